"""The paged KV cache and the attention over it (gwa_kv_append, gwa_kv_read,
gwa_rope_table, gwa_sdpa_paged) against plain CPU implementations.

Append: codes, scales, biases and rotated queries bit for bit (the definition
decides them in fp32), nothing else of the cache touched.

Attention tolerance, against fp64 on the same cache.  With P = max |v| over
the visible values of a head: the weights times the value scales are rounded
to fp16 (relative 2^-12 each, and the centred code carries at most the group's
range, <= 2 P), the biases enter in fp32, and the output is rounded to bf16
(2^-9 of itself).  Scores carry the fp32 rounding of sums of 64 products:
below 2^-16 absolute at |score| <= 32, i.e. 2^-16 relative in each weight.
Together below 2^-9 |out| + (2^-11 + 2^-14) P; the tests allow 2^-8 |out| +
2^-10 P.
"""
import numpy as np
import pytest
import torch

import group_wise_affine_gb300 as gwa
from helpers import bf16_to_f64, dev_bf16, host_u16
from oracle import serving

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    gwa.build()
    gwa.load()
    assert torch.cuda.is_available()


def rand_bf16(rng, *shape, scale=1.0):
    return serving.bf16_round((rng.standard_normal(shape) * scale).astype(np.float32))


def i32(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()


class Case:
    """A batch over a cache filled with random keys and values."""

    def __init__(self, seed, lens, Hq=8, Hkv=2, D=128, bits=4, page=16,
                 spread=1.0, vscale=1.0, spare=2):
        rng = self.rng = np.random.default_rng(seed)
        self.ql = np.array([a for a, _ in lens])
        self.kl = np.array([b for _, b in lens])
        self.Hq, self.Hkv, self.D, self.bits, self.page = Hq, Hkv, D, bits, page
        need = -(-self.kl // page)
        P = int(need.sum()) + spare
        width = max(1, int(need.max()))
        order = rng.permutation(P)
        self.table = np.full((len(lens), width), -7, dtype=np.int32)  # never read past the end
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = order[at:at + n]
            at += n
        self.q_start = np.concatenate([[0], np.cumsum(self.ql)])
        self.T = int(self.q_start[-1])
        ch = np.exp(spread * rng.standard_normal(D)) if spread != 1.0 else np.ones(D)
        kbits = serving.bf16_round((rng.standard_normal((P, Hkv, page, D)) * ch).astype(np.float32))
        vbits = rand_bf16(rng, P, Hkv, page, D, scale=vscale)
        kc, self.kp = serving.quantize(kbits, bits)
        vc, self.vp = serving.quantize(vbits, bits)
        self.kq, self.vq = serving.pack(kc, bits), serving.pack(vc, bits)

    def device(self):
        self.cache = gwa.KVCache(
            torch.from_numpy(self.kq.view(np.int32)).cuda(), dev_bf16(self.kp),
            torch.from_numpy(self.vq.view(np.int32)).cuda(), dev_bf16(self.vp),
            bits=self.bits)
        self.batch = gwa.KVBatch(i32(self.q_start), i32(self.kl), i32(self.table), self.T,
                                 int(self.ql.max()), int(self.kl.max()))
        return self

    def sequence(self, b):
        """fp64 keys and values of a sequence."""
        n = int(self.kl[b])
        t = np.arange(n)
        pg, sl = self.table[b, t // self.page], t % self.page
        return (serving.values(self.kq[pg, :, sl], self.kp[pg, :, sl], self.bits),
                serving.values(self.vq[pg, :, sl], self.vp[pg, :, sl], self.bits))


def check_attention(c, causal=True, qscale=0.7, scale=None, strided=False, tight=2.0 ** -10):
    q = rand_bf16(c.rng, c.T, c.Hq, c.D, scale=qscale)
    scale = 1.0 / np.sqrt(c.D) if scale is None else scale
    c.device()
    qd = dev_bf16(q)
    if strided:
        wide = torch.full((c.T, c.Hq + 3, c.D), float("nan"), dtype=torch.bfloat16, device="cuda")
        wide[:, 1:1 + c.Hq] = qd
        qd = wide[:, 1:1 + c.Hq]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = bf16_to_f64(gwa.sdpa_paged(qd, c.cache, c.batch, scale=scale, causal=causal,
                                     status=status))
    assert int(status) == 0
    kv = [c.sequence(b) for b in range(len(c.kl))]
    want = serving.attention(serving.bf16_value(q).astype(np.float64), [k for k, _ in kv],
                             [v for _, v in kv], c.q_start, c.kl, scale, causal)
    peak = max([np.abs(v).max() for _, v in kv if v.size] + [1e-30])
    bar = 2.0 ** -8 * np.abs(want) + tight * peak
    worst = np.max(np.abs(got - want) / bar)
    assert np.isfinite(got).all() and worst <= 1, worst
    return got


# ------------------------------------------------------------------ attention
@pytest.mark.parametrize("kv", [1, 2, 15, 16, 17, 31, 33, 127, 128, 129, 1000, 4097])
def test_one_token_lengths(kv):
    check_attention(Case(kv, [(1, kv)], Hq=10, Hkv=2))


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("rep,q", [(1, 1), (5, 1), (8, 1), (5, 3), (4, 8), (3, 1), (7, 5)])
def test_widths_heads_and_rows(bits, D, rep, q):
    check_attention(Case(D + bits + rep, [(q, 300), (max(1, q - 1), 70)], Hq=2 * rep, Hkv=2,
                         D=D, bits=bits, page=32))


@pytest.mark.parametrize("page", [16, 64, 256, 4096])
def test_page_sizes(page):
    check_attention(Case(page, [(1, 500), (2, 17), (1, 256)], page=page))


def test_ragged_batch_with_empty_sequences():
    rng = np.random.default_rng(0)
    lens = [(int(rng.integers(0, 3)), int(n)) for n in rng.integers(3, 700, 70)]
    lens[3], lens[11], lens[40] = (0, 0), (0, 50), (2, 2)
    check_attention(Case(5, lens, Hq=4, Hkv=1))


@pytest.mark.parametrize("q", [9, 33, 130, 300])
@pytest.mark.parametrize("causal", [True, False])
def test_prompts(q, causal):
    check_attention(Case(q, [(q, q), (q // 2, q + 61)], Hq=4, Hkv=2), causal=causal)


@pytest.mark.parametrize("D,bits,rep", [(64, 4, 8), (256, 4, 3), (256, 8, 1), (128, 8, 5), (64, 8, 2)])
def test_prompts_of_every_format(D, bits, rep):
    check_attention(Case(D + rep, [(150, 290), (1, 40), (37, 37)], Hq=2 * rep, Hkv=2, D=D,
                         bits=bits, page=32))


@pytest.mark.parametrize("q", [2, 40, 200])
def test_rows_that_see_nothing_are_zero(q):
    # more new tokens than the cache is long: the first rows see no key
    c = Case(1, [(q, q - 1), (q, q)], Hq=4, Hkv=2)
    got = check_attention(c)
    assert (got[0] == 0).all()
    # no keys at all
    c = Case(2, [(q, 0), (1, 40)], Hq=4, Hkv=2)
    got = check_attention(c)
    assert (got[:q] == 0).all()


@pytest.mark.parametrize("q", [1, 90])
def test_masked_places_may_hold_anything(q):
    # what lies past a sequence's end in its last page: NaN, infinities
    c = Case(3, [(q, q + 7), (q, q + 4)], Hq=4, Hkv=2, page=128)
    ref = check_attention(c)
    for b in range(2):
        pg = c.table[b, int(c.kl[b]) // 128] if int(c.kl[b]) % 128 else None
        assert pg is not None
        for a in (c.kp, c.vp):
            a[pg, :, int(c.kl[b]) % 128:] = np.array([0x7fc0, 0x7f80], dtype=np.uint16)
        c.kq[pg, :, int(c.kl[b]) % 128:] = 0xffffffff
        c.vq[pg, :, int(c.kl[b]) % 128:] = 0xffffffff
    c.rng = np.random.default_rng(3)
    c2 = Case(3, [(q, q + 7), (q, q + 4)], Hq=4, Hkv=2, page=128)
    c.rng = c2.rng
    got = check_attention(c)
    assert np.array_equal(got, ref)


@pytest.mark.parametrize("q,kv", [(3, 20), (70, 90)])
def test_a_later_key_that_is_not_finite_stays_with_its_readers(q, kv):
    # a token's own key and value are NaN: rows before it do not see it
    c = Case(4, [(q, kv)], Hq=4, Hkv=2, page=32)
    ref = check_attention(c)
    last = kv - 1
    pg, sl = c.table[0, last // 32], last % 32
    for bad in (0x7fc0, 0x7f80):
        d = Case(4, [(q, kv)], Hq=4, Hkv=2, page=32)
        d.kp[pg, :, sl] = bad
        d.vp[pg, :, sl] = bad
        qb = rand_bf16(d.rng, d.T, d.Hq, d.D, scale=0.7)
        d.device()
        got = bf16_to_f64(gwa.sdpa_paged(dev_bf16(qb), d.cache, d.batch))
        assert np.array_equal(got[:-1], ref[:-1])
        if bad == 0x7fc0:
            assert np.isnan(got[-1]).all()


@pytest.mark.parametrize("q", [1, 80])
@pytest.mark.parametrize("vscale", [1e-30, 1e-6, 1e4, 1e30])
def test_value_range(q, vscale):
    check_attention(Case(6, [(q, 400)], Hq=4, Hkv=2, vscale=vscale))


@pytest.mark.parametrize("q", [1, 80])
def test_key_and_query_range(q):
    # keys and queries far from 1 whose scores are ordinary
    for kscale in (1e-20, 1e20):
        c = Case(7, [(q, 300)], Hq=4, Hkv=2)
        f = serving.bf16_value(c.kp) * np.float32(kscale)
        c.kp = serving.bf16_round(f)
        check_attention(c, qscale=0.7 / kscale)


@pytest.mark.parametrize("q", [1, 80])
def test_value_scales_that_grow_and_shrink_along_the_cache(q):
    c = Case(8, [(q, 1500)], Hq=4, Hkv=2, page=16)
    t = np.arange(c.kl[0])
    f = serving.bf16_value(c.vp)
    for i in range(0, len(t), 16):
        f[c.table[0, i // 16]] *= np.float32(2.0 ** ((i // 16) % 13 - 6))
    c.vp = serving.bf16_round(f)
    check_attention(c)


@pytest.mark.parametrize("q", [1, 80])
def test_sharp_scores_and_outlier_channels(q):
    check_attention(Case(9, [(q, 700)], Hq=4, Hkv=2, spread=1.5), qscale=2.0)


@pytest.mark.parametrize("scale", [0.0, -0.1])
def test_unusual_scales(scale):
    check_attention(Case(10, [(2, 200), (40, 60)], Hq=4, Hkv=2), scale=scale)


def test_strided_queries_and_more_heads_than_a_row_block():
    check_attention(Case(11, [(1, 333), (2, 90)], Hq=40, Hkv=1), strided=True)
    check_attention(Case(12, [(60, 100)], Hq=6, Hkv=3), strided=True)


def test_a_long_cache_is_the_average_of_its_halves():
    # equal keys make every weight equal: the output is the mean value, a
    # small number among large ones.  The weights' fp16 roundings are
    # independent, 2^-12 of peak / sqrt(n) together, and an fp32 sum of n/16
    # products with one sign loses at most n/16 2^-24 of itself: 2^-14 peak
    # holds both
    c = Case(13, [(1, 20000)], Hq=4, Hkv=1, D=64, page=64)
    c.kp[:] = serving.bf16_round(np.array([0.1, 0.2], np.float32))
    c.kq[:] = 0x55555555
    check_attention(c, tight=2.0 ** -14)


def test_results_do_not_depend_on_the_bounds_or_the_workspace_contents():
    c = Case(14, [(1, 900), (3, 40)], Hq=8, Hkv=2).device()
    q = dev_bf16(rand_bf16(c.rng, c.T, c.Hq, c.D))
    a = gwa.sdpa_paged(q, c.cache, c.batch)
    loose = gwa.KVBatch(i32(c.q_start), i32(c.kl), i32(c.table), c.T, int(c.ql.max()), 900)
    ws = gwa.make_sdpa_paged_workspace(c.cache, loose, 8)
    ws.fill_(255)
    b = gwa.sdpa_paged(q, c.cache, loose, workspace=ws)
    assert torch.equal(a, b)
    assert torch.equal(a, gwa.sdpa_paged(q, c.cache, c.batch, workspace=ws))


def test_rows_of_no_sequence_are_not_written():
    c = Case(15, [(1, 50), (2, 30)], Hq=4, Hkv=2).device()
    q = dev_bf16(rand_bf16(c.rng, c.T + 2, c.Hq, c.D))
    batch = gwa.KVBatch(i32(c.q_start), i32(c.kl), i32(c.table), c.T + 2, 2, 50)
    out = torch.full((c.T + 2, 4, c.D), 7.0, dtype=torch.bfloat16, device="cuda")
    gwa.sdpa_paged(q, c.cache, batch, out=out)
    assert (out[c.T:] == 7).all()
    want = gwa.sdpa_paged(q[:c.T].contiguous(), c.cache, c.batch)
    assert torch.equal(out[:c.T], want)


def test_bad_pages_raise_the_status():
    for q in (1, 64):
        c = Case(16, [(q, 100), (q, 90)], Hq=4, Hkv=2).device()
        for bad in (-1, 1 << 20):
            t = c.table.copy()
            t[1, 1] = bad
            batch = gwa.KVBatch(i32(c.q_start), i32(c.kl), i32(t), c.T, q, 100)
            x = dev_bf16(rand_bf16(c.rng, c.T, c.Hq, c.D))
            status = torch.zeros(1, dtype=torch.int32, device="cuda")
            got = gwa.sdpa_paged(x, c.cache, batch, status=status)
            assert int(status) == 1
            good = gwa.sdpa_paged(x, c.cache, c.batch)
            assert torch.equal(got[:q], good[:q])


@pytest.mark.parametrize("D,rep,causal", [(64, 2, True), (128, 8, True), (256, 4, False)])
def test_many_short_prompts(D, rep, causal):
    # hundreds of blocks of a tile or two, cut anywhere: lengths from none to
    # several tiles, some with more new tokens than keys
    rng = np.random.default_rng(D)
    lens = [(int(q), int(kv)) for q, kv in zip(rng.integers(0, 90, 60), rng.integers(0, 300, 60))]
    lens += [(70, 0), (1, 1), (64, 64), (33, 129), (200, 128)]
    check_attention(Case(D + 1, lens, Hq=4 * rep, Hkv=4, D=D), causal=causal)


@pytest.mark.parametrize("bits", [4, 8])
def test_many_sequences_in_long_runs(bits):
    # enough work for runs of many steps a CTA, over segments from one step to
    # dozens and sequences without keys
    rng = np.random.default_rng(bits)
    kv = np.concatenate([rng.integers(0, 6000, 40), rng.integers(0, 200, 40), [0, 1, 127, 128, 129]])
    check_attention(Case(bits + 40, [(1, int(n)) for n in kv], Hq=8, Hkv=8, D=64, bits=bits))


def test_scores_that_grow_along_the_keys():
    # the running maximum moves in nearly every step, in either half of it
    # (scores reach a few dozen, so a key's 2^-12 counts for more: twice the bar)
    for q in (1, 48):
        c = Case(50 + q, [(q, 400)], Hq=4, Hkv=2, D=128, bits=8)
        pg, sl = c.table[0, np.arange(400) // c.page], np.arange(400) % c.page
        grow = serving.bf16_value(c.kp[pg, :, sl]) * np.linspace(0.1, 12, 400)[:, None, None, None]
        c.kp[pg, :, sl] = serving.bf16_round(grow.astype(np.float32))
        check_attention(c, qscale=1.0, tight=2.0 ** -9)


def test_another_stream():
    c = Case(17, [(1, 3000)] * 4, Hq=8, Hkv=2).device()
    q = dev_bf16(rand_bf16(c.rng, c.T, c.Hq, c.D))
    want = gwa.sdpa_paged(q, c.cache, c.batch)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    outs = [gwa.sdpa_paged(q, c.cache, c.batch, stream=s) for _ in range(8)]
    s.synchronize()
    for o in outs:
        assert torch.equal(o, want)


def test_in_a_graph():
    c = Case(18, [(1, 700), (1, 90)], Hq=8, Hkv=2).device()
    q = dev_bf16(rand_bf16(c.rng, c.T, c.Hq, c.D))
    ws = gwa.make_sdpa_paged_workspace(c.cache, c.batch, 8)
    out = torch.empty_like(q)
    gwa.sdpa_paged(q, c.cache, c.batch, out=out, workspace=ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        gwa.sdpa_paged(q, c.cache, c.batch, out=out, workspace=ws)
    # lengths are read on the device: the same graph serves a shorter cache
    c.batch.kv_len.copy_(i32([500, 80]))
    g.replay()
    torch.cuda.synchronize()
    again = gwa.sdpa_paged(q, c.cache, c.batch)
    assert torch.equal(out, again)


# ------------------------------------------------------------------ append
def run_append(seed, lens, Hq=4, Hkv=2, D=128, bits=4, page=16, rot=128, strided=False,
               spread=1.0):
    c = Case(seed, lens, Hq, Hkv, D, bits, page).device()
    kq0, vq0 = c.cache.kq.clone(), c.cache.vq.clone()
    rng = c.rng
    x = serving.bf16_round((rng.standard_normal((c.T, Hq + 2 * Hkv, D)) *
                            np.exp(spread * rng.standard_normal((c.T, Hq + 2 * Hkv, 1)))
                            ).astype(np.float32))
    q, k, v = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
    xd = dev_bf16(x)
    qd, kd, vd = xd[:, :Hq], xd[:, Hq:Hq + Hkv], xd[:, Hq + Hkv:]
    if not strided:
        qd, kd, vd = qd.contiguous(), kd.contiguous(), vd.contiguous()
    n = int(max(1, c.kl.max()))
    table = serving.rope_table(n, rot, 1e4) if rot else np.zeros((n, 0, 2), np.float32)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    qo = gwa.kv_append(kd, vd, c.cache, c.batch, q=qd if Hq else None,
                       rope=torch.from_numpy(table).cuda() if rot else None, status=status)
    assert int(status) == 0
    seq, pos = serving.positions(c.q_start, c.kl, c.T)
    if Hq:
        assert np.array_equal(host_u16(qo), serving.rotate(q, table, pos))
    kr = serving.rotate(k, table, pos)
    live = np.nonzero(pos >= 0)[0]
    pg, sl = c.table[seq[live], pos[live] // page], pos[live] % page
    for name, src in (("k", kr), ("v", v)):
        codes, par = serving.quantize(src[live], bits)
        want_q = getattr(c, name + "q").copy()
        want_p = getattr(c, name + "p").copy()
        want_q[pg, :, sl] = serving.pack(codes, bits)
        want_p[pg, :, sl] = par
        got_q = getattr(c.cache, name + "q").cpu().numpy().view(np.uint32)
        assert np.array_equal(got_q, want_q)                  # nothing else moved
        assert np.array_equal(host_u16(getattr(c.cache, name + "p")), want_p)
        setattr(c, name + "q", want_q)
        setattr(c, name + "p", want_p)
    k2, v2 = gwa.kv_read(c.cache, c.batch, status=status)
    assert int(status) == 0
    for got, name in ((k2, "k"), (v2, "v")):
        want = np.zeros((c.T, Hkv, D), np.float32)
        want[live] = serving.values(getattr(c, name + "q")[pg, :, sl],
                                    getattr(c, name + "p")[pg, :, sl], bits).astype(np.float32)
        assert np.array_equal(host_u16(got), serving.bf16_round(want))
    return c


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("D,rot", [(64, 64), (64, 16), (128, 128), (128, 32), (128, 0),
                                   (256, 256), (256, 64), (256, 48)])
def test_append_formats(bits, D, rot):
    run_append(D + rot + bits, [(1, 40), (3, 3), (17, 50)], D=D, bits=bits, rot=rot)


@pytest.mark.parametrize("Hq,Hkv", [(40, 8), (0, 1), (0, 3), (1, 1), (7, 7)])
@pytest.mark.parametrize("strided", [True, False])
def test_append_heads_and_strides(Hq, Hkv, strided):
    run_append(Hq, [(2, 9), (1, 17)], Hq=Hq, Hkv=Hkv, strided=strided)


def test_append_ragged_batch():
    rng = np.random.default_rng(1)
    lens = [(int(a), int(a + b)) for a, b in zip(rng.integers(0, 40, 75), rng.integers(0, 90, 75))]
    run_append(2, lens, page=32)


def test_append_many_tokens():
    run_append(3, [(2500, 2500), (700, 1000)], Hq=6, Hkv=2, page=64, strided=True)


def test_append_before_the_start_has_no_place():
    # more new tokens than the length: the first have no position
    run_append(4, [(5, 3), (2, 0)])


def test_append_constant_and_wide_ranged_rows():
    run_append(5, [(64, 64)], spread=6.0)
    c = Case(6, [(1, 1)], Hq=1, Hkv=1).device()
    z = torch.zeros((1, 1, 128), dtype=torch.bfloat16, device="cuda")
    for fill in (0.0, -0.0, 3.5):
        z.fill_(fill)
        gwa.kv_append(z, z, c.cache, c.batch)
        k, v = gwa.kv_read(c.cache, c.batch)
        assert (k == fill).all() and (v == fill).all()


def test_append_status_and_skips():
    c = Case(7, [(2, 40), (1, 20)], Hq=2, Hkv=2).device()
    x = dev_bf16(rand_bf16(c.rng, 3, 2, 128))
    before = c.cache.kq.clone()
    t = c.table.copy()
    t[1, 1] = 1 << 20
    batch = gwa.KVBatch(i32(c.q_start), i32(c.kl), i32(t), 3, 2, 40)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    gwa.kv_append(x, x, c.cache, batch, status=status)
    assert int(status) == 1
    moved = (c.cache.kq != before).nonzero()[:, 0].unique()
    assert moved.numel() == 1                       # the first sequence's page alone
    status.zero_()
    k, _ = gwa.kv_read(c.cache, batch, status=status)
    assert int(status) == 1 and (k[2] == 0).all() and (k[0] != 0).any()
    status.zero_()
    table = gwa.rope_table(39, 128, 1e4)            # the second new token is at 39
    before = c.cache.kq.clone()
    gwa.kv_append(x, x, c.cache, c.batch, rope=table, status=status)
    assert int(status) == 2


def test_append_in_place_queries():
    c = Case(8, [(3, 30)], Hq=4, Hkv=2).device()
    x = rand_bf16(c.rng, 3, 4, 128)
    kv = dev_bf16(rand_bf16(c.rng, 3, 2, 128))
    table = gwa.rope_table(64, 128, 1e4)
    a = dev_bf16(x)
    want = gwa.kv_append(kv, kv, c.cache, c.batch, q=a, rope=table).clone()
    gwa.kv_append(kv, kv, c.cache, c.batch, q=a, rope=table, q_out=a)
    assert torch.equal(a, want)


def test_rope_table_matches_fp64_angles():
    n, rot, base = 70000, 64, 1e6
    got = gwa.rope_table(n, rot, base).cpu().numpy().astype(np.float64)
    a = np.arange(n)[:, None] * base ** (-np.arange(0, rot, 2) / rot)
    # the angle is accurate to ~1e-11 at 7e4; fp32 sine and cosine to 2^-23
    assert np.abs(got - np.stack([np.cos(a), np.sin(a)], -1)).max() < 4e-7


def test_append_then_attend_matches_plain_attention():
    # the whole way once: rotate and quantize a prompt, then attend over it
    c = Case(20, [(50, 50), (1, 61)], Hq=4, Hkv=2).device()
    rng = np.random.default_rng(21)
    x = rand_bf16(rng, c.T, 8, c.D)
    xd = dev_bf16(x)
    table = gwa.rope_table(64, c.D, 1e4)
    q = gwa.kv_append(xd[:, 4:6], xd[:, 6:8], c.cache, c.batch, q=xd[:, :4], rope=table)
    out = bf16_to_f64(gwa.sdpa_paged(q, c.cache, c.batch))
    full = gwa.KVBatch(i32([0, 50, 111]), i32(c.kl), i32(c.table), 111, 61, 61)
    k, v = (bf16_to_f64(t) for t in gwa.kv_read(c.cache, full))
    want = serving.attention(bf16_to_f64(q), [k[:50], k[50:]], [v[:50], v[50:]], c.q_start,
                             c.kl, 1 / np.sqrt(c.D), True)
    # keys and values read back are rounded to bf16 once more (2^-9): a key's
    # rounding moves a score of |q||k|/sqrt(D) ~ 4 by below 2^-7
    assert np.abs(out - want).max() < 2.0 ** -5


# ------------------------------------------------------------------ refusals
def test_refusals():
    c = Case(30, [(1, 20)], Hq=4, Hkv=2).device()
    q = dev_bf16(rand_bf16(c.rng, 1, 4, 128))
    kv = dev_bf16(rand_bf16(c.rng, 1, 2, 128))
    with pytest.raises(ValueError):
        gwa.sdpa_paged(q[..., :64], c.cache, c.batch)
    with pytest.raises(ValueError):
        gwa.sdpa_paged(q.float(), c.cache, c.batch)
    with pytest.raises(ValueError):
        gwa.sdpa_paged(q.cpu(), c.cache, c.batch)
    with pytest.raises(gwa.GwaError):
        gwa.sdpa_paged(q[:, :3].contiguous(), c.cache, c.batch)      # 3 heads over 2
    with pytest.raises(gwa.GwaError) as e:
        gwa.sdpa_paged(q, c.cache, c.batch, workspace=torch.empty(16, dtype=torch.uint8,
                                                                  device="cuda"))
    assert e.value.code == gwa.GWA_ERR_WORKSPACE
    with pytest.raises(gwa.GwaError):
        gwa.sdpa_paged(q, c.cache, c.batch, scale=float("nan"))
    with pytest.raises(ValueError):
        gwa.kv_append(kv[:, :1], kv, c.cache, c.batch)
    with pytest.raises(gwa.GwaError):
        gwa.kv_append(kv, kv, c.cache, c.batch, rope=gwa.rope_table(64, 24, 1e4))
    with pytest.raises(TypeError):
        gwa.KVBatch(i32([0, 1]).long(), i32([1]), i32([[0]]), 1, 1, 1)
    with pytest.raises(ValueError):
        gwa.KVCache(c.cache.kq, c.cache.kp[:1], c.cache.vq, c.cache.vp)
    bad = torch.empty((2, 2, 24, 16), dtype=torch.int32, device="cuda")
    par = torch.empty((2, 2, 24, 2, 2), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(gwa.GwaError):                                # page of 24
        gwa.kv_append(kv, kv, gwa.KVCache(bad, par, bad, par), c.batch)
