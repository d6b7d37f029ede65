"""Edges of the paged cache and the attention over it: values far apart in
size, lengths past the page table, rows without a place, loose bounds.

Attention tolerances are those of ``test_gpu_paged`` (2^-8 of the output and
2^-10 of the largest value that the row can see).
"""
import numpy as np
import pytest
import torch

import group_wise_affine_gb300 as gwa
from helpers import bf16_to_f64, dev_bf16
from oracle import serving
from test_gpu_paged import Case, check_attention, i32, rand_bf16

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    gwa.build()
    gwa.load()
    assert torch.cuda.is_available()


def scale_values(c, b, first, last, factor):
    """Multiplies the values of keys [first, last) of sequence b."""
    t = np.arange(first, last)
    pg, sl = c.table[b, t // c.page], t % c.page
    c.vp[pg, :, sl] = serving.bf16_round(serving.bf16_value(c.vp[pg, :, sl]) * np.float32(factor))


def attend(c, q, **kw):
    """Output and fp64 reference of one call over the case's cache."""
    c.device()
    got = bf16_to_f64(gwa.sdpa_paged(dev_bf16(q), c.cache, c.batch, **kw))
    kv = [c.sequence(b) for b in range(len(c.kl))]
    want = serving.attention(serving.bf16_value(q).astype(np.float64), [k for k, _ in kv],
                             [v for _, v in kv], c.q_start, c.kl, 1 / np.sqrt(c.D), True)
    return got, want, kv


def within(got, want, peak):
    return np.isfinite(got).all() and (
        np.abs(got - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -10 * peak).all()


@pytest.mark.parametrize("ratio", [2.0 ** 10, 2.0 ** 16, 2.0 ** 24])
@pytest.mark.parametrize("D,bits", [(64, 4), (128, 4), (256, 4), (64, 8), (128, 8), (256, 8)])
def test_a_later_value_that_is_large_stays_with_its_readers_prompts(D, bits, ratio):
    # the last token's value is finite and much larger than all others: the
    # rows before it do not see it, and their values keep their precision
    c = Case(D + bits, [(70, 100)], Hq=4, Hkv=2, D=D, bits=bits)
    scale_values(c, 0, 99, 100, ratio)
    got, want, kv = attend(c, rand_bf16(c.rng, c.T, c.Hq, c.D, scale=0.7))
    v = np.abs(kv[0][1])
    assert within(got[:-1], want[:-1], v[:-1].max())
    assert within(got[-1:], want[-1:], v.max())


@pytest.mark.parametrize("D,bits", [(128, 4), (256, 8)])
def test_a_large_value_of_no_weight_leaves_the_others_prompts(D, bits):
    # the first key's score is hundreds below the others'
    c = Case(D, [(70, 400)], Hq=4, Hkv=2, D=D, bits=bits)
    scale_values(c, 0, 0, 1, 2.0 ** 24)
    pg = c.table[0, 0]
    c.kp[pg, :, 0] = serving.bf16_round(np.array([0.0, -100.0], np.float32))
    q = serving.bf16_round(np.abs(serving.bf16_value(rand_bf16(c.rng, c.T, c.Hq, c.D, scale=0.7))))
    got, want, kv = attend(c, q)
    assert within(got, want, np.abs(kv[0][1])[1:].max())


@pytest.mark.parametrize("D", [128, 256])
@pytest.mark.parametrize("first,then", [(1e30, 1e-10), (1e-10, 1e30), (1e-30, 1e30)])
def test_values_that_fall_and_rise_by_many_powers_prompts(D, first, then):
    c = Case(31, [(80, 700)], Hq=4, Hkv=2, D=D)
    scale_values(c, 0, 0, 256, first)
    scale_values(c, 0, 256, 700, then)
    check_attention(c)


@pytest.mark.parametrize("vscale", [1e-36, 1e34, 3e37])
@pytest.mark.parametrize("D,bits", [(128, 4), (256, 8)])
def test_values_near_the_ends_of_the_range_prompts(D, bits, vscale):
    # (blocks of one CTA, and blocks cut over many)
    check_attention(Case(32, [(80, 1500)], Hq=4, Hkv=2, D=D, bits=bits, vscale=vscale))
    check_attention(Case(33, [(80, 90)] * 2, Hq=4, Hkv=2, D=D, bits=bits, vscale=vscale))


@pytest.mark.parametrize("q", [1, 80])
def test_many_small_weights_beside_one_that_takes_all(q):
    # one key takes the weight and has a value of zero, 131071 others take
    # 2^-25.2 each of it: the output is a few thousandths of their values.  152
    # sequences over the same pages, so that a block's keys are not cut
    n, B = 131072, 152
    c = Case(35, [(q, n + q)], Hq=2, Hkv=1, D=64, page=4096)
    c.kq[:] = 0
    c.kp[:] = 0
    c.vp[:] = serving.bf16_round(np.array([2.0 ** -6, 1.0], np.float32))
    pg = c.table[0, 0]
    c.kp[pg, :, 0] = serving.bf16_round(np.array([0.0, 4.375], np.float32))
    c.vp[pg, :, 0] = 0
    qb = serving.bf16_round(np.full((c.T, 2, 64), 0.5, np.float32))
    _, want, kv = attend(c, qb)     # scores 4.375 * 32 / 8 = 17.5 and 0
    assert 0.003 < want.min() and want.max() < 0.005
    batch = gwa.KVBatch(i32(np.arange(B + 1) * q), i32([n + q] * B), i32(np.repeat(c.table, B, 0)),
                        B * q, q, n + q)
    got = bf16_to_f64(gwa.sdpa_paged(dev_bf16(np.tile(qb, (B, 1, 1))), c.cache, batch))
    for b in range(B):
        assert within(got[b * q:(b + 1) * q], want, np.abs(kv[0][1]).max())


@pytest.mark.parametrize("ratio", [2.0 ** 10, 2.0 ** 16, 2.0 ** 24])
@pytest.mark.parametrize("D,bits", [(64, 4), (128, 4), (256, 4), (64, 8), (128, 8), (256, 8)])
def test_a_later_value_that_is_large_stays_with_its_readers_few_rows(D, bits, ratio):
    for kv_len in (20, 300):
        c = Case(D + bits, [(3, kv_len)], Hq=4, Hkv=2, D=D, bits=bits)
        scale_values(c, 0, kv_len - 1, kv_len, ratio)
        got, want, kv = attend(c, rand_bf16(c.rng, c.T, c.Hq, c.D, scale=0.7))
        v = np.abs(kv[0][1])
        assert within(got[:-1], want[:-1], v[:-1].max())
        assert within(got[-1:], want[-1:], v.max())


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("q,kv", [(3, 129), (3, 385), (3, 1537), (80, 385), (80, 2049)])
def test_scores_far_below_zero_in_cut_segments(D, q, kv):
    # every score lies hundreds below zero, and the last piece of a cut
    # segment holds keys that the earlier rows do not see
    c = Case(D + kv, [(q, kv)], Hq=4, Hkv=2, D=D)
    f = serving.bf16_value(c.kp).copy()
    f[..., 1] -= np.float32(3000.0 / D)
    c.kp = serving.bf16_round(f)
    x = np.abs(serving.bf16_value(rand_bf16(c.rng, c.T, c.Hq, c.D, scale=0.7)))
    got, want, cache = attend(c, serving.bf16_round(x))
    assert within(got, want, np.abs(cache[0][1]).max())


@pytest.mark.parametrize("q,kv", [(3, 3000), (80, 3000)])
def test_a_query_that_is_not_a_number_leaves_the_others(q, kv):
    c = Case(41, [(q, kv)], Hq=4, Hkv=2)
    x = rand_bf16(c.rng, c.T, c.Hq, c.D, scale=0.7)
    c.device()
    good = gwa.sdpa_paged(dev_bf16(x), c.cache, c.batch)
    x[1, 2, 5] = 0x7fc0
    got = gwa.sdpa_paged(dev_bf16(x), c.cache, c.batch)
    assert torch.isnan(got[1, 2]).all()
    got[1, 2], good[1, 2] = 0, 0
    assert torch.equal(got, good)


@pytest.mark.parametrize("first,then", [(1e30, 1e-10), (1e-10, 1e30), (1e-30, 1e30)])
@pytest.mark.parametrize("D", [128, 256])
def test_values_that_fall_and_rise_by_many_powers_few_rows(D, first, then):
    c = Case(31, [(1, 700)], Hq=4, Hkv=2, D=D)
    scale_values(c, 0, 0, 256, first)
    scale_values(c, 0, 256, 700, then)
    check_attention(c)


@pytest.mark.parametrize("vscale", [1e-36, 1e34, 3e37])
@pytest.mark.parametrize("D,bits", [(64, 8), (128, 4), (256, 8)])
def test_values_near_the_ends_of_the_range_few_rows(D, bits, vscale):
    check_attention(Case(32, [(1, 30000)], Hq=4, Hkv=1, D=D, bits=bits, vscale=vscale))
    check_attention(Case(33, [(5, 90)] * 2, Hq=4, Hkv=2, D=D, bits=bits, vscale=vscale))


@pytest.mark.parametrize("bits", [4, 8])
def test_biases_far_above_their_scales_few_rows(bits):
    # constant groups: a scale of zero and a large bias; their neighbours' 1e6
    # times smaller
    c = Case(34, [(2, 500)], Hq=4, Hkv=2, bits=bits)
    f = serving.bf16_value(c.vp).copy()
    f[::2, ..., 0] = 0.0
    f[::2, ..., 1] = 3e38
    f[1::2] *= np.float32(1e32)
    c.vp = serving.bf16_round(f)
    check_attention(c)


@pytest.mark.parametrize("q", [3, 80])
@pytest.mark.parametrize("causal", [True, False])
def test_lengths_past_the_page_table(q, causal):
    # tokens past the table have no place; the others keep their own
    page, width = 16, 8
    cap = page * width
    c = Case(36, [(q, cap), (q, 40 + q)], Hq=4, Hkv=2, page=page).device()
    table = np.full((2, width), -7, dtype=np.int32)
    table[:, :c.table.shape[1]] = c.table
    kl = np.array([cap + 2, 40 + q])     # the first sequence's last two are past it
    batch = gwa.KVBatch(i32(c.q_start), i32(kl), i32(table), c.T, q, int(kl.max()))
    x = rand_bf16(c.rng, c.T, 8, c.D)
    xd = dev_bf16(x)
    kq0 = c.cache.kq.clone()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    gwa.kv_append(xd[:, 4:6], xd[:, 6:8], c.cache, batch, status=status)
    assert int(status) == 1
    pos = cap + 2 - q + np.arange(q)
    live = pos < cap
    codes, _ = serving.quantize(x[:q][live][:, 4:6], 4)
    want_q = kq0.cpu().numpy().view(np.uint32).copy()
    want_q[table[0, pos[live] // page], :, pos[live] % page] = serving.pack(codes, 4)
    p2 = 40 + np.arange(q)
    codes, _ = serving.quantize(x[q:, 4:6], 4)
    want_q[table[1, p2 // page], :, p2 % page] = serving.pack(codes, 4)
    assert np.array_equal(c.cache.kq.cpu().numpy().view(np.uint32), want_q)
    status.zero_()
    k, v = gwa.kv_read(c.cache, batch, status=status)
    assert int(status) == 1
    assert (k[q - 2:q] == 0).all() and (v[q - 2:q] == 0).all() and (k[:q - 2] != 0).any()
    # attention: rows see the keys that are there, up to their own position
    for name in ("kq", "kp", "vq", "vp"):
        t = getattr(c.cache, name)
        setattr(c, name, t.cpu().view(torch.int16).numpy().view(np.uint16).reshape(t.shape)
                if t.dtype == torch.bfloat16 else t.cpu().numpy().view(np.uint32))
    status.zero_()
    got = bf16_to_f64(gwa.sdpa_paged(xd[:, :4], c.cache, batch, causal=causal, status=status))
    assert int(status) == 1
    kv = [c.sequence(b) for b in range(2)]
    qf = serving.bf16_value(x[:, :4]).astype(np.float64)
    for i in range(2 * q):
        b, j = divmod(i, q)
        seen = min(int(c.kl[b]), int(kl[b]) - q + j + 1) if causal else int(c.kl[b])
        for h in range(4):
            s = kv[b][0][:seen, h // 2] @ qf[i, h] / np.sqrt(c.D)
            p = np.exp(s - s.max())
            want = (p / p.sum()) @ kv[b][1][:seen, h // 2]
            assert within(got[i, h], want, np.abs(kv[b][1]).max())


def test_rotated_queries_of_tokens_without_a_place():
    # seven tokens: two of the first sequence (its page is bad), two of the
    # second, of which the last is past the rotary table, three of none
    c = Case(37, [(2, 40), (2, 21)], Hq=4, Hkv=2).device()
    t = c.table.copy()
    t[0, 2] = 1 << 20
    batch = gwa.KVBatch(i32(c.q_start), i32(c.kl), i32(t), 7, 2, 40)
    x = rand_bf16(c.rng, 7, 8, c.D)
    xd = dev_bf16(x)
    table = gwa.rope_table(40, c.D, 1e4)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = torch.full((7, 4, c.D), float("nan"), dtype=torch.bfloat16, device="cuda")

    def append(rope, b=batch):
        status.zero_()
        out.fill_(float("nan"))
        return gwa.kv_append(xd[:, 4:6], xd[:, 6:8], c.cache, b, q=xd[:, :4], rope=rope,
                             q_out=out, status=status)

    pos = np.array([38, 39, 19, 20, -1, -1, -1])
    rot = serving.bf16_value(serving.rotate(x[:, :4], serving.rope_table(40, c.D, 1e4), pos))
    got = append(table).float().cpu().numpy()
    assert int(status) == 1
    assert np.array_equal(got[:4], rot[:4])         # a bad page: rotated all the same
    assert (got[4:] == 0).all()                     # of no sequence: zero
    got = append(table[:20].contiguous()).float().cpu().numpy()
    assert int(status) == 3
    assert np.array_equal(got[2], rot[2])
    assert (got[[0, 1, 3, 4, 5, 6]] == 0).all()     # past the rotary table: zero
    none = gwa.KVBatch(i32([0]), i32([]), i32(np.zeros((0, 1))), 7, 2, 40)
    assert (append(table, none) == 0).all()
    k, v = gwa.kv_read(c.cache, none)
    assert (k == 0).all() and (v == 0).all()


def test_a_prompt_chunk_beside_single_tokens_under_a_wide_page_table():
    # 128 sequences, tables wide enough for a million positions each
    rng = np.random.default_rng(38)
    lens = [(260, 300)] + [(1, int(n)) for n in rng.integers(1, 200, 127)]
    c = Case(38, lens, Hq=40, Hkv=8, D=64, page=4096)
    wide = np.full((128, 256), -7, dtype=np.int32)
    wide[:, :c.table.shape[1]] = c.table
    c.table = wide
    check_attention(c)


@pytest.mark.parametrize("lens,Hq,Hkv,D,causal", [
    ([(1, 900), (3, 40)], 8, 2, 128, True),
    ([(1, 1000)], 8, 8, 64, True),
    ([(80, 640)], 1, 1, 256, False),
    ([(80, 640), (1, 64)], 2, 1, 128, True),
    ([(100, 60), (90, 200), (1, 3000)], 4, 2, 256, True)])
def test_results_do_not_depend_on_the_longest_length_given(lens, Hq, Hkv, D, causal):
    c = Case(39, lens, Hq=Hq, Hkv=Hkv, D=D).device()
    q = dev_bf16(rand_bf16(c.rng, c.T, c.Hq, c.D))
    want = gwa.sdpa_paged(q, c.cache, c.batch, causal=causal)
    for longest in (int(c.kl.max()) + 1, 4096, 100000):
        loose = gwa.KVBatch(i32(c.q_start), i32(c.kl), i32(c.table), c.T, int(c.ql.max()), longest)
        ws = gwa.make_sdpa_paged_workspace(c.cache, loose, Hq)
        ws.fill_(255)
        got = gwa.sdpa_paged(q, c.cache, loose, causal=causal, workspace=ws)
        assert torch.equal(want, got)


@pytest.mark.parametrize("q", [1, 3])
def test_one_sequence_does_not_depend_on_a_padded_number_of_new_tokens(q):
    c = Case(40, [(q, 700)], Hq=8, Hkv=2).device()
    x = dev_bf16(rand_bf16(c.rng, c.T, c.Hq, c.D))
    want = gwa.sdpa_paged(x, c.cache, c.batch)
    padded = gwa.KVBatch(i32(c.q_start), i32(c.kl), i32(c.table), c.T, 64, 700)
    assert torch.equal(want, gwa.sdpa_paged(x, c.cache, padded))
