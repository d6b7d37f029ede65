"""Low-rank adapters of many requests (gwa_lora_add, gwa_lora_gate_up_silu)
against the formula in 64 bits on the same bf16 inputs.

Tolerance.  The output is rounded once: 2^-8 of itself (bf16, half a step).
t = A x is a sum of K exact products in fp32, in any order and with whatever
rounding the tensor cores use: K/8 additions of at most 2^-22 of sum |A x| =
T.  It enters the second product in two bf16 parts, 2^-16 of it, and that sum
of R products and the base's value is again fp32: (R/8 + 4) 2^-22 of sum |B|
|t| + |base|.  So |err| <= 2^-8 |out| + scale sum_r |B_r| (2^-16 + (K/8 + R/8
+ 4) 2^-22) T_r + 2^-20 |base|.  Through the gate, h = SiLU(g) u: |SiLU'(g) u|
e_g + |SiLU(g)| e_u + 2^-8 |h| and the gate's own fp32 roundings, 2^-19 |h|.
"""
import numpy as np
import pytest
import torch

import group_wise_affine_gb300 as gwa
from helpers import bf16_to_f64, dev_bf16
from oracle import serving

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    gwa.build()
    gwa.load()
    assert torch.cuda.is_available()


def rand(rng, *shape, scale=1.0):
    return serving.bf16_round((rng.standard_normal(shape) * scale).astype(np.float32))


def f64(bits):
    return serving.bf16_value(bits).astype(np.float64)


class Case:
    def __init__(self, seed, ids, K=256, sizes=(64, 32), rank=16, adapters=4, ranks=None, scale=True):
        rng = self.rng = np.random.default_rng(seed)
        self.ids, self.K, self.sizes, self.rank = np.asarray(ids, np.int32), K, sizes, rank
        M, N, S = len(self.ids), sum(sizes), len(sizes)
        self.x = rand(rng, M, K)
        self.a = rand(rng, adapters, S, rank, K, scale=K ** -0.5)
        self.b = rand(rng, adapters, N, rank, scale=0.5)
        self.base = [rand(rng, M, n) for n in sizes]
        self.scale = (rng.random(adapters) * 2 - 0.5).astype(np.float32) if scale else None
        self.ranks = None if ranks is None else np.asarray(ranks, np.int32)

    def device(self):
        t = lambda a: None if a is None else torch.from_numpy(a).cuda()  # noqa: E731
        self.lora = gwa.LoRA(dev_bf16(self.a), dev_bf16(self.b), scale=t(self.scale), ranks=t(self.ranks))
        return (dev_bf16(self.x), [dev_bf16(v) for v in self.base], self.lora, t(self.ids))

    def want(self):
        """The sections' outputs and their bars (without the last rounding)."""
        x, a, b, base = f64(self.x), f64(self.a), f64(self.b), [f64(v) for v in self.base]
        out = serving.lora(x, base, a, b, self.ids, self.scale, self.ranks)
        zero = [np.zeros_like(v) for v in base]
        size = None if self.scale is None else np.abs(self.scale)
        mag = serving.lora(np.abs(x), zero, np.abs(a), np.abs(b), self.ids, size, self.ranks)
        rel = 2.0 ** -16 + (self.K / 8 + self.rank / 8 + 4) * 2.0 ** -22
        return out, [rel * m + 2.0 ** -20 * np.abs(v) for m, v in zip(mag, base)]


def check(got, want, bar):
    worst = np.max(np.abs(got - want) / (2.0 ** -8 * np.abs(want) + bar + 1e-30), initial=0.0)
    assert np.isfinite(got).all() and worst <= 1, worst


def run(c, **kw):
    args = c.device()
    got = gwa.lora_add(*args, **kw)
    for g, w, b in zip(got, *c.want()):
        check(bf16_to_f64(g), w, b)
    return got


def ids_of(seed, M, adapters, none=0.2):
    rng = np.random.default_rng(seed)
    return np.where(rng.random(M) < none, -1, rng.integers(0, adapters, M))


# ------------------------------------------------------------------ values
@pytest.mark.parametrize("M", [1, 2, 7, 8, 9, 16, 17, 33, 64, 255, 256, 257, 300])
def test_tokens_in_any_order(M):
    run(Case(M, ids_of(M, M, 4)))


@pytest.mark.parametrize("M", [1, 40, 300])
@pytest.mark.parametrize("rank", [8, 16, 24, 32, 40, 64, 96, 128])
def test_ranks(rank, M):
    run(Case(rank, ids_of(rank, M, 3), rank=rank, adapters=3, K=160))


@pytest.mark.parametrize("M", [5, 290])
@pytest.mark.parametrize("rank", [16, 64])
def test_an_adapters_own_rank(rank, M):
    """0 to rank, odd ones and ones outside; what lies past it is not taken."""
    ranks = [0, 1, 3, rank - 1, rank, rank + 5, -2, rank // 2 + 3]
    c = Case(rank, ids_of(M, M, 8, 0.0), rank=rank, adapters=8, ranks=ranks)
    for e, r in enumerate(ranks):
        r = min(max(r, 0), rank)
        c.a[e, :, r:] = 0x7fc0      # NaN
        c.b[e, :, r:] = 0x7f80      # infinity
    c2 = Case(rank, c.ids, rank=rank, adapters=8, ranks=ranks)
    got = gwa.lora_add(*c.device())
    for g, w, b in zip(got, *c2.want()):
        check(bf16_to_f64(g), w, b)


@pytest.mark.parametrize("K", [32, 64, 96, 512, 1056, 5120, 13824])
@pytest.mark.parametrize("M", [1, 20, 270])
def test_row_lengths(K, M):
    run(Case(K, ids_of(K, M, 3), K=K, adapters=3))


@pytest.mark.parametrize("sizes", [(1,), (8,), (31,), (7, 9, 1), (0, 16), (1024, 256, 256), (33, 5000), (8,) * 8])
@pytest.mark.parametrize("M", [3, 270])
def test_sections(sizes, M):
    run(Case(len(sizes), ids_of(M, M, 4), sizes=sizes))


@pytest.mark.parametrize("runs", [(300,), (200, 1, 99), (128, 128, 128), (17, 500, 3, 40), (2500, 2500), (8191, 1, 900)])
def test_prompts(runs):
    """Runs of neighbours, past what is sorted, and past one launch."""
    ids = np.repeat(np.arange(len(runs)) % 3 - (len(runs) > 3), runs)
    run(Case(sum(runs), ids, sizes=(48, 8), adapters=3))


@pytest.mark.parametrize("rank", [8, 16, 40, 64, 72])
@pytest.mark.parametrize("runs", [(128, 128, 128), (127, 129, 16, 15, 1, 130), (1000, 3, 300), (31, 1, 2, 300, 17), (2000, 15, 129, 200)])
def test_prompts_of_whole_rows(runs, rank):
    """Outputs in units of 16 bytes, ends of tiles and of sections anywhere,
    ranks of the adapters' own, in place and not."""
    ids = np.repeat(np.arange(len(runs)) % 3 - (len(runs) == 5), runs)
    c = Case(sum(runs) + rank, ids, sizes=(136, 64, 8, 200), rank=rank, adapters=3, K=96,
             ranks=[rank, max(1, rank // 2 - 1), rank - 3])
    out = run(c)
    x, base, lora, ids = c.device()
    gwa.lora_add(x, base, lora, ids, out=base)
    assert all(torch.equal(a, b) for a, b in zip(out, base))


@pytest.mark.parametrize("more", [0, 1600])
@pytest.mark.parametrize("rank", [16, 40, 64])
@pytest.mark.parametrize("I", [8, 64, 200])
def test_gate_up_of_prompts(I, rank, more):
    c = Case(I + rank, np.repeat([0, -1, 2, 1], (300, 20, 129 + more, 15)), sizes=(I, I), rank=rank, adapters=3,
             ranks=[rank, rank // 2, rank - 5])
    x, (gate, up), lora, ids = c.device()
    h = bf16_to_f64(gwa.lora_gate_up_silu(x, (gate, up), lora, ids))
    (g, u), (eg, eu) = c.want()
    sig = 1 / (1 + np.exp(-g))
    want = g * sig * u
    slope = np.abs(sig * (1 + g * (1 - sig))) + eg
    check(h, want, slope * np.abs(u) * eg + (np.abs(g * sig) + eg) * eu + 2.0 ** -19 * np.abs(want))
    for at in (0, 1):
        x, y, lora, ids = c.device()
        again = gwa.lora_gate_up_silu(x, y, lora, ids, h=y[at])
        assert torch.equal(again.float(), torch.from_numpy(h).cuda().float())


@pytest.mark.parametrize("M", [257, 511, 512, 700, 9000])
def test_short_runs_that_are_told(M):
    """256 tokens at a time, in order; the same values up to the order of sums."""
    run(Case(M, ids_of(M, M, 5), adapters=5, K=96), runs=M)
    run(Case(M, np.repeat(ids_of(M, M // 10 + 1, 5), 10)[:M], adapters=5, K=96), runs=M // 10 + 1)
    c = Case(M + 1, ids_of(M, M, 5), sizes=(24, 24), rank=32, adapters=5, K=64)
    x, (gate, up), lora, ids = c.device()
    a, b = (gwa.lora_gate_up_silu(x, (gate, up), lora, ids, runs=r).double() for r in (0, M))
    assert ((a - b).abs() <= 2.0 ** -7 * a.abs() + 1e-3).all()


@pytest.mark.parametrize("M,rank", [(3, 16), (40, 64), (40, 128), (600, 64)])
def test_rows_on_16_bytes(M, rank):
    """x, A and B that begin on 16 bytes and not on 32: the same values."""
    c = Case(M, ids_of(M, M, 4), rank=rank, K=2080)
    x, base, lora, ids = c.device()

    def moved(t):
        room = torch.empty(t.numel() + 16, dtype=t.dtype, device="cuda")
        at = 8 if room.data_ptr() % 32 == 0 else 0
        return room[at:at + t.numel()].view(t.shape).copy_(t)

    other = gwa.LoRA(moved(lora.a), moved(lora.b), scale=lora.scale)
    x = moved(x)
    assert x.data_ptr() % 32 == 16 and other.a.data_ptr() % 32 == 16 and other.b.data_ptr() % 32 == 16
    for g, w, b in zip(gwa.lora_add(x, base, other, ids), *c.want()):
        check(bf16_to_f64(g), w, b)


def test_sections_without_outputs():
    run(Case(2100, np.repeat([0, 1, -1], 700), sizes=(0, 64, 0, 8), adapters=2, K=64))
    run(Case(2101, np.repeat([0, 1, -1], 700), sizes=(0, 64, 0, 0, 8, 0), rank=40, adapters=2, K=64))


def test_one_adapter_for_all_and_one_for_each():
    run(Case(1, np.zeros(200), adapters=1))
    run(Case(2, np.arange(200), adapters=200, K=64))
    run(Case(3, np.arange(700) % 350, adapters=350, K=64))


def test_without_scale():
    run(Case(4, ids_of(1, 21, 4), scale=False))


def test_no_adapter_leaves_the_base_as_it_is():
    for M in (9, 300):
        c = Case(M, np.full(M, -1))
        c.base[0][0, :4] = [0x7fc1, 0x8000, 0x0001, 0xff80]  # NaN, -0, the smallest, -infinity
        x, base, lora, ids = c.device()
        for g, b in zip(gwa.lora_add(x, base, lora, ids), base):
            assert torch.equal(torch.nan_to_num(g, 7.0), torch.nan_to_num(b, 7.0))


@pytest.mark.parametrize("M", [6, 300])
def test_in_place_is_the_same(M):
    c = Case(M, ids_of(M, M, 4), sizes=(40, 17))
    x, base, lora, ids = c.device()
    want = gwa.lora_add(x, base, lora, ids)
    got = gwa.lora_add(x, base, lora, ids, out=base)
    for w, g, b in zip(want, got, base):
        assert g is b and torch.equal(w, g)


@pytest.mark.parametrize("M", [1, 13, 80, 300])
@pytest.mark.parametrize("I,rank", [(1, 8), (40, 16), (77, 32), (512, 64), (96, 128)])
def test_gate_up(M, I, rank):
    c = Case(M + I, ids_of(I, M, 4), sizes=(I, I), rank=rank)
    x, (gate, up), lora, ids = c.device()
    h = bf16_to_f64(gwa.lora_gate_up_silu(x, (gate, up), lora, ids))
    (g, u), (eg, eu) = c.want()
    sig = 1 / (1 + np.exp(-g))
    want = g * sig * u
    slope = np.abs(sig * (1 + g * (1 - sig))) + eg  # (|SiLU''| <= 1/2)
    check(h, want, slope * np.abs(u) * eg + (np.abs(g * sig) + eg) * eu + 2.0 ** -19 * np.abs(want))
    again = gwa.lora_gate_up_silu(x, (gate, up), lora, ids, h=gate)
    assert again is gate and torch.equal(again.float(), torch.from_numpy(h).cuda().float())


@pytest.mark.parametrize("M", [5, 300])
def test_no_adapters_at_all(M):
    """A server without one loaded: the base as it is, every id told."""
    c = Case(M, np.zeros(M), adapters=1, sizes=(40, 40))
    x, base, _, ids = c.device()
    lora = gwa.LoRA(*(torch.empty(0, *s, dtype=torch.bfloat16, device="cuda") for s in ((2, 16, 256), (80, 16))))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = gwa.lora_add(x, base, lora, ids, status=status)
    assert all(torch.equal(g, b) for g, b in zip(got, base)) and int(status) == 1
    h = gwa.lora_gate_up_silu(x, base, lora, ids).float()
    g, u = (b.double() for b in base)
    assert ((h - g * torch.sigmoid(g) * u).abs() <= 2.0 ** -7 * h.abs() + 1e-30).all()


def test_many_sections_of_wide_adapters():
    """More rows of A than one pass of the tensor cores takes (256)."""
    run(Case(9, ids_of(9, 400, 3), sizes=(16,) * 8, rank=64, adapters=3, K=96))
    run(Case(10, ids_of(10, 400, 2), sizes=(16, 24, 8), rank=128, adapters=2, K=96))


def test_ids_past_the_adapters_are_told():
    for M in (10, 300):
        c = Case(M, ids_of(3, M, 4))
        c.ids[3] = 4
        c.ids[7] = 0x7fffffff
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        run(c, status=status)
        assert int(status) == 1
        c.ids[[3, 7]] = -5
        status.zero_()
        run(c, status=status)
        assert int(status) == 0


def test_other_tokens_do_not_matter():
    """Not finite inputs stay in their own rows, and a row's bits do not
    depend on the others'."""
    for M in (30, 300):
        c = Case(M, ids_of(M, M, 3), adapters=3)
        want = run(c)
        x, base, lora, ids = c.device()
        bad = torch.arange(M, device="cuda") % 5 == 2
        x[bad] = float("nan")
        got = gwa.lora_add(x, base, lora, ids)
        for g, w in zip(got, want):
            assert torch.equal(g[~bad], w[~bad])
            assert torch.isnan(g[bad & (ids >= 0)]).all()


def test_runs_repeat_and_replay():
    c = Case(5, ids_of(5, 70, 4), sizes=(300, 20), rank=32)
    x, base, lora, ids = c.device()
    out = [torch.empty_like(b) for b in base]
    work = gwa.make_lora_workspace(lora, 70)
    first = [t.clone() for t in gwa.lora_add(x, base, lora, ids, out=out, workspace=work)]
    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=side):
        gwa.lora_add(x, base, lora, ids, out=out, workspace=work)
    c.ids = ids_of(6, 70, 4).astype(np.int32)  # other adapters, same graph
    ids.copy_(torch.from_numpy(c.ids))
    graph.replay()
    torch.cuda.synchronize()
    for g, w, b in zip(out, *c.want()):
        check(bf16_to_f64(g), w, b)
    ids.copy_(torch.from_numpy(ids_of(5, 70, 4).astype(np.int32)))
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, out))


@pytest.mark.parametrize("M,rank", [(700, 16), (2100, 40)])
def test_prompts_replay(M, rank):
    """A captured call of prompts, replayed with other runs, in place."""
    lens = [M // 3, 40, M // 2, 9]
    ids_a = np.repeat([1, -1, 0, 2, 1], lens + [M - sum(lens)]).astype(np.int32)
    c = Case(M, ids_a, sizes=(64, 24), rank=rank, adapters=3, K=96)
    x, base, lora, ids = c.device()
    y = [b.clone() for b in base]
    work = gwa.make_lora_workspace(lora, M)
    gwa.lora_add(x, y, lora, ids, out=y, workspace=work)
    first = [t.clone() for t in y]
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        gwa.lora_add(x, y, lora, ids, out=y, workspace=work)
    for order in (ids_a[::-1].copy(), np.full(M, 2, np.int32), ids_a):
        c.ids = order
        ids.copy_(torch.from_numpy(order))
        for t, b in zip(y, base):
            t.copy_(b)
        graph.replay()
        torch.cuda.synchronize()
        for g, w, b in zip(y, *c.want()):
            check(bf16_to_f64(g), w, b)
    assert all(torch.equal(a, b) for a, b in zip(first, y))


def test_two_streams_at_once():
    cases = [Case(i, np.repeat([0, 2, 1], 800), sizes=(128, 8), rank=rank, adapters=3, K=512) for i, rank in ((1, 16), (2, 64))]
    args = [c.device() for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    work = [gwa.make_lora_workspace(a[2], 2400) for a in args]
    out = [[torch.empty_like(b) for b in a[1]] for a in args]
    torch.cuda.synchronize()
    for _ in range(20):
        for a, s, w, o in zip(args, streams, work, out):
            gwa.lora_add(*a, out=o, workspace=w, stream=s)
    torch.cuda.synchronize()
    for c, o in zip(cases, out):
        for g, w, b in zip(o, *c.want()):
            check(bf16_to_f64(g), w, b)


def test_another_stream():
    c = Case(6, ids_of(6, 300, 4))
    s = torch.cuda.Stream()
    args = c.device()
    torch.cuda.synchronize()
    got = gwa.lora_add(*args, stream=s)
    s.synchronize()
    for g, w, b in zip(got, *c.want()):
        check(bf16_to_f64(g), w, b)


def test_rows_outside_are_not_touched():
    """Buffers between guards, with rows that are no 16-byte units."""
    c = Case(7, ids_of(7, 270, 4), sizes=(13,))
    x, (base,), lora, ids = c.device()
    wide = torch.full((270 * 13 + 6,), 3.0, dtype=torch.bfloat16, device="cuda")
    out = wide[3:-3].view(270, 13)
    gwa.lora_add(x, [base], lora, ids, out=[out])
    check(bf16_to_f64(out), c.want()[0][0], c.want()[1][0])
    assert (wide[:3] == 3).all() and (wide[-3:] == 3).all()
