"""Attention over the paged cache through a sliding window, with first tokens
that stay visible (gwa_sdpa_paged_window), against fp64 on the same cache.

Tolerance as in test_gpu_paged: with P the largest |v| that a token of the
case sees, 2^-8 |out| + 2^-10 P (weights 2^-11 of themselves times values of
at most 2 P after the centre's shift, fp32 biases, scores within 2^-16, one
bf16 rounding).
"""
import numpy as np
import pytest
import torch

import group_wise_affine_gb300 as gwa
from helpers import bf16_to_f64, dev_bf16
from oracle import serving
from test_gpu_paged import Case, rand_bf16

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    gwa.build()
    gwa.load()
    assert torch.cuda.is_available()


def want(c, q, window, sinks, scale):
    kv = [c.sequence(b) for b in range(len(c.kl))]
    return serving.attention_window(serving.bf16_value(q).astype(np.float64), [k for k, _ in kv],
                                    [v for _, v in kv], c.q_start, c.kl, scale, window, sinks)


def peak(c):
    return max([np.abs(c.sequence(b)[1]).max() for b in range(len(c.kl)) if c.kl[b]] + [1e-30])


def check(c, window, sinks=0, status_want=0, big=None, ref=None, **kw):
    q = rand_bf16(c.rng, c.T, c.Hq, c.D, scale=0.7)
    scale = 1.0 / np.sqrt(c.D)
    ref = want(c, q, window, sinks, scale) if ref is None else ref(q, scale)
    big = peak(c) if big is None else big
    c.device()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = bf16_to_f64(gwa.sdpa_paged(dev_bf16(q), c.cache, c.batch, scale=scale, status=status, window=window,
                                     sinks=sinks, **kw))
    assert int(status) == status_want
    worst = np.max(np.abs(got - ref) / (2.0 ** -8 * np.abs(ref) + 2.0 ** -10 * big))
    assert np.isfinite(got).all() and worst <= 1, worst
    return got


@pytest.mark.parametrize("kv", [1, 2, 16, 17, 127, 128, 129, 300, 1000, 4097])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (2, 4), (16, 0), (17, 3), (128, 4), (129, 128), (500, 16),
                                          (1000, 129), (5000, 4), (40, 6000), (2 ** 31 - 1, 2 ** 31 - 1)])
def test_one_token(kv, window, sinks):
    check(Case(kv, [(1, kv)], Hq=10, Hkv=2), window, sinks)


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("rep,q", [(1, 1), (5, 1), (8, 1), (5, 3), (4, 8), (7, 5), (1, 17)])
def test_widths_heads_and_rows(bits, D, rep, q):
    c = lambda: Case(D + bits + rep, [(q, 700), (max(1, q - 1), 70), (q, 1300)], Hq=2 * rep, Hkv=2, D=D, bits=bits, page=32)  # noqa: E731
    check(c(), 150, 4)
    check(c(), 3, 0)


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("window,sinks", [(1, 0), (7, 1), (64, 0), (100, 4), (128, 64), (257, 130), (900, 3), (5000, 0)])
def test_prompts(D, bits, window, sinks):
    check(Case(window + D, [(300, 300), (130, 700), (77, 78)], Hq=8, Hkv=2, D=D, bits=bits), window, sinks)


@pytest.mark.parametrize("page", [16, 64, 4096])
def test_prompt_chunks_and_pages(page):
    check(Case(page, [(513, 2100)], Hq=5, Hkv=1, page=page), 600, 4)
    check(Case(page, [(2, 5000), (1, 17), (3, 256)], page=page), 400, 20)


def test_ragged_batch_with_empty_sequences():
    rng = np.random.default_rng(0)
    lens = [(int(rng.integers(0, 3)), int(n)) for n in rng.integers(3, 700, 70)]
    lens[3], lens[11], lens[40] = (0, 0), (0, 50), (2, 2)
    check(Case(5, lens, Hq=4, Hkv=1), 90, 5)
    # single tokens beside prompts: both kernels
    check(Case(6, [(1, 900), (200, 800), (0, 4), (5, 60), (90, 90)], Hq=8, Hkv=2), 120, 4)


@pytest.mark.parametrize("q", [6, 200])
def test_more_new_tokens_than_the_cache_holds(q):
    """Rows at negative positions see nothing, and are zero."""
    got = check(Case(q, [(q, q - 3)], Hq=4, Hkv=2), 2, 1)
    assert (got[:3] == 0).all() and (got[3:] != 0).any()


@pytest.mark.parametrize("lens", [[(1, 1500)], [(4, 700), (1, 9)], [(300, 1200)]])
def test_a_window_past_the_start_is_the_causal_mask(lens):
    c = Case(9, lens, Hq=8, Hkv=2).device()
    q = dev_bf16(rand_bf16(c.rng, c.T, c.Hq, c.D))
    plain = gwa.sdpa_paged(q, c.cache, c.batch)
    for window in (1500, 10 ** 6):
        assert torch.equal(gwa.sdpa_paged(q, c.cache, c.batch, window=window, sinks=window % 7), plain)


@pytest.mark.parametrize("lens", [[(1, 2000)], [(5, 2000), (3, 900)], [(150, 2000)]])
@pytest.mark.parametrize("D", [128, 256])
def test_pages_that_no_token_sees_are_not_read(lens, D):
    window, sinks, page = 300, 20, 16
    c = Case(D, lens, Hq=8, Hkv=2, D=D, page=page)
    plain = check(Case(D, lens, Hq=8, Hkv=2, D=D, page=page), window, sinks)
    for b, (n, m) in enumerate(lens):
        low = max(0, m - n - window + 1)
        used = {t // page for t in range(m) if t >= low or t < sinks}
        for j in range(-(-m // page)):
            if j not in used:
                c.table[b, j] = (-1, 2 ** 30, 7 - 2 ** 31)[j % 3]
    q_like = Case(D, lens, Hq=8, Hkv=2, D=D, page=page)  # (the same draws)
    got = check(c, window, sinks, big=peak(q_like), ref=lambda q, s: want(q_like, q, window, sinks, s))
    assert (got == plain).all()


def hide(c, seen, kbits, vbits):
    """Puts parameters into the keys of sequence 0 outside ``seen``."""
    for t in range(int(c.kl[0])):
        if not seen(t):
            pg, sl = c.table[0, t // c.page], t % c.page
            c.kp[pg, :, sl], c.vp[pg, :, sl] = kbits, vbits


@pytest.mark.parametrize("kbits,vbits", [(0x7fc0, 0x7fc0), (0x7f80, 0xff80), (0x0000, 0x7f80), (0x7f00, 0x7f00)])
@pytest.mark.parametrize("q", [1, 40])
def test_whatever_hidden_keys_hold(q, kbits, vbits):
    """NaN, infinities and values near bf16's end in front of every window and
    behind the first keys."""
    lens, window, sinks = [(q, 900)], 200, 5
    plain = Case(q, lens, Hq=4, Hkv=1)
    low = 900 - q - window + 1
    c = Case(q, lens, Hq=4, Hkv=1)
    hide(c, lambda t: t >= low or t < sinks, kbits, vbits)
    check(c, window, sinks, big=peak(plain), ref=lambda q, s: want(plain, q, window, sinks, s))


@pytest.mark.parametrize("q", [3, 60])
def test_large_values_in_front_of_some_windows(q):
    """A key that the first token sees and the others do not, 2^12 times the
    others' values: those rows keep their tolerance, which is relative to what
    they see."""
    lens, window = [(q, 700)], 100
    c = Case(q, lens, Hq=4, Hkv=1)
    t = 700 - q - window + 1  # the first token's first key
    pg, sl = c.table[0, t // c.page], t % c.page
    big = serving.bf16_value(c.vp[pg, :, sl]) * np.float32(4096)
    c.vp[pg, :, sl] = serving.bf16_round(big)
    qb = rand_bf16(c.rng, c.T, c.Hq, c.D, scale=0.7)
    scale = 1.0 / np.sqrt(c.D)
    ref = want(c, qb, window, 0, scale)
    small = peak(Case(q, lens, Hq=4, Hkv=1))
    c.device()
    got = bf16_to_f64(gwa.sdpa_paged(dev_bf16(qb), c.cache, c.batch, scale=scale, window=window))
    bar = 2.0 ** -8 * np.abs(ref) + 2.0 ** -10 * small
    bar[0] += 2.0 ** -10 * 4096 * small
    assert (np.abs(got - ref) <= bar).all()


@pytest.mark.parametrize("lens", [[(1, 3000)], [(3, 900), (1, 2000)], [(100, 1500), (1, 5)]])
def test_looser_bounds_change_nothing(lens):
    c = Case(2, lens, Hq=8, Hkv=2).device()
    q = dev_bf16(rand_bf16(c.rng, c.T, c.Hq, c.D))
    first = gwa.sdpa_paged(q, c.cache, c.batch, window=250, sinks=4)
    c.batch.max_kv = 100000
    assert torch.equal(gwa.sdpa_paged(q, c.cache, c.batch, window=250, sinks=4), first)


def test_a_captured_step_follows_the_lengths():
    c = Case(3, [(1, 700), (2, 300)], Hq=8, Hkv=2).device()
    c.batch.max_kv = 700
    q = rand_bf16(c.rng, c.T, c.Hq, c.D, scale=0.7)
    qd = dev_bf16(q)
    work = gwa.make_sdpa_paged_workspace(c.cache, c.batch, c.Hq, window=130, sinks=4)
    out = torch.empty_like(qd)
    run = lambda: gwa.sdpa_paged(qd, c.cache, c.batch, window=130, sinks=4, workspace=work, out=out)  # noqa: E731
    run()
    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=side):
        run()
    for kl in ([700, 300], [5, 299], [129, 134], [0, 2], [650, 17]):
        c.kl = np.array(kl)
        c.batch.kv_len.copy_(torch.tensor(kl, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        ref = want(c, q, 130, 4, 1.0 / np.sqrt(c.D))
        bar = 2.0 ** -8 * np.abs(ref) + 2.0 ** -10 * peak(c)
        assert (np.abs(bf16_to_f64(out) - ref) <= bar).all()


def test_refusals_of_the_binding():
    c = Case(1, [(1, 20)]).device()
    q = dev_bf16(rand_bf16(c.rng, 1, c.Hq, c.D))
    for kw in (dict(window=5, causal=False), dict(sinks=3)):
        with pytest.raises(ValueError):
            gwa.sdpa_paged(q, c.cache, c.batch, **kw)
    for kw in (dict(window=0), dict(window=-1), dict(window=3, sinks=-1)):
        with pytest.raises(gwa.GwaError):
            gwa.sdpa_paged(q, c.cache, c.batch, **kw)
        with pytest.raises(gwa.GwaError):
            gwa.make_sdpa_paged_workspace(c.cache, c.batch, c.Hq, **kw)
