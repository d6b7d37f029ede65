"""Token sampling (gwa_sample) against a plain CPU implementation in 64 bits.

The rule decides by whole-number masses, each within 2^-18 of the real one:
the exponent's two fp32 roundings at |y| <= 40 (2^-23 |y| ln 2 < 2^-18.2) and
exp2f's two ulps.  So a cut or a draw may differ from the real-valued rule
only where a cumulative mass lies within 2^-17 of the total of its goal; the
check accepts every token that some boundary within that distance allows, and
the probability within 2^-16 relative.
"""
import numpy as np
import pytest
import torch

import group_wise_affine_gb300 as gwa
from helpers import dev_bf16
from oracle import serving

pytestmark = pytest.mark.gpu
EPS = 2.0 ** -17


@pytest.fixture(scope="module", autouse=True)
def _lib():
    gwa.build()
    gwa.load()
    assert torch.cuda.is_available()


def logits(rng, rows, V, peaks=8):
    x = rng.standard_normal((rows, V)).astype(np.float32) * 2
    for r in range(rows):
        n = min(peaks, V)
        x[r, rng.integers(0, V, n)] += rng.uniform(2, 9, n).astype(np.float32)
    return x


def allowed(x, u, T, k, p, mp):
    """(token, probability) pairs that the rule allows for one row."""
    V = len(x)
    x = np.where(np.isnan(x), -np.inf, x)
    if x.max() == -np.inf:
        return [(-1, 0.0)]
    order = serving.sample_order(x)
    if not T > 0:
        return [(int(order[0]), 1.0)]
    w = serving.sample_masses(x, T)
    n = k if 0 < k < V else V
    ws = w[order[:n]]
    W = ws.sum()
    lens = {n}
    if p < 1:
        before = np.cumsum(ws) - ws
        lo = max(1, int((before < (p - EPS) * W).sum()))
        hi = max(1, int((before < (p + EPS) * W).sum()))
        lens = set(range(lo, hi + 1)) if hi - lo < 50 else {lo, hi}
    if mp > 0:
        lo = int((ws >= min(mp, 1.0) * (1 + EPS)).sum())
        hi = int((ws >= min(mp, 1.0) * (1 - EPS)).sum())
        lens = {max(1, min(m, c)) for m in lens for c in range(lo, hi + 1)}
    out = []
    for m in lens:
        keep = np.sort(order[:m])
        c = np.cumsum(w[keep])
        tot = c[-1]
        a = int(np.searchsorted(c, (u - EPS) * tot, side="right"))
        b = int(np.searchsorted(c, (u + EPS) * tot, side="right"))
        for i in range(a, min(b, m - 1) + 1):
            out.append((int(keep[i]), w[keep[i]] / tot))
    return out


def run(x, u, T=None, k=None, p=None, mp=None, bf16=False, pad=0):
    rows, V = x.shape
    f = lambda a, t: None if a is None else torch.from_numpy(np.asarray(a, dtype=t)).cuda()
    if bf16:
        bits = serving.bf16_round(np.where(np.isfinite(x), x, 0))
        bits = np.where(x == np.inf, 0x7f80, np.where(x == -np.inf, 0xff80,
                                                      np.where(np.isnan(x), 0x7fc0, bits)))
        x = serving.bf16_value(bits.astype(np.uint16))
        d = dev_bf16(bits.astype(np.uint16))
    else:
        d = torch.from_numpy(np.ascontiguousarray(x)).cuda()
    if pad:
        wide = torch.full((rows, V + pad), 99.0, dtype=d.dtype, device="cuda")
        wide[:, pad // 2:pad // 2 + V] = d
        d = wide[:, pad // 2:pad // 2 + V]
    tok, prob = gwa.sample(d, f(u, np.float32), f(T, np.float32), f(k, np.int32),
                           f(p, np.float32), f(mp, np.float32))
    tok, prob = tok.cpu().numpy(), prob.cpu().numpy()
    for r in range(rows):
        ok = allowed(x[r].astype(np.float64), float(np.float32(u[r])),
                     1.0 if T is None else float(np.float32(T[r])), 0 if k is None else int(k[r]),
                     1.0 if p is None else float(np.float32(p[r])),
                     0.0 if mp is None else float(np.float32(mp[r])))
        hit = [q for t, q in ok if t == tok[r]]
        assert hit, (r, tok[r], ok[:5])
        assert min(abs(prob[r] - q) for q in hit) <= 2.0 ** -16 * prob[r] + 1e-12, (r, prob[r], hit)
    return tok, prob


@pytest.mark.parametrize("V", [1, 2, 7, 8, 31, 33, 1000, 4097, 50257, 151669, 524288])
@pytest.mark.parametrize("bf16", [False, True])
def test_vocabularies(V, bf16):
    rng = np.random.default_rng(V)
    n = 4
    run(logits(rng, n, V), rng.random(n), T=rng.uniform(0.5, 1.5, n),
        k=rng.integers(1, 60, n), p=rng.uniform(0.3, 1, n), mp=rng.uniform(0, 0.1, n), bf16=bf16)


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("on", ["", "k", "p", "m", "kp", "km", "pm", "kpm"])
def test_each_filter(on, bf16):
    rng = np.random.default_rng(len(on) + 10 * bf16)
    n, V = 40, 3001
    run(logits(rng, n, V), rng.random(n), T=rng.uniform(0.2, 2.0, n),
        k=rng.integers(0, 300, n) if "k" in on else None,
        p=rng.uniform(0, 1.05, n) if "p" in on else None,
        mp=rng.uniform(0, 0.3, n) if "m" in on else None, bf16=bf16, pad=5)


@pytest.mark.parametrize("rows", [1, 3, 19, 160, 700])
def test_row_counts(rows):
    rng = np.random.default_rng(rows)
    run(logits(rng, rows, 2500), rng.random(rows), T=rng.uniform(0.5, 1.5, rows),
        k=rng.integers(0, 50, rows), p=rng.uniform(0.3, 1, rows))


def test_the_token_does_not_depend_on_the_split():
    # the same row alone (a large cluster) and among many (a small one)
    rng = np.random.default_rng(5)
    for bf16 in (False, True):
        x = torch.from_numpy(logits(rng, 1, 130001, peaks=200)).cuda()
        x = x.bfloat16() if bf16 else x
        many = 300
        for i in range(6):
            f = lambda v: torch.full((many,), v, device="cuda")
            u = f(float(rng.random()))
            a = dict(temperature=f(1.3), top_p=f(0.97),
                     top_k=torch.full((many,), [0, 5000][i % 2], dtype=torch.int32, device="cuda"))
            one = {k: v[:1] for k, v in a.items()}
            t1, p1 = gwa.sample(x, u[:1], **one)
            t2, p2 = gwa.sample(x.expand(many, -1).contiguous(), u, **a)
            assert (t2 == t1).all() and (p2 == p1).all()


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("V", [9001, 40011, 200001])
def test_rows_that_keep_many_tokens(V, bf16):
    # nearly flat rows, whose kept tokens no short list holds: each filter,
    # from few tokens to nearly all, few rows (wide clusters) and many
    rng = np.random.default_rng(V + bf16)
    for n in (2, 160):
        x = rng.standard_normal((n, V)).astype(np.float32) * 0.4
        off = lambda a, z: np.where(rng.random(n) < 0.4, z, a)
        run(x, rng.random(n), T=rng.uniform(0.5, 1.5, n),
            k=off(rng.integers(400, V, n), 0), p=off(rng.uniform(0.05, 0.999, n), 1.0),
            mp=off(rng.uniform(0.0, 0.5, n), 0.0), bf16=bf16)
        if n * V > 2e6:
            break


@pytest.mark.parametrize("bf16", [False, True])
def test_many_equal_logits_around_the_cut(bf16):
    # a few values only: thousands of equals at the cut of a small top-k
    rng = np.random.default_rng(11)
    x = np.round(rng.standard_normal((24, 30011)) * 1.5).astype(np.float32)
    x = np.minimum(x, 2)
    k = np.resize([1, 2, 60, 512, 513, 2500], 24)
    run(x, rng.random(24), T=rng.uniform(0.5, 1.5, 24), k=k, bf16=bf16)
    run(x, rng.random(24), T=rng.uniform(0.5, 1.5, 24), k=k, p=rng.uniform(0.1, 0.99, 24),
        mp=rng.uniform(0, 0.3, 24), bf16=bf16)
    run(x, rng.random(24), p=rng.uniform(0.01, 0.99, 24), mp=rng.uniform(0, 1, 24), bf16=bf16)


def test_ties_go_to_the_lowest_index():
    V, n = 5000, 64
    x = np.zeros((n, V), np.float32)
    u = (np.arange(n) + 0.5) / n
    tok, prob = run(x, u, k=np.full(n, 7))
    assert set(tok) == set(range(7)) and np.allclose(prob, 1 / 7)
    tok, _ = run(x, u, p=np.full(n, 0.01))            # 50 of 5000
    assert set(tok) == set(range(0, 50)) & set(tok) and tok.max() < 50
    x[:, 3::5] = 1.0                                  # 1000 equal tops
    tok, _ = run(x, u, k=np.full(n, 3), p=np.full(n, 0.99))
    assert set(tok) <= {3, 8, 13}
    tok, _ = run(x, u, T=np.zeros(n))
    assert set(tok) == {3}


def test_zeros_of_both_signs_are_equal():
    x = np.zeros((4, 9), np.float32)
    x[:, 0] = -0.0
    for bf16 in (False, True):
        tok, _ = run(x, [0.1, 0.5, 0.9, 0.99], k=[1] * 4, bf16=bf16)
        assert (tok == 0).all()


@pytest.mark.parametrize("bf16", [False, True])
def test_infinities_and_nan(bf16):
    V = 300
    x = np.random.default_rng(1).standard_normal((6, V)).astype(np.float32)
    x[0, :] = -np.inf
    x[1, :] = np.nan
    x[2, 5:] = -np.inf
    x[3, 7] = x[3, 200] = np.inf
    x[4, ::2] = np.nan
    x[5, 1:] = -np.inf
    for p in (1.0, 0.5):
        tok, prob = run(x, [0.3, 0.5, 0.7, 0.9, 0.2, 0.999], p=[p] * 6, k=[0, 0, 40, 0, 30, 250],
                        bf16=bf16)
        assert tok[0] == -1 and tok[1] == -1 and prob[0] == 0
        assert tok[2] < 5 and tok[3] in (7, 200) and tok[4] % 2 == 1 and tok[5] == 0
    run(x, [0.3] * 6, T=[0.0] * 6, bf16=bf16)


def test_extreme_parameters():
    rng = np.random.default_rng(2)
    x = logits(rng, 8, 1000)
    for T in (1e-30, 1e-3, 50.0, 1e30):
        run(x, rng.random(8), T=[T] * 8)
    x[:, ::3] = -np.inf
    tok, _ = run(x, rng.random(8), T=[np.inf] * 8)
    assert (tok % 3 != 0).all()
    run(x, [0.0, 0.9999999, 0.0, 0.9999999] * 2, p=[0.0] * 4 + [1e-9] * 4)
    run(x, rng.random(8), mp=[1.0] * 8)
    run(x, rng.random(8), k=[-5, 0, 1, 2, 999, 1000, 1001, 1 << 30])
    # random numbers outside [0, 1) are drawn as its ends
    t, _ = gwa.sample(torch.zeros((4, 10), device="cuda"),
                      torch.tensor([-1.0, 1.0, 7.0, float("nan")], device="cuda"))
    assert t.tolist() == [0, 9, 9, 0]


def test_frequencies_follow_the_probabilities():
    n = 20000
    x = np.tile(np.log(np.array([0.1, 0.2, 0.3, 0.4], np.float32)), (n, 1))
    t, _ = gwa.sample(torch.from_numpy(x).cuda(), torch.from_numpy(
        ((np.arange(n) + 0.5) / n).astype(np.float32)).cuda())
    c = np.bincount(t.cpu().numpy(), minlength=4) / n
    assert np.abs(c - [0.1, 0.2, 0.3, 0.4]).max() < 1e-3


def test_another_stream_and_a_graph():
    rng = np.random.default_rng(3)
    x = torch.from_numpy(logits(rng, 5, 40000)).cuda()
    u = torch.rand(5, device="cuda")
    want, _ = gwa.sample(x, u)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got, _ = gwa.sample(x, u, stream=s)
    s.synchronize()
    assert torch.equal(got, want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got, _ = gwa.sample(x, u)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(got, want)


def test_refusals():
    x = torch.zeros((2, 10), device="cuda")
    u = torch.zeros(2, device="cuda")
    with pytest.raises(ValueError):
        gwa.sample(x.half(), u)
    with pytest.raises(ValueError):
        gwa.sample(x, u[:1])
    with pytest.raises(ValueError):
        gwa.sample(x, u.double())
    with pytest.raises(ValueError):
        gwa.sample(x.t(), torch.zeros(10, device="cuda"))
    with pytest.raises(ValueError):
        gwa.sample(x, u, top_k=torch.zeros(2, dtype=torch.int64, device="cuda"))
    with pytest.raises(ValueError):
        gwa.sample(x.cpu(), u)
    with pytest.raises(gwa.GwaError):
        gwa.sample(torch.zeros((1, 524289), device="cuda"), u[:1])
    with pytest.raises(gwa.GwaError):
        gwa.sample(torch.zeros((1, 0), device="cuda"), u[:1])
