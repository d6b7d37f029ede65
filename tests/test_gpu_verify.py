"""Verification of drafted tokens (gwa_verify_draft) against the rule in 64
bits with real-valued masses.

Whole-number masses are within 2^-18 of the real ones (test_gpu_sample), so a
share p or q is within 2^-16 relative (its own mass and the sum's), a filter's
cut can move where a cumulative mass lies within 2^-17 of its goal, and the
running mass of max(p - q, 0) within 2^-15 of the row's whole mass.  The check
accepts every decision that some value within these distances allows.
"""
import itertools

import numpy as np
import pytest
import torch

import group_wise_affine_gb300 as gwa
from helpers import dev_bf16
from oracle import serving
from test_gpu_sample import EPS, logits

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    gwa.build()
    gwa.load()
    assert torch.cuda.is_available()


def shares(x, T, k, p, mp):
    """Every set of shares that the rounding of the filters' cuts allows."""
    base = serving.kept_shares(x, T, k, p, mp)
    if not T > 0 or not base.any():
        return [base]
    x = np.where(np.isnan(x), -np.inf, x)
    order, w = serving.sample_order(x), serving.sample_masses(x, T)
    n = int(k) if 0 < k < len(x) else len(x)
    ws = w[order[:n]]
    lens = {n}
    if p < 1:
        before, W = np.cumsum(ws) - ws, ws.sum()
        lens = set(range(max(1, int((before < (p - EPS) * W).sum())), max(1, int((before < (p + EPS) * W).sum())) + 1))
        lens = lens if len(lens) < 20 else {min(lens), max(lens)}
    if mp > 0:
        lo, hi = (int((ws >= min(mp, 1.0) * (1 + e)).sum()) for e in (EPS, -EPS))
        lens = {max(1, min(m, c)) for m in lens for c in range(lo, hi + 1)}
    return [serving.kept_shares(x, T, k, p, mp, count=m) for m in lens]


def check_sequence(token, accepted, prob, xs, ys, drafts, us, u_draw, f):
    """One sequence: xs its target rows, ys its draft rows (or None)."""
    n = len(drafts)
    ps = [shares(x, *f) for x in xs]
    qs = [shares(y, *f) for y in ys] if ys is not None else None
    assert 0 <= accepted <= n
    V = len(xs[0])
    for j, d in enumerate(drafts):
        may = []
        for a, q in itertools.product(ps[j], qs[j] if qs is not None else [None]):
            pd = a[d] if 0 <= d < V else 0.0
            qd = (q[d] if 0 <= d < V else 0.0) if q is not None else 1.0
            may.append((us[j] * qd * (1 - 2.0 ** -15) < pd, not us[j] * qd * (1 + 2.0 ** -15) < pd,
                        min(1.0, pd / qd) if qd > 0 else float(pd > 0)))
        assert min(abs(prob[j] - m[2]) for m in may) <= 2.0 ** -15 * prob[j] + 1e-9, (j, prob[j], may)
        if j < accepted:
            assert token[j] == d and any(m[0] for m in may), (j, us[j], may)
        if j == accepted:
            assert any(m[1] for m in may), (j, us[j], may)
    assert prob[n] == 0
    assert (token[accepted + 1:n + 1] == -1).all()
    j, ok = accepted, False
    for a, q in itertools.product(ps[j], qs[j] if qs is not None and j < n else [None]):
        if not a.any():
            ok = ok or token[j] == -1
            continue
        rest = a
        if j < n:
            rest = a.copy()
            if q is not None:
                rest = np.maximum(a - q, 0.0)
            elif 0 <= drafts[j] < V:
                rest[drafts[j]] = 0.0
            if rest.sum() <= 2.0 ** -15:  # nothing but roundings
                ok = ok or a[token[j]] > 0
                continue
        c = np.cumsum(rest)
        lo = int(np.searchsorted(c, u_draw * c[-1] - 2.0 ** -15, side="right"))
        hi = min(int(np.searchsorted(c, u_draw * c[-1] + 2.0 ** -15, side="right")), V - 1)
        # (a token of the run may have lost its own mass to the rounding, or won one from it)
        ok = ok or (lo <= token[j] <= hi and rest[token[j]] > -2.0 ** -15 and a[token[j]] > 0)
    assert ok, (j, token[j], u_draw)


def to_device(x, bf16):
    if bf16:
        bits = serving.bf16_round(np.where(np.isfinite(x), x, 0))
        bits = np.where(x == np.inf, 0x7f80, np.where(x == -np.inf, 0xff80, np.where(np.isnan(x), 0x7fc0, bits)))
        return dev_bf16(bits.astype(np.uint16)), serving.bf16_value(bits.astype(np.uint16))
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32)).cuda(), x.astype(np.float32)


def uniform(rng, n):
    return (rng.integers(0, 1 << 24, n) * 2.0 ** -24).astype(np.float32)


def run(rng, lens, x, y, drafts=None, T=None, k=None, p=None, mp=None, bf16=False, pad=0, lead=0):
    """lens: drafts of each sequence + 1 (0: none).  Filters by sequence."""
    lens = np.asarray(lens)
    R, V = x.shape
    start = lead + np.concatenate([[0], np.cumsum(lens)])
    dx, x = to_device(x, bf16)
    dy, y = to_device(y, bf16) if y is not None else (None, None)
    if pad:
        wide = torch.full((2, R, V + pad), 77.0, dtype=dx.dtype, device="cuda")
        wide[0, :, 1:V + 1] = dx
        dx = wide[0, :, 1:V + 1]
        if dy is not None:
            wide[1, :, pad:] = dy
            dy = wide[1, :, pad:]
    B = len(lens)
    val = lambda a, off: np.full(B, off) if a is None else np.asarray(a)  # noqa: E731
    seq = np.clip(np.searchsorted(start, np.arange(R), side="right") - 1, 0, B - 1)
    f = [val(T, 1.0).astype(np.float32), val(k, 0).astype(np.int32), val(p, 1.0).astype(np.float32), val(mp, 0.0).astype(np.float32)]
    if drafts is None:  # drawn from the drafts' rows, or the target's likelier tokens
        drafts = np.zeros(R, np.int64)
        for i in range(R - 1):
            b = seq[i]
            s = serving.kept_shares((x if y is None else y)[i], *(float(v[b]) for v in f))
            c = np.cumsum(s)
            drafts[i + 1] = min(int(np.searchsorted(c, rng.random() * c[-1], side="right")), V - 1) if c[-1] > 0 else 0
    us, ud = uniform(rng, R), uniform(rng, B)
    t = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
    token, accepted, prob = gwa.verify_draft(
        dx, t(drafts.astype(np.int32)), t(start.astype(np.int32)), t(us), t(ud), draft_logits=dy,
        **{n: None if given is None else t(v[seq]) for n, given, v in
           zip(("temperature", "top_k", "top_p", "min_p"), (T, k, p, mp), f)})
    token, accepted, prob = token.cpu().numpy(), accepted.cpu().numpy(), prob.cpu().numpy()
    for b in range(B):
        a, e = start[b], start[b + 1]
        if a == e:
            assert accepted[b] == 0
            continue
        check_sequence(token[a:e], int(accepted[b]), prob[a:e], x[a:e].astype(np.float64),
                       None if y is None else y[a:e - 1].astype(np.float64), [int(d) for d in drafts[a + 1:e]],
                       us[a:e - 1].astype(np.float64), float(ud[b]), [float(v[b]) for v in f])
    outside = np.ones(R, bool)
    outside[start[0]:start[-1]] = False
    assert (token[outside] == -1).all() and (prob[outside] == 0).all()
    return token, accepted


def pair(rng, R, V, noise=0.7, peaks=8):
    x = logits(rng, R, V, peaks)
    return x, x + rng.standard_normal((R, V)).astype(np.float32) * np.float32(noise)


@pytest.mark.parametrize("V", [1, 2, 7, 33, 1000, 4097, 50257, 151669, 524288])
@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("with_draft", [True, False])
def test_vocabularies(V, bf16, with_draft):
    rng = np.random.default_rng(V)
    lens = [3, 1, 5, 0, 2] if V < 60000 else [3, 2]
    x, y = pair(rng, sum(lens), V)
    n = len(lens)
    run(rng, lens, x, y if with_draft else None, T=rng.uniform(0.5, 1.5, n), k=rng.integers(1, 60, n),
        p=rng.uniform(0.3, 1, n), mp=rng.uniform(0, 0.1, n), bf16=bf16)


@pytest.mark.parametrize("on", ["", "k", "p", "m", "kp", "km", "pm", "kpm"])
@pytest.mark.parametrize("bf16", [False, True])
def test_each_filter(on, bf16):
    rng = np.random.default_rng(len(on) + 10 * bf16)
    lens = [4] * 12
    x, y = pair(rng, 48, 3001)
    n = 12
    run(rng, lens, x, y, T=rng.uniform(0.2, 2.0, n), k=rng.integers(0, 300, n) if "k" in on else None,
        p=rng.uniform(0, 1.05, n) if "p" in on else None, mp=rng.uniform(0, 0.3, n) if "m" in on else None, bf16=bf16, pad=5)


@pytest.mark.parametrize("B", [1, 3, 40, 200])
def test_batches(B):
    rng = np.random.default_rng(B)
    lens = rng.integers(0, 6, B)
    lens[0] = 4
    x, y = pair(rng, int(lens.sum()), 1500)
    run(rng, lens, x, y, T=rng.uniform(0.5, 1.5, B), p=rng.uniform(0.5, 1, B))


def test_greedy_rows():
    rng = np.random.default_rng(1)
    x, y = pair(rng, 60, 800, noise=0.2)
    x[:, 5] = x[:, 700] = x.max(1) + 1      # equal largest: the lower index
    y[:30] = x[:30]
    token, accepted = run(rng, [6] * 10, x, y, T=[0.0] * 5 + [-1.0, 0.7, 0.0, 1.0, 0.0])
    assert (accepted[:5] == 5).all() and (token[:30] == 5).all()
    d = np.full(60, 5)
    d[8] = 700                               # certain drafts, one of them the other equal
    token, accepted = run(rng, [6] * 10, x, None, drafts=d, T=[0.0] * 10)
    assert accepted.tolist() == [5, 1] + [5] * 8 and token[7] == 5 and (token[8:12] == -1).all()


def test_a_draft_model_that_agrees_always_stands():
    rng = np.random.default_rng(2)
    x = logits(rng, 80, 2000)
    _, accepted = run(rng, [80], x, x.copy(), T=[0.9], p=[0.9])
    assert accepted[0] == 79                 # more than two warps of drafts


def test_drafts_that_the_target_excludes():
    rng = np.random.default_rng(3)
    x, y = pair(rng, 12, 500)
    x[:, 100:] = -np.inf
    y[:, :100] = -np.inf
    _, accepted = run(rng, [4, 4, 4], x, y)
    assert (accepted == 0).all()
    _, accepted = run(rng, [4, 4, 4], x, y, drafts=np.array([0, -1, 500, 1 << 30] * 3))
    assert (accepted == 0).all()
    _, accepted = run(rng, [4, 4, 4], x, None, drafts=np.array([0, -1, 500, 1 << 30] * 3))
    assert (accepted == 0).all()


def test_a_certain_draft_is_all_that_is_left():
    """p is the draft alone: it stands, whatever u."""
    x = np.full((2, 50), -np.inf, np.float32)
    x[:, 7] = 1.0
    token, accepted = run(np.random.default_rng(4), [2], x, None, drafts=np.array([0, 7]))
    assert token.tolist() == [7, 7] and accepted[0] == 1


def test_rows_without_a_token():
    rng = np.random.default_rng(5)
    x, y = pair(rng, 9, 300)
    x[1] = -np.inf
    x[4] = np.nan
    y[6] = -np.inf
    token, accepted = run(rng, [3, 3, 3], x, y, drafts=np.array([0, 3, 5, 0, 2, 9, 0, 1, 2]))
    assert accepted[0] <= 1


def test_infinite_and_nan_logits():
    rng = np.random.default_rng(6)
    x, y = pair(rng, 12, 300)
    x[rng.random(x.shape) < 0.1] = np.nan
    y[rng.random(x.shape) < 0.1] = -np.inf
    x[2, 40] = x[2, 41] = np.inf
    y[5, 17] = np.inf
    run(rng, [4, 4, 4], x, y, T=[1.0, 0.5, np.inf])


def test_equal_logits():
    rng = np.random.default_rng(7)
    x = np.zeros((4, 5000), np.float32)
    y = np.zeros((4, 5000), np.float32)
    y[:, ::2] = 0.5
    run(rng, [4], x, y)
    run(rng, [4], x, y, k=[77])
    run(rng, [4], x, x.copy(), p=[0.5])


def test_rows_outside_every_sequence():
    rng = np.random.default_rng(8)
    x, y = pair(rng, 14, 400)
    run(rng, [3, 0, 4], x, y, lead=2)


def test_no_rows_at_all():
    z = lambda *s, t=torch.float32: torch.zeros(s, dtype=t, device="cuda")  # noqa: E731
    token, accepted, prob = gwa.verify_draft(z(0, 50), z(0, t=torch.int32), z(4, t=torch.int32), z(0), z(3))
    assert token.numel() == prob.numel() == 0 and accepted.tolist() == [0, 0, 0]


@pytest.mark.parametrize("with_draft", [True, False])
def test_the_tokens_are_the_targets(with_draft):
    """Over many sequences the first token has the target's distribution, and
    so has the second where the first draft stood."""
    g = torch.Generator(device="cuda").manual_seed(0)
    n, V = 200000, 6
    p1 = torch.tensor([0.30, 0.05, 0.20, 0.05, 0.25, 0.15], device="cuda")
    p2 = torch.tensor([0.10, 0.30, 0.10, 0.20, 0.10, 0.20], device="cuda")
    q = torch.tensor([0.10, 0.25, 0.20, 0.15, 0.05, 0.25], device="cuda")
    x = torch.stack([p1.log(), p2.log()]).repeat(n, 1)
    y = q.log().repeat(2 * n, 1)
    ids = torch.multinomial(q, 2 * n, replacement=True, generator=g).to(torch.int32)
    start = torch.arange(n + 1, device="cuda", dtype=torch.int32) * 2
    u, ud = torch.rand(2 * n, device="cuda", generator=g), torch.rand(n, device="cuda", generator=g)
    token, accepted, _ = gwa.verify_draft(x, ids, start, u, ud, draft_logits=y if with_draft else None)
    token = token.view(n, 2)
    for got, p in ((token[:, 0], p1), (token[accepted == 1, 1], p2)):
        m = got.numel()
        share = torch.bincount(got.long(), minlength=V) / m
        assert (share - p).abs().max() < 5 * 0.5 / m ** 0.5, (share, p)
    assert abs(float(accepted.float().mean()) - float(torch.minimum(p1, q).sum() if with_draft else (q * p1).sum())) < 0.01


def test_the_result_does_not_depend_on_the_split():
    """One sequence alone (wide clusters) and among many (narrow ones)."""
    rng = np.random.default_rng(9)
    x, y = pair(rng, 5, 130001, peaks=200)
    many = 160
    for bf16 in (False, True):
        dx, dy = to_device(x, bf16)[0], to_device(y, bf16)[0]
        for i in range(3):
            u = torch.from_numpy(uniform(rng, 5)).cuda()
            ud = torch.from_numpy(uniform(rng, 1)).cuda()
            ids = torch.from_numpy(rng.integers(0, 130001, 5).astype(np.int32)).cuda()
            ids[1:] = dy[:-1].float().argmax(-1).to(torch.int32)
            f = lambda v, n, t=torch.float32: torch.full((n,), v, device="cuda", dtype=t)  # noqa: E731
            start = torch.arange(many + 1, device="cuda", dtype=torch.int32) * 5
            a = gwa.verify_draft(dx, ids, start[:2], u, ud, draft_logits=dy, temperature=f(1.2, 5),
                                 top_p=f([1.0, 0.97, 0.5][i], 5))
            r = lambda t: t.repeat(many, *[1] * (t.dim() - 1))  # noqa: E731
            b = gwa.verify_draft(r(dx), r(ids), start, r(u), r(ud), draft_logits=r(dy), temperature=f(1.2, 5 * many),
                                 top_p=f([1.0, 0.97, 0.5][i], 5 * many))
            for s, t in zip(a, b):
                assert torch.equal(r(s), t)


def test_a_captured_step_and_another_stream():
    rng = np.random.default_rng(10)
    x, y = pair(rng, 8, 2000)
    dx, dy = to_device(x, True)[0], to_device(y, True)[0]
    ids = torch.from_numpy(rng.integers(0, 2000, 8).astype(np.int32)).cuda()
    start = torch.tensor([0, 4, 8], dtype=torch.int32, device="cuda")
    u, ud = (torch.from_numpy(uniform(rng, n)).cuda() for n in (8, 2))
    work = gwa.make_verify_workspace(8)
    run = lambda **kw: gwa.verify_draft(dx, ids, start, u, ud, draft_logits=dy, workspace=work, **kw)  # noqa: E731
    run()
    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=side):
        out = run()
    for i in range(3):
        ids.copy_(torch.from_numpy(rng.integers(0, 2000, 8).astype(np.int32)))
        start.copy_(torch.tensor([[0, 4, 8], [0, 1, 7], [0, 0, 8]][i], dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        kept = [t.clone() for t in out]
        assert all(torch.equal(a, b) for a, b in zip(kept, run()))
    torch.cuda.synchronize()
    got = run(stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, kept))
