"""Verification of drafted tokens (gwa_verify_draft): the drawn token against
the same whole-number masses, and calls at once.

Masses are floor(2^40 exp2f(y)) with y = (x - top) * fl(fl(1/T) log2 e) in fp32
(exp2f, taken here from torch on the GPU, is what the kernels use), so shares
and cuts can be had exactly and the drawn token's only distance is the
residual's own rounding.  A token's max(p - q, 0) in units of p's likeliest is
t_p - c t_q with c = SP / SQ held to 2^-46 of itself as hi + lo: b lo is
rounded (2^-24 of at most 2^-24 of c t_q), the fma rounds to 2^-24 of c t_q,
the difference to 2^-24 of itself, and the floor takes less than 2^-40.  With
t_p >= the difference: less than 2^-23 c t_q + 2^-24 t_p + 2^-40 a token, and
the sum of that is the distance that the running mass may have.
"""
import numpy as np
import pytest
import torch

import group_wise_affine_gb300 as gwa
from test_gpu_sample import logits
from test_gpu_verify import pair, to_device, uniform

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    gwa.build()
    gwa.load()
    assert torch.cuda.is_available()


def parts(x, T):
    """exp2f of the exponents, fp64 arrays of fp32 values, NaN and -inf zero."""
    x = torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32)).cuda()
    per = np.float32(np.float32(1) / np.float32(T)) * np.float32(1.4426950408889634)
    y = (x - x.max(-1, keepdim=True).values) * torch.tensor(float(per), dtype=torch.float32, device="cuda")
    return torch.exp2(y).nan_to_num(0.0).double().cpu().numpy()


def cut(t, x, k):
    """Those of the first k logits (equal ones by index) stay."""
    if not 0 < k < t.shape[-1]:
        return t
    out = np.zeros_like(t)
    for r, row in enumerate(x):
        keep = np.lexsort((np.arange(len(row)), -row))[:k]
        out[r, keep] = t[r, keep]
    return out


def mass(t):
    return np.floor(t * 2.0 ** 40)


def check_drawn(token, rest, unsure, u):
    """``token`` at share u of the running sum of rest, each entry of which may
    be off by its ``unsure``."""
    c, far = np.cumsum(rest), unsure.sum()
    goal = u * c[-1]
    assert rest[token] > -unsure[token]
    assert c[token] + 2 * far >= goal and c[token] - rest[token] - 2 * far <= goal, (token, goal, c[token], far)


@pytest.mark.parametrize("V,k", [(50, 0), (1000, 0), (1000, 37), (33001, 0), (151669, 0), (151669, 400)])
@pytest.mark.parametrize("noise", [2.0 ** -12, 0.02, 1.0])
@pytest.mark.parametrize("with_draft", [True, False])
def test_the_drawn_token_by_whole_numbers(V, k, noise, with_draft):
    """Drafts that fall at once (u near 1), of draft models that differ by much
    and by little."""
    rng = np.random.default_rng(V + k)
    B, T = 24, 0.8
    x = logits(rng, 2 * B, V)
    y = x + (rng.standard_normal(x.shape) * noise).astype(np.float32)
    tp, tq = cut(parts(x, T), x, k), cut(parts(y, T), y, k)
    P, Q = mass(tp), mass(tq)
    SP, SQ = P.sum(1), Q.sum(1)     # (below 2^53 of 2^-40: exact)
    assert SP.max() < 2.0 ** 53 and SQ.max() < 2.0 ** 53
    drafts = np.zeros(2 * B, np.int32)
    for b in range(B):  # a token that the draft takes for likelier than the target does
        over = Q[2 * b] / SQ[2 * b] - P[2 * b] / SP[2 * b] if with_draft else P[2 * b]
        drafts[2 * b + 1] = int(over.argmax())
    u = np.full(2 * B, 1 - 2.0 ** -24, np.float32)
    ud = uniform(rng, B)
    t = lambda a: torch.from_numpy(a).cuda()  # noqa: E731
    f = lambda v, d: torch.full((2 * B,), v, dtype=d, device="cuda")  # noqa: E731
    token, accepted, _ = gwa.verify_draft(
        t(x), t(drafts), torch.arange(B + 1, dtype=torch.int32, device="cuda") * 2, t(u), t(ud),
        draft_logits=t(y) if with_draft else None, temperature=f(T, torch.float32), top_k=f(k, torch.int32))
    token, accepted = token.cpu().numpy(), accepted.cpu().numpy()
    fell = 0
    for b in range(B):
        d, r = int(drafts[2 * b + 1]), 2 * b
        p, q = int(P[r, d]), int(Q[r, d]) if with_draft else 1
        sq = int(SQ[r]) if with_draft else 1
        stands = ((1 << 24) - 1) * q * int(SP[r]) < (p * sq << 24)
        assert bool(accepted[b]) == stands
        if stands:
            check_drawn(int(token[r + 1]), P[r + 1], np.zeros(V), float(ud[b]))
            continue
        fell += 1
        got = int(token[r])
        if with_draft:
            other = SP[r] / SQ[r] * tq[r]
            unsure = np.where(tp[r] > 0, 2.0 ** -23 * other + 2.0 ** -24 * tp[r] + 2.0 ** -40, 0.0)
            check_drawn(got, np.maximum(tp[r] - other, 0.0), unsure, float(ud[b]))
            assert tp[r, got] - other[got] > -unsure[got] and got != d
        else:
            rest = P[r].copy()
            rest[d] = 0
            check_drawn(got, rest, np.zeros(V), float(ud[b]))
            assert got != d and rest[got] > 0
    assert fell > B // 2


def test_two_calls_at_once():
    """On two streams, wide clusters beside narrow ones."""
    rng = np.random.default_rng(3)
    sets = []
    for lens, V in (([5], 131072), ([4] * 60, 20011)):
        rows = sum(lens)
        x, y = pair(rng, rows, V)
        dx, dy = to_device(x, True)[0], to_device(y, True)[0]
        start = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device="cuda")
        ids = torch.zeros(rows, dtype=torch.int32, device="cuda")
        ids[1:] = dy[:-1].float().argmax(-1).to(torch.int32)
        u, ud = (torch.from_numpy(uniform(rng, n)).cuda() for n in (rows, len(lens)))
        p = torch.full((rows,), 0.9, device="cuda")
        sets.append((dict(logits=dx, ids=ids, q_start=start, u=u, u_draw=ud, draft_logits=dy, top_p=p),
                     gwa.make_verify_workspace(rows), torch.cuda.Stream()))
    want = [gwa.verify_draft(**kw, workspace=w) for kw, w, _ in sets]
    torch.cuda.synchronize()
    got = [[] for _ in sets]
    for _ in range(12):
        for g, (kw, w, s) in zip(got, sets):
            g.append(gwa.verify_draft(**kw, workspace=w, stream=s))
    torch.cuda.synchronize()
    for g, w in zip(got, want):
        for outs in g:
            assert all(torch.equal(a, b) for a, b in zip(outs, w))
