"""Attention through a sliding window (gwa_sdpa_paged_window): strided queries,
other streams, calls at once.  Tolerance as in test_gpu_window."""
import numpy as np
import pytest
import torch

import group_wise_affine_gb300 as gwa
from helpers import bf16_to_f64, dev_bf16
from test_gpu_paged import Case, rand_bf16
from test_gpu_window import peak, want

pytestmark = pytest.mark.gpu

# few rows, both kernels, prompts
BATCHES = [[(1, 1900), (2, 90)], [(1, 900), (150, 800), (0, 4), (7, 60)], [(300, 1500)]]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    gwa.build()
    gwa.load()
    assert torch.cuda.is_available()
    gwa.pipeline_status()
    yield
    assert gwa.pipeline_status() == 0


def made(seed, lens, **kw):
    c = Case(seed, lens, **{"Hq": 8, "Hkv": 2, **kw})
    q = rand_bf16(c.rng, c.T, c.Hq, c.D, scale=0.7)
    return c.device(), q


@pytest.mark.parametrize("lens", BATCHES)
@pytest.mark.parametrize("D,bits", [(64, 8), (128, 4), (256, 4)])
def test_strided_queries(lens, D, bits):
    """Heads that lie among others, NaN on both sides of them."""
    c, q = made(D, lens, D=D, bits=bits)
    ref = want(c, q, 200, 5, 1.0 / np.sqrt(D))
    wide = torch.full((c.T, c.Hq + 3, D), float("nan"), dtype=torch.bfloat16, device="cuda")
    wide[:, 1:1 + c.Hq] = dev_bf16(q)
    got = gwa.sdpa_paged(wide[:, 1:1 + c.Hq], c.cache, c.batch, window=200, sinks=5)
    bar = 2.0 ** -8 * np.abs(ref) + 2.0 ** -10 * peak(c)
    assert (np.abs(bf16_to_f64(got) - ref) <= bar).all()
    assert torch.equal(got, gwa.sdpa_paged(dev_bf16(q), c.cache, c.batch, window=200, sinks=5))


def test_other_streams_and_calls_at_once():
    """Calls of several kinds on a stream each, on workspaces that hold
    anything: the bits of the same calls one after the other."""
    sets = [made(i, lens) for i, lens in enumerate(BATCHES)]
    kw = [dict(window=w, sinks=s) for w, s in ((700, 4), (64, 0), (333, 20))]
    queries = [dev_bf16(q) for _, q in sets]
    one = [gwa.sdpa_paged(q, c.cache, c.batch, **k) for q, (c, _), k in zip(queries, sets, kw)]
    works = [gwa.make_sdpa_paged_workspace(c.cache, c.batch, c.Hq, **k).fill_(0xff) for (c, _), k in zip(sets, kw)]
    streams = [torch.cuda.Stream() for _ in sets]
    torch.cuda.synchronize()
    got = [[] for _ in sets]
    for _ in range(10):
        for i, (c, _) in enumerate(sets):
            got[i].append(gwa.sdpa_paged(queries[i], c.cache, c.batch, workspace=works[i], stream=streams[i], **kw[i]))
    torch.cuda.synchronize()
    for outs, w in zip(got, one):
        assert all(torch.equal(o, w) for o in outs)
