"""Adapters (gwa_lora_add, gwa_lora_gate_up_silu): workspaces, alignment, far
gates, and what lies around and in front of their buffers.  Values against the
formula in 64 bits, tolerances as in test_gpu_lora; the rest bit for bit.
"""
import numpy as np
import pytest
import torch

import group_wise_affine_gb300 as gwa
from helpers import bf16_to_f64
from oracle import serving
from test_gpu_lora import Case, check, ids_of

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    gwa.build()
    gwa.load()
    assert torch.cuda.is_available()
    gwa.pipeline_status()
    yield
    assert gwa.pipeline_status() == 0


def some(M):
    """Ids of three adapters: in no order, of more than 256 tokens runs of a
    third, 20, a half, 9 and what is left."""
    if M <= 256:
        return ids_of(M, M, 3)
    lens = [M // 3, 20, M // 2, 9]
    return np.repeat([1, -1, 0, 2, 1], lens + [M - sum(lens)])


# ---------------------------------------------------------------- workspaces
def test_a_workspace_for_more_tokens_serves_fewer():
    """Made once, for the largest step."""
    rank, most = 64, 5000
    work = None
    for M in (most, 4096, 4999, 2731, 2000, 257, 256, 1):
        c = Case(M, ids_of(M, M, 3), K=64, sizes=(48,), rank=rank, adapters=3)
        args = c.device()
        if work is None:
            work = gwa.make_lora_workspace(c.lora, most)
        got = gwa.lora_add(*args, workspace=work)
        for g, w, b in zip(got, *c.want()):
            check(bf16_to_f64(g), w, b)
    for M in (500, 6144, 8200):
        c = Case(M, ids_of(M, M, 3), K=64, sizes=(48,), rank=rank, adapters=3)
        args = c.device()
        got = gwa.lora_add(*args, workspace=gwa.make_lora_workspace(c.lora, M + 1), runs=M)
        for g, w, b in zip(got, *c.want()):
            check(bf16_to_f64(g), w, b)


# ---------------------------------------------------------------- dispatch
def test_long_runs_of_a_long_call_that_are_told():
    """200 runs in 16384 tokens are long ones, in each of the launches that the
    call is made of: the same kernels, and bits, as where nothing is told."""
    M = 16384
    c = Case(1, np.repeat(np.arange(200) % 4, 82)[:M], K=64, sizes=(256,), rank=40)
    x, base, lora, ids = c.device()
    plain, = gwa.lora_add(x, base, lora, ids)
    told, = gwa.lora_add(x, base, lora, ids, runs=200)
    assert torch.equal(plain, told)
    check(bf16_to_f64(told[-600:]), c.want()[0][0][-600:], c.want()[1][0][-600:])


# ---------------------------------------------------------------- alignment
def moved(t):
    """A copy that begins on 16 bytes and not on 32."""
    room = torch.empty(t.numel() + 16, dtype=t.dtype, device="cuda")
    at = 8 if room.data_ptr() % 32 == 0 else 0
    out = room[at:at + t.numel()].view(t.shape).copy_(t)
    assert out.data_ptr() % 32 == 16
    return out


@pytest.mark.parametrize("M", [1, 40, 256])
@pytest.mark.parametrize("rank", [16, 64, 128])
@pytest.mark.parametrize("own", [False, True])
def test_bits_do_not_depend_on_where_buffers_begin(M, rank, own):
    c = Case(M, ids_of(M, M, 4, none=0.0), K=4128, sizes=(4096, 1024), rank=rank, ranks=[rank] * 4 if own else None)
    x, base, lora, ids = c.device()
    want = gwa.lora_add(x, base, lora, ids)
    for what in ("x", "a", "b", "xab"):
        other = gwa.LoRA(moved(lora.a) if "a" in what else lora.a, moved(lora.b) if "b" in what else lora.b,
                         scale=lora.scale, ranks=lora.ranks)
        got = gwa.lora_add(moved(x) if "x" in what else x, base, other, ids)
        assert all(torch.equal(a, b) for a, b in zip(got, want)), what


# ---------------------------------------------------------------- far gates
@pytest.mark.parametrize("M", [3, 60, 300, 2100])
@pytest.mark.parametrize("size", [0, 100])
def test_gates_far_from_zero(M, size):
    """Gates of 60 to 100 on either side, where e^-g leaves fp32's range, and
    up to 2^100 on the other half.  Beside the bar of test_gpu_lora: the fast
    exponential is off by 2 + 1.173 |g| steps of fp32 (2^-23), the quotient by
    2, the slope is taken at the far end of g's error, and below fp32's normal
    range e^-|g| is a whole number of 2^-149 (a bf16 of 2^-133)."""
    I, rank = 64, 16
    c = Case(M + size, some(M), sizes=(I, I), rank=rank, adapters=3, K=96)
    rng = np.random.default_rng(M)
    g0 = rng.uniform(60, 100, (M, I)) * rng.choice([-1.0, 1.0], (M, I))
    c.base[0] = serving.bf16_round(g0.astype(np.float32))
    c.base[1] = serving.bf16_round((rng.standard_normal((M, I)) * 2.0 ** size).astype(np.float32))
    x, (gate, up), lora, ids = c.device()
    h = bf16_to_f64(gwa.lora_gate_up_silu(x, (gate, up), lora, ids))
    (g, u), (eg, eu) = c.want()
    e = np.exp(-np.abs(g))
    sig = np.where(g < 0, e, 1.0) / (1 + e)
    want = g * sig * u
    slope = (np.abs(sig * (1 + g * (1 - sig))) + np.minimum(eg, e)) * np.exp(eg)
    fast = (4 + 1.173 * np.abs(g)) * 2.0 ** -23 + 2.0 ** -22
    bar = slope * np.abs(u) * eg + np.abs(g * sig) * eu * (1 + eg) + fast * np.abs(want) \
        + np.abs(g * u) * 2.0 ** -149 + 2.0 ** -133
    check(h, want, bar)
    if size:
        assert (np.abs(h[(g < -88) & (g > -95)]) > 0).all()
