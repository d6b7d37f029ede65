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


@pytest.mark.parametrize("M", [5, 250, 700, 2100])
@pytest.mark.parametrize("rank", [16, 40, 128])
def test_whatever_the_workspace_holds(M, rank):
    """Nothing is taken from it that the call has not put there: the rows of
    tokens without an adapter, what lies past an adapter's rank, shares of K
    that are not used."""
    c = Case(M + rank, some(M), K=2080, sizes=(64, 24), rank=rank, adapters=3, ranks=[rank, 0, rank // 2 - 3])
    x, base, lora, ids = c.device()
    work = gwa.make_lora_workspace(lora, M)
    outs = []
    for fill in (0x00, 0xff, 0x7f):  # zeros, NaN, 3.4e38
        work.fill_(fill)
        outs.append(gwa.lora_add(x, base, lora, ids, workspace=work))
    for g, w, b in zip(outs[0], *c.want()):
        check(bf16_to_f64(g), w, b)
    for other in outs[1:]:
        assert all(torch.equal(a, b) for a, b in zip(outs[0], other))


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


@pytest.mark.parametrize("M", [3, 300, 2100])
def test_infinite_gates_and_inputs(M):
    """An infinite gate makes its own output not finite, an infinite input its
    own token's outputs; no other bit moves."""
    I = 64
    c = Case(M, np.full(M, 1), sizes=(I, I), rank=16, adapters=2, K=96)
    x, (gate, up), lora, ids = c.device()
    want = gwa.lora_gate_up_silu(x, (gate, up), lora, ids)
    gate[0, 3], gate[1, 5], gate[2, 63] = float("inf"), float("-inf"), float("nan")
    got = gwa.lora_gate_up_silu(x, (gate, up), lora, ids)
    hit = torch.zeros(M, I, dtype=torch.bool, device="cuda")
    hit[0, 3] = hit[1, 5] = hit[2, 63] = True
    assert torch.equal(got[~hit], want[~hit]) and not got[hit].isfinite().any()
    x, base, lora, ids = c.device()
    want = gwa.lora_add(x, base, lora, ids)
    x[M // 2, 7] = float("-inf")
    rows = torch.arange(M, device="cuda") != M // 2
    for g, w in zip(gwa.lora_add(x, base, lora, ids), want):
        assert torch.equal(g[rows], w[rows]) and not g[M // 2].isfinite().any()


# ---------------------------------------------------------------- buffers
def guarded(M, n, dtype=torch.bfloat16):
    wide = torch.full((M * n + 256,), 3.0, dtype=dtype, device="cuda")
    return wide, wide[128:-128].view(M, n)


@pytest.mark.parametrize("M,rank", [(40, 16), (300, 24), (2100, 16), (700, 40), (513, 64), (2050, 128)])
@pytest.mark.parametrize("in_place", [False, True])
def test_buffers_between_guards(M, rank, in_place):
    """Rows of 16-byte units, ends of tiles and of blocks of outputs anywhere."""
    sizes = (136, 8, 200)
    c = Case(M + rank, some(M), sizes=sizes, rank=rank, adapters=3, K=96, ranks=[rank, rank - 3, rank // 2])
    x, base, lora, ids = c.device()
    rooms = [guarded(M, n) for n in sizes]
    out = [o for _, o in rooms]
    if in_place:
        for o, b in zip(out, base):
            o.copy_(b)
    gwa.lora_add(x, out if in_place else base, lora, ids, out=out)
    for o, w, b in zip(out, *c.want()):
        check(bf16_to_f64(o), w, b)
    for wide, _ in rooms:
        assert (wide[:128] == 3).all() and (wide[-128:] == 3).all()


@pytest.mark.parametrize("M,rank,I", [(40, 16, 72), (300, 24, 72), (2100, 16, 200), (700, 40, 8), (700, 64, 136)])
def test_gate_up_between_guards(M, rank, I):
    c = Case(M + I, some(M), sizes=(I, I), rank=rank, adapters=3, K=96)
    x, base, lora, ids = c.device()
    want = gwa.lora_gate_up_silu(x, base, lora, ids)
    wide, h = guarded(M, I)
    gwa.lora_gate_up_silu(x, base, lora, ids, h=h)
    assert torch.equal(h, want)
    for at in (0, 1):
        (wide, h), x_base = guarded(M, I), list(base)
        x_base[at] = h.copy_(base[at])
        gwa.lora_gate_up_silu(x, x_base, lora, ids, h=h)
        assert torch.equal(h, want)
        assert (wide[:128] == 3).all() and (wide[-128:] == 3).all()


@pytest.mark.parametrize("M,rank,runs", [(40, 64, 0), (700, 16, 0), (700, 16, 700), (2100, 16, 0), (9000, 64, 0)])
def test_calls_repeat_bit_for_bit(M, rank, runs):
    c = Case(M, ids_of(M, M, 3) if runs else some(M), sizes=(264, 64), rank=rank, adapters=3, K=1056)
    args = c.device()
    first = gwa.lora_add(*args, runs=runs)
    for _ in range(5):
        assert all(torch.equal(a, b) for a, b in zip(first, gwa.lora_add(*args, runs=runs)))
