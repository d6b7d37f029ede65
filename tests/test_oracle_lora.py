"""The plain implementation of the adapters pinned by hand, and the refusals
of their entry points, all without a GPU."""
import ctypes

import numpy as np
import pytest

from oracle import serving


def test_adapters_worked_by_hand():
    x = np.array([[1.0, 2.0], [3.0, -1.0], [5.0, 5.0]])
    a = np.zeros((2, 2, 2, 2))
    a[0, 0] = [[1, 0], [0, 1]]      # section 0: t = x
    a[0, 1] = [[1, 1], [9, 9]]      # section 1: t = (x0 + x1, ..), the second past the rank
    b = np.zeros((2, 3, 2))
    b[0] = [[1, 10], [0, 2], [4, 7]]  # two outputs of section 0, one of section 1
    base = [np.ones((3, 2)), np.zeros((3, 1))]
    out = serving.lora(x, base, a, b, [0, -1, 2], scale=[0.5, 1.0], ranks=[1, 2])
    assert out[0].tolist() == [[1.5, 1.0], [1, 1], [1, 1]]
    assert out[1].tolist() == [[6.0], [0], [0]]
    out = serving.lora(x, base, a, b, [0, 0, 1])
    assert out[0].tolist() == [[22.0, 5.0], [-6.0, -1.0], [1, 1]]


@pytest.fixture(scope="module")
def lib():
    import group_wise_affine_gb300 as gwa
    gwa.build()
    return gwa.load()


def lora(gwa, **kw):
    a = dict(a=1 << 20, b=1 << 20, scale=None, ranks=None, N=96, K=256, sections=2, rank=16, adapters=3)
    a.update(kw)
    return gwa._Lora(**a)


BAD = [("rank", 4, "UNSUPPORTED"), ("rank", 12, "UNSUPPORTED"), ("rank", 136, "UNSUPPORTED"), ("sections", 0, "UNSUPPORTED"),
       ("sections", 9, "UNSUPPORTED"), ("K", 0, "INVALID_ARG"), ("K", 40, "INVALID_ARG"), ("K", 1 << 21, "INVALID_ARG"),
       ("N", -2, "INVALID_ARG"), ("adapters", -1, "INVALID_ARG"), ("a", 0, "INVALID_ARG"), ("b", 0, "INVALID_ARG"),
       ("a", (1 << 20) + 2, "MISALIGNED"), ("b", (1 << 20) + 8, "MISALIGNED"), ("scale", (1 << 20) + 2, "MISALIGNED"),
       ("ranks", (1 << 20) + 1, "MISALIGNED")]


def call(lib, l, x=1 << 20, M=4, ids=1 << 20, runs=0, sizes=(64, 32), base=(1 << 20, 1 << 20), out=(1 << 20, 1 << 20), ws=1 << 20,
         n=1 << 30, status=None):
    c = lambda t, v: (t * len(v))(*v)  # noqa: E731
    return lib.gwa_lora_add(x, M, l, ids, runs, c(ctypes.c_int64, sizes), c(ctypes.c_void_p, base), c(ctypes.c_void_p, out), ws, n,
                            status, None)


@pytest.mark.parametrize("field,value,code", BAD)
def test_adapters_are_checked(lib, field, value, code):
    import group_wise_affine_gb300 as gwa
    want = getattr(gwa, "GWA_ERR_" + code)
    assert call(lib, lora(gwa, **{field: value})) == want
    assert gwa.last_error()
    assert lib.gwa_lora_gate_up_silu(1 << 20, 4, lora(gwa, **{field: value}), 1 << 20, 0, 1 << 20, 1 << 20, 1 << 20, 1 << 20, 1 << 30,
                                     None, None) == want


@pytest.mark.parametrize("kw,code", [
    (dict(x=None), "INVALID_ARG"), (dict(ids=None), "INVALID_ARG"), (dict(runs=-1), "INVALID_ARG"), (dict(M=-1), "INVALID_ARG"),
    (dict(sizes=(64, 31)), "INVALID_ARG"), (dict(sizes=(-1, 97)), "INVALID_ARG"), (dict(base=(1 << 20, None)), "INVALID_ARG"),
    (dict(out=(None, 1 << 20)), "INVALID_ARG"), (dict(out=((1 << 20) + 1, 1 << 20)), "MISALIGNED"),
    (dict(x=(1 << 20) + 8), "MISALIGNED"), (dict(ids=(1 << 20) + 2), "MISALIGNED"), (dict(status=(1 << 20) + 2), "MISALIGNED"),
    (dict(ws=None), "WORKSPACE"), (dict(n=100), "WORKSPACE"), (dict(ws=(1 << 20) + 8), "MISALIGNED")])
def test_arguments_are_checked(lib, kw, code):
    import group_wise_affine_gb300 as gwa
    assert call(lib, lora(gwa), **kw) == getattr(gwa, "GWA_ERR_" + code)


def test_gate_up_wants_two_equal_sections(lib):
    import group_wise_affine_gb300 as gwa
    p = 1 << 20
    for l in (lora(gwa, sections=3), lora(gwa, N=97), lora(gwa, sections=1)):
        assert lib.gwa_lora_gate_up_silu(p, 4, l, p, 0, p, p, p, p, 1 << 30, None, None) == gwa.GWA_ERR_INVALID_ARG


def test_rows_past_31_bits_are_refused(lib):
    import group_wise_affine_gb300 as gwa
    assert call(lib, lora(gwa, adapters=1 << 27)) == gwa.GWA_ERR_INVALID_ARG
    assert "adapters=134217728" in gwa.last_error()


def test_nothing_to_do_and_workspaces(lib):
    import group_wise_affine_gb300 as gwa
    assert call(lib, lora(gwa), M=0) == 0
    assert call(lib, lora(gwa, N=0), sizes=(0, 0)) == 0
    size = lambda M: lib.gwa_lora_workspace_bytes(lora(gwa), M)  # noqa: E731
    assert size(0) == 0 and not gwa.last_error()
    assert size(1) >= 2 * 16 * 4 and size(300) >= 300 * 2 * 16 * 4 and size(100000) > 0
    assert size(-1) == 0 and gwa.last_error()


def test_binding_refuses_mismatched_tensors():
    import torch

    import group_wise_affine_gb300 as gwa
    z = lambda *s, t=torch.bfloat16: torch.zeros(s, dtype=t)  # noqa: E731
    for a, b, kw in ((z(2, 1, 8), z(2, 9, 8), {}), (z(2, 1, 8, 32), z(3, 9, 8), {}), (z(2, 1, 8, 32), z(2, 9, 16), {}),
                     (z(2, 1, 8, 32), z(2, 9, 8), dict(scale=z(2))), (z(2, 1, 8, 32), z(2, 9, 8), dict(ranks=z(3, t=torch.int32)))):
        with pytest.raises(ValueError):
            gwa.LoRA(a, b, **kw)
    with pytest.raises(TypeError):
        gwa.LoRA(z(2, 1, 8, 32, t=torch.float32), z(2, 9, 8))
