"""The plain windowed attention pinned to independent statements, and the
refusals of its entry point, all without a GPU."""
import ctypes

import numpy as np
import pytest

from oracle import serving
from test_oracle_serving import BAD, BAD_BATCH, batch, cache


def problem(seed=0, lens=((1, 5), (0, 3), (4, 4), (2, 0), (3, 9))):
    rng = np.random.default_rng(seed)
    q_start = np.concatenate([[0], np.cumsum([a for a, _ in lens])])
    kl = np.array([b for _, b in lens])
    q = rng.standard_normal((q_start[-1], 4, 8))
    k = [rng.standard_normal((n, 2, 8)) for n in kl]
    v = [rng.standard_normal((n, 2, 8)) for n in kl]
    return q, k, v, q_start, kl


def test_a_long_window_is_the_causal_mask():
    p = problem()
    want = serving.attention(*p, 0.3, True)
    for window, sinks in ((9, 0), (100, 3), (1, 9)):
        assert np.allclose(serving.attention_window(*p, 0.3, window, sinks), want, atol=1e-12)


def test_a_window_of_one_is_the_tokens_own_value():
    q, k, v, q_start, kl = problem()
    got = serving.attention_window(q, k, v, q_start, kl, 0.3, 1, 0)
    for b in range(len(kl)):
        for i in range(q_start[b], q_start[b + 1]):
            p = kl[b] - q_start[b + 1] + i
            own = np.repeat(v[b][p], 2, 0) if p >= 0 else 0.0
            assert np.allclose(got[i], own)


def test_window_and_first_keys_by_hand():
    """Equal scores: the mean of the values that a token sees."""
    v = np.arange(6.0).reshape(6, 1, 1)
    z = np.zeros((2, 1, 1))
    got = serving.attention_window(z, [np.zeros((6, 1, 1))], [v], [0, 2], [6], 1.0, 2, 1)
    # positions 4 and 5: keys {3, 4} and {4, 5}, each with key 0
    assert np.allclose(got[:, 0, 0], [7 / 3, 3.0])


@pytest.fixture(scope="module")
def lib():
    import group_wise_affine_gb300 as gwa
    gwa.build()
    return gwa.load()


def call(lib, c, b, window=4, sinks=1, q=1 << 20, out=1 << 20, ws=1 << 20, n=1 << 30):
    return lib.gwa_sdpa_paged_window(q, 512, 4, c, b, 0.1, window, sinks, out, ws, n, None, None)


@pytest.mark.parametrize("field,value,code", BAD + BAD_BATCH)
def test_cache_and_batch_are_checked(lib, field, value, code):
    import group_wise_affine_gb300 as gwa
    c = cache(gwa, **({field: value} if (field, value, code) in BAD else {}))
    b = batch(gwa, **({field: value} if (field, value, code) in BAD_BATCH else {}))
    assert call(lib, c, b) == getattr(gwa, "GWA_ERR_" + code)
    assert gwa.last_error()


@pytest.mark.parametrize("kw,code", [(dict(window=0), "INVALID_ARG"), (dict(window=-3), "INVALID_ARG"),
                                     (dict(sinks=-1), "INVALID_ARG"), (dict(q=None), "INVALID_ARG"),
                                     (dict(out=(1 << 20) + 8), "MISALIGNED"), (dict(ws=None), "WORKSPACE"),
                                     (dict(n=16), "WORKSPACE")])
def test_arguments_are_checked(lib, kw, code):
    import group_wise_affine_gb300 as gwa
    assert call(lib, cache(gwa), batch(gwa), **kw) == getattr(gwa, "GWA_ERR_" + code)


def test_workspace(lib):
    import group_wise_affine_gb300 as gwa
    f = lib.gwa_sdpa_paged_window_workspace_bytes
    c, b = cache(gwa, num_pages=1 << 20), batch(gwa, max_pages=1 << 16, max_kv=1 << 20)
    whole = lib.gwa_sdpa_paged_workspace_bytes(4, c, b)
    assert 0 < f(4, c, b, 100, 4) <= whole and f(4, c, b, 2 ** 31 - 1, 0) == whole
    assert f(4, c, b, 0, 0) == 0 and gwa.last_error()
    assert f(3, c, b, 5, 0) == 0
    assert call(lib, c, batch(gwa, tokens=0)) == 0
