"""The plain verification of drafted tokens pinned by hand and by what it
promises, and the refusals of its entry point, all without a GPU."""
import numpy as np
import pytest

from oracle import serving


def test_by_hand():
    p = np.array([0.5, 0.3, 0.2, 0.0])
    q = np.array([0.2, 0.6, 0.2, 0.0])
    run = lambda d, u, v, qq=q: serving.verify([p, p], None if qq is None else [qq], [d], [u], v)  # noqa: E731
    assert run(0, 0.99, 0.6) == ([0, 1], 1)          # p > q always stands; then 0.6 of p falls on 1
    assert run(1, 0.49, 0.0) == ([1, 0], 1)          # 0.49 x 0.6 < 0.3
    assert run(1, 0.5, 0.99) == ([0], 0)             # falls: max(p - q, 0) has token 0 alone
    assert run(3, 0.5, 0.7) == ([0], 0)              # a share of zero never stands
    assert run(1, 0.29, 0.9, None) == ([1, 2], 1)    # certain drafts stand with p
    assert run(1, 0.31, 0.72, None) == ([2], 0)      # without token 1: shares 5/7 and 2/7


def test_the_first_token_is_the_targets():
    rng = np.random.default_rng(0)
    p, q = np.array([0.1, 0.2, 0.3, 0.4]), np.array([0.4, 0.1, 0.1, 0.4])
    for qq in ([q], None):
        n = 40000
        got = np.zeros(4)
        for _ in range(n):
            d = int(rng.choice(4, p=q))
            got[serving.verify([p, p], qq, [d], [rng.random()], rng.random())[0][0]] += 1
        assert (np.abs(got / n - p) < 5 * np.sqrt(p * (1 - p) / n)).all()


def test_kept_shares():
    x = np.array([1.0, 3.0, 2.0, -np.inf, np.nan, 2.0])
    s = serving.kept_shares(x, 1.0, 2, 1.0, 0.0)
    e = np.exp(-1.0)
    assert np.allclose(s, [0, 1 / (1 + e), e / (1 + e), 0, 0, 0])
    assert serving.kept_shares(x, 0.0, 0, 0.5, 0.0).tolist() == [0, 1, 0, 0, 0, 0]
    assert np.allclose(serving.kept_shares(x, 1.0, 0, 1.0, 0.5), [0, 1, 0, 0, 0, 0])
    assert np.allclose(serving.kept_shares(x, 1.0, 0, 0.6, 0.0), s)
    assert serving.kept_shares(np.full(3, -np.inf), 1.0, 0, 1.0, 0.0).sum() == 0


@pytest.fixture(scope="module")
def lib():
    import group_wise_affine_gb300 as gwa
    gwa.build()
    return gwa.load()


P = 1 << 20
ARGS = dict(logits=P, dtype=0, rows=4, V=100, stride=100, draft=P, draft_stride=100, ids=P, q_start=P, batch=2, u=P, u_draw=P, T=None,
            k=None, p=None, m=None, token=P, accepted=P, prob=None, ws=P, n=1 << 20, stream=None)


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=2), "UNSUPPORTED"), (dict(V=524289, stride=1 << 20, draft_stride=1 << 20), "UNSUPPORTED"),
    (dict(V=0), "INVALID_ARG"), (dict(rows=-1), "INVALID_ARG"), (dict(rows=(1 << 23) + 1), "INVALID_ARG"),
    (dict(stride=99), "INVALID_ARG"), (dict(draft_stride=99), "INVALID_ARG"), (dict(batch=-1), "INVALID_ARG"),
    (dict(batch=0), "INVALID_ARG"), (dict(logits=None), "INVALID_ARG"), (dict(ids=None), "INVALID_ARG"),
    (dict(q_start=None), "INVALID_ARG"), (dict(u=None), "INVALID_ARG"), (dict(u_draw=None), "INVALID_ARG"),
    (dict(token=None), "INVALID_ARG"), (dict(accepted=None), "INVALID_ARG"), (dict(logits=P + 1), "MISALIGNED"),
    (dict(draft=P + 1), "MISALIGNED"), (dict(u=P + 2), "MISALIGNED"), (dict(k=P + 2), "MISALIGNED"), (dict(prob=P + 1), "MISALIGNED"),
    (dict(ws=None), "WORKSPACE"), (dict(n=64), "WORKSPACE"), (dict(ws=P + 8), "MISALIGNED")])
def test_arguments_are_checked(lib, kw, code):
    import group_wise_affine_gb300 as gwa
    assert lib.gwa_verify_draft(*{**ARGS, **kw}.values()) == getattr(gwa, "GWA_ERR_" + code)
    assert gwa.last_error()


def test_nothing_to_do_and_workspaces(lib):
    assert lib.gwa_verify_draft(*{**ARGS, "rows": 0, "batch": 0}.values()) == 0
    f = lib.gwa_verify_draft_workspace_bytes
    assert f(0) == 0 and f(5) >= 5 * 2 * 32 and f(-1) == 0 and f((1 << 23) + 1) == 0


def test_binding_refuses_mismatched_tensors():
    import torch

    import group_wise_affine_gb300 as gwa
    z = lambda *s, t=torch.float32: torch.zeros(s, dtype=t)  # noqa: E731
    i = torch.int32
    with pytest.raises(ValueError):
        gwa.verify_draft(z(3, 10, t=torch.float16), z(3, t=i), z(2, t=i), z(3), z(1))
    with pytest.raises(ValueError):
        gwa.verify_draft(z(3, 10), z(3, t=i), z(2, t=i), z(3), z(1), draft_logits=z(3, 9))
    with pytest.raises(ValueError):
        gwa.verify_draft(z(3, 10), z(3, t=i), z(2, t=i), z(3), z(1), draft_logits=z(3, 10, t=torch.bfloat16))
