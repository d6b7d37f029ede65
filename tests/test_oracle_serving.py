"""The plain implementations of the serving operators (oracle/serving.py)
pinned to independent statements of the same definitions, and the refusals of
their C entry points, all without a GPU."""
import ctypes

import numpy as np
import pytest

from oracle import serving

RNG = np.random.default_rng


def test_bf16_rounds_to_nearest_even():
    x = np.array([1.0, 1.0 + 2.0 ** -8, 1.0 + 3 * 2.0 ** -8, 1.0 + 2.0 ** -8 + 2.0 ** -20, -2.5],
                 np.float32)
    got = serving.bf16_value(serving.bf16_round(x))
    assert got.tolist() == [1.0, 1.0, 1.0 + 2.0 ** -6, 1.0 + 2.0 ** -7, -2.5]


@pytest.mark.parametrize("bits", [4, 8])
def test_quantized_values_are_within_half_a_step(bits):
    x = serving.bf16_round(RNG(bits).standard_normal((5, 3, 128)).astype(np.float32))
    code, par = serving.quantize(x, bits)
    assert code.min() >= 0 and code.max() <= 2 ** bits - 1
    got = serving.values(serving.pack(code, bits), par, bits)
    v = serving.bf16_value(x).astype(np.float64)
    step = np.repeat(serving.bf16_value(par[..., 0]), 64, axis=-1).astype(np.float64)
    # half a step, and what the scale's rounding to bf16 takes from the top
    assert (np.abs(got - v) <= step * (0.5 + (2 ** bits - 1) * 2.0 ** -8)).all()


@pytest.mark.parametrize("rot", [16, 64, 128])
def test_rotation_turns_pairs_by_the_position(rot):
    D, base = 128, 1e4
    x = serving.bf16_round(RNG(rot).standard_normal((4, 2, D)).astype(np.float32))
    pos = np.array([0, 1, 7, 200])
    got = serving.bf16_value(serving.rotate(x, serving.rope_table(256, rot, base), pos))
    v = serving.bf16_value(x).astype(np.float64)
    want = v.copy()
    for t in range(4):
        for i in range(rot // 2):
            a = pos[t] * base ** (-2 * i / rot)
            z = (v[t, :, i] + 1j * v[t, :, i + rot // 2]) * np.exp(1j * a)
            want[t, :, i], want[t, :, i + rot // 2] = z.real, z.imag
    assert np.abs(got - want).max() <= 2.0 ** -8 * np.abs(v).max() * 2
    assert (got[0] == v[0]).all() and (got[..., rot:] == v[..., rot:]).all()


@pytest.mark.parametrize("causal", [True, False])
def test_attention_against_one_row_at_a_time(causal):
    rng = RNG(3)
    lens = [(1, 5), (0, 3), (4, 4), (2, 0), (3, 9)]  # (new tokens, cache length)
    q_start = np.concatenate([[0], np.cumsum([a for a, _ in lens])])
    kl = np.array([b for _, b in lens])
    q = rng.standard_normal((q_start[-1], 4, 8))
    k = [rng.standard_normal((n, 2, 8)) for n in kl]
    v = [rng.standard_normal((n, 2, 8)) for n in kl]
    got = serving.attention(q, k, v, q_start, kl, 0.3, causal)
    for b, (n, length) in enumerate(lens):
        for i in range(n):
            pos = length - n + i
            see = min(length, pos + 1) if causal else length
            for h in range(4):
                want = np.zeros(8)
                if see > 0:
                    s = np.array([0.3 * (q[q_start[b] + i, h] * k[b][t, h // 2]).sum()
                                  for t in range(see)])
                    p = np.exp(s - s.max())
                    want = (p[:, None] * v[b][:see, h // 2]).sum(0) / p.sum()
                assert np.allclose(got[q_start[b] + i, h], want, atol=1e-12)


def test_sampling_order_and_masses():
    x = np.array([0.5, 2.0, -np.inf, 2.0, 1.0])
    assert serving.sample_order(x).tolist()[:4] == [1, 3, 4, 0]
    w = serving.sample_masses(x, 0.5)
    assert np.allclose(w / w.max(), np.exp((x - 2.0) / 0.5)) and w[2] == 0


@pytest.fixture(scope="module")
def lib():
    import group_wise_affine_gb300 as gwa
    gwa.build()
    return gwa.load()


def cache(gwa, **kw):
    a = dict(kq=1 << 20, kp=1 << 20, vq=1 << 20, vp=1 << 20, num_pages=4, heads=2, head_dim=128,
             page_size=16, bits=4, group=64)
    a.update(kw)
    return gwa._KVCache(**a)


def batch(gwa, **kw):
    a = dict(q_start=1 << 20, kv_len=1 << 20, page_table=1 << 20, batch=1, max_pages=4, tokens=3,
             max_q=3, max_kv=10)
    a.update(kw)
    return gwa._KVBatch(**a)


BAD = [("head_dim", 96, "UNSUPPORTED"), ("bits", 3, "UNSUPPORTED"), ("group", 32, "UNSUPPORTED"),
       ("page_size", 24, "UNSUPPORTED"), ("page_size", 8192, "UNSUPPORTED"),
       ("heads", 0, "INVALID_ARG"), ("kq", 0, "INVALID_ARG"), ("vp", (1 << 20) + 4, "MISALIGNED")]
BAD_BATCH = [("q_start", 0, "INVALID_ARG"), ("tokens", -1, "INVALID_ARG"),
             ("kv_len", (1 << 20) + 2, "MISALIGNED"), ("max_pages", -1, "INVALID_ARG")]


@pytest.mark.parametrize("field,value,code", BAD + BAD_BATCH)
def test_cache_and_batch_are_checked(lib, field, value, code):
    import group_wise_affine_gb300 as gwa
    want = getattr(gwa, "GWA_ERR_" + code)
    c = cache(gwa, **({field: value} if (field, value, code) in BAD else {}))
    b = batch(gwa, **({field: value} if (field, value, code) in BAD_BATCH else {}))
    p = ctypes.c_void_p(1 << 20)
    assert lib.gwa_kv_append(None, 0, None, 0, p, 256, p, 256, c, b, None, 0, 0, None, None) == want
    assert lib.gwa_kv_read(c, b, p, p, None, None) == want
    assert lib.gwa_sdpa_paged(p, 512, 4, c, b, 0.1, 1, p, p, 1 << 30, None, None) == want
    assert gwa.last_error()


def test_append_attend_and_sample_arguments_are_checked(lib):
    import group_wise_affine_gb300 as gwa
    c, b, p, odd = cache(gwa), batch(gwa), ctypes.c_void_p(1 << 20), ctypes.c_void_p((1 << 20) + 2)
    invalid, misaligned = gwa.GWA_ERR_INVALID_ARG, gwa.GWA_ERR_MISALIGNED

    def append(q=None, qs=0, qo=None, Hq=0, k=p, ks=256, v=p, vs=256, rope=None, rows=0, rot=0):
        return lib.gwa_kv_append(q, qs, qo, Hq, k, ks, v, vs, c, b, rope, rows, rot, None, None)

    assert append(k=None) == invalid and append(k=odd) == misaligned
    assert append(ks=252) in (invalid, misaligned) and append(vs=128) == invalid
    assert append(rope=p, rows=10, rot=24) == gwa.GWA_ERR_UNSUPPORTED
    assert append(rope=None, rows=10, rot=64) == invalid
    assert append(q=p, qs=512, qo=None, Hq=4) == invalid

    def attend(q=p, qs=512, Hq=4, scale=0.1, out=p, ws=p, size=1 << 30):
        return lib.gwa_sdpa_paged(q, qs, Hq, c, b, scale, 1, out, ws, size, None, None)

    assert attend(Hq=3) == invalid and attend(scale=float("inf")) == invalid
    assert attend(q=odd) == misaligned and attend(out=None) == invalid
    assert attend(size=16) == gwa.GWA_ERR_WORKSPACE

    def draw(x=p, dtype=0, rows=2, V=100, stride=100, u=p, token=p):
        return lib.gwa_sample(x, dtype, rows, V, stride, u, None, None, None, None, token, None,
                              None)

    assert draw(dtype=2) == gwa.GWA_ERR_UNSUPPORTED and draw(V=524289, stride=1 << 20) == \
        gwa.GWA_ERR_UNSUPPORTED
    assert draw(V=0) == invalid and draw(stride=99) == invalid and draw(u=None) == invalid
    assert draw(x=ctypes.c_void_p((1 << 20) + 1)) == misaligned
    assert draw(rows=0) == 0


def test_a_wide_page_table_beside_a_prompt_is_not_refused(lib):
    # 128 sequences, one chunk of 2048 tokens among them, tables for 131072
    # positions; and what passes the documented count of work
    import group_wise_affine_gb300 as gwa
    c, p = cache(gwa, heads=8, page_size=64), ctypes.c_void_p(1 << 20)
    b = batch(gwa, batch=128, max_pages=2048, tokens=2175, max_q=2048, max_kv=131072)
    assert lib.gwa_sdpa_paged_workspace_bytes(40, c, b) > 16
    assert lib.gwa_sdpa_paged(p, 5120, 40, c, b, 0.1, 1, p, p, 16, None, None) == \
        gwa.GWA_ERR_WORKSPACE
    for kw in (dict(batch=1 << 20, tokens=1 << 20, max_q=1), dict(tokens=1 << 30, max_q=1 << 25)):
        b = batch(gwa, **{**dict(batch=64, max_pages=1 << 16, max_kv=1 << 22), **kw})
        assert lib.gwa_sdpa_paged_workspace_bytes(40, c, b) == 0
        assert lib.gwa_sdpa_paged(p, 5120, 40, c, b, 0.1, 1, p, p, 1 << 40, None, None) == \
            gwa.GWA_ERR_UNSUPPORTED
        assert "units of work" in gwa.last_error()


@pytest.mark.parametrize("dim,bits,rep", [(64, 4, 1), (128, 8, 5), (256, 4, 3), (256, 8, 16)])
def test_batches_within_the_documented_count_of_work_pass(lib, dim, bits, rep):
    import group_wise_affine_gb300 as gwa
    rng = RNG(dim + rep)
    seen = set()
    for _ in range(3000):
        B, H = int(2 ** rng.uniform(0, 17)), int(2 ** rng.uniform(0, 7))
        T, mp = int(2 ** rng.uniform(0, 30)), int(2 ** rng.uniform(0, 24))
        mq = max(1, min(T, int(2 ** rng.uniform(0, 22))))
        c = cache(gwa, heads=H, head_dim=dim, bits=bits, page_size=64)
        b = batch(gwa, batch=B, max_pages=mp, tokens=T, max_q=mq, max_kv=1 << 20)
        n = H * (B + T * rep / 256) * (mp * 64 / 128 + 5) * (4 if dim == 256 else 1)
        ok = lib.gwa_sdpa_paged_workspace_bytes(H * rep, c, b) > 0
        assert ok or n >= 2e9, (B, H, T, mp, mq)
        seen.add(ok)
    assert seen == {True, False}


def test_a_workspace_for_what_is_refused_is_an_error(lib):
    from types import SimpleNamespace as S

    import group_wise_affine_gb300 as gwa
    dev = dict(device="cpu")
    good = gwa.make_sdpa_paged_workspace(S(c=cache(gwa), **dev), S(c=batch(gwa)), 4)
    assert good.numel() == lib.gwa_sdpa_paged_workspace_bytes(4, cache(gwa), batch(gwa)) > 0
    for c, b, Hq in ((cache(gwa), batch(gwa), 3), (cache(gwa, bits=3), batch(gwa), 4),
                     (cache(gwa), batch(gwa, tokens=-1), 4)):
        with pytest.raises(gwa.GwaError, match="gwa_sdpa_paged_workspace_bytes"):
            gwa.make_sdpa_paged_workspace(S(c=c, **dev), S(c=b), Hq)


def test_a_batch_and_what_the_library_is_told_of_it_stay_the_same(monkeypatch):
    import torch

    import group_wise_affine_gb300 as gwa
    monkeypatch.setattr(gwa, "_ptr", lambda t: t.data_ptr())
    i = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    b = gwa.KVBatch(i(3), i(2), i(2, 4), tokens=9, max_q=5, max_kv=40)
    for name, value in (("tokens", 4), ("max_q", 2), ("max_kv", 64)):
        setattr(b, name, value)
        assert getattr(b, name) == getattr(b.c, name) == value
    c = gwa.KVCache.empty(2, 1, 16, 64, device="cpu")
    for obj, name, value in ((b, "kv_len", i(2)), (b, "q_start", i(3)), (b, "page_table", i(2, 9)),
                             (c, "kq", c.kq.clone()), (c, "heads", 2), (c, "dim", 128)):
        was = getattr(obj, name)
        with pytest.raises(AttributeError):
            setattr(obj, name, value)
        assert getattr(obj, name) is was
