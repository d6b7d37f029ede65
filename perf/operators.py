"""Measured cases of the serving operators: a token's way through the cache.

Three operators, each in two forms.  ``kv_append`` rotates the new tokens' queries and keys, quantizes keys and values
and writes them into a paged cache (``kv_read`` gives back the values that the cache then stands for); ``sdpa_paged`` is
softmax attention over that cache; ``sample`` draws one token a row from logits under temperature, top-k, top-p and
min-p.  With ``own`` false, ``run`` computes them from elementary torch operations in 32 bits, rounded once at the end;
with ``own`` true it calls the library.
"""
import math

import numpy as np
import torch

own = False

GROUP = 64            # head dimensions that share one scale and one bias
MASS = float(2 ** 40)  # a token's probability mass is counted in units of 2^-40 of the likeliest token's


# ------------------------------------------------------------------ cases

def _append(name, **k):
    return {"name": name, "kind": "append", "Hq": 40, "Hkv": 8, "D": 128, "bits": 4, "page": 64, "rot": 128, "strided": True,
            "mix": 1, **k}


def _attend(name, **k):
    return {"name": name, "kind": "attend", "Hq": 40, "Hkv": 8, "D": 128, "bits": 4, "page": 64, "causal": True, "mix": 1, **k}


def _sample(name, **k):
    return {"name": name, "kind": "sample", "mix": 1, **k}


def listed():
    return [
        # one token of one conversation: launch and latency are all there is
        _append("append, one token", B=1, q=1, kv=4097),
        # a decode step of a server: 64 sequences of many lengths, one token each, small pages
        _append("append, 64 sequences", B=64, q=1, kv=8192, page=16),
        # a long prompt written in one go
        _append("append, prompt of 8192", B=1, q=8192, kv=8192),
        # ragged prompts on wide heads, of which a quarter is rotated, into an 8-bit cache
        _append("append, ragged wide u8", B=3, q=1501, kv=4099, Hq=16, Hkv=2, D=256, bits=8, rot=64, page=32, strided=False),
        # one conversation, one new token, a cache of ordinary length
        _attend("attend, 1 x 4096", B=1, q=1, kv=4096),
        # one conversation at the longest context that the benchmark of this repository runs, ending inside a page
        _attend("attend, 1 x 131071", B=1, q=1, kv=131071),
        # a decode step of a server over sequences of many lengths, some of them empty
        _attend("attend, 64 ragged", B=64, q=1, kv=8192, Hq=32, page=16),
        # drafted tokens checked in one pass, 8-bit cache, narrow heads
        _attend("attend, 16 x 4 drafted u8", B=16, q=4, kv=3001, Hq=16, Hkv=4, D=64, bits=8, page=32),
        # a chunk of a long prompt: the cache holds what came before
        _attend("attend, chunk 2048 of 8192", B=1, q=2048, kv=8192),
        # ragged prompts on wide heads
        _attend("attend, ragged prompts wide", B=3, q=1100, kv=1733, Hq=16, Hkv=2, D=256, page=16),
        # one conversation's next token, every filter on
        _sample("sample, 1 x 131072 fp32", rows=1, V=131072, type="fp32", filters="all"),
        # a server's step: every row with filters of its own, some greedy, bf16 logits, odd vocabulary
        _sample("sample, 256 x 151669 bf16", rows=256, V=151669, type="bf16", filters="mixed"),
    ]


def _log(rng, lo, hi):
    """A whole number, spread evenly over its logarithm."""
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["append", "attend", "attend", "sample"])
    if kind == "sample":
        V = _log(rng, 300, 150000) | rng.randint(0, 1)
        rows = min(256, _log(rng, 1, 300))
        return {"kind": kind, "rows": rows, "V": V, "type": rng.choice(["fp32", "bf16"]) if rows * V < 19e6 else "bf16",
                "filters": rng.choice(["all", "top_p", "top_k", "none", "mixed"]), "mix": rng.randint(1, 1 << 20)}
    Hkv = rng.choice([1, 2, 4, 8])
    rep = rng.choice([1, 2, 3, 4, 5, 6, 7, 8])
    D = rng.choice([64, 128, 128, 256])
    c = {"kind": kind, "Hq": Hkv * rep, "Hkv": Hkv, "D": D, "bits": rng.choice([4, 4, 8]), "page": rng.choice([16, 32, 64, 128]),
         "mix": rng.randint(1, 1 << 20)}
    if kind == "append":
        c["B"] = _log(rng, 1, 64)
        c["q"] = max(1, min(_log(rng, 1, 8192), 8192 // c["B"]))
        c["kv"] = c["q"] + _log(rng, 1, 4096)
        c["rot"] = rng.choice([D, D, D // 2, D // 4, 0])
        c["strided"] = rng.choice([True, False])
        return c
    c["causal"] = rng.choice([True, True, False])
    if rng.random() < 0.6:      # decode: a few tokens a sequence
        c["B"] = _log(rng, 1, 64)
        c["q"] = rng.choice([1, 1, 1, 2, 4, 5, 8])
        c["kv"] = max(c["q"], min(_log(rng, 16, 131072), 524288 // c["B"] * 128 // D))
    else:                       # prompts and chunks of them
        c["B"] = rng.choice([1, 1, 2, 3, 4])
        c["q"] = max(9, min(_log(rng, 9, 1700), 1700 // c["B"] * 128 // D * 5 // max(5, rep)))
        c["kv"] = c["q"] + rng.choice([0, _log(rng, 1, 6144 // c["B"])])
    return c


def _lens(c):
    """New tokens and cache lengths (new tokens included) of each sequence: the first as the case says, the others spread below it; from the sixth
    sequence on, every sixth has no tokens at all."""
    B, q, kv = c["B"], c["q"], c["kv"]
    r = np.random.RandomState(c["mix"])
    ql = np.concatenate([[q], r.randint(max(1, q // 2), q + 1, B - 1)]).astype(np.int64)
    kl = np.maximum(np.concatenate([[kv], r.randint(1, kv + 1, B - 1)]), ql).astype(np.int64)
    empty = np.arange(B) % 6 == 5
    return np.where(empty, 0, ql), np.where(empty, 0, kl)


# ------------------------------------------------------------------ inputs

def _randn(g, *shape):
    return torch.randn(shape, device="cuda", generator=g)


def _quantize(x, bits):
    """bf16 values in groups of 64 of the last axis: codes (whole numbers in fp32), scale and bias."""
    x = x.reshape(*x.shape[:-1], -1, GROUP)
    lo = x.amin(-1, keepdim=True) + 0.0
    s = ((x.amax(-1, keepdim=True) - lo) / float(2 ** bits - 1)).bfloat16().float()
    code = torch.where(s == 0, torch.zeros_like(x), torch.round((x - lo) / s)).clamp(0, 2 ** bits - 1)
    return code.flatten(-2), torch.stack([s[..., 0], lo[..., 0]], -1).bfloat16()


def _pack(code, bits):
    per = 32 // bits
    shift = torch.arange(per, device=code.device, dtype=torch.int64) * bits
    w = (code.to(torch.int64).reshape(*code.shape[:-1], -1, per) << shift).sum(-1)
    return torch.where(w >= 2 ** 31, w - 2 ** 32, w).to(torch.int32)


def _values(words, par, bits):
    """The fp32 values that packed words and their (scale, bias) pairs stand for."""
    shift = torch.arange(32 // bits, device=words.device, dtype=torch.int32) * bits
    code = ((words[..., None] >> shift) & (2 ** bits - 1)).flatten(-2).float()
    code = code.reshape(*code.shape[:-1], -1, GROUP)
    par = par.float()
    return (code * par[..., 0:1] + par[..., 1:2]).flatten(-2)


def _cache(c, g, filled):
    """A paged cache whose pages lie in no order; filled with keys and values of ordinary size, a few key channels of them large, as rotated keys have."""
    ql, kl = _lens(c)
    need = np.maximum(1, -(-kl // c["page"]))
    pages = int(need.sum()) + 3
    perm = torch.randperm(pages, device="cuda", generator=g).to(torch.int32)
    table = torch.full((c["B"], int(need.max())), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(need.tolist()):
        table[b, :n] = perm[at:at + n]
        at += n
    shape = (pages, c["Hkv"], c["page"])
    D, bits = c["D"], c["bits"]
    s = {"table": table, "kv_len": torch.from_numpy(kl.astype(np.int32)).cuda(),
         "q_start": torch.from_numpy(np.concatenate([[0], np.cumsum(ql)]).astype(np.int32)).cuda()}
    for n in ("k", "v"):
        if filled:
            size = torch.ones(D, device="cuda")
            if n == "k":
                size[torch.randperm(D, device="cuda", generator=g)[:D // 16]] = 4.0
            words = torch.empty(*shape, D * bits // 32, dtype=torch.int32, device="cuda")
            par = torch.empty(*shape, D // GROUP, 2, dtype=torch.bfloat16, device="cuda")
            step = max(1, (1 << 25) // (c["Hkv"] * c["page"] * D))
            for i in range(0, pages, step):
                n_i = min(step, pages - i)
                code, p = _quantize((_randn(g, n_i, *shape[1:], D) * size).bfloat16().float(), bits)
                words[i:i + n_i], par[i:i + n_i] = _pack(code, bits), p
        else:
            words = torch.zeros(*shape, D * bits // 32, dtype=torch.int32, device="cuda")
            par = torch.zeros(*shape, D // GROUP, 2, dtype=torch.bfloat16, device="cuda")
        s[n + "q"], s[n + "p"] = words, par
    return s


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    if c["kind"] == "sample":
        return _prepare_sample(c, g)
    ql, kl = _lens(c)
    T, D = int(ql.sum()), c["D"]
    s = _cache(c, g, c["kind"] == "attend")
    s.update(case=c, T=T, scale=1.0 / math.sqrt(D))
    if c["kind"] == "append":
        n = (c["Hq"], c["Hkv"], c["Hkv"])
        x = _randn(g, T, sum(n), D).bfloat16()
        parts = list(x.split(n, dim=1))         # views of one fused projection's rows
        s["q"], s["k"], s["v"] = parts if c["strided"] else [t.contiguous() for t in parts]
        r = c["rot"]
        angle = torch.arange(int(kl.max()), device="cuda", dtype=torch.float64)[:, None] * 1e6 ** (
            -torch.arange(0, r, 2, device="cuda", dtype=torch.float64) / max(1, r))
        s["rope"] = torch.stack([angle.cos(), angle.sin()], -1).float() if r else None
    else:
        s["q"] = (_randn(g, T, c["Hq"], D) * 0.7).bfloat16()
    # token i of the batch: its sequence and its place in it (the plain form's plan)
    seq = np.repeat(np.arange(c["B"]), ql)
    first = np.concatenate([[0], np.cumsum(ql)])[:-1]
    pos = np.arange(T) - first[seq] + (kl - ql)[seq]
    s["seq"], s["pos"] = torch.from_numpy(seq).cuda(), torch.from_numpy(pos).cuda()
    s["row"] = torch.from_numpy(np.arange(T) - first[seq]).cuda()
    s["max_q"], s["max_kv"] = int(ql.max()), int(kl.max())
    if own:                                     # the handles that a program keeps beside its cache
        import group_wise_affine_gb300 as gwa
        s["cache"] = gwa.KVCache(s["kq"], s["kp"], s["vq"], s["vp"], bits=c["bits"])
        s["batch"] = gwa.KVBatch(s["q_start"], s["kv_len"], s["table"], tokens=T, max_q=s["max_q"], max_kv=s["max_kv"])
        if c["kind"] == "attend":
            s["workspace"] = gwa.make_sdpa_paged_workspace(s["cache"], s["batch"], c["Hq"])
    return s


def _prepare_sample(c, g):
    R, V = c["rows"], c["V"]
    x = _randn(g, R, V) * 2.0
    likely = torch.randint(0, V, (R, 24), device="cuda", generator=g)
    x.scatter_add_(1, likely, torch.rand((R, 24), device="cuda", generator=g) * 8.0 + 3.0)
    x[:, V - V // 50:] = -math.inf              # padding of the vocabulary
    u = lambda lo, hi: torch.rand(R, device="cuda", generator=g) * (hi - lo) + lo  # noqa: E731
    f = c["filters"]
    on = lambda name, t, off: torch.full_like(t, off) if f not in (name, "all", "mixed") else (  # noqa: E731
        torch.where(torch.rand(R, device="cuda", generator=g) < 0.4, torch.full_like(t, off), t) if f == "mixed" else t)
    s = {"case": c, "logits": x.bfloat16() if c["type"] == "bf16" else x,
         "top_k": on("top_k", torch.randint(1, 200, (R,), device="cuda", generator=g, dtype=torch.int32), 0),
         "top_p": on("top_p", u(0.5, 0.99), 1.0), "min_p": on("min_p", u(0.0, 0.1), 0.0), "u": u(0.0, 1.0)}
    t = u(0.6, 1.3)
    s["temperature"] = torch.where(torch.arange(R, device="cuda") % 8 == 7, torch.zeros_like(t), t) if f == "mixed" else t
    return s


# ------------------------------------------------------------------ one pass

def run(state):
    return {"append": _run_append, "attend": _run_attend, "sample": _run_sample}[state["case"]["kind"]](state)


def _run_append(s):
    if own:
        import group_wise_affine_gb300 as gwa
        q = gwa.kv_append(s["k"], s["v"], s["cache"], s["batch"], q=s["q"], rope=s["rope"])
        k, v = gwa.kv_read(s["cache"], s["batch"])
        return {"q": q, "k": k, "v": v}
    c = s["case"]
    q, k = _rotate(s["q"], s), _rotate(s["k"], s)
    page = s["table"][s["seq"], s["pos"] // c["page"]].long()
    slot = s["pos"] % c["page"]
    out = {"q": q}
    for n, x in (("k", k), ("v", s["v"])):
        code, par = _quantize(x.float(), c["bits"])
        s[n + "q"][page, :, slot] = _pack(code, c["bits"])
        s[n + "p"][page, :, slot] = par
        out[n] = _values(s[n + "q"][page, :, slot], s[n + "p"][page, :, slot], c["bits"]).bfloat16()
    return out


def _rotate(x, s):
    r = s["case"]["rot"]
    if not r:
        return x.contiguous()
    x = x.float()
    cs = s["rope"][s["pos"]]
    cos, sin = cs[:, None, :, 0], cs[:, None, :, 1]
    a, b = x[..., :r // 2], x[..., r // 2:r]
    return torch.cat([a * cos - b * sin, b * cos + a * sin, x[..., r:]], -1).bfloat16()


def _run_attend(s):
    c = s["case"]
    if own:
        import group_wise_affine_gb300 as gwa
        return gwa.sdpa_paged(s["q"], s["cache"], s["batch"], scale=s["scale"], causal=c["causal"], workspace=s["workspace"])
    B, Hq, Hkv, D, n, m = c["B"], c["Hq"], c["Hkv"], c["D"], s["max_q"], s["max_kv"]
    at = torch.arange(m, device="cuda")
    page = s["table"][:, at // c["page"]].long().clamp(min=0)
    k = _values(s["kq"][page, :, at % c["page"]], s["kp"][page, :, at % c["page"]], c["bits"]).permute(0, 2, 3, 1)
    v = _values(s["vq"][page, :, at % c["page"]], s["vp"][page, :, at % c["page"]], c["bits"]).permute(0, 2, 1, 3)
    q = torch.zeros((B, n, Hq, D), device="cuda")
    q[s["seq"], s["row"]] = s["q"].float()
    q = q.reshape(B, n, Hkv, Hq // Hkv, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, -1, D)
    x = (torch.matmul(q, k) * s["scale"]).reshape(B, Hkv, Hq // Hkv, n, m)
    length = s["kv_len"].long()
    last = length[:, None] - 1
    if c["causal"]:
        last = last - (s["q_start"].diff().long()[:, None] - 1 - torch.arange(n, device="cuda"))
    x = x.masked_fill(at > last[:, None, None, :, None], -math.inf)
    x = torch.exp(x - x.amax(-1, keepdim=True).clamp(min=-3e38))
    p = x / x.sum(-1, keepdim=True).clamp(min=1e-30)
    o = torch.matmul(p.reshape(B, Hkv, -1, m), v).reshape(B, Hkv, Hq // Hkv, n, D).permute(0, 3, 1, 2, 4).reshape(B, n, Hq, D)
    return o[s["seq"], s["row"]].bfloat16()


def _run_sample(s):
    if own:
        import group_wise_affine_gb300 as gwa
        token, prob = gwa.sample(s["logits"], s["u"], temperature=s["temperature"], top_k=s["top_k"], top_p=s["top_p"], min_p=s["min_p"])
        return {"token": token, "prob": prob}
    x = s["logits"].float()
    x = x.masked_fill(x != x, -math.inf)
    R, V = x.shape
    top = x.amax(-1, keepdim=True)
    per = (1.0 / s["temperature"][:, None]) * 1.4426950408889634
    w = (torch.exp2(((x - top) * per).masked_fill(x == top, 0.0)) * MASS).to(torch.int64)
    order = torch.sort(x, dim=-1, descending=True, stable=True)[1]
    ws = w.gather(1, order)
    rank = torch.arange(V, device="cuda")
    k = s["top_k"][:, None]
    keep = (rank < k) | (k <= 0)
    ws = ws * keep
    cum = ws.cumsum(-1)
    p = s["top_p"][:, None]
    goal = (cum[:, -1:].double() * p.double()).to(torch.int64)
    keep = keep & ((cum - ws < goal) | (rank == 0) | (p >= 1.0))
    keep = keep & (ws >= (s["min_p"][:, None] * MASS).to(torch.int64))
    w = w * torch.zeros_like(keep).scatter_(1, order, keep)
    cum = w.cumsum(-1)
    all_ = cum[:, -1:]
    at = torch.minimum((s["u"][:, None].double() * all_.double()).to(torch.int64), all_ - 1)
    token = torch.searchsorted(cum, at, right=True)
    prob = w.gather(1, token.clamp(max=V - 1)).double() / all_.double()
    greedy = s["temperature"][:, None] <= 0
    token = torch.where(greedy, torch.where(x == top, rank, V).amin(-1, keepdim=True), token)
    none = top == -math.inf
    prob = torch.where(none, 0.0, torch.where(greedy, 1.0, prob))
    return {"token": torch.where(none, -1, token)[:, 0].to(torch.int32), "prob": prob[:, 0].float()}


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    c = case
    if c["kind"] == "sample":
        n = c["rows"] * c["V"]
        return {"bytes": n * (4 if c["type"] == "fp32" else 2) + c["rows"] * 28, "flops": 4 * n}
    ql, kl = _lens(c)
    T, D = int(ql.sum()), c["D"]
    token = 2 * c["Hkv"] * (D * c["bits"] // 8 + D // GROUP * 4)    # a token's codes, scales and biases, keys and values
    tables = 4 * (2 * c["B"] + 1 + int((-(-kl // c["page"])).sum()))
    if c["kind"] == "append":
        return {"bytes": T * ((c["Hq"] * 2 + c["Hkv"] * 4) * D * 2 + token + c["rot"] * 4) + tables,
                "flops": T * ((c["Hq"] + c["Hkv"]) * c["rot"] * 3 + c["Hkv"] * 2 * D * 6)}
    pairs = int((ql * kl - (ql * (ql - 1) // 2 if c["causal"] else 0)).sum())
    return {"bytes": int(kl.sum()) * token + T * c["Hq"] * D * 4 + tables, "flops": pairs * c["Hq"] * D * 4}


# ------------------------------------------------------------------ the definitions in 64 bits

def exact(case, seed):
    c = case
    s = prepare(c, seed)
    if c["kind"] == "sample":
        return _exact_sample(s)
    return _exact_append(s) if c["kind"] == "append" else _exact_attend(s)


def _bf16(x):
    return x.to(torch.bfloat16).double()


def _exact_append(s):
    c, (ql, kl) = s["case"], _lens(s["case"])
    r, D, top = c["rot"], c["D"], 2.0 ** c["bits"] - 1
    out = {"q": s["q"].double(), "k": s["k"].double(), "v": s["v"].double()}
    if r:
        turn = torch.view_as_complex(s["rope"][s["pos"]].double())[:, None]
        for n in ("q", "k"):
            z = torch.complex(out[n][..., :r // 2], out[n][..., r // 2:r]) * turn
            out[n] = torch.cat([z.real, z.imag, out[n][..., r:]], -1)
    for n in ("k", "v"):
        x = _bf16(out[n]).reshape(-1, D // GROUP, GROUP)
        lo, hi = x.min(-1).values[..., None], x.max(-1).values[..., None]
        step = _bf16((hi - lo) / top)
        code = torch.where(step > 0, ((x - lo) / step).round(), torch.zeros_like(x)).clamp(max=top)
        out[n] = (lo + code * step).reshape(out[n].shape)
    return out


def _exact_attend(s):
    c, (ql, kl) = s["case"], _lens(s["case"])
    D, rep, page, bits = c["D"], c["Hq"] // c["Hkv"], c["page"], c["bits"]
    out = torch.zeros((s["T"], c["Hq"], D), dtype=torch.float64, device="cuda")
    mask = (1 << bits) - 1
    start = 0
    for b in range(c["B"]):
        n, m = int(ql[b]), int(kl[b])
        if not n:
            continue
        ids = s["table"][b, :-(-m // page)].long()
        for h in range(c["Hkv"]):
            kv = []
            for w in ("k", "v"):
                words = s[w + "q"][ids, h].reshape(-1, D * bits // 32)[:m].to(torch.int64)
                par = s[w + "p"][ids, h].reshape(-1, D // GROUP, 2)[:m].double().repeat_interleave(GROUP, 1)
                code = torch.stack([(words >> i) & mask for i in range(0, 32, bits)], -1).reshape(m, D).double()
                kv.append(code * par[..., 0] + par[..., 1])
            q = s["q"][start:start + n, h * rep:(h + 1) * rep].double()
            x = torch.einsum("ihd,jd->hij", q, kv[0]) * s["scale"]
            if c["causal"]:
                j = torch.arange(m, device="cuda")
                x = x.masked_fill(j > m - n + torch.arange(n, device="cuda")[:, None], -math.inf)
            out[start:start + n, h * rep:(h + 1) * rep] = torch.einsum("hij,jd->ihd", torch.softmax(x, -1), kv[1])
        start += n
    return out


def _exact_sample(s):
    x = s["logits"].double()
    prob = torch.zeros(x.shape[0], dtype=torch.float64, device="cuda")
    for i in range(x.shape[0]):
        t = float(s["temperature"][i])
        if t <= 0:
            prob[i] = 1.0
            continue
        e = torch.exp((x[i] - x[i].max()) / t)
        order = torch.sort(x[i], descending=True, stable=True)[1]
        n = int(s["top_k"][i]) or len(order)
        e_o = e[order[:n]]
        if float(s["top_p"][i]) < 1:
            before = e_o.cumsum(0) - e_o
            n = max(1, int((before < float(s["top_p"][i]) * e_o.sum()).sum()))
            e_o = e_o[:n]
        n = int((e_o >= float(s["min_p"][i])).sum())
        kept = torch.sort(order[:n])[0]
        cum = e[kept].cumsum(0)
        at = min(int((cum <= float(s["u"][i]) * cum[-1]).sum()), n - 1)
        prob[i] = e[kept[at]] / cum[-1]
    return {"token": None, "prob": prob}
