"""Measured cases of three further serving operators: what a step of many conversations needs beside the shared weights.

``lora_add`` and ``lora_gate_up_silu`` add each token's own low-rank adapter to a shared projection's output;
``sdpa_paged`` with a window is attention over the paged cache where a token sees the last keys and a few first ones;
``verify_draft`` settles which drafted tokens stand against the target's probabilities, and draws the token after them.
With ``own`` false, ``run`` computes them from elementary torch operations in 32 bits, rounded once at the end (the
shares of probability in 64); with ``own`` true it calls the library.
"""
import math

import numpy as np
import torch

own = False

GROUP = 64            # head dimensions that share one scale and one bias
MASS = float(2 ** 40)  # a token's probability mass is counted in units of 2^-40 of the likeliest token's


# ------------------------------------------------------------------ cases

def _lora(name, **k):
    return {"name": name, "kind": "lora", "K": 5120, "sections": "5120,1024,1024", "silu": False, "rank": 16, "mixed": False,
            "adapters": 8, "mix": 1, **k}


def _window(name, **k):
    return {"name": name, "kind": "window", "Hq": 40, "Hkv": 8, "D": 128, "bits": 4, "page": 64, "mix": 1, **k}


def _verify(name, **k):
    return {"name": name, "kind": "verify", "draft": True, "mix": 1, **k}


def listed():
    return [
        # one conversation's next token through the fused query, key and value projection: launches and latency
        _lora("adapters, one token", B=1, q=1),
        # a decode step: 64 conversations in no order over 32 adapters of many ranks
        _lora("adapters, 64 tokens mixed", B=64, q=1, adapters=32, rank=64, mixed=True),
        # drafted tokens of 16 conversations through the gated projection, the activation applied on the way out
        _lora("adapters, 16 x 5 gate up", B=16, q=5, sections="13824,13824", silu=True, adapters=6, rank=32),
        # prompts of a few conversations through the down projection's long rows
        _lora("adapters, prompts down", B=5, q=1501, K=13824, sections="5120", adapters=4, rank=64),
        # a long conversation's next token: the cache is long, what it sees is not
        _window("window, 1 x 131071", B=1, q=1, kv=131071, window=4096, sinks=4),
        # drafted tokens of many conversations, small pages, 8-bit cache
        _window("window, 64 x 4 drafted u8", B=64, q=4, kv=8192, Hq=32, bits=8, page=16, window=1024, sinks=16),
        # a chunk of a long prompt
        _window("window, chunk 2048 of 16384", B=1, q=2048, kv=16384, window=2048, sinks=4),
        # ragged prompts on wide heads, a window that is no multiple of anything
        _window("window, ragged prompts wide", B=3, q=1100, kv=4099, Hq=16, Hkv=2, D=256, page=16, window=501, sinks=3),
        # one conversation, four drafted tokens, every filter on
        _verify("verify, 1 x 4 fp32", B=1, q=5, V=131072, type="fp32", filters="all"),
        # a server's step: filters of its own for every conversation, some greedy, odd vocabulary
        _verify("verify, 64 x 4 bf16", B=64, q=5, V=151669, type="bf16", filters="mixed"),
        # drafts looked up in the text so far: no draft probabilities
        _verify("verify, 16 x 7 looked up", B=16, q=8, V=50021, type="bf16", filters="top_p", draft=False),
    ]


def _log(rng, lo, hi):
    """A whole number, spread evenly over its logarithm."""
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["lora", "window", "verify"])
    c = {"kind": kind, "mix": rng.randint(1, 1 << 20)}
    if kind == "lora":
        c["silu"] = rng.random() < 0.3
        c["K"] = rng.choice([1024, 2048, 5120, 13824, 64 * rng.randint(1, 96)])
        if c["silu"]:
            n = rng.choice([512, 2048, 13824, rng.randint(1, 9000)])
            c["sections"] = f"{n},{n}"
        else:
            c["sections"] = rng.choice(["5120,1024,1024", "1024,256,256", "5120", "2048", str(rng.randint(1, 7000))])
        c["rank"] = rng.choice([8, 16, 16, 32, 64, 24])
        c["mixed"] = rng.random() < 0.5
        c["adapters"] = _log(rng, 1, 48)
        c["B"] = _log(rng, 1, 128)
        # (no more rows than the largest listed case has bytes for)
        width = c["K"] + 2 * sum(map(int, c["sections"].split(",")))
        c["q"] = max(1, min(_log(rng, 1, 2000) if rng.random() < 0.5 else rng.choice([1, 1, 4, 5]), 90_000_000 // width // c["B"]))
        return c
    if kind == "verify":
        c["V"] = _log(rng, 300, 150000) | rng.randint(0, 1)
        c["B"] = _log(rng, 1, 64)
        c["q"] = max(1, min(rng.choice([2, 3, 4, 5, 8, 9]), 45_000_000 // c["V"] // c["B"]))
        c["type"] = rng.choice(["fp32", "bf16"]) if c["B"] * c["q"] * c["V"] < 19e6 else "bf16"
        c["filters"] = rng.choice(["all", "top_p", "top_k", "none", "mixed"])
        c["draft"] = rng.random() < 0.75
        return c
    c["Hkv"] = rng.choice([1, 2, 4, 8])
    rep = rng.choice([1, 2, 3, 4, 5, 6, 7, 8])
    c["Hq"] = c["Hkv"] * rep
    c["D"] = rng.choice([64, 128, 128, 256])
    c["bits"] = rng.choice([4, 4, 8])
    c["page"] = rng.choice([16, 32, 64, 128])
    c["window"] = _log(rng, 1, 8192)
    c["sinks"] = rng.choice([0, 1, 4, 4, 16, 64, 130])
    if rng.random() < 0.6:      # decode: a few tokens a sequence
        c["B"] = _log(rng, 1, 64)
        c["q"] = rng.choice([1, 1, 1, 2, 4, 5, 8])
        c["kv"] = max(c["q"], min(_log(rng, 16, 131072), 524288 // c["B"] * 128 // c["D"]))
    else:                       # prompts and chunks of them
        c["B"] = rng.choice([1, 1, 2, 3, 4])
        c["q"] = max(9, min(_log(rng, 9, 1700), 1700 // c["B"] * 128 // c["D"] * 5 // max(5, rep)))
        c["kv"] = c["q"] + rng.choice([0, _log(rng, 1, 6144 // c["B"])])
    return c


def _lens(c):
    """Tokens of each sequence, and its cache length with them: the first as the case says, the others spread below it; from the sixth sequence on,
    every sixth has no tokens at all."""
    B, q, kv = c["B"], c["q"], c.get("kv", c["q"])
    r = np.random.RandomState(c["mix"])
    ql = np.concatenate([[q], r.randint(max(1, q // 2), q + 1, B - 1)]).astype(np.int64)
    kl = np.maximum(np.concatenate([[kv], r.randint(1, kv + 1, B - 1)]), ql).astype(np.int64)
    empty = np.arange(B) % 6 == 5
    return np.where(empty, 0, ql), np.where(empty, 0, kl)


def _sections(c):
    return [int(n) for n in c["sections"].split(",")]


def _adapters(c):
    """Each token's adapter (-1: one conversation in eight has none), and each adapter's rank."""
    r = np.random.RandomState(c["mix"] + 7)
    ql = _lens(c)[0]
    of = np.where(r.rand(c["B"]) < 0.125, -1, r.randint(0, c["adapters"], c["B"]))
    of[0] = 0
    ranks = r.randint(1, c["rank"] // 8 + 1, c["adapters"]) * 8 if c["mixed"] else np.full(c["adapters"], c["rank"])
    return np.repeat(of, ql), ranks


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


def _cache(c, g):
    """A paged cache whose pages lie in no order, filled with keys and values of ordinary size, a few key channels of them large, as rotated keys have."""
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
    s = {"table": table, "kv_len": torch.from_numpy(kl.astype(np.int32)).cuda()}
    for n in ("k", "v"):
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
        s[n + "q"], s[n + "p"] = words, par
    return s


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    ql, kl = _lens(case)
    T = int(ql.sum())
    start = np.concatenate([[0], np.cumsum(ql)])
    seq = np.repeat(np.arange(case["B"]), ql)
    s = {"case": case, "T": T, "q_start": torch.from_numpy(start.astype(np.int32)).cuda(),
         # token i of the batch: its sequence and its place in it (the plain forms' plan)
         "seq": torch.from_numpy(seq).cuda(), "row": torch.from_numpy(np.arange(T) - start[:-1][seq]).cuda()}
    {"lora": _prepare_lora, "window": _prepare_window, "verify": _prepare_verify}[case["kind"]](case, g, s)
    return s


def _prepare_lora(c, g, s):
    K, N, r = c["K"], _sections(c), c["rank"]
    s["x"] = _randn(g, s["T"], K).bfloat16()
    s["a"] = (_randn(g, c["adapters"], len(N), r, K) * K ** -0.5).bfloat16()
    s["b"] = (_randn(g, c["adapters"], sum(N), r) * 0.3).bfloat16()
    s["y"] = [_randn(g, s["T"], n).bfloat16() for n in N]      # the shared projection's output
    s["scale"] = torch.rand(c["adapters"], device="cuda", generator=g) + 0.5
    ids, ranks = _adapters(c)
    s["ids"] = torch.from_numpy(ids.astype(np.int32)).cuda()
    s["ranks"] = torch.from_numpy(ranks.astype(np.int32)).cuda()
    # rows by adapter (the plain form's plan)
    s["groups"] = [(int(a), int(ranks[a]) if a >= 0 else 0, torch.from_numpy(np.nonzero(ids == a)[0]).cuda()) for a in np.unique(ids)]
    if own:
        import group_wise_affine_gb300 as gwa
        s["lora"] = gwa.LoRA(s["a"], s["b"], scale=s["scale"], ranks=s["ranks"])
        s["workspace"] = gwa.make_lora_workspace(s["lora"], s["T"])


def _prepare_window(c, g, s):
    s.update(_cache(c, g))
    ql, kl = _lens(c)
    s["scale"] = 1.0 / math.sqrt(c["D"])
    s["q"] = (_randn(g, s["T"], c["Hq"], c["D"]) * 0.7).bfloat16()
    s["max_q"], s["max_kv"] = int(ql.max()), int(kl.max())
    if own:
        import group_wise_affine_gb300 as gwa
        s["cache"] = gwa.KVCache(s["kq"], s["kp"], s["vq"], s["vp"], bits=c["bits"])
        s["batch"] = gwa.KVBatch(s["q_start"], s["kv_len"], s["table"], tokens=s["T"], max_q=s["max_q"], max_kv=s["max_kv"])
        s["workspace"] = gwa.make_sdpa_paged_workspace(s["cache"], s["batch"], c["Hq"], window=c["window"], sinks=c["sinks"])


def _prepare_verify(c, g, s):
    B, T, V = c["B"], s["T"], c["V"]
    x = _randn(g, T, V) * 2.0
    likely = torch.randint(0, V, (T, 24), device="cuda", generator=g)
    x.scatter_add_(1, likely, torch.rand((T, 24), device="cuda", generator=g) * 8.0 + 3.0)
    x[:, V - V // 50:] = -math.inf              # padding of the vocabulary
    kind = torch.bfloat16 if c["type"] == "bf16" else torch.float32
    u = lambda n, lo, hi: torch.rand(n, device="cuda", generator=g) * (hi - lo) + lo  # noqa: E731
    f = c["filters"]
    on = lambda name, t, off: torch.full_like(t, off) if f not in (name, "all", "mixed") else (  # noqa: E731
        torch.where(torch.rand(B, device="cuda", generator=g) < 0.4, torch.full_like(t, off), t) if f == "mixed" else t)
    # a conversation's settings, for each of its rows
    t = u(B, 0.6, 1.3)
    t = torch.where(torch.arange(B, device="cuda") % 8 == 7, torch.zeros_like(t), t) if f == "mixed" else t
    per = {"temperature": t, "top_k": on("top_k", torch.randint(1, 200, (B,), device="cuda", generator=g, dtype=torch.int32), 0),
           "top_p": on("top_p", u(B, 0.5, 0.99), 1.0), "min_p": on("min_p", u(B, 0.0, 0.1), 0.0)}
    s.update({n: v[s["seq"]].contiguous() for n, v in per.items()})
    s["logits"] = x.to(kind)
    s["u"], s["u_draw"] = u(T, 0.0, 1.0), u(B, 0.0, 1.0)
    # the draft model's opinion is near the target's; its tokens are drawn from it
    y = (x + _randn(g, T, V) * 0.6).to(kind)
    s["draft_logits"] = y if c["draft"] else None
    w = _masses(y, s).double().cumsum(-1)
    token = torch.searchsorted(w, u(T, 0.0, 1.0)[:, None].double() * w[:, -1:], right=True).clamp(max=V - 1)[:, 0]
    # row i's token was drawn from row i - 1's opinion (the first of a sequence is given)
    s["ids"] = torch.roll(token, 1, 0).to(torch.int32)
    s["has"] = torch.zeros(T, dtype=torch.bool, device="cuda")
    s["has"][:-1] = s["seq"][1:] == s["seq"][:-1]       # rows with a drafted token behind them


# ------------------------------------------------------------------ one pass

def run(state):
    return {"lora": _run_lora, "window": _run_window, "verify": _run_verify}[state["case"]["kind"]](state)


def _run_lora(s):
    c = s["case"]
    if own:
        import group_wise_affine_gb300 as gwa
        if c["silu"]:
            return gwa.lora_gate_up_silu(s["x"], s["y"], s["lora"], s["ids"], workspace=s["workspace"])
        return gwa.lora_add(s["x"], s["y"], s["lora"], s["ids"], workspace=s["workspace"])
    y = [t.float() for t in s["y"]]
    for a, r, rows in s["groups"]:
        if a < 0:
            continue
        x = s["x"][rows].float()
        at = 0
        for i, t in enumerate(y):
            low = torch.matmul(x, s["a"][a, i, :r].float().t())
            t[rows] += torch.matmul(low, s["b"][a, at:at + t.shape[1], :r].float().t()) * s["scale"][a]
            at += t.shape[1]
    if c["silu"]:
        return (y[0] / (1.0 + torch.exp(-y[0])) * y[1]).bfloat16()
    return [t.bfloat16() for t in y]


def _run_window(s):
    c = s["case"]
    if own:
        import group_wise_affine_gb300 as gwa
        return gwa.sdpa_paged(s["q"], s["cache"], s["batch"], scale=s["scale"], window=c["window"], sinks=c["sinks"], workspace=s["workspace"])
    B, Hq, Hkv, D, n = c["B"], c["Hq"], c["Hkv"], c["D"], s["max_q"]
    W, first = c["window"], c["sinks"]
    length, new = s["kv_len"].long(), s["q_start"].diff().long()
    # the keys that some row of a sequence may see: the first ones, then those from its first token's window on
    m = min(s["max_kv"], first + W + n - 1)
    j = torch.arange(m, device="cuda")
    low = (length - new - W + 1).clamp(min=first)
    at = torch.where(j < first, j, low[:, None] + j - first)
    inside = at < length[:, None]
    at = torch.where(inside, at, 0)
    page = s["table"].long().gather(1, at // c["page"]).clamp(min=0)
    k = _values(s["kq"][page, :, at % c["page"]], s["kp"][page, :, at % c["page"]], c["bits"]).permute(0, 2, 3, 1)
    v = _values(s["vq"][page, :, at % c["page"]], s["vp"][page, :, at % c["page"]], c["bits"]).permute(0, 2, 1, 3)
    q = torch.zeros((B, n, Hq, D), device="cuda")
    q[s["seq"], s["row"]] = s["q"].float()
    q = q.reshape(B, n, Hkv, Hq // Hkv, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, -1, D)
    x = (torch.matmul(q, k) * s["scale"]).reshape(B, Hkv, Hq // Hkv, n, m)
    pos = (length - new)[:, None] + torch.arange(n, device="cuda")
    at = at[:, None, :]
    seen = inside[:, None, :] & (at <= pos[:, :, None]) & ((at > pos[:, :, None] - W) | (at < first))
    x = x.masked_fill(~seen[:, None, None], -math.inf)
    x = torch.exp(x - x.amax(-1, keepdim=True).clamp(min=-3e38))
    p = x / x.sum(-1, keepdim=True).clamp(min=1e-30)
    o = torch.matmul(p.reshape(B, Hkv, -1, m), v).reshape(B, Hkv, Hq // Hkv, n, D).permute(0, 3, 1, 2, 4).reshape(B, n, Hq, D)
    return o[s["seq"], s["row"]].bfloat16()


def _masses(x, s):
    """The kept tokens' whole-number masses, zero elsewhere, row by row under its filters."""
    x = x.float()
    x = x.masked_fill(x != x, -math.inf)
    V = x.shape[1]
    top = x.amax(-1, keepdim=True)
    greedy = s["temperature"][:, None] <= 0
    per = torch.where(greedy, 0.0, (1.0 / s["temperature"][:, None]) * 1.4426950408889634)
    w = (torch.exp2(((x - top) * per).masked_fill(x == top, 0.0)) * MASS).to(torch.int64)
    order = torch.sort(x, dim=-1, descending=True, stable=True)[1]
    ws = w.gather(1, order)
    rank = torch.arange(V, device="cuda")
    k = torch.where(greedy, 1, s["top_k"][:, None])
    keep = (rank < k) | (k <= 0)
    ws = ws * keep
    cum = ws.cumsum(-1)
    p = s["top_p"][:, None]
    goal = (cum[:, -1:].double() * p.double()).to(torch.int64)
    keep = keep & ((cum - ws < goal) | (rank == 0) | (p >= 1.0))
    keep = keep & (ws >= (s["min_p"][:, None] * MASS).to(torch.int64))
    return w * torch.zeros_like(keep).scatter_(1, order, keep)


def _run_verify(s):
    c = s["case"]
    if own:
        import group_wise_affine_gb300 as gwa
        token, accepted, prob = gwa.verify_draft(s["logits"], s["ids"], s["q_start"], s["u"], s["u_draw"], draft_logits=s["draft_logits"],
                                                 temperature=s["temperature"], top_k=s["top_k"], top_p=s["top_p"], min_p=s["min_p"])
        return {"token": token, "accepted": accepted, "prob": prob}
    T, B = s["T"], c["B"]
    has, seq, row = s["has"], s["seq"], s["row"]
    p = _masses(s["logits"], s).double()
    p = p / p.sum(-1, keepdim=True)
    draft = torch.roll(s["ids"], -1, 0).long()[:, None]
    if c["draft"]:
        q = _masses(s["draft_logits"], s).double()
        q = q / q.sum(-1, keepdim=True)
    else:
        q = torch.zeros_like(p).scatter_(1, draft, 1.0)
    q = q * has[:, None]                            # behind the last draft the token is the target's own
    pd, qd = p.gather(1, draft)[:, 0], q.gather(1, draft)[:, 0]
    stands = has & (s["u"].double() * qd < pd)
    # rows of a sequence up to its first draft that falls
    fell = torch.full((B,), c["q"], dtype=torch.int64, device="cuda").scatter_reduce_(0, seq, torch.where(stands, c["q"], row), "amin")
    new = s["q_start"].diff().long()
    accepted = torch.where(new > 0, fell, 0)
    at = (s["q_start"][:-1].long() + accepted).clamp(max=T - 1)
    rest = (p[at] - q[at]).clamp(min=0)
    rest = torch.where(rest.sum(-1, keepdim=True) > 0, rest, p[at]).cumsum(-1)
    goal = s["u_draw"][:, None].double() * rest[:, -1:]
    drawn = torch.searchsorted(rest, goal, right=True)[:, 0].clamp(max=c["V"] - 1)
    mine = accepted[seq]
    token = torch.where(row < mine, draft[:, 0], torch.where(row == mine, drawn[seq], -1))
    prob = torch.where(has, (pd / qd.clamp(min=1e-300)).clamp(max=1.0), 0.0)
    return {"token": token.to(torch.int32), "accepted": accepted.to(torch.int32), "prob": prob.float()}


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    c = case
    ql, kl = _lens(c)
    T = int(ql.sum())
    if c["kind"] == "lora":
        ids, ranks = _adapters(c)
        N, used = _sections(c), [int(a) for a in np.unique(ids) if a >= 0]
        weights = sum(int(ranks[a]) * (len(N) * c["K"] + sum(N)) for a in used)
        out = N[0] if c["silu"] else sum(N)
        have = ids >= 0
        return {"bytes": 2 * (weights + int(have.sum()) * c["K"] + T * (sum(N) + out)) + 4 * T,
                "flops": 2 * int(ranks[ids[have]].sum()) * (len(N) * c["K"] + sum(N)) + T * out}
    if c["kind"] == "verify":
        rows = T + (int((ql - 1).clip(0).sum()) if c["draft"] else 0)
        return {"bytes": rows * c["V"] * (4 if c["type"] == "fp32" else 2) + T * 32, "flops": 4 * rows * c["V"]}
    D, W, first = c["D"], c["window"], c["sinks"]
    token = 2 * c["Hkv"] * (D * c["bits"] // 8 + D // GROUP * 4)    # a token's codes, scales and biases, keys and values
    keys = pairs = 0
    for n, m in zip(ql.tolist(), kl.tolist()):
        if n:
            pos = np.arange(m - n, m)
            pairs += int((np.minimum(pos + 1, W) + np.clip(np.minimum(first, pos + 1 - W), 0, None)).sum())
            low = max(m - n - W + 1, 0)
            keys += m - low + min(first, low)
    return {"bytes": keys * token + T * c["Hq"] * D * 4 + 4 * (2 * c["B"] + 1 + keys // c["page"]), "flops": pairs * c["Hq"] * D * 4}


# ------------------------------------------------------------------ the definitions in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return {"lora": _exact_lora, "window": _exact_window, "verify": _exact_verify}[case["kind"]](case, s)


def _exact_lora(c, s):
    N = _sections(c)
    ids, ranks = _adapters(c)
    y = torch.cat(s["y"], 1).double()
    of = np.repeat(np.arange(len(N)), N)            # the section of an output
    for a in range(c["adapters"]):
        rows = torch.from_numpy(np.flatnonzero(ids == a)).cuda()
        if not len(rows):
            continue
        r = int(ranks[a])
        for i in range(len(N)):
            cols = torch.from_numpy(np.flatnonzero(of == i)).cuda()
            delta = s["b"][a, cols, :r].double() @ s["a"][a, i, :r].double()
            for part in rows.split(512):
                y[part[:, None], cols] += float(s["scale"][a]) * (s["x"][part].double() @ delta.t())
    if c["silu"]:
        gate, up = y.split(N, 1)
        return gate * torch.sigmoid(gate) * up
    return list(y.split(N, 1))


def _exact_window(c, s):
    ql, kl = _lens(c)
    D, rep, page, bits = c["D"], c["Hq"] // c["Hkv"], c["page"], c["bits"]
    out = torch.zeros((s["T"], c["Hq"], D), dtype=torch.float64, device="cuda")
    mask = (1 << bits) - 1
    start = 0
    for b in range(c["B"]):
        n, m = int(ql[b]), int(kl[b])
        if not n:
            continue
        low = max(0, m - n - c["window"] + 1)
        key = torch.cat([torch.arange(min(c["sinks"], low), device="cuda"), torch.arange(low, m, device="cuda")])
        ids, slot = s["table"][b, key // page].long(), key % page
        pos = torch.arange(m - n, m, device="cuda")[:, None]
        hidden = (key > pos) | ((pos - key >= c["window"]) & (key >= c["sinks"]))
        for h in range(c["Hkv"]):
            kv = []
            for w in ("k", "v"):
                words = s[w + "q"][ids, h, slot].to(torch.int64)
                par = s[w + "p"][ids, h, slot].double().repeat_interleave(GROUP, 1)
                code = torch.stack([(words >> i) & mask for i in range(0, 32, bits)], -1).reshape(len(key), D).double()
                kv.append(code * par[..., 0] + par[..., 1])
            q = s["q"][start:start + n, h * rep:(h + 1) * rep].double()
            x = torch.einsum("ihd,jd->hij", q, kv[0]) * s["scale"]
            x = torch.softmax(x.masked_fill(hidden, -math.inf), -1)
            out[start:start + n, h * rep:(h + 1) * rep] = torch.einsum("hij,jd->ihd", x, kv[1])
        start += n
    return out


def _exact_verify(c, s):
    def share(x, token, t, k, p, m):
        """One token's share of what the filters keep."""
        x = x.double()
        if t <= 0:
            return 1.0 if token == int((x == x.max()).nonzero()[0]) else 0.0
        e = torch.exp((x - x.max()) / t)
        order = torch.sort(x, descending=True, stable=True)[1]
        if k > 0:
            order = order[:k]
        if p < 1:
            before = e[order].cumsum(0) - e[order]
            order = order[:max(1, int((before < p * e[order].sum()).sum()))]
        order = order[e[order] >= m]
        return float((e[order] * (order == token)).sum() / e[order].sum())

    prob = torch.zeros(s["T"], dtype=torch.float64)
    has, ids = s["has"].tolist(), s["ids"].tolist()
    rule = list(zip(*(s[n].tolist() for n in ("temperature", "top_k", "top_p", "min_p"))))
    for i in range(s["T"]):
        if not has[i]:
            continue
        p = share(s["logits"][i], ids[i + 1], *rule[i])
        q = share(s["draft_logits"][i], ids[i + 1], *rule[i]) if c["draft"] else 1.0
        prob[i] = min(1.0, p / q) if q > 0 else float(p > 0)
    return {"token": None, "accepted": None, "prob": prob.cuda()}
