"""Tokens for several conversations at once, the whole way on the library's
kernels: quantized projections with each conversation's own low-rank adapter
beside them, a paged 4-bit KV cache with the rotary embedding on the way in,
attention over it (whole, or through a sliding window whose pages behind it go
back to the pool), sampling, or the verification of tokens drafted from the
conversation's own text.

    python examples/serve.py            # a synthetic model, a few conversations

A step takes whatever every conversation has to compute, the prompt of a new
one in chunks beside one token each of the running ones, as one ragged batch.
Weights are random; the point is the calls and their order.  Normalisation and
the residual sums are plain PyTorch.
"""
import os
import sys
from dataclasses import dataclass, field
from typing import List

import torch

if __name__ == "__main__":
    sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import group_wise_affine_gb300 as gwa


@dataclass
class Config:
    layers: int = 2
    hidden: int = 1024
    heads: int = 8
    kv_heads: int = 2
    head_dim: int = 128
    ffn: int = 2048
    vocab: int = 4096
    rope_base: float = 1e4
    longest: int = 4096      # tokens of a conversation
    page: int = 16           # tokens of a page
    pages: int = 512         # of the pool, for every layer
    chunk: int = 256         # prompt tokens of a step
    window: int = 0          # keys that a token sees (0: all), and the first ones
    sinks: int = 4           # that it sees beside them
    drafts: int = 0          # tokens that a step may guess ahead


@dataclass
class Sampling:
    temperature: float = 0.8
    top_k: int = 50
    top_p: float = 0.95
    min_p: float = 0.0
    seed: int = 0


@dataclass
class Conversation:
    tokens: List[int]
    sampling: Sampling
    new: int                                    # tokens still to draw
    done: int = 0                               # tokens in the cache
    pages: List[int] = field(default_factory=list)  # (-1: given back)
    adapter: int = -1                           # of the server's (-1: none)
    random: torch.Generator = None


def random_weights(c: Config, seed: int = 0, device="cuda") -> dict:
    g = torch.Generator(device=device).manual_seed(seed)

    def w(n, k):
        return gwa.quantize_affine((torch.randn((n, k), device=device, generator=g)
                                    * k ** -0.5).bfloat16())

    q, kv = c.heads * c.head_dim, c.kv_heads * c.head_dim
    return {"embed": torch.randn((c.vocab, c.hidden), device=device, generator=g).bfloat16(),
            "head": w(c.vocab, c.hidden),
            "layers": [{"qkv": w(q + 2 * kv, c.hidden), "o": w(c.hidden, q),
                        "gate_up": w(2 * c.ffn, c.hidden), "down": w(c.hidden, c.ffn)}
                       for _ in range(c.layers)]}


def random_adapters(c: Config, count: int, rank: int, seed: int = 0, size: float = 0.3, device="cuda") -> list:
    """Adapters for every projection of every layer."""
    g = torch.Generator(device=device).manual_seed(seed)

    def w(sizes, k):
        r = lambda *s: torch.randn(s, device=device, generator=g)  # noqa: E731
        return gwa.LoRA((r(count, len(sizes), rank, k) * k ** -0.5).bfloat16(),
                        (r(count, sum(sizes), rank) * size * rank ** -0.5).bfloat16(),
                        scale=torch.ones(count, device=device))

    q, kv = c.heads * c.head_dim, c.kv_heads * c.head_dim
    return [{"qkv": w([q, kv, kv], c.hidden), "o": w([c.hidden], q), "gate_up": w([c.ffn, c.ffn], c.hidden),
             "down": w([c.hidden], c.ffn)} for _ in range(c.layers)]


def rms(x: torch.Tensor) -> torch.Tensor:
    f = x.float()
    return (f * torch.rsqrt(f.square().mean(-1, keepdim=True) + 1e-6)).bfloat16()


class Server:
    def __init__(self, config: Config, weights: dict, device="cuda", adapters: list = None):
        self.c, self.w, self.device = config, weights, device
        self.adapters = adapters
        self.caches = [gwa.KVCache.empty(config.pages, config.kv_heads, config.page,
                                         config.head_dim, 4, device) for _ in range(config.layers)]
        self.rope = gwa.rope_table(config.longest, config.head_dim, config.rope_base, device)
        self.status = torch.zeros(1, dtype=torch.int32, device=device)
        self.free = list(range(config.pages))
        self.running: List[Conversation] = []

    def add(self, prompt: List[int], new: int, sampling: Sampling = None, adapter: int = -1) -> Conversation:
        if not prompt or len(prompt) + new > self.c.longest:
            raise ValueError("a prompt of 1 to `longest` tokens, with the new ones")
        s = sampling or Sampling()
        conv = Conversation(list(prompt), s, new, adapter=adapter, random=torch.Generator().manual_seed(s.seed))
        self.running.append(conv)
        return conv

    def _batch(self, todo):
        """The step's tokens as one batch; pages are taken from the pool."""
        c = self.c
        for conv, n, drafts in todo:
            while len(conv.pages) * c.page < conv.done + n + len(drafts):
                if not self.free:
                    raise RuntimeError("the pool has no pages left")
                conv.pages.append(self.free.pop())
        width = max(len(conv.pages) for conv, _, _ in todo)
        start, length, table = [0], [], []
        for conv, n, drafts in todo:
            start.append(start[-1] + n + len(drafts))
            length.append(conv.done + n + len(drafts))
            table.append(conv.pages + [0] * (width - len(conv.pages)))
        dev = lambda a: torch.tensor(a, dtype=torch.int32).to(self.device)  # noqa: E731
        return gwa.KVBatch(dev(start), dev(length), dev(table), start[-1],
                           max(n + len(d) for _, n, d in todo), max(length))

    def _give_back(self, conv):
        """The pages that no later token sees."""
        c = self.c
        for j in range(max(0, conv.done - c.window + 1) // c.page if c.window else 0):
            if j * c.page >= c.sinks and conv.pages[j] >= 0:
                self.free.append(conv.pages[j])
                conv.pages[j] = -1

    def forward(self, todo) -> torch.Tensor:
        """Runs (conversation, tokens) pairs, or (conversation, tokens, drafted
        tokens behind them); the logits of each one's last token and of its
        drafts."""
        c = self.c
        todo = [(t[0], t[1], t[2] if len(t) > 2 else []) for t in todo]
        ids = [t for conv, n, d in todo for t in conv.tokens[conv.done:conv.done + n] + d]
        batch = self._batch(todo)
        dev = lambda a: torch.tensor(a, dtype=torch.int32).to(self.device)  # noqa: E731
        own = dev([conv.adapter for conv, n, d in todo for _ in range(n + len(d))]) if self.adapters else None
        x = self.w["embed"][torch.tensor(ids, device=self.device)]
        T, q_size, kv_size = len(ids), c.heads * c.head_dim, c.kv_heads * c.head_dim
        seen = {"window": c.window, "sinks": c.sinks} if c.window else {}
        work = gwa.make_sdpa_paged_workspace(self.caches[0], batch, c.heads, **seen)
        for i, (cache, w) in enumerate(zip(self.caches, self.w["layers"])):
            lora = self.adapters[i] if self.adapters else None

            def adapt(name, x, ys):
                if lora:
                    gwa.lora_add(x, ys, lora[name], own, out=ys, status=self.status, runs=len(todo))
                return ys

            h = rms(x)
            q, k, v = adapt("qkv", h, gwa.qmv_fused_sections(h, w["qkv"], [q_size, kv_size, kv_size]))
            k, v = (t.view(T, c.kv_heads, c.head_dim) for t in (k, v))
            q = gwa.kv_append(k, v, cache, batch, q=q.view(T, c.heads, c.head_dim),
                              rope=self.rope, status=self.status)
            a = gwa.sdpa_paged(q, cache, batch, workspace=work, status=self.status, **seen).view(T, q_size)
            x = x + adapt("o", a, [gwa.qmv_affine(a, w["o"])])[0]
            h = rms(x)
            if lora:
                h = gwa.lora_gate_up_silu(h, gwa.qmv_fused_sections(h, w["gate_up"], [c.ffn, c.ffn]), lora["gate_up"],
                                          own, status=self.status, runs=len(todo))
            else:
                h = gwa.qmv_gate_up_silu(h, w["gate_up"])
            x = x + adapt("down", h, [gwa.qmv_affine(h, w["down"])])[0]
        rows, at = [], 0
        for conv, n, d in todo:
            conv.done += n
            rows += range(at + n - 1, at + n + len(d))
            at += n + len(d)
        return gwa.qmv_affine(rms(x[torch.tensor(rows, device=self.device)]), self.w["head"])

    def _draft(self, conv) -> List[int]:
        """What followed the conversation's last two tokens before."""
        t, most = conv.tokens, min(self.c.drafts, conv.new - 1)
        for i in range(len(t) - 3, 0, -1):
            if most > 0 and t[i - 1:i + 1] == t[-2:]:
                return t[i + 1:i + 1 + most]
        return []

    def _draw(self, convs, drafts, logits) -> List[List[int]]:
        """The next tokens of conversations that have their last token's logits
        (and their drafts')."""
        f = lambda a, t=torch.float32: torch.tensor(a, dtype=t).to(self.device)  # noqa: E731
        rand = lambda conv: float(torch.rand((), generator=conv.random))  # noqa: E731
        each = [conv.sampling for conv, d in zip(convs, drafts) for _ in range(1 + len(d))]
        filters = dict(temperature=f([p.temperature for p in each]), top_k=f([p.top_k for p in each], torch.int32),
                       top_p=f([p.top_p for p in each]), min_p=f([p.min_p for p in each]))
        if not self.c.drafts:
            token, _ = gwa.sample(logits, f([rand(conv) for conv in convs]), **filters)
            return [[t] for t in token.tolist()]
        start = [0]
        for d in drafts:
            start.append(start[-1] + 1 + len(d))
        ids = [t for conv, d in zip(convs, drafts) for t in [conv.tokens[-1]] + d]
        u = [rand(conv) for conv, d in zip(convs, drafts) for _ in range(1 + len(d))]
        token, stand, _ = gwa.verify_draft(logits, f(ids, torch.int32), f(start, torch.int32), f(u),
                                           f([rand(conv) for conv in convs]), **filters)
        token, stand = token.tolist(), stand.tolist()
        return [token[a:a + 1 + n] for a, n in zip(start, stand)]

    def step(self) -> int:
        """One step for every running conversation; the tokens it drew."""
        todo = []
        for conv in self.running:
            n = min(self.c.chunk, len(conv.tokens) - conv.done)
            todo.append((conv, n, self._draft(conv) if conv.done + n == len(conv.tokens) else []))
        if not todo:
            return 0
        logits = self.forward(todo)
        # those whose prompt is through draw their next tokens
        rows, convs, drafts, at = [], [], [], 0
        for conv, _, d in todo:
            if conv.done == len(conv.tokens):
                convs.append(conv)
                drafts.append(d)
                rows += range(at, at + 1 + len(d))
            at += 1 + len(d)
        drawn = 0
        if rows:
            for conv, tokens in zip(convs, self._draw(convs, drafts, logits[rows])):
                # (those that stood are in the cache already)
                conv.done += len(tokens) - 1
                conv.tokens += tokens
                conv.new -= len(tokens)
                drawn += len(tokens)
                if conv.new == 0:
                    self.free += [j for j in conv.pages if j >= 0]
                    conv.pages = []
                    self.running.remove(conv)
        for conv in self.running:
            self._give_back(conv)
        if int(self.status):
            raise RuntimeError(f"cache status {int(self.status)}")
        return drawn


def main():
    import time
    c = Config(window=512, drafts=3)
    server = Server(c, random_weights(c), adapters=random_adapters(c, count=3, rank=16))
    g = torch.Generator().manual_seed(1)
    convs = [server.add(torch.randint(0, c.vocab, (n,), generator=g).tolist() * 2, new=64, adapter=i - 1,
                        sampling=Sampling(seed=i, temperature=0.0 if i == 0 else 0.8))
             for i, n in enumerate((5, 450, 64, 333))]
    server.step()
    torch.cuda.synchronize()
    t, n = time.perf_counter(), 0
    while server.running:
        n += server.step()
    print(f"{n} tokens in {time.perf_counter() - t:.3f} s")
    for conv in convs:
        print(conv.tokens[-8:])


if __name__ == "__main__":
    main()
