"""Tokens for several conversations at once, the whole way on the library's
kernels: quantized projections, a paged 4-bit KV cache with the rotary
embedding on the way in, attention over it, sampling.

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
    pages: List[int] = field(default_factory=list)
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


def rms(x: torch.Tensor) -> torch.Tensor:
    f = x.float()
    return (f * torch.rsqrt(f.square().mean(-1, keepdim=True) + 1e-6)).bfloat16()


class Server:
    def __init__(self, config: Config, weights: dict, device="cuda"):
        self.c, self.w, self.device = config, weights, device
        self.caches = [gwa.KVCache.empty(config.pages, config.kv_heads, config.page,
                                         config.head_dim, 4, device) for _ in range(config.layers)]
        self.rope = gwa.rope_table(config.longest, config.head_dim, config.rope_base, device)
        self.status = torch.zeros(1, dtype=torch.int32, device=device)
        self.free = list(range(config.pages))
        self.running: List[Conversation] = []

    def add(self, prompt: List[int], new: int, sampling: Sampling = None) -> Conversation:
        if not prompt or len(prompt) + new > self.c.longest:
            raise ValueError("a prompt of 1 to `longest` tokens, with the new ones")
        s = sampling or Sampling()
        conv = Conversation(list(prompt), s, new, random=torch.Generator().manual_seed(s.seed))
        self.running.append(conv)
        return conv

    def _batch(self, todo):
        """The step's tokens as one batch; pages are taken from the pool."""
        c = self.c
        for conv, n in todo:
            while len(conv.pages) * c.page < conv.done + n:
                if not self.free:
                    raise RuntimeError("the pool has no pages left")
                conv.pages.append(self.free.pop())
        width = max(len(conv.pages) for conv, _ in todo)
        start, length, table = [0], [], []
        for conv, n in todo:
            start.append(start[-1] + n)
            length.append(conv.done + n)
            table.append(conv.pages + [0] * (width - len(conv.pages)))
        dev = lambda a: torch.tensor(a, dtype=torch.int32).to(self.device)  # noqa: E731
        return gwa.KVBatch(dev(start), dev(length), dev(table), start[-1],
                           max(n for _, n in todo), max(length))

    def forward(self, todo) -> torch.Tensor:
        """Runs (conversation, tokens) pairs; the logits of each one's last."""
        c = self.c
        ids = [t for conv, n in todo for t in conv.tokens[conv.done:conv.done + n]]
        batch = self._batch(todo)
        x = self.w["embed"][torch.tensor(ids, device=self.device)]
        T, q_size, kv_size = len(ids), c.heads * c.head_dim, c.kv_heads * c.head_dim
        work = gwa.make_sdpa_paged_workspace(self.caches[0], batch, c.heads)
        for cache, w in zip(self.caches, self.w["layers"]):
            q, k, v = gwa.qmv_fused_sections(rms(x), w["qkv"], [q_size, kv_size, kv_size])
            k, v = (t.view(T, c.kv_heads, c.head_dim) for t in (k, v))
            q = gwa.kv_append(k, v, cache, batch, q=q.view(T, c.heads, c.head_dim),
                              rope=self.rope, status=self.status)
            a = gwa.sdpa_paged(q, cache, batch, workspace=work, status=self.status)
            x = x + gwa.qmv_affine(a.view(T, q_size), w["o"])
            x = x + gwa.qmv_affine(gwa.qmv_gate_up_silu(rms(x), w["gate_up"]), w["down"])
        for conv, n in todo:
            conv.done += n
        last = (batch.q_start[1:] - 1).long()
        return gwa.qmv_affine(rms(x[last]), self.w["head"])

    def step(self) -> int:
        """One step for every running conversation; the tokens it drew."""
        todo = [(conv, min(self.c.chunk, len(conv.tokens) - conv.done)) for conv in self.running]
        if not todo:
            return 0
        logits = self.forward(todo)
        # those whose prompt is through draw a token
        rows = [i for i, (conv, _) in enumerate(todo) if conv.done == len(conv.tokens)]
        if rows:
            convs = [todo[i][0] for i in rows]
            f = lambda a, t=torch.float32: torch.tensor(a, dtype=t).to(self.device)  # noqa: E731
            u = f([float(torch.rand((), generator=conv.random)) for conv in convs])
            s = [conv.sampling for conv in convs]
            token, _ = gwa.sample(logits[rows], u, temperature=f([p.temperature for p in s]),
                                  top_k=f([p.top_k for p in s], torch.int32),
                                  top_p=f([p.top_p for p in s]), min_p=f([p.min_p for p in s]))
            for conv, t in zip(convs, token.tolist()):
                conv.tokens.append(t)
                conv.new -= 1
                if conv.new == 0:
                    self.free += conv.pages
                    conv.pages = []
                    self.running.remove(conv)
        if int(self.status):
            raise RuntimeError(f"cache status {int(self.status)}")
        return len(rows)


def main():
    import time
    c = Config()
    server = Server(c, random_weights(c))
    g = torch.Generator().manual_seed(1)
    convs = [server.add(torch.randint(0, c.vocab, (n,), generator=g).tolist(), new=64,
                        sampling=Sampling(seed=i, temperature=0.0 if i == 0 else 0.8))
             for i, n in enumerate((5, 900, 64, 333))]
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
