"""The serving path as one: examples/serve.py runs projections, append,
attention over the paged cache and sampling together.

Logits tolerance.  A conversation computed token by token and the same one
computed as one prompt go through different kernels, which round the same
values at different sums: bf16 activations (2^-9 each, some ten roundings on
the way), and where such a rounding moves a key or value across a code's
boundary (about 2 in 100 of them) the cache holds a neighbouring code, 1/15 of
the group's range or about 0.35 of its deviation away.  0.35 sqrt(0.02) = 0.05
of a key or value, rms, carries over to the logits at no more than its own
size; the test allows twice that.
"""
import importlib.util
import os

import pytest
import torch

import group_wise_affine_gb300 as gwa

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "examples", "serve.py")


@pytest.fixture(scope="module")
def serve():
    gwa.build()
    gwa.load()
    import sys
    spec = importlib.util.spec_from_file_location("serve_example", PATH)
    m = importlib.util.module_from_spec(spec)
    sys.modules["serve_example"] = m  # (dataclasses look their module up)
    spec.loader.exec_module(m)
    return m


def prompts(serve, c, lens):
    g = torch.Generator().manual_seed(7)
    return [torch.randint(0, c.vocab, (n,), generator=g).tolist() for n in lens]


def run(serve, c, w, lens, new):
    server = serve.Server(c, w)
    convs = [server.add(p, new, serve.Sampling(seed=i, temperature=0.0 if i == 1 else 0.9))
             for i, p in enumerate(prompts(serve, c, lens))]
    steps = 0
    while server.running:
        server.step()
        steps += 1
    assert sorted(server.free) == list(range(c.pages))
    return [v.tokens for v in convs], steps


def test_conversations_run_to_their_end_and_repeat(serve):
    c = serve.Config(layers=2, chunk=64)
    w = serve.random_weights(c)
    lens, new = (1, 150, 17, 64), 9
    a, steps = run(serve, c, w, lens, new)
    assert steps == 3 - 1 + new  # the longest prompt takes three chunks
    for t, n in zip(a, lens):
        assert len(t) == n + new and all(0 <= i < c.vocab for i in t)
    b, _ = run(serve, c, w, lens, new)
    assert a == b


def test_token_by_token_agrees_with_one_prompt(serve):
    c = serve.Config(layers=2, chunk=512)
    w = serve.random_weights(c, seed=3)
    p = prompts(serve, c, [90])[0]
    whole, single = serve.Server(c, w), serve.Server(c, w)
    conv = whole.add(p, 1)
    want = whole.forward([(conv, len(p))]).float()
    conv = single.add(p, 1)
    for _ in p:
        got = single.forward([(conv, 1)]).float()
    err = (got - want).square().mean().sqrt() / want.square().mean().sqrt()
    assert float(err) < 0.1, float(err)


def test_the_pool_runs_out_with_an_error(serve):
    c = serve.Config(layers=1, pages=4)
    server = serve.Server(c, serve.random_weights(c))
    server.add([1] * 65, 2)
    with pytest.raises(RuntimeError):
        server.step()
    with pytest.raises(ValueError):
        server.add([], 1)
