"""The serving path with adapters, a sliding window and drafted tokens
together: examples/serve.py beside what test_gpu_serve runs of it.

Logits tolerance as there: kernels for few and for many tokens round the same
values at different sums, and where that moves a key or value across a code's
boundary the cache holds a neighbouring code; 0.05 rms of the logits' own size,
twice that allowed.
"""
import pytest
import torch

from test_gpu_serve import prompts, serve  # noqa: F401 (the example, as a fixture)

pytestmark = pytest.mark.gpu


def rms_error(got, want):
    return float((got.float() - want.float()).square().mean().sqrt() / want.float().square().mean().sqrt())


def run(serve, c, w, lens, new, adapters=None, repeat=1):  # noqa: F811
    server = serve.Server(c, w, adapters=adapters)
    convs = [server.add(p * repeat, new, serve.Sampling(seed=i, temperature=0.0 if i == 1 else 0.9),
                        adapter=i % 3 - 1 if adapters else -1) for i, p in enumerate(prompts(serve, c, lens))]
    steps = 0
    while server.running:
        server.step()
        steps += 1
    assert sorted(server.free) == list(range(c.pages))
    return [v.tokens for v in convs], steps


def test_everything_together_runs_to_its_end_and_repeats(serve):  # noqa: F811
    c = serve.Config(layers=2, chunk=64, window=96, sinks=4, drafts=3)
    w, ad = serve.random_weights(c), serve.random_adapters(c, 2, 16)
    lens, new = (3, 150, 17, 64), 24
    a, _ = run(serve, c, w, lens, new, ad, repeat=2)
    for t, n in zip(a, lens):
        assert len(t) == 2 * n + new and all(0 <= i < c.vocab for i in t)
    b, _ = run(serve, c, w, lens, new, ad, repeat=2)
    assert a == b


def test_a_window_longer_than_the_text_changes_nothing(serve):  # noqa: F811
    c = serve.Config(layers=2, chunk=64)
    w = serve.random_weights(c)
    lens, new = (1, 150, 40), 9
    wide = serve.Config(layers=2, chunk=64, window=4096)
    assert run(serve, c, w, lens, new) == run(serve, wide, w, lens, new)


def test_a_window_needs_its_own_pages_only(serve):  # noqa: F811
    """400 tokens through a pool of 11 pages of 16: a window of 64 holds 4 to 5,
    the first keys' page and a chunk's 4 beside them."""
    c = serve.Config(layers=2, chunk=64, window=64, sinks=4, pages=11)
    a, _ = run(serve, c, serve.random_weights(c), (380,), 20)
    assert len(a[0]) == 400


def test_windowed_prompt_agrees_with_token_by_token(serve):  # noqa: F811
    c = serve.Config(layers=2, chunk=512, window=40, sinks=3)
    w, ad = serve.random_weights(c, seed=3), serve.random_adapters(c, 1, 8, seed=4)
    p = prompts(serve, c, [120])[0]
    whole, single = (serve.Server(c, w, adapters=ad) for _ in range(2))
    want = whole.forward([(whole.add(p, 1, adapter=0), len(p))])
    conv = single.add(p, 1, adapter=0)
    for _ in p:
        got = single.forward([(conv, 1)])
        single._give_back(conv)
    assert rms_error(got, want) < 0.1


def test_many_prompt_tokens_with_adapters_agree_with_chunks(serve):  # noqa: F811
    """500 tokens at once (the many-token kernels) and by 100 (the others)."""
    c = serve.Config(layers=1, chunk=512)
    w, ad = serve.random_weights(c, seed=5), serve.random_adapters(c, 3, 24, seed=6)
    p = prompts(serve, c, [500])[0]
    whole, parts = (serve.Server(c, w, adapters=ad) for _ in range(2))
    want = whole.forward([(whole.add(p, 1, adapter=2), 500)])
    conv = parts.add(p, 1, adapter=2)
    for _ in range(5):
        got = parts.forward([(conv, 100)])
    assert rms_error(got, want) < 0.1


def test_adapters_matter_to_their_conversations_alone(serve):  # noqa: F811
    c = serve.Config(layers=2)
    w = serve.random_weights(c, seed=7)
    ad = serve.random_adapters(c, 2, 16, seed=8, size=1.0)
    p = prompts(serve, c, [30])[0]
    plain, server = serve.Server(c, w), serve.Server(c, w, adapters=ad)
    want = plain.forward([(plain.add(p, 1), 30)])
    got = server.forward([(server.add(p, 1, adapter=i), 30) for i in (-1, 0, 1)])
    assert rms_error(got[:1], want) < 0.1
    assert rms_error(got[1:2], want) > 0.3 and rms_error(got[2:], got[1:2]) > 0.3


def test_a_step_verifies_what_it_drafted(serve):  # noqa: F811
    """Drafts' logits are those of the same text taken as a prompt."""
    c = serve.Config(layers=2, drafts=4)
    w = serve.random_weights(c, seed=9)
    p = prompts(serve, c, [60])[0]
    server = serve.Server(c, w)
    a, b = server.add(p[:56], 8), server.add(p, 8)
    got = server.forward([(a, 56, p[56:])])
    assert a.done == 56 and got.shape[0] == 5
    want = server.forward([(b, 60)])
    assert rms_error(got[-1:], want) < 0.1
    # greedy drafts: the model's own next tokens stand, another does not
    for s in (a, b):
        s.sampling.temperature = 0.0
    best = got.float().argmax(-1).tolist()
    out = server._draw([a], [[best[0], best[1], (best[2] + 1) % c.vocab, 0]], got)
    assert out == [[best[0], best[1], best[2]]]
    assert server._draw([a], [best[:4]], got) == [best]


def test_ids_past_the_adapters_raise(serve):  # noqa: F811
    c = serve.Config(layers=1)
    server = serve.Server(c, serve.random_weights(c), adapters=serve.random_adapters(c, 2, 8))
    server.add([1, 2, 3], 2, adapter=2)
    with pytest.raises(RuntimeError):
        server.step()
