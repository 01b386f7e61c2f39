"""The example layer works on the rows that a call's tokens need, whatever its
buffers hold: the same launches, and so the same bits, as a layer made for the call."""
import pytest
import torch

from tests.test_gpu_moe_example import example  # noqa: F401  (the fixture)

pytestmark = pytest.mark.gpu

K, E, H, F = 4, 16, 512, 384


def made(example, tokens, training=False):  # noqa: F811
    g = torch.Generator(device="cuda").manual_seed(0)
    randn = lambda *s: torch.randn(*s, device="cuda", generator=g)  # noqa: E731
    l = example.MoELayer(tokens, K, E, H, F, training)
    l.load(randn(E, F, H) / H ** 0.5, randn(E, H, F) / F ** 0.5, 0.1 * randn(E, F))
    return l


def batch(example, T, seed):  # noqa: F811
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(T, H, device="cuda", generator=g).bfloat16()
    return (x, *example.route(x, torch.randn(E, H, device="cuda", generator=g), K))


def test_a_large_layer_serves_few_tokens_as_a_small_one(example):  # noqa: F811
    small, large = made(example, 8), made(example, 4096)
    used = []
    for lin in (large.up, large.down):
        run = lin.run
        lin.run = lambda rows, *a, run=run: (used.append(rows), run(rows, *a))
    large.serve(*batch(example, 4096, 1))              # rows of an earlier, larger call lie behind
    b = batch(example, 8, 2)
    got, want = large.serve(*b), small.serve(*b)
    rows = [example.m.mxa2a_moe_rows(t, K, E, example.ALIGN) for t in (4096, 8)]
    assert used == [rows[0], rows[0], rows[1], rows[1]]
    assert torch.equal(got, want)
    assert all(l.status()["code"] == 0 for l in (small.up, small.down, large.up, large.down))


def test_a_smaller_training_batch_gives_the_same_gradients(example):  # noqa: F811
    small, large = made(example, 40, True), made(example, 700, True)
    out = large.forward(*batch(example, 700, 1))
    large.backward(torch.ones_like(out))
    b = batch(example, 40, 2)
    d = torch.randn(40, H, device="cuda").bfloat16()
    assert torch.equal(small.forward(*b), large.forward(*b))
    for a, c in zip(small.backward(d), large.backward(d)):
        assert torch.equal(a, c)
