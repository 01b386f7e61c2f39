"""The example layer's own refusals: its buffers hold a fixed number of tokens, and
the sort only knows how many rows there are.  No device is needed: every call is
refused before its first launch."""
import importlib.util
import os

import pytest
import torch

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "moe_layer.py")


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("moe_layer_checks", PATH)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)

    class NoLaunch:      # stands for the binding: a call that gets this far was not refused
        def __getattr__(self, name):
            raise AssertionError(f"{name} was called")

    mod.m = NoLaunch()
    return mod


def layer(example, tokens=8, topk=4, experts=16, hidden=64, ffn=96, training=True):
    l = object.__new__(example.MoELayer)
    l.tokens, l.k, l.E, l.H, l.F, l.training, l.rows, l.T = tokens, topk, experts, hidden, ffn, training, 544, None
    return l


def batch(T, k=4, H=64):
    return torch.zeros(T, H, dtype=torch.bfloat16), torch.zeros(T, k, dtype=torch.int32), torch.zeros(T, k)


@pytest.mark.parametrize("call", ["serve", "forward"])
def test_a_batch_that_does_not_fit_is_refused(example, call):
    # 8 tokens x 4 of 16 experts and 9 .. 12 tokens all need 544 rows: rows alone do not tell
    for T in (9, 12, 13):
        with pytest.raises(ValueError):
            getattr(layer(example), call)(*batch(T))


@pytest.mark.parametrize("call", ["serve", "forward"])
def test_other_arguments_that_would_be_misread_are_refused(example, call):
    x, ids, w = batch(8)
    bad = [(x[:7], ids, w), (x[:, :32], ids, w), (x.float(), ids, w), (x.t().contiguous().t(), ids, w),
           (x, ids.long(), w), (x, ids[:, :3], w), (x, torch.zeros(4, 8, dtype=torch.int32).t(), w),
           (x, ids, w[:7]), (x, ids, w.double()), (x, ids, w[:, :3])]
    for b in bad:
        with pytest.raises(ValueError):
            getattr(layer(example), call)(*b)


def test_backward_takes_the_gradient_of_the_last_forward(example):
    l = layer(example)
    with pytest.raises(ValueError):       # no forward pass yet
        l.backward(torch.zeros(8, 64, dtype=torch.bfloat16))
    l.T = 8
    for d in (torch.zeros(7, 64, dtype=torch.bfloat16), torch.zeros(8, 64), torch.zeros(8, 96, dtype=torch.bfloat16)):
        with pytest.raises(ValueError):
            l.backward(d)


def test_weights_of_another_shape_are_refused(example):
    l = layer(example)
    W1, W2, b1 = torch.zeros(16, 96, 64), torch.zeros(16, 64, 96), torch.zeros(16, 96)
    for bad in ((W1[:15], W2, b1), (W1, W2.transpose(1, 2), b1), (W1.bfloat16(), W2, b1), (W1, W2, b1[:, :64]), (W1, W2, b1.double())):
        with pytest.raises(ValueError):
            l.load(*bad)
