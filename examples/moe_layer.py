"""A mixture-of-experts feed-forward layer on the library's row operators and linear layer.

    out[t] = x[t] + sum_j weight[t][j] * ( silu(x[t] W1[e]^T + b1[e]) W2[e]^T ),   e = expert[t][j]

Serving keeps every operand of the products in MXFP8 (sort, dispatch quantised, experts with MXFP8 output,
experts, combine: five launches); training keeps BF16 rows and quantises them along both of their dimensions.

    python examples/moe_layer.py        # a few steps of gradient descent, then a decode batch through the result
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from all_mxfp8_block_gb300 import mxa2a as m  # noqa: E402

ALIGN = 32            # rows of a segment: the MX block along the rows, what the linear layer asks for
BF16, F32, E4M3, E5M2 = m.MXA2A_TYPE_BF16, m.MXA2A_TYPE_F32, m.MXA2A_TYPE_E4M3, m.MXA2A_TYPE_E5M2


def up(x, a):
    return -(-x // a) * a


def codes(*shape):
    return torch.zeros(*shape, dtype=torch.uint8, device="cuda")


def tiles(rows, cols, *groups):
    return torch.zeros(*groups, -(-cols // 128), -(-rows // 128), 512, dtype=torch.uint8, device="cuda")


def bf16(*shape):
    return torch.zeros(*shape, dtype=torch.bfloat16, device="cuda")


def check(name, t, dtype, *shape):
    """The library takes addresses: what a call reads or writes has to be what it is taken for."""
    if t.dtype != dtype or tuple(t.shape) != shape or not t.is_contiguous():
        raise ValueError(f"{name}: contiguous {dtype} {list(shape)} wanted, got {t.dtype} {list(t.shape)}")


class MoELayer:
    """Buffers and plans for up to ``tokens`` tokens a call; hidden and ffn multiples of 32."""

    def __init__(self, tokens, topk, experts, hidden, ffn, training=False):
        self.tokens, self.k, self.E, self.H, self.F = tokens, topk, experts, hidden, ffn
        self.T = None         # tokens of the forward pass that a backward pass may follow
        rows = self.rows_of(tokens)
        i32 = lambda n: torch.zeros(n, dtype=torch.int32, device="cuda")  # noqa: E731
        self.offsets, self.counts, self.pos = i32(experts + 1), i32(experts), i32(tokens * topk)
        self.up = m.Linear(experts, rows, ffn, hidden, training)
        self.down = m.Linear(experts, rows, hidden, ffn, training)
        self.x, self.x_s = codes(rows, hidden), tiles(rows, hidden)
        self.h, self.h_s = codes(rows, ffn), tiles(rows, ffn)
        self.y = bf16(rows, hidden)
        self.w1, self.w1_s = codes(experts, ffn, hidden), tiles(ffn, hidden, experts)
        self.w2, self.w2_s = codes(experts, hidden, ffn), tiles(hidden, ffn, experts)
        self.training = training
        if training:
            r32 = up(rows, 32)
            self.xb, self.z, self.hb = bf16(rows, hidden), bf16(rows, ffn), bf16(rows, ffn)
            self.x_t, self.x_ts = codes(hidden, r32), tiles(hidden, rows)
            self.h_t, self.h_ts = codes(ffn, r32), tiles(ffn, rows)
            self.w1_t, self.w1_ts = codes(experts, hidden, ffn), tiles(hidden, ffn, experts)
            self.w2_t, self.w2_ts = codes(experts, ffn, hidden), tiles(ffn, hidden, experts)
            self.dy, self.dh, self.dxs = bf16(rows, hidden), bf16(rows, ffn), bf16(rows, hidden)

    def rows_of(self, tokens):
        """Rows that a call with so many tokens works on.  A call passes its own, not the layer's most: the
        kernels' tiles and splits are chosen by them (a decode step's by a decode step's)."""
        return max(ALIGN, m.mxa2a_moe_rows(tokens, self.k, self.E, ALIGN))

    def load(self, W1, W2, b1=None):
        """W1 fp32 [experts][ffn][hidden], W2 [experts][hidden][ffn], b1 [experts][ffn]: quantised once per update."""
        check("W1", W1, torch.float32, self.E, self.F, self.H)
        check("W2", W2, torch.float32, self.E, self.H, self.F)
        if b1 is not None:
            check("b1", b1, torch.float32, self.E, self.F)
        t = self.training
        m.mxa2a_quantize(W1, F32, self.H, self.E, self.F, self.H, E4M3, self.w1, self.w1_s,
                         self.w1_t if t else None, self.w1_ts if t else None)
        m.mxa2a_quantize(W2, F32, self.F, self.E, self.H, self.F, E4M3, self.w2, self.w2_s,
                         self.w2_t if t else None, self.w2_ts if t else None)
        self.b1 = b1

    def _sort(self, x, expert, weight):
        # (pos holds `tokens` tokens: the sort only checks the rows, whose padding has room for more)
        T = expert.shape[0]
        if T > self.tokens:
            raise ValueError(f"{T} tokens: this layer takes up to {self.tokens}")
        check("x", x, torch.bfloat16, T, self.H)
        check("expert", expert, torch.int32, T, self.k)
        check("weight", weight, torch.float32, T, self.k)
        self.rows = self.rows_of(T)
        m.mxa2a_moe_sort(T, self.k, self.E, ALIGN, self.rows, expert, self.offsets, self.counts, self.pos, None)
        return T

    def serve(self, x, expert, weight):
        """x bf16 [T][hidden], expert int32 [T][topk], weight fp32 [T][topk]; returns bf16 [T][hidden]."""
        T, out = self._sort(x, expert, weight), torch.empty_like(x)
        self.T = None         # (the rows of a forward pass are no longer there)
        m.mxa2a_moe_dispatch(T, self.k, self.E, self.H, self.rows, x, BF16, self.H, self.pos, self.offsets, self.counts,
                             self.x, E4M3, self.x_s)
        self.up.run(self.rows, self.x, self.x_s, self.w1, self.w1_s, self.h, E4M3, self.h_s, self.offsets, self.counts,
                    self.b1, m.MXA2A_ACT_SILU)
        self.down.run(self.rows, self.h, self.h_s, self.w2, self.w2_s, self.y, BF16, None, self.offsets, self.counts)
        m.mxa2a_moe_combine(T, self.k, self.H, self.rows, self.y, BF16, self.pos, weight, x, out)
        return out

    def forward(self, x, expert, weight):
        """As serve, keeping what backward needs."""
        T, H, F, rows, out = self._sort(x, expert, weight), self.H, self.F, self.rows, torch.empty_like(x)
        self.T, self.weight = T, weight
        m.mxa2a_moe_dispatch(T, self.k, self.E, H, rows, x, BF16, H, self.pos, self.offsets, self.counts, self.xb, BF16)
        m.mxa2a_quantize(self.xb, BF16, H, 1, rows, H, E4M3, self.x, self.x_s, self.x_t, self.x_ts)
        self.up.run(rows, self.x, self.x_s, self.w1, self.w1_s, self.hb, BF16, None, self.offsets, self.counts,
                    self.b1, m.MXA2A_ACT_SILU, None, self.z)
        m.mxa2a_quantize(self.hb, BF16, F, 1, rows, F, E4M3, self.h, self.h_s, self.h_t, self.h_ts)
        self.down.run(rows, self.h, self.h_s, self.w2, self.w2_s, self.y, BF16, None, self.offsets, self.counts)
        m.mxa2a_moe_combine(T, self.k, H, rows, self.y, BF16, self.pos, weight, x, out)
        return out

    def backward(self, dout):
        """dout bf16 [T][hidden]: gradients of x, the routing weights, W1, W2 (fp32) and b1."""
        if self.T is None:
            raise ValueError("no forward pass to take the gradient of")
        check("dout", dout, torch.bfloat16, self.T, self.H)
        T, E, H, F, rows = self.T, self.E, self.H, self.F, self.rows
        f32 = lambda *s: torch.empty(*s, device="cuda")  # noqa: E731
        dweight, dW1, dW2, db1 = f32(T, self.k), f32(E, F, H), f32(E, H, F), f32(E, F)
        seg = (self.offsets, self.counts)
        m.mxa2a_moe_combine_backward(T, self.k, E, H, rows, dout, BF16, self.y, self.pos, *seg, self.weight, self.dy,
                                     dweight)
        self.down.backward(rows, self.dy, None, m.MXA2A_ACT_NONE, E5M2, self.h_t, self.h_ts, self.w2_t, self.w2_ts,
                           self.dh, dW2, F32, None, *seg)
        self.up.backward(rows, self.dh, self.z, m.MXA2A_ACT_SILU, E5M2, self.x_t, self.x_ts, self.w1_t, self.w1_ts,
                         self.dxs, dW1, F32, db1, *seg)
        dx = torch.empty_like(dout)      # the copies' gradients summed, plus the residual's
        m.mxa2a_moe_combine(T, self.k, H, rows, self.dxs, BF16, self.pos, None, dout, dx)
        return dx, dweight, dW1, dW2, db1


def route(x, router, topk):
    """Expert ids and softmax weights of the topk largest router scores."""
    top, ids = (x.float() @ router.t()).topk(topk, dim=1)
    return ids.to(torch.int32).contiguous(), top.softmax(1).contiguous()


def main(tokens=512, topk=4, experts=16, hidden=512, ffn=384, steps=30, lr=2.0):
    g = torch.Generator(device="cuda").manual_seed(0)
    randn = lambda *s: torch.randn(*s, device="cuda", generator=g)  # noqa: E731
    router = randn(experts, hidden) / hidden ** 0.5
    W1, W2 = randn(experts, ffn, hidden) / hidden ** 0.5, randn(experts, hidden, ffn) / ffn ** 0.5
    b1 = 0.1 * randn(experts, ffn)
    x = randn(tokens, hidden).bfloat16()
    ids, weight = route(x, router, topk)
    layer = MoELayer(tokens, topk, experts, hidden, ffn, training=True)
    layer.load(W1, W2, b1)
    target = layer.forward(x, ids, weight).float() + 0.3 * randn(tokens, hidden)    # learn a perturbed output
    losses = []
    for _ in range(steps):
        layer.load(W1, W2, b1)
        diff = layer.forward(x, ids, weight).float() - target
        losses.append(float((diff * diff).sum(1).mean()) / 2)
        _, _, dW1, dW2, db1 = layer.backward((diff / tokens).bfloat16())
        for p, d in ((W1, dW1), (W2, dW2), (b1, db1)):
            p -= lr * d
    layer.load(W1, W2, b1)
    print("training loss %.3f -> %.3f in %d steps" % (losses[0], losses[-1], steps))
    server = MoELayer(8, topk, experts, hidden, ffn)
    server.load(W1, W2, b1)
    got = server.serve(x[:8].contiguous(), ids[:8].contiguous(), weight[:8].contiguous()).float()
    want = layer.forward(x, ids, weight).float()[:8]
    print("8 tokens served: largest difference from the training path %.3g of %.3g" % ((got - want).abs().max(), want.abs().max()))
    for lin in (layer.up, layer.down, server.up, server.down):
        if lin.status()["code"]:
            raise RuntimeError(f"device status {lin.status()}")
    return losses, got, want


if __name__ == "__main__":
    main()
