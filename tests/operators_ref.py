"""64-bit references of the mixture-of-experts row operators and the linear
layer (numpy), sharing no code with the package."""
from __future__ import annotations

import math

import numpy as np
import torch

MANT = {"e4m3": (3, -6, 8, 448.0, torch.float8_e4m3fn), "e5m2": (2, -14, 15, 57344.0, torch.float8_e5m2)}
F32_EPS = 2.0 ** -24           # half a unit in the last place of 1.0f
ROUND = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11, "f32": 2.0 ** -24}   # unit roundoff: 2^-p for p significant bits
TINY = {"bf16": 2.0 ** -134, "f16": 2.0 ** -25, "f32": 2.0 ** -150}  # half the smallest subnormal
DTYPE = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def up(x, a):
    return -(-x // a) * a


def routing(tokens, topk, experts, seed, drop=0.0, only=None):
    """int32 [tokens][topk] distinct experts of each token (from `only`, if given); -1 with probability drop."""
    rng = np.random.default_rng(seed)
    pool = np.arange(experts) if only is None else np.asarray(only)
    ids = np.stack([rng.permutation(pool)[:topk] for _ in range(tokens)]) if tokens else np.zeros((0, topk), np.int64)
    ids = np.where(rng.random(ids.shape) < drop, -1, ids)
    return ids.astype(np.int32)


def sort(ids, experts, align, rows):
    """offsets, counts, pos, src, by walking the assignments in order."""
    flat = ids.reshape(-1)
    counts = [0] * experts
    for e in flat:
        if 0 <= e < experts:
            counts[e] += 1
    offsets = [0]
    for c in counts:
        offsets.append(offsets[-1] + up(c, align))
    nxt = list(offsets[:-1])
    pos = np.full(flat.size, -1, np.int64)
    src = np.full(rows, -1, np.int64)
    for i, e in enumerate(flat):
        if 0 <= e < experts:
            pos[i] = nxt[e]
            src[nxt[e]] = i
            nxt[e] += 1
    return np.array(offsets), np.array(counts), pos.reshape(ids.shape), src


def quant(x, fmt):
    """(code values, scale exponents X) of float64 [..., K], blocks of 32: values are x / 2^X rounded to the format."""
    bits, emin, emax, vmax, _ = MANT[fmt]
    b = np.asarray(x, np.float64).reshape(*x.shape[:-1], x.shape[-1] // 32, 32)
    amax = np.abs(b).max(-1)
    _, e = np.frexp(amax)
    X = np.where(amax > 0, np.clip(e - 1 - emax, -127, 127), -127)
    v = b / np.exp2(X)[..., None]
    _, m = np.frexp(np.where(v == 0, 2.0 ** -300, v))
    step = np.exp2(np.maximum(m - 1, emin) - bits)
    q = np.clip(np.rint(v / step) * step, -vmax, vmax)
    return q.reshape(x.shape), X


def quant_values(x, fmt):
    q, X = quant(x, fmt)
    return q * np.repeat(np.exp2(X), 32, axis=-1)


def tie_slack(x, fmt, err):
    """Per element: how far its quantised value may move when the element moves by err (a neighbouring code, or the
    whole block where its largest magnitude is that near a power of two)."""
    sign = np.where(x < 0, -1.0, 1.0)
    lo, hi = quant_values(x - sign * err, fmt), quant_values(x + sign * err, fmt)
    return np.abs(hi - lo)


def tiles(s):
    """Scale bytes [..., R, B] in tiles [..., ceil(B/4), ceil(R/128), 512], byte by byte."""
    *lead, R, B = s.shape
    out = np.zeros((*lead, -(-B // 4), -(-R // 128), 512), np.uint8)
    r, b = np.meshgrid(np.arange(R), np.arange(B), indexing="ij")
    out[..., b // 4, r // 128, (r % 32) * 16 + (r % 128) // 32 * 4 + b % 4] = s
    return out


def untile(t, R, B):
    r, b = np.meshgrid(np.arange(R), np.arange(B), indexing="ij")
    return t[..., b // 4, r // 128, (r % 32) * 16 + (r % 128) // 32 * 4 + b % 4]


def encode(values, fmt):
    """Code bytes of values that the format holds exactly."""
    return torch.from_numpy(np.ascontiguousarray(values)).to(MANT[fmt][4]).view(torch.uint8)


def decode(codes, fmt):
    return codes.cpu().view(MANT[fmt][4]).to(torch.float64).numpy()


def mx(x, fmt="e4m3"):
    """Device (codes, scale tiles) of float64 [..., R, K], and the values they stand for."""
    q, X = quant(x, fmt)
    t = torch.from_numpy(tiles((X + 127).astype(np.uint8)))
    return encode(q, fmt).cuda(), t.cuda(), q * np.repeat(np.exp2(X), 32, axis=-1)


def act(z, name):
    if name == "relu":
        return np.maximum(z, 0)
    if name == "gelu":
        return 0.5 * z * (1 + np.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))
    if name == "silu":
        return z / (1 + np.exp(-z))
    return z


def slope(z, name):
    if name == "relu":
        return (z > 0).astype(np.float64)
    if name == "gelu":
        a = math.sqrt(2 / math.pi)
        t = np.tanh(a * (z + 0.044715 * z ** 3))
        return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * a * (1 + 3 * 0.044715 * z * z)
    if name == "silu":
        s = 1 / (1 + np.exp(-z))
        return s * (1 + z * (1 - s))
    return np.ones_like(z)


def slope_size(z, name):
    """Sum of the magnitudes of the two terms that slope() adds (they cancel near gelu's and silu's lowest point)."""
    if name == "gelu":
        a = math.sqrt(2 / math.pi)
        s = 0.5 * (1 + np.tanh(a * (z + 0.044715 * z ** 3)))
        return s + np.abs(slope(z, name) - s)
    if name == "silu":
        s = 1 / (1 + np.exp(-z))
        return s + np.abs(slope(z, name) - s)
    return np.abs(slope(z, name))


def f64(t):
    return t.detach().cpu().to(torch.float64).numpy()


def check(got, ref, bound, what=""):
    got = f64(got) if isinstance(got, torch.Tensor) else got
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    assert np.isfinite(got).all(), what
    over = np.abs(got - ref) - bound
    assert (over <= 0).all(), (what, float(over.max()), np.unravel_index(over.argmax(), over.shape))
