"""Cases of the mixture-of-experts operators and of the block-scaled linear layer.

Five operators, each as a user calls it:

* ``dispatch``  tokens sorted by expert (stable counting sort of the expert ids into aligned segments) and
  their rows copied into that order, as they are or quantised to MXFP8 on the way;
* ``combine``   the experts' rows back in token order, weighted, summed over a token's experts, plus a residual;
* ``combine_backward``  its gradient: the experts' rows' and the weights';
* ``linear``    an MXFP8 product per expert (or one for all rows) with bias, activation and residual, written as
  BF16 or as the next product's MXFP8 operand;
* ``linear_backward``   the gradient of that product: input rows, weights and bias, through products of the
  quantised gradient.

Shared layout: expert e's rows are [offsets[e], offsets[e] + counts[e]), segments start at multiples of 32 rows, the
rows between a segment's last token and the next segment are zero.  MXFP8: E4M3 or E5M2 codes, one E8M0 scale per
32 elements along the contraction, scales in tiles: for every 128 elements along the contraction and every 128 rows
512 bytes, row r's four scales at (r % 32) * 16 + (r % 128) / 32 * 4.
"""
import math

import torch

own = False

ALIGN = 32
FMT = {"e4m3": (8, 448.0, torch.float8_e4m3fn, 3, -6), "e5m2": (15, 57344.0, torch.float8_e5m2, 2, -14)}
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


# ---------------------------------------------------------------- cases

def listed():
    return [
        # one token of a decode step to its 8 experts, quantised for their first product: latency only
        {"name": "dispatch 1 token", "op": "dispatch", "tokens": 1, "topk": 8, "experts": 64, "hidden": 4096,
         "type": "bf16", "out": "e4m3", "drop": False},
        # a prefill batch with tokens that lost their expert (capacity or another rank's), quantised on the way
        {"name": "dispatch 4096 tokens", "op": "dispatch", "tokens": 4096, "topk": 4, "experts": 32, "hidden": 7168,
         "type": "bf16", "out": "e4m3", "drop": True},
        # a training batch of an odd number of tokens, rows kept in BF16 (they are quantised both ways later)
        {"name": "dispatch 16001 tokens", "op": "dispatch", "tokens": 16001, "topk": 2, "experts": 8, "hidden": 4096,
         "type": "bf16", "out": "bf16", "drop": False},
        # a decode batch's experts' rows back onto the residual stream
        {"name": "combine 8 tokens", "op": "combine", "tokens": 8, "topk": 8, "experts": 64, "hidden": 4096,
         "type": "bf16", "weighted": True, "residual": True, "drop": False},
        # a prefill batch's
        {"name": "combine 8192 tokens", "op": "combine", "tokens": 8192, "topk": 4, "experts": 32, "hidden": 7168,
         "type": "bf16", "weighted": True, "residual": True, "drop": True},
        # the gradient of a small batch in 32 bits, odd token count
        {"name": "combine backward 509", "op": "combine_backward", "tokens": 509, "topk": 8, "experts": 64,
         "hidden": 2048, "type": "f32", "drop": True},
        # the gradient of a training batch
        {"name": "combine backward 8192", "op": "combine_backward", "tokens": 8192, "topk": 4, "experts": 32,
         "hidden": 4096, "type": "bf16", "drop": False},
        # one token through one dense layer (the benchmark's small-M weights), residual added: bound by the weights' bytes
        {"name": "linear 1 token", "op": "linear", "tokens": 1, "topk": 1, "experts": 1, "dense": True, "N": 7168,
         "K": 8192, "act": "none", "bias": True, "residual": True, "out": "bf16", "preact": False},
        # a decode batch's first expert products, written as the second products' operand
        {"name": "linear experts decode", "op": "linear", "tokens": 8, "topk": 4, "experts": 16, "dense": False,
         "N": 2048, "K": 7168, "act": "silu", "bias": False, "residual": False, "out": "e4m3", "preact": False},
        # a prefill batch's expert products on the MoE-projection-like shape, pre-activation kept for the gradient
        {"name": "linear experts 4096", "op": "linear", "tokens": 4096, "topk": 4, "experts": 32, "dense": False,
         "N": 2048, "K": 7168, "act": "gelu", "bias": True, "residual": False, "out": "bf16", "preact": True},
        # the gradient of a small dense layer, odd row count
        {"name": "linear backward 300", "op": "linear_backward", "tokens": 300, "topk": 1, "experts": 1,
         "dense": True, "N": 1056, "K": 1024, "act": "gelu", "grad": "e4m3"},
        # the gradient of a training batch's expert products
        {"name": "linear backward 8192", "op": "linear_backward", "tokens": 8192, "topk": 2, "experts": 8,
         "dense": False, "N": 4096, "K": 4096, "act": "silu", "grad": "e5m2"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo, hi):
    """A multiple of 32, the scale block; 96 blocks become 97."""
    n = _log(rng, lo // 32, hi // 32)
    return 32 * (n + 1 if n == 96 else n)


def draw(rng):
    op = rng.choice(["dispatch", "combine", "combine_backward", "linear", "linear", "linear_backward"])
    c = {"op": op, "topk": rng.randint(1, 8)}
    if op in ("dispatch", "combine", "combine_backward"):
        c["hidden"] = _width(rng, 256, 7168)
        c["experts"] = max(c["topk"], _log(rng, 2, 256))
        most = {"dispatch": 16384 * 4096 * 2, "combine": 8192 * 7168 * 5, "combine_backward": 8192 * 4096 * 5}[op]
        c["type"] = rng.choice(["bf16", "bf16", "f16", "f32"])
        room = most * 2 // ((c["topk"] + 1) * c["hidden"] * (4 if c["type"] == "f32" else 2))
        c["tokens"] = min(_log(rng, 1, 20000), room)
        c["drop"] = rng.random() < 0.3
        if op == "dispatch":
            c["out"] = rng.choice([c["type"], "e4m3", "e5m2"])
        if op == "combine":
            c["weighted"], c["residual"] = rng.random() < 0.7, rng.random() < 0.5
        return c
    c["dense"] = rng.random() < 0.4
    c["experts"] = 1 if c["dense"] else max(c["topk"], _log(rng, 2, 64))
    if c["dense"]:
        c["topk"] = 1
    c["K"], c["N"] = _width(rng, 256, 8192), _width(rng, 256, 8192)
    while c["experts"] * c["N"] * c["K"] > 32 * 2048 * 7168:
        c["experts"] = max(c["topk"], c["experts"] // 2)
        c["N"] = max(256, c["N"] // 64 * 32)
    c["N"] += 32 if c["N"] == 32 * 96 else 0
    room = (16384 * 2048 * 7168 if op == "linear" else 16384 * 4096 * 4096) // (c["N"] * c["K"] * c["topk"])
    c["tokens"] = max(1, min(_log(rng, 1, 8192), room, 16384 // c["topk"]))
    c["act"] = rng.choice(["none", "relu", "gelu", "silu"])
    if op == "linear":
        c["bias"], c["residual"] = rng.random() < 0.5, rng.random() < 0.4
        c["out"] = rng.choice(["bf16", "bf16", "e4m3"])
        c["preact"] = c["act"] != "none" and rng.random() < 0.5
    else:
        c["grad"] = rng.choice(["e4m3", "e5m2"])
    return c


# ---------------------------------------------------------------- inputs

def _up(x, a):
    return -(-x // a) * a


def _rows(c):
    """Rows that hold any routing of the case's tokens: every segment may need ALIGN - 1 rows of padding."""
    a = c["tokens"] * c["topk"]
    return c["tokens"] if c.get("dense") else _up(a + min(c["experts"], a) * (ALIGN - 1), ALIGN)


def _route(c, g):
    """Distinct experts of every token (some preferred over others), -1 where a token lost one, and softmax weights."""
    T, k, E = c["tokens"], c["topk"], c["experts"]
    logits = torch.randn(T, E, device="cuda", generator=g) + 0.5 * torch.randn(1, E, device="cuda", generator=g)
    top, ids = logits.topk(k, dim=1)
    ids = ids.to(torch.int32)
    if c.get("drop"):
        ids = torch.where(torch.rand(T, k, device="cuda", generator=g) < 0.03, torch.full_like(ids, -1), ids)
    return ids.contiguous(), top.softmax(dim=1).contiguous()


def _segments(ids, E, rows):
    """(offsets, counts, pos, src) of the stable sort: elementary operations, no order kept from one call to the next."""
    flat = ids.reshape(-1).long()
    ok = (flat >= 0) & (flat < E)
    e = torch.where(ok, flat, torch.zeros_like(flat))
    hot = ((flat[:, None] == torch.arange(E, device=flat.device)[None, :])).to(torch.int32)
    counts = hot.sum(0, dtype=torch.int32)
    ends = torch.cumsum((counts + ALIGN - 1) // ALIGN * ALIGN, 0)
    offsets = torch.cat([torch.zeros_like(ends[:1]), ends])
    rank = torch.cumsum(hot, 0, dtype=torch.int32).gather(1, e[:, None])[:, 0].long() - 1
    pos = torch.where(ok, offsets[e] + rank, torch.full_like(rank, -1))
    src = torch.full((rows + 1,), -1, dtype=torch.int32, device=flat.device)
    src[torch.where(ok, pos, torch.full_like(pos, rows))] = torch.arange(flat.numel(), dtype=torch.int32, device=flat.device)
    return offsets.to(torch.int32), counts, pos.to(torch.int32), src[:rows].contiguous()


def _quant(x, fmt):
    """Codes (uint8) and E8M0 bytes of fp32 [..., K], 32 to a scale along the last axis: scale 2^(floor(log2 amax) - emax)."""
    emax, vmax, dt, _, _ = FMT[fmt]
    b = x.reshape(*x.shape[:-1], x.shape[-1] // 32, 32)
    amax = b.abs().amax(-1)
    _, e = torch.frexp(amax)
    X = torch.where(amax > 0, e.to(torch.int32) - 1 - emax, torch.full_like(e, -127, dtype=torch.int32)).clamp(-127, 127)
    q = torch.ldexp(b, -X[..., None]).clamp(-vmax, vmax).to(dt).view(torch.uint8).reshape(x.shape)
    return q, (X + 127).to(torch.uint8)


def _tiles(s):
    """Scale bytes [..., rows, blocks] in tiles [..., ceil(blocks / 4), ceil(rows / 128), 512]."""
    *lead, R, B = s.shape
    Rt, Bt = -(-R // 128), -(-B // 4)
    p = torch.zeros(*lead, Rt * 128, Bt * 4, dtype=torch.uint8, device=s.device)
    p[..., :R, :B] = s
    p = p.reshape(*lead, Rt, 4, 32, Bt, 4)
    n = len(lead)
    return p.permute(*range(n), n + 3, n, n + 2, n + 1, n + 4).reshape(*lead, Bt, Rt, 512).contiguous()


def _untiles(t, R, B):
    """The reverse of _tiles."""
    *lead, Bt, Rt, _ = t.shape
    n = len(lead)
    p = t.reshape(*lead, Bt, Rt, 32, 4, 4).permute(*range(n), n + 1, n + 3, n + 2, n, n + 4)
    return p.reshape(*lead, Rt * 128, Bt * 4)[..., :R, :B]


def _values(codes, scale, fmt):
    """fp32 values of codes [..., K] under E8M0 bytes [..., K / 32]."""
    s = scale.contiguous().view(torch.float8_e8m0fnu).float()
    v = codes.view(FMT[fmt][2]).float()
    return (v.reshape(*s.shape, 32) * s[..., None]).reshape(v.shape)


def _chunked_quant(x, fmt):
    """_quant of a [G][R][K] tensor group by group: weights need no temporaries of their whole size."""
    parts = [_quant(x[i].float(), fmt) for i in range(x.shape[0])]
    return torch.stack([p[0] for p in parts]), torch.stack([p[1] for p in parts])


def _pick(x, at):
    """x's rows at `at`, zeros where it is negative."""
    v = x[at.clamp(min=0).long()]
    return torch.where((at >= 0).reshape(-1, *([1] * (x.dim() - 1))), v, torch.zeros_like(v))


def _inputs(c, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    op, T, k, E, rows = c["op"], c["tokens"], c["topk"], c["experts"], _rows(c)
    randn = lambda *s: torch.randn(*s, device="cuda", generator=g)  # noqa: E731
    s = {"case": dict(c), "rows": rows}
    if op in ("dispatch", "combine", "combine_backward"):
        H, dt = c["hidden"], TYPES[c["type"]]
        ids, w = _route(c, g)
        s["ids"], s["weight"] = ids, w
        offsets, counts, pos, src = _segments(ids, E, rows)
        if op == "dispatch":
            s["x"] = randn(T, H).to(dt)
            s.update(offsets=torch.zeros_like(offsets), counts=torch.zeros_like(counts), pos=torch.zeros_like(pos), src=torch.zeros_like(src))
            if c["out"] in FMT:
                s["out"] = torch.zeros(rows, H, dtype=torch.uint8, device="cuda")
                s["out_scale"] = torch.zeros(-(-H // 128), -(-rows // 128), 512, dtype=torch.uint8, device="cuda")
            else:
                s["out"] = torch.zeros(rows, H, dtype=dt, device="cuda")
            return s
        s.update(offsets=offsets, counts=counts, pos=pos)
        s["y"] = torch.where((src >= 0)[:, None], randn(rows, H), torch.zeros((), device="cuda")).to(dt)
        if op == "combine":
            s["residual"] = randn(T, H).to(dt) if c["residual"] else None
            s["out"] = torch.zeros(T, H, dtype=dt, device="cuda")
        else:
            s["dout"] = randn(T, H).to(dt)
            s["dy"] = torch.zeros(rows, H, dtype=dt, device="cuda")
            s["dweight"] = torch.zeros(T, k, device="cuda")
        return s
    N, K = c["N"], c["K"]
    src = None
    s["offsets"] = s["counts"] = None
    s["lens"], s["starts"] = [T], [0]
    if not c["dense"]:
        ids, _ = _route(c, g)
        s["offsets"], s["counts"], _, src = _segments(ids, E, rows)
        s["lens"], s["starts"] = s["counts"].tolist(), s["offsets"].tolist()[:E]
    s["longest"] = max(s["lens"])
    at = torch.arange(T, dtype=torch.int32, device="cuda") if src is None else src // k * (src >= 0) - (src < 0).to(torch.int32)
    x = _pick(randn(T, K) * (0.25 + torch.rand(T, 1, device="cuda", generator=g)), at)
    W = torch.randn(E, N, K, device="cuda", generator=g, dtype=torch.bfloat16) / math.sqrt(K)
    if op == "linear":
        q, sc = _quant(x, "e4m3")
        s["x"], s["x_scale"] = q, _tiles(sc)
        q, sc = _chunked_quant(W, "e4m3")
        s["w"], s["w_scale"] = q, _tiles(sc)
        s["bias"] = 0.1 * randn(E, N) if c["bias"] else None
        s["residual"] = randn(rows, N).to(torch.bfloat16) if c["residual"] else None
        s["preact"] = torch.zeros(rows, N, dtype=torch.bfloat16, device="cuda") if c["preact"] else None
        if c["out"] in FMT:
            s["out"] = torch.zeros(rows, N, dtype=torch.uint8, device="cuda")
            s["out_scale"] = torch.zeros(-(-N // 128), -(-rows // 128), 512, dtype=torch.uint8, device="cuda")
        else:
            s["out"], s["out_scale"] = torch.zeros(rows, N, dtype=torch.bfloat16, device="cuda"), None
        return s
    pad = _up(rows, 32) - rows
    xt = torch.nn.functional.pad(x, (0, 0, 0, pad)).t().contiguous()
    q, sc = _quant(xt, "e4m3")
    s["x_t"], s["x_t_scale"] = q, _tiles(sc)
    q, sc = _chunked_quant(W.transpose(1, 2).contiguous(), "e4m3")
    s["w_t"], s["w_t_scale"] = q, _tiles(sc)
    s["preact"] = (1.5 * randn(rows, N)).to(torch.bfloat16) if c["act"] != "none" else None
    s["dy"] = (_pick(randn(T, N), at) / math.sqrt(N)).to(torch.bfloat16)
    s["dx"] = torch.zeros(rows, K, dtype=torch.bfloat16, device="cuda")
    s["dw"] = torch.zeros(E, N, K, dtype=torch.bfloat16, device="cuda")
    s["dbias"] = torch.zeros(E, N, device="cuda")
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    if own and case["op"].startswith("linear"):  # the handle that a program keeps for a layer
        from all_mxfp8_block_gb300 import mxa2a
        s["layer"] = mxa2a.Linear(case["experts"], s["rows"], case["N"], case["K"],
                                  training=case["op"] == "linear_backward")
    return s


# ---------------------------------------------------------------- plain forms (32 bits, rounded once at the end)

def _act(z, act):
    if act == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z))
    if act == "gelu":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)))
    if act == "silu":
        return z / (1 + torch.exp(-z))
    return z


def _act_grad(z, act):
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "gelu":
        a = math.sqrt(2 / math.pi)
        t = torch.tanh(a * (z + 0.044715 * z * z * z))
        return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * a * (1 + 3 * 0.044715 * z * z)
    if act == "silu":
        sg = 1 / (1 + torch.exp(-z))
        return sg * (1 + z * (1 - sg))
    return torch.ones_like(z)


def _by_group(s, E):
    """[E][longest] row of each expert's i-th token, -1 past its last."""
    i = torch.arange(max(1, s["longest"]), device="cuda")[None, :]
    if s["offsets"] is None:
        return i
    return torch.where(i < s["counts"][:, None], s["offsets"][:E, None] + i, torch.full_like(i, -1))


def _ungroup(v, at, rows):
    """Rows [E][longest] back to their places in [rows], zeros elsewhere."""
    out = torch.zeros(rows + 1, v.shape[-1], dtype=v.dtype, device=v.device)
    out[torch.where(at >= 0, at, torch.full_like(at, rows)).reshape(-1).long()] = v.reshape(-1, v.shape[-1])
    return out[:rows]


def _as_values(codes, fmt, scale):
    """What is held in 8 bits, as the values it stands for: the codes' and the scales'."""
    return {"codes": codes.view(FMT[fmt][2]), "scale": scale.view(torch.float8_e8m0fnu)}


def _plain(s):
    c = s["case"]
    op, T, k, E, rows = c["op"], c["tokens"], c["topk"], c["experts"], s["rows"]
    if op == "dispatch":
        offsets, counts, pos, src = _segments(s["ids"], E, rows)
        tok = torch.where(src >= 0, src // k, src)
        r = {"offsets": offsets, "counts": counts, "pos": pos, "src": src}
        if c["out"] in FMT:
            q, sc = _quant(s["x"].float(), c["out"])
            r.update(_as_values(_pick(q, tok), c["out"], _tiles(_pick(sc, tok))))
        else:
            r["out"] = _pick(s["x"], tok)
        return r
    if op == "combine":
        at = s["pos"].reshape(T, k)
        v = _pick(s["y"], s["pos"]).float().reshape(T, k, -1)
        if c["weighted"]:
            v = v * torch.where(at >= 0, s["weight"], torch.zeros_like(s["weight"]))[..., None]
        v = v.sum(1)
        return (v if s["residual"] is None else v + s["residual"].float()).to(s["out"].dtype)
    if op == "combine_backward":
        at = s["pos"].reshape(T, k)
        d = s["dout"].float()
        dw = (d[:, None, :] * _pick(s["y"], s["pos"]).float().reshape(T, k, -1)).sum(2)
        v = (d[:, None, :] * s["weight"][..., None]).to(s["dy"].dtype).reshape(T * k, -1)
        return {"dy": _ungroup(v, s["pos"], rows), "dweight": torch.where(at >= 0, dw, torch.zeros_like(dw))}
    N, K = c["N"], c["K"]
    at = _by_group(s, E)
    flat = at.reshape(-1)
    if op == "linear":
        x = _values(s["x"], _untiles(s["x_scale"], rows, K // 32), "e4m3")
        w = _values(s["w"], _untiles(s["w_scale"], N, K // 32), "e4m3")
        z = torch.bmm(_pick(x, flat).reshape(E, -1, K), w.transpose(1, 2))
        if s["bias"] is not None:
            z = z + s["bias"][:, None, :]
        y = _act(z, c["act"])
        if s["residual"] is not None:
            y = y + _pick(s["residual"], flat).float().reshape(y.shape)
        y = _ungroup(y, at, rows)
        if c["out"] in FMT:
            q, sc = _quant(y, c["out"])
            r = _as_values(q, c["out"], _tiles(sc))
        else:
            r = {"out": y.to(torch.bfloat16)}
        if c["preact"]:
            r["preact"] = _ungroup(z, at, rows).to(torch.bfloat16)
        return r
    dz = _pick(s["dy"], flat).float().reshape(E, -1, N)
    if s["preact"] is not None:
        dz = dz * _act_grad(_pick(s["preact"], flat).float().reshape(dz.shape), c["act"])
    r = {"dbias": dz.sum(1)}
    dz = _ungroup(dz, at, _up(rows, 32))
    q, sc = _quant(dz, c["grad"])
    dzr = _pick(_values(q, sc, c["grad"]), flat).reshape(E, -1, N)
    w = _values(s["w_t"], _untiles(s["w_t_scale"], K, N // 32), "e4m3")
    r["dx"] = _ungroup(torch.bmm(dzr, w.transpose(1, 2)), at, rows).to(torch.bfloat16)
    q, sc = _quant(dz.t().contiguous(), c["grad"])
    dzt = _pick(_values(q, sc, c["grad"]).t(), flat).reshape(E, -1, N)
    xt = _values(s["x_t"], _untiles(s["x_t_scale"], K, s["x_t"].shape[1] // 32), "e4m3")
    r["dw"] = torch.bmm(dzt.transpose(1, 2), _pick(xt.t(), flat).reshape(E, -1, K)).to(torch.bfloat16)
    return r


# ---------------------------------------------------------------- the framework's operators

def _own(s):
    from all_mxfp8_block_gb300 import mxa2a as m
    c = s["case"]
    op, T, k, E, rows = c["op"], c["tokens"], c["topk"], c["experts"], s["rows"]
    types = {"bf16": m.MXA2A_TYPE_BF16, "f16": m.MXA2A_TYPE_F16, "f32": m.MXA2A_TYPE_F32,
             "e4m3": m.MXA2A_TYPE_E4M3, "e5m2": m.MXA2A_TYPE_E5M2}
    acts = {"none": m.MXA2A_ACT_NONE, "relu": m.MXA2A_ACT_RELU, "gelu": m.MXA2A_ACT_GELU, "silu": m.MXA2A_ACT_SILU}
    if op == "dispatch":
        H = c["hidden"]
        m.mxa2a_moe_sort(T, k, E, ALIGN, rows, s["ids"], s["offsets"], s["counts"], s["pos"], s["src"])
        m.mxa2a_moe_dispatch(T, k, E, H, rows, s["x"], types[c["type"]], H, s["pos"], s["offsets"], s["counts"],
                             s["out"], types[c["out"]], s.get("out_scale"))
        r = {n: s[n] for n in ("offsets", "counts", "pos", "src")}
        if c["out"] in FMT:
            r.update(_as_values(s["out"], c["out"], s["out_scale"]))
        else:
            r["out"] = s["out"]
        return r
    if op == "combine":
        m.mxa2a_moe_combine(T, k, c["hidden"], rows, s["y"], types[c["type"]], s["pos"],
                            s["weight"] if c["weighted"] else None, s["residual"], s["out"])
        return s["out"]
    if op == "combine_backward":
        m.mxa2a_moe_combine_backward(T, k, E, c["hidden"], rows, s["dout"], types[c["type"]], s["y"], s["pos"],
                                     s["offsets"], s["counts"], s["weight"], s["dy"], s["dweight"])
        return {"dy": s["dy"], "dweight": s["dweight"]}
    if op == "linear":
        s["layer"].run(rows, s["x"], s["x_scale"], s["w"], s["w_scale"], s["out"], types[c["out"]], s["out_scale"],
                       s["offsets"], s["counts"], s["bias"], acts[c["act"]], s["residual"], s["preact"])
        r = _as_values(s["out"], c["out"], s["out_scale"]) if c["out"] in FMT else {"out": s["out"]}
        if c["preact"]:
            r["preact"] = s["preact"]
        return r
    s["layer"].backward(rows, s["dy"], s["preact"], acts[c["act"]], types[c["grad"]], s["x_t"], s["x_t_scale"],
                        s["w_t"], s["w_t_scale"], s["dx"], s["dw"], m.MXA2A_TYPE_BF16, s["dbias"],
                        s["offsets"], s["counts"])
    return {"dbias": s["dbias"], "dx": s["dx"], "dw": s["dw"]}


def run(state):
    return _own(state) if own else _plain(state)


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    c = case
    op, T, k, E = c["op"], c["tokens"], c["topk"], c["experts"]
    a = T * k
    size = {"bf16": 2, "f16": 2, "f32": 4, "e4m3": 33 / 32, "e5m2": 33 / 32}
    hit = 1 if c.get("dense") else E * (1 - (1 - k / E) ** T)  # experts that some token is sent to
    if op == "dispatch":
        H = c["hidden"]
        return {"bytes": 12 * a + 8 * E + T * H * size[c["type"]] + a * H * size[c["out"]], "flops": 0}
    if op == "combine":
        return {"bytes": 8 * a + (a + T * (2 if c["residual"] else 1)) * c["hidden"] * size[c["type"]],
                "flops": 2 * a * c["hidden"]}
    if op == "combine_backward":
        return {"bytes": 12 * a + (2 * a + T) * c["hidden"] * size[c["type"]], "flops": 3 * a * c["hidden"]}
    N, K = c["N"], c["K"]
    if op == "linear":
        b = (a * K + hit * N * K) * 33 / 32 + a * N * size[c["out"]]
        b += (4 * hit * N if c["bias"] else 0) + a * N * 2 * (int(c["residual"]) + int(c["preact"]))
        return {"bytes": b, "flops": 2 * a * N * K}
    b = a * N * 2 * (1 if c["act"] == "none" else 2) + (a * K + hit * N * K) * 33 / 32 + a * K * 2 + E * N * K * 2 + E * N * 4
    return {"bytes": b, "flops": 4 * a * N * K}


# ---------------------------------------------------------------- from the definitions, in 64 bits

def _quant64(x, fmt):
    """Values of the codes and scales of fp64 [..., K]: the format's rounding written out (nearest, ties to even)."""
    emax, vmax, _, bits, emin = FMT[fmt]
    b = x.reshape(*x.shape[:-1], -1, 32)
    amax = b.abs().amax(-1, keepdim=True)
    X = torch.where(amax > 0, torch.floor(torch.log2(amax.clamp(min=2.0 ** -1000))), torch.full_like(amax, -300.0))
    X = torch.where((amax > 0) & (torch.exp2(X) > amax), X - 1, X)
    X = torch.where((amax > 0) & (torch.exp2(X + 1) <= amax), X + 1, X)
    X = (X - emax).clamp(-127, 127)
    v = b / torch.exp2(X)
    m = torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -60)))
    step = torch.exp2(m.clamp(min=emin) - bits)
    q = (torch.round(v / step) * step).clamp(-vmax, vmax)
    return q.reshape(x.shape), torch.exp2(X)[..., 0]


def _tiles64(s, fill):
    *lead, R, B = s.shape
    Rt, Bt = -(-R // 128), -(-B // 4)
    p = torch.full((*lead, Rt * 128, Bt * 4), fill, dtype=s.dtype, device=s.device)
    p[..., :R, :B] = s
    out = p.reshape(*lead, Rt, 4, 32, Bt, 4).movedim(-2, -5)
    return out.transpose(-2, -3).reshape(*lead, Bt, Rt, 512)


def _values64(codes, tiles, fmt, R, B):
    s = tiles.view(torch.float8_e8m0fnu).to(torch.float64)
    s = s.reshape(*tiles.shape[:-1], 32, 4, 4).transpose(-2, -3).movedim(-5, -2)
    s = s.reshape(*tiles.shape[:-3], tiles.shape[-2] * 128, tiles.shape[-3] * 4)[..., :R, :B]
    return codes.view(FMT[fmt][2]).to(torch.float64) * s.repeat_interleave(32, -1)


def _spans(s):
    return list(zip(s["starts"], s["lens"]))


def exact(case, seed):
    c = case
    op, T, k, E = c["op"], c["tokens"], c["topk"], c["experts"]
    if c["op"].startswith("linear") and (2 if op == "linear" else 4) * T * k * c["N"] * c["K"] > 6e12:
        return None
    s = _inputs(c, seed)
    rows = s["rows"]
    if op in ("dispatch", "combine", "combine_backward"):
        H = c["hidden"]
        flat = s["ids"].reshape(-1).tolist()
        count = [0] * E
        for e in flat:
            if 0 <= e < E:
                count[e] += 1
        at, nxt = 0, []
        for n in count:
            nxt.append(at)
            at += _up(n, ALIGN)
        pos = []
        for e in flat:
            pos.append(nxt[e] if 0 <= e < E else -1)
            if 0 <= e < E:
                nxt[e] += 1
        there = torch.tensor([p for p in pos if p >= 0], dtype=torch.long, device="cuda")
        a = torch.tensor([i for i, p in enumerate(pos) if p >= 0], dtype=torch.long, device="cuda")
    if op == "dispatch":
        x = s["x"].double()
        none = {n: None for n in ("offsets", "counts", "pos", "src")}
        if c["out"] in FMT:
            q, sc = _quant64(x, c["out"])
            codes = torch.zeros(rows, H, dtype=torch.float64, device="cuda")
            scale = torch.full((rows, H // 32), 2.0 ** -127, dtype=torch.float64, device="cuda")
            codes[there], scale[there] = q[a // k], sc[a // k]
            return {**none, "codes": codes, "scale": _tiles64(scale, 2.0 ** -127)}
        out = torch.zeros(rows, H, dtype=torch.float64, device="cuda")
        out[there] = x[a // k]
        return {**none, "out": out}
    if op == "combine":
        out = torch.zeros(T, H, dtype=torch.float64, device="cuda") if s["residual"] is None else s["residual"].double()
        w = s["weight"].double().reshape(-1) if c["weighted"] else torch.ones(T * k, dtype=torch.float64, device="cuda")
        for j in range(k):
            m = a % k == j
            out[a[m] // k] += w[a[m], None] * s["y"][there[m]].double()
        return out
    if op == "combine_backward":
        d = s["dout"].double()
        dy = torch.zeros(rows, H, dtype=torch.float64, device="cuda")
        dw = torch.zeros(T * k, dtype=torch.float64, device="cuda")
        for j in range(k):
            m = a % k == j
            dy[there[m]] = s["weight"].double().reshape(-1)[a[m], None] * d[a[m] // k]
            dw[a[m]] = (d[a[m] // k] * s["y"][there[m]].double()).sum(1)
        return {"dy": dy, "dweight": dw.reshape(T, k)}
    N, K = c["N"], c["K"]
    if op == "linear":
        x = _values64(s["x"], s["x_scale"], "e4m3", rows, K // 32)
        pre = torch.zeros(rows, N, dtype=torch.float64, device="cuda")
        out = torch.zeros(rows, N, dtype=torch.float64, device="cuda")
        for e, (o, n) in enumerate(_spans(s)):
            if n:
                z = x[o:o + n] @ _values64(s["w"][e], s["w_scale"][e], "e4m3", N, K // 32).t()
                z = z if s["bias"] is None else z + s["bias"][e].double()
                pre[o:o + n] = z
                out[o:o + n] = _act(z, c["act"]) + (0 if s["residual"] is None else s["residual"][o:o + n].double())
        # codes of the sums in 64 bits say little: a value near the middle of two codes rounds either way
        r = {"codes": None, "scale": None} if c["out"] in FMT else {"out": out}
        r = {**r, "preact": pre} if c["preact"] else r
        return r if any(v is not None for v in r.values()) else None
    up = _up(rows, 32)
    dz = torch.zeros(up, N, dtype=torch.float64, device="cuda")
    dbias = torch.zeros(E, N, dtype=torch.float64, device="cuda")
    for e, (o, n) in enumerate(_spans(s)):
        d = s["dy"][o:o + n].double()
        dz[o:o + n] = d if s["preact"] is None else d * _act_grad(s["preact"][o:o + n].double(), c["act"])
        dbias[e] = dz[o:o + n].sum(0)
    q, sc = _quant64(dz, c["grad"])
    by_row = q * sc.repeat_interleave(32, -1)
    q, sc = _quant64(dz.t().contiguous(), c["grad"])
    by_col = q * sc.repeat_interleave(32, -1)
    xt = _values64(s["x_t"], s["x_t_scale"], "e4m3", K, up // 32)
    dx = torch.zeros(rows, K, dtype=torch.float64, device="cuda")
    dw = torch.zeros(E, N, K, dtype=torch.float64, device="cuda")
    for e, (o, n) in enumerate(_spans(s)):
        if n:
            dx[o:o + n] = by_row[o:o + n] @ _values64(s["w_t"][e], s["w_t_scale"][e], "e4m3", K, N // 32).t()
            dw[e] = by_col[:, o:o + n] @ xt[:, o:o + n].t()
    return {"dbias": dbias, "dx": dx, "dw": dw}
