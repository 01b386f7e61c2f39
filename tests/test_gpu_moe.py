"""The mixture-of-experts row operators against their 64-bit definitions.

Tolerances: whole numbers, copies and quantised rows are exact.  A combine sums
at most topk + 1 terms in fp32 and rounds once: (topk + 2) half-ulps of the sum
of magnitudes plus the output's rounding.  dy is one product and one rounding.
dweight sums `hidden` products in some fixed order: at most hidden + 1 half-ulps
of the sum of magnitudes.
"""
import numpy as np
import pytest
import torch

from all_mxfp8_block_gb300 import inputs, mxa2a
from tests import operators_ref as R

pytestmark = pytest.mark.gpu

TYPE = {"bf16": mxa2a.MXA2A_TYPE_BF16, "f16": mxa2a.MXA2A_TYPE_F16, "f32": mxa2a.MXA2A_TYPE_F32,
        "e4m3": mxa2a.MXA2A_TYPE_E4M3, "e5m2": mxa2a.MXA2A_TYPE_E5M2}


def run_sort(ids, experts, align, rows=None, stream=None):
    T, k = ids.shape
    rows = mxa2a.mxa2a_moe_rows(T, k, experts, align) if rows is None else rows
    d = {"ids": torch.from_numpy(ids).cuda(), "rows": rows}
    for name, n in (("offsets", experts + 1), ("counts", experts), ("pos", max(1, T * k)), ("src", max(1, rows))):
        d[name] = torch.full((n,), -7, dtype=torch.int32, device="cuda")
    if stream is not None:
        stream.wait_stream(torch.cuda.current_stream())
    mxa2a.mxa2a_moe_sort(T, k, experts, align, rows, d["ids"], d["offsets"], d["counts"], d["pos"], d["src"], stream)
    return d


def routed(T, k, E, seed, align=32, drop=0.0, only=None):
    ids = R.routing(T, k, E, seed, drop, only)
    return ids, run_sort(ids, E, align)


SORTS = [(1, 1, 1, 1), (1, 8, 64, 32), (3, 2, 1024, 32), (33, 4, 7, 1), (509, 8, 64, 32), (512, 8, 1000, 128),
         (513, 8, 9, 24), (4097, 1, 3, 32), (20000, 4, 256, 32), (30011, 8, 1024, 16)]


@pytest.mark.parametrize("T,k,E,align", SORTS)
@pytest.mark.parametrize("drop", [0.0, 0.2])
def test_sort(T, k, E, align, drop):
    ids = R.routing(T, k, E, T + k, drop) if E >= k else np.zeros((T, k), np.int32)
    d = run_sort(ids, E, align)
    offsets, counts, pos, src = R.sort(ids, E, align, d["rows"])
    assert (d["offsets"].cpu().numpy() == offsets).all()
    assert (d["counts"].cpu().numpy() == counts).all()
    assert (d["pos"].cpu().numpy() == pos.reshape(-1)).all()
    assert (d["src"].cpu().numpy() == src).all()


def test_sort_of_equal_and_foreign_ids():
    # every assignment to one expert; ids past the range and negative ones go nowhere; repeated experts in a token
    ids = np.full((1000, 4), 5, np.int32)
    ids[::3, 1] = 17
    ids[::5, 2] = -2147483648
    ids[::7, 3] = 2147483647
    d = run_sort(ids, 9, 32)
    offsets, counts, pos, src = R.sort(ids, 9, 32, d["rows"])
    assert (d["offsets"].cpu().numpy() == offsets).all() and (d["counts"].cpu().numpy() == counts).all()
    assert (d["pos"].cpu().numpy() == pos.reshape(-1)).all() and (d["src"].cpu().numpy() == src).all()


def test_sort_without_tokens_or_takers():
    d = run_sort(np.zeros((0, 2), np.int32), 4, 32, rows=96)
    assert (d["offsets"].cpu().numpy() == 0).all() and (d["counts"].cpu().numpy() == 0).all()
    assert (d["src"].cpu().numpy() == -1).all()
    d = run_sort(np.full((40, 2), -1, np.int32), 4, 32)
    assert (d["offsets"].cpu().numpy() == 0).all() and (d["pos"].cpu().numpy() == -1).all()
    assert (d["src"].cpu().numpy() == -1).all()


def test_sort_optional_src_and_other_stream():
    ids = R.routing(700, 3, 20, 4)
    s = torch.cuda.Stream()
    d = run_sort(ids, 20, 32, stream=s)
    s.synchronize()
    pos = d["pos"].clone()
    mxa2a.mxa2a_moe_sort(700, 3, 20, 32, d["rows"], d["ids"], d["offsets"], d["counts"], d["pos"], None)
    assert (pos == d["pos"]).all()
    assert (pos.cpu().numpy() == R.sort(ids, 20, 32, d["rows"])[2].reshape(-1)).all()


def make_rows(n, H, dtype, seed, pad=0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(n, H + pad, generator=g) * torch.exp2(torch.randint(-9, 10, (n, 1), generator=g).float())
    return x.to(R.DTYPE[dtype]).cuda()


@pytest.mark.parametrize("T,k,E,H,dtype,pad", [(1, 8, 64, 256, "bf16", 0), (37, 3, 5, 1, "bf16", 0), (37, 3, 5, 129, "f16", 3),
                                               (200, 2, 16, 1000, "f32", 8), (65, 1, 1, 6, "bf16", 2), (301, 4, 8, 4096, "bf16", 0)])
def test_dispatch_copy(T, k, E, H, dtype, pad):
    ids, d = routed(T, k, E, H, drop=0.1)
    x = make_rows(T, H, dtype, H, pad)
    out = torch.full((d["rows"], H), -3.0, dtype=R.DTYPE[dtype], device="cuda")
    mxa2a.mxa2a_moe_dispatch(T, k, E, H, d["rows"], x, TYPE[dtype], H + pad, d["pos"], d["offsets"], d["counts"], out, TYPE[dtype])
    _, _, _, src = R.sort(ids, E, 32, d["rows"])
    used = int(d["offsets"][E])
    want = torch.zeros(used, H, dtype=R.DTYPE[dtype])
    have = src[:used] >= 0
    want[torch.from_numpy(have)] = x.cpu()[:, :H][torch.from_numpy(src[:used][have] // k)]
    assert torch.equal(out[:used].cpu(), want)
    assert (out[used:] == -3.0).all()          # rows past the last segment are left alone


@pytest.mark.parametrize("T,k,E,H,dtype,fmt", [(1, 8, 64, 4096, "bf16", "e4m3"), (77, 3, 5, 32, "f16", "e5m2"), (50, 2, 4, 160, "f32", "e4m3"),
                                               (300, 4, 32, 1056, "bf16", "e4m3"), (129, 1, 2, 2016, "f32", "e5m2")])
def test_dispatch_quantised(T, k, E, H, dtype, fmt):
    ids, d = routed(T, k, E, H + 1, drop=0.1)
    x = make_rows(T, H, dtype, H)
    x[0, :32] = 0                              # a block of zeros
    x[T // 2, -1] = 0.0 if dtype == "f16" else 1e-30
    out = torch.full((d["rows"], H), 0x55, dtype=torch.uint8, device="cuda")
    sc = torch.full((-(-H // 128), -(-d["rows"] // 128), 512), 0x55, dtype=torch.uint8, device="cuda")
    mxa2a.mxa2a_moe_dispatch(T, k, E, H, d["rows"], x, TYPE[dtype], H, d["pos"], d["offsets"], d["counts"], out, TYPE[fmt], sc)
    _, _, _, src = R.sort(ids, E, 32, d["rows"])
    used = int(d["offsets"][E])
    rows = np.zeros((used, H))
    have = src[:used] >= 0
    rows[have] = R.f64(x)[src[:used][have] // k]
    q, X = R.quant(rows, fmt)
    assert (R.decode(out, fmt)[:used] == q).all()
    assert (R.untile(sc.cpu().numpy(), used, H // 32) == X + 127).all()
    codes, scales = inputs.quantize_mx_rows(x.float().cpu(), fmt)     # the library's own input quantiser
    assert (out.cpu()[:used][torch.from_numpy(have)] == codes[torch.from_numpy(src[:used][have] // k)]).all()
    assert (out[used:] == 0x55).all()


def test_dispatch_quantised_infinities():
    ids, d = routed(3, 1, 1, 0)
    x = make_rows(3, 96, "bf16", 1)
    x[1, 40], x[2, 3] = float("inf"), float("nan")
    out = torch.zeros(d["rows"], 96, dtype=torch.uint8, device="cuda")
    sc = torch.zeros(1, 1, 512, dtype=torch.uint8, device="cuda")
    mxa2a.mxa2a_moe_dispatch(3, 1, 1, 96, d["rows"], x, 0, 96, d["pos"], d["offsets"], d["counts"], out, TYPE["e4m3"], sc)
    s = R.untile(sc.cpu().numpy(), 3, 3)
    assert (s == 255).tolist() == [[False] * 3, [False, True, False], [True, False, False]]
    v = R.decode(out, "e4m3")[:3].reshape(3, 3, 32)
    assert np.isnan(v[1, 1]).all() and np.isnan(v[2, 0]).all() and np.isfinite(v[0]).all() and np.isfinite(v[1, [0, 2]]).all()


COMBINES = [(1, 1, 1, 8, "bf16"), (8, 8, 64, 4096, "bf16"), (100, 3, 7, 33, "f16"), (100, 3, 7, 2048, "f32"), (257, 4, 16, 7168, "bf16"),
            (65, 9, 40, 520, "bf16"), (31, 64, 80, 130, "f32")]


@pytest.mark.parametrize("T,k,E,H,dtype", COMBINES)
@pytest.mark.parametrize("weighted,residual", [(True, True), (False, False)])
def test_combine(T, k, E, H, dtype, weighted, residual):
    ids, d = routed(T, k, E, 3 * H, drop=0.15)
    y = make_rows(d["rows"], H, dtype, 5)
    _, _, pos, src = R.sort(ids, E, 32, d["rows"])
    y[torch.from_numpy(src < 0).cuda()] = float("nan")     # padding and unused rows must not be read into a sum
    w = torch.rand(T, k).cuda() if weighted else None
    res = make_rows(T, H, dtype, 6) if residual else None
    out = torch.empty(T, H, dtype=R.DTYPE[dtype], device="cuda")
    mxa2a.mxa2a_moe_combine(T, k, H, d["rows"], y, TYPE[dtype], d["pos"], w, res, out)
    wv = np.ones((T, k)) if w is None else R.f64(w)
    ref = np.zeros((T, H)) if res is None else R.f64(res)
    size = np.abs(ref)
    yv = R.f64(y)
    for j in range(k):
        ok = pos[:, j] >= 0
        t = wv[ok, j, None] * yv[pos[ok, j]]
        ref[ok] += t
        size[ok] += np.abs(t)
    bound = (k + 2) * R.F32_EPS * size * 1.01
    R.check(out, ref, bound + R.ROUND[dtype] * (np.abs(ref) + bound) + R.TINY[dtype])
    again = torch.empty_like(out)
    mxa2a.mxa2a_moe_combine(T, k, H, d["rows"], y, TYPE[dtype], d["pos"], w, res, again)
    assert torch.equal(out, again)


def test_combine_of_tokens_without_experts():
    pos = torch.full((5, 2), -1, dtype=torch.int32, device="cuda")
    res = make_rows(5, 64, "bf16", 2)
    out = torch.full((5, 64), 9.0, dtype=torch.bfloat16, device="cuda")
    mxa2a.mxa2a_moe_combine(5, 2, 64, 0, None, 0, pos, None, res, out)
    assert torch.equal(out, res)
    mxa2a.mxa2a_moe_combine(5, 2, 64, 0, None, 0, pos, None, None, out)
    assert (out == 0).all()


@pytest.mark.parametrize("T,k,E,H,dtype", COMBINES)
def test_combine_backward(T, k, E, H, dtype):
    ids, d = routed(T, k, E, 5 * H, drop=0.15)
    y, dout = make_rows(d["rows"], H, dtype, 7), make_rows(T, H, dtype, 8)
    _, _, pos, src = R.sort(ids, E, 32, d["rows"])
    y[torch.from_numpy(src < 0).cuda()] = float("nan")
    w = torch.rand(T, k).cuda()
    dy = torch.full((d["rows"], H), 5.0, dtype=R.DTYPE[dtype], device="cuda")
    dw = torch.full((T, k), 5.0, device="cuda")
    mxa2a.mxa2a_moe_combine_backward(T, k, E, H, d["rows"], dout, TYPE[dtype], y, d["pos"], d["offsets"], d["counts"], w, dy, dw)
    used = int(d["offsets"][E])
    ref, refw, size = np.zeros((used, H)), np.zeros((T, k)), np.zeros((T, k))
    dv, yv, wv = R.f64(dout), R.f64(y), R.f64(w)
    for j in range(k):
        ok = pos[:, j] >= 0
        ref[pos[ok, j]] = wv[ok, j, None] * dv[ok]
        refw[ok, j] = (dv[ok] * yv[pos[ok, j]]).sum(1)
        size[ok, j] = np.abs(dv[ok] * yv[pos[ok, j]]).sum(1)
    R.check(dy[:used], ref, (R.F32_EPS + R.ROUND[dtype]) * 1.01 * np.abs(ref) + R.TINY[dtype], "dy")
    R.check(dw, refw, (H + 1) * R.F32_EPS * 1.01 * size, "dweight")
    assert (dy[used:] == 5.0).all()


def test_combine_gradient_against_differences():
    # out = sum_j w_j y_j: linear in y and in w, so differences of the 64-bit form are the gradient up to rounding
    T, k, E, H = 9, 3, 6, 40
    ids, d = routed(T, k, E, 1)
    _, _, pos, _ = R.sort(ids, E, 32, d["rows"])
    y, dout, w = make_rows(d["rows"], H, "f32", 1), make_rows(T, H, "f32", 2), torch.rand(T, k).cuda()
    dy, dw = torch.zeros_like(y), torch.zeros_like(w)
    mxa2a.mxa2a_moe_combine_backward(T, k, E, H, d["rows"], dout, 2, y, d["pos"], d["offsets"], d["counts"], w, dy, dw)

    def loss(yv, wv):
        return (R.f64(dout) * (wv[..., None] * yv[pos]).sum(1)).sum()

    rng = np.random.default_rng(0)
    yv, wv = R.f64(y), R.f64(w)
    for _ in range(20):
        t, j, h = rng.integers(T), rng.integers(k), rng.integers(H)
        e = 1e-3
        a, b = wv.copy(), wv.copy()
        a[t, j] += e
        b[t, j] -= e
        num = (loss(yv, a) - loss(yv, b)) / (2 * e)
        assert abs(float(dw[t, j]) - num) <= 1e-4 * np.abs(R.f64(dout)[t] * yv[pos[t, j]]).sum()
        a, b = yv.copy(), yv.copy()
        a[pos[t, j], h] += e
        b[pos[t, j], h] -= e
        num = (loss(a, wv) - loss(b, wv)) / (2 * e)
        assert abs(float(dy[pos[t, j], h]) - num) <= 1e-4 * abs(num) + 1e-6 * np.abs(R.f64(dout)).max()


def test_dispatch_gradient_is_combine_without_weights():
    T, k, E, H = 70, 4, 9, 256
    ids, d = routed(T, k, E, 2, drop=0.1)
    g = make_rows(d["rows"], H, "f32", 3)
    dx = torch.empty(T, H, device="cuda")
    mxa2a.mxa2a_moe_combine(T, k, H, d["rows"], g, 2, d["pos"], None, None, dx)
    _, _, pos, _ = R.sort(ids, E, 32, d["rows"])
    ref, size = np.zeros((T, H)), np.zeros((T, H))
    for j in range(k):
        ok = pos[:, j] >= 0
        ref[ok] += R.f64(g)[pos[ok, j]]
        size[ok] += np.abs(R.f64(g)[pos[ok, j]])
    R.check(dx, ref, (k + 2) * R.F32_EPS * 1.01 * size)


def test_rows_out_of_range_are_not_touched():
    # pos, offsets and counts that point past the buffers: skipped by the kernels' own checks
    T, k, E, H, rows = 4, 2, 3, 64, 64
    x = make_rows(T, H, "bf16", 1)
    pos = torch.tensor([0, 64, 1, 1 << 30, 2, -5, 3, 63], dtype=torch.int32, device="cuda")
    offsets = torch.tensor([0, 32, 64, 4096], dtype=torch.int32, device="cuda")
    counts = torch.tensor([4, 31, 1], dtype=torch.int32, device="cuda")
    out = torch.full((rows + 64, H), 7.0, dtype=torch.bfloat16, device="cuda")
    mxa2a.mxa2a_moe_dispatch(T, k, E, H, rows, x, 0, H, pos, offsets, counts, out, 0)
    assert (out[rows:] == 7.0).all()
    for r, t in ((0, 0), (1, 1), (2, 2), (3, 3)):
        assert torch.equal(out[r], x[t])
    res = torch.empty(T, H, dtype=torch.bfloat16, device="cuda")
    mxa2a.mxa2a_moe_combine(T, k, H, rows, out, 0, pos, None, None, res)
    assert torch.equal(res[1], x[1])


def test_graph_capture():
    T, k, E, H = 64, 4, 16, 512
    ids, d = routed(T, k, E, 6)
    x = make_rows(T, H, "bf16", 1)
    y = torch.zeros(d["rows"], H, dtype=torch.bfloat16, device="cuda")
    out = torch.zeros(T, H, dtype=torch.bfloat16, device="cuda")

    def step():
        mxa2a.mxa2a_moe_sort(T, k, E, 32, d["rows"], d["ids"], d["offsets"], d["counts"], d["pos"], d["src"])
        mxa2a.mxa2a_moe_dispatch(T, k, E, H, d["rows"], x, 0, H, d["pos"], d["offsets"], d["counts"], y, 0)
        mxa2a.mxa2a_moe_combine(T, k, H, d["rows"], y, 0, d["pos"], None, None, out)

    step()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    x.copy_(make_rows(T, H, "bf16", 9))
    d["ids"].copy_(torch.from_numpy(R.routing(T, k, E, 77)))
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, (x.float() * k).to(torch.bfloat16))
