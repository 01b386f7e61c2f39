"""Refusals of the mixture-of-experts and linear-layer calls: decided on the host
before any launch, so they need no GPU (the pointers are never read)."""
import pytest

from all_mxfp8_block_gb300 import mxa2a as m
from all_mxfp8_block_gb300 import build as mxbuild

P = 4096          # an aligned address that no refused call reads


@pytest.fixture(scope="module")
def lib():
    mxbuild.build()
    return m.load()


def test_moe_rows(lib):
    r = m.mxa2a_moe_rows
    assert r(1, 8, 64, 32) == 256
    assert r(4096, 4, 32, 32) == 17376
    assert r(0, 1, 1, 32) == 0
    assert r(3, 2, 4, 1) == 6
    assert r(5, 1, 2, 24) == 72                 # 5 + 2 * 23 rounded up to 24
    for bad in ((-1, 1, 1, 1), (1, 0, 1, 1), (1, 65, 1, 1), (1, 1, 0, 1), (1, 1, 1025, 1), (1, 1, 1, 0), (1, 1, 1, 1025), (1 << 26, 2, 1, 1)):
        assert r(*bad) == -1, bad


def test_scale_tiles_bytes(lib):
    b = m.mxa2a_scale_tiles_bytes
    assert b(1, 32) == 512 and b(129, 128) == 1024 and b(0, 128) == 0 and b(300, 1056) == 3 * 9 * 512 and b(-1, 32) == -1


def sort(lib, T=4, k=2, E=3, align=32, rows=1 << 20, expert=P, offsets=P, counts=P, pos=P, src=P):
    return lib.mxa2a_moe_sort(T, k, E, align, rows, expert, offsets, counts, pos, src, None)


def test_sort_refusals(lib):
    shape, null, mis = m.MXA2A_ERR_INVALID_SHAPE, m.MXA2A_ERR_NULL_PTR, m.MXA2A_ERR_MISALIGNED
    assert sort(lib, T=-1) == shape and sort(lib, k=0) == shape and sort(lib, E=0) == shape and sort(lib, align=0) == shape
    assert sort(lib, rows=95) == shape          # 8 assignments to 3 experts may need 8 + 3 * 31 -> 128 rows
    assert sort(lib, rows=1 << 31) == shape
    assert sort(lib, expert=None) == null and sort(lib, offsets=None) == null and sort(lib, counts=None) == null and sort(lib, pos=None) == null
    assert sort(lib, expert=P + 2) == mis and sort(lib, src=P + 1) == mis


def dispatch(lib, T=4, k=2, E=3, H=64, rows=128, x=P, xt=0, ldx=64, pos=P, off=P, cnt=P, out=P, ot=3, osc=P):
    return lib.mxa2a_moe_dispatch(T, k, E, H, rows, x, xt, ldx, pos, off, cnt, out, ot, osc, None)


def test_dispatch_refusals(lib):
    shape, null, mis, opt = m.MXA2A_ERR_INVALID_SHAPE, m.MXA2A_ERR_NULL_PTR, m.MXA2A_ERR_MISALIGNED, m.MXA2A_ERR_INVALID_OPTION
    assert dispatch(lib, xt=3) == opt and dispatch(lib, ot=5 + 1) == opt and dispatch(lib, xt=0, ot=2) == opt
    assert dispatch(lib, H=48, ldx=48) == shape and dispatch(lib, ldx=63) == shape and dispatch(lib, H=0) == shape and dispatch(lib, rows=-1) == shape
    assert dispatch(lib, osc=None) == null and dispatch(lib, out=None) == null and dispatch(lib, x=None) == null and dispatch(lib, off=None) == null
    assert dispatch(lib, x=P + 8) == mis and dispatch(lib, ldx=68) == mis and dispatch(lib, out=P + 8) == mis and dispatch(lib, osc=P + 2) == mis
    assert dispatch(lib, ot=0, x=P + 1) == mis


def test_combine_refusals(lib):
    f = lambda T=4, k=2, H=64, rows=128, y=P, t=0, pos=P, w=P, res=P, out=P: lib.mxa2a_moe_combine(T, k, H, rows, y, t, pos, w, res, out, None)  # noqa: E731
    shape, null, mis, opt = m.MXA2A_ERR_INVALID_SHAPE, m.MXA2A_ERR_NULL_PTR, m.MXA2A_ERR_MISALIGNED, m.MXA2A_ERR_INVALID_OPTION
    assert f(t=3) == opt and f(T=-1) == shape and f(k=65) == shape and f(H=0) == shape
    assert f(y=None) == null and f(pos=None) == null and f(out=None) == null
    assert f(y=P + 1) == mis and f(t=2, res=P + 2) == mis and f(w=P + 2) == mis
    g = lambda T=4, k=2, E=3, H=64, rows=128, d=P, t=0, y=P, pos=P, off=P, cnt=P, w=P, dy=P, dw=P: lib.mxa2a_moe_combine_backward(  # noqa: E731
        T, k, E, H, rows, d, t, y, pos, off, cnt, w, dy, dw, None)
    assert g(t=4) == opt and g(E=0) == shape and g(dw=None) == null and g(dy=None) == null and g(cnt=None) == null and g(dw=P + 2) == mis


def test_quantize_refusals(lib):
    f = lambda x=P, t=0, ldx=64, G=1, r=8, c=64, fmt=3, q=P, s=P, qt=None, st=None: lib.mxa2a_quantize(x, t, ldx, G, r, c, fmt, q, s, qt, st, None)  # noqa: E731
    shape, null, mis, opt = m.MXA2A_ERR_INVALID_SHAPE, m.MXA2A_ERR_NULL_PTR, m.MXA2A_ERR_MISALIGNED, m.MXA2A_ERR_INVALID_OPTION
    assert f(t=4) == opt and f(fmt=0) == opt and f(c=40) == shape and f(ldx=32) == shape and f(r=-1) == shape
    assert f(x=None) == null and f(s=None) == null and f(q=None, s=None) == null and f(qt=P) == null
    assert f(x=P + 2) == mis and f(ldx=65) == mis and f(q=P + 4) == mis and f(s=P + 1) == mis
    t = lambda s=P, G=1, r=8, c=64, o=P: lib.mxa2a_scale_tiles(s, G, r, c, o, None)  # noqa: E731
    assert t(c=33) == shape and t(s=None) == null and t(o=None) == null and t(o=P + 2) == mis


def test_linear_rules(lib):
    v, ok, bad = m.mxa2a_linear_validate, m.MXA2A_OK, m.MXA2A_ERR_INVALID_SHAPE
    assert v(1, 1, 32, 32) == ok and v(32, 17376, 2048, 7168) == ok and v(1024, 65536, 2048, 1024) == ok
    for a in ((0, 1, 32, 32), (1025, 1, 32, 32), (1, 0, 32, 32), (1, (1 << 22) + 1, 32, 32), (1, 1, 48, 32), (1, 1, 32, 0), (1, 1, 32, (1 << 20) + 32),
              (1024, 1 << 22, 1 << 20, 1 << 20)):
        assert v(*a) == bad, a
    assert not lib.mxa2a_linear_create(1, 1, 33, 32, 0) and m.mxa2a_last_error() == bad


def test_linear_null_plan(lib):
    null = m.MXA2A_ERR_NULL_PTR
    assert lib.mxa2a_linear_run(None, 1, P, P, P, P, P, 0, None, None, None, None, 0, None, None, None) == null
    assert lib.mxa2a_linear_backward(None, 1, P, P, 0, 3, P, P, P, P, P, P, 0, P, None, None, None) == null
    assert lib.mxa2a_linear_get_status(None, None) == null and lib.mxa2a_linear_set_option(None, 1, 1) == null
    assert lib.mxa2a_linear_get_option(None, 1, None) == null
    lib.mxa2a_linear_destroy(None)
