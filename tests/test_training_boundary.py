"""The training operators' C ABI without a GPU: workspace sizes and the refusal of invalid
arguments before any HIP call (nothing here launches a kernel)."""
import ctypes as C
import os

import pytest

import exact_inner_product_amd as mips

F32, BF16, FP8 = 0, 1, 2
OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3
vp = C.c_void_p


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(mips.LIB_PATH):
        from exact_inner_product_amd import build
        build.build()
    return mips.lib()


def test_lookup_refusals(L):
    def call(table=0x1000, dt=BF16, rows=10, d=16, stride=16, ids=0x2000, bits=32, t=5, out=0x3000):
        return L.mips_embedding_lookup(vp(table), dt, rows, d, stride, vp(ids), bits, t, 1.0, vp(out), None)

    assert call(t=0) == OK and call(t=0, table=None, ids=None, out=None) == OK
    for bad in (dict(table=None), dict(ids=None), dict(out=None), dict(rows=0), dict(d=0), dict(stride=15),
                dict(t=-1), dict(table=0x1001), dict(ids=0x2002), dict(out=0x3001), dict(bits=64, ids=0x2004)):
        assert call(**bad) == INVALID, bad
    for bad in (dict(dt=FP8), dict(bits=16), dict(d=16385, stride=16385)):
        assert call(**bad) == UNSUPPORTED, bad


def test_embedding_grad_refusals(L):
    def call(grad=0x1000, dt=BF16, t=5, d=16, stride=16, ids=0x2000, bits=32, rows=10, out=0x3000, odt=BF16,
             ostride=16, ws=0x10000, wsb=1 << 20):
        return L.mips_embedding_grad(vp(grad), dt, t, d, stride, vp(ids), bits, rows, 1.0, 0, vp(out), odt, ostride,
                                     vp(ws), wsb, None)

    for bad in (dict(grad=None), dict(ids=None), dict(out=None), dict(ws=None), dict(rows=0), dict(d=0), dict(t=-1),
                dict(stride=15), dict(ostride=15), dict(grad=0x1001), dict(ids=0x2002), dict(out=0x3001),
                dict(ws=0x10080), dict(odt=F32, out=0x3002)):
        assert call(**bad) == INVALID, bad
    for bad in (dict(dt=FP8), dict(dt=F32, odt=BF16), dict(bits=8), dict(rows=1 << 31), dict(t=(1 << 30) + 1),
                dict(d=16385, stride=16385, ostride=16385)):
        assert call(**bad) == UNSUPPORTED, bad
    assert call(wsb=256) == WORKSPACE


def test_embedding_grad_workspace(L):
    size = L.mips_embedding_grad_workspace_size
    assert size(-1, 10, 16) == 0 and size(5, 0, 16) == 0 and size(5, 10, 0) == 0
    assert size((1 << 30) + 1, 10, 16) == 0 and size(5, 1 << 31, 16) == 0 and size(5, 10, 16385) == 0
    assert size(0, 10, 16) > 0
    last = 0
    for t in (1, 8, 100, 8192, 8193, 100000, 1 << 20):
        n = size(t, 1000, 64)
        assert n >= 8 * t and n >= last
        last = n


def test_clip_refusals(L):
    n = 3

    def call(ptrs=(0x1000, 0x2000, 0x3000), outs=(0x1000, 0x2000, 0x3000), counts=(4, 0, 7), codes=(F32, BF16, BF16),
             k=n, mx=1.0, norm=0x4000, ws=0x10000, wsb=1 << 20):
        return L.mips_clip_grad_norm((vp * n)(*ptrs), (vp * n)(*outs), (C.c_int64 * n)(*counts),
                                     (C.c_int32 * n)(*codes), k, mx, vp(norm), vp(ws), wsb, None)

    for bad in (dict(ptrs=(None, 0x2000, 0x3000)), dict(outs=(0x1000, 0x2000, None)), dict(counts=(4, -1, 7)),
                dict(k=0), dict(mx=-1.0), dict(mx=float("nan")), dict(norm=None), dict(ws=None), dict(ws=0x10008),
                dict(ptrs=(0x1002, 0x2000, 0x3000)), dict(outs=(0x1000, 0x2000, 0x3001)),
                dict(counts=(4, 0, (1 << 38) + 1))):
        assert call(**bad) == INVALID, bad
    assert call(codes=(F32, BF16, FP8)) == UNSUPPORTED
    assert call(wsb=256) == WORKSPACE
    assert L.mips_clip_grad_norm(None, None, None, None, 1, 1.0, vp(0x4000), vp(0x10000), 1 << 20, None) == INVALID


def test_clip_workspace(L):
    size = L.mips_clip_workspace_size
    assert size(0) == 0 and size(-1) == 0
    assert size(1) >= 1024 * 8
    assert 2048 * 8 <= size(1000) and 16 * 8 * 1563 <= size(100000)
