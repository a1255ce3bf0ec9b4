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
    assert call(wsb=128) == WORKSPACE
    assert call(t=20000, wsb=256) == WORKSPACE


def test_embedding_grad_workspace(L):
    size = L.mips_embedding_grad_workspace_size
    assert size(-1, 10, 16) == 0 and size(5, 0, 16) == 0 and size(5, 10, 0) == 0
    assert size((1 << 30) + 1, 10, 16) == 0 and size(5, 1 << 31, 16) == 0 and size(5, 10, 16385) == 0
    assert size(0, 10, 16) > 0
    last = 0
    for t in (1, 8, 100, 8192, 8193, 100000, 1 << 20):
        n = size(t, 1000, 64)
        assert n >= (8 * t if t > 16384 else 1) and n >= last  # (few tokens are sorted in LDS)
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


def test_logprobs_refusals(L):
    def call(q=0x1000, qs=64, b=5, items=0x2000, layout=0, istr=64, n=100, d=64, dt=BF16, bias=None, ex=None, xw=0,
             scale=1.0, ids=0x3000, bits=32, g=1, k=2, lp=0x4000, lse=0x5000, ent=0x6000, ai=0x7000, al=0x8000,
             ws=0x10000, wsb=1 << 30):
        return L.mips_logprobs(vp(q), qs, b, vp(items), layout, istr, n, d, dt, vp(bias), vp(ex), xw, scale, vp(ids), bits,
                               g, k, vp(lp), vp(lse), vp(ent), vp(ai), vp(al), vp(ws), wsb, None)

    for bad in (dict(q=None), dict(items=None), dict(lse=None), dict(ws=None), dict(ids=None), dict(lp=None),
                dict(ai=None), dict(al=None), dict(b=0), dict(n=0), dict(d=0), dict(g=-1), dict(k=-1), dict(layout=2),
                dict(q=0x1008), dict(items=0x2008), dict(qs=56), dict(istr=68), dict(qs=65), dict(istr=1 << 25),
                dict(ws=0x10010), dict(bias=0x2), dict(ex=0x2), dict(lse=0x5002), dict(ent=0x6001), dict(xw=-1),
                dict(xw=4), dict(ex=0x9000, xw=3), dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")),
                dict(scale=float("inf")), dict(scale=1e7), dict(bits=64, ids=0x3004)):
        assert call(**bad) == INVALID, bad
    for bad in (dict(dt=FP8), dict(d=60, qs=64), dict(d=264, qs=264, istr=264), dict(dt=F32, d=132, qs=132, istr=132),
                dict(n=(1 << 31)), dict(b=mips.B_MAX + 1), dict(k=65), dict(bits=16), dict(layout=1, d=24)):
        assert call(**bad) == UNSUPPORTED, bad
    assert call(wsb=16) == WORKSPACE


def test_logprobs_workspace(L):
    size = L.mips_logprobs_workspace_size
    assert size(0, 10, 64, BF16, 0) == 0 and size(1, 0, 64, BF16, 0) == 0 and size(1, 10, 60, BF16, 0) == 0
    assert size(1, 10, 64, FP8, 0) == 0 and size(1, 10, 64, BF16, 65) == 0 and size(1, 10, 64, BF16, -1) == 0
    assert 0 < size(1, 10, 64, BF16, 0) <= size(1, 10, 64, BF16, 5)
    # tile maxima: about 4 bytes per query and 32 or 64 items, in batches of queries beyond 1 GiB
    assert size(100, 1000000, 128, BF16, 1) >= 100 * 1000000 // 32 * 4
    assert size(100000, 10000000, 128, BF16, 1) < 2 << 30


def test_logprobs_backward_refusals(L):
    def call(q=0x1000, qs=64, b=5, items=0x2000, istr=64, n=100, d=64, dt=BF16, bias=None, ex=None, xw=0, scale=1.0,
             ids=0x3000, bits=32, g=1, lse=0x5000, ent=0x6000, gl=0x7000, ge=0x8000, dq=0x9000, di=0xA000, db=None,
             ws=0x10000, wsb=1 << 30):
        return L.mips_logprobs_backward(vp(q), qs, b, vp(items), istr, n, d, dt, vp(bias), vp(ex), xw, scale, vp(ids),
                                        bits, g, vp(lse), vp(ent), vp(gl), vp(ge), vp(dq), vp(di), vp(db), vp(ws), wsb,
                                        None)

    for bad in (dict(q=None), dict(items=None), dict(lse=None), dict(ws=None), dict(ids=None), dict(gl=None),
                dict(ent=None), dict(dq=None, di=None), dict(b=0), dict(n=0), dict(d=0), dict(g=-1), dict(q=0x1008),
                dict(items=0x2008), dict(qs=56), dict(istr=68), dict(dq=0x9008), dict(di=0xA008), dict(db=0x2),
                dict(ws=0x10010), dict(gl=0x7002), dict(ge=0x8002), dict(xw=-1), dict(xw=4), dict(ex=0x9000, xw=3),
                dict(scale=0.0), dict(scale=float("nan"))):
        assert call(**bad) == INVALID, bad
    for bad in (dict(dt=FP8), dict(d=60), dict(d=264, qs=264, istr=264), dict(dt=F32, d=132, qs=132, istr=132),
                dict(n=(1 << 30) + 1), dict(g=65), dict(bits=8), dict(b=mips.B_MAX + 1)):
        assert call(**bad) == UNSUPPORTED, bad
    assert call(wsb=256) == WORKSPACE
    size = L.mips_logprobs_backward_workspace_size
    assert size(0, 10, 64, BF16, 1) == 0 and size(5, 10, 64, BF16, 65) == 0 and size(5, 10, 60, BF16, 1) == 0
    assert size(5, 10, 64, BF16, 1) > 0


def test_limits_match_the_binding():
    import re
    text = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "mips.h")).read()
    limits = dict(re.findall(r"#define (MIPS_\w+_MAX) (\d+)", text))
    assert int(limits["MIPS_ALTERNATIVES_MAX"]) == mips.ALTERNATIVES_MAX
    assert int(limits["MIPS_TARGETS_MAX"]) == mips.TARGETS_MAX


def test_the_stream_handle_has_a_public_source(monkeypatch):
    """Without torch's internal function the handle comes from the current stream's object."""
    import types

    import torch

    from exact_inner_product_amd import training
    asked = []

    def current_stream(device):
        asked.append(device)
        return types.SimpleNamespace(cuda_stream=77)

    monkeypatch.setattr(torch.cuda, "current_stream", current_stream)
    monkeypatch.setattr(training, "_raw_stream", None)
    device = torch.device("cuda", 0)
    assert training._stream(device) == 77 and asked == [device]
    monkeypatch.setattr(training, "_raw_stream", lambda index: 100 + index)
    assert training._stream(device) == 100 and len(asked) == 1
