"""The C ABI of the operators over histories without a GPU: sizes, and the refusal of invalid
arguments before any HIP call (nothing here launches a kernel); the generator's known answers."""
import ctypes as C
import os
import re

import numpy as np
import pytest
import torch

import exact_inner_product_amd as mips
from exact_inner_product_amd.histories import _Rows, _Sequences
from tests import histories_check as hc

F32, BF16, FP8 = 0, 1, 2
OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3
vp = C.c_void_p


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(mips.LIB_PATH):
        from exact_inner_product_amd import build
        build.build()
    return mips.lib()


def seq(b=4, bits=0, t=50, n=0, offsets=None, lengths=None):
    return _Sequences(b, bits, t, n, offsets, lengths)


def rows(p=0x1000, row=64, step=64 * 50):
    return _Rows(p, row, step)


BAD_SEQ = (dict(b=0), dict(t=0), dict(t=-1), dict(bits=32, offsets=0x100, lengths=0x200), dict(bits=32, offsets=0x102, n=5),
           dict(bits=64, lengths=0x104), dict(bits=32, offsets=0x100, n=-1))
NO_SEQ = (dict(bits=16, lengths=0x100), dict(bits=0, offsets=0x100, n=5), dict(t=(1 << 30) + 1), dict(b=1 << 20, t=1 << 11),
          dict(b=mips.B_MAX + 1, t=1), dict(bits=32, offsets=0x100, n=(1 << 30) + 1))


def test_scan_sizes(L):
    tiles = lambda q, d, t=BF16: L.mips_gated_scan_carries(C.byref(q), d, t)  # noqa: E731
    size = lambda q, d, t=BF16: L.mips_gated_scan_workspace_size(C.byref(q), d, t)  # noqa: E731
    for q, n in ((seq(4096, t=127), 4096 * 127), (seq(1, t=1), 1), (seq(2, t=1280), 2560), (seq(2, 32, 0, 10, 0x100), 10),
                 (seq(2, 32, 0, 100000, 0x100), 100000)):
        for d in (1, 128, 16384):
            assert n <= 8 * tiles(q, d) and n <= 4 * tiles(q, d, F32)   # a state for every 8 or 4 rows at least
    assert size(seq(4096, t=127), 128) == 0 and size(seq(4096, t=127), 128, F32) == 0  # whole sequences in a tile
    for bad in BAD_SEQ + NO_SEQ:
        assert tiles(seq(**bad), 64) == -1 and size(seq(**bad), 64) == 0, bad
    assert tiles(seq(), 0) == -1 and tiles(seq(), 16385) == -1 and size(seq(), 0) == 0
    assert tiles(seq(), 64, FP8) == -1 and size(seq(), 64, FP8) == 0 and tiles(seq(2, t=1280), 128, F32) > 1
    assert L.mips_gated_scan_carries(None, 4, F32) == -1 and L.mips_gated_scan_workspace_size(None, 4, F32) == 0
    assert size(seq(2, t=1280), 128) >= 8 * 128 * 2560 // 128 and size(seq(2, 32, 0, 100000, 0x100), 128) >= 400000


def test_scan_refusals(L):
    def call(s=seq(), d=64, dt=BF16, x=rows(), f=rows(0x2000), g=rows(0x3000), init=0x4000, states=0x5000, last=0x6000,
             carries=None, ws=None, wsb=0):
        ref = lambda v: None if v is None else C.byref(v)  # noqa: E731
        return L.mips_gated_scan(ref(s), d, dt, ref(x), ref(f), ref(g), vp(init), vp(states), vp(last), vp(carries), vp(ws),
                                 wsb, None)

    for bad in [dict(s=seq(**b)) for b in BAD_SEQ] + [dict(s=None), dict(d=0), dict(x=None), dict(f=None), dict(last=None),
                dict(x=rows(None)), dict(x=rows(0x1001)), dict(f=rows(0x2000, 63)), dict(g=rows(0x3000, 64, 63)),
                dict(init=0x4002), dict(states=0x5001), dict(last=0x6002), dict(ws=0x10010), dict(dt=F32, x=rows(0x1002)),
                dict(carries=0x7002), dict(s=seq(t=1280)), dict(s=seq(4, 32, 0, 200, 0x100))]:
        assert call(**bad) == INVALID, bad
    for bad in [dict(s=seq(**b)) for b in NO_SEQ] + [dict(dt=FP8), dict(d=16385, x=rows(row=1 << 20, step=1 << 30))]:
        assert call(**bad) == UNSUPPORTED, bad
    assert call(s=seq(t=1280), ws=0x10000, wsb=1024) == WORKSPACE
    assert call(s=seq(4, 32, 0, 200, 0x100), ws=0x10000, wsb=512) == WORKSPACE


def test_scan_backward_refusals(L):
    def call(s=seq(), d=64, dt=BF16, x=rows(), f=rows(0x2000), g=rows(0x3000), init=0x4000, gs=rows(0x5000), gl=0x6000,
             carries=0xB000, dx=0x7000, df=0x8000, dg=0x9000, di=0xA000, ws=None, wsb=0):
        ref = lambda v: None if v is None else C.byref(v)  # noqa: E731
        return L.mips_gated_scan_backward(ref(s), d, dt, ref(x), ref(f), ref(g), vp(init), ref(gs), vp(gl), vp(carries), vp(dx),
                                          vp(df), vp(dg), vp(di), vp(ws), wsb, None)

    for bad in [dict(s=seq(**b)) for b in BAD_SEQ] + [dict(s=None), dict(d=0), dict(x=None), dict(f=None), dict(gs=None, gl=None),
                dict(gs=rows(0x5001)), dict(gl=0x6002), dict(dx=None), dict(df=None), dict(dg=None), dict(dx=0x7001),
                dict(df=0x8001), dict(dg=0x9001), dict(di=0xA002), dict(ws=0x10010), dict(s=seq(t=1280)),
                dict(carries=None), dict(carries=0xB002)]:
        assert call(**bad) == INVALID, bad
    for bad in [dict(s=seq(**b)) for b in NO_SEQ] + [dict(dt=FP8)]:
        assert call(**bad) == UNSUPPORTED, bad
    assert call(s=seq(t=1280), ws=0x10000, wsb=1024) == WORKSPACE


def test_step_refusals(L):
    def call(x=0x1000, xs=64, f=0x2000, fs=64, g=0x3000, gs=64, dt=BF16, b=5, d=64, state=0x4000, ss=64, out=0x4000, os_=64,
             n=10, ids=0x5000, bits=32, h=0x6000):
        return L.mips_gated_step(vp(x), xs, vp(f), fs, vp(g), gs, dt, b, d, vp(state), ss, vp(out), os_, n, vp(ids), bits, vp(h),
                                 None)

    assert call(b=0) == OK and call(b=0, x=None, f=None, g=None, state=None, out=None, ids=None, h=None) == OK
    for bad in (dict(x=None), dict(f=None), dict(state=None), dict(out=None), dict(ids=None), dict(h=None), dict(b=-1), dict(d=0),
                dict(n=0), dict(xs=63), dict(fs=63), dict(gs=63), dict(ss=63), dict(os_=63), dict(x=0x1001), dict(f=0x2001),
                dict(g=0x3001), dict(state=0x4002), dict(out=0x7002), dict(ids=0x5002), dict(bits=64, ids=0x5004), dict(h=0x6001),
                dict(os_=128), dict(out=0x4004), dict(state=0x4100), dict(ss=128, out=0x4100)):
        assert call(**bad) == INVALID, bad
    for bad in (dict(dt=FP8), dict(bits=16), dict(b=65537), dict(d=16385, xs=1 << 15, fs=1 << 15, gs=1 << 15, ss=1 << 15, os_=1 << 15)):
        assert call(**bad) == UNSUPPORTED, bad


def test_dropout_refusals(L):
    def call(x=0x1000, dt=BF16, n=5, p=0.5, counter=0x2000, res=0x3000, out=0x4000):
        return L.mips_dropout(vp(x), dt, n, p, 1, 2, vp(counter), vp(res), vp(out), None)

    assert call(n=0) == OK
    for bad in (dict(x=None), dict(out=None), dict(n=-1), dict(p=-0.1), dict(p=1.1), dict(p=float("nan")), dict(x=0x1001),
                dict(res=0x3001), dict(out=0x4001), dict(counter=0x2004)):
        assert call(**bad) == INVALID, bad
    assert call(dt=FP8) == UNSUPPORTED and call(n=(1 << 40) + 1) == UNSUPPORTED


def test_pool_refusals(L):
    def call(s=seq(), d=64, dt=BF16, x=rows(), v=0x2000, m=0x3000, n=0x4000, ws=0x10000, wsb=1 << 30):
        return L.mips_pool_normalize(None if s is None else C.byref(s), d, dt, None if x is None else C.byref(x), 1, vp(v), vp(m),
                                     vp(n), vp(ws), wsb, None)

    def back(s=seq(), d=64, dt=BF16, g=0x1000, gs=64, m=0x3000, n=0x4000, dx=0x5000):
        return L.mips_pool_normalize_backward(None if s is None else C.byref(s), d, dt, vp(g), gs, 1, vp(m), vp(n), vp(dx), None)

    for bad in [dict(s=seq(**b)) for b in BAD_SEQ] + [dict(s=None), dict(d=0), dict(x=None), dict(x=rows(None)), dict(v=None),
                dict(m=None), dict(n=None), dict(v=0x2001), dict(m=0x3002), dict(n=0x4002), dict(ws=0x10010), dict(x=rows(row=63)),
                dict(s=seq(t=1280), ws=None)]:
        assert call(**bad) == INVALID, bad
    for bad in [dict(s=seq(**b)) for b in BAD_SEQ] + [dict(s=None), dict(d=0), dict(g=None), dict(gs=63), dict(m=None), dict(n=None),
                dict(dx=None), dict(g=0x1001), dict(dx=0x5001)]:
        assert back(**bad) == INVALID, bad
    for bad in [dict(s=seq(**b)) for b in NO_SEQ] + [dict(dt=FP8)]:
        assert call(**bad) == UNSUPPORTED and back(**bad) == UNSUPPORTED, bad
    assert call(s=seq(t=1280), wsb=256) == WORKSPACE
    size = L.mips_pool_workspace_size
    assert size(None, 4) == 0 and size(C.byref(seq(b=0)), 4) == 0 and size(C.byref(seq()), 0) == 0 and size(C.byref(seq()), 64) == 0
    assert size(C.byref(seq(t=1280)), 64) > 0 and size(C.byref(seq(4, 32, 0, 200, 0x100)), 64) > 0


def test_python_refusals():
    """What the binding checks before it looks at devices: shapes and types."""
    x, f = torch.zeros(3, 5, 8), torch.zeros(3, 5, 8)
    three = torch.tensor([1, 2, 3])
    for call in (lambda: mips.gated_scan(x[0], f[0]), lambda: mips.gated_scan(x, f[:, :4]), lambda: mips.gated_scan(x, f, f[:2]),
                 lambda: mips.gated_scan(x, f, lengths=three[:2]), lambda: mips.gated_scan(x, f, offsets=three),
                 lambda: mips.gated_scan(x[0], f[0], offsets=three, lengths=three), lambda: mips.gated_scan(x[0], f[0], offsets=three[:1]),
                 lambda: mips.gated_scan(x[:, :0], f[:, :0]), lambda: mips.gated_scan(x, f, initial=torch.zeros(3, 7)),
                 lambda: mips.gated_scan(x, f.bfloat16()), lambda: mips.gated_scan(x, f, initial=torch.zeros(3, 8).double()),
                 lambda: mips.gated_scan_backward(None, None, x, f, None, None),
                 lambda: mips.gated_step(x[0], f[0], torch.zeros(9, 8), three), lambda: mips.gated_step(x[0], f[0], torch.zeros(9, 7), three),
                 lambda: mips.gated_step(x[:, 0], f[:, 0], torch.zeros(9, 8).double(), three),
                 lambda: mips.gated_step(x[:, 0], f[:, 0], torch.zeros(9, 8), three, out=torch.zeros(8, 8)),
                 lambda: mips.gated_step(x[:, 0], f[:, 0], torch.zeros(8, 9).t(), three),
                 lambda: mips.dropout(x, 1.5, 0), lambda: mips.dropout(x, -0.5, 0), lambda: mips.dropout(x, 0.5, 0, residual=x[:2]),
                 lambda: mips.dropout(x, 0.5, 0, counter=torch.zeros(2, dtype=torch.int64)),
                 lambda: mips.dropout(x, 0.5, 0, counter=torch.zeros(1)),
                 lambda: mips.pool_normalize(x[0]), lambda: mips.pool_normalize(x, lengths=three[:1])):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: mips.gated_scan(x.half(), f.half()), lambda: mips.gated_scan(x, f, lengths=three.float()),
                 lambda: mips.dropout(x.double(), 0.5, 0), lambda: mips.pool_normalize(x.half()),
                 lambda: mips.gated_step(x[:, 0].half(), f[:, 0].half(), torch.zeros(9, 8), three)):
        with pytest.raises(TypeError):
            call()
    for call in (lambda: mips.gated_scan(x, f), lambda: mips.dropout(x, 0.5, 0), lambda: mips.pool_normalize(x),
                 lambda: mips.gated_step(x[:, 0], f[:, 0], torch.zeros(9, 8), three)):
        with pytest.raises(ValueError, match="GPU"):
            call()


def test_sizes_past_32_bits_are_refused():
    """Before anything of such a size is looked at: the C interface would see them cut short."""
    wide, far = 1 << 32, (1 << 32) + 1
    one = torch.zeros(1, 1, 1)
    for x in (one.expand(far, 1, 1), one.expand(1, 1, far)):
        for call in (lambda: mips.gated_scan(x, x), lambda: mips.pool_normalize(x),
                     lambda: mips.pool_normalize_backward(one[0], x.shape, None)):
            with pytest.raises(mips.MipsError):
                call()
    row = torch.zeros(1, 1)
    for x in (row.expand(far, 1), row.expand(1, wide + 4)):
        with pytest.raises(mips.MipsError):
            mips.gated_step(x, x, row, torch.zeros(1, dtype=torch.int32).expand(x.shape[0]))
    with pytest.raises(mips.MipsError):
        mips.gated_scan(row, row, offsets=torch.zeros(1, dtype=torch.int32).expand(far + 1))


def test_limits_match_the_binding():
    text = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "mips.h")).read()
    assert int(re.search(r"#define MIPS_EVENTS_MAX (\d+)", text)[1]) == mips.EVENTS_MAX


def test_generator_known_answers():
    """Philox4x32-10's published known answers (the authors' test vectors)."""
    one = 0xFFFFFFFF
    for ctr, key, want in (((0, 0, 0, 0), (0, 0), (0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8)),
                           ((one,) * 4, (one,) * 2, (0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD)),
                           ((0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344), (0xA4093822, 0x299F31D0),
                            (0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1))):
        got = hc.philox([np.array([v], dtype=np.uint64) for v in ctr], key)
        assert tuple(int(v[0]) for v in got) == want


def test_bounds_of_the_plain_forms():
    """The 64-bit loops against torch's autograd of the same recurrence."""
    rng = np.random.default_rng(0)
    n, d = 23, 5
    seqs = [(0, 7), (7, 7), (7, 20), (20, 21)]
    x, f, g = (rng.standard_normal((n, d)) for _ in range(3))
    init, gs, gl = rng.standard_normal((4, d)), rng.standard_normal((n, d)), rng.standard_normal((4, d))
    for gate in (g, None):
        t = [None if v is None else torch.from_numpy(v).requires_grad_() for v in (x, f, gate, init)]
        a = torch.sigmoid(t[1])
        w = 1 - a if gate is None else torch.sigmoid(t[2])
        loss, states = 0, {}
        for s, (lo, hi) in enumerate(seqs):
            h = t[3][s]
            for r in range(lo, hi):
                h = a[r] * h + w[r] * t[0][r]
                states[r] = h.detach().numpy()
                loss = loss + (h * torch.from_numpy(gs[r])).sum()
            loss = loss + (h * torch.from_numpy(gl[s])).sum()
        loss.backward()
        h, _, _, _ = hc.scan(x, f, gate, seqs, init)
        assert all(np.allclose(h[r], v, rtol=1e-12) for r, v in states.items()) and not h[21:].any()
        for got, v in zip(hc.scan_grad(x, f, gate, seqs, init, gs, gl), t):
            assert v is None or np.allclose(got[0], v.grad.numpy(), rtol=1e-10, atol=1e-14)
