"""The global gradient norm and clipping, against 64-bit sums on the CPU.

Tolerances. Squares are summed in binary64 (relative error below 2^-30 at these sizes), so the
norm is its exact value rounded to binary32: 2^-23. The factor is rounded once and the product
once in binary32: 2^-22 of each value. A bf16 output is such a value rounded to nearest, which
is monotone: it lies between the roundings of the interval's two ends."""
import math

import pytest
import torch

import exact_inner_product_amd as mips

pytestmark = pytest.mark.gpu


def _dev():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    return torch.device("cuda:0")


def _exact(ts, max_norm):
    total = math.sqrt(sum(float(t.double().cpu().square().sum()) for t in ts))
    return total, min(1.0, max_norm / (total + 1e-6))


def _check(got, ts, coef):
    for i, (g, t) in enumerate(zip(got, ts)):
        want = t.double().cpu() * coef
        tol = want.abs() * 2.0 ** -22 + 1e-40
        lo, hi = want - tol, want + tol
        if t.dtype == torch.bfloat16:
            lo, hi = lo.bfloat16().double(), hi.bfloat16().double()
        g = g.double().cpu()
        assert ((lo <= g) & (g <= hi)).all(), i


SETS = [
    [(1,)], [(5, 3), (0,), (7,)], [(16384,)], [(16385,), (16383,), (3, 1)], [(400, 16), (16,), (128, 64)],
    [(i * 37 + 1,) for i in range(150)], [(1,)] * 64, [(2,)] * 65, [(1000003,), (64, 1001)], [(5_000_000,)],
]


@pytest.mark.parametrize("sizes", SETS, ids=[str(i) for i in range(len(SETS))])
@pytest.mark.parametrize("mix", ["f32", "bf16", "mixed"])
@pytest.mark.parametrize("max_norm", [0.5, 1e9])
def test_clip(sizes, mix, max_norm):
    dev = _dev()
    print(f"clip {len(sizes)} tensors {sizes[:3]} {mix} max_norm={max_norm}", flush=True)
    gen = torch.Generator().manual_seed(len(sizes))
    ts = []
    for i, s in enumerate(sizes):
        t = torch.randn(s, generator=gen)
        ts.append((t.bfloat16() if mix == "bf16" or (mix == "mixed" and i % 2) else t).to(dev))
    total, coef = _exact(ts, max_norm)
    keep = [t.clone() for t in ts]
    out = [torch.full_like(t, 9.0) for t in ts]
    norm, got = mips.clip_grad_norm(ts, max_norm, out=out)
    assert norm.dtype == torch.float32 and norm.shape == ()
    assert abs(float(norm) - total) <= total * 2.0 ** -23
    assert all(torch.equal(a, b) for a, b in zip(ts, keep))
    _check(got, keep, coef)
    norm2, inplace = mips.clip_grad_norm(ts, max_norm)
    assert float(norm2) == float(norm) and inplace[0] is ts[0]
    assert all(torch.equal(a, b) for a, b in zip(ts, out))
    if max_norm == 1e9:
        assert all(torch.equal(a, b) for a, b in zip(ts, keep))


def test_misaligned_views_and_permuted_tensors():
    dev = _dev()
    base = torch.randn(4099, device=dev)
    half = torch.randn(4099, device=dev).bfloat16()
    ts = [base[1:], half[1:], half[3:3], torch.randn(33, 7, device=dev).t(), torch.randn(1, 5, device=dev).t()]
    total, coef = _exact(ts, 1.0)
    keep = [t.clone(memory_format=torch.preserve_format) for t in ts]
    first = base[0].item(), half[0].item()
    norm, got = mips.clip_grad_norm(ts, 1.0)
    assert abs(float(norm) - total) <= total * 2.0 ** -23
    _check(got, keep, coef)
    assert (base[0].item(), half[0].item()) == first


def test_extreme_values():
    """Squares outside binary32's range; NaN and infinity follow the formula."""
    dev = _dev()
    for v in (1e30, 1e-30):
        ts = [torch.full((100,), v, device=dev), torch.full((17,), v, device=dev)]
        total, coef = _exact(ts, 1.0)
        norm, got = mips.clip_grad_norm([t.clone() for t in ts], 1.0)
        assert abs(float(norm) - total) <= total * 2.0 ** -23
        _check(got, ts, coef)
    bad = torch.ones(40, device=dev)
    bad[3] = float("nan")
    norm, got = mips.clip_grad_norm([torch.ones(5, device=dev), bad], 1.0)
    assert math.isnan(float(norm)) and all(torch.isnan(g).all() for g in got)
    big = torch.ones(40, device=dev)
    big[3] = float("inf")
    norm, got = mips.clip_grad_norm([torch.ones(5, device=dev), big], 1.0)
    assert math.isinf(float(norm)) and (got[0] == 0).all() and torch.isnan(got[1][3])
    ts = [torch.ones(4, device=dev)]
    norm, got = mips.clip_grad_norm(ts, 0.0)
    assert float(norm) == 2.0 and (got[0] == 0).all()
    norm, got = mips.clip_grad_norm([torch.full((4,), 3.0, device=dev)], math.inf)
    assert float(norm) == 6.0 and (got[0] == 3).all()
    norm, got = mips.clip_grad_norm([torch.empty(0, device=dev)], 1.0)
    assert float(norm) == 0.0


def test_side_stream_and_graph():
    dev = _dev()
    ts = [torch.randn(70001, device=dev), torch.randn(513, device=dev).bfloat16()]
    out = [torch.empty_like(t) for t in ts]
    want_n, want = mips.clip_grad_norm(ts, 1.0, out=[torch.empty_like(t) for t in ts])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        n, got = mips.clip_grad_norm(ts, 1.0, out=out)
    side.synchronize()
    assert float(n) == float(want_n) and all(torch.equal(a, b) for a, b in zip(got, want))
    ws = mips.empty_workspace(mips.lib().mips_clip_workspace_size(2), dev)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gn, _ = mips.clip_grad_norm(ts, 1.0, out=out, workspace=ws)
    for _ in range(3):
        ts[0].copy_(torch.randn(70001, device=dev))
        graph.replay()
        torch.cuda.synchronize()
        n, got = mips.clip_grad_norm(ts, 1.0, out=[torch.empty_like(t) for t in ts])
        assert float(gn) == float(n) and all(torch.equal(a, b) for a, b in zip(out, got))


def test_refusals():
    dev = _dev()
    t = torch.ones(8, device=dev)
    for bad in ([], [t[::2]], [t, t.cpu()]):
        with pytest.raises(ValueError):
            mips.clip_grad_norm(bad, 1.0)
    with pytest.raises(TypeError):
        mips.clip_grad_norm([t.half()], 1.0)
    with pytest.raises(ValueError):
        mips.clip_grad_norm([t], -1.0)
    with pytest.raises(ValueError):
        mips.clip_grad_norm([t], 1.0, out=[t.bfloat16()])
    with pytest.raises(mips.MipsError, match="workspace too small"):
        mips.clip_grad_norm([t], 1.0, workspace=mips.empty_workspace(256, dev))


@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_an_infinite_max_norm_only_takes_the_norm(bad, dtype):
    """Gradients that overflowed are left (and copied) bit by bit, whatever the norm."""
    dev = _dev()
    ts = [torch.randn(70001, device=dev).to(dtype), torch.randn(33, 7, device=dev).to(dtype)]
    ts[0][4321] = bad
    keep = [t.clone() for t in ts]
    as_ints = lambda t: t.view(torch.int32 if dtype == torch.float32 else torch.int16)  # noqa: E731
    norm, got = mips.clip_grad_norm(ts, math.inf, out=[torch.zeros_like(t) for t in ts])
    assert math.isnan(float(norm)) if math.isnan(bad) else float(norm) == math.inf
    assert all(torch.equal(as_ints(a), as_ints(b)) for a, b in zip(got, keep))
    norm, _ = mips.clip_grad_norm(ts, math.inf)
    assert math.isnan(float(norm)) if math.isnan(bad) else float(norm) == math.inf
    assert all(torch.equal(as_ints(a), as_ints(b)) for a, b in zip(ts, keep))


def test_empty_tensors_among_permuted_ones():
    """A tensor without elements is dense whatever its strides: also beside one that is permuted."""
    dev = _dev()
    ts = [torch.randn(33, 7, device=dev).t(), torch.empty(5, 0, device=dev), torch.empty(0, 5, device=dev).t()]
    keep = ts[0].clone(memory_format=torch.preserve_format)
    total, coef = _exact(ts[:1], 1.0)
    norm, got = mips.clip_grad_norm(ts, 1.0)
    assert abs(float(norm) - total) <= total * 2.0 ** -23
    _check(got[:1], [keep], coef)
    out = [torch.empty_like(t) for t in ts]
    norm2, got2 = mips.clip_grad_norm([keep, *ts[1:]], 1.0, out=out)
    assert float(norm2) == float(norm) and torch.equal(got2[0], got[0])


def test_the_stride_of_a_single_element_does_not_matter():
    """out may have any stride along an axis of length 1, also beside a permuted tensor."""
    dev = _dev()
    ts = [torch.randn(33, 7, device=dev).t(), torch.randn(1, 5, device=dev).t()]
    out = [torch.empty(33, 7, device=dev).t(), torch.empty(5, 1, device=dev)]
    assert ts[1].stride() != out[1].stride()
    total, coef = _exact(ts, 1.0)
    norm, got = mips.clip_grad_norm(ts, 1.0, out=out)
    assert abs(float(norm) - total) <= total * 2.0 ** -23
    _check(got, ts, coef)
    with pytest.raises(ValueError):
        mips.clip_grad_norm(ts, 1.0, out=[torch.empty(7, 33, device=dev), out[1]])
