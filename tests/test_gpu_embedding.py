"""Embedding lookup with scaling and its gradient by sorted tokens, against plain 64-bit
implementations on the CPU.

Tolerances. Lookup: one binary32 product and one rounding to the table's type, both to
nearest, as torch's own conversions do: bitwise. Gradient: a sum of m values in binary32 in any
order is within m * 2^-24 * sum|g| of the exact sum (m - 1 additions, each within half a unit in
the last place of a partial sum of at most sum|g|, to first order), the scale adds one
rounding (2^-24) and an accumulated output another: within (m + 4) * 2^-24 * sum|g|. A bf16
output is such a value rounded to nearest, which is monotone: it lies between the roundings of
the interval's two ends."""
import numpy as np
import pytest
import torch

import exact_inner_product_amd as mips

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def _dev():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    return torch.device("cuda:0")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("idt", [torch.int32, torch.int64])
@pytest.mark.parametrize("rows,d,shape", [(1, 1, (1,)), (7, 8, (0,)), (400, 16, (3, 5)), (1000, 100, (257,)),
                                          (1000, 64, (4, 33)), (50, 600, (70,)), (300, 33, (129,)),
                                          (20, 2056, (9,))])
def test_lookup(dtype, idt, rows, d, shape):
    dev = _dev()
    print(f"lookup {dtype} {idt} rows={rows} d={d} ids={shape}", flush=True)
    gen = torch.Generator().manual_seed(rows + d)
    table = torch.randn(rows, d, generator=gen).to(DT[dtype])
    ids = torch.randint(0, rows, shape, generator=gen).to(idt)
    flat = ids.view(-1)
    if flat.numel() > 3:  # padding: below and past the table
        flat[1], flat[2] = -1, rows
    got = mips.embedding_lookup(table.to(dev), ids.to(dev), scale=1.7).cpu()
    ok = (ids >= 0) & (ids < rows)
    want = (table[torch.where(ok, ids, 0).long()].float() * 1.7).to(DT[dtype])
    want[~ok] = 0
    assert got.shape == (*shape, d) and got.dtype == DT[dtype]
    assert torch.equal(got, want)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_lookup_of_strided_and_misaligned_tables(dtype):
    dev = _dev()
    base = torch.randn(60, 96, generator=torch.Generator().manual_seed(3)).to(DT[dtype])
    ids = torch.tensor([59, 0, 7, 7, 31])
    for cut in (slice(0, 64), slice(1, 65), slice(8, 40), slice(3, 4)):
        table = base.to(dev)[:, cut]
        got = mips.embedding_lookup(table, ids.to(dev), scale=0.5)
        assert torch.equal(got.cpu(), (base[:, cut][ids].float() * 0.5).to(DT[dtype])), cut
    turned = base.to(dev).t()  # unit stride along the rows: copied
    assert torch.equal(mips.embedding_lookup(turned, ids.to(dev)).cpu(), base.t()[ids])


def test_lookup_carries_infinities_and_nan():
    dev = _dev()
    for dtype in (torch.float32, torch.bfloat16):
        table = torch.tensor([[float("inf"), -float("inf"), float("nan"), 0.0] * 4], dtype=dtype, device=dev)
        got = mips.embedding_lookup(table, torch.zeros(2, dtype=torch.int32, device=dev), scale=2.0).cpu()
        assert torch.equal(torch.nan_to_num(got), torch.nan_to_num(table.cpu().repeat(2, 1)))
        assert torch.isnan(got[:, 2::4]).all() and torch.isinf(got[:, 0::4]).all()


def _ids_like(kind, rows, t, rng):
    if kind == "one":
        return np.full(t, min(3, rows - 1))
    if kind == "uniform":
        return rng.integers(0, rows, t)
    if kind == "padded":
        i = rng.integers(-2, rows + 2, t)
        return i
    u = rng.random(t)  # zipf
    return np.minimum(np.exp(u * np.log(rows + 1)).astype(np.int64) - 1, rows - 1)


def _check_grad(got, grad, ids, rows, scale, base=None):
    g = grad.double().cpu().numpy()
    want = np.zeros((rows, g.shape[1]))
    mag = np.zeros_like(want)
    cnt = np.zeros((rows, 1))
    ok = (ids >= 0) & (ids < rows)
    np.add.at(want, ids[ok], g[ok])
    np.add.at(mag, ids[ok], np.abs(g[ok]))
    np.add.at(cnt, ids[ok], 1.0)
    want, mag = want * scale, mag * abs(scale)
    if base is not None:
        want += base
        mag += np.abs(base)
    tol = (cnt + 4) * 2.0 ** -24 * mag
    lo, hi = want - tol, want + tol
    if got.dtype == torch.bfloat16:
        lo, hi = (torch.from_numpy(x).bfloat16().double().numpy() for x in (lo, hi))
    got = got.double().cpu().numpy()
    assert ((lo <= got) & (got <= hi)).all(), f"worst {np.max(np.abs(got - want) - tol)}"


CASES = [
    # kind, rows, t, d
    ("uniform", 1, 1, 1), ("uniform", 10, 1, 64), ("one", 5, 7, 8), ("one", 400, 9, 16), ("uniform", 400, 8, 16),
    ("zipf", 1000, 513, 100), ("padded", 300, 1000, 33), ("one", 3, 8192, 32), ("zipf", 65536, 8192, 64),
    ("zipf", 65535, 8193, 64), ("uniform", 255, 8200, 16), ("uniform", 256, 9001, 24), ("one", 70000, 20000, 128),
    ("padded", 50, 30000, 8), ("zipf", 100000, 120001, 64), ("uniform", 900000, 40000, 16), ("zipf", 200, 9000, 700),
    ("zipf", 5000, 16384, 16), ("zipf", 5000, 16385, 16), ("uniform", 1 << 24, 17000, 1), ("padded", 70, 1100000, 8),
    ("zipf", 3000, 1024, 64), ("uniform", 65536, 1025, 8), ("uniform", 1 << 22, 5000, 1), ("one", 1 << 23, 700, 1),
    ("one", 600, 16384, 8), ("padded", 1025, 16000, 40),
    ("zipf", 1 << 21, 16000, 8), ("uniform", 1 << 23, 9000, 1),  # few tokens, sorted: many rows
]


@pytest.mark.parametrize("dtype,out", [("f32", "f32"), ("bf16", "bf16"), ("bf16", "f32")])
@pytest.mark.parametrize("kind,rows,t,d", CASES)
def test_grad(kind, rows, t, d, dtype, out):
    dev = _dev()
    print(f"embedding grad {dtype}->{out} {kind} rows={rows} t={t} d={d}", flush=True)
    rng = np.random.default_rng(rows + t)
    ids = _ids_like(kind, rows, t, rng)
    grad = torch.from_numpy(rng.standard_normal((t, d)).astype(np.float32)).to(DT[dtype])
    idt = torch.int64 if t % 2 else torch.int32
    buf = torch.full((rows, d), 7.0, dtype=DT[out], device=dev)
    got = mips.embedding_grad(grad.to(dev), torch.from_numpy(ids).to(idt).to(dev), rows, scale=1.25, out=buf)
    assert got.data_ptr() == buf.data_ptr()
    _check_grad(got, grad, ids, rows, 1.25)
    again = mips.embedding_grad(grad.to(dev), torch.from_numpy(ids).to(idt).to(dev), rows, scale=1.25,
                                out=torch.empty_like(buf))
    assert torch.equal(got, again)


@pytest.mark.parametrize("dtype,out", [("f32", "f32"), ("bf16", "bf16"), ("bf16", "f32")])
@pytest.mark.parametrize("t", [0, 37, 9000])
def test_grad_accumulates_and_writes_strided_rows(dtype, out, t):
    dev = _dev()
    rows, d = 500, 40
    rng = np.random.default_rng(t)
    ids = _ids_like("zipf", rows, t, rng)
    wide = torch.from_numpy(rng.standard_normal((t, d + 8)).astype(np.float32)).to(DT[dtype]).to(dev)
    for cut in (slice(0, d), slice(1, d + 1)):
        base = torch.from_numpy(rng.standard_normal((rows, d + 4)).astype(np.float32)).to(DT[out]).to(dev)
        want_rest = base[:, d:].clone()
        start = base[:, :d].double().cpu().numpy()
        grad = wide[:, cut]
        mips.embedding_grad(grad, torch.from_numpy(ids).to(dev), rows, scale=-0.5, out=base[:, :d], accumulate=True)
        _check_grad(base[:, :d], grad, ids, rows, -0.5, start)
        assert torch.equal(base[:, d:], want_rest)
        mips.embedding_grad(grad, torch.from_numpy(ids).to(dev), rows, scale=-0.5, out=base[:, :d])
        _check_grad(base[:, :d], grad, ids, rows, -0.5)
        assert torch.equal(base[:, d:], want_rest)


def test_grad_is_the_lookups_gradient_by_differences():
    """sum(lookup(table + h e) * y) - sum(lookup(table - h e) * y) over 2h, for every element:
    the lookup is linear, so the quotient is exact up to rounding (values on a grid: exact)."""
    dev = _dev()
    rows, d, t = 6, 8, 21
    rng = np.random.default_rng(5)
    table = torch.from_numpy(rng.integers(-8, 9, (rows, d)).astype(np.float32)).to(dev)
    y = torch.from_numpy(rng.integers(-8, 9, (t, d)).astype(np.float32)).to(dev)
    ids = torch.from_numpy(rng.integers(-1, rows, t)).to(dev)
    got = mips.embedding_grad(y, ids, rows, scale=0.5).cpu()
    for v in range(rows):
        for j in range(d):
            e = torch.zeros_like(table)
            e[v, j] = 1.0
            up = (mips.embedding_lookup(table + e, ids, 0.5) * y).sum()
            dn = (mips.embedding_lookup(table - e, ids, 0.5) * y).sum()
            assert float((up - dn) / 2) == float(got[v, j])


def test_on_another_stream_and_in_a_graph():
    """The gradient on a side stream, then captured and replayed with fresh inputs, equals
    the eager result bit by bit."""
    dev = _dev()
    rows, d, t = 3000, 64, 20000
    rng = np.random.default_rng(9)
    ids = torch.from_numpy(rng.integers(0, rows, t)).to(torch.int32).to(dev)
    grad = torch.randn(t, d, device=dev)
    table = torch.randn(rows, d, device=dev)
    want, looked = mips.embedding_grad(grad, ids, rows), mips.embedding_lookup(table, ids)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        a, b = mips.embedding_grad(grad, ids, rows), mips.embedding_lookup(table, ids)
    side.synchronize()
    assert torch.equal(a, want) and torch.equal(b, looked)
    out = torch.empty_like(want)
    ws = mips.empty_workspace(mips.lib().mips_embedding_grad_workspace_size(t, rows, d), dev)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mips.embedding_grad(grad, ids, rows, out=out, workspace=ws)
    for i in range(3):
        grad.copy_(torch.randn(t, d, device=dev))
        ids.copy_(torch.from_numpy(rng.integers(0, rows, t)).to(torch.int32))
        out.fill_(5.0)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, mips.embedding_grad(grad, ids, rows)), i


def test_refusals():
    dev = _dev()
    table = torch.zeros(4, 8, device=dev)
    ids = torch.zeros(3, dtype=torch.int32, device=dev)
    with pytest.raises(TypeError):
        mips.embedding_lookup(table.half(), ids)
    with pytest.raises(TypeError):
        mips.embedding_lookup(table, ids.float())
    with pytest.raises(ValueError):
        mips.embedding_lookup(table, ids.cpu())
    with pytest.raises(ValueError):
        mips.embedding_lookup(table[0], ids)
    with pytest.raises(ValueError):
        mips.embedding_grad(torch.zeros(4, 8, device=dev), ids, 4)
    with pytest.raises(ValueError):
        mips.embedding_grad(torch.zeros(3, 8, device=dev), ids, 4, accumulate=True)
    with pytest.raises(TypeError):
        mips.embedding_grad(torch.zeros(3, 8, device=dev), ids, 4,
                            out=torch.zeros(4, 8, device=dev, dtype=torch.bfloat16))
    with pytest.raises(mips.MipsError, match="workspace too small"):
        mips.embedding_grad(torch.zeros(20000, 8, device=dev), ids[:1].repeat(20000), 4,
                            workspace=mips.empty_workspace(256, dev))
