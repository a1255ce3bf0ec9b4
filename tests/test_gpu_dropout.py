"""Dropout against the generator's definition on the CPU (itself checked with its published known
answers in test_histories_boundary.py).

Tolerance: one product (half a unit in the last place of x * scale) and, with a residual, one sum (or
both in one rounding), in binary32: within 2^-24 (|x scale| + |x scale + residual|), and the rounding to the type on top.
The scale is a ratio of integers rounded to binary32 on both sides. Which elements are kept is exact."""
import numpy as np
import pytest
import torch

import exact_inner_product_amd as mips
from tests import histories_check as hc
from tests.histories_check import DT

pytestmark = pytest.mark.gpu


def _dev():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    return torch.device("cuda:0")


def check(got, x, p, seed, offset, residual=None, start=0):
    n = x.numel()
    keep = hc.kept(n, p, seed, offset, start)
    c = int(p * 65536 + 0.5)
    scale = float(np.float32(65536 / (65536 - c))) if c < 65536 else 0.0
    v = np.where(keep, x.double().numpy().reshape(-1) * scale, 0.0)
    want = v if residual is None else v + residual.double().numpy().reshape(-1)
    hc.within(got.reshape(-1), want, hc.U * (np.abs(v) + np.abs(want)), "dropout")
    if residual is None:
        assert np.array_equal(got.cpu().float().numpy().reshape(-1) != 0, keep & (x.float().numpy().reshape(-1) != 0))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape", [(1,), (7,), (8,), (9,), (1000, 64), (33, 5, 3), (4097, 129), (300000,)])
def test_dropout(shape, dtype):
    dev = _dev()
    print(f"dropout {shape} {dtype}", flush=True)
    gen = torch.Generator().manual_seed(len(shape) + shape[0])
    x, r = (torch.randn(shape, generator=gen).to(DT[dtype]) for _ in range(2))
    for k, p in enumerate((0.0, 0.1, 0.5, 0.999, 1.0, 1e-6)):
        seed, offset = 0x123456789ABCDEF0 + k, (k << 33) + 5
        check(mips.dropout(x.to(dev), p, seed, offset), x, p, seed, offset)
        check(mips.dropout(x.to(dev), p, seed, offset, residual=r.to(dev)), x, p, seed, offset, r)


def test_seeds_offsets_and_the_counter():
    dev = _dev()
    x = torch.ones(5000, device=dev)
    a = mips.dropout(x, 0.5, 0)
    assert torch.equal(a, mips.dropout(x, 0.5, 1 << 64)) and torch.equal(a, mips.dropout(x, 0.5, 0, 1 << 64))
    for other in (mips.dropout(x, 0.5, 1), mips.dropout(x, 0.5, 1 << 32), mips.dropout(x, 0.5, 0, 1),
                  mips.dropout(x, 0.5, 0, 1 << 32)):
        assert 0.4 < float((a == other).float().mean()) < 0.6  # 5000 fair coins: 14 standard deviations
    check(mips.dropout(x, 0.5, -1, -1), x.cpu(), 0.5, (1 << 64) - 1, (1 << 64) - 1)
    for c in (0, 3, -1):
        counter = torch.tensor(c, device=dev)
        assert torch.equal(mips.dropout(x, 0.5, 9, 7, counter=counter), mips.dropout(x, 0.5, 9, 7 + c))


def test_layouts():
    """The mask goes by the element's place in the shape, not in memory."""
    dev = _dev()
    for dtype in (torch.float32, torch.bfloat16):
        x = torch.randn(70, 50, device=dev).to(dtype)
        want = mips.dropout(x, 0.3, 5)
        assert torch.equal(mips.dropout(x.t().contiguous().t(), 0.3, 5), want)
        big = torch.randn(70, 60, device=dev).to(dtype)
        big[:, 3:53] = x
        assert torch.equal(mips.dropout(big[:, 3:53], 0.3, 5), want)
        odd = torch.empty(3501, dtype=dtype, device=dev)  # not aligned: one by one
        odd[1:] = x.view(-1)
        assert torch.equal(mips.dropout(odd[1:], 0.3, 5), want.view(-1))
        assert torch.equal(mips.dropout(x, 0.3, 5, residual=x.t().contiguous().t()), mips.dropout(x, 0.3, 5, residual=x))
    assert mips.dropout(torch.empty(0, 4, device=dev), 0.5, 1).shape == (0, 4)


def test_dropped_values_may_be_anything():
    dev = _dev()
    keep = torch.from_numpy(hc.kept(4000, 0.4, 3, 0)).to(dev)
    for bad in (float("nan"), float("inf"), -float("inf")):
        y = mips.dropout(torch.full((4000,), bad, device=dev), 0.4, 3)
        assert not y[~keep].any() and not torch.isfinite(y[keep]).any()
    # all dropped: only the residual is left
    r = torch.randn(4000, device=dev)
    assert torch.equal(mips.dropout(torch.full((4000,), float("nan"), device=dev), 1.0, 3, residual=r), r)


def test_rates():
    """Share of kept elements and of kept neighbours over 2^20 draws, to six standard deviations."""
    dev = _dev()
    n = 1 << 20
    for p in (0.1, 0.5, 0.9):
        k = (mips.dropout(torch.ones(n, device=dev), p, 77) != 0).double()
        q = 1 - int(p * 65536 + 0.5) / 65536
        assert abs(float(k.mean()) - q) < 6 * (q * (1 - q) / n) ** 0.5
        for lag in (1, 2, 8, 64):
            c = float(((k[lag:] - q) * (k[:-lag] - q)).mean())
            assert abs(c) < 6 * q * (1 - q) / n ** 0.5


def test_places_past_32_bits():
    """Elements whose places and byte offsets pass 2^32."""
    dev = _dev()
    n, tail = (1 << 32) + 4104, 8192
    x = torch.ones(n, dtype=torch.bfloat16, device=dev)
    y = mips.dropout(x, 0.25, 11, 2)
    check(y[n - tail:], x[n - tail:].cpu(), 0.25, 11, 2, start=n - tail)
    del x, y
    torch.cuda.empty_cache()


def test_one_rounding_with_a_residual():
    """Sums that cancel: within half a unit in the last place of x scale + residual itself (64 bits hold the
    product, and the sum to 2^-53, which is below a millionth of the room where the sum is above 2^-20 of its terms)."""
    dev = _dev()
    gen = torch.Generator().manual_seed(8)
    n, p, seed = 1 << 17, 0.1, 21
    c = int(p * 65536 + 0.5)
    scale = float(np.float32(65536 / (65536 - c)))
    x = torch.randn(n, generator=gen)
    r = -(x.double() * scale * (1 + torch.randn(n, generator=gen).double() * 1e-3)).float()
    keep = torch.from_numpy(hc.kept(n, p, seed, 0))
    want = torch.where(keep, x.double() * scale, 0.0) + r.double()
    sure = want.abs() > r.double().abs() * 2.0 ** -20
    assert sure.double().mean() > 0.99
    got = mips.dropout(x.to(dev), p, seed, residual=r.to(dev)).cpu().double()
    assert ((got - want).abs() <= hc.U * want.abs() * (1 + 1e-6))[sure].all()
    assert torch.equal(got[~keep], r.double()[~keep])
