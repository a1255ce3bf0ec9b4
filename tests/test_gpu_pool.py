"""Pooled and normalised vectors and their gradient against plain 64-bit forms.

Tolerances, u = 2^-24. A mean of m rows in binary32 in any order: (m + 3) u mean|x| =: e (m - 1
additions, the reciprocal of m, a product). The norm n of d squares: relative (d + 4) u, and what the
means' errors add, |e| / n in the 2-norm, at most; u = m / n then has e / n + |u| ((d + 8) u + |e| / n). The
gradient with w = g . m and t = m w / n^2, W = sum |g m|: errors of w ((d + 2) u W + sum |g| e),
of m and of n carry into t in proportion, then a difference, a quotient and a product."""
import numpy as np
import pytest
import torch

import exact_inner_product_amd as mips
from tests import histories_check as hc
from tests.histories_check import DT
from tests.test_gpu_scan import make

pytestmark = pytest.mark.gpu


def _dev():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    return torch.device("cuda:0")


def reference(x, seqs, normalize):
    """(vectors, bound, means, their bound, norms, count)."""
    d, b = x.shape[1], len(seqs)
    m, e, cnt = np.zeros((b, d)), np.zeros((b, d)), np.zeros((b, 1))
    for s, (lo, hi) in enumerate(seqs):
        cnt[s] = hi - lo
        if hi > lo:
            m[s] = x[lo:hi].mean(0)
            e[s] = (hi - lo + 3) * hc.U * np.abs(x[lo:hi]).mean(0)
    if not normalize:
        return m, e + hc.U * np.abs(m) + 1e-36, m, e, np.ones((b, 1)), cnt
    n = np.sqrt(np.maximum((m * m).sum(1, keepdims=True), 1e-12))
    rel = (d + 8) * hc.U + np.sqrt((e * e).sum(1, keepdims=True)) / n
    return m / n, e / n + np.abs(m / n) * rel + 1e-36, m, e, n, cnt


def reference_grad(x, seqs, normalize, g):
    d = x.shape[1]
    _, _, m, e, n, cnt = reference(x, seqs, normalize)
    inv = 1 / np.maximum(cnt, 1)
    square = (m * m).sum(1, keepdims=True)
    rel = (d + 8) * hc.U + np.sqrt((e * e).sum(1, keepdims=True)) / n
    if normalize:
        w, we = (g * m).sum(1, keepdims=True), (d + 2) * hc.U * np.abs(g * m).sum(1, keepdims=True) + (np.abs(g) * e).sum(1, keepdims=True)
        live = square > 1e-12
        t = np.where(live, m * w / n ** 2, 0.0)
        te = np.where(live, (np.abs(m) * we + e * np.abs(w) + np.abs(m * w) * (2 * rel + 6 * hc.U)) / n ** 2, 0.0)
    else:
        t = te = np.zeros_like(m)
        rel = np.zeros_like(rel)
    v = (g - t) / n * inv
    ve = (te + hc.U * (np.abs(g) + np.abs(t))) / n * inv + np.abs(v) * (rel + 6 * hc.U)
    dx, de = np.zeros_like(x), np.zeros_like(x)
    for s, (lo, hi) in enumerate(seqs):
        dx[lo:hi], de[lo:hi] = v[s], ve[s]
    return dx, de + 1e-36


CASES = [("dense", 1, 1, 1), ("dense", 5, 1, 128), ("dense", 700, 1, 64), ("dense", 16, 50, 64), ("dense", 30, 127, 128),
         ("dense", 3, 256, 100), ("dense", 3, 257, 128), ("dense", 2, 3000, 64), ("dense", 1, 1000, 1032), ("dense", 9, 31, 8),
         ("padded", 1, 3, 16), ("padded", 40, 33, 33), ("padded", 20, 127, 128), ("padded", 5, 600, 256), ("padded", 4, 90, 700),
         ("packed", 1, 5, 8), ("packed", 50, 40, 100), ("packed", 8, 900, 128), ("packed", 3000, 3, 64), ("packed", 3, 4000, 20)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("layout,b,t,d,lens", [(*c, lens) for c in CASES for lens in ("ends", "holes", "none")
                                                if c[0] != "dense" or lens == "ends"])  # dense rows have no lengths
def test_pool(layout, b, t, d, lens, dtype):
    dev = _dev()
    print(f"pool {layout} b={b} t={t} d={d} {lens} {dtype}", flush=True)
    c = make(layout, b, t, d, dtype, False, False, lens=lens)
    at = {k: None if c[k] is None else c[k].to(dev) for k in ("lengths", "offsets")}
    x = c["x"].double().numpy().reshape(-1, d)
    g = c["gl"].to(DT[dtype])
    for normalize in (True, False):
        f = mips.pool_normalize(c["x"].to(dev), normalize=normalize, **at)
        v, e, m, me, n, _ = reference(x, c["seqs"], normalize)
        hc.within(f.vectors, v, e, "vectors")
        hc.within(f.mean, m, me + 1e-36, "mean")
        dx = mips.pool_normalize_backward(g.to(dev), c["x"].shape, f, **at)
        want, tol = reference_grad(x, c["seqs"], normalize, g.double().numpy())
        hc.within(dx, want, tol, "grad_x")


@pytest.mark.parametrize("layout,b,t,d", [("dense", 5, 40, 64), ("dense", 3, 700, 64), ("padded", 6, 60, 128), ("packed", 6, 300, 72)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_strides_and_padding(layout, b, t, d, dtype):
    dev = _dev()
    c = make(layout, b, t, d, dtype, False, False)
    at = {k: None if c[k] is None else c[k].to(dev) for k in ("lengths", "offsets")}
    pad = torch.ones(c["x"].numel() // d, dtype=torch.bool)
    for lo, hi in c["seqs"]:
        pad[lo:hi] = False
    x = c["x"].clone()
    x.view(-1, d)[pad] = float("nan")
    x = x.to(dev)
    want = mips.pool_normalize(c["x"].to(dev), **at)
    assert torch.equal(mips.pool_normalize(x, **at).vectors, want.vectors)
    for k, shift in ((8, 8), (3, 1)):
        big = torch.full((*x.shape[:-2], x.shape[-2] + 2, d + k), float("nan"), dtype=x.dtype, device=dev)
        cut = big[..., 1:1 + x.shape[-2], shift:shift + d]
        cut.copy_(x)
        assert torch.equal(mips.pool_normalize(cut, **at).vectors, want.vectors)
    g = c["gl"].to(DT[dtype]).to(dev)
    dx = mips.pool_normalize_backward(g, x.shape, want, **at)
    wide = torch.zeros(b, d + 5, dtype=g.dtype, device=dev)
    wide[:, 1:1 + d] = g
    assert torch.equal(mips.pool_normalize_backward(wide[:, 1:1 + d], x.shape, want, **at), dx)
    row = g[:1].expand(b, d)
    assert torch.equal(mips.pool_normalize_backward(row, x.shape, want, **at),
                       mips.pool_normalize_backward(row.contiguous(), x.shape, want, **at))


def test_small_and_non_finite_sums():
    dev = _dev()
    x = torch.zeros(5, 3, 32, device=dev)
    x[1] = 1e-9           # below the epsilon's root
    x[2, 1, 4] = float("nan")
    x[3, 0, 7] = float("inf")
    x[4] = 1.0
    f = mips.pool_normalize(x)
    assert not f.vectors[0].any() and float(f.norm[0]) == pytest.approx(1e-6)
    assert torch.allclose(f.vectors[1], torch.full((32,), 1e-3, device=dev), rtol=1e-5)
    assert torch.isnan(f.vectors[2]).all() and not torch.isfinite(f.vectors[3, 7])
    assert torch.allclose(f.vectors[4], torch.full((32,), 32 ** -0.5, device=dev), rtol=1e-6)
    g = torch.randn(5, 32, device=dev)
    dx = mips.pool_normalize_backward(g, x.shape, f)
    for s in (0, 1):
        assert torch.allclose(dx[s], (g[s] * 1e6 / 3).expand(3, 32), rtol=1e-5)
    assert torch.isfinite(dx[4]).all()


def test_agrees_with_l2_normalize():
    """One row a sequence: the index's own normalisation, to a few units in the last place."""
    dev = _dev()
    x = torch.randn(1000, 128, device=dev)
    got = mips.pool_normalize(x[:, None]).vectors
    assert torch.allclose(got, mips.l2_normalize(x), rtol=136 * 2.0 ** -24, atol=0)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("d", [2, 7, 8, 9, 12, 15, 17, 63, 65, 513, 1031])
def test_widths(d, dtype):
    """Widths beside those that move by eight, whole sequences and ones that are joined."""
    dev = _dev()
    rng = np.random.default_rng(d)
    for b, t in ((3, 5), (2, 400)):
        x = torch.from_numpy(rng.standard_normal((b, t, d)).astype(np.float32)).to(DT[dtype])
        g = torch.from_numpy(rng.standard_normal((b, d)).astype(np.float32)).to(DT[dtype])
        n = torch.tensor([t] + [t // 3] * (b - 1))
        f = mips.pool_normalize(x.to(dev), lengths=n.to(dev))
        dx = mips.pool_normalize_backward(g.to(dev), x.shape, f, lengths=n.to(dev))
        for s in range(b):
            k = int(n[s])
            rows = x[s, :k].double()
            m = rows.mean(0)
            norm = float(m.norm())
            u = m / norm
            # the mean is off by (k + 3) u of the rows' mean size at most, the norm's sum by d u more
            room = (k + 3 + d + 8) * 2.0 ** -24 * rows.abs().mean(0).norm() / norm
            half = 2.0 ** -24 if dtype == "f32" else 2.0 ** -8
            assert (f.vectors[s].cpu().double() - u).abs().max() <= room + half
            want = (g[s].double() - u * float(u @ g[s].double())) / norm / k
            err = (dx[s].cpu().double() - torch.cat([want.expand(k, d), torch.zeros(t - k, d, dtype=torch.float64)])).abs().max()
            assert err <= (4 * room + half) * g[s].double().norm() / norm / k


@pytest.mark.parametrize("d", [5, 64, 100, 700])
@pytest.mark.parametrize("layout", ["padded", "packed"])
def test_gradient_of_a_mean_that_is_not_finite(layout, d):
    """Without normalisation the gradient is g / rows whatever the rows hold."""
    dev = _dev()
    for dtype in ("f32", "bf16"):
        c = make(layout, 5, 300, d, dtype, False, False)
        at = {k: None if c[k] is None else c[k].to(dev) for k in ("lengths", "offsets")}
        g = c["gl"].to(DT[dtype]).to(dev)
        want = mips.pool_normalize_backward(g, c["x"].shape, mips.pool_normalize(c["x"].to(dev), normalize=False, **at), **at)
        assert torch.isfinite(want).all() and want.any()
        x = c["x"].view(-1, d)
        for k, (lo, hi) in enumerate(c["seqs"]):
            if hi > lo:
                x[hi - 1, k % d] = (float("inf"), float("nan"), -float("inf"))[k % 3]
        f = mips.pool_normalize(c["x"].to(dev), normalize=False, **at)
        assert not torch.isfinite(f.mean).all()
        assert torch.equal(mips.pool_normalize_backward(g, c["x"].shape, f, **at), want)
