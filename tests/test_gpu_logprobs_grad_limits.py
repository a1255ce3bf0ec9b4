"""The gradient of the log probabilities and entropy where biases mask items: -inf or the lowest float.

Formulas, bounds and check() as in tests/test_gpu_logprobs_grad.py: a masked item has p = 0, so its
weight is that of the targets that name it, sum_i g_i [id_i = j], and it adds nothing to the errors."""
import numpy as np
import pytest
import torch

import exact_inner_product_amd as mips
from tests.test_gpu_logprobs import U, grid, logits64
from tests.test_gpu_logprobs_grad import check, run

pytestmark = pytest.mark.gpu
LOWEST = float(np.finfo(np.float32).min)
SHAPES = [("f32", 40, 333, 16), ("bf16", 70, 1000, 64), ("bf16", 300, 600, 128), ("f32", 130, 700, 128),
          ("bf16", 33, 290, 256)]


def _dev():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    return torch.device("cuda:0")


def masking_bias(rng, n, kind):
    """Biases of which two in five, and the first block of 32, mask their items."""
    low = rng.random(n) < 0.4
    low[:32] = True
    bias = rng.uniform(-8, 8, n).astype(np.float32)
    bias[low] = {"inf": -np.inf, "lowest": LOWEST, "both": np.where(np.arange(low.sum()) % 2, -np.inf, LOWEST)}[kind]
    return torch.from_numpy(bias)


def gradients64(q, items, scale, ids, gl, gh, bias):
    """(dq, dc, dbias and the magnitudes of their error bounds, r) as test_gpu_logprobs_grad.reference,
    with the targets of masked items."""
    b, n = q.shape[0], items.shape[0]
    l = logits64(q, items, scale, bias).astype(np.float64)
    live = l > -1e30
    m = np.where(live, l, -np.inf).max(1, keepdims=True)
    some = np.isfinite(m)
    e = np.where(live, np.exp(np.where(live, l, 0) - np.where(some, m, 0)), 0.0)
    z = np.where(some, e.sum(1, keepdims=True), 1.0)
    p = e / z
    lp = np.where(p > 0, np.log(np.where(p > 0, p, 1)), 0.0)
    ent = -(p * lp).sum(1, keepdims=True)
    h = np.zeros((b, 1)) if gh is None else gh.double().numpy()[:, None]
    hot, ahot = np.zeros((b, n)), np.zeros((b, n))
    for r in range(b):
        for c in range(ids.shape[1]):
            j = int(ids[r, c])
            if 0 <= j < n and some[r, 0]:
                hot[r, j] += float(gl[r, c])
                ahot[r, j] += abs(float(gl[r, c]))
    G, aG = hot.sum(1, keepdims=True), ahot.sum(1, keepdims=True)
    w = hot - p * (G + h * (lp + ent))
    a = ahot + p * (aG + np.abs(h) * (np.abs(lp) + ent + 2))
    qd, cd = q.double().numpy(), items.double().numpy()
    big = np.abs(np.where(live, l, 0)).max(initial=0)
    r = 2 * (4 * U * big + (n / 32 + 264) * U) + 8 * U
    return [(scale * w @ cd, scale * a @ np.abs(cd), n), (scale * w.T @ qd, scale * a.T @ np.abs(qd), b),
            (w.sum(0), a.sum(0), b)], r


def inputs(rng, dtype, b, n, d, kind):
    q, items = grid(rng, b, d, dtype), grid(rng, n, d, dtype)
    bias = masking_bias(rng, n, kind)
    ids = torch.from_numpy(rng.integers(-1, n + 1, (b, 2))).to(torch.int32)
    ids[::3, 0] = 5  # a masked item as a target
    gl = torch.from_numpy(rng.uniform(-1, 1, (b, 2)).astype(np.float32))
    return q, items, bias, ids, gl


@pytest.mark.parametrize("dtype,b,n,d", SHAPES)
@pytest.mark.parametrize("kind", ["inf", "lowest", "both"])
@pytest.mark.parametrize("need_bias", [False, True])
def test_masking_biases(dtype, b, n, d, kind, need_bias):
    dev = _dev()
    print(f"logprobs grad masking bias {kind} {dtype} b={b} n={n} d={d} need_bias={need_bias}", flush=True)
    rng = np.random.default_rng(n + d + len(kind))
    q, items, bias, ids, gl = inputs(rng, dtype, b, n, d, kind)
    refs, r = gradients64(q, items, 10.0, ids, gl, None, bias)
    check(run(q, items, ids, gl, None, 10.0, bias, None, dev, need_bias), refs, r, dtype == "bf16")


@pytest.mark.parametrize("scale", [1e-6, 1e6])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_masking_biases_at_the_scales_limits(dtype, scale):
    """The bias is divided by the scale on its way: neither end overflows into a NaN. (At a scale of
    1e6 one item has all the probability up to the logits' rounding: only finiteness is asked.)"""
    dev = _dev()
    rng = np.random.default_rng(3)
    q, items, bias, ids, gl = inputs(rng, dtype, 30, 200, 32, "both")
    bias[40:60] = -1e33
    got = run(q, items, ids, gl, None, scale, bias, None, dev)
    if scale < 1:
        refs, r = gradients64(q, items, scale, ids, gl, None, bias)
        check(got, refs, r, dtype == "bf16")
    assert all(torch.isfinite(x.float()).all() for x in got)


@pytest.mark.parametrize("dtype,b,n,d", SHAPES)
@pytest.mark.parametrize("kind", ["inf", "lowest", "both"])
def test_masking_biases_with_entropy(dtype, b, n, d, kind):
    """0 log 0 = 0: neither the pass that owns the items nor the one that streams them makes it a NaN.
    The forward pass' entropy is given from 64 bits."""
    dev = _dev()
    print(f"logprobs grad entropy, masking bias {kind} {dtype} b={b} n={n} d={d}", flush=True)
    rng = np.random.default_rng(n + d + len(kind))
    q, items, bias, ids, gl = inputs(rng, dtype, b, n, d, kind)
    gh = torch.from_numpy(rng.uniform(-1, 1, b).astype(np.float32))
    gh[::4] = 0.0
    refs, r = gradients64(q, items, 10.0, ids, gl, gh, bias)
    l = logits64(q, items, 10.0, bias).astype(np.float64)
    l[l < -1e30] = -np.inf
    lp = l - np.logaddexp.reduce(l, axis=1, keepdims=True)
    entropy = torch.from_numpy((-(np.exp(lp) * np.where(np.isfinite(lp), lp, 0)).sum(1)).astype(np.float32))
    args = [x.to(dev) for x in (q, items, ids)]
    f = mips.item_logprobs(*args, scale=10.0, bias=bias.to(dev), entropy=False)
    f.entropy = entropy.to(dev)
    got = mips.item_logprobs_backward(gl.to(dev), *args, f, scale=10.0, bias=bias.to(dev), grad_entropy=gh.to(dev),
                                      need_bias=True)
    check(got, refs, r, dtype == "bf16")


def test_large_entropy_gradients_of_masked_items():
    """h log p overflows where log p is that of a masked item; p = 0 all the same."""
    dev = _dev()
    rng = np.random.default_rng(9)
    q, items, bias, _, _ = inputs(rng, "bf16", 40, 300, 64, "both")
    low = bias < -1e30
    q, items, bias = q.to(dev), items.to(dev), bias.to(dev)
    f = mips.item_logprobs(q, items, scale=5.0, bias=bias)
    f.entropy = torch.ones(40, device=dev)
    dq, di, db = mips.item_logprobs_backward(None, q, items, None, f, scale=5.0, bias=bias, need_bias=True,
                                             grad_entropy=torch.full((40,), 1e12, device=dev))
    assert torch.isfinite(dq.float()).all() and torch.isfinite(di.float()).all() and torch.isfinite(db).all()
    assert (di[low] == 0).all() and (db[low] == 0).all()


@pytest.mark.parametrize("dtype,d", [("f32", 16), ("bf16", 64)])
def test_scores_of_minus_infinity_with_entropy(dtype, d):
    """Items of p = 0 by their own rows have no gradient either (the queries' would multiply 0 with
    those rows)."""
    dev = _dev()
    rng = np.random.default_rng(d)
    b, n = 50, 200
    q, items = grid(rng, b, d, dtype), grid(rng, n, d, dtype)
    q[:, 0] = q[:, 0].abs() + 2.0 ** -8
    low = np.arange(n) % 3 == 0
    items[torch.from_numpy(low), 0] = -float("inf")
    gh = torch.from_numpy(rng.uniform(-1, 1, b).astype(np.float32)).to(dev)
    q, items = q.to(dev), items.to(dev)
    f = mips.item_logprobs(q, items, scale=5.0)
    f.entropy = torch.ones(b, device=dev)
    _, di, db = mips.item_logprobs_backward(None, q, items, None, f, scale=5.0, grad_entropy=gh, need_queries=False,
                                            need_bias=True)
    for x in (di.float().cpu(), db.cpu()):
        assert torch.isfinite(x).all() and (x[low] == 0).all() and (x[~low] != 0).any()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("kind", ["inf", "lowest"])
@pytest.mark.parametrize("entropy", [False, True])
def test_queries_that_biases_leave_without_an_item(dtype, kind, entropy):
    """No gradient, as under a bitmap that leaves nothing; also where only some queries are left so."""
    dev = _dev()
    rng = np.random.default_rng(4)
    b, n, d = 70, 150, 32
    q, items = grid(rng, b, d, dtype).to(dev), grid(rng, n, d, dtype).to(dev)
    ids = torch.from_numpy(rng.integers(0, n, (b, 2))).to(dev)
    gl = torch.ones(b, 2, device=dev)
    gh = torch.ones(b, device=dev) if entropy else None
    bias = torch.full((n,), -np.inf if kind == "inf" else LOWEST, device=dev)
    f = mips.item_logprobs(q, items, ids, scale=5.0, bias=bias)
    got = mips.item_logprobs_backward(gl, q, items, ids, f, scale=5.0, bias=bias, grad_entropy=gh, need_bias=True)
    assert all((x == 0).all() for x in got)
    # every item masked but number 7, which a bitmap takes from the odd queries
    bias[7] = 0.0
    words = torch.zeros((b, (n + 31) // 32), dtype=torch.int32, device=dev)
    words[1::2, 0] = 1 << 7
    kw = dict(scale=5.0, bias=bias, exclude=words)
    f = mips.item_logprobs(q, items, ids, **kw)
    dq, di, db = mips.item_logprobs_backward(gl, q, items, ids, f, grad_entropy=gh, need_bias=True, **kw)
    assert (dq[1::2] == 0).all() and torch.isfinite(dq.float()).all() and torch.isfinite(di.float()).all()
    # even queries have p_7 = 1, and so w = sum_i g_i ([id_i = j] - [j = 7])
    want = torch.zeros(n, device=dev)
    want.index_add_(0, ids[::2].reshape(-1), torch.ones(b, device=dev))
    want[7] -= float(b)
    assert (db - want).abs().max() <= 1e-3
