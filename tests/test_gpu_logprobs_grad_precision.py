"""How much of a bf16 call's gradient the rounding of its weights may cost.

Formulas and the binary32 part of the bound as in tests/test_gpu_logprobs_grad.py. The weights
w_bj = sum_i g_bi [id_bi = j] - p_bj G_b are rounded to bf16 for the second product, to nearest:
2^-8 of the weight that the formula has, not of the terms it is the difference of. A target that has
nearly all of the probability has a weight of nearly 0, and its query a gradient that is small beside
p G."""
import numpy as np
import pytest
import torch

import exact_inner_product_amd as mips
from tests.test_gpu_logprobs import U, grid, logits64

pytestmark = pytest.mark.gpu


def _dev():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    return torch.device("cuda:0")


def bounds(q, items, scale, ids, gl, at_targets=2.0 ** -8):
    """For queries and items: (formula in 64 bits, tolerance), both before the output's rounding."""
    b, n = q.shape[0], items.shape[0]
    l = logits64(q, items, scale).astype(np.float64)
    p = np.exp(l - l.max(1, keepdims=True))
    p /= p.sum(1, keepdims=True)
    hot, ahot = np.zeros((b, n)), np.zeros((b, n))
    for c in range(ids.shape[1]):
        np.add.at(hot, (np.arange(b), ids[:, c].numpy()), gl[:, c].double().numpy())
        np.add.at(ahot, (np.arange(b), ids[:, c].numpy()), gl[:, c].double().abs().numpy())
    w = hot - p * hot.sum(1, keepdims=True)
    a = ahot + p * ahot.sum(1, keepdims=True)
    lost = np.abs(w) * np.where(ahot > 0, at_targets, 2.0 ** -8)
    r = 2 * (4 * U * np.abs(l).max() + (n / 32 + 264) * U) + 8 * U
    qd, cd = q.double().numpy(), items.double().numpy()
    return ((scale * w @ cd, scale * ((r + (n + 70) * U) * a + lost) @ np.abs(cd)),
            (scale * w.T @ qd, scale * ((r + (b + 70) * U) * a + lost).T @ np.abs(qd)), 1 - p[np.arange(b), ids[:, 0]])


def check(got, want, tol, name):
    lo, hi = (torch.from_numpy(want + s * tol).bfloat16().double().numpy() for s in (-1, 1))
    y = got.double().cpu().numpy()
    assert ((lo <= y) & (y <= hi)).all(), \
        f"{name}: error {np.linalg.norm(y - want) / np.linalg.norm(want):.2g} of the gradient's norm"


@pytest.mark.parametrize("b,n,d,g", [(64, 500, 64, 1), (300, 2000, 128, 1), (90, 777, 256, 3), (130, 300, 24, 2),
                                     (20, 9000, 32, 1), (257, 300, 128, 64)])
@pytest.mark.parametrize("sign", [-1.0, 1.0, 0.0])
@pytest.mark.parametrize("confident", [False, True])
@pytest.mark.parametrize("extra", [False, True])
def test_weights_keep_what_the_formula_leaves(b, n, d, g, sign, confident, extra):
    dev = _dev()
    print(f"logprobs grad precision b={b} n={n} d={d} g={g} sign={sign} confident={confident} extra={extra}", flush=True)
    rng = np.random.default_rng(b + n)
    items = grid(rng, n, d, "bf16")
    ids = torch.from_numpy(rng.integers(0, n, (b, 1))).repeat(1, g)
    ids[:, g // 2:] = torch.from_numpy(rng.integers(0, n, (b, g - g // 2))) if g > 1 else ids
    if confident:  # queries lie on their target
        q, scale = items[ids[:, 0]], 24.0
    else:
        q, scale = grid(rng, b, d, "bf16"), 10.0
    gl = torch.from_numpy(rng.uniform(0.5, 1.5, (b, g)).astype(np.float32)) * (sign or 1.0)
    if sign == 0.0:  # both signs in a batch
        gl[::2] *= -1
    if g > 1 and confident:
        gl[:, g // 2:] *= 2.0 ** -10
    dq, di, rest = bounds(q, items, scale, ids, gl)
    if confident and d >= 64 and g == 1:
        assert np.median(rest) < 0.02  # the case it says it is
    args = [x.to(dev) for x in (q, items, ids)]
    f = mips.item_logprobs(*args, scale=scale)
    got = mips.item_logprobs_backward(gl.to(dev), *args, f, scale=scale, need_bias=extra)
    check(got[0], *dq, "queries")
    check(got[1], *di, "items")


@pytest.mark.parametrize("b,n,d,g", [(64, 500, 64, 1), (300, 2000, 128, 1), (90, 777, 256, 3), (20, 9000, 32, 1),
                                     (700, 700, 24, 1)])
@pytest.mark.parametrize("extra", [False, True])
def test_a_targets_weight_is_kept_to_16_bits(b, n, d, g, extra):
    """It is most of its item's gradient: 2^-16 of it may be lost, 2^-8 of the others."""
    dev = _dev()
    print(f"logprobs grad precision at targets b={b} n={n} d={d} g={g} extra={extra}", flush=True)
    rng = np.random.default_rng(b + n)
    items, q = grid(rng, n, d, "bf16"), grid(rng, b, d, "bf16")
    ids = torch.from_numpy(rng.integers(0, n, (b, g)))
    gl = torch.from_numpy(rng.uniform(-1.5, 1.5, (b, g)).astype(np.float32))
    dq, di, _ = bounds(q, items, 10.0, ids, gl, 2.0 ** -16)
    args = [x.to(dev) for x in (q, items, ids)]
    f = mips.item_logprobs(*args, scale=10.0)
    got = mips.item_logprobs_backward(gl.to(dev), *args, f, scale=10.0, need_bias=extra)
    check(got[0], *dq, "queries")
    check(got[1], *di, "items")
