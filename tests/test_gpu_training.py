"""The training operators together: the example's model learns, and the differentiable
functions give torch's own gradients of the same formulas.

The differentiable functions are compared with torch's autograd in binary64 on the CPU. Vectors
lie on a grid (exact inner products); binary32 sums of at most 64 terms and exponents of logits of
at most 8 leave relative errors below 1e-5 of the largest gradient, the tolerance."""
import importlib.util
import math
import os

import numpy as np
import pytest
import torch

from exact_inner_product_amd import autograd as mag
from tests.test_gpu_logprobs import bitmap, grid

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _dev():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    return torch.device("cuda:0")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_example_learns(dtype):
    _dev()
    spec = importlib.util.spec_from_file_location("train_two_tower", os.path.join(ROOT, "examples", "train_two_tower.py"))
    ex = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ex)
    print(f"example {dtype}", flush=True)
    table, losses = ex.train(steps=150, dtype=dtype, log=None)
    assert all(math.isfinite(x) for x in losses)
    assert sum(losses[-10:]) / 10 < losses[0] - 1.0
    hit, prob, entropy = ex.evaluate(table, dtype=dtype)
    # untrained: one group in eight, one item in 400, log 400 = 5.99 nats
    assert hit > 0.9 and prob > 4 / 400 and entropy < 5.5


def test_differentiable_functions_match_torch():
    dev = _dev()
    rng = np.random.default_rng(0)
    table = grid(rng, 40, 32, "f32")
    items = grid(rng, 60, 32, "f32")
    history = torch.from_numpy(rng.integers(0, 40, (30, 2)))
    ids = torch.from_numpy(rng.integers(0, 60, (30, 2)))
    mask = rng.random(60) < 0.1
    mask[ids.numpy().ravel()] = False
    bias = torch.from_numpy(rng.uniform(-1, 1, 60).astype(np.float32))

    def total(lp, h):
        return lp.sum() * 0.5 + (lp[:, 0] * lp[:, 1]).sum() * 0.25 - 0.3 * h.sum()

    t, i, b = (x.to(dev).requires_grad_() for x in (table, items, bias))
    q = mag.embedding(t, history.to(dev), scale=0.5).sum(1)
    lp, h = mag.item_logprobs(q, i, ids.to(dev), scale=4.0, bias=b, exclude=bitmap(mask).to(dev), entropy=True)
    total(lp, h).backward()

    t2, i2, b2 = (x.double().requires_grad_() for x in (table, items, bias))
    q2 = (t2[history] * 0.5).sum(1)
    l2 = (q2 @ i2.T) * 4.0 + b2
    l2 = l2.masked_fill(torch.from_numpy(mask), -math.inf)
    logp = torch.log_softmax(l2, 1)
    p = logp.exp()
    h2 = -(p * logp.masked_fill(torch.from_numpy(mask), 0.0)).sum(1)
    total(logp.gather(1, ids), h2).backward()
    for name, a, w in (("table", t, t2), ("items", i, i2), ("bias", b, b2)):
        err = (a.grad.double().cpu() - w.grad).abs().max()
        assert err <= 1e-5 * w.grad.abs().max(), (name, float(err))


def test_only_what_is_asked_for_is_computed():
    dev = _dev()
    rng = np.random.default_rng(1)
    items, q = grid(rng, 50, 16, "bf16").to(dev), grid(rng, 5, 16, "bf16").to(dev).requires_grad_()
    ids = torch.zeros((5, 1), dtype=torch.int32, device=dev)
    lp, h = mag.item_logprobs(q, items, ids, scale=2.0)
    assert h is None
    lp.sum().backward()
    assert q.grad is not None and q.grad.dtype == torch.bfloat16 and items.grad is None
