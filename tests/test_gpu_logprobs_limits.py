"""Log probabilities where logits are infinite, of the lowest value or NaN: biases that mask items,
scores of -inf, rows of NaN, and queries that such values leave without an item.

Definitions as in tests/test_gpu_logprobs.py, whose tolerances hold: a logit of -inf (or far below
every other one) has probability 0 and adds 0 to the entropy, so the finite logits alone decide the
sums and the bounds. The log probability of an item with the lowest finite bias is that bias: what is
subtracted is below its last place."""
import numpy as np
import pytest
import torch

import exact_inner_product_amd as mips
from tests.test_gpu_logprobs import bitmap, check, grid, logits64

pytestmark = pytest.mark.gpu
LOWEST = float(np.finfo(np.float32).min)


def _dev():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    return torch.device("cuda:0")


def masking_bias(rng, n, kind, share=0.4):
    """(bias, which items it masks): -inf, the lowest float, or both in turn."""
    low = rng.random(n) < share
    bias = rng.uniform(-8, 8, n).astype(np.float32)
    bias[low] = {"inf": -np.inf, "lowest": LOWEST, "both": np.where(np.arange(low.sum()) % 2, -np.inf, LOWEST)}[kind]
    return torch.from_numpy(bias), low


SHAPES = [("f32", 5, 333, 16), ("bf16", 40, 2000, 64), ("bf16", 300, 1000, 128), ("f32", 70, 70000, 32),
          ("bf16", 9, 3333, 256), ("bf16", 600, 90000, 16)]


@pytest.mark.parametrize("dtype,b,n,d", SHAPES)
@pytest.mark.parametrize("kind", ["inf", "lowest", "both"])
def test_entropy_under_masking_biases(dtype, b, n, d, kind):
    dev = _dev()
    print(f"logprobs masking bias {kind} {dtype} b={b} n={n} d={d}", flush=True)
    rng = np.random.default_rng(n + len(kind))
    items, q = grid(rng, n, d, dtype), grid(rng, b, d, dtype)
    bias, low = masking_bias(rng, n, kind)
    low[:64] = True  # whole tiles too
    bias[:64] = -np.inf if kind != "lowest" else LOWEST
    ids = torch.from_numpy(np.flatnonzero(~low)[rng.integers(0, (~low).sum(), (b, 2))]).to(torch.int32)
    r = mips.item_logprobs(q.to(dev), items.to(dev), ids.to(dev), scale=10.0, bias=bias.to(dev))
    l = logits64(q, items, 10.0, bias)
    l[:, low] = -np.inf
    check(r, l, ids)


@pytest.mark.parametrize("dtype,d", [("f32", 16), ("bf16", 64), ("bf16", 128)])
def test_entropy_with_scores_of_minus_infinity(dtype, d):
    """Items whose rows hold -inf against queries that are positive there: p = 0 without a bias."""
    dev = _dev()
    rng = np.random.default_rng(d)
    items, q = grid(rng, 3000, d, dtype), grid(rng, 40, d, dtype)
    q[:, 0] = q[:, 0].abs() + 2.0 ** -8
    low = rng.random(3000) < 0.3
    low[:32] = True
    items[torch.from_numpy(low), 0] = -float("inf")
    ids = torch.from_numpy(np.flatnonzero(~low)[:80].reshape(40, 2))
    r = mips.item_logprobs(q.to(dev), items.to(dev), ids.to(dev), scale=10.0)
    l = logits64(q, torch.where(torch.from_numpy(low)[:, None], 0, items), 10.0)
    l[:, low] = -np.inf
    check(r, l, ids)


@pytest.mark.parametrize("first", [0, 9984, 19968])
@pytest.mark.parametrize("what", ["rows", "bias"])
@pytest.mark.parametrize("k", [0, 4])
def test_a_block_of_nan_reaches_every_query(first, what, k):
    """So many queries that a wave takes several tiles of 64 items: the NaN are in its first, a middle
    or the last one, as whole rows or biases."""
    dev = _dev()
    rng = np.random.default_rng(3)
    n, b, d = 20032, 2100, 64
    items, q = grid(rng, n, d, "bf16").to(dev), grid(rng, b, d, "bf16").to(dev)
    bias = torch.zeros(n, device=dev)
    if what == "rows":
        items[first:first + 64] = float("nan")
    else:
        bias[first:first + 64] = float("nan")
    ids = torch.full((b, 1), 5000, device=dev)
    r = mips.item_logprobs(q, items, ids, scale=10.0, bias=bias if what == "bias" else None, alternatives=k)
    assert torch.isnan(r.logsumexp).all() and torch.isnan(r.entropy).all() and torch.isnan(r.logprobs).all()
    # few queries over many items, f32, and a single wide tile of a wave
    items, q = grid(rng, 300000, 16, "f32").to(dev), grid(rng, 3, 16, "f32").to(dev)
    items[first:first + 64] = float("nan")
    r = mips.item_logprobs(q, items, scale=10.0, alternatives=k)
    assert torch.isnan(r.logsumexp).all() and torch.isnan(r.entropy).all()


def test_nan_rows_behind_a_bitmap_stay_out():
    """The block of NaN is excluded for some queries: those are finite, the others NaN."""
    dev = _dev()
    rng = np.random.default_rng(6)
    n, b, d = 5000, 70, 64
    items, q = grid(rng, n, d, "bf16"), grid(rng, b, d, "bf16")
    held = items.clone()
    held[:64] = float("nan")
    mask = np.zeros((b, n), bool)
    mask[::2, :64] = True
    r = mips.item_logprobs(q.to(dev), held.to(dev), scale=10.0, exclude=bitmap(mask).to(dev))
    assert torch.isnan(r.logsumexp[1::2]).all() and torch.isnan(r.entropy[1::2]).all()
    even = mips.ItemLogprobs(None, r.logsumexp[::2], r.entropy[::2], None, None)
    check(even, logits64(q, items, 10.0, None, mask)[::2])


@pytest.mark.parametrize("k", [0, 5])
@pytest.mark.parametrize("kind", ["inf", "lowest", "both"])
def test_given_ids_of_masked_items(kind, k):
    """logp = l - lse: -inf, or the lowest float itself."""
    dev = _dev()
    rng = np.random.default_rng(1)
    n, b = 777, 37
    items, q = grid(rng, n, 64, "bf16"), grid(rng, b, 64, "bf16")
    bias, low = masking_bias(rng, n, kind)
    ids = torch.from_numpy(np.flatnonzero(low)[rng.integers(0, low.sum(), (b, 3))])
    r = mips.item_logprobs(q.to(dev), items.to(dev), ids.to(dev), scale=10.0, bias=bias.to(dev), alternatives=k)
    assert torch.equal(r.logprobs.cpu(), bias[ids])


@pytest.mark.parametrize("k", [0, 5])
@pytest.mark.parametrize("kind", ["inf", "lowest"])
def test_biases_that_leave_nothing(kind, k):
    """As under a bitmap that leaves nothing: lse and log probabilities -inf, entropy 0, no alternatives."""
    dev = _dev()
    rng = np.random.default_rng(2)
    n, b = 700, 35
    items, q = grid(rng, n, 32, "bf16").to(dev), grid(rng, b, 32, "bf16").to(dev)
    bias = torch.full((n,), -np.inf if kind == "inf" else LOWEST, device=dev)
    ids = torch.from_numpy(rng.integers(-1, n, (b, 2))).to(dev)
    r = mips.item_logprobs(q, items, ids, scale=10.0, bias=bias, alternatives=k)
    assert (r.logsumexp == -np.inf).all() and (r.entropy == 0).all()
    assert torch.equal(r.logprobs, torch.where(ids < 0, 0.0, -np.inf).float())
    if k:
        assert (r.alt_ids == -1).all() and (r.alt_logprobs == -np.inf).all()


@pytest.mark.parametrize("dtype,b,n,d", SHAPES)
@pytest.mark.parametrize("kind", ["inf", "lowest", "both"])
@pytest.mark.parametrize("left", [3, None])
def test_alternatives_under_masking_biases(dtype, b, n, d, kind, left):
    """Masked items are no alternatives, wherever they lie; fewer live items than alternatives too."""
    dev = _dev()
    print(f"logprobs alternatives, masking bias {kind} {dtype} b={b} n={n} d={d} left={left}", flush=True)
    rng = np.random.default_rng(n + len(kind))
    items, q = grid(rng, n, d, dtype), grid(rng, b, d, dtype)
    bias, low = masking_bias(rng, n, kind)
    if left:
        keep = rng.permutation(n)[:left]
        low[:] = True
        low[keep] = False
        bias[:] = torch.where(torch.arange(n) % 2 == 0, LOWEST, -np.inf) if kind == "both" else bias[bias < -1e30][0]
        bias[torch.from_numpy(keep)] = torch.arange(left).float()
    r = mips.item_logprobs(q.to(dev), items.to(dev), scale=10.0, bias=bias.to(dev), entropy=False, alternatives=17)
    l = logits64(q, items, 10.0, bias)
    l[:, low] = -np.inf
    check(r, l, None, 17)


def test_nan_logits_are_no_alternatives():
    """The others keep their order; their log probabilities are NaN, as the log-sum-exp is."""
    dev = _dev()
    rng = np.random.default_rng(5)
    for n, d in ((700, 64), (90000, 16)):
        items, q = grid(rng, n, d, "bf16"), grid(rng, 40, d, "bf16")
        bad = rng.random(n) < 0.02
        bad[64:128] = True
        held = items.clone()
        held[torch.from_numpy(bad)] = float("nan")
        r = mips.item_logprobs(q.to(dev), held.to(dev), scale=5.0, alternatives=9)
        l = logits64(q, items, 5.0)
        l[:, bad] = -np.inf
        want = np.lexsort((np.broadcast_to(np.arange(n), l.shape), -l), axis=1)[:, :9]
        assert np.array_equal(r.alt_ids.cpu().numpy(), want)
        assert torch.isnan(r.logsumexp).all() and torch.isnan(r.alt_logprobs).all()
