"""The gradient of the log probabilities and entropy over an item table, against the formulas in
64 bits and against differences of the definition in 64 bits.

Tolerances, u = 2^-24, vectors on a grid (exact inner products; tests/test_gpu_logprobs.py). A
probability's relative error is at most r = 2 (4 u L + (n/32 + 264) u) + 8 u, L = max |l|: the
exponent's and the log-sum-exp's errors. With a_bj = p_bj (|G_b| + |h_b| (|log p_bj| + H_b)) +
sum_i |g_bi| [id_bi = j], the magnitudes that make up a weight, a gradient's error is at most
scale * (k r + (m + 70) u) * sum a |row| for a sum of m terms; k = 3 covers the entropy term's log p
and H, each with an error of at most r (1 + |log p|), through the factor |log p| + H + 2 in
place of |log p| + H. In bf16 each weight is rounded once to 8 significant bits (2^-8), and the
result, a value of that interval, to nearest: it lies between the roundings of the interval's
ends."""
import numpy as np
import pytest
import torch

import exact_inner_product_amd as mips
from tests.test_gpu_logprobs import U, bitmap, grid, logits64

pytestmark = pytest.mark.gpu


def _dev():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    return torch.device("cuda:0")


def reference(q, items, scale, ids, gl, gh, bias, mask):
    """(dq, dc, dbias, and for each the magnitudes of its error bound) in 64 bits."""
    b, n = q.shape[0], items.shape[0]
    l = logits64(q, items, scale, bias, mask).astype(np.float64)
    m = l.max(1, keepdims=True)
    some = np.isfinite(m)
    e = np.where(np.isfinite(l), np.exp(l - np.where(some, m, 0)), 0.0)
    z = e.sum(1, keepdims=True)
    p = e / np.where(some, z, 1)
    with np.errstate(divide="ignore"):
        lp = np.where(p > 0, np.log(np.where(p > 0, p, 1)), 0.0)
    ent = -(p * lp).sum(1, keepdims=True)
    h = np.zeros((b, 1)) if gh is None else gh.double().numpy()[:, None]
    hot, ahot = np.zeros((b, n)), np.zeros((b, n))
    if ids is not None:
        i, g = ids.numpy().astype(np.int64), gl.double().numpy()
        for r in range(b):
            for c in range(i.shape[1]):
                if 0 <= i[r, c] < n and np.isfinite(l[r, i[r, c]]):
                    hot[r, i[r, c]] += g[r, c]
                    ahot[r, i[r, c]] += abs(g[r, c])
    G, aG = hot.sum(1, keepdims=True), ahot.sum(1, keepdims=True)
    w = hot - p * (G + h * (lp + ent))
    a = ahot + p * (aG + np.abs(h) * (np.abs(lp) + ent + 2))
    qd, cd = q.double().numpy(), items.double().numpy()
    big = np.abs(np.where(np.isfinite(l), l, 0)).max(initial=0)
    r = 2 * (4 * U * big + (n / 32 + 264) * U) + 8 * U
    return [(scale * w @ cd, scale * a @ np.abs(cd), n), (scale * w.T @ qd, scale * a.T @ np.abs(qd), b),
            (w.sum(0), a.sum(0), b)], r


def check(got, refs, r, bf16):
    for name, x, (want, mag, m) in zip(("queries", "items", "bias"), got, refs):
        if x is None:
            continue
        tol = (3 * r + (m + 70) * U) * mag
        lo, hi = want - tol, want + tol
        if x.dtype == torch.bfloat16:
            lo, hi = (want + s * (tol + 2.0 ** -8 * mag) for s in (-1, 1))
            lo, hi = (torch.from_numpy(v).bfloat16().double().numpy() for v in (lo, hi))
        y = x.double().cpu().numpy()
        assert y.shape == want.shape
        assert ((lo <= y) & (y <= hi)).all(), f"{name}: off by {np.abs(y - want).max()}, magnitude {mag.max()}"


def run(q, items, ids, gl, gh, scale, bias, words, dev, need_bias=True):
    put = lambda t: None if t is None else t.to(dev)  # noqa: E731
    kw = dict(scale=scale, bias=put(bias), exclude=put(words))
    f = mips.item_logprobs(put(q), put(items), put(ids), **kw)
    return mips.item_logprobs_backward(put(gl), put(q), put(items), put(ids), f, grad_entropy=put(gh),
                                       need_bias=need_bias, **kw)


CASES = [
    # dtype, b, n, d, g
    ("f32", 1, 1, 16, 1), ("bf16", 1, 1, 16, 1), ("f32", 3, 31, 4, 2), ("bf16", 2, 33, 8, 1), ("f32", 64, 64, 32, 1),
    ("bf16", 65, 63, 24, 3), ("f32", 100, 100, 100, 1), ("bf16", 128, 300, 100, 1), ("f32", 1000, 1000, 64, 1),
    ("f32", 70, 513, 128, 9), ("bf16", 300, 1000, 128, 1), ("bf16", 130, 777, 256, 20), ("bf16", 33, 500, 200, 64),
    ("bf16", 20, 9000, 64, 1), ("bf16", 1500, 130, 32, 1), ("f32", 10, 5000, 16, 1), ("bf16", 257, 257, 128, 1),
]


@pytest.mark.parametrize("dtype,b,n,d,g", CASES)
def test_logprobs_gradient(dtype, b, n, d, g):
    dev = _dev()
    print(f"logprobs grad {dtype} b={b} n={n} d={d} g={g}", flush=True)
    rng = np.random.default_rng(b + n + d)
    q, items = grid(rng, b, d, dtype), grid(rng, n, d, dtype)
    ids = torch.from_numpy(rng.integers(-1, n + 1, (b, g))).to(torch.int64 if b % 2 else torch.int32)
    gl = torch.from_numpy(rng.uniform(-1, 1, (b, g)).astype(np.float32))
    refs, r = reference(q, items, 15.0, ids, gl, None, None, None)
    got = run(q, items, ids, gl, None, 15.0, None, None, dev)
    check(got, refs, r, dtype == "bf16")
    plain = run(q, items, ids, gl, None, 15.0, None, None, dev, need_bias=False)
    check(plain, refs, r, dtype == "bf16")
    again = run(q, items, ids, gl, None, 15.0, None, None, dev, need_bias=False)
    assert torch.equal(plain[0], again[0]) and torch.equal(plain[1], again[1])


@pytest.mark.parametrize("dtype,b,n,d", [("f32", 40, 333, 16), ("bf16", 70, 1000, 64), ("bf16", 300, 600, 128),
                                         ("f32", 130, 700, 128), ("bf16", 33, 290, 256)])
@pytest.mark.parametrize("kind", ["entropy", "bias", "shared", "own", "all", "entropy only", "bias+own+entropy"])
def test_entropy_bias_and_masks(dtype, b, n, d, kind):
    dev = _dev()
    print(f"logprobs grad {kind} {dtype} b={b} n={n} d={d}", flush=True)
    rng = np.random.default_rng(n + d + len(kind))
    q, items = grid(rng, b, d, dtype), grid(rng, n, d, dtype)
    ids = gl = gh = bias = mask = None
    if kind != "entropy only":
        ids = torch.from_numpy(rng.integers(-1, n + 1, (b, 2))).to(torch.int32)
        ids[:, 1] = ids[:, 0].clone()  # one item twice
        gl = torch.from_numpy(rng.uniform(-1, 1, (b, 2)).astype(np.float32))
    if "entropy" in kind:
        gh = torch.from_numpy(rng.uniform(-1, 1, b).astype(np.float32))
    if "bias" in kind:
        bias = torch.from_numpy(rng.uniform(-8, 8, n).astype(np.float32))
    if kind == "shared":
        mask = np.broadcast_to(rng.random(n) < 0.3, (b, n))
    elif "own" in kind:
        mask = rng.random((b, n)) < rng.random((b, 1))
        mask[0] = True
        mask[1] = True
        mask[1, n - 1] = False
    elif kind == "all":
        mask = np.ones((b, n), bool)
    words = None if mask is None else bitmap(mask if "own" in kind else mask[0])
    held = items.clone()
    if kind in ("shared", "all"):
        bad = np.flatnonzero(mask[0])
        held[bad[::3]] = float("nan")
        held[bad[1::3]] = float("inf")
    refs, r = reference(q, items, 10.0, ids, gl, gh, bias, mask)
    if kind in ("shared", "all"):  # excluded rows: exactly zero
        got = run(q, held, ids, gl, gh, 10.0, bias, words, dev)
        assert (got[1].cpu()[torch.from_numpy(mask[0].copy())] == 0).all()
        assert (got[2].cpu()[torch.from_numpy(mask[0].copy())] == 0).all()
    else:
        got = run(q, held, ids, gl, gh, 10.0, bias, words, dev)
    check(got, refs, r, dtype == "bf16")


def test_against_differences():
    """Central differences of sum(G * logp) + sum(h * H), the definition in 64 bits, for every
    element of queries, items and bias: within the formula's bound plus the differences' own error
    (step 1e-5, third derivatives of at most scale^3: 1e-7)."""
    dev = _dev()
    rng = np.random.default_rng(1)
    b, n, d, scale = 4, 7, 8, 3.0
    q, items = grid(rng, b, d, "f32"), grid(rng, n, d, "f32")
    ids = torch.from_numpy(rng.integers(0, n, (b, 2)))
    gl = torch.from_numpy(rng.uniform(-1, 1, (b, 2)).astype(np.float32))
    gh = torch.from_numpy(rng.uniform(-1, 1, b).astype(np.float32))
    bias = torch.from_numpy(rng.uniform(-1, 1, n).astype(np.float32))
    mask = rng.random((b, n)) < 0.2
    mask[np.arange(b), ids[:, 0]] = mask[np.arange(b), ids[:, 1]] = False

    def loss(qd, cd, bd):
        l = np.where(mask, -np.inf, qd @ cd.T * scale + bd)
        lse = np.log(np.exp(l).sum(1, keepdims=True))
        p = np.exp(l - lse)
        h = -(p * np.where(p > 0, l - lse, 0)).sum(1)
        return float((gl.double().numpy() * (np.take_along_axis(l, ids.numpy(), 1) - lse)).sum() + (gh.double().numpy() * h).sum())

    x = [q.double().numpy(), items.double().numpy(), bias.double().numpy()]
    refs, r = reference(q, items, scale, ids, gl, gh, bias, mask)
    got = run(q, items, ids, gl, gh, scale, bias, bitmap(mask), dev)
    for k in range(3):
        y = got[k].double().cpu().numpy()
        for at in np.ndindex(x[k].shape):
            up, dn = [v.copy() for v in x], [v.copy() for v in x]
            up[k][at] += 1e-5
            dn[k][at] -= 1e-5
            diff = (loss(*up) - loss(*dn)) / 2e-5
            tol = (3 * r + (refs[k][2] + 70) * U) * refs[k][1][at] + 1e-7
            assert abs(diff - y[at]) <= tol, (k, at)


def test_strided_rows_streams_and_graph():
    dev = _dev()
    rng = np.random.default_rng(2)
    wide_q, wide_i = grid(rng, 90, 80, "bf16"), grid(rng, 700, 80, "bf16")
    ids = torch.from_numpy(rng.integers(0, 700, (90, 1)))
    gl = torch.ones(90, 1) / 90
    for cut in (slice(0, 64), slice(1, 65), slice(4, 41)):
        q, items = wide_q[:, cut], wide_i[:, cut]
        refs, r = reference(q, items, 6.0, ids, gl, None, None, None)
        dq, di = wide_q.to(dev)[:, cut], wide_i.to(dev)[:, cut]
        f = mips.item_logprobs(dq, di, ids.to(dev), scale=6.0)
        check(mips.item_logprobs_backward(gl.to(dev), dq, di, ids.to(dev), f, scale=6.0), refs, r, True)
    q, items, ids, gl = wide_q[:, :64].to(dev), wide_i[:, :64].to(dev), ids.to(dev), gl.to(dev)
    f = mips.item_logprobs(q, items, ids, scale=6.0)
    want = mips.item_logprobs_backward(gl, q, items, ids, f, scale=6.0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = mips.item_logprobs_backward(gl, q, items, ids, f, scale=6.0)
    side.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        f = mips.item_logprobs(q, items, ids, scale=6.0)
        res = mips.item_logprobs_backward(gl, q, items, ids, f, scale=6.0)
    for i in range(3):
        wide_q = grid(rng, 90, 80, "bf16").to(dev)
        q.copy_(wide_q[:, :64])
        graph.replay()
        torch.cuda.synchronize()
        f2 = mips.item_logprobs(q, items, ids, scale=6.0)
        want = mips.item_logprobs_backward(gl, q, items, ids, f2, scale=6.0)
        assert torch.equal(res[0], want[0]) and torch.equal(res[1], want[1]), i


def test_refusals():
    dev = _dev()
    q, items = torch.zeros(3, 32, device=dev), torch.zeros(10, 32, device=dev)
    ids = torch.zeros((3, 1), dtype=torch.int32, device=dev)
    f = mips.item_logprobs(q, items, ids, entropy=False)
    g = torch.zeros(3, 1, device=dev)
    with pytest.raises(ValueError):
        mips.item_logprobs_backward(g, q, items, ids, f, grad_entropy=torch.zeros(3, device=dev))
    with pytest.raises(ValueError):
        mips.item_logprobs_backward(g[:2], q, items, ids, f)
    with pytest.raises(ValueError):
        mips.item_logprobs_backward(None, q, items, ids, f)
    with pytest.raises(ValueError):
        mips.item_logprobs_backward(g.bfloat16(), q, items, ids, f)
    with pytest.raises(TypeError):
        mips.item_logprobs_backward(g, q, mips.empty_corpus(100, 32, "f32", dev), ids, f)
    with pytest.raises(mips.MipsError, match="invalid argument"):
        mips.item_logprobs_backward(g, q, items, ids, f, need_queries=False, need_items=False)
    with pytest.raises(mips.MipsError, match="workspace too small"):
        mips.item_logprobs_backward(g, q, items, ids, f, workspace=mips.empty_workspace(256, dev))
    many = torch.zeros((3, 65), dtype=torch.int32, device=dev)
    f = mips.item_logprobs(q, items, many)
    with pytest.raises(mips.MipsError, match="unsupported"):
        mips.item_logprobs_backward(torch.zeros(3, 65, device=dev), q, items, many, f)
