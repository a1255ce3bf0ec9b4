"""Log probabilities over an item table against the definition in 64 bits on the CPU.

Vectors lie on a grid (multiples of 2^-8, or 2^-10 in f32), so that every inner product is exact
in binary32 and the logits l = fl(fl(s * scale) + bias) are the same numbers on both sides: the
alternatives' ids must be equal, ties by the lowest id.

Tolerances, u = 2^-24. The kernel's exponents are y = s * (scale * log2 e) in binary32: with
L = max |l|, each is off by at most d = 4 u L (the rounded constant and product, and the
reference's own rounding), an exp2 by 2 u, and the sums run over at most C = n/32 + 200 additions a
lane and join: rho = d + (C + 64) u bounds the relative error of a sum (64 u covers the exponents'
own rounding, |y - m| <= 40 where a term counts). lse is then within rho + 2 u (|lse| + 1), a log
probability within twice that, and the entropy, an average of |log p| with those weights, within
4 rho (H + 1 + 40) + 2 u H."""
import math

import numpy as np
import pytest
import torch

import exact_inner_product_amd as mips

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
U = 2.0 ** -24


def _dev():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    return torch.device("cuda:0")


def grid(rng, n, d, dtype):
    step = 256.0 if dtype == "bf16" else 1024.0
    x = rng.standard_normal((n, d))
    x /= np.sqrt((x * x).sum(1, keepdims=True)) + 1e-30
    return torch.from_numpy((np.round(x * step) / step).astype(np.float32)).to(DT[dtype])


def bitmap(mask):
    """int32 words of a boolean [.., n] (True: excluded)."""
    m = np.asarray(mask, bool)
    n = m.shape[-1]
    pad = np.zeros((*m.shape[:-1], (n + 31) // 32 * 32), np.uint8)
    pad[..., :n] = m
    words = np.packbits(pad.reshape(*m.shape[:-1], -1, 32), axis=-1, bitorder="little")
    return torch.from_numpy(np.ascontiguousarray(words).view(np.int32)[..., 0])


def logits64(q, items, scale, bias=None, mask=None):
    """The logits as binary32 numbers (exact on the grid), masked ones -inf."""
    s = (q.double().numpy() @ items.double().numpy().T).astype(np.float32)
    l = s * np.float32(scale)
    if bias is not None:
        l = l + bias.numpy()
    if mask is not None:
        l = np.where(mask, np.float32(-np.inf), l)
    return l


def check(r, l, ids=None, k=0):
    b, n = l.shape
    x = l.astype(np.float64)
    m = x.max(1, keepdims=True)
    some = np.isfinite(m[:, 0])
    with np.errstate(invalid="ignore", divide="ignore"):
        e = np.where(np.isfinite(x), np.exp(x - np.where(np.isfinite(m), m, 0)), 0.0)
        z = e.sum(1)
        lse = np.where(some, np.where(some, m[:, 0], 0) + np.log(np.where(some, z, 1)), -np.inf)
        ent = np.where(some, -(e * np.where(e > 0, x - lse[:, None], 0)).sum(1) / np.where(some, z, 1), 0.0)
    big = np.abs(np.where(np.isfinite(x), x, 0)).max(1)
    rho = 4 * U * big + (n / 32 + 264) * U
    tol = rho + 2 * U * (np.abs(np.where(some, lse, 0)) + 1)
    got = r.logsumexp.double().cpu().numpy()
    assert np.array_equal(np.isfinite(got), some)
    assert (np.abs(got - lse)[some] <= tol[some]).all(), f"lse off by {np.abs(got - lse)[some].max()}"
    if r.entropy is not None:
        h = r.entropy.double().cpu().numpy()
        assert (np.abs(h - ent) <= 4 * rho * (ent + 41) + 2 * U * ent).all(), f"entropy off by {np.abs(h - ent).max()}"
    if ids is not None:
        i = ids.numpy().astype(np.int64)
        pad = (i < 0) | (i >= n)
        with np.errstate(invalid="ignore"):
            want = np.take_along_axis(x, np.where(pad, 0, i), 1) - lse[:, None]
        want = np.where(pad, 0.0, np.where(np.isnan(want), -np.inf, want))
        lp = r.logprobs.double().cpu().numpy()
        fin = np.isfinite(want)
        assert np.array_equal(lp[~fin], want[~fin])
        assert (np.abs(lp - want) <= 2 * tol[:, None])[fin].all()
    if k:
        key = np.lexsort((np.broadcast_to(np.arange(n), l.shape), -l), axis=1)[:, :k]
        best = np.take_along_axis(l, key, 1)
        want_ids = np.full((b, k), -1)
        want_ids[:, :key.shape[1]] = np.where(np.isfinite(best), key, -1)
        assert np.array_equal(r.alt_ids.cpu().numpy(), want_ids)
        alt = r.alt_logprobs.double().cpu().numpy()
        ok = want_ids >= 0
        assert (alt[~ok] == -np.inf).all()
        with np.errstate(invalid="ignore"):
            ref = np.full((b, k), -np.inf)
            ref[:, :key.shape[1]] = best - lse[:, None]
        assert (np.abs(alt - ref) <= 2 * tol[:, None])[ok].all()


CASES = [
    # dtype, b, n, d, g, k
    ("f32", 1, 1, 16, 1, 1), ("bf16", 1, 1, 16, 1, 64), ("bf16", 1, 31, 8, 2, 5), ("f32", 3, 32, 4, 33, 3),
    ("bf16", 33, 33, 24, 1, 40), ("f32", 1, 400, 16, 1, 10), ("bf16", 64, 401, 32, 3, 20), ("f32", 65, 400, 100, 130, 7),
    ("bf16", 31, 5000, 100, 1, 1), ("bf16", 300, 3001, 128, 8, 20), ("f32", 257, 2500, 128, 1, 64),
    ("bf16", 17, 2049, 256, 4, 20), ("bf16", 130, 4100, 200, 1, 0), ("f32", 40, 6000, 64, 0, 20),
    ("bf16", 5, 70001, 128, 1, 20), ("f32", 2, 140003, 16, 2, 64), ("bf16", 70, 80000, 64, 1, 33),
    ("bf16", 1, 300000, 32, 1, 20), ("bf16", 600, 1024, 16, 1, 5),
]


@pytest.mark.parametrize("dtype,b,n,d,g,k", CASES)
def test_rows(dtype, b, n, d, g, k):
    dev = _dev()
    print(f"logprobs {dtype} b={b} n={n} d={d} g={g} k={k}", flush=True)
    rng = np.random.default_rng(b * 1000 + n)
    items, q = grid(rng, n, d, dtype), grid(rng, b, d, dtype)
    ids = torch.from_numpy(rng.integers(-1, n + 1, (b, g))).to(torch.int64 if n % 2 else torch.int32) if g else None
    r = mips.item_logprobs(q.to(dev), items.to(dev), None if ids is None else ids.to(dev), scale=20.0, alternatives=k)
    check(r, logits64(q, items, 20.0), ids, k)


@pytest.mark.parametrize("dtype,b,n,d", [("f32", 5, 333, 16), ("bf16", 40, 2000, 64), ("bf16", 300, 1000, 128),
                                         ("f32", 70, 70000, 32), ("bf16", 9, 3333, 256)])
@pytest.mark.parametrize("kind", ["bias", "shared", "own", "all", "bias+own"])
def test_bias_and_masks(dtype, b, n, d, kind):
    dev = _dev()
    print(f"logprobs {kind} {dtype} b={b} n={n} d={d}", flush=True)
    rng = np.random.default_rng(n + len(kind))
    items, q = grid(rng, n, d, dtype), grid(rng, b, d, dtype)
    bias = torch.from_numpy(rng.uniform(-8, 8, n).astype(np.float32)) if "bias" in kind else None
    mask = None
    if kind == "shared":
        mask = np.broadcast_to(rng.random(n) < 0.3, (b, n))
    elif "own" in kind:
        mask = rng.random((b, n)) < rng.random((b, 1))
        mask[0] = True        # nothing left
        mask[1] = True
        mask[1, n - 1] = False  # one item left
    elif kind == "all":
        mask = np.ones((b, n), bool)
    words = None if mask is None else bitmap(mask if "own" in kind else mask[0])
    # excluded rows may hold anything
    poisoned = items.clone()
    if kind in ("shared", "all"):
        bad = np.flatnonzero(mask[0])
        poisoned[bad[::3]] = float("nan")
        poisoned[bad[1::3]] = float("inf")
    ids = torch.from_numpy(rng.integers(-1, n + 1, (b, 3))).to(torch.int32)
    r = mips.item_logprobs(q.to(dev), poisoned.to(dev), ids.to(dev), scale=10.0,
                           bias=None if bias is None else bias.to(dev),
                           exclude=None if words is None else words.to(dev), alternatives=17)
    check(r, logits64(q, items, 10.0, bias, mask), ids, 17)


@pytest.mark.parametrize("scale", [1e-6, 0.3, 1000.0])
def test_scales(scale):
    dev = _dev()
    rng = np.random.default_rng(3)
    items, q = grid(rng, 3000, 64, "bf16"), grid(rng, 20, 64, "bf16")
    ids = torch.zeros((20, 1), dtype=torch.int32)
    r = mips.item_logprobs(q.to(dev), items.to(dev), ids.to(dev), scale=scale, alternatives=9)
    check(r, logits64(q, items, scale), ids, 9)


def test_ties_go_to_the_lowest_id():
    dev = _dev()
    rng = np.random.default_rng(4)
    base = grid(rng, 5, 32, "bf16")
    items = base[torch.from_numpy(rng.integers(0, 5, 90000))]
    q = grid(rng, 3, 32, "bf16")
    r = mips.item_logprobs(q.to(dev), items.to(dev), scale=5.0, alternatives=64)
    check(r, logits64(q, items, 5.0), None, 64)


@pytest.mark.parametrize("dtype,d", [("f32", 16), ("f32", 128), ("bf16", 16), ("bf16", 128), ("bf16", 256)])
def test_packed_corpus_equals_its_rows(dtype, d):
    """An index gives what a table of its stored rows gives: bitwise in bf16; in f32 the two
    layouts sum an inner product in another order."""
    from tests.mips_check import untile
    dev = _dev()
    n, b = 5003, 37
    rng = np.random.default_rng(d)
    x = torch.from_numpy(rng.standard_normal((n, d)).astype(np.float32))
    corpus = mips.prepare_corpus(x.to(dev), dtype, model_version="a")
    packed = corpus.packed.cpu().numpy()
    if dtype == "bf16":
        codes = untile(packed, n, d, "bf16")
        stored = torch.from_numpy(np.ascontiguousarray(codes).view(np.int16)).view(torch.bfloat16).reshape(n, d)
    else:
        stored = torch.from_numpy(np.ascontiguousarray(untile(packed, n, d, "f32")).view(np.float32).reshape(n, d).copy())
    q = mips.l2_normalize(torch.from_numpy(rng.standard_normal((b, d)).astype(np.float32)).to(dev), dtype)
    ids = torch.from_numpy(rng.integers(0, n, (b, 2))).to(dev)
    ex = bitmap(rng.random(n) < 0.1).to(dev)
    a = mips.item_logprobs(q, corpus, ids, scale=20.0, exclude=ex, alternatives=10, model_version="a")
    w = mips.item_logprobs(q, stored.to(dev), ids, scale=20.0, exclude=ex, alternatives=10)
    if dtype == "bf16":
        for name in ("logprobs", "logsumexp", "entropy", "alt_ids", "alt_logprobs"):
            assert torch.equal(getattr(a, name), getattr(w, name)), name
    else:
        # unit vectors: |s| error <= d u each way, times the scale; entropy as in the module's bound
        tol = 20.0 * 2 * d * U + (n / 32 + 264) * U * 2 + 40 * U
        fin = torch.isfinite(w.logprobs)
        assert torch.equal(fin, torch.isfinite(a.logprobs))
        assert (a.logprobs - w.logprobs)[fin].abs().max() <= 2 * tol
        assert (a.logsumexp - w.logsumexp).abs().max() <= tol
        assert (a.entropy - w.entropy).abs().max() <= 4 * tol * 60
    with pytest.raises(mips.VersionSkew):
        mips.item_logprobs(q, corpus, ids, model_version="b")


def test_alternatives_whose_runs_fall_to_few_threads():
    """The best items 512 tiles apart, so that the threads that look through the tiles' maxima
    find them all in the same places: more candidates than are ranked at once."""
    dev = _dev()
    for n, d in ((65000, 128), (1_300_000, 16)):
        items = torch.full((n, d), 2.0 ** -8)
        items[:, 0] = 0.0
        k = 64
        where = torch.arange(0, n, 32)
        # rising over tiles t = 0, 512, 1024 .. more than over their neighbours
        items[where, 0] = ((where // 32 % 512 < 2).float() * 0.5).clamp(min=0)
        items[where, 1] = (where // 32 % 251).float() / 256
        q = torch.zeros(2, d)
        q[:, 0] = 1.0
        q[:, 1] = 0.25
        items, q = items.bfloat16(), q.bfloat16()
        r = mips.item_logprobs(q.to(dev), items.to(dev), scale=3.0, alternatives=k)
        check(r, logits64(q, items, 3.0), None, k)


def test_alternatives_are_the_searchs_results():
    dev = _dev()
    rng = np.random.default_rng(8)
    corpus = mips.prepare_corpus(torch.from_numpy(rng.standard_normal((200000, 64)).astype(np.float32)).to(dev), "bf16")
    q = mips.l2_normalize(torch.from_numpy(rng.standard_normal((12, 64)).astype(np.float32)).to(dev), "bf16")
    s, i = mips.topk(q, corpus, 30)
    r = mips.item_logprobs(q, corpus, i, scale=1.0, alternatives=30)
    assert torch.equal(r.alt_ids, i)
    assert torch.equal(r.alt_logprobs, s - r.logsumexp[:, None])
    assert torch.equal(r.logprobs, r.alt_logprobs)


def test_strided_misaligned_and_odd_rows():
    dev = _dev()
    rng = np.random.default_rng(5)
    for dtype in ("f32", "bf16"):
        wide_i, wide_q = grid(rng, 700, 96, dtype), grid(rng, 20, 96, dtype)
        for cut in (slice(0, 64), slice(8, 72), slice(1, 65), slice(3, 40), slice(5, 6)):
            i, q = wide_i[:, cut], wide_q[:, cut]
            r = mips.item_logprobs(wide_q.to(dev)[:, cut], wide_i.to(dev)[:, cut], scale=7.0, alternatives=6)
            check(r, logits64(q, i, 7.0), None, 6)
        r = mips.item_logprobs(wide_q.to(dev).t().contiguous().t(), wide_i.to(dev).t().contiguous().t(), scale=7.0,
                               alternatives=6)
        check(r, logits64(wide_q, wide_i, 7.0), None, 6)
        r = mips.item_logprobs(wide_q.to(dev)[::3], wide_i.to(dev)[1::2], scale=7.0, alternatives=6)
        check(r, logits64(wide_q[::3], wide_i[1::2], 7.0), None, 6)


def test_nan_and_infinite_scores_propagate():
    dev = _dev()
    rng = np.random.default_rng(6)
    items, q = grid(rng, 500, 32, "bf16"), grid(rng, 3, 32, "bf16")
    for bad in (float("nan"), float("inf")):
        q2 = q.clone()
        q2[1, 0] = bad
        r = mips.item_logprobs(q2.to(dev), items.to(dev), torch.zeros((3, 1), dtype=torch.int32, device=dev), scale=4.0)
        assert torch.isnan(r.logsumexp[1]) and torch.isnan(r.entropy[1]) and torch.isnan(r.logprobs[1, 0])
        assert torch.isfinite(r.logsumexp[[0, 2]]).all()


def test_batch_split_by_the_tile_maxima_workspace():
    """So many tiles that the queries are taken in several batches; equal to single calls."""
    dev = _dev()
    n, d, b = 4_200_000, 16, 2100
    rng = np.random.default_rng(7)
    items = grid(rng, 50000, d, "bf16").to(dev).repeat(84, 1)
    q = grid(rng, b, d, "bf16").to(dev)
    print(f"logprobs split n={n} b={b}", flush=True)
    r = mips.item_logprobs(q, items, scale=9.0, alternatives=3)
    for i in (0, 1000, b - 1):
        one = mips.item_logprobs(q[i:i + 1], items, scale=9.0, alternatives=3)
        assert torch.equal(one.alt_ids[0], r.alt_ids[i])
        assert abs(float(one.logsumexp) - float(r.logsumexp[i])) <= (n / 32 + 264) * U * 2 + 40 * U


def test_other_stream_and_graph():
    dev = _dev()
    rng = np.random.default_rng(9)
    items, q = grid(rng, 90000, 64, "bf16").to(dev), grid(rng, 40, 64, "bf16").to(dev)
    ids = torch.from_numpy(rng.integers(0, 90000, (40, 2))).to(dev)
    names = ("logprobs", "logsumexp", "entropy", "alt_ids", "alt_logprobs")
    want = mips.item_logprobs(q, items, ids, scale=20.0, alternatives=8)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = mips.item_logprobs(q, items, ids, scale=20.0, alternatives=8)
    side.synchronize()
    assert all(torch.equal(getattr(want, k), getattr(got, k)) for k in names)
    ws = mips.empty_workspace(mips.lib().mips_logprobs_workspace_size(40, 90000, 64, 1, 8), dev)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        res = mips.item_logprobs(q, items, ids, scale=20.0, alternatives=8, workspace=ws)
    for i in range(3):
        q.copy_(grid(rng, 40, 64, "bf16"))
        graph.replay()
        torch.cuda.synchronize()
        want = mips.item_logprobs(q, items, ids, scale=20.0, alternatives=8)
        assert all(torch.equal(getattr(want, k), getattr(res, k)) for k in names), i


def test_refusals():
    dev = _dev()
    q, items = torch.zeros(3, 32, device=dev), torch.zeros(10, 32, device=dev)
    ids = torch.zeros((3, 1), dtype=torch.int32, device=dev)
    for bad in (dict(ids=ids[:2]), dict(ids=ids[0]), dict(ids=ids.cpu()), dict(bias=torch.zeros(9, device=dev)),
                dict(exclude=torch.zeros(0, dtype=torch.int32, device=dev)),
                dict(exclude=torch.zeros((2, 1), dtype=torch.int32, device=dev))):
        with pytest.raises(ValueError):
            mips.item_logprobs(q, items, **bad)
    with pytest.raises(ValueError):
        mips.item_logprobs(q, items[:, :16])
    for bad in (dict(ids=ids.float()), dict(exclude=torch.zeros(1, device=dev))):
        with pytest.raises(TypeError):
            mips.item_logprobs(q, items, **bad)
    with pytest.raises(TypeError):
        mips.item_logprobs(q, items.bfloat16())
    with pytest.raises(TypeError):
        mips.item_logprobs(q, mips.empty_corpus(100, 32, "int8", dev))
    for bad in (dict(scale=0.0), dict(scale=-1.0), dict(scale=math.inf), dict(scale=math.nan)):
        with pytest.raises(mips.MipsError, match="invalid argument"):
            mips.item_logprobs(q, items, **bad)
    with pytest.raises(mips.MipsError, match="unsupported"):
        mips.item_logprobs(q, items, alternatives=65)
    with pytest.raises(mips.MipsError, match="unsupported"):
        mips.item_logprobs(torch.zeros(3, 129, device=dev), torch.zeros(10, 129, device=dev))
    with pytest.raises(mips.MipsError, match="workspace too small"):
        mips.item_logprobs(q, items, workspace=mips.empty_workspace(256, dev)[:128])
