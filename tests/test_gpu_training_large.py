"""Tables and batches whose element offsets pass 32 bits: lookups, their gradients and the softmax
over more than 2^31 numbers. Values are chosen so that the answers are known in closed form;
everything large stays on the GPU."""
import numpy as np
import pytest
import torch

import exact_inner_product_amd as mips

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


def _dev():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GiB of GPU memory")
    return torch.device("cuda:0")


@pytest.mark.parametrize("t", [300, 20000])
def test_lookup_and_gradient_of_a_table_past_32_bit_offsets(t):
    """Gradients are whole numbers, exact in any order: the few rows with tokens are compared,
    and that no other row holds anything."""
    dev = _dev()
    rows, d = (1 << 24) + 40, 136
    print(f"large table: {rows} x {d}, {t} tokens", flush=True)
    rng = np.random.default_rng(t)
    edge = (1 << 31) // d
    ids = rng.integers(0, rows, t)
    ids[:8] = [0, edge - 1, edge, edge + 1, 1 << 24, rows - 1, rows - 1, rows]
    ids = torch.from_numpy(ids).to(dev)
    ok = ids < rows
    grad = torch.from_numpy(rng.integers(-4, 5, (t, d)).astype(np.float32)).to(dev).bfloat16()
    table = torch.full((rows, d), 7.0, dtype=torch.bfloat16, device=dev)
    mips.embedding_grad(grad, ids, rows, out=table)
    used, inv = torch.unique(ids[ok], return_inverse=True)
    want = torch.zeros(len(used), d, device=dev).index_add_(0, inv, grad[ok].float())
    assert torch.equal(table[used].float(), want)
    full = sum(int(torch.count_nonzero(part)) for part in table.split(1 << 20))
    assert full == int(torch.count_nonzero(want))
    got = mips.embedding_lookup(table, ids, scale=2.0)
    assert torch.equal(got[ok].float(), 2 * want[inv]) and not got[~ok].any()


def test_lookup_and_gradient_of_tokens_past_32_bit_offsets():
    """Every token's gradient is its own row, a small whole number: a row's sum is its count
    times the row, exact in binary32."""
    dev = _dev()
    t, rows, d = (1 << 24) + 40, 1000, 136
    print(f"large batch: {t} tokens of {rows} x {d}", flush=True)
    gen = torch.Generator(device=dev).manual_seed(1)
    table = torch.randint(-3, 4, (rows, d), generator=gen, device=dev).bfloat16()
    ids = torch.randint(0, rows, (t,), generator=gen, device=dev)
    out = mips.embedding_lookup(table, ids)
    for part, i in zip(out.split(1 << 20), ids.split(1 << 20)):
        assert torch.equal(part, table[i])
    got = mips.embedding_grad(out, ids, rows, out=torch.empty(rows, d, device=dev))
    assert torch.equal(got, torch.bincount(ids, minlength=rows)[:, None] * table.float())


def test_log_probabilities_and_gradient_past_32_bit_offsets():
    """All rows are zero but a few, whose logits are known: the log-sum-exp, the alternatives
    (zeros tie, lowest ids first) and the gradients follow in closed form. Tolerances are those of the
    smaller tests: tests/test_gpu_logprobs.py, tests/test_gpu_logprobs_grad.py."""
    dev = _dev()
    n, d, b, k, scale = (1 << 24) + 1000, 128, 3, 8, 8.0
    print(f"large softmax: {n} x {d}", flush=True)
    rng = np.random.default_rng(3)
    special = np.array([5, 1 << 20, (1 << 24) - 1, 1 << 24, n - 1])
    rows = torch.from_numpy(np.round(rng.standard_normal((5, d)) * 16) / 64).bfloat16()
    q = torch.from_numpy(np.round(rng.standard_normal((b, d)) * 16) / 64).bfloat16()
    items = torch.zeros(n, d, dtype=torch.bfloat16, device=dev)
    items[torch.from_numpy(special).to(dev)] = rows.to(dev)
    l = scale * (q.double().numpy() @ rows.double().numpy().T)          # exact in binary32
    lse = np.log(n - 5 + np.exp(l).sum(1))
    ids = torch.tensor([[5, n - 1], [1 << 24, 77], [n - 2, (1 << 24) - 1]])
    r = mips.item_logprobs(q.to(dev), items, ids.to(dev), scale=scale, alternatives=k)
    big = np.abs(l).max()
    rho = 4 * U * big + (n / 32 + 264) * U
    tol = rho + 2 * U * (lse + 1)
    assert (np.abs(r.logsumexp.double().cpu().numpy() - lse) <= tol).all()
    logit = np.zeros((b, 2))
    for x in range(b):
        for c in range(2):
            at = np.flatnonzero(special == int(ids[x, c]))
            logit[x, c] = l[x, at[0]] if len(at) else 0.0
    assert (np.abs(r.logprobs.double().cpu().numpy() - (logit - lse[:, None])) <= 2 * tol[:, None]).all()
    for x in range(b):
        up = special[l[x] > 0][np.argsort(-l[x][l[x] > 0], kind="stable")]
        zeros = [i for i in range(2 * k) if i not in special][:k]
        assert r.alt_ids[x].tolist() == [*up, *zeros][:k]

    g = torch.from_numpy(rng.standard_normal((b, 2)).astype(np.float32))
    dq, dc, _ = mips.item_logprobs_backward(g.to(dev), q.to(dev), items, ids.to(dev), r, scale=scale)
    # the weights of the rows that are looked at: the special ones, the targets and one more
    look = np.array([*special, 77, n - 2, 123456])
    ll = np.concatenate([l, np.zeros((b, 3))], 1)
    p = np.exp(ll - lse[:, None])
    hot, ahot = np.zeros_like(p), np.zeros_like(p)
    for x in range(b):
        for c in range(2):
            hot[x, look == int(ids[x, c])] += float(g[x, c])
            ahot[x, look == int(ids[x, c])] += abs(float(g[x, c]))
    G = g.double().numpy().sum(1, keepdims=True)
    w, a = hot - p * G, ahot + p * np.abs(hot.sum(1, keepdims=True))
    a = np.maximum(a, np.abs(w))
    qd, cd = q.double().numpy(), rows.double().numpy()
    rr = 2 * rho + 8 * U
    for got, want, mag, m in ((dc[torch.from_numpy(look).to(dev)], scale * w.T @ qd, scale * a.T @ np.abs(qd), b),
                              (dq, scale * w[:, :5] @ cd, scale * a[:, :5] @ np.abs(cd), n)):
        e = (3 * rr + (m + 70) * U + 2.0 ** -8) * mag
        lo, hi = (torch.from_numpy(want + s * e).bfloat16().double().numpy() for s in (-1, 1))
        y = got.double().cpu().numpy()
        assert ((lo <= y) & (y <= hi)).all(), np.abs(y - want).max()
    # every other row has the same weights, and so the same bits
    same = sum(int((part == dc[123456]).all(1).sum()) for part in dc.split(1 << 20))
    assert same == n - 7
