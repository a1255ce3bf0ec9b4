"""Cases of the training and evaluation operators, with the operators in plain torch.

Four operators meet here, as a two-tower retrieval model uses them:

- ``answer``: log probabilities of given items under a softmax over a whole item table, its
  log-sum-exp and entropy, and the most likely alternatives (evaluation and serving);
- ``train``: the same log probabilities of the training targets, and the gradient of the loss
  for queries and item rows;
- ``gather`` / ``scatter``: embedding lookup with scaling, and its gradient by sorted tokens;
- ``clip``: the global gradient norm over a model's tensors, and clipping by it.

With ``own`` false, ``run`` is elementary torch in 32 bits; with ``own`` true it is the calls a
user makes of ``exact_inner_product_amd``.

Where ids are compared, vectors lie on a grid of 2^-8 (bf16) or 2^-10 (f32): an inner product
of such vectors is exact in binary32 in any order of summation, so that the order of the
alternatives, ties by the lowest id, is the same for every correct program.
"""
import math

import numpy as np
import torch

own = False

_DT = {"bf16": torch.bfloat16, "f32": torch.float32}
_SIZE = {"bf16": 2, "f32": 4}


def listed():
    return [
        # One user against the toy catalogue (400 items, width 16): what a call costs when it
        # has nothing to do; latency alone.
        dict(name="answer_toy", op="answer", dtype="f32", b=1, n=400, d=16, g=1, k=10, drop=0, tau=0.1),
        # A serving batch of 16 users over a million items: bound by reading the table.
        dict(name="answer_1m", op="answer", dtype="bf16", b=16, n=1000000, d=128, g=1, k=20, drop=0, tau=0.05),
        # The headline index, 50 users over 10M items with 5% of them excluded: eight given
        # items a user (the impressions to be scored) and the 20 best alternatives.
        dict(name="answer_10m", op="answer", dtype="bf16", b=50, n=10000000, d=128, g=8, k=20, drop=5, tau=0.05),
        # In-batch negatives with the logQ correction: 1000 pairs in f32, every item the
        # positive of one query.
        dict(name="train_inbatch_f32", op="train", dtype="f32", b=1000, n=1000, d=64, bias=True, tau=0.1),
        # In-batch negatives and as many mixed negatives in bf16, with logQ.
        dict(name="train_mixed_bf16", op="train", dtype="bf16", b=4096, n=8192, d=128, bias=True, tau=0.05),
        # Full softmax over a quarter of a million items, the largest training step here.
        dict(name="train_full_bf16", op="train", dtype="bf16", b=4096, n=250000, d=128, bias=False, tau=0.05),
        # One user's history of 50 items from a million-row table.
        dict(name="gather_user", op="gather", dtype="f32", v=1000000, d=64, t=50),
        # A training batch's histories (4096 users, 127 items each) from a million-row table.
        dict(name="gather_batch", op="gather", dtype="bf16", v=1000000, d=128, t=4096 * 127),
        # The gradient of a small table (65,536 rows) for an odd number of Zipf tokens.
        dict(name="scatter_small", op="scatter", dtype="f32", v=65536, d=64, t=8191),
        # The gradient of a million-row table for a batch's histories: hot ids hold thousands
        # of tokens, most ids none.
        dict(name="scatter_batch", op="scatter", dtype="bf16", v=1000000, d=128, t=4096 * 127),
        # A pair of towers: 48 small tensors, where launches and latency count.
        dict(name="clip_towers", op="clip", dtype="bf16", tensors=48, most=1 << 18, table=0),
        # Towers and their tables: 1.2 GB of gradients in f32.
        dict(name="clip_tables", op="clip", dtype="f32", tensors=24, most=1 << 20, table=2000000 * 128),
    ]


def _log_uniform(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


# Scores of one call, and scores of its first 256 queries: in the plain form's binary32
# product, rows of the result further than 2 GiB from a tile's first one came out wrong.
_SCORES, _TILE = 1050000000, 530000000


def draw(rng):
    op = rng.choice(("answer", "answer", "train", "train", "gather", "scatter", "scatter", "clip"))
    dtype = rng.choice(("bf16", "f32"))
    if op == "answer":
        d = rng.choice((16, 32, 64, 128, 128, 256) if dtype == "bf16" else (16, 32, 64, 128))
        b = _log_uniform(rng, 1, 1024)
        n = _log_uniform(rng, 400, min(10000000, _SCORES // b, _TILE // min(b, 256), 1280000000 // d // (1 if dtype == "bf16" else 4)))
        return dict(op=op, dtype=dtype, b=b, n=n, d=d, g=rng.choice((1, 1, 4, 8)), k=rng.choice((0, 1, 5, 10, 20)),
                    drop=rng.choice((0, 0, 5)), tau=rng.choice((0.05, 0.1, 0.2)))
    if op == "train":
        d = rng.choice((16, 32, 64, 128, 128, 256) if dtype == "bf16" else (16, 32, 64, 128))
        b = _log_uniform(rng, 64, 4096)
        cost = 4096 * 250000 * 128 // (1 if dtype == "bf16" else 8)
        n = _log_uniform(rng, b, max(b, min(1000000, _SCORES // b, cost // b // d)))
        return dict(op=op, dtype=dtype, b=b, n=n, d=d, bias=rng.random() < 0.5, tau=rng.choice((0.05, 0.1, 0.2)))
    if op in ("gather", "scatter"):
        d = rng.choice((16, 32, 64, 100, 128, 256, 512))
        v = _log_uniform(rng, 1000, 128000000 // d)
        return dict(op=op, dtype=dtype, v=v, d=d, t=_log_uniform(rng, 1 if op == "gather" else 64, 67000000 // d))
    return dict(op=op, dtype=dtype, tensors=rng.randint(1, 60), most=_log_uniform(rng, 64, 1 << 21),
                table=rng.choice((0, 0, _log_uniform(rng, 1000000, 200000000))))


def _shapes(case):
    """Element counts of a clip case's tensors: spread evenly over the logarithm, odd ones among them."""
    c = case["tensors"]
    sizes = [max(1, int(case["most"] ** ((i + 1) / c)) + i % 2) for i in range(c)]
    return sizes + ([case["table"]] if case["table"] else [])


def _vectors(gen, n, d, dtype):
    """Unit vectors on a grid: an index or a batch as a quantised store keeps it."""
    step = 256.0 if dtype == "bf16" else 1024.0
    x = torch.randn(n, d, generator=gen, device="cuda")
    x = x / x.square().sum(1, keepdim=True).sqrt()
    return (torch.round(x * step) / step).to(_DT[dtype])


def _zipf(gen, v, t):
    """t ids below v, rank r about as often as 1/r, spread over the table."""
    u = torch.rand(t, generator=gen, device="cuda", dtype=torch.float64)
    r = (torch.exp(u * math.log(v + 1.0)).long() - 1).clamp_(0, v - 1)
    return (r * 2654435761 % v).to(torch.int32)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    op, dtype = case["op"], case["dtype"]
    s = dict(case=case)
    if op in ("answer", "train"):
        b, n, d = case["b"], case["n"], case["d"]
        s["scale"] = 1.0 / case["tau"]
        s["items"] = _vectors(gen, n, d, dtype)
        if op == "train":
            # in a batch every query's target is a row of its own; the rest are negatives
            s["ids"] = torch.randperm(n, generator=gen, device="cuda")[:b].to(torch.int32)[:, None].contiguous()
        else:
            s["ids"] = torch.randint(0, n, (b, case["g"]), generator=gen, device="cuda", dtype=torch.int32)
        # a trained query points at its target, with noise
        step = 256.0 if dtype == "bf16" else 1024.0
        q = s["items"][s["ids"][:, 0].long()].float() + 1.5 / math.sqrt(d) * torch.randn(b, d, generator=gen, device="cuda")
        q = q / q.square().sum(1, keepdim=True).sqrt()
        s["queries"] = (torch.round(q * step) / step).to(_DT[dtype])
        s["exclude"] = s["bias"] = None
        if case.get("drop"):
            bits = (torch.rand((n + 31) // 32, 32, generator=gen, device="cuda") < case["drop"] / 100.0).long()
            words = (bits << torch.arange(32, device="cuda")).sum(1)
            s["exclude"] = torch.where(words >= 2 ** 31, words - 2 ** 32, words).to(torch.int32)
        if case.get("bias"):
            # - log q of items drawn by popularity
            s["bias"] = torch.empty(n, device="cuda").uniform_(0.0, 8.0, generator=gen)
        if op == "train":
            s["grad"] = torch.empty(b, 1, device="cuda").uniform_(-1.5, -0.5, generator=gen)
    elif op == "gather":
        s["table"] = torch.randn(case["v"], case["d"], generator=gen, device="cuda").to(_DT[dtype])
        s["ids"] = _zipf(gen, case["v"], case["t"])
        s["scale"] = math.sqrt(case["d"])
    elif op == "scatter":
        s["grad"] = torch.randn(case["t"], case["d"], generator=gen, device="cuda").to(_DT[dtype])
        s["ids"] = _zipf(gen, case["v"], case["t"])
        s["scale"] = math.sqrt(case["d"])
    else:
        s["grads"] = [torch.randn(m, generator=gen, device="cuda").to(_DT[dtype]) for m in _shapes(case)]
        s["out"] = [torch.empty_like(g) for g in s["grads"]]
        s["max_norm"] = 1.0
    return s


# ------------------------------------------------------------------- plain forms
def _excluded(words, n):
    bits = (words[:, None].long() >> torch.arange(32, device=words.device)) & 1
    return bits.reshape(-1)[:n] == 1


def _logits(s):
    x = (s["queries"].float() @ s["items"].float().T) * s["scale"]
    if s["bias"] is not None:
        x = x + s["bias"]
    if s["exclude"] is not None:
        x = x.masked_fill(_excluded(s["exclude"], x.shape[1]), -math.inf)
    return x


def _softmax_stats(x):
    """(log sum exp, entropy) of each row."""
    m = x.max(1, keepdim=True).values
    e = torch.exp(x - m)
    z = e.sum(1)
    ex = (e * x.clamp(min=-3e38)).sum(1)
    lse = m[:, 0] + torch.log(z)
    return lse, lse - ex / z


def _best(x, k):
    """The k largest of each row, ties by the lowest index: (indices, values)."""
    bits = (x + 0.0).view(torch.int32).long()
    key = torch.where(bits < 0, -(bits & 0x7FFFFFFF), bits) * 2 ** 32 - torch.arange(x.shape[1], device=x.device)
    ids = torch.topk(key, k, dim=1).indices
    return ids.to(torch.int32), x.gather(1, ids)


def _plain_answer(s):
    x = _logits(s)
    lse, entropy = _softmax_stats(x)
    out = dict(logprobs=x.gather(1, s["ids"].long()) - lse[:, None], logsumexp=lse, entropy=entropy)
    if s["case"]["k"]:
        ids, best = _best(x, s["case"]["k"])
        out.update(alt_ids=ids, alt_logprobs=best - lse[:, None])
    return out


def _plain_train(s):
    x = _logits(s)
    lse, _ = _softmax_stats(x)
    ids = s["ids"].long()
    logprobs = x.gather(1, ids) - lse[:, None]
    # d logp / d x_j = [j is the target] - p_j
    w = torch.exp(x.sub_(lse[:, None])).mul_(-s["grad"])
    w.scatter_add_(1, ids, s["grad"])
    w.mul_(s["scale"])
    q, c = s["queries"], s["items"]
    return dict(logprobs=logprobs, grad_queries=(w @ c.float()).to(q.dtype), grad_items=(w.T @ q.float()).to(c.dtype))


def _plain_gather(s):
    return (s["table"][s["ids"].long()].float() * s["scale"]).to(s["table"].dtype)


def _plain_scatter(s):
    out = torch.zeros(s["case"]["v"], s["case"]["d"], device="cuda")
    out.index_add_(0, s["ids"].long(), s["grad"].float())
    return (out * s["scale"]).to(s["grad"].dtype)


def _plain_clip(s):
    norm = torch.stack([g.float().square().sum() for g in s["grads"]]).sum().sqrt()
    coef = (s["max_norm"] / (norm + 1e-6)).clamp(max=1.0)
    return dict(norm=norm, grads=[(g.float() * coef).to(g.dtype) for g in s["grads"]])


_PLAIN = dict(answer=_plain_answer, train=_plain_train, gather=_plain_gather, scatter=_plain_scatter, clip=_plain_clip)


# ------------------------------------------------------------- the framework's calls
def _own_answer(mips, s):
    r = mips.item_logprobs(s["queries"], s["items"], s["ids"], scale=s["scale"], exclude=s["exclude"],
                           alternatives=s["case"]["k"])
    out = dict(logprobs=r.logprobs, logsumexp=r.logsumexp, entropy=r.entropy)
    if s["case"]["k"]:
        out.update(alt_ids=r.alt_ids, alt_logprobs=r.alt_logprobs)
    return out


def _own_train(mips, s):
    kw = dict(scale=s["scale"], bias=s["bias"])
    r = mips.item_logprobs(s["queries"], s["items"], s["ids"], entropy=False, **kw)
    dq, dc, _ = mips.item_logprobs_backward(s["grad"], s["queries"], s["items"], s["ids"], r, **kw)
    return dict(logprobs=r.logprobs, grad_queries=dq, grad_items=dc)


def _own_gather(mips, s):
    return mips.embedding_lookup(s["table"], s["ids"], scale=s["scale"])


def _own_scatter(mips, s):
    return mips.embedding_grad(s["grad"], s["ids"], s["case"]["v"], scale=s["scale"])


def _own_clip(mips, s):
    norm, out = mips.clip_grad_norm(s["grads"], s["max_norm"], out=s["out"])
    return dict(norm=norm, grads=out)


_OWN = dict(answer=_own_answer, train=_own_train, gather=_own_gather, scatter=_own_scatter, clip=_own_clip)


def run(state):
    op = state["case"]["op"]
    if own:
        import exact_inner_product_amd as mips
        return _OWN[op](mips, state)
    return _PLAIN[op](state)


def work(case):
    op, e = case["op"], _SIZE[case["dtype"]]
    if op in ("answer", "train"):
        b, n, d = case["b"], case["n"], case["d"]
        if op == "answer":
            out = b * (4 * case["g"] + 8 + 8 * case["k"]) + (n // 8 if case["drop"] else 0) + 4 * b * case["g"]
            return dict(bytes=(n + b) * d * e + out, flops=2 * b * n * d)
        return dict(bytes=2 * (n + b) * d * e + (4 * n if case["bias"] else 0) + 12 * b, flops=6 * b * n * d)
    if op == "gather":
        rows = min(case["v"], case["t"])  # at most so many distinct rows are read
        return dict(bytes=(rows + case["t"]) * case["d"] * e + 4 * case["t"], flops=case["t"] * case["d"])
    if op == "scatter":
        return dict(bytes=(case["v"] + case["t"]) * case["d"] * e + 4 * case["t"], flops=case["t"] * case["d"])
    m = sum(_shapes(case))
    return dict(bytes=2 * m * e, flops=3 * m)


# -------------------------------------------------- the definitions, in 64 bits
def _exact_rows(s, rows):
    """Logits of some queries as 64-bit floats."""
    q = s["queries"][rows].double()
    x = torch.mm(q, s["items"].double().t()).mul_(float(s["scale"]))
    if s["bias"] is not None:
        x.add_(s["bias"].double())
    if s["exclude"] is not None:
        ids = torch.arange(x.shape[1], device=x.device)
        word = s["exclude"][ids // 32].long()
        x[:, torch.bitwise_right_shift(word, ids % 32).bitwise_and(1).bool()] = -float("inf")
    return x


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("answer", "train"):
        b, n = case["b"], case["n"]
        step = max(1, min(b, 400000000 // n))
        parts, dc = [], torch.zeros(n, case["d"], dtype=torch.float64, device="cuda") if op == "train" else None
        for r0 in range(0, b, step):
            rows = slice(r0, min(b, r0 + step))
            x = _exact_rows(s, rows)
            lse = torch.logsumexp(x, 1)
            ids = s["ids"][rows].long()
            lp = torch.gather(x, 1, ids) - lse[:, None]
            if op == "answer":
                p = torch.exp(x - lse[:, None])
                ent = -(p * torch.where(p > 0, x - lse[:, None], torch.zeros_like(x))).sum(1)
                top = torch.topk(x, case["k"], dim=1).values - lse[:, None] if case["k"] else None
                parts.append((lp, lse, ent, top))
            else:
                g = s["grad"][rows].double()
                w = torch.exp(x - lse[:, None]) * (-g)
                at = torch.arange(w.shape[0], device="cuda")
                w[at, ids[:, 0]] += g[:, 0]
                w = w * float(s["scale"])
                parts.append((lp, torch.mm(w, s["items"].double())))
                dc += torch.mm(w.t(), s["queries"][rows].double())
        if op == "train":
            return dict(logprobs=torch.cat([p[0] for p in parts]), grad_queries=torch.cat([p[1] for p in parts]), grad_items=dc)
        out = dict(logprobs=torch.cat([p[0] for p in parts]), logsumexp=torch.cat([p[1] for p in parts]),
                   entropy=torch.cat([p[2] for p in parts]))
        if case["k"]:
            out.update(alt_ids=None, alt_logprobs=torch.cat([p[3] for p in parts]))
        return out
    if op == "gather":
        return torch.index_select(s["table"], 0, s["ids"].long()).double() * s["scale"]
    if op == "scatter":
        order = torch.argsort(s["ids"].long(), stable=True)
        out = torch.zeros(case["v"], case["d"], dtype=torch.float64, device="cuda")
        out.index_add_(0, s["ids"].long()[order], s["grad"].double()[order])
        return out * s["scale"]
    total = float(np.sqrt(sum(float((g.double() ** 2).sum()) for g in s["grads"])))
    coef = min(1.0, s["max_norm"] / (total + 1e-6))
    return dict(norm=torch.tensor(total, dtype=torch.float64), grads=[g.double() * coef for g in s["grads"]])
