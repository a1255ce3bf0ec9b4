"""Cases of the user tower's operators over histories of events, with the operators in plain torch.

Four operators meet here, as a user tower that reads a history uses them:

- ``encode`` / ``train``: a gated linear recurrence over sequences, h_t = a_t h_{t-1} + b_t x_t with
  a = sigmoid(forget logits) and b = 1 - a or sigmoid(input logits); its states and the last ones,
  and their gradient;
- ``step``: the same recurrence for single events, against a table with the state of every user;
- ``dropout``: dropout from a counter-based generator (Philox4x32-10: Salmon, Moraes, Dror and
  Shaw, "Parallel random numbers: as easy as 1, 2, 3", 2011), with an optional residual, and its gradient;
- ``pool``: the mean of a history's rows, L2-normalised, and its gradient.

Sequences are dense ([b, t, d]), padded (dense, with a length each) or packed ([n, d], with b + 1
offsets). With ``own`` false, ``run`` is elementary torch in 32 bits; with ``own`` true it is the calls
a user makes of ``exact_inner_product_amd``.
"""
import math

import numpy as np
import torch

own = False

_DT = {"bf16": torch.bfloat16, "f32": torch.float32}
_SIZE = {"bf16": 2, "f32": 4}


def listed():
    return [
        # One user's history of 50 events: what a call costs when it has next to nothing to do.
        dict(name="encode_user", op="encode", dtype="f32", layout="dense", b=1, t=50, d=64, gate=False, initial=False, states=True),
        # A log of 65,536 events encoded in one go from a given state: few channels, one long axis.
        dict(name="encode_long", op="encode", dtype="bf16", layout="dense", b=1, t=65536, d=256, gate=False, initial=True, states=True),
        # A training batch's histories, 4096 users with 127 events each; every state is used.
        dict(name="train_batch", op="train", dtype="bf16", layout="dense", b=4096, t=127, d=128, gate=False, initial=False, states=True),
        # The same batch with histories of 0 to 127 events, of which the last state is the user's vector.
        dict(name="train_last", op="train", dtype="bf16", layout="padded", b=4096, t=127, d=128, gate=False, initial=False, states=False),
        # Packed histories of 0 to 600 events in f32, an odd width, a gate of its own for the input.
        dict(name="train_packed", op="train", dtype="f32", layout="packed", b=2000, t=600, d=100, gate=True, initial=True, states=True),
        # Long sequences at the width of the embedding table, the largest training step here.
        dict(name="train_long", op="train", dtype="bf16", layout="dense", b=4, t=16384, d=1024, gate=False, initial=False, states=True),
        # Sixteen users' new events, as a server applies them: latency alone.
        dict(name="step_few", op="step", dtype="f32", b=16, v=100000, d=64, gate=False),
        # A micro-batch of 4096 events against a million users, one in ten of a user met before.
        dict(name="step_batch", op="step", dtype="bf16", b=4096, v=1000000, d=128, gate=True),
        # Dropout of a small batch of user vectors.
        dict(name="dropout_small", op="dropout", dtype="f32", n=1000, d=64, p=0.1, residual=False),
        # Dropout of a training batch's histories, added to the branch beside it.
        dict(name="dropout_batch", op="dropout", dtype="bf16", n=4096 * 127, d=128, p=0.1, residual=True),
        # Sixteen users' histories as vectors to search with.
        dict(name="pool_few", op="pool", dtype="f32", layout="padded", b=16, t=50, d=64, train=False),
        # A training batch's histories pooled, with the gradient.
        dict(name="pool_batch", op="pool", dtype="bf16", layout="padded", b=4096, t=127, d=128, train=True),
    ]


def _log_uniform(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("encode", "train", "train", "step", "dropout", "pool"))
    dtype = rng.choice(("bf16", "f32"))
    d = rng.choice((16, 32, 64, 100, 128, 128, 256, 512, 1024))
    if op == "step":
        return dict(op=op, dtype=dtype, b=_log_uniform(rng, 1, 16384), v=_log_uniform(rng, 1000, 128000000 // d), d=d,
                    gate=rng.random() < 0.5)
    # a quarter of the largest case's elements in f32, where a gate of its own doubles the work
    most = 67108864 // (1 if dtype == "bf16" else 4) // d
    if op == "dropout":
        return dict(op=op, dtype=dtype, n=_log_uniform(rng, 1, most), d=d, p=rng.choice((0.05, 0.1, 0.2, 0.5)),
                    residual=rng.random() < 0.5)
    b = _log_uniform(rng, 1, 4096)
    t = _log_uniform(rng, 1, min(32768, most // b))
    layout = rng.choice(("dense", "padded", "packed"))
    if op == "pool":
        return dict(op=op, dtype=dtype, layout=layout, b=b, t=t, d=d, train=rng.random() < 0.5)
    return dict(op=op, dtype=dtype, layout=layout, b=b, t=t, d=d, gate=rng.random() < 0.5, initial=rng.random() < 0.5,
                states=rng.random() < 0.7)


def _lengths(case):
    """The length of each sequence: 0 to t, spread evenly, in an order that looks random."""
    if case["layout"] == "dense":
        return np.full(case["b"], case["t"], dtype=np.int64)
    u = np.arange(1, case["b"] + 1, dtype=np.uint64) * np.uint64(2654435761) % np.uint64(1 << 32)
    return (u * np.uint64(case["t"] + 1) >> np.uint64(32)).astype(np.int64)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    op, dt, d = case["op"], _DT[case["dtype"]], case["d"]

    def normal(*shape, scale=1.0, mean=0.0, dtype=dt):
        return (torch.randn(*shape, generator=gen, device="cuda") * scale + mean).to(dtype)

    s = dict(case=case)
    if op == "dropout":
        s.update(x=normal(case["n"], d), grad=normal(case["n"], d), residual=normal(case["n"], d) if case["residual"] else None,
                 seed=int(torch.randint(0, 1 << 62, (1,), generator=gen, device="cuda")), offset=seed % 1000)
        return s
    if op == "step":
        b, v = case["b"], case["v"]
        rows = torch.randint(0, v, (b,), generator=gen, device="cuda")
        earlier = (torch.rand(b, generator=gen, device="cuda") * torch.arange(b, device="cuda")).long()
        rows = torch.where(torch.rand(b, generator=gen, device="cuda") < 0.1, rows[earlier], rows)
        state = normal(v, d, dtype=torch.float32)
        s.update(x=normal(b, d), forget=normal(b, d, mean=2.0), gate=normal(b, d) if case["gate"] else None,
                 rows=rows.to(torch.int32), state=state, out=state.clone())
        return s
    b, t = case["b"], case["t"]
    lengths = _lengths(case)
    packed = case["layout"] == "packed"
    shape = (int(lengths.sum()), d) if packed else (b, t, d)
    s["x"] = normal(*shape)
    s["lengths"] = torch.from_numpy(lengths.astype(np.int32)).cuda() if case["layout"] == "padded" else None
    s["offsets"] = torch.from_numpy(np.concatenate([[0], np.cumsum(lengths)]).astype(np.int32)).cuda() if packed else None
    if op == "pool":
        s["grad"] = normal(b, d) if case["train"] else None
        return s
    # gates that remember some ten events in the mean, some channels and events a hundred
    s["forget"] = normal(*shape, scale=1.5, mean=2.0)
    s["gate"] = normal(*shape) if case["gate"] else None
    s["initial"] = normal(b, d, dtype=torch.float32) if case["initial"] else None
    if op == "train":
        s["grad_states"] = normal(*shape) if case["states"] else None
        s["grad_last"] = normal(b, d, dtype=torch.float32)
    return s


# ------------------------------------------------------------------- plain forms
def _rows(s):
    """(sequence of each row, first row of its sequence, last one, row of no sequence) over the rows
    of x laid out flat."""
    x = s["x"]
    at = torch.arange(x.numel() // x.shape[-1], device=x.device)
    if s["offsets"] is not None:
        off = s["offsets"].long()
        seq = torch.searchsorted(off, at, right=True) - 1
        return seq, at == off[seq], at == off[seq + 1] - 1, torch.zeros_like(at, dtype=torch.bool)
    t = x.shape[1]
    seq, pos = at // t, at % t
    end = torch.full_like(seq, t) if s["lengths"] is None else s["lengths"].long()[seq]
    return seq, pos == 0, pos == end - 1, pos >= end


def _recur(a, b, steps):
    """y_r = a_r y_{r-1} + b_r over the rows, by doubling: after k rounds each row holds its last 2^k."""
    k = 1
    while k < steps:
        b = torch.cat([b[:k], torch.addcmul(b[k:], a[k:], b[:-k])])
        a = torch.cat([a[:k], a[k:] * a[:-k]])
        k *= 2
    return b


def _gates(s, d):
    f = s["forget"].reshape(-1, d).float()
    return torch.sigmoid(f), torch.sigmoid(-f if s["gate"] is None else s["gate"].reshape(-1, d).float())


def _plain_scan(s):
    case, x = s["case"], s["x"]
    d, nseq = case["d"], case["b"]
    seq, first, last, pad = _rows(s)
    init = s["initial"] if s["initial"] is not None else torch.zeros(nseq, d, device=x.device)
    xf = x.reshape(-1, d).float()
    a, b = _gates(s, d)
    a, b = a.masked_fill(pad[:, None], 0.0), b.masked_fill(pad[:, None], 0.0)
    before = init[seq].masked_fill(~first[:, None], 0.0)       # what a first row finds
    inner = a.masked_fill(first[:, None], 0.0)
    h = _recur(inner, torch.addcmul(b * xf, a, before), case["t"])
    ends = torch.where(last)[0]
    end = init.index_copy(0, seq[ends], h[ends])
    out = dict(last=end)
    if case["states"]:
        out["states"] = h.reshape(x.shape).to(x.dtype)
    if case["op"] == "encode":
        return out
    # D_r = g_r + a_{r+1} D_{r+1}, by the same recurrence over the rows from the last to the first
    g = torch.zeros_like(xf) if s["grad_states"] is None else s["grad_states"].reshape(-1, d).float()
    g = (g + s["grad_last"][seq].masked_fill(~last[:, None], 0.0)).masked_fill(pad[:, None], 0.0)
    after = torch.cat([inner[1:], torch.zeros_like(inner[:1])]).masked_fill(last[:, None], 0.0)
    grad = _recur(after.flip(0), g.flip(0), case["t"]).flip(0)
    prev = torch.cat([torch.zeros_like(h[:1]), h[:-1]]).masked_fill(first[:, None], 0.0) + before
    out["grad_x"] = (grad * b).reshape(x.shape).to(x.dtype)
    if s["gate"] is None:
        df = grad * (prev - xf) * a * b
    else:
        df = grad * prev * a * torch.sigmoid(-s["forget"].reshape(-1, d).float())
        out["grad_gate"] = (grad * xf * b * torch.sigmoid(-s["gate"].reshape(-1, d).float())).reshape(x.shape).to(x.dtype)
    out["grad_forget"] = df.reshape(x.shape).to(x.dtype)
    if s["initial"] is not None:
        starts = torch.where(first & ~pad)[0]
        out["grad_initial"] = s["grad_last"].index_copy(0, seq[starts], (a * grad)[starts])
    return out


def _plain_step(s):
    b, d = s["case"]["b"], s["case"]["d"]
    order = torch.argsort(s["rows"], stable=True)              # a row's events together, in their order
    rows = s["rows"].long()[order]
    first = torch.cat([torch.ones_like(rows[:1]), rows[1:] - rows[:-1]]) != 0
    final = torch.cat([rows[1:] - rows[:-1], torch.ones_like(rows[:1])]) != 0
    a, g = _gates(s, d)
    a, g = a[order], g[order]
    before = s["state"][rows].masked_fill(~first[:, None], 0.0)
    h = _recur(a.masked_fill(first[:, None], 0.0), torch.addcmul(g * s["x"].float()[order], a, before), b)
    ends = torch.where(final)[0]
    s["out"].index_copy_(0, rows[ends], h[ends])
    return dict(states=torch.empty_like(s["x"]).index_copy_(0, order, h.to(s["x"].dtype)), table=s["out"])


def _kept(case, seed, offset, device):
    """Which elements dropout keeps: 16 bits each of Philox4x32-10 of (element // 8, offset) under the seed."""
    m = case["n"] * case["d"]
    low = 0xFFFFFFFF
    i = torch.arange((m + 7) // 8, device=device)
    c0, c1, c2, c3 = i & low, i >> 32, torch.full_like(i, offset & low), torch.full_like(i, offset >> 32)
    k0, k1 = seed & low, seed >> 32
    for _ in range(10):
        p, q = c0 * 0xD2511F53, c2 * 0xCD9E8D57
        c0, c1, c2, c3 = ((q >> 32) & low) ^ c1 ^ k0, q & low, ((p >> 32) & low) ^ c3 ^ k1, p & low
        k0, k1 = (k0 + 0x9E3779B9) & low, (k1 + 0xBB67AE85) & low
    words = torch.stack([c0, c1, c2, c3], 1)
    halves = torch.stack([words & 0xFFFF, words >> 16], 2).reshape(-1)[:m]
    return (halves >= round(case["p"] * 65536)).reshape(case["n"], case["d"])


def _plain_dropout(s):
    case, x = s["case"], s["x"]
    keep = _kept(case, s["seed"], s["offset"], x.device)
    scale = 65536 / (65536 - round(case["p"] * 65536))
    out = (x.float() * scale).masked_fill(~keep, 0.0)
    if s["residual"] is not None:
        out = out + s["residual"].float()
    return dict(out=out.to(x.dtype), grad=(s["grad"].float() * scale).masked_fill(~keep, 0.0).to(x.dtype))


def _plain_pool(s):
    case, x = s["case"], s["x"]
    b, d = case["b"], case["d"]
    seq, _, _, pad = _rows(s)
    count = torch.zeros(b, device=x.device).index_add_(0, seq, (~pad).float()).clamp(min=1.0)[:, None]
    if s["offsets"] is None:
        total = x.float().masked_fill(pad.reshape(b, -1)[:, :, None], 0.0).sum(1)
    else:
        total = torch.zeros(b, d, device=x.device).index_add_(0, seq, x.float())
    mean = total / count
    norm = mean.square().sum(1, keepdim=True).clamp(min=1e-12).sqrt()
    unit = mean / norm
    out = dict(vectors=unit.to(x.dtype))
    if case["train"]:
        g = s["grad"].float()
        dm = (g - unit * (unit * g).sum(1, keepdim=True)) / norm / count
        dm = torch.where(norm > 1e-6, dm, g / norm / count)
        out["grad_x"] = dm.to(x.dtype)[seq].masked_fill(pad[:, None], 0.0).reshape(x.shape)
    return out


_PLAIN = dict(encode=_plain_scan, train=_plain_scan, step=_plain_step, dropout=_plain_dropout, pool=_plain_pool)


# ------------------------------------------------------------- the framework's calls
def _own_scan(mips, s):
    case = s["case"]
    at = dict(lengths=s["lengths"], offsets=s["offsets"], initial=s["initial"])
    f = mips.gated_scan(s["x"], s["forget"], s["gate"], states=case["states"], **at)
    out = dict(last=f.last)
    if case["states"]:
        out["states"] = f.states
    if case["op"] == "encode":
        return out
    dx, df, dg, di = mips.gated_scan_backward(s["grad_states"], s["grad_last"], s["x"], s["forget"], s["gate"], f, **at)
    out.update(grad_x=dx, grad_forget=df)
    if s["gate"] is not None:
        out["grad_gate"] = dg
    if s["initial"] is not None:
        out["grad_initial"] = di
    return out


def _own_step(mips, s):
    h = mips.gated_step(s["x"], s["forget"], s["state"], s["rows"], s["gate"], out=s["out"])
    return dict(states=h, table=s["out"])


def _own_dropout(mips, s):
    p, seed, offset = s["case"]["p"], s["seed"], s["offset"]
    return dict(out=mips.dropout(s["x"], p, seed, offset, residual=s["residual"]), grad=mips.dropout(s["grad"], p, seed, offset))


def _own_pool(mips, s):
    at = dict(lengths=s["lengths"], offsets=s["offsets"])
    f = mips.pool_normalize(s["x"], **at)
    out = dict(vectors=f.vectors)
    if s["case"]["train"]:
        out["grad_x"] = mips.pool_normalize_backward(s["grad"], s["x"].shape, f, **at)
    return out


_OWN = dict(encode=_own_scan, train=_own_scan, step=_own_step, dropout=_own_dropout, pool=_own_pool)


def run(state):
    op = state["case"]["op"]
    if own:
        import exact_inner_product_amd as mips
        return _OWN[op](mips, state)
    return _PLAIN[op](state)


def work(case):
    op, e, d = case["op"], _SIZE[case["dtype"]], case["d"]
    if op == "dropout":
        m = case["n"] * d
        return dict(bytes=m * e * (5 if case["residual"] else 4), flops=3 * m)
    if op == "step":
        m = case["b"] * d
        return dict(bytes=m * (8 + e * (4 if case["gate"] else 3)) + 4 * case["b"], flops=8 * m)
    m, ends = int(_lengths(case).sum()) * d, case["b"] * d
    if op == "pool":
        return dict(bytes=m * e * (2 if case["train"] else 1) + ends * e * (2 if case["train"] else 1), flops=m * (2 if case["train"] else 1))
    # x, forget and gate, the states; then their gradients
    tensors = 2 + case["gate"] + case["states"]
    small = 1 + case["initial"]
    if op == "train":
        tensors, small = 2 * tensors, 2 * small
    return dict(bytes=m * e * tensors + 4 * ends * small, flops=m * (10 if op == "encode" else 30))


# -------------------------------------------------- the definitions, in 64 bits
def _padded(v, lengths, t):
    """Packed rows as [t, b, d] in 64 bits, zeros behind each sequence's end; (also its inverse's index)."""
    b = len(lengths)
    rows = np.repeat(np.arange(b), lengths)
    pos = np.arange(int(lengths.sum())) - np.repeat(np.cumsum(lengths) - lengths, lengths)
    at = (torch.from_numpy(pos).cuda(), torch.from_numpy(rows).cuda())
    out = torch.zeros(t, b, v.shape[-1], dtype=torch.float64, device="cuda")
    if v.dim() == 3:
        out[at] = v[at[1], at[0]].double()
    else:
        out[at] = v.double()
    return out, at


def _exact_scan(s):
    case = s["case"]
    b, t, d = case["b"], case["t"], case["d"]
    lengths = _lengths(case)
    x, at = _padded(s["x"], lengths, t)
    f = _padded(s["forget"], lengths, t)[0]
    a, w = 1.0 / (1.0 + torch.exp(-f)), 1.0 / (1.0 + torch.exp(f))
    if s["gate"] is not None:
        w = 1.0 / (1.0 + torch.exp(-_padded(s["gate"], lengths, t)[0]))
    live = torch.zeros(t, b, 1, dtype=torch.bool, device="cuda")
    live[at] = True
    a, w = torch.where(live, a, 1.0), torch.where(live, w, 0.0)   # behind the end the state stays
    h = torch.zeros(b, d, dtype=torch.float64, device="cuda") if s["initial"] is None else s["initial"].double()
    u = w * x
    hs = torch.empty(t + 1, b, d, dtype=torch.float64, device="cuda")
    hs[0] = h
    for i in range(t):
        torch.addcmul(u[i], a[i], hs[i], out=hs[i + 1])

    def whole(v):
        if s["x"].dim() == 2:
            return v[at]
        out = torch.zeros(b, t, d, dtype=torch.float64, device="cuda")
        out[at[1], at[0]] = v[at]
        return out

    out = dict(last=hs[t].clone())
    if case["states"]:
        out["states"] = whole(hs[1:])
    if case["op"] == "encode":
        return out
    g = s["grad_last"].double()
    gs = torch.zeros_like(u) if s["grad_states"] is None else _padded(s["grad_states"], lengths, t)[0]
    total = u                                                  # its values are no longer needed
    for i in range(t - 1, -1, -1):
        torch.add(gs[i], g, out=total[i])
        g = total[i] * a[i]
    out["grad_x"] = whole(total * w)
    if s["gate"] is None:
        out["grad_forget"] = whole(total * (hs[:-1] - x) * a * (1 - a))
    else:
        out["grad_forget"] = whole(total * hs[:-1] * a * (1 - a))
        out["grad_gate"] = whole(total * x * w * (1 - w))
    if s["initial"] is not None:
        out["grad_initial"] = g
    return out


def _exact_step(s):
    table = s["state"].double()
    x, f = s["x"].double(), s["forget"].double()
    a = torch.exp(-torch.log1p(torch.exp(-f)))
    w = 1.0 - a if s["gate"] is None else torch.exp(-torch.log1p(torch.exp(-s["gate"].double())))
    rows = s["rows"].cpu().numpy()
    seen, wave = {}, np.empty(len(rows), dtype=np.int64)
    for e, r in enumerate(rows.tolist()):                      # an event's place among its row's
        wave[e] = seen[r] = seen.get(r, -1) + 1
    h = torch.empty_like(x)
    for k in range(int(wave.max()) + 1):
        e = torch.from_numpy(np.nonzero(wave == k)[0]).cuda()
        r = s["rows"][e].long()
        h[e] = a[e] * table[r] + w[e] * x[e]
        table[r] = h[e]
    return dict(states=h, table=table)


def _exact_dropout(s):
    case = s["case"]
    m = case["n"] * case["d"]
    i = np.arange((m + 7) // 8, dtype=np.uint64)
    mask, half = np.uint64(0xFFFFFFFF), np.uint64(32)
    ctr = [i & mask, i >> half, np.full_like(i, s["offset"] % (1 << 32)), np.full_like(i, s["offset"] >> 32)]
    key = [s["seed"] % (1 << 32), s["seed"] >> 32]
    for _ in range(10):
        hi_lo = [ctr[0] * np.uint64(0xD2511F53), ctr[2] * np.uint64(0xCD9E8D57)]
        ctr = [(hi_lo[1] >> half) ^ ctr[1] ^ np.uint64(key[0]), hi_lo[1] & mask,
               (hi_lo[0] >> half) ^ ctr[3] ^ np.uint64(key[1]), hi_lo[0] & mask]
        key = [(key[0] + 0x9E3779B9) % (1 << 32), (key[1] + 0xBB67AE85) % (1 << 32)]
    bits = np.stack([c.astype(np.uint32) for c in ctr], 1).astype("<u4").view("<u2").reshape(-1)[:m]
    cut = int(math.floor(case["p"] * 65536 + 0.5))
    factor = torch.from_numpy((bits >= cut).reshape(case["n"], case["d"])).cuda().double() * (65536.0 / (65536 - cut))
    out = s["x"].double() * factor
    if s["residual"] is not None:
        out += s["residual"].double()
    return dict(out=out, grad=s["grad"].double() * factor)


def _exact_pool(s):
    case = s["case"]
    lengths = _lengths(case)
    n = torch.from_numpy(lengths).cuda().double().clamp(min=1)[:, None]
    x, at = _padded(s["x"], lengths, case["t"])
    mean = x.sum(0) / n
    square = (mean * mean).sum(1, keepdim=True)
    norm = torch.sqrt(torch.clamp(square, min=1e-12))
    out = dict(vectors=mean / norm)
    if case["train"]:
        g = s["grad"].double()
        dm = g / norm - torch.where(square > 1e-12, mean * (mean * g).sum(1, keepdim=True) / norm ** 3, torch.zeros_like(mean))
        if s["x"].dim() == 2:
            out["grad_x"] = (dm / n)[at[1]]
        else:
            out["grad_x"] = torch.zeros(s["x"].shape, dtype=torch.float64, device="cuda")
            out["grad_x"][at[1], at[0]] = (dm / n)[at[1]]
    return out


def exact(case, seed):
    s = prepare(case, seed)
    kinds = dict(encode=_exact_scan, train=_exact_scan, step=_exact_step, dropout=_exact_dropout, pool=_exact_pool)
    return kinds[case["op"]](s)
