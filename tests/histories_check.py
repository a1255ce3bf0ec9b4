"""Plain 64-bit forms of the operators over histories, on the CPU, with bounds on what binary32 may
be off by. u = 2^-24 is half a unit in the last place, relative to the value.

Gates. sigmoid(v) is 1 / (1 + e) or e / (1 + e) with e = 2^(-|v| log2 e) in binary32: the rounded
constant and its product leave 2 |v| u in e, the exponential and the reciprocal (one unit in the last
place each) 2 u each, the sum and the product u each: within (2 |v| + 8) u =: k(v) u of the value.

States. A state is a sum of terms (product of gates) * b x; each row multiplies a term by a gate with
error k u and rounds once or twice (product, sum), joins of runs, waves and tiles round a term about
twice each, fewer than 32 times within a tile and twice a wave of rows beyond it. With M the same
recurrence over absolute values, the error is below E + 32 u M, E_r = a E_{r-1} + (k + 4) u (a M_{r-1} + b |x|).
The gradient's recurrence has the same form the other way.

Values below 2^-126 may be flushed to 0: 1e-36 is added to every bound."""
import numpy as np
import torch

U = 2.0 ** -24
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def spans(layout, shape, lengths=None, offsets=None):
    """[(first row, one past the last)] of each sequence, in rows as they lie."""
    if layout == "packed":
        return [(int(offsets[s]), int(offsets[s + 1])) for s in range(len(offsets) - 1)]
    b, t, _ = shape
    n = [t] * b if lengths is None else [min(max(int(v), 0), t) for v in lengths]
    return [(s * t, s * t + n[s]) for s in range(b)]


def gates(f, g):
    """(a, 1 - a, k_a, b, 1 - b, k_b) in 64 bits."""
    with np.errstate(over="ignore"):
        a, na = 1 / (1 + np.exp(-f)), 1 / (1 + np.exp(f))
        b, nb = (na, a) if g is None else (1 / (1 + np.exp(-g)), 1 / (1 + np.exp(g)))
    big = lambda v: 2 * np.minimum(np.abs(v), 200.0) + 8  # noqa: E731
    return a, na, big(f), b, nb, big(f if g is None else g)


def scan(x, f, g, seqs, initial):
    """(states, their bound, last, its bound); x, f, g: 64-bit [rows, d]."""
    n, d = x.shape
    a, na, ka, b, nb, kb = gates(f, g)
    h, e, m = np.zeros((n, d)), np.zeros((n, d)), np.zeros((n, d))
    last, laste = np.zeros((len(seqs), d)), np.zeros((len(seqs), d))
    for s, (lo, hi) in enumerate(seqs):
        hh = np.zeros(d) if initial is None else initial[s]
        ee, mm = np.zeros(d), np.abs(hh)
        for r in range(lo, hi):
            k = np.maximum(ka[r], kb[r]) + 4
            ee = a[r] * ee + k * U * (a[r] * mm + b[r] * np.abs(x[r]))
            mm = a[r] * mm + b[r] * np.abs(x[r])
            hh = a[r] * hh + b[r] * x[r]
            h[r], e[r], m[r] = hh, ee, mm
        last[s], laste[s] = hh, ee + 32 * U * mm
    return h, e + 32 * U * m + 1e-36, last, laste + 1e-36


def scan_grad(x, f, g, seqs, initial, gs, gl):
    """[(gradient, bound)] of x, forget, gate (None without) and initial."""
    n, d = x.shape
    a, na, ka, b, nb, kb = gates(f, g)
    h, he, _, _ = scan(x, f, g, seqs, initial)
    D, E, M = np.zeros((n, d)), np.zeros((n, d)), np.zeros((n, d))
    P, PE, PM = np.zeros((n, d)), np.zeros((n, d)), np.zeros((n, d))  # the state before each row
    live = np.zeros(n, dtype=bool)
    di, die = np.zeros((len(seqs), d)), np.zeros((len(seqs), d))
    hm = scan(np.abs(x), f, g, seqs, None if initial is None else np.abs(initial))[0]
    for s, (lo, hi) in enumerate(seqs):
        v = np.zeros(d) if gl is None else gl[s].copy()
        ve, vm = np.zeros(d), np.abs(v)
        for r in range(hi - 1, lo - 1, -1):
            live[r] = True
            q = np.zeros(d) if gs is None else gs[r]
            D[r], M[r] = q + v, np.abs(q) + vm
            E[r] = ve + 2 * U * M[r]
            v, vm = a[r] * D[r], a[r] * M[r]
            ve = a[r] * E[r] + (ka[r] + 4) * U * vm
            if r > lo:
                P[r], PE[r], PM[r] = h[r - 1], he[r - 1], hm[r - 1]
            elif initial is not None:
                P[r], PM[r] = initial[s], np.abs(initial[s])
        di[s], die[s] = v, ve + 32 * U * vm + 1e-36
    E = E + 32 * U * M
    x, f, b, nb = (np.where(live[:, None], w, 0.0) for w in (x, f, b, nb))
    out = [(D * b, E * b + (kb + 4) * U * M * b)]
    if g is None:
        w = a * na
        out += [(D * (P - x) * w, (E * np.abs(P - x) + M * PE + (2 * ka + 8) * U * M * (PM + np.abs(x))) * w), None]
    else:
        w = a * na
        out += [(D * P * w, (E * np.abs(P) + M * PE + (2 * ka + 8) * U * M * PM) * w),
                (D * x * b * nb, (E + (2 * kb + 8) * U * M) * np.abs(x) * b * nb)]
    out = [None if o is None else (np.where(live[:, None], o[0], 0.0), np.where(live[:, None], o[1], 0.0) + 1e-36) for o in out]
    return out + [(di, die)]


def within(got, want, tol, what):
    """got lies between the roundings of want - tol and want + tol to its type."""
    lo, hi = want - tol, want + tol
    if got.dtype == torch.bfloat16:
        lo, hi = (torch.from_numpy(v).bfloat16().double().numpy() for v in (lo, hi))
    v = got.detach().cpu().double().numpy().reshape(want.shape)
    bad = ~((lo <= v) & (v <= hi))
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} outside; worst {np.max(np.where(bad, np.abs(v - want) / tol, 0))} bounds at " \
        f"{np.unravel_index(np.argmax(np.where(bad, np.abs(v - want) / tol, 0)), bad.shape)}"


# ------------------------------------------------------------------------ dropout
def philox(c, key, rounds=10):
    """Philox4x32 over arrays: c a list of four, key of two (numpy uint64 below 2^32)."""
    low, half = np.uint64(0xFFFFFFFF), np.uint64(32)
    c, (k0, k1) = [np.asarray(v, dtype=np.uint64) for v in c], key
    for _ in range(rounds):
        p, q = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = [(q >> half) ^ c[1] ^ np.uint64(k0), q & low, (p >> half) ^ c[3] ^ np.uint64(k1), p & low]
        k0, k1 = (k0 + 0x9E3779B9) % (1 << 32), (k1 + 0xBB67AE85) % (1 << 32)
    return c


def kept(n, p, seed, offset, start=0):
    """Which of the elements start .. start + n - 1 dropout keeps (start a multiple of 8)."""
    i = np.arange(start // 8, (start + n + 7) // 8, dtype=np.uint64)
    full = lambda v: np.full_like(i, v)  # noqa: E731
    w = philox([i & np.uint64(0xFFFFFFFF), i >> np.uint64(32), full(offset % (1 << 32)), full(offset >> 32)],
               (seed % (1 << 32), seed >> 32))
    half = np.stack([v for x in w for v in (x & np.uint64(0xFFFF), x >> np.uint64(16))], 1).reshape(-1)[:n]
    return half >= int(p * 65536 + 0.5)
