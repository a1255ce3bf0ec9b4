"""The gated recurrence over sequences and its gradient against a plain loop in 64 bits; the bounds
are derived in histories_check."""
import numpy as np
import pytest
import torch

import exact_inner_product_amd as mips
from tests import histories_check as hc
from tests.histories_check import DT

pytestmark = pytest.mark.gpu


def _dev():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    return torch.device("cuda:0")


def _lengths(kind, b, t, rng):
    n = rng.integers(0, t + 1, b)
    if kind == "none":
        n[:] = 0
    elif kind == "ends":
        n[0], n[-1] = 0, t
    elif kind == "holes":
        n[rng.random(b) < 0.6] = 0
    return n


def make(layout, b, t, d, dtype, gate, initial, seed=0, lens="ends"):
    """Inputs on the CPU: a dict of tensors and how they are laid out."""
    rng = np.random.default_rng(seed + b * 1000 + t * 10 + d)
    c = dict(layout=layout, b=b, t=t, d=d, lengths=None, offsets=None)
    shape = (b, t, d)
    if layout == "padded":
        c["lengths"] = torch.from_numpy(_lengths(lens, b, t, rng))
    if layout == "packed":
        n = _lengths(lens, b, t, rng)
        before, after = (3, 2) if lens == "ends" else (0, 0)  # rows of no sequence
        off = before + np.concatenate([[0], np.cumsum(n)])
        c["offsets"] = torch.from_numpy(off)
        shape = (int(off[-1]) + after, d)
    t32 = lambda *s, m=0.0, k=1.0: torch.from_numpy((rng.standard_normal(s) * k + m).astype(np.float32))  # noqa: E731
    c["x"] = t32(*shape).to(DT[dtype])
    c["forget"] = t32(*shape, m=1.5, k=2.0).to(DT[dtype])
    c["gate"] = t32(*shape, k=2.0).to(DT[dtype]) if gate else None
    c["initial"] = t32(b, d) if initial else None
    c["gs"], c["gl"] = t32(*shape).to(DT[dtype]), t32(b, d)
    c["seqs"] = hc.spans(layout, shape, c["lengths"], c["offsets"])
    return c


def flat(v):
    return None if v is None else v.double().numpy().reshape(-1, v.shape[-1])


def place(c, dev, index=torch.int32):
    """The case on the GPU."""
    out = {k: (v.to(dev) if isinstance(v, torch.Tensor) else v) for k, v in c.items()}
    for k in ("lengths", "offsets"):
        out[k] = None if out[k] is None else out[k].to(index)
    return out


def run(c, dev, states=True, grads=("gs", "gl"), index=torch.int32):
    p = place(c, dev, index)
    at = dict(lengths=p["lengths"], offsets=p["offsets"], initial=p["initial"])
    f = mips.gated_scan(p["x"], p["forget"], p["gate"], states=states, **at)
    g = mips.gated_scan_backward(p["gs"] if "gs" in grads else None, p["gl"] if "gl" in grads else None, p["x"], p["forget"],
                                 p["gate"], f, **at)
    return f, g


def check(c, f, g, grads=("gs", "gl")):
    x, ff, gg, init = (flat(c[k]) for k in ("x", "forget", "gate", "initial"))
    h, e, last, le = hc.scan(x, ff, gg, c["seqs"], init)
    if f.states is not None:
        assert f.states.shape == c["x"].shape and f.states.dtype == c["x"].dtype
        pad = np.ones(len(x), dtype=bool)
        for lo, hi in c["seqs"]:
            pad[lo:hi] = False
        assert not f.states.reshape(-1, c["d"])[torch.from_numpy(pad).to(f.states.device)].any()
        hc.within(f.states, h, e, "states")
    hc.within(f.last, last, le, "last")
    want = hc.scan_grad(x, ff, gg, c["seqs"], init, flat(c["gs"]) if "gs" in grads else None, flat(c["gl"]) if "gl" in grads else None)
    for name, got, w in zip(("grad_x", "grad_forget", "grad_gate", "grad_initial"), g, want):
        if got is None:
            assert (name == "grad_gate" and gg is None) or (name == "grad_initial" and init is None)
            continue
        hc.within(got, w[0], w[1], name)


CASES = [
    # layout, b, t, d
    ("dense", 1, 1, 1), ("dense", 3, 1, 128), ("dense", 300, 1, 16), ("dense", 1, 2, 4), ("dense", 5, 7, 3),
    ("dense", 1, 50, 64), ("dense", 40, 50, 16), ("dense", 9, 127, 128), ("dense", 4, 128, 132), ("dense", 4, 129, 128),
    ("dense", 2, 300, 100), ("dense", 3, 1000, 16), ("dense", 1, 2500, 30), ("dense", 2, 1500, 260), ("dense", 1, 700, 64),
    ("padded", 1, 1, 8), ("padded", 7, 20, 33), ("padded", 30, 127, 128), ("padded", 6, 400, 64), ("padded", 3, 900, 128),
    ("padded", 500, 3, 16), ("packed", 1, 1, 16), ("packed", 1, 300, 128), ("packed", 40, 60, 100), ("packed", 12, 500, 128),
    ("packed", 2000, 3, 32), ("packed", 3, 2500, 16), ("packed", 30, 200, 1), ("packed", 5, 700, 260),
]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("layout,b,t,d", CASES)
def test_scan(layout, b, t, d, dtype):
    dev = _dev()
    for gate, initial in ((False, False), (True, True)):
        print(f"scan {layout} b={b} t={t} d={d} {dtype} gate={gate} initial={initial}", flush=True)
        c = make(layout, b, t, d, dtype, gate, initial)
        check(c, *run(c, dev))


@pytest.mark.parametrize("lens", ["none", "holes"])
@pytest.mark.parametrize("layout,b,t,d", [("padded", 9, 40, 64), ("padded", 9, 400, 64), ("packed", 9, 40, 64),
                                          ("packed", 3000, 9, 128), ("packed", 200, 400, 20)])
def test_sequences_without_rows(layout, b, t, d, lens):
    dev = _dev()
    print(f"scan {lens} {layout} b={b} t={t} d={d}", flush=True)
    c = make(layout, b, t, d, "f32", True, True, lens=lens)
    check(c, *run(c, dev, index=torch.int64))
    c = make(layout, b, t, d, "bf16", False, False, lens=lens)
    check(c, *run(c, dev))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("t", [2, 3, 4, 5, 7, 8, 9, 12, 15, 16, 17])
def test_sequences_about_as_long_as_a_run(t, dtype):
    """Padded sequences that begin and end at every place of a thread's rows, many of them empty."""
    dev = _dev()
    for lens in ("ends", "holes"):
        c = make("padded", 70, t, 20, dtype, t % 2 == 0, True, lens=lens)
        check(c, *run(c, dev))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("layout,b,t,d,gate", [("dense", 1, 6000, 128, False), ("dense", 2, 3500, 70, True), ("padded", 2, 4500, 130, False),
                                               ("packed", 3, 3000, 128, True), ("dense", 1, 30000, 3, False)])
def test_states_that_reach_far(layout, b, t, d, gate, dtype):
    """Gates near 1: what a row sees comes from thousands of rows before, over many tiles and groups of
    them, as do the gradients from behind."""
    dev = _dev()
    c = make(layout, b, t, d, dtype, gate, True)
    c["forget"] = (c["forget"].float() * 0.5 + 8.0).to(DT[dtype])
    check(c, *run(c, dev))


@pytest.mark.parametrize("layout,b,t,d", [("dense", 3, 40, 64), ("dense", 2, 600, 128), ("padded", 8, 200, 100), ("packed", 8, 200, 64)])
def test_parts_of_the_gradient(layout, b, t, d):
    """Only the last state's gradient, only the states'; without states the last ones stay the same."""
    dev = _dev()
    print(f"parts {layout} b={b} t={t} d={d}", flush=True)
    c = make(layout, b, t, d, "bf16", False, True)
    f, g = run(c, dev)
    for grads in (("gl",), ("gs",)):
        f2, g2 = run(c, dev, states=False, grads=grads)
        assert f2.states is None and torch.equal(f2.last, f.last)
        check(c, f2, g2, grads)
    p = place(c, dev)
    at = dict(lengths=p["lengths"], offsets=p["offsets"], initial=p["initial"])
    f3 = mips.gated_scan(p["x"], p["forget"], carries=False, **at)
    assert f3.carries is None and torch.equal(f3.states, f.states) and torch.equal(f3.last, f.last)
    with pytest.raises(ValueError, match="carries"):
        mips.gated_scan_backward(p["gs"], None, p["x"], p["forget"], None, f3, **at)


@pytest.mark.parametrize("layout,b,t,d", [("dense", 2, 50, 64), ("dense", 3, 700, 64), ("padded", 5, 200, 128), ("packed", 5, 300, 36)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_strides(layout, b, t, d, dtype):
    """Views with wider rows, gaps between sequences, rows that are not aligned, turned and broadcast ones."""
    dev = _dev()
    print(f"strides {layout} b={b} t={t} d={d} {dtype}", flush=True)
    c = make(layout, b, t, d, dtype, True, True)
    p = place(c, dev)
    at = dict(lengths=p["lengths"], offsets=p["offsets"], initial=p["initial"])
    f = mips.gated_scan(p["x"], p["forget"], p["gate"], **at)
    want = mips.gated_scan_backward(p["gs"], p["gl"], p["x"], p["forget"], p["gate"], f, **at)

    def wide(v, k, shift):  # [..., rows + 3, d + k] cut back
        big = torch.full((*v.shape[:-2], v.shape[-2] + 3, v.shape[-1] + k), float("nan"), dtype=v.dtype, device=dev)
        cut = big[..., 1:1 + v.shape[-2], shift:shift + v.shape[-1]]
        cut.copy_(v)
        return cut

    def turned(v):
        return v.transpose(-1, -2).contiguous().transpose(-1, -2)

    for change in (lambda v: wide(v, 8, 4), lambda v: wide(v, 3, 1), turned):
        x, fg, gt, gs = (change(p[k]) for k in ("x", "forget", "gate", "gs"))
        f2 = mips.gated_scan(x, fg, gt, **at)
        g2 = mips.gated_scan_backward(gs, p["gl"], x, fg, gt, f2, **at)
        assert torch.equal(f2.states, f.states) and torch.equal(f2.last, f.last)
        assert all(torch.equal(u, v) for u, v in zip(g2, want))
    one = p["gs"].reshape(-1, d)[:1].expand(p["gs"].numel() // d, d).reshape(p["gs"].shape)
    broad = p["gs"].reshape(-1, d)[:1].expand(*p["gs"].shape)
    g2 = mips.gated_scan_backward(broad, p["gl"], p["x"], p["forget"], p["gate"], f, **at)
    g3 = mips.gated_scan_backward(one.contiguous(), p["gl"], p["x"], p["forget"], p["gate"], f, **at)
    assert all(torch.equal(u, v) for u, v in zip(g2, g3))


@pytest.mark.parametrize("layout,b,t,d", [("padded", 6, 90, 64), ("padded", 4, 600, 128), ("packed", 6, 150, 64)])
def test_padding_may_hold_anything(layout, b, t, d):
    dev = _dev()
    print(f"padding {layout} b={b} t={t} d={d}", flush=True)
    c = make(layout, b, t, d, "bf16", True, True)
    f, g = run(c, dev)
    pad = torch.ones(c["x"].numel() // d, dtype=torch.bool)
    for lo, hi in c["seqs"]:
        pad[lo:hi] = False
    for bad in (float("nan"), float("inf"), -float("inf"), torch.finfo(torch.bfloat16).min):
        c2 = dict(c)
        for k in ("x", "forget", "gate", "gs"):
            c2[k] = c[k].clone()
            c2[k].view(-1, d)[pad] = bad
        f2, g2 = run(c2, dev)
        assert torch.equal(f2.states, f.states) and torch.equal(f2.last, f.last)
        assert all(torch.equal(u, v) for u, v in zip(g2, g))


def test_nan_stays_in_its_sequence_and_channel():
    dev = _dev()
    for layout, b, t, d in (("dense", 6, 40, 64), ("dense", 4, 700, 64), ("packed", 7, 300, 128)):
        print(f"nan {layout}", flush=True)
        c = make(layout, b, t, d, "f32", False, False)
        f, g = run(c, dev)
        lo, hi = next((lo, hi) for lo, hi in c["seqs"][1:] if hi - lo > 5)
        for bad in (float("nan"), float("inf")):
            c2 = dict(c)
            c2["x"] = c["x"].clone()
            c2["x"].view(-1, d)[lo + 3, 5] = bad
            f2, g2 = run(c2, dev)
            h, h2 = f.states.view(-1, d), f2.states.view(-1, d)
            hit = torch.zeros_like(h, dtype=torch.bool)
            hit[lo + 3:hi, 5] = True
            assert not torch.isfinite(h2[hit]).any() and torch.equal(h2[~hit], h[~hit])
            # the gradient for x does not depend on x
            assert torch.equal(g2[0], g[0])
            same = ~hit
            assert torch.equal(g2[1].view(-1, d)[same], g[1].view(-1, d)[same])


def test_extreme_gates():
    """Logits of +inf and -inf: a state that is kept for good, and one that is replaced. sigmoid(-inf) is
    held at 2^-126, which changes no state here, and a gradient by less than |D| (|h| + |x|) 2^-126."""
    dev = _dev()
    for t in (90, 1500):
        c = make("dense", 2, t, 64, "f32", False, True)
        c["forget"][0] = float("inf")       # kept
        c["forget"][1] = -float("inf")      # replaced
        f, g = run(c, dev)
        assert torch.equal(f.states[0].cpu(), c["initial"][0].expand(t, 64))
        assert torch.equal(f.states[1].cpu(), c["x"][1])
        assert not g[0][0].any() and not g[1][0].any() and (g[1][1].abs() < 1e-36).all()
        want = c["gs"].clone()
        want[1, -1] += c["gl"][1]
        assert torch.equal(g[0][1].cpu(), want[1])
        c["forget"][0], c["forget"][1] = 300.0, -300.0
        f, _ = run(c, dev)
        assert torch.equal(f.states[0].cpu(), c["initial"][0].expand(t, 64)) and torch.equal(f.states[1].cpu(), c["x"][1])


def test_same_call_same_bits():
    dev = _dev()
    for layout, b, t, d in (("dense", 2, 9000, 64), ("packed", 700, 90, 128), ("dense", 1, 40000, 16)):
        c = make(layout, b, t, d, "bf16", True, True)
        f, g = run(c, dev)
        for _ in range(4):
            f2, g2 = run(c, dev)
            assert torch.equal(f2.states, f.states) and torch.equal(f2.last, f.last)
            assert all(torch.equal(u, v) for u, v in zip(g2, g))


def test_broken_offsets_stay_in_bounds():
    """Decreasing offsets and ones outside the rows: results are meaningless, neighbours are not touched."""
    dev = _dev()
    n, d = 1000, 64
    big = torch.randn(3, n, d, device=dev)
    for off in ([5, -7, 2000, 3, 10 ** 9, 600, 1000], [1000, 0], [0, 0, 0, 0], [-1, -1], [n + 5, n + 9], [900, 100, 900, 100]):
        o = torch.tensor(off, dtype=torch.int32, device=dev)
        print(f"offsets {off}", flush=True)
        f = mips.gated_scan(big[0], big[1], offsets=o)
        g = mips.gated_scan_backward(big[2], None, big[0], big[1], None, f, offsets=o)
        p = mips.pool_normalize(big[0], offsets=o)
        mips.pool_normalize_backward(p.vectors, big[0].shape, p, offsets=o)
        torch.cuda.synchronize()
        assert f.last.shape == (len(off) - 1, d) and g[0].shape == (n, d)
    padded = torch.tensor([-5, 400, 7], dtype=torch.int64, device=dev)
    x = torch.randn(3, 300, d, device=dev)
    want = mips.gated_scan(x, x, lengths=torch.tensor([0, 300, 7], device=dev))
    got = mips.gated_scan(x, x, lengths=padded)
    assert torch.equal(got.states, want.states) and torch.equal(got.last, want.last)


@pytest.mark.parametrize("layout,b,t,d,dtype", [("dense", 1, 60000, 128, "f32"), ("dense", 1, 120000, 100, "bf16"), ("dense", 2, 40000, 130, "bf16"),
                                                ("padded", 3, 30000, 65, "f32"), ("packed", 4, 50000, 66, "f32"), ("packed", 300, 900, 128, "bf16"),
                                                ("dense", 1, 300000, 16, "f32")])
def test_exact_sums_over_long_chains(layout, b, t, d, dtype):
    """Gates of infinity keep the state and take the input whole: states are sums of small whole numbers, exact
    in binary32 in whatever order maps are joined (below 2^24), and gradients are sums from behind."""
    dev = _dev()
    gen = torch.Generator().manual_seed(t)
    lengths = torch.randint(0, t + 1, (b,), generator=gen)
    lengths[0] = t
    if layout == "dense":
        lengths[:] = t
    offsets = torch.cat([torch.zeros(1, dtype=torch.int64), lengths.cumsum(0)])
    shape = (int(offsets[-1]), d) if layout == "packed" else (b, t, d)
    x, gs = (torch.randint(-3, 4, shape, generator=gen) for _ in range(2))
    initial, gl = (torch.randint(-9, 10, (b, d), generator=gen) for _ in range(2))
    h, dx, last, di = torch.zeros_like(x), torch.zeros_like(x), initial.clone(), gl.clone()
    for s in range(b):
        n = int(lengths[s])
        rows = (lambda v: v[offsets[s]:offsets[s] + n]) if layout == "packed" else (lambda v: v[s, :n])  # noqa: E731
        if n:
            rows(h)[:] = rows(x).cumsum(0) + initial[s]
            rows(dx)[:] = rows(gs).flip(0).cumsum(0).flip(0) + gl[s]
            last[s], di[s] = rows(h)[-1], rows(dx)[0]
    at = {"padded": dict(lengths=lengths.to(dev)), "packed": dict(offsets=offsets.to(dev))}.get(layout, {})
    at["initial"] = initial.float().to(dev)
    dt, gates = DT[dtype], torch.full(shape, float("inf"), dtype=DT[dtype], device=dev)
    xd, gd, gld = x.to(dev, dt), gs.to(dev, dt), gl.float().to(dev)
    want_h, want_dx = h.to(dev).to(dt), dx.to(dev).to(dt)
    for _ in range(5):
        f = mips.gated_scan(xd, gates, gates, **at)
        g = mips.gated_scan_backward(gd, gld, xd, gates, gates, f, **at)
        assert torch.equal(f.states, want_h) and torch.equal(f.last, last.to(dev).float())
        assert torch.equal(g[0], want_dx) and torch.equal(g[3], di.to(dev).float())
        assert not g[1].any() and not g[2].any()
        assert torch.equal(mips.gated_scan(xd, gates, gates, states=False, carries=False, **at).last, f.last)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("layout,b,t,d", [("dense", 3, 9, 4), ("padded", 5, 60, 33), ("dense", 2, 1500, 64), ("packed", 4, 900, 128)])
def test_gates_of_minus_infinity_are_zero(layout, b, t, d, dtype):
    """Inputs of the type's lowest value behind gates of -inf leave nothing in the state, and a forget logit
    of -inf nothing of a state that large: what is left are sums of small whole numbers, exact in binary32.
    Likewise for the gradients of what such gates keep out."""
    dev = _dev()
    c = make(layout, b, t, d, dtype, True, True)
    rng = np.random.default_rng(t)
    shape, low = c["x"].shape, torch.finfo(DT[dtype]).min
    whole = lambda *s: torch.from_numpy(rng.integers(-3, 4, s)).float()  # noqa: E731
    masked, first = torch.from_numpy(rng.random(shape) < 0.4), torch.zeros(shape, dtype=torch.bool)
    for lo, hi in c["seqs"]:
        if hi > lo:
            first.view(-1, d)[lo] = True
    x, c["initial"] = whole(*shape), torch.full((b, d), torch.finfo(torch.float32).min)
    inf = torch.full(shape, float("inf"))
    c["x"] = torch.where(masked, low, x).to(DT[dtype])
    c["gate"] = torch.where(masked, -inf, inf).to(DT[dtype])
    c["forget"] = torch.where(first, -inf, inf).to(DT[dtype])  # nothing is left of the initial state
    h, last = torch.zeros(shape).view(-1, d), c["initial"].clone()
    kept, want_dx = torch.where(masked, 0.0, x).view(-1, d), torch.zeros(shape).view(-1, d)
    c["gs"] = whole(*shape).to(DT[dtype])
    f, (dx, df, dg, di) = run(c, dev, grads=("gs",))
    for s, (lo, hi) in enumerate(c["seqs"]):
        if hi > lo:
            h[lo:hi] = kept[lo:hi].cumsum(0)
            last[s] = h[hi - 1]
            want_dx[lo:hi] = c["gs"].float().view(-1, d)[lo:hi].flip(0).cumsum(0).flip(0)
    assert torch.equal(f.states.cpu().view(-1, d), h.to(DT[dtype])) and torch.equal(f.last.cpu(), last)
    assert torch.equal(dx.cpu().view(-1, d), torch.where(masked.view(-1, d), 0.0, want_dx).to(DT[dtype]))
    assert not di.any() and not df.any()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("layout,b,t,d", [("dense", 2, 7, 5), ("padded", 3, 90, 64), ("dense", 1, 900, 128)])
def test_gate_gradients_of_large_inputs(layout, b, t, d, dtype):
    """grad_gate = D x b (1 - b) where D x alone is past the largest value: small with a gate far below 0,
    0 with one of -inf."""
    dev = _dev()
    c = make(layout, b, t, d, dtype, True, False)
    c["x"] = torch.sign(c["x"].float()).mul(3e38).to(DT[dtype])
    c["gate"] = c["gate"].float().sub(24.0).to(DT[dtype])
    c["forget"][..., 1, :] = 0.0
    c["gs"], c["gl"] = (torch.where(v < 0, -8.0, 8.0).to(v.dtype) for v in (c["gs"], c["gl"]))
    check(c, *run(c, dev))
    c["gate"].fill_(-float("inf"))
    f, g = run(c, dev)
    assert not f.states.any() and not g[0].any() and not g[1].any() and not g[2].any()
