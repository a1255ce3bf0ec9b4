"""The recurrence for single events against a table of states, against a plain loop in 64 bits
(bounds: histories_check; an event's state has been through as many rows as its row had events)."""
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


def make(kind, b, v, d, dtype, gate, seed=0):
    rng = np.random.default_rng(seed + b + v + d)
    f32 = lambda *s, m=0.0, k=1.0: torch.from_numpy((rng.standard_normal(s) * k + m).astype(np.float32))  # noqa: E731
    if kind == "one":
        rows = np.full(b, v // 2)
    elif kind == "pairs":
        rows = np.arange(b) // 2 % v
    elif kind == "few":
        rows = rng.integers(0, min(v, 5), b)
    elif kind == "padded":
        rows = rng.integers(-3, v + 3, b)
    else:
        rows = rng.integers(0, v, b)
    return dict(x=f32(b, d).to(DT[dtype]), forget=f32(b, d, m=1.0, k=2.0).to(DT[dtype]),
                gate=f32(b, d, k=2.0).to(DT[dtype]) if gate else None, state=f32(v, d), rows=torch.from_numpy(rows))


def reference(c):
    x, f = c["x"].double().numpy(), c["forget"].double().numpy()
    a, _, ka, w, _, kb = hc.gates(f, None if c["gate"] is None else c["gate"].double().numpy())
    table = c["state"].double().numpy().copy()
    err, mag = np.zeros_like(table), np.abs(table)
    h, he = np.zeros_like(x), np.zeros_like(x)
    for e, r in enumerate(c["rows"].tolist()):
        if not 0 <= r < len(table):
            continue
        err[r] = a[e] * err[r] + (np.maximum(ka[e], kb[e]) + 4) * hc.U * (a[e] * mag[r] + w[e] * np.abs(x[e]))
        mag[r] = a[e] * mag[r] + w[e] * np.abs(x[e])
        table[r] = a[e] * table[r] + w[e] * x[e]
        h[e], he[e] = table[r], err[r] + 1e-36
    return h, he, table, err


CASES = [("any", 1, 1, 1), ("any", 16, 1000, 64), ("any", 1000, 300, 128), ("padded", 300, 100, 33), ("few", 700, 20, 16),
         ("one", 900, 3, 128), ("pairs", 4096, 2048, 16), ("any", 513, 60, 260), ("padded", 5, 2, 1024), ("any", 64, 10, 4),
         ("one", 3000, 9, 20), ("few", 5000, 5, 8), ("any", 20000, 700, 8), ("any", 65536, 100000, 4), ("one", 65536, 2, 16)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("kind,b,v,d", CASES)
def test_step(kind, b, v, d, dtype):
    dev = _dev()
    print(f"step {kind} b={b} v={v} d={d} {dtype}", flush=True)
    for gate in (False, True):
        c = make(kind, b, v, d, dtype, gate)
        p = {k: None if t is None else t.to(dev) for k, t in c.items()}
        h, he, table, te = reference(c)
        kept = p["state"].clone()
        into = torch.full_like(kept, 7.0)
        got = mips.gated_step(p["x"], p["forget"], p["state"], p["rows"].to(torch.int32), p["gate"], out=into)
        assert torch.equal(p["state"], kept)
        hc.within(got, h, he, "states")
        named = torch.zeros(v, dtype=torch.bool)
        named[[r for r in c["rows"].tolist() if 0 <= r < v]] = True
        assert (into[~named.to(dev)] == 7.0).all()      # rows without an event are left as they were
        hc.within(into[named.to(dev)], table[named.numpy()], te[named.numpy()] + 1e-36, "table")
        again = mips.gated_step(p["x"], p["forget"], p["state"], p["rows"], p["gate"])  # in place, int64
        assert torch.equal(again, got) and torch.equal(p["state"][named.to(dev)], into[named.to(dev)])
        assert torch.equal(p["state"][~named.to(dev)], kept[~named.to(dev)])


def test_steps_make_the_scan():
    """A history event by event ends in the states of the scan over it, to their bounds."""
    dev = _dev()
    b, t, d = 50, 30, 64
    rng = np.random.default_rng(0)
    x, f, g = (torch.from_numpy(rng.standard_normal((b, t, d)).astype(np.float32)) for _ in range(3))
    want = mips.gated_scan(x.to(dev), f.to(dev), g.to(dev))
    state = torch.zeros(80, d, device=dev)
    rows = torch.randperm(80, device=dev)[:b]
    steps = [mips.gated_step(x[:, i].to(dev), f[:, i].to(dev), state, rows, g[:, i].to(dev)) for i in range(t)]
    flat = [v.double().numpy().reshape(-1, d) for v in (x, f, g)]
    _, e, _, le = hc.scan(*flat, [(s * t, s * t + t) for s in range(b)], None)
    assert (np.abs((torch.stack(steps, 1) - want.states).cpu().double().numpy()).reshape(-1, d) <= 2 * e).all()
    assert (np.abs((state[rows] - want.last).cpu().double().numpy()) <= 2 * le).all()


def test_strides_and_alignment():
    dev = _dev()
    for dtype in ("f32", "bf16"):
        c = make("any", 200, 50, 64, dtype, True)
        p = {k: t.to(dev) for k, t in c.items()}
        first = p["state"].clone()
        want = mips.gated_step(p["x"], p["forget"], first, p["rows"], p["gate"])
        for k, shift in ((4, 4), (3, 1)):
            cut = []
            for t in (p["x"], p["forget"], p["gate"], p["state"]):
                big = torch.full((t.shape[0], t.shape[1] + k + 1), float("nan"), dtype=t.dtype, device=dev)
                cut.append(big[:, shift:shift + t.shape[1]])
                cut[-1].copy_(t)
            got = mips.gated_step(cut[0], cut[1], cut[3], p["rows"], cut[2])
            assert torch.equal(got, want) and torch.equal(cut[3], first)
        got = mips.gated_step(p["x"], p["forget"], p["state"].clone(), p["rows"].repeat_interleave(2)[::2], p["gate"])
        assert torch.equal(got, want)


def test_offsets_past_32_bits():
    """Rows beyond 2^32 bytes and 2^31 elements of a table."""
    dev = _dev()
    v, d = 9_000_000, 256
    table = torch.empty(v, d, device=dev)
    rows = torch.tensor([v - 1, 3, 8_400_001, v - 1], device=dev)
    table[rows] = 2.0
    x, f = torch.ones(4, d, device=dev), torch.zeros(4, d, device=dev)
    h = mips.gated_step(x, f, table, rows)
    assert h[:, 0].tolist() == [1.5, 1.5, 1.5, 1.25] and table[rows, d - 1].tolist() == [1.25, 1.5, 1.5, 1.25]


def test_autograd_notices_the_table():
    dev = _dev()
    t = torch.ones(30, 8, device=dev, requires_grad=True)
    state = t * 1.0
    y = (state * state).sum()
    mips.gated_step(torch.ones(2, 8, device=dev), torch.ones(2, 8, device=dev), state.detach(), torch.tensor([0, 1], device=dev))
    with pytest.raises(RuntimeError, match="inplace operation"):
        y.backward()


def test_tables_that_overlap():
    """Tables beside each other in one tensor are taken, ones that share elements refused."""
    dev = _dev()
    x, f = torch.randn(5, 8, device=dev), torch.randn(5, 8, device=dev)
    rows = torch.tensor([0, 3, 1, 3, 9], device=dev)
    big = torch.randn(21, 20, device=dev)
    state = big[:10, :8].clone()
    want, out = mips.gated_step(x, f, state.clone(), rows), torch.zeros(10, 8, device=dev)
    mips.gated_step(x, f, state, rows, out=out)
    for into in (big[:10, 8:16], big[:10, 12:], big[10:20, :8], big[11:, 4:12]):
        into.zero_()
        assert torch.equal(mips.gated_step(x, f, big[:10, :8], rows, out=into), want) and torch.equal(into, out)
    for into in (big[1:11, :8], big[:10, 4:12], big[9:19, 7:15], big[:20:2, :8]):
        with pytest.raises(mips.MipsError):
            mips.gated_step(x, f, big[:10, :8], rows, out=into)
        with pytest.raises(mips.MipsError):
            mips.gated_step(x, f, into, rows, out=big[:10, :8])


def test_gates_of_minus_infinity_are_zero():
    """An event of the type's lowest value behind a gate of -inf leaves the state as it is, and a forget logit
    of -inf leaves nothing of a state that large."""
    dev = _dev()
    for dtype in (torch.float32, torch.bfloat16):
        inf, low = float("inf"), torch.finfo(dtype).min
        state = torch.tensor([2.0, torch.finfo(torch.float32).min], device=dev)[:, None].repeat(1, 20)
        x, forget, gate = (torch.tensor(v, device=dev)[:, None].expand(3, 20).to(dtype) for v in ([low, 5.0, low], [inf, -inf, inf], [-inf, inf, -inf]))
        h = mips.gated_step(x, forget, state, torch.tensor([0, 1, 1], device=dev), gate)
        assert h[:, 0].tolist() == [2.0, 5.0, 5.0] and state[:, 19].tolist() == [2.0, 5.0]
        assert (h == h[:, :1]).all() and (state == state[:, :1]).all()


def test_columns_of_one_tensor_with_other_rows():
    """A table beside every second (third) row's other columns shares nothing with it; of the same columns it does."""
    dev = _dev()
    x, f = torch.randn(5, 8, device=dev), torch.randn(5, 8, device=dev)
    rows = torch.tensor([0, 3, 1, 3, 9], device=dev)
    big = torch.randn(60, 20, device=dev)
    state = big[:10, :8].clone()
    out = torch.zeros(10, 8, device=dev)
    want = mips.gated_step(x, f, state, rows, out=out)
    for table, into in ((big[:10, :8], big[:20:2, 8:16]), (big[:10, :8], big[1:31:3, 12:]), (big[:30:3, :8], big[:20:2, 9:17])):
        table.copy_(state)
        into.zero_()
        assert torch.equal(mips.gated_step(x, f, table, rows, out=into), want) and torch.equal(into, out)
        assert torch.equal(table, state)
    for table, into in ((big[:10, :8], big[1:21:2, 4:12]), (big[:30:3, 8:16], big[:20:2, 9:17]), (big[:10, :8], big[1:21:2, 15:].as_strided((10, 8), (40, 1)))):
        for a, b in ((table, into), (into, table)):
            with pytest.raises(mips.MipsError):
                mips.gated_step(x, f, a, rows, out=b)


def crowd(kind, b, v, d, dtype, seed=0):
    """Events of which many are padding, or of one row, beside rows that come again."""
    c = make("any", b, v, d, dtype, True, seed)
    rng = np.random.default_rng(seed)
    rows = rng.integers(0, v, b)
    if kind in ("padding", "both"):
        rows[rng.random(b) < 0.5] = -1
    if kind in ("hot", "both"):
        rows[rng.random(b) < 0.3] = v // 3
    if kind == "outside":
        rows[rng.random(b) < 0.5] = v + (1 << 40)
        rows[rng.random(b) < 0.1] = -(1 << 62)
    if kind == "late":  # one row's events all behind those that other workgroups have
        rows[b // 2:] = np.where(rng.random(b - b // 2) < 0.6, v - 1, rows[b // 2:])
    c["rows"] = torch.from_numpy(rows)
    return c


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("kind,b,v,d", [("padding", 4096, 700, 16), ("padding", 65536, 20000, 4), ("both", 1000, 60, 33), ("hot", 4096, 1500, 20),
                                        ("outside", 6000, 900, 8), ("both", 40000, 9000, 8), ("hot", 65536, 30000, 4), ("late", 50000, 40000, 4),
                                        ("late", 17000, 300, 12), ("both", 2500, 100, 520)])
def test_padding_and_rows_that_come_again(kind, b, v, d, dtype):
    dev = _dev()
    print(f"crowd {kind} b={b} v={v} d={d} {dtype}", flush=True)
    c = crowd(kind, b, v, d, dtype)
    p = {k: t.to(dev) for k, t in c.items()}
    h, he, table, te = reference(c)
    into, kept = torch.full_like(p["state"], 7.0), p["state"].clone()
    got = mips.gated_step(p["x"], p["forget"], p["state"], p["rows"], p["gate"], out=into)
    assert torch.equal(p["state"], kept)
    hc.within(got, h, he, "states")
    named = torch.zeros(v, dtype=torch.bool)
    rows = c["rows"][(c["rows"] >= 0) & (c["rows"] < v)]
    named[rows] = True
    assert (into[~named.to(dev)] == 7.0).all()
    hc.within(into[named.to(dev)], table[named.numpy()], te[named.numpy()] + 1e-36, "table")
    for _ in range(3):
        state = kept.clone()
        again = mips.gated_step(p["x"], p["forget"], state, p["rows"], p["gate"])
        assert torch.equal(again, got) and torch.equal(state[named.to(dev)], into[named.to(dev)])
        assert torch.equal(state[~named.to(dev)], kept[~named.to(dev)])


def _in_a_graph(call, reps):
    """Microseconds of a call, the least of some replays."""
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for _ in range(reps):
            call()
    best = float("inf")
    for _ in range(6):
        a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        a.record()
        graph.replay()
        b.record()
        b.synchronize()
        best = min(best, a.elapsed_time(b) / reps * 1e3)
    return best


@pytest.mark.parametrize("b", [4096, 65536])
def test_padding_takes_no_longer_than_events(b):
    """Half of the events padding, beside distinct rows and rows that come again: less work than without. (With
    padding looked up as a row this took 2.5 and 5 times as long for 4096, 26 and 32 times for 65,536.)"""
    dev = _dev()
    gen = torch.Generator(device=dev).manual_seed(b)
    v, d = 200000, 128
    state = torch.randn(v, d, device=dev, generator=gen)
    x, f = (torch.randn(b, d, device=dev, generator=gen).bfloat16() for _ in range(2))
    distinct = torch.randperm(v, device=dev, generator=gen)[:b]
    again = distinct[torch.randint(0, b // 2, (b,), device=dev, generator=gen)]
    half = torch.rand(b, device=dev, generator=gen) < 0.5
    for rows in (distinct, again):
        with_padding = torch.where(half, -1, rows)
        full, padded = (_in_a_graph(lambda r=r: mips.gated_step(x, f, state, r), 5) for r in (rows, with_padding))
        print(f"b={b}: {full:.1f} us, half of them padding {padded:.1f} us", flush=True)
        assert padded <= 1.5 * full
