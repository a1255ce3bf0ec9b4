"""The operators over histories as a program uses them: one after another, under autograd, on several
streams, in captured graphs, with workspaces of the caller, and at sizes past 32 bits."""
import importlib.util
import math
import os
import re
import runpy

import numpy as np
import pytest
import torch

import exact_inner_product_amd as mips
from exact_inner_product_amd import autograd as mag
from tests import histories_check as hc
from tests.histories_check import U
from tests.test_gpu_scan import flat, make, place, run

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _dev():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    return torch.device("cuda:0")


def plain_scan(x, f, g, lengths, initial):
    """The recurrence by torch in 64 bits over padded rows; (states, last)."""
    a, b = torch.sigmoid(f), torch.sigmoid(-f if g is None else g)
    h = torch.zeros_like(x[:, 0]) if initial is None else initial
    out = []
    for r in range(x.shape[1]):
        live = (r < lengths)[:, None]
        h = torch.where(live, a[:, r] * h + b[:, r] * x[:, r], h)
        out.append(torch.where(live, h, torch.zeros_like(h)))
    return torch.stack(out, 1), h


@pytest.mark.parametrize("layout", ["padded", "packed"])
def test_a_user_tower(layout):
    """lookup -> dropout -> recurrence -> dropout with residual -> pooling -> softmax loss, with the
    gradients of the table, the gates' weights and the initial state, against torch in 64 bits with
    the same dropped elements.

    All is in binary32. A row of the recurrence loses at most (2 * 8 + 12 + 32) u = 60 u of its terms
    (gates below 8 in size), 20 rows 7e-5, its gradient's recurrence as much again; the softmax
    loss' own tolerance is 1e-5; pooling and dropout add a few u: below 2e-4 of the largest value."""
    dev = _dev()
    gen = torch.Generator().manual_seed(3)
    b, t, d, n, p, seed = 24, 20, 32, 50, 0.25, 11
    table = torch.randn(n, d, generator=gen)
    weight = torch.randn(d, d, generator=gen) * 0.1
    initial = torch.randn(b, d, generator=gen)
    history = torch.randint(0, n, (b, t), generator=gen)
    lengths = torch.randint(0, t + 1, (b,), generator=gen)
    lengths[:3] = torch.tensor([0, 1, t])
    targets = torch.randint(0, n, (b, 1), generator=gen)
    live = torch.arange(t)[None] < lengths[:, None]
    offsets = torch.cat([torch.zeros(1, dtype=torch.int64), lengths.cumsum(0)])

    ids = history if layout == "padded" else history[live]
    args = {"lengths": lengths.to(dev)} if layout == "padded" else {"offsets": offsets.to(dev)}
    leaves = [v.to(dev).requires_grad_() for v in (table, weight, initial)]
    T, W, I = leaves  # noqa: E741
    e = mag.dropout(mag.embedding(T, ids.to(dev)), p, seed, 0)
    h, last = mag.gated_scan(e, e @ W, initial=I, **args)
    y = mag.dropout(h, p, seed, 1, residual=e)
    users = mag.pool_normalize(y, **args)
    lp, _ = mag.item_logprobs(users, T, targets.to(dev), scale=4.0)
    loss = -lp.mean() + 0.1 * (last * last).mean()
    loss.backward()

    masks = [mips.dropout(torch.ones(ids.shape + (d,), device=dev), p, seed, k).cpu().double() for k in (0, 1)]
    if layout == "packed":  # back into rows of t, padding dropped
        full = [torch.zeros(b, t, d, dtype=torch.float64) for _ in masks]
        for f, m in zip(full, masks):
            f[live] = m
        masks = full
    T2, W2, I2 = (v.double().requires_grad_() for v in (table, weight, initial))
    e2 = T2[history] * masks[0]
    h2, last2 = plain_scan(e2, e2 @ W2, None, lengths, I2)
    y2 = torch.where(live[:, :, None], h2 * masks[1] + e2, 0.0)
    mean = y2.sum(1) / lengths.clamp(min=1)[:, None]
    users2 = mean / mean.square().sum(1, keepdim=True).clamp(min=1e-12).sqrt()
    loss2 = (-torch.log_softmax((users2 @ T2.T) * 4.0, 1).gather(1, targets).mean() + 0.1 * (last2 * last2).mean())
    loss2.backward()
    loss, loss2 = loss.detach(), loss2.detach()
    assert abs(float(loss) - float(loss2)) <= 2e-4 * abs(float(loss2))
    for name, got, want in (("table", T, T2), ("weight", W, W2), ("initial", I, I2)):
        err = float((got.grad.double().cpu() - want.grad).abs().max() / want.grad.abs().max())
        assert err <= 2e-4, (name, err)


@pytest.mark.parametrize("gate", [False, True])
@pytest.mark.parametrize("layout,b,t,d", [("dense", 2, 300, 5), ("padded", 4, 37, 8), ("packed", 5, 41, 3)])
def test_scan_gradient_against_differences(layout, b, t, d, gate):
    """The gradient along directions of all inputs together, against central differences of the
    64-bit plain form. With steps e and 2e their truncation errors are C e^2 and 4 C e^2 up to terms in
    e^4: three times their difference is nine times the former; at e = 1e-4 the differences' own
    rounding is below 2^-53 / 1e-4 = 1.2e-12 of the sum of |terms|."""
    dev = _dev()
    c = make(layout, b, t, d, "f32", gate, True, seed=5)
    f, grads = run(place(c, dev), dev)
    rows = [flat(c[k]) for k in ("x", "forget", "gate")] + [c["initial"].double().numpy()]
    gs, gl = flat(c["gs"]), c["gl"].double().numpy()
    bounds = [w[1] for w in hc.scan_grad(*rows[:3], c["seqs"], rows[3], gs, gl) if w is not None]
    got = [flat(g) if g.dim() > 2 or layout == "packed" else g.double().numpy() for g in
           (v.cpu() for v in grads if v is not None)]
    if gate is False:
        rows.pop(2)
    live = np.zeros(rows[0].shape[0], dtype=bool)
    for lo, hi in c["seqs"]:
        live[lo:hi] = True

    def loss(inputs):
        x, fo, ga, i = (inputs[0], inputs[1], inputs[2] if gate else None, inputs[-1])
        h, _, last, _ = hc.scan(x, fo, ga, c["seqs"], i)
        return float((h * gs)[live].sum() + (last * gl).sum()), float(np.abs(h * gs).sum() + np.abs(last * gl).sum())

    rng = np.random.default_rng(1)
    for _ in range(6):
        v = [rng.standard_normal(r.shape) for r in rows]
        at = lambda e: loss([r + e * w for r, w in zip(rows, v)])  # noqa: E731
        d1, d2 = ((at(e)[0] - at(-e)[0]) / (2 * e) for e in (1e-4, 2e-4))
        want = sum(float((g * w).sum()) for g, w in zip(got, v))
        room = sum(float((e * np.abs(w)).sum()) for e, w in zip(bounds, v))
        assert abs(want - d1) <= room + 3 * abs(d2 - d1) + 1e-10 * at(0)[1], (want, d1, room)


@pytest.mark.parametrize("normalize", [True, False])
def test_pool_gradient_against_differences(normalize):
    """As above. The gradient's terms are at most |w| / norm / rows, its rounding 64 u of them: the mean's
    (rows + 3) u, the norm's and the product's (d + 8) u each."""
    dev = _dev()
    rng = np.random.default_rng(2)
    b, t, d = 5, 13, 9
    x = rng.standard_normal((b, t, d)).astype(np.float32)
    lengths = np.array([0, 1, 13, 7, 20])
    w = rng.standard_normal((b, d)).astype(np.float32)
    xt = torch.from_numpy(x).to(dev).requires_grad_()
    y = mag.pool_normalize(xt, lengths=torch.from_numpy(lengths).to(dev), normalize=normalize)
    (y * torch.from_numpy(w).to(dev)).sum().backward()
    got = xt.grad.double().cpu().numpy()

    def loss(z):
        total = 0.0
        for s in range(b):
            k = min(lengths[s], t)
            m = z[s, :k].sum(0) / max(k, 1)
            total += float((m * w[s]).sum() / (math.sqrt(max((m * m).sum(), 1e-12)) if normalize else 1.0))
        return total

    z = x.astype(np.float64)
    assert all(np.linalg.norm(z[s, :min(n, t)].mean(0)) > 0.5 for s, n in enumerate(lengths) if n)
    for _ in range(6):
        v = rng.standard_normal(z.shape)
        d1, d2 = ((loss(z + e * v) - loss(z - e * v)) / (2 * e) for e in (1e-4, 2e-4))
        room = 64 * U * float((np.linalg.norm(v, axis=2) * np.linalg.norm(w, axis=1)[:, None]).sum() / 0.5)
        assert abs(float((got * v).sum()) - d1) <= room + 3 * abs(d2 - d1) + 1e-9, normalize


def test_functions_without_a_gradient():
    """Results that nothing uses, inputs that need none, and a second-order gradient."""
    dev = _dev()
    x = torch.randn(3, 50, 16, device=dev)
    f = torch.randn(3, 50, 16, device=dev, requires_grad=True)
    h, last = mag.gated_scan(x, f, states=False)
    assert h is None
    (g,) = torch.autograd.grad(last.sum(), f, create_graph=True)
    with pytest.raises(RuntimeError):
        g.sum().backward()
    h, last = mag.gated_scan(x, f)
    (g,) = torch.autograd.grad(h.sum(), f)
    want = mips.gated_scan_backward(torch.ones_like(x), None, x, f.detach(), None, mips.gated_scan(x, f.detach()))
    assert torch.equal(g, want[1])
    with torch.no_grad():
        assert not mag.gated_scan(x, f)[0].requires_grad
    r = torch.randn_like(x).requires_grad_()
    y = mag.dropout(x, 0.5, 1, residual=r)
    y.sum().backward()
    assert torch.equal(r.grad, torch.ones_like(r))
    x = x.clone().requires_grad_()
    h, _ = mag.gated_scan(x * 1.0, f)
    with torch.no_grad():
        f.add_(1.0)
    with pytest.raises(RuntimeError, match="inplace operation"):
        h.sum().backward()


def test_broadcast_inputs():
    """One row of gates for all rows and one history for all users: their gradients are sums."""
    dev = _dev()
    b, t, d = 6, 90, 24
    x, g = torch.randn(1, t, d, device=dev), torch.randn(b, t, d, device=dev)
    w = torch.randn(d, device=dev)
    leaves = [v.clone().requires_grad_() for v in (x, w)]
    h, _ = mag.gated_scan(leaves[0].expand(b, t, d), leaves[1].expand(b, t, d))
    h.backward(g)
    f = mips.gated_scan(x.expand(b, t, d), w.expand(b, t, d))
    full = mips.gated_scan_backward(g, None, x.expand(b, t, d), w.expand(b, t, d), None, f)
    for leaf, v, over in ((leaves[0], full[0], (0,)), (leaves[1], full[1], (0, 1))):
        want = v.double().sum(over)
        room = b * t * U * v.double().abs().sum(over)  # the order of the sum is torch's
        assert bool(((leaf.grad.double().reshape(want.shape) - want).abs() <= room).all())


def test_the_counter_may_advance_before_the_backward_pass():
    dev = _dev()
    x = torch.randn(1000, device=dev, requires_grad=True)
    counter = torch.tensor([5], device=dev)
    y = mag.dropout(x, 0.5, 3, 1, counter=counter)
    counter += 1
    y.sum().backward()
    assert torch.equal(x.grad != 0, y != 0)
    assert torch.equal(x.grad, mips.dropout(torch.ones_like(x), 0.5, 3, 6))


def calls(c, state, rows, counter):
    """One of every operator on the inputs in c; the results."""
    n = c["x"].shape[-1]
    args = {k: c[k] for k in ("lengths", "offsets")}
    x = mips.dropout(c["x"], 0.3, 7, 2, counter=counter)
    f = mips.gated_scan(x, c["forget"], c["gate"], initial=c["initial"], **args)
    p = mips.pool_normalize(f.states, **args)
    dh = mips.pool_normalize_backward(p.vectors, f.states.shape, p, **args)
    g = mips.gated_scan_backward(dh, f.last, x, c["forget"], c["gate"], f, initial=c["initial"], **args)
    flat_ = lambda v: v.reshape(-1, n)[:rows.shape[0]]  # noqa: E731
    out = mips.gated_step(flat_(x), flat_(c["forget"]), state, rows)
    return [x, f.states, f.last, p.vectors, dh, out, state] + [v for v in g if v is not None]


@pytest.mark.parametrize("layout,b,t,d,dtype", [("dense", 3, 40, 64, "f32"), ("padded", 3, 2000, 256, "bf16"),
                                                ("packed", 5, 900, 100, "bf16"), ("packed", 1, 20000, 32, "f32")])
def test_captured_and_replayed(layout, b, t, d, dtype):
    """All operators in one graph, replayed with new inputs and a counter that the graph advances, with
    eager calls of the same sizes and others between the replays."""
    dev = _dev()
    cases = [place(make(layout, b, t, d, dtype, True, True, seed=s), dev) for s in (0, 1, 2)]
    shape = cases[0]["x"].shape
    if layout == "packed":  # the same number of rows in each
        k = min(c["x"].shape[0] for c in cases)
        for c in cases:
            c.update({n: c[n][:k].contiguous() for n in ("x", "forget", "gate", "gs")})
        shape = cases[0]["x"].shape
    rows = torch.randint(0, 40, (30,), device=dev)
    tensors = ("x", "forget", "gate", "initial", "lengths", "offsets")
    held = {k: (None if cases[0][k] is None else cases[0][k].clone()) for k in tensors}
    state, counter = torch.zeros(40, d, device=dev), torch.zeros(1, dtype=torch.int64, device=dev)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        calls(held, state.clone(), rows, counter)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = calls(held, state, rows, counter)
        counter += 1
    state.zero_()
    counter.zero_()
    other = torch.zeros(40, d, device=dev)
    for k in range(5):
        c = cases[k % 3]
        for n in tensors:
            if held[n] is not None:
                held[n].copy_(c[n])
        want = calls(c, other, rows, torch.tensor([k], device=dev))
        torch.cuda.synchronize()
        graph.replay()
        mips.gated_scan(torch.ones(2, 3000, 64, device=dev), torch.ones(2, 3000, 64, device=dev))
        torch.cuda.synchronize()
        for i, (a, w) in enumerate(zip(got, want)):
            assert a.shape == w.shape and torch.equal(a, w), (k, i, shape)


def test_a_captured_training_step():
    """Forward and backward through autograd in one graph, on leaves of the graph alone."""
    dev = _dev()
    xs = [[torch.randn(4, 700, 64, device=dev) for _ in range(2)] for _ in range(3)]
    lengths = torch.tensor([700, 0, 13, 450], device=dev)
    grad = torch.randn(4, 64, device=dev)

    def step(x, f):
        x, f = x.clone().requires_grad_(), f.clone().requires_grad_()
        h, _ = mag.gated_scan(x, f, lengths=lengths)
        y = mag.pool_normalize(mag.dropout(h, 0.1, 3, residual=x), lengths=lengths)
        return torch.autograd.grad(y, [x, f], grad)

    want = [step(*v) for v in xs]
    held = [torch.zeros_like(v) for v in xs[0]]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(*held)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(*held)
    for k in range(5):
        for h, v in zip(held, xs[k % 3]):
            h.copy_(v)
        graph.replay()
        step(*xs[0])
        torch.cuda.synchronize()
        assert all(torch.equal(g, w) for g, w in zip(got, want[k % 3])), k


def test_two_calls_at_once():
    """Long recurrences on two streams, each with its own workspace, many times over."""
    dev = _dev()
    streams = [torch.cuda.Stream() for _ in range(2)]
    cases = [place(make("dense", 2, 5000, 256, "bf16", False, True, seed=s), dev) for s in range(2)]
    want = [run(c, dev) for c in cases]
    torch.cuda.synchronize()
    for _ in range(10):
        got = []
        for s, c in zip(streams, cases):
            with torch.cuda.stream(s):
                got.append(run(c, dev))
        torch.cuda.synchronize()
        for (f, g), (fw, gw) in zip(got, want):
            assert torch.equal(f.states, fw.states) and torch.equal(f.last, fw.last)
            assert all(torch.equal(a, w) for a, w in zip(g, gw) if w is not None)


def test_workspaces_of_the_caller():
    """A workspace that holds anything gives the same bits call after call; one on the host or too
    small a one is refused."""
    dev = _dev()
    c = place(make("packed", 7, 600, 128, "f32", True, True), dev)
    args = dict(offsets=c["offsets"], initial=c["initial"])
    want, wg = run(c, dev)
    ws = torch.randint(0, 256, (1 << 23,), dtype=torch.uint8, device=dev)
    for fill in (None, 0, 255):
        if fill is not None:
            ws.fill_(fill)
        f = mips.gated_scan(c["x"], c["forget"], c["gate"], workspace=ws, **args)
        g = mips.gated_scan_backward(c["gs"], c["gl"], c["x"], c["forget"], c["gate"], f, workspace=ws, **args)
        p = mips.pool_normalize(c["x"], offsets=c["offsets"], workspace=ws)
        assert torch.equal(f.states, want.states) and all(torch.equal(a, b) for a, b in zip(g, wg))
        assert torch.equal(p.vectors, mips.pool_normalize(c["x"], offsets=c["offsets"]).vectors)
    for bad, error in ((ws.cpu(), ValueError), (ws[:256], mips.MipsError), (ws[:1].expand(1 << 23), ValueError)):
        with pytest.raises(error):
            mips.gated_scan(c["x"], c["forget"], c["gate"], workspace=bad, **args)
        with pytest.raises(error):
            mips.gated_scan_backward(c["gs"], c["gl"], c["x"], c["forget"], c["gate"], f, workspace=bad, **args)
    with pytest.raises(ValueError):
        mips.pool_normalize(c["x"], offsets=c["offsets"], workspace=ws.cpu())
    with pytest.raises(ValueError):
        mips.gated_scan(c["x"], c["forget"].cpu(), c["gate"], **args)
    with pytest.raises(ValueError):
        mips.gated_scan(c["x"], c["forget"], c["gate"], offsets=c["offsets"].cpu())
    with pytest.raises(ValueError):
        mips.gated_step(c["x"], c["forget"], torch.zeros(5, 128), torch.zeros(c["x"].shape[0], dtype=torch.int32, device=dev))
    with pytest.raises(ValueError):
        mips.dropout(c["x"], 0.5, 1, counter=torch.zeros(1, dtype=torch.int64))


def test_wide_strides():
    """Packed rows further apart than are used in place, sequences that begin past 32 bits, and rows
    that interleave (time before batch)."""
    dev = _dev()
    big = torch.zeros(9, 600000, device=dev)
    off = torch.tensor([0, 4, 4, 9], device=dev)
    x, f = torch.randn(9, 40, device=dev), torch.randn(9, 40, device=dev)
    big[:, :40], big[:, 100:140] = x, f
    a, w = mips.gated_scan(big[:, :40], big[:, 100:140], offsets=off), mips.gated_scan(x, f, offsets=off)
    assert torch.equal(a.states, w.states) and torch.equal(a.last, w.last)
    assert torch.equal(mips.pool_normalize(big[:, :40], offsets=off).vectors, mips.pool_normalize(x, offsets=off).vectors)
    del big

    room = torch.empty((1 << 32) + 4096, dtype=torch.bfloat16, device=dev)
    far = room.as_strided((2, 6, 64), (1 << 32, 64, 1))
    x, f = torch.randn(2, 6, 64, device=dev).bfloat16(), torch.randn(2, 6, 64, device=dev).bfloat16()
    far.copy_(x)
    g = torch.randn(2, 6, 64, device=dev).bfloat16()
    fa, fw = mips.gated_scan(far, f), mips.gated_scan(x, f)
    assert torch.equal(fa.states, fw.states)
    ga, gw = (mips.gated_scan_backward(g, None, v, f, None, fw) for v in (far, x))
    assert all(torch.equal(p, q) for p, q in zip(ga[:2], gw[:2]))
    assert torch.equal(mips.pool_normalize(far).vectors, mips.pool_normalize(x).vectors)
    del far, room

    tb = torch.randn(300, 5, 2, 64, device=dev)  # time, batch, (x and forget), channels
    x, f = tb[:, :, 0].transpose(0, 1), tb[:, :, 1].transpose(0, 1)
    a, w = mips.gated_scan(x, f), mips.gated_scan(x.contiguous(), f.contiguous())
    assert torch.equal(a.states, w.states) and torch.equal(a.last, w.last)
    assert torch.equal(mips.pool_normalize(x).vectors, mips.pool_normalize(x.contiguous()).vectors)


@pytest.mark.parametrize("layout", ["dense", "packed"])
def test_elements_past_32_bits(layout):
    """A sequence of more than 2^31 elements. A gate of -inf shortly before the end makes the rows behind it a
    short sequence of its own, whose states and gradients a plain loop gives."""
    dev = _dev()
    t, d, k = (1 << 21) + 77, 1024, 9
    x, f = torch.empty((t, d), dtype=torch.bfloat16, device=dev), torch.empty((t, d), dtype=torch.bfloat16, device=dev)
    x.fill_(0.5)
    f.fill_(1.0)
    rng = np.random.default_rng(0)
    tail = lambda m=0.0: torch.from_numpy(rng.standard_normal((k, d)).astype(np.float32) + np.float32(m)).bfloat16()  # noqa: E731
    xt, ft, gt = tail(), tail(1.0), tail()
    ft[0] = -math.inf  # forgets what came before, and takes x whole
    x[-k:], f[-k:] = xt.to(dev), ft.to(dev)
    if layout == "packed":
        args = dict(offsets=torch.tensor([0, t], device=dev))
    else:
        x, f, args = x[None], f[None], {}
    scan = mips.gated_scan(x, f, **args)
    rows = [v.double().numpy() for v in (xt, ft)]
    h, e, last, le = hc.scan(rows[0], rows[1], None, [(0, k)], None)
    got = scan.states.reshape(t, d)[-k:].double().cpu().numpy()
    assert (np.abs(got - h) <= e + 2.0 ** -8 * (np.abs(h) + e)).all()
    assert (np.abs(scan.last.double().cpu().numpy() - last) <= le).all()
    gs = torch.zeros_like(x)
    gs.reshape(t, d)[-k:] = gt.to(dev)
    dx, df, _, _ = mips.gated_scan_backward(gs, None, x, f, None, scan, **args)
    # (row 0's gradient for the gate is D (h - x) a (1 - a) with a = 0, whatever came before)
    for name, out, (want, bound) in zip(("x", "forget"), (dx, df), hc.scan_grad(rows[0], rows[1], None, [(0, k)], None, gt.double().numpy(), None)):
        out = out.reshape(t, d)[-k:].double().cpu().numpy()
        assert (np.abs(out - want) <= bound + 2.0 ** -8 * (np.abs(want) + bound) + 1e-36).all(), name
    assert not bool(dx.reshape(t, d)[:-k].any()) or float(dx.reshape(t, d)[:-k].abs().max()) < 1e-36
    del dx, df, gs, scan, f
    x.reshape(t, d)[:-k] = 0
    m = mips.pool_normalize(x, normalize=False, **args).mean[0].double().cpu().numpy()
    want = rows[0].sum(0) / t
    assert (np.abs(m - want) <= (64 + 4) * U * np.abs(rows[0]).sum(0) / t).all()


def test_example_with_an_encoder():
    """The example with its recurrent user side runs, its gradients are those of torch in 64 bits, and a
    user's state from single events is that of the whole history (tolerances as of the tower above)."""
    dev = _dev()
    spec = importlib.util.spec_from_file_location("train_two_tower", os.path.join(ROOT, "examples", "train_two_tower.py"))
    ex = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ex)
    for dtype in ("f32", "bf16"):
        params, losses = ex.train_encoder(steps=3, dtype=dtype, log=None, device=str(dev))
        assert len(losses) == 3 and all(math.isfinite(v) for v in losses)
        assert all(bool(torch.isfinite(p).all()) for p in params)
    gen = torch.Generator(device=dev)
    gen.manual_seed(4)
    history, clicked = ex.sample(gen, 16, dev)
    lengths = torch.randint(0, ex.HISTORY + 1, (16,), generator=gen, device=dev)
    leaves = [torch.randn(s, generator=gen, device=dev).requires_grad_() for s in ((ex.N, ex.D), (ex.D, ex.D), (ex.D,))]
    users = ex.encode(*leaves, history, lengths)
    (users * users.detach().roll(1, 0)).sum().backward()
    t2, w2, b2 = (v.detach().double().cpu().requires_grad_() for v in leaves)
    e2 = t2[history.long().cpu()]
    h2, last2 = plain_scan(e2, e2 @ w2.T + b2, None, lengths.cpu(), None)
    mean = h2.sum(1) / lengths.cpu().clamp(min=1)[:, None]
    users2 = mean / mean.square().sum(1, keepdim=True).clamp(min=1e-12).sqrt()
    (users2 * users2.detach().roll(1, 0)).sum().backward()
    for got, want in zip(leaves, (t2, w2, b2)):
        assert (got.grad.double().cpu() - want.grad).abs().max() <= 2e-4 * want.grad.abs().max()
    with torch.no_grad():
        states = ex.follow(*leaves, history, lengths)
    assert (states.double().cpu() - last2.detach()).abs().max() <= 1e-4 * last2.abs().max()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_example_serves_what_it_trained(dtype, monkeypatch, capsys):
    """The program itself: it trains, searches for new users and follows them event by event. States are sums
    of b x over at most five events, within (2 * 16 + 12 + 32) u of five of the largest input on either side."""
    _dev()
    path = os.path.join(ROOT, "examples", "train_two_tower.py")
    monkeypatch.setattr("sys.argv", [path, "--encoder", "recurrence", "--steps", "2", "--dtype", dtype])
    with pytest.raises(SystemExit) as end:
        runpy.run_path(path, run_name="__main__")
    assert not end.value.code
    text = capsys.readouterr().out
    found = re.search(r"([\d.]+)% lie in the user's group; states followed event by event are within (\S+) of", text)
    assert found, text
    assert 0 <= float(found[1]) <= 100 and float(found[2]) <= 2 * 76 * U * 5 * 1.0
