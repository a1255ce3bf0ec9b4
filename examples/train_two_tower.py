"""A small two-tower retrieval model trained, indexed and searched on one GPU.

The toy world of "Two-tower retrieval" (mhtirogla.ai): 8 groups of 50 items; a user likes one
group, has a history in it and clicks another of its items, popular ones more often. Items have
one embedding table, which the user side shares (a user is the mean of the history's rows).
Each step is

    embedding_lookup -> mean -> item_logprobs (in-batch softmax with the logQ correction)
    -> item_logprobs_backward -> embedding_grad, added to the item side's gradient
    -> clip_grad_norm -> a plain gradient step.

Afterwards the table is packed into an index, users are searched, and the same softmax over the
index gives the probability of their next item and its most likely alternatives.

With --encoder recurrence the user is what a gated recurrence makes of the history instead,

    embedding -> dropout -> gated_scan -> pool_normalize -> item_logprobs,

trained through the differentiable functions. Afterwards new users are encoded and searched, and their states
followed event by event with gated_step, as a server has them.

    python3 examples/train_two_tower.py [--steps 300] [--dtype f32|bf16] [--encoder mean|recurrence]
"""
import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import exact_inner_product_amd as mips  # noqa: E402
from exact_inner_product_amd import autograd as mag  # noqa: E402

GROUPS, PER, D, HISTORY, TAU = 8, 50, 16, 5, 0.1
N = GROUPS * PER


def sample(gen, b, device):
    """(history [b, HISTORY], clicked item [b]): items of one group, rank r with weight 1 / (r + 1)."""
    weight = 1.0 / torch.arange(1, PER + 1, device=device)
    rank = torch.multinomial(weight, b * (HISTORY + 1), replacement=True, generator=gen).view(b, HISTORY + 1)
    group = torch.randint(0, GROUPS, (b, 1), generator=gen, device=device)
    items = (rank * GROUPS + group).to(torch.int32)
    return items[:, :HISTORY].contiguous(), items[:, HISTORY].contiguous()


def train(steps=300, b=128, dtype="f32", seed=0, device="cuda:0", log=print):
    """(table, losses): the trained item table and the loss of every step."""
    dt = torch.float32 if dtype == "f32" else torch.bfloat16
    gen = torch.Generator(device=device)
    gen.manual_seed(seed)
    table = torch.randn(N, D, generator=gen, device=device) * 0.1
    weight = (1.0 / torch.arange(1, PER + 1, device=device)).repeat_interleave(GROUPS)
    log_q = torch.log(weight / weight.sum())
    targets = torch.arange(b, device=device, dtype=torch.int32)[:, None]
    losses = []
    for step in range(steps):
        history, clicked = sample(gen, b, device)
        rows = table.to(dt)
        users = mips.embedding_lookup(rows, history).float().mean(1).to(dt)
        items = mips.embedding_lookup(rows, clicked)          # in-batch: every user's item is a candidate
        bias = -log_q[clicked.long()]
        f = mips.item_logprobs(users, items, targets, scale=1 / TAU, bias=bias, entropy=False)
        losses.append(-f.logprobs.mean())
        grad = torch.full((b, 1), -1.0 / b, device=device)
        d_users, d_items, _ = mips.item_logprobs_backward(grad, users, items, targets, f, scale=1 / TAU, bias=bias)
        # the table's gradient: the items' rows, and each user's gradient for its history's rows
        d_table = mips.embedding_grad(d_items, clicked, N, out=torch.empty(N, D, device=device))
        d_history = (d_users / HISTORY)[:, None, :].expand(b, HISTORY, D)
        mips.embedding_grad(d_history.contiguous(), history, N, out=d_table, accumulate=True)
        norm, _ = mips.clip_grad_norm([d_table], 1.0)
        table -= 0.5 * d_table
        if log and (step + 1) % 100 == 0:
            log(f"step {step + 1}: loss {float(losses[-1]):.3f}, gradient norm {float(norm):.3f}")
    return table, [float(x) for x in losses]


def evaluate(table, users=256, seed=1, dtype="f32"):
    """(share of the 10 best items that lie in the user's group, mean probability of the clicked
    item, mean entropy in nats)."""
    device = table.device
    gen = torch.Generator(device=device)
    gen.manual_seed(seed)
    history, clicked = sample(gen, users, device)
    corpus = mips.prepare_corpus(table.contiguous(), dtype)
    q = mips.l2_normalize(mips.embedding_lookup(table, history).mean(1), dtype)
    _, best = mips.topk(q, corpus, 10)
    f = mips.item_logprobs(q, corpus, clicked[:, None], scale=1 / TAU, alternatives=10)
    assert torch.equal(f.alt_ids, best)  # the alternatives are the search's results
    group = (history[:, :1] % GROUPS)
    return (float((best % GROUPS == group).float().mean()), float(f.logprobs.exp().mean()),
            float(f.entropy.mean()))


def encode(table, weight, bias, history, lengths, drop=0.0, seed=0, step=0):
    """Unit vectors [b, D] of the users whose first `lengths` events are in history [b, HISTORY]."""
    events = mag.dropout(mag.embedding(table, history), drop, seed, step)
    states, _ = mag.gated_scan(events, torch.nn.functional.linear(events, weight, bias), lengths=lengths)
    return mag.pool_normalize(states, lengths=lengths)


def train_encoder(steps=300, b=128, dtype="f32", seed=0, device="cuda:0", log=print):
    """((table, gates' weight and bias), losses) with a recurrence on the user side."""
    dt = torch.float32 if dtype == "f32" else torch.bfloat16
    gen = torch.Generator(device=device)
    gen.manual_seed(seed)
    params = [torch.randn(N, D, generator=gen, device=device) * 0.1, torch.randn(D, D, generator=gen, device=device) * 0.1,
              torch.zeros(D, device=device)]
    weight = (1.0 / torch.arange(1, PER + 1, device=device)).repeat_interleave(GROUPS)
    log_q = torch.log(weight / weight.sum())
    targets = torch.arange(b, device=device, dtype=torch.int32)[:, None]
    losses = []
    for step in range(steps):
        history, clicked = sample(gen, b, device)
        lengths = torch.randint(1, HISTORY + 1, (b,), generator=gen, device=device)
        leaves = [p.to(dt).detach().requires_grad_() for p in params]
        users = encode(*leaves, history, lengths, drop=0.1, seed=seed, step=step)
        logprobs, _ = mag.item_logprobs(users, mag.embedding(leaves[0], clicked), targets, scale=1 / TAU,
                                        bias=-log_q[clicked.long()])
        loss = -logprobs.mean()
        grads = [g.float() for g in torch.autograd.grad(loss, leaves)]
        norm, _ = mips.clip_grad_norm(grads, 1.0)
        for p, g in zip(params, grads):
            p -= 0.5 * g
        losses.append(loss.detach())
        if log and (step + 1) % 100 == 0:
            log(f"step {step + 1}: loss {float(losses[-1]):.3f}, gradient norm {float(norm):.3f}")
    return params, [float(x) for x in losses]


def follow(table, weight, bias, history, lengths):
    """The users' states [b, D] after their events, taken one at a time as a server sees them."""
    b = history.shape[0]
    states = torch.zeros(b, D, device=table.device)
    users = torch.arange(b, device=table.device)
    for k in range(HISTORY):
        events = mips.embedding_lookup(table, history[:, k].contiguous())
        # a user without a k-th event is no row of the table: skipped
        mips.gated_step(events, torch.nn.functional.linear(events, weight, bias), states, torch.where(k < lengths, users, -1))
    return states


def serve(table, weight, bias, users=256, seed=1):
    """(share of the 10 best items that lie in the user's group, largest difference between a state from single
    events and that of the whole history) of new users with histories of 1 to HISTORY events."""
    device = table.device
    gen = torch.Generator(device=device)
    gen.manual_seed(seed)
    history, _ = sample(gen, users, device)
    lengths = torch.randint(1, HISTORY + 1, (users,), generator=gen, device=device)
    with torch.no_grad():
        q = encode(table, weight, bias, history, lengths)
        _, best = mips.topk(q, mips.prepare_corpus(table.float(), "f32" if table.dtype == torch.float32 else "bf16"), 10)
        events = mips.embedding_lookup(table, history)
        gates = torch.nn.functional.linear(events, weight, bias)
        whole = mips.gated_scan(events, gates, lengths=lengths, states=False, carries=False).last
        apart = (follow(table, weight, bias, history, lengths) - whole).abs().max()
    return float((best % GROUPS == history[:, :1] % GROUPS).float().mean()), float(apart)


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--steps", type=int, default=300)
    ap.add_argument("--dtype", choices=("f32", "bf16"), default="f32")
    ap.add_argument("--encoder", choices=("mean", "recurrence"), default="mean")
    a = ap.parse_args()
    if a.encoder == "recurrence":
        params, losses = train_encoder(a.steps, dtype=a.dtype)
        hit, apart = serve(*(p.to(torch.float32 if a.dtype == "f32" else torch.bfloat16) for p in params))
        print(f"loss {losses[0]:.3f} -> {losses[-1]:.3f} (log of the batch: {math.log(128):.3f}); of the 10 best items "
              f"{100 * hit:.1f}% lie in the user's group; states followed event by event are within {apart:.1e} of the histories'")
        sys.exit()
    table, losses = train(a.steps, dtype=a.dtype)
    hit, prob, entropy = evaluate(table, dtype=a.dtype)
    print(f"loss {losses[0]:.3f} -> {losses[-1]:.3f} (log of the batch: {math.log(128):.3f}); of the 10 best items "
          f"{hit:.1%} in the user's group; clicked item's probability {prob:.4f}; entropy {entropy:.2f} nats")
