"""What the training operators' Python calls check and lay out before a kernel reads it."""
import dataclasses

import numpy as np
import pytest
import torch

import exact_inner_product_amd as mips
from tests.test_gpu_logprobs import grid

pytestmark = pytest.mark.gpu


def _dev():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    return torch.device("cuda:0")


def softmax_call(dev, dtype="bf16", b=20, n=100, d=32):
    rng = np.random.default_rng(0)
    q, items = grid(rng, b, d, dtype).to(dev), grid(rng, n, d, dtype).to(dev)
    ids = torch.from_numpy(rng.integers(0, n, (b, 2))).to(dev)
    gl = torch.from_numpy(rng.standard_normal((b, 2)).astype(np.float32)).to(dev)
    gh = torch.from_numpy(rng.standard_normal(b).astype(np.float32)).to(dev)
    return q, items, ids, gl, gh, mips.item_logprobs(q, items, ids, scale=3.0)


def test_strided_results_of_the_forward_call():
    """The log-sum-exp and the entropy as columns of one tensor, and as every second row of another."""
    dev = _dev()
    q, items, ids, gl, gh, f = softmax_call(dev)
    want = mips.item_logprobs_backward(gl, q, items, ids, f, scale=3.0, grad_entropy=gh)
    plain = mips.item_logprobs_backward(gl, q, items, ids, f, scale=3.0)
    both = torch.stack([f.logsumexp, f.entropy], 1)
    wide = torch.full((2, 40), 7.0, device=dev)
    wide[0, ::2], wide[1, ::2] = f.logsumexp, f.entropy
    for lse, ent in ((both[:, 0], both[:, 1]), (wide[0, ::2], wide[1, ::2])):
        g = dataclasses.replace(f, logsumexp=lse, entropy=ent)
        got = mips.item_logprobs_backward(gl, q, items, ids, g, scale=3.0, grad_entropy=gh)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        got = mips.item_logprobs_backward(gl, q, items, ids, g, scale=3.0)
        assert torch.equal(got[0], plain[0]) and torch.equal(got[1], plain[1])


def test_an_entropy_that_does_not_fit_is_refused():
    dev = _dev()
    q, items, ids, gl, gh, f = softmax_call(dev)
    for bad in (f.entropy[:-1], f.entropy[:, None], f.entropy.bfloat16(), f.entropy.double(), f.entropy.cpu()):
        g = dataclasses.replace(f, entropy=bad)
        with pytest.raises(ValueError):
            mips.item_logprobs_backward(gl, q, items, ids, g, scale=3.0, grad_entropy=gh)
        mips.item_logprobs_backward(gl, q, items, ids, g, scale=3.0)  # not used, not looked at


def test_a_workspace_on_the_host_is_refused():
    dev = _dev()
    q, items, ids, gl, _, f = softmax_call(dev)
    host = torch.empty(1 << 24, dtype=torch.uint8)
    calls = (lambda ws: mips.item_logprobs(q, items, ids, workspace=ws),
             lambda ws: mips.item_logprobs(q, items, ids, alternatives=3, workspace=ws),
             lambda ws: mips.item_logprobs_backward(gl, q, items, ids, f, workspace=ws),
             lambda ws: mips.embedding_grad(torch.zeros(20, 2, 8, device=dev), ids, 100, workspace=ws),
             lambda ws: mips.clip_grad_norm([q], 1.0, workspace=ws))
    for call in calls:
        with pytest.raises(ValueError):
            call(host)
        call(host.to(dev))


def test_autograd_notices_what_is_written_in_place():
    """As after torch's own in-place operations: a backward pass that saved the tensor refuses."""
    dev = _dev()

    def refused(write, rg=torch.ones(30, 8, device=dev)):
        t = rg.clone().requires_grad_()
        x = t * 1.0
        y = (x * x).sum()  # saves x
        write(x.detach())
        with pytest.raises(RuntimeError, match="inplace operation"):
            y.backward()

    ids = torch.zeros(4, dtype=torch.int32, device=dev)
    grad = torch.ones(4, 8, device=dev)
    refused(lambda x: mips.clip_grad_norm([x], 1.0))
    refused(lambda x: mips.clip_grad_norm([torch.ones_like(x)], 1.0, out=[x]))
    refused(lambda x: mips.embedding_grad(grad, ids, 30, out=x))
    refused(lambda x: mips.embedding_grad(grad, ids, 30, out=x, accumulate=True))
    # what is only read stays as it was
    x = torch.ones(30, 8, device=dev)
    version = x._version
    mips.clip_grad_norm([x], 1.0, out=[torch.empty_like(x)])
    mips.embedding_lookup(x, ids)
    mips.embedding_grad(x, torch.zeros(30, dtype=torch.int32, device=dev), 5)
    assert x._version == version
