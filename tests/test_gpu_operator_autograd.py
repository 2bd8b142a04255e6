"""The rotary and cross-attention calls record no autograd graph: an input that
asks for a gradient is worth a warning, and a torch.autograd.Function around the
calls trains."""
import warnings

import pytest
import torch

import context_attention_partial_gb300 as cp
import plain_operators as plain

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def inputs(dtype=torch.float32):
    g = torch.Generator("cpu").manual_seed(90)
    q, k, v, dout = (torch.randn(2, h, s, 64, generator=g).to(dtype).to(DEV)
                     for h, s in ((4, 30), (2, 50), (2, 50), (4, 30)))
    return q, k, v, dout, torch.rand(30, 1, generator=g).to(DEV) * 20


def calls(q, k, v, dout, pos):
    yield lambda: cp.rotary(q, pos, (64,))
    yield lambda: cp.cross_attention(q, k, v)
    with torch.no_grad():
        out, lse = cp.cross_attention(q, k, v)
    yield lambda: cp.cross_attention_backward(q, k, v, out, lse, dout)


@pytest.mark.parametrize("which", [0, 1, 2])
def test_an_input_that_asks_for_a_gradient_is_warned_of(which):
    q, k, v, dout, pos = inputs()
    plain_calls, asking = list(calls(q, k, v, dout, pos)), list(calls(q.clone().requires_grad_(), k, v, dout, pos))
    with warnings.catch_warnings():
        warnings.simplefilter("error")
        want = plain_calls[which]()
        with torch.no_grad():
            asking[which]()
    with pytest.warns(UserWarning, match="no autograd graph") as seen:
        got = asking[which]()
    assert seen[0].filename.endswith("test_gpu_operator_autograd.py")
    for a, b in zip(got if isinstance(got, tuple) else [got], want if isinstance(want, tuple) else [want]):
        assert torch.equal(a, b) and not a.requires_grad
    with warnings.catch_warnings():
        warnings.simplefilter("error")
        with pytest.raises(UserWarning):
            asking[which]()


class Block(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, pos):
        rq = cp.rotary(q, pos, (64,))
        out, lse = cp.cross_attention(rq, k, v)
        ctx.save_for_backward(rq, k, v, out, lse, pos)
        return out

    @staticmethod
    def backward(ctx, dout):
        rq, k, v, out, lse, pos = ctx.saved_tensors
        drq, dk, dv = cp.cross_attention_backward(rq, k, v, out, lse, dout)
        return cp.rotary(drq, pos, (64,), inverse=True), dk, dv, None


def test_an_autograd_function_around_the_calls():
    q, k, v, _, pos = inputs()
    leaves = [t.clone().requires_grad_() for t in (q, k, v)]
    with warnings.catch_warnings():
        warnings.simplefilter("error")
        Block.apply(*leaves, pos).sum().backward()
    rq = cp.rotary(q, pos, (64,))
    want = plain.cross(rq, k, v, dout=torch.ones_like(q))
    for name, leaf in (("dk", leaves[1]), ("dv", leaves[2])):
        assert plain.worst(leaf.grad, *want[name]) <= 1.0
    # dq turned back: orthogonal, so a pair's error is at most the sum of its members'
    value, tol = want["dq"]
    turned, mag = plain.rotary(value.float(), pos, (64,), inverse=True)
    pair = lambda t: t.unflatten(-1, (32, 2)).sum(-1, keepdim=True).expand(*t.shape[:-1], 32, 2).flatten(-2)
    limit = pair(tol) + plain.rotary_tolerance(turned, mag, torch.float32) + 2.0 ** -24 * pair(value.abs())
    assert plain.worst(leaves[0].grad, turned, limit) <= 1.0


def test_readme_blocks_run_as_they_stand():
    """The README's Python blocks, with tensors of the kind it names."""
    import os
    import re
    with open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "README.md")) as f:
        blocks = re.findall(r"```python\n(.*?)```", f.read(), re.S)
    assert len(blocks) >= 2
    g = torch.Generator("cpu").manual_seed(91)
    bf = lambda h, s: torch.randn(2, h, s, 128, generator=g).bfloat16().to(DEV)
    have = dict(cp=cp, q=bf(4, 90), k=bf(4, 90), v=bf(4, 90), text_k=bf(2, 77), text_v=bf(2, 77), dy=bf(4, 90),
                positions=torch.rand(90, 3, generator=g).to(DEV) * 30, n=torch.tensor([77, 20], dtype=torch.int32, device=DEV))
    for block in blocks:
        names = dict(have)
        exec(block, names)
        assert names["y"].shape == have["q"].shape and torch.isfinite(names["y"].float()).all()
        if "dq" in names:
            want = plain.cross(names["rq"], names["text_k"], names["text_v"], (77, 20), dout=names["dy"])
            for name, got in (("out", names["y"]), ("lse", names["lse"]), ("dq", names["drq"]), ("dk", names["dk"]),
                              ("dv", names["dv"])):
                assert plain.worst(got, *want[name]) <= 1.0
            turned, mag = plain.rotary(names["drq"], names["positions"], (16, 56, 56), inverse=True)
            assert plain.worst(names["dq"], turned, plain.rotary_tolerance(turned, mag, torch.bfloat16)) <= 1.0
