"""Multi-axis rotary positions against a plain 64-bit form; tolerances count
roundings (plain_operators.py)."""
import pytest
import torch

import context_attention_partial_gb300 as cp
import plain_operators as plain

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def normal(seed, *shape, dtype=torch.bfloat16):
    g = torch.Generator("cpu").manual_seed(seed)
    return torch.randn(*shape, generator=g).to(dtype).to(DEV)


def grid_positions(t, h, w, start=0):
    g = torch.meshgrid(torch.arange(t), torch.arange(h), torch.arange(w), indexing="ij")
    return (torch.stack(g, -1).reshape(-1, 3) + start).float().to(DEV)


def check(x, y, pos, axes, **kw):
    want, mag = plain.rotary(x, pos, axes, **kw)
    assert plain.worst(y, want, plain.rotary_tolerance(want, mag, x.dtype)) <= 1.0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("interleaved", [True, False])
@pytest.mark.parametrize("B,H,Hk,thw,D,axes", [
    (1, 24, 24, (1, 7, 9), 128, (16, 56, 56)),
    (2, 3, 1, (2, 5, 5), 64, (16, 24, 24)),
    (1, 2, 2, (1, 1, 1), 128, (44, 42, 42)),      # one token
    (3, 4, 2, (4, 3, 3), 64, (22, 22, 20)),
    (2, 1, 1, (3, 1, 7), 128, (2, 4, 6)),         # most features copied
    (1, 2, 1, (2, 2, 9), 256, (64, 96, 96)),
    (1, 3, 2, (1, 4, 5), 24, (8, 8, 8)),
    (1, 5, 2, (1, 3, 3), 8, (2, 2, 2)),
])
def test_rotary_matches_plain(B, H, Hk, thw, D, axes, interleaved, dtype):
    n = thw[0] * thw[1] * thw[2]
    q, k = normal(1, B, H, n, D, dtype=dtype), normal(2, B, Hk, n, D, dtype=dtype)
    pos = grid_positions(*thw, start=3)
    for inverse in (False, True):
        a, b = cp.rotary([q, k], pos, axes, interleaved=interleaved, inverse=inverse)
        check(q, a, pos, axes, interleaved=interleaved, inverse=inverse)
        check(k, b, pos, axes, interleaved=interleaved, inverse=inverse)


@pytest.mark.parametrize("axes,theta", [((128,), 10000.0), ((64, 64), 500000.0), ((32, 32, 32, 32), 100.0)])
@pytest.mark.parametrize("interleaved", [True, False])
def test_rotary_one_to_four_axes_far_and_fractional_positions(axes, theta, interleaved):
    B, S = 2, 37
    x = normal(3, B, 2, S, 128, dtype=torch.float32)
    pos = torch.arange(S, dtype=torch.float32, device=DEV).view(1, S, 1) + torch.tensor(
        [0.25, 9_999_000.0], device=DEV).view(2, 1, 1)
    pos = pos.expand(B, S, len(axes)) * torch.tensor([1.0, -0.5, 2.0, 0.125], device=DEV)[: len(axes)]
    y = cp.rotary(x, pos, axes, theta=theta, interleaved=interleaved)
    check(x, y, pos, axes, theta=theta, interleaved=interleaved)


@pytest.mark.parametrize("interleaved", [True, False])
def test_rotary_layouts_in_place_and_round_trip(interleaved):
    """A [B,S,H,D] tensor as its [B,H,S,D] view, q and k as views of one fused
    projection, in place; features past the axes stay bit for bit."""
    B, S, H, D, axes = 2, 45, 6, 128, (16, 40, 40)
    pos = grid_positions(1, 5, 9)
    qkv = normal(4, B, S, 3, H, D)
    q, k, v = (qkv[:, :, i].transpose(1, 2) for i in range(3))
    want = [cp.rotary(t.contiguous(), pos, axes, interleaved=interleaved) for t in (q, k)]
    away = cp.rotary([q, k], pos, axes, interleaved=interleaved)
    assert away[0].stride()[1] == D                 # a [B,S,H,D] tensor again
    v0, q0 = v.clone(), q.clone()
    got = cp.rotary([q, k], pos, axes, interleaved=interleaved, outs=[q, k])
    for a, b, c in zip(got, want, away):
        assert torch.equal(a, b) and torch.equal(c, b)
    assert torch.equal(v, v0)
    assert torch.equal(q[..., 96:], q0[..., 96:])
    back = cp.rotary(q, pos, axes, interleaved=interleaved, inverse=True)
    # two roundings to bf16, each at most 2^-8 of a turned pair's length
    pair = q0.float().abs().amax(-1, keepdim=True)
    assert float(((back.float() - q0.float()).abs() / (pair * 2 * 2 ** -8 * 1.5)).max()) <= 1.0


def test_rotary_broadcast_positions_and_inputs():
    """Positions and inputs may be expanded views; outputs may not."""
    x = normal(5, 1, 2, 9, 64).expand(3, 2, 9, 64)
    pos = grid_positions(1, 3, 3)
    y = cp.rotary(x, pos.expand(3, 9, 3), (16, 24, 24))
    check(x, y, pos, (16, 24, 24))
    with pytest.raises(cp.CpattnError) as e:
        cp.rotary(x, pos, (16, 24, 24), outs=torch.empty(1, 2, 9, 64, device=DEV, dtype=x.dtype).expand(3, 2, 9, 64))
    assert e.value.name == "CPATTN_ERR_LAYOUT"


@pytest.mark.parametrize("interleaved", [True, False])
def test_rotary_gradient_is_the_inverse_turn(interleaved):
    """d/dx of sum(w y): the inverse turn of w, against differences of the fp32 kernel."""
    B, H, S, D, axes = 1, 2, 5, 64, (16, 24, 24)
    x, w = normal(6, B, H, S, D, dtype=torch.float32), normal(7, B, H, S, D, dtype=torch.float32)
    pos = torch.rand(S, 3, generator=torch.Generator("cpu").manual_seed(8)).to(DEV) * 40
    f = lambda t: (cp.rotary(t, pos, axes, interleaved=interleaved).double() * w.double())
    grad = cp.rotary(w, pos, axes, interleaved=interleaved, inverse=True)
    step = 0.5                                       # (linear: any step)
    for i in range(0, D, 7):
        d = torch.zeros_like(x)
        d[..., i] = step
        num = (f(x + d) - f(x - d)).sum(-1) / (2 * step)
        # fp32 roundings of values up to |x| + step, over the step
        assert float((num - grad[..., i].double()).abs().max()) <= 64 * 2 ** -24 * 16 / step


def test_rotary_canary_and_empty():
    big = torch.full((2, 5, 40, 80), 7.0, device=DEV, dtype=torch.bfloat16)
    y = big[:, 1:4, 3:36, 8:72]
    x = normal(9, 2, 3, 33, 64)
    pos = grid_positions(1, 3, 11)
    cp.rotary(x, pos, (16, 24, 24), outs=y)
    check(x, y, pos, (16, 24, 24))
    mask = torch.ones_like(big, dtype=torch.bool)
    mask[:, 1:4, 3:36, 8:72] = False
    assert torch.all(big[mask] == 7.0)
    assert cp.rotary(x[:, :, :0], pos[:0], (16, 24, 24)).shape == (2, 3, 0, 64)
    a, b = cp.rotary([x, x[:, :0]], pos, (16, 24, 24))     # no key heads on this rank
    check(x, a, pos, (16, 24, 24))
    assert b.numel() == 0


def test_rotary_captured_and_on_another_stream():
    x, pos = normal(10, 1, 4, 33, 128), grid_positions(1, 3, 11)
    axes = (16, 56, 56)
    want = cp.rotary(x, pos, axes)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    y = cp.rotary(x, pos, axes, stream=s)
    s.synchronize()
    assert torch.equal(y, want)
    out = torch.zeros_like(x)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        cp.rotary(x, pos, axes, outs=out)
    x.neg_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, -want)
    assert cp.last_device_status() == 0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("interleaved", [True, False])
def test_rotary_gradient_of_a_sum(interleaved, dtype):
    """The gradient that (w y).sum() sends back is one value for every element."""
    pos = grid_positions(1, 3, 11)
    dy = torch.full((), 0.75, dtype=dtype, device=DEV).expand(2, 3, 33, 64)
    want = cp.rotary(dy.contiguous(), pos, (16, 24, 24), interleaved=interleaved, inverse=True)
    got = cp.rotary(dy, pos, (16, 24, 24), interleaved=interleaved, inverse=True)
    assert got.shape == dy.shape and torch.equal(got, want)
    check(dy, got, pos, (16, 24, 24), interleaved=interleaved, inverse=True)


@pytest.mark.parametrize("interleaved", [True, False])
@pytest.mark.parametrize("theta", [1.0, 1.5, 1e4, 1e7])
@pytest.mark.parametrize("axes", [(64,), (128,), (256,), (22, 20, 22)])
def test_rotary_angles_up_to_two_to_the_24(axes, theta, interleaved):
    """The header's bound: 2^-23 turns at positions of up to 2^24 in magnitude.
    With it, cos and sin of two steps, two products and a sum:
    (2 pi 2^-23 + 2 * 2^-24 + 3 * 2^-24) / 2^-24 < 18 of the pair's magnitudes."""
    g = torch.Generator("cpu").manual_seed(12)
    D = max(64, sum(axes) + 2)
    D += -D % 8
    S = 64
    x = normal(13, 1, 2, S, D, dtype=torch.float32)
    pos = ((torch.rand(S, len(axes), generator=g) * 2 - 1) * 2 ** 24)
    pos[:4] = torch.tensor([2.0 ** 24, -(2.0 ** 24), 2.0 ** 24 - 1, 0.0]).view(4, 1)
    pos = pos.to(DEV)
    if D > 256:
        x, D = x[..., :256].contiguous(), 256
    y = cp.rotary(x, pos, axes, theta=theta, interleaved=interleaved)
    want, mag = plain.rotary(x, pos, axes, theta=theta, interleaved=interleaved)
    assert plain.worst(y, want, 18 * 2.0 ** -24 * mag) <= 1.0
