"""Per-head norms with rotary positions, and their gradient, against the formulas in 64 bits."""
import warnings

import pytest
import torch

import context_attention_partial_gb300 as cp
import plain_cache as C
import plain_operators as P

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32


def tensors(B, heads, S, D, dtype, seed, layout="bhsd"):
    g = torch.Generator("cpu").manual_seed(seed)
    out = []
    for h in heads:
        x = torch.randn((B, h, S, D) if layout == "bhsd" else (B, S, h, D), generator=g).to(dtype).to(DEV)
        out.append(x if layout == "bhsd" else x.transpose(1, 2))
    return out


def weights(n, D, dtype, seed):
    g = torch.Generator("cpu").manual_seed(seed)
    return None if dtype is None else [(1 + 0.3 * torch.randn(D, generator=g)).to(dtype).to(DEV) for _ in range(n)]


def positions(B, S, axes, per_batch, seed):
    g = torch.Generator("cpu").manual_seed(seed)
    return torch.randint(0, 500, (B, S, len(axes)) if per_batch else (S, len(axes)), generator=g).float().to(DEV)


def check(got, want_tol):
    want, tol = want_tol
    assert got.shape == want.shape
    assert P.worst(got, want, tol) <= 1


# (B, heads, S, D, axes, per_batch, weights)
CASES = [
    (1, (3, 1), 33, 128, (16, 56, 56), False, BF),
    (2, (2,), 1, 64, (64,), True, F32),
    (3, (5, 2, 1), 17, 24, (8, 8), True, None),
    (1, (24, 24), 300, 128, (44, 42, 42), False, F32),
    (2, (4, 4, 2, 2), 19, 256, (64, 32, 96, 64), False, BF),
    (1, (7,), 2000, 8, (2,), False, BF),
    (1, (2,), 5, 136, (32, 104), False, None),
    (4, (16, 4), 130, 64, (32, 32), True, BF),
    (1, (1,), 40, 96, (6, 10), False, F32),
    (2, (40, 8), 3, 128, (128,), False, F32),
]
SLOW = [(1, (2, 1), 40, 160, (64, 96), False, F32), (1, (3,), 9, 252, (36, 108), True, F32)]


def ident(c):
    return "x".join(map(str, (c[0], *c[1], c[2], c[3])))


@pytest.mark.parametrize("layout", ["bhsd", "bshd"])
@pytest.mark.parametrize("interleaved", [True, False])
@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("case", CASES + SLOW, ids=ident)
def test_both_directions(case, dtype, interleaved, layout):
    B, heads, S, D, axes, per_batch, wtype = case
    if D * (2 if dtype == BF else 4) % 16:
        pytest.skip("rows are whole 16-byte vectors")
    xs, dys = tensors(B, heads, S, D, dtype, 1, layout), tensors(B, heads, S, D, dtype, 2, layout)
    ws, pos = weights(len(heads), D, wtype, 3), positions(B, S, axes, per_batch, 4)
    kw = dict(eps=1e-5, theta=500.0, interleaved=interleaved)
    ys = cp.norm_rotary(xs, ws, pos, axes, **kw)
    dxs, dws = cp.norm_rotary_backward(xs, ws, pos, axes, dys, **kw)
    assert (dws is None) == (ws is None)
    for i, x in enumerate(xs):
        w = None if ws is None else ws[i]
        assert ys[i].dtype == dtype and ys[i].stride() == x.stride()
        check(ys[i], C.norm_rotary(x, w, pos, axes, **kw))
        dx, dw = C.norm_rotary_backward(x, w, pos, axes, dys[i], **kw)
        check(dxs[i], dx)
        if w is not None:
            assert dws[i].dtype == w.dtype
            check(dws[i], dw)
    assert cp.last_device_status() == 0
    again = cp.norm_rotary_backward(xs, ws, pos, axes, dys, **kw)
    assert all(torch.equal(a, b) for a, b in zip(dxs, again[0]))
    if ws is not None:
        assert all(torch.equal(a, b) for a, b in zip(dws, again[1]))


def test_against_differences():
    """The fp32 gradient along random directions against central differences of the
    plain 64-bit form."""
    torch.manual_seed(0)
    x, dy, vx = (torch.randn(1, 2, 7, 32, device=DEV) for _ in range(3))
    w, vw = 1 + 0.3 * torch.randn(32, device=DEV), torch.randn(32, device=DEV)
    pos = torch.arange(7, device=DEV).float()[:, None]
    dx, dw = cp.norm_rotary_backward(x, w, pos, (32,), dy)

    def f(t):
        xx, ww = x.double() + t * vx.double(), w.double() + t * vw.double()
        z = xx * torch.rsqrt(xx.square().mean(-1, keepdim=True) + 1e-6) * ww
        return float((P.rotary(z, pos, (32,))[0] * dy.double()).sum())

    h = 1e-4
    slope = (f(h) - f(-h)) / (2 * h)
    got = float((dx.double() * vx.double()).sum() + (dw.double() * vw.double()).sum())
    # differences: h^2 of a third derivative of some hundreds; fp32: 2^-18 of the magnitudes
    assert abs(got - slope) <= 1e-4 + 2.0 ** -18 * float((dx * vx).abs().sum() + (dw * vw).abs().sum())


@pytest.mark.parametrize("interleaved", [True, False])
@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_in_place(dtype, interleaved):
    axes = (12, 20)   # (halves that are not whole vectors)
    xs, dys = tensors(2, (3, 2), 37, 64, dtype, 5), tensors(2, (3, 2), 37, 64, dtype, 6)
    ws, pos = weights(2, 64, F32, 7), positions(2, 37, axes, False, 8)
    kw = dict(interleaved=interleaved)
    want = cp.norm_rotary(xs, ws, pos, axes, **kw)
    wdx, wdw = cp.norm_rotary_backward(xs, ws, pos, axes, dys, **kw)
    mine = [x.clone() for x in xs]
    got = cp.norm_rotary(mine, ws, pos, axes, outs=mine, **kw)
    assert all(a is b and torch.equal(a, c) for a, b, c in zip(got, mine, want))
    for over in ("dy", "x"):
        a, b = [x.clone() for x in xs], [d.clone() for d in dys]
        dx, dw = cp.norm_rotary_backward(a, ws, pos, axes, b, dxs=b if over == "dy" else a, **kw)
        assert all(torch.equal(x, y) for x, y in zip(dx + dw, wdx + wdw))


def test_broadcast_inputs_and_single_tensors():
    x = torch.randn(1, 4, 1, 64, device=DEV).expand(3, 4, 50, 64)
    dy = torch.ones(1, device=DEV).expand(3, 4, 50, 64)
    w, pos = torch.ones(1, device=DEV).expand(64), torch.arange(50, device=DEV).float()[:, None]
    y = cp.norm_rotary(x, w, pos, (64,))
    check(y, C.norm_rotary(x, w, pos, (64,)))
    dx, dw = cp.norm_rotary_backward(x, w, pos, (64,), dy)
    a, b = C.norm_rotary_backward(x, w, pos, (64,), dy)
    check(dx, a)
    check(dw, b)
    assert cp.norm_rotary_backward(x, None, pos, (64,), dy)[1] is None


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_extreme_rows(dtype):
    """Rows of zeros, with and without eps, large and tiny rows, and rows that are not
    finite beside them."""
    x = torch.randn(1, 1, 8, 64, device=DEV)
    x[0, 0, 0] = 0
    x[0, 0, 1] *= 1e15
    x[0, 0, 2] *= 1e-15
    x[0, 0, 3, 5] = float("nan")
    x[0, 0, 4, 5] = float("inf")
    x, pos = x.to(dtype), torch.zeros(8, 1, device=DEV)
    for eps in (1e-6, 1.0):
        y = cp.norm_rotary(x, None, pos, (64,), eps=eps)
        want, tol = C.norm_rotary(x, None, pos, (64,), eps=eps)
        rows = [0, 1, 2, 5, 6, 7]
        assert P.worst(y[:, :, rows], want[:, :, rows], tol[:, :, rows]) <= 1
        assert y[0, 0, 3].isnan().all() and y[0, 0, 4, 5].isnan()
    y = cp.norm_rotary(x[:, :, 1:3], None, pos[:2], (64,), eps=0.0)
    check(y, C.norm_rotary(x[:, :, 1:3], None, pos[:2], (64,), eps=0.0))
    # (not a number, or below 0: 1e-6)
    for eps in (float("nan"), -1.0):
        assert torch.equal(cp.norm_rotary(x[:, :, 5:], None, pos[:3], (64,), eps=eps),
                           cp.norm_rotary(x[:, :, 5:], None, pos[:3], (64,)))


@pytest.mark.parametrize("interleaved", [True, False])
@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_an_infinite_weight_of_a_feature_that_does_not_turn(dtype, interleaved):
    """It is that feature's alone: infinite of x's sign there, every other feature as ever."""
    axes, D = (6, 4), 24   # (10 features turn: some vectors in part)
    x, = tensors(2, (3,), 9, D, dtype, 5)
    pos = positions(2, 9, axes, False, 6)
    w, = weights(1, D, F32, 7)
    for f in (10, 11, 17):
        bad = w.clone()
        bad[f] = float("inf")
        got = cp.norm_rotary(x, bad, pos, axes, interleaved=interleaved)
        want = cp.norm_rotary(x, w, pos, axes, interleaved=interleaved)
        others = [i for i in range(D) if i != f]
        assert torch.equal(got[..., others], want[..., others])
        assert torch.equal(got[..., f].float(), x[..., f].float().sign() * float("inf"))


def test_no_rows():
    w = torch.ones(64, device=DEV)
    for shape in ((0, 2, 5, 64), (1, 0, 5, 64), (1, 2, 0, 64)):
        x = torch.empty(shape, device=DEV)
        pos = torch.zeros(shape[2], 1, device=DEV)
        assert cp.norm_rotary(x, w, pos, (64,)).shape == shape
        dw = torch.full((64,), 3.0, device=DEV)
        dx, got = cp.norm_rotary_backward(x, w, pos, (64,), x, dweights=dw)
        assert got is dw and torch.all(dw == 0) and dx.shape == shape
    # one tensor without heads beside one with
    x, e = torch.randn(1, 2, 5, 64, device=DEV), torch.empty(1, 0, 5, 64, device=DEV)
    pos = torch.zeros(5, 1, device=DEV)
    dxs, dws = cp.norm_rotary_backward([e, x], [w, w], pos, (64,), [e, x])
    assert torch.all(dws[0] == 0) and torch.equal(dws[1], cp.norm_rotary_backward(x, w, pos, (64,), x)[1])


def test_many_tokens_and_heads():
    """More tiles than blocks, and more heads than a block takes."""
    for B, heads, S, D in ((2, (1,), 70001, 64), (1, (300,), 3, 128)):
        x, dy = tensors(B, heads, S, D, BF, 11)[0], tensors(B, heads, S, D, BF, 12)[0]
        w, pos = weights(1, D, F32, 13)[0], positions(B, S, (D,), False, 14)
        check(cp.norm_rotary(x, w, pos, (D,)), C.norm_rotary(x, w, pos, (D,)))
        dx, dw = cp.norm_rotary_backward(x, w, pos, (D,), dy)
        a, b = C.norm_rotary_backward(x, w, pos, (D,), dy)
        check(dx, a)
        check(dw, b)


def test_streams_graphs_and_autograd():
    x, dy = tensors(1, (4,), 100, 64, BF, 15)[0], tensors(1, (4,), 100, 64, BF, 16)[0]
    w, pos = weights(1, 64, BF, 17)[0], positions(1, 100, (64,), False, 18)
    want = cp.norm_rotary(x, w, pos, (64,))
    wdx, wdw = cp.norm_rotary_backward(x, w, pos, (64,), dy)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    y = cp.norm_rotary(x, w, pos, (64,), stream=side)
    dx, dw = cp.norm_rotary_backward(x, w, pos, (64,), dy, stream=side)
    side.synchronize()
    assert torch.equal(y, want) and torch.equal(dx, wdx) and torch.equal(dw, wdw)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = cp.norm_rotary(x, w, pos, (64,))
        dx, dw = cp.norm_rotary_backward(x, w, pos, (64,), dy)
    for t in (y, dx, dw):
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, want) and torch.equal(dx, wdx) and torch.equal(dw, wdw)

    class Norm(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, w):
            ctx.save_for_backward(x, w)
            return cp.norm_rotary(x, w, pos, (64,))

        @staticmethod
        def backward(ctx, dy):
            return cp.norm_rotary_backward(*ctx.saved_tensors, pos, (64,), dy)

    xr, wr = x.clone().requires_grad_(), w.clone().requires_grad_()
    with warnings.catch_warnings():
        warnings.simplefilter("error")
        (Norm.apply(xr, wr) * dy).sum().backward()
    assert torch.equal(xr.grad, wdx) and torch.equal(wr.grad, wdw)
    with pytest.warns(UserWarning, match="no autograd graph"):
        cp.norm_rotary(x, wr, pos, (64,))


def test_workspace_of_the_caller():
    x = torch.randn(1, 4, 100, 64, device=DEV)
    w, pos = torch.ones(64, device=DEV), torch.zeros(100, 1, device=DEV)
    need = cp.norm_rotary_backward_workspace_bytes(x)
    assert need > 0 and cp.norm_rotary_backward_workspace_bytes([x]) == need
    want = cp.norm_rotary_backward(x, w, pos, (64,), x)
    got = cp.norm_rotary_backward(x, w, pos, (64,), x, workspace=torch.full((need,), 255, dtype=torch.uint8, device=DEV))
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    with pytest.raises(cp.CpattnError) as e:
        cp.norm_rotary_backward(x, w, pos, (64,), x, workspace=torch.empty(need - 4, dtype=torch.uint8, device=DEV))
    assert e.value.name == "CPATTN_ERR_WORKSPACE"
