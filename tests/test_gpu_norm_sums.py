"""Gradients of norms' weights, exactly, at the sizes where many blocks share them.

x is +-1 everywhere and eps 0, so each row's factor is 1; positions are 0, so nothing turns; and
dy = c x with c of 0 to 3.  Then dw is the sum of c over tokens and heads: whole numbers below
2^24, whose sums are exact in fp32 in any order, and a row that is left out or added twice shows."""
import pytest
import torch

import context_attention_partial_gb300 as cp

DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32


def inputs(B, H, S, D, dtype, device, seed, most):
    """x, dy and the exact dw: c is 0 or 1 (most 1), or 1 to 3."""
    g = torch.Generator(device).manual_seed(seed)
    sign = torch.randint(0, 2, (B, H, S, D), generator=g, dtype=torch.int8, device=device).mul_(2).sub_(1)
    x = sign.to(dtype)
    c = torch.randint(0 if most == 1 else 1, most + 1, (B, H, S, D), generator=g, dtype=torch.int8, device=device)
    dw = c.sum((0, 1, 2), dtype=torch.int64)
    dy = sign.mul_(c).to(dtype)
    assert int(dw.max()) < 2 ** 24
    return x, dy, dw


# (B, heads, S, D, dtype, interleaved)
CASES = [
    (2, (1,), 70001, 64, BF, True),              # more tiles of tokens than blocks
    (1, (300,), 3, 128, BF, False),              # more heads than a block takes
    (30000, (4, 2), 1, 64, BF, True),            # many sequences
    (1, (24, 24), 32768, 128, BF, True),
    (1, (24, 8), 4609, 128, F32, False),
    (2, (3, 1, 2, 5), 10007, 256, F32, True),    # two vectors a lane
    (1, (7, 2), 20011, 256, BF, False),
    (3, (5,), 9001, 24, BF, False),              # rows that do not fill their lanes
    (1, (1, 1), 1, 8, BF, True),
]


@pytest.mark.gpu
@pytest.mark.parametrize("case", CASES, ids=lambda c: "x".join(map(str, (c[0], *c[1], c[2], c[3]))))
def test_sums_are_exact(case):
    B, heads, S, D, dtype, interleaved = case
    xs, dys, want = zip(*(inputs(B, H, S, D, dtype, DEV, i, 3) for i, H in enumerate(heads)))
    ws, pos = [torch.ones(D, device=DEV) for _ in heads], torch.zeros(S, 1, device=DEV)
    kw = dict(eps=0.0, interleaved=interleaved)
    for y, x in zip(cp.norm_rotary(list(xs), ws, pos, (D,), **kw), xs):
        assert torch.equal(y, x)                 # (the rows' factors are 1)
    dxs, dws = cp.norm_rotary_backward(list(xs), ws, pos, (D,), list(dys), **kw)
    for dw, n in zip(dws, want):
        assert torch.equal(dw.long(), n) and torch.equal(dw, dw.round())
    assert cp.last_device_status() == 0


@pytest.mark.gpu
def test_sums_past_2_31_elements():
    H, S, D = 2, 2 ** 23 + 5, 128
    x, dy, want = inputs(1, H, S, D, BF, DEV, 1, 1)
    assert x.numel() > 2 ** 31
    w, pos = torch.ones(D, device=DEV), torch.zeros(S, 1, device=DEV)
    dx, dw = cp.norm_rotary_backward(x, w, pos, (D,), dy, eps=0.0, dxs=dy)
    assert torch.equal(dw.long(), want) and torch.equal(dw, dw.round())


@pytest.mark.parametrize("case", CASES, ids=lambda c: "x".join(map(str, (c[0], *c[1], c[2], c[3]))))
def test_a_lost_tile_shows(case):
    """The check of the sums notices the smallest share that a kernel could lose or add twice: one head of
    one token."""
    B, heads, S, D, dtype, _ = case
    H, S = heads[0], min(S, 64)
    x, dy, want = inputs(min(B, 2), H, S, D, dtype, "cpu", 0, 3)
    r = torch.rsqrt(x.double().square().mean(-1, keepdim=True))
    terms = x.double() * r * dy.double()
    assert torch.equal(terms.sum((0, 1, 2)).long(), want)
    for row in (terms[0, 0, 0], terms[-1, -1, -1]):
        assert bool(((terms.sum((0, 1, 2)) - row).long() != want).all())
        assert bool(((terms.sum((0, 1, 2)) + row).long() != want).all())
