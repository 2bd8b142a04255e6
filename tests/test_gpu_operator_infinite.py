"""Scores of -inf in cross attention: a key that a query's score puts at -inf has
no weight there, and the rest of the row is what it is without that key.

Two ways to such scores.  "inf": the keys hold -inf in feature 0 and every query
is positive there.  "overflow": they hold -3e38 and some queries 1e3 (a product
past fp32), the others 0 -- so those keys have weight in some rows only."""
import math

import pytest
import torch

import context_attention_partial_gb300 as cp
import plain_operators as plain

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32


def inputs(kind, B, H, Hk, M, N, D, dtype, dead, seed):
    """q, k, v, dout with the keys `dead` (a slice, or None: all) at -inf, and per
    row whether they are (bool [M])."""
    g = torch.Generator("cpu").manual_seed(seed)
    q, k, v, dout = (torch.randn(B, h, s, D, generator=g) for h, s in ((H, M), (Hk, N), (Hk, N), (H, M)))
    k[..., 0] = 0
    rows = torch.ones(M, dtype=torch.bool)
    if kind == "inf":
        q[..., 0] = q[..., 0].abs() + 0.5
        k[:, :, dead, 0] = -math.inf
    else:
        rows = torch.arange(M) % 3 != 1
        q[..., 0] = rows.float() * 1e3
        k[:, :, dead, 0] = -3e38
    q, k, v, dout = (t.to(dtype).to(DEV) for t in (q, k, v, dout))
    return q, k, v, dout, rows.to(DEV)


def expected(q, k, v, dout, rows, dead, lengths):
    """plain.cross without the dead keys for `rows`, with them (their feature 0 is
    met by zeros) for the others: name -> (value, tolerance)."""
    B, H, M, D = q.shape
    N = k.shape[2]
    alive = torch.ones(N, dtype=torch.bool, device=DEV)
    alive[dead] = False
    k0 = k.clone()
    k0[:, :, dead, 0] = 0
    full = {}
    for part, keys in ((rows, alive), (~rows, torch.ones_like(alive))):
        if not part.any():
            continue
        left = None if lengths is None else [int(keys[: max(0, n)].sum()) for n in lengths]
        got = plain.cross(q[:, :, part], k0[:, :, keys], v[:, :, keys], left, dout=dout[:, :, part])
        for name, pair in got.items():
            shape = {"out": (B, H, M, D), "dq": (B, H, M, D), "lse": (B, H, M)}.get(name, tuple(k.shape))
            if name not in full:
                full[name] = [torch.zeros(shape, dtype=torch.float64, device=DEV) for _ in range(2)]
            for whole, x in zip(full[name], pair):
                if name in ("dk", "dv"):
                    whole[:, :, keys] += x
                else:
                    whole[:, :, part] = x
    return full


def ratio(got, pair, skip_first=False):
    value, tol = pair
    cut = slice(1, None) if skip_first else slice(None)
    return plain.worst(got[..., cut] if skip_first else got, value[..., cut] if skip_first else value,
                       tol[..., cut] if skip_first else tol)


def lengths_of(n):
    return None if n is None else torch.tensor(n, dtype=torch.int32, device=DEV)


# (B, H, H_kv, S_q, S_kv, D, dead keys, lengths)
CASES = [
    (1, 2, 2, 128, 129, 128, slice(128, 129), None),          # a lone key in the second chain of tiles
    (1, 2, 2, 128, 129, 64, slice(0, 128), None),             # a whole first tile
    (1, 3, 3, 300, 400, 128, slice(0, 128), None),
    (2, 4, 2, 200, 257, 64, slice(0, 256), (257, 200)),       # (a sequence of dead keys only: below)
    (1, 2, 1, 77, 4481, 64, slice(0, 1200), None),            # whole key parts
    (1, 2, 2, 100, 2500, 128, slice(1300, 2500), None),
    (1, 1, 1, 400, 1100, 128, slice(128, 1100), None),
    (2, 8, 2, 1, 3000, 128, slice(0, 2900), (3000, 2999)),    # few rows
    (1, 6, 2, 9, 500, 64, slice(64, 128), None),
    (1, 4, 4, 33, 70, 64, slice(69, 70), None),
]
IDS = ["x".join(map(str, c[:6])) for c in CASES]


def whole(case):
    """The case, its lengths raised so that every sequence keeps a live key."""
    *sizes, dead, lengths = case
    if lengths is not None:
        last = dead.stop + 1
        lengths = tuple(max(n, last) for n in lengths)
    return sizes, dead, lengths


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("kind", ["inf", "overflow"])
@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_keys_at_minus_infinity_have_no_weight(case, kind, dtype):
    sizes, dead, lengths = whole(case)
    q, k, v, dout, rows = inputs(kind, *sizes, dtype, dead, seed=1)
    want = expected(q, k, v, dout, rows, dead, lengths)
    out, lse = cp.cross_attention(q, k, v, kv_lengths=lengths_of(lengths))
    assert cp.last_device_status() == 0
    assert ratio(out, want["out"]) <= 1.0
    assert ratio(lse, want["lse"]) <= 1.0


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("kind", ["inf", "overflow"])
@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_gradient_with_keys_at_minus_infinity(case, kind, dtype):
    """dk and dv of such a key are 0 where no row gives it weight, also when the
    last tile of queries is not full.  (dq's feature 0 is 0 * inf, or past bf16.)"""
    sizes, dead, lengths = whole(case)
    q, k, v, dout, rows = inputs(kind, *sizes, dtype, dead, seed=2)
    want = expected(q, k, v, dout, rows, dead, lengths)
    n = lengths_of(lengths)
    out, lse = cp.cross_attention(q, k, v, kv_lengths=n)
    dq, dk, dv = cp.cross_attention_backward(q, k, v, out, lse, dout, kv_lengths=n)
    assert cp.last_device_status() == 0
    assert ratio(dq, want["dq"], skip_first=True) <= 1.0
    assert ratio(dk, want["dk"]) <= 1.0
    assert ratio(dv, want["dv"]) <= 1.0
    if kind == "inf":
        assert torch.all(dk[:, :, dead] == 0) and torch.all(dv[:, :, dead] == 0)


# S_q, S_kv, D: the few-rows kernel, one chain and two, key parts (cluster and
# workspace), 64-row and small fp32 blocks
ALL = [(1, 5, 64), (3, 700, 128), (1, 9000, 128), (40, 130, 64), (77, 4481, 64), (130, 128, 128), (300, 300, 128), (1000, 200, 64)]


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("kind", ["inf", "overflow"])
@pytest.mark.parametrize("M,N,D", ALL)
def test_rows_without_a_finite_score_are_rows_without_keys(M, N, D, kind, dtype):
    """(0, -inf) forward, and no part in any gradient."""
    dead = slice(0, N)
    q, k, v, dout, rows = inputs(kind, 1, 4, 2, M, N, D, dtype, dead, seed=3)
    want = expected(q, k, v, dout, rows, dead, None)
    out, lse = cp.cross_attention(q, k, v)
    dq, dk, dv = cp.cross_attention_backward(q, k, v, out, lse, dout)
    assert cp.last_device_status() == 0
    assert torch.all(out[:, :, rows] == 0) and torch.all(lse[:, :, rows] == -math.inf)
    assert ratio(out, want["out"]) <= 1.0 and ratio(lse, want["lse"]) <= 1.0
    assert torch.all(dq[:, :, rows, 1:] == 0)
    assert ratio(dq, want["dq"], skip_first=True) <= 1.0
    assert ratio(dk, want["dk"]) <= 1.0 and ratio(dv, want["dv"]) <= 1.0
    if kind == "overflow":
        assert torch.all(dq[:, :, rows] == 0)
