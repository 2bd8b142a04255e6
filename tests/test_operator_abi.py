"""Refusals of the rotary and cross-attention entry points (host side, no GPU)."""
import ctypes

import pytest
import torch

import context_attention_partial_gb300 as cp
from context_attention_partial_gb300 import _lib
from test_abi import DIV, DTYPE, FAKE, LAYOUT, NULL, OK, SHAPE, UNSUP, WS, t


def arr(*ts):
    return (_lib.CTensor * len(ts))(*ts)


def rotary(x, y=None, pos=None, axes=(16, 56, 56), n=None, **kw):
    lib = cp.load_library()
    xs = x if isinstance(x, (list, tuple)) else [x]
    ys = y if isinstance(y, (list, tuple)) else [y] if y is not None else \
        [t(tuple(a.shape[: a.ndim]), a.dtype, data=FAKE + (i + 9) * (1 << 24)) for i, a in enumerate(xs)]
    pos = pos if pos is not None else t((xs[0].shape[2], len(axes)), _lib.F32)
    dims = (ctypes.c_int32 * max(1, len(axes)))(*axes)
    return lib.cpattn_rotary(len(xs) if n is None else n, arr(*xs), pos, len(axes), dims, 1e4,
                             kw.get("interleaved", 1), kw.get("inverse", 0), arr(*ys), None)


def test_rotary_validation():
    x = t((1, 4, 16, 128))
    lib = cp.load_library()
    dims = (ctypes.c_int32 * 3)(16, 56, 56)
    assert rotary([x], n=0) == SHAPE
    assert rotary([x] * 5) == SHAPE
    assert lib.cpattn_rotary(1, None, t((16, 3), _lib.F32), 3, dims, 1e4, 1, 0, arr(x), None) == NULL
    assert lib.cpattn_rotary(1, arr(x), None, 3, dims, 1e4, 1, 0, arr(x), None) == NULL
    assert lib.cpattn_rotary(1, arr(x), t((16, 3), _lib.F32), 3, None, 1e4, 1, 0, arr(x), None) == NULL
    assert rotary(x, pos=t((16, 3))) == DTYPE                            # bf16 positions
    assert rotary(x, y=t((1, 4, 16, 128), _lib.F32)) == DTYPE
    assert rotary([x, t((1, 2, 16, 128), _lib.F32)]) == DTYPE
    assert rotary(t((1, 4, 16, 128), _lib.I32)) == DTYPE
    assert rotary(x, axes=()) == SHAPE
    assert rotary(x, axes=(32,) * 5) == SHAPE
    assert rotary(x, axes=(16, 57, 55)) == SHAPE                         # odd
    assert rotary(x, axes=(0, 64, 64)) == SHAPE
    assert rotary(x, axes=(-2, 64, 64)) == SHAPE
    assert rotary(x, axes=(64, 64, 2)) == SHAPE                          # past D
    assert rotary(x, pos=t((15, 3), _lib.F32)) == SHAPE
    assert rotary(x, pos=t((16, 2), _lib.F32)) == SHAPE
    assert rotary(x, pos=t((2, 16, 3), _lib.F32)) == SHAPE               # B is 1
    assert rotary([x, t((1, 4, 15, 128))]) == SHAPE
    assert rotary([x, t((1, 4, 16, 64))]) == SHAPE
    assert rotary(x, y=t((1, 4, 16, 64))) == SHAPE
    assert rotary(t((1, 4, 16, 12)), axes=(4, 4, 4)) == UNSUP            # 24-byte rows
    assert rotary(t((1, 4, 16, 264)), axes=(4, 4, 4)) == UNSUP
    assert rotary(t((1, 4, 16, 128), data=FAKE + 2)) == LAYOUT
    assert rotary(t((1, 4, 16, 128), stride=(8192, 2048, 132, 1))) == LAYOUT
    assert rotary(x, y=t((1, 4, 16, 128), data=FAKE + (1 << 24), stride=(0, 0, 128, 1))) == LAYOUT
    # in place only element for element
    assert rotary(x, y=t((1, 4, 16, 128), stride=(8192, 128, 512, 1))) == LAYOUT
    assert rotary(x, pos=t((16, 3), _lib.F32, data=FAKE + 2)) == LAYOUT
    assert rotary(x, pos=t((16, 3), _lib.F32, stride=(-3, 1))) == LAYOUT
    assert rotary(x, pos=t((16, 3), _lib.F32, data=0)) == NULL
    assert rotary(t((1, 4, 16, 128), data=0)) == NULL
    e = t((1, 4, 0, 128), data=0)
    assert rotary(e, y=e, pos=t((0, 3), _lib.F32, data=0)) == OK
    e = t((1, 0, 16, 128), data=0)
    assert rotary(e, y=e) == OK


def cross(q, k, v=None, out=None, lse=None, lengths=None, ws=None, ws_bytes=0):
    v = v if v is not None else t(tuple(k.shape[:4]), k.dtype)
    out = out if out is not None else t(tuple(q.shape[:4]), q.dtype)
    lse = lse if lse is not None else t(tuple(q.shape[:3]), _lib.F32)
    return cp.load_library().cpattn_cross_attention(q, k, v, lengths, 0.0, out, lse, ws, ws_bytes, None)


def grad(q, k, dout=None, dq=None, dk=None, dv=None, out=None, lse=None, lengths=None, ws=FAKE, ws_bytes=1 << 40):
    sq, sk = tuple(q.shape[:4]), tuple(k.shape[:4])
    return cp.load_library().cpattn_cross_attention_backward(
        q, k, t(sk, k.dtype), out or t(sq, q.dtype), lse or t(sq[:3], _lib.F32), dout or t(sq, q.dtype),
        lengths, 0.0, dq or t(sq, q.dtype), dk or t(sk, k.dtype), dv or t(sk, k.dtype), ws, ws_bytes, None)


def test_cross_validation():
    lib = cp.load_library()
    q, k = t((2, 8, 300, 128)), t((2, 2, 77, 128))
    n = t((2,), _lib.I32)
    assert lib.cpattn_cross_attention(None, k, k, None, 0.0, q, t((2, 8, 300), _lib.F32), None, 0, None) == NULL
    assert lib.cpattn_cross_attention(q, k, k, None, 0.0, q, None, None, 0, None) == NULL
    for call in (cross, grad):
        assert call(q, t((2, 2, 77, 128), _lib.F32)) == DTYPE
        assert call(t((2, 8, 300, 128), _lib.I32), t((2, 2, 77, 128), _lib.I32)) == DTYPE
        assert call(q, k, lengths=t((2,), _lib.F32)) == DTYPE
        assert call(q, k, lengths=t((3,), _lib.I32)) == SHAPE
        assert call(q, k, lengths=t((2, 1), _lib.I32)) == SHAPE
        assert call(q, t((1, 2, 77, 128))) == SHAPE                      # another batch
        assert call(q, t((2, 2, 77, 64))) == SHAPE
        assert call(q, t((2, 0, 77, 128))) == SHAPE
        assert call(q, t((2, 3, 77, 128))) == DIV                        # 8 % 3
        assert call(t((2, 8, 300, 96)), t((2, 2, 77, 96))) == UNSUP
        assert call(q, k, lse=t((2, 8, 299), _lib.F32)) == SHAPE
        assert call(q, k, lse=t((2, 8, 300))) == DTYPE
        assert call(q, k, out=t((2, 8, 300, 128), _lib.F32)) == DTYPE
        assert call(q, k, out=t((2, 8, 301, 128))) == SHAPE
        assert call(t((2, 8, 300, 128), data=FAKE + 8), k) == LAYOUT
        assert call(q, t((2, 2, 77, 128), stride=(0, 77 * 128, 128, 1))) == LAYOUT   # broadcast batch
        assert call(q, t((2, 2, 77, 128), stride=(2 * 77 * 128, 77 * 128, 132, 1))) == LAYOUT
        assert call(q, k, out=t((2, 8, 300, 128), stride=(0, 300 * 128, 128, 1))) == LAYOUT
        assert call(q, k, lse=t((2, 8, 300), _lib.F32, stride=(2400, 1, 8))) == LAYOUT
        assert call(q, k, lengths=t((2,), _lib.I32, stride=(2,))) == LAYOUT
        assert call(q, k, lengths=t((2,), _lib.I32, data=FAKE + 2)) == LAYOUT
        assert call(q, k, lengths=t((2,), _lib.I32, data=0)) == NULL
        assert call(t((2, 8, 300, 128), data=0), k) == NULL
        assert call(q, t((2, 2, 77, 128), data=0)) == NULL
        z = t((2, 8, 0, 128), data=0)
        assert call(z, t((2, 2, 0, 128), data=0)) == OK
    assert cross(t((2, 8, 0, 128), data=0), k) == OK
    assert cross(q, k, v=t((2, 2, 78, 128))) == SHAPE
    assert cross(q, k, v=t((2, 2, 77, 128), _lib.F32)) == DTYPE
    # few queries over many keys: the split's partials need a workspace
    few, far = t((1, 2, 1, 128)), t((1, 2, 9000, 128))
    need = lib.cpattn_cross_workspace_bytes(few, far)
    assert need > 0 and need % 4 == 0
    assert cross(few, far) == WS
    assert cross(few, far, ws=FAKE, ws_bytes=need - 4) == WS
    assert cross(few, far, ws=FAKE + 4, ws_bytes=need) == WS
    assert lib.cpattn_cross_workspace_bytes(q, t((2, 3, 77, 128))) == 0
    assert lib.cpattn_cross_workspace_bytes(None, k) == 0


def test_cross_backward_validation():
    lib = cp.load_library()
    q, k = t((2, 8, 300, 128)), t((2, 2, 77, 128))
    lse = t((2, 8, 300), _lib.F32)
    back = lib.cpattn_cross_attention_backward
    assert back(q, k, k, q, lse, None, None, 0.0, q, k, k, FAKE, 1 << 40, None) == NULL
    assert back(q, k, k, q, lse, q, None, 0.0, q, k, None, FAKE, 1 << 40, None) == NULL
    need = lib.cpattn_cross_backward_workspace_bytes(q, k)
    assert need >= 2 * 8 * 300 * 4
    assert grad(q, k, ws=None, ws_bytes=need) == WS
    assert grad(q, k, ws_bytes=need - 4) == WS
    assert grad(q, k, ws=FAKE + 4, ws_bytes=need) == WS
    assert grad(q, k, dout=t((2, 8, 300, 128), _lib.F32)) == DTYPE
    assert grad(q, k, dk=t((2, 2, 77, 128), _lib.F32)) == DTYPE
    assert grad(q, k, dv=t((2, 8, 77, 128))) == SHAPE                    # shared heads sum
    assert grad(q, k, dq=t((2, 8, 299, 128))) == SHAPE
    assert grad(q, k, dk=t((2, 2, 77, 128), stride=(0, 77 * 128, 128, 1))) == LAYOUT
    assert grad(q, k, dout=t((2, 8, 300, 128), stride=(0, 300 * 128, 128, 1))) == LAYOUT
    assert grad(q, k, dq=t((2, 8, 300, 128), data=0)) == NULL


def test_python_binding_refusals():
    q = torch.zeros(1, 1, 4, 64)
    with pytest.raises(ValueError):
        cp.rotary(q, torch.zeros(4, 1), (64,))
    with pytest.raises(ValueError):
        cp.cross_attention(q, q, q)
    with pytest.raises(ValueError):
        cp.cross_attention_backward(q, q, q, q, torch.zeros(1, 1, 4), q)


@pytest.mark.parametrize("theta", [1.0, 1.5, 100.0, 1e4, 1e7])
@pytest.mark.parametrize("d", [64, 256])
def test_rotary_angle_arithmetic(d, theta):
    """The kernel's angle step by step on the host, in exact fractions where fp32
    rounds: within the header's 2^-23 turns at positions of up to 2^24."""
    import math
    import random
    from decimal import Decimal, getcontext

    import numpy as np
    f32 = np.float32
    getcontext().prec = 50
    two_pi = 2 * Decimal("3.14159265358979323846264338327950288419716939937511")
    rate, rng = -2.0 / d * math.log(theta), random.Random(1)
    step, f, worst = math.exp(rate), 0.0, Decimal(0)
    for i in range(d // 2):
        f = 0.15915494309189535 * math.exp(i * rate) if i % 16 == 0 else f * step
        hi_w = f32(f)
        lo_w = f32(f - float(hi_w))
        exact = (Decimal(-2 * i) / d * Decimal(theta).ln()).exp() / two_pi
        for pos in [f32(2.0 ** 24), f32(2.0 ** 24 - 1)] + [f32(rng.uniform(-2.0 ** 24, 2.0 ** 24)) for _ in range(8)]:
            product = float(pos) * float(hi_w)                 # (48 bits: exact in fp64)
            hi = f32(product)
            lo = f32(Decimal(float(pos)) * Decimal(float(lo_w)) + Decimal(product - float(hi)))
            turns = f32(f32(hi - np.rint(hi)) + lo)
            off = Decimal(float(turns)) - Decimal(float(pos)) * exact
            worst = max(worst, abs(off - off.to_integral_value()))
    assert worst < Decimal(2) ** -23


def test_workspace_sizes_without_a_device():
    """The sizes need no GPU and no CUDA tensor: shapes say all."""
    q, k = torch.zeros(1, 2, 1, 128).bfloat16(), torch.zeros(1, 2, 9000, 128).bfloat16()
    assert cp.cross_workspace_bytes(q, k) == cp.load_library().cpattn_cross_workspace_bytes(
        t((1, 2, 1, 128)), t((1, 2, 9000, 128))) > 0
    assert cp.cross_backward_workspace_bytes(q, k) >= 2 * 4
    assert cp.cross_workspace_bytes(torch.empty(1, 2, 1, 96, device="meta").bfloat16(), k) == 0
