"""Refusals of the norm and paged-cache entry points (host side, no GPU), and the
arithmetic that finds a token's place."""
import ctypes

import pytest
import torch

import context_attention_partial_gb300 as cp
from context_attention_partial_gb300 import _lib
from test_abi import DIV, DTYPE, FAKE, LAYOUT, NULL, OK, SHAPE, UNSUP, WS, t

F32, I32, BF16 = _lib.F32, _lib.I32, _lib.BF16
FAR = FAKE + (1 << 30)


def arr(xs):
    return None if xs is None else (_lib.CTensor * len(xs))(*xs)


def listed(x):
    return x if x is None or isinstance(x, (list, tuple)) else [x]


def dims(axes):
    return (ctypes.c_int32 * max(1, len(axes)))(*axes)


def norm(x, w=None, y=None, pos=None, axes=(16, 56, 56), n=None):
    xs = listed(x)
    ys = listed(y) or [t(tuple(a.shape[:a.ndim]), a.dtype, data=FAR + (i << 24)) for i, a in enumerate(xs)]
    pos = pos or t((xs[0].shape[2], len(axes)), F32)
    return cp.load_library().cpattn_norm_rotary(len(xs) if n is None else n, arr(xs), arr(listed(w)), 1e-6, pos, len(axes),
                                                dims(axes), 1e4, 1, arr(ys), None)


def grad(x, w=None, y=None, pos=None, axes=(16, 56, 56), n=None, dy=None, dw=None, ws=FAKE, ws_bytes=1 << 40):
    xs = listed(x)
    ys = listed(y) or [t(tuple(a.shape[:a.ndim]), a.dtype, data=FAR + (i << 24)) for i, a in enumerate(xs)]
    dys = listed(dy) or [t(tuple(a.shape[:a.ndim]), a.dtype, data=2 * FAR + (i << 24)) for i, a in enumerate(xs)]
    dws = listed(dw) or listed(w)
    pos = pos or t((xs[0].shape[2], len(axes)), F32)
    return cp.load_library().cpattn_norm_rotary_backward(
        len(xs) if n is None else n, arr(xs), arr(listed(w)), 1e-6, pos, len(axes), dims(axes), 1e4, 1, arr(dys), arr(ys),
        arr(dws), ws, ws_bytes, None)


@pytest.mark.parametrize("call", [norm, grad])
def test_norm_validation(call):
    x, w = t((1, 4, 16, 128)), t((128,))
    assert call([x], n=0) == SHAPE
    assert call([x] * 5) == SHAPE
    assert call(x, pos=t((16, 3))) == DTYPE
    assert call(x, y=t((1, 4, 16, 128), F32)) == DTYPE
    assert call([x, t((1, 2, 16, 128), F32)]) == DTYPE
    assert call(t((1, 4, 16, 128), I32)) == DTYPE
    assert call(x, w=t((128,), I32)) == DTYPE
    assert call([x, x], w=[w, t((128,), F32)]) == DTYPE
    for axes in ((), (32,) * 5, (16, 57, 55), (0, 64, 64), (-2, 64, 64), (64, 64, 2)):
        assert call(x, axes=axes) == SHAPE
    assert call(x, pos=t((15, 3), F32)) == SHAPE
    assert call(x, pos=t((2, 16, 3), F32)) == SHAPE
    assert call([x, t((1, 4, 15, 128))]) == SHAPE
    assert call([x, t((1, 4, 16, 64))]) == SHAPE
    assert call(x, y=t((1, 4, 16, 64))) == SHAPE
    assert call(x, w=t((64,))) == SHAPE
    assert call(x, w=t((1, 128))) == SHAPE
    assert call(t((1, 4, 16, 12)), axes=(4, 4, 4)) == UNSUP
    assert call(t((1, 4, 16, 264)), axes=(4, 4, 4)) == UNSUP
    assert call(t((1, 70000, 1, 128))) == UNSUP
    assert call(t((1, 4, 16, 128), data=FAKE + 2)) == LAYOUT
    assert call(t((1, 4, 16, 128), stride=(8192, 2048, 132, 1))) == LAYOUT
    assert call(x, y=t((1, 4, 16, 128), data=FAR, stride=(0, 0, 128, 1))) == LAYOUT
    assert call(x, y=t((1, 4, 16, 128), stride=(8192, 128, 512, 1))) == LAYOUT
    assert call(x, w=t((128,), stride=(2,))) == LAYOUT
    assert call(x, w=t((128,), F32, data=FAKE + 2)) == LAYOUT
    assert call(x, pos=t((16, 3), F32, data=FAKE + 2)) == LAYOUT
    assert call(x, pos=t((16, 3), F32, stride=(-3, 1))) == LAYOUT
    assert call(x, pos=t((16, 3), F32, data=0)) == NULL
    assert call(x, w=t((128,), data=0)) == NULL
    assert call(t((1, 4, 16, 128), data=0)) == NULL
    for e in (t((1, 4, 0, 128), data=0), t((1, 0, 16, 128), data=0), t((0, 4, 16, 128), data=0)):
        assert call(e, y=e, **({"dy": e} if call is grad else {})) == OK


def test_norm_backward_validation():
    lib = cp.load_library()
    x, w, pos = t((1, 4, 16, 128)), t((128,)), t((16, 1), F32)
    one = arr([x])
    args = (1, one, None, 1e-6, pos, 1, dims((128,)), 1e4, 1)
    assert lib.cpattn_norm_rotary_backward(*args, None, one, None, None, 0, None) == NULL
    weighted = (1, one, arr([w]), 1e-6, pos, 1, dims((128,)), 1e4, 1)
    assert lib.cpattn_norm_rotary_backward(*weighted, one, one, None, FAKE, 1 << 40, None) == NULL
    need = lib.cpattn_norm_rotary_backward_workspace_bytes(1, one)
    assert need > 0 and need % (128 * 4) == 0
    assert grad(x, w=w, ws=None, ws_bytes=need) == WS
    assert grad(x, w=w, ws_bytes=need - 4) == WS
    assert grad(x, w=w, ws=FAKE + 4, ws_bytes=need) == WS
    assert grad(x, dy=t((1, 4, 16, 128), F32)) == DTYPE
    assert grad(x, dy=t((1, 4, 15, 128))) == SHAPE
    assert grad(x, dy=t((1, 4, 16, 128), data=0)) == NULL
    assert grad(x, dy=t((1, 4, 16, 128), data=FAKE + 8)) == LAYOUT
    assert grad(x, dy=t((1, 4, 16, 128), data=FAR, stride=(8192, 128, 512, 1))) == LAYOUT   # in place, other strides
    assert grad(x, w=w, dw=t((128,), F32)) == DTYPE
    assert grad(x, w=w, dw=t((64,))) == SHAPE
    assert grad(x, w=w, dw=t((128,), data=0)) == NULL
    assert lib.cpattn_norm_rotary_backward_workspace_bytes(0, one) == 0
    assert lib.cpattn_norm_rotary_backward_workspace_bytes(1, None) == 0
    assert lib.cpattn_norm_rotary_backward_workspace_bytes(1, arr([t((1, 4, 16, 100), BF16)])) == 0


K, PAGES, TABLE, LEN = t((2, 2, 3, 64)), t((9, 2, 16, 64)), t((2, 5), I32), t((2,), I32)


def append(k=K, v=None, q=None, qw=None, kw=None, pos=None, axes=(64,), kp=PAGES, vp=None, table=TABLE, lengths=LEN,
           counts=None, q_out=None):
    v = v or t(tuple(k.shape[:4]), k.dtype)
    vp = vp or t(tuple(kp.shape[:4]), kp.dtype, data=FAR)
    q_out = q_out or (t(tuple(q.shape[:4]), q.dtype, data=FAR) if q is not None else None)
    return cp.load_library().cpattn_cache_append(q, k, v, qw, kw, 1e-6, pos, len(axes), dims(axes), 1e4, 1, kp, vp, table,
                                                 lengths, counts, q_out, None)


def attend(q=t((2, 4, 3, 64)), kp=PAGES, vp=None, table=TABLE, lengths=LEN, counts=None, parents=None, out=None, lse=None,
           ws=FAKE, ws_bytes=1 << 40):
    vp = vp or t(tuple(kp.shape[:4]), kp.dtype, data=FAR)
    out = out or t(tuple(q.shape[:4]), q.dtype, data=2 * FAR)
    lse = lse or t(tuple(q.shape[:3]), F32, data=3 * FAR)
    return cp.load_library().cpattn_cache_attention(q, kp, vp, table, lengths, counts, parents, 0.0, out, lse, ws, ws_bytes,
                                                    None)


@pytest.mark.parametrize("call", [append, attend])
def test_cache_validation(call):
    assert call(kp=t((9, 2, 16, 64), F32)) == DTYPE
    assert call(vp=t((9, 2, 16, 64), F32)) == DTYPE
    assert call(table=t((2, 5), F32)) == DTYPE
    assert call(lengths=t((2,), F32)) == DTYPE
    assert call(counts=t((2,), F32)) == DTYPE
    assert call(vp=t((8, 2, 16, 64))) == SHAPE
    assert call(table=t((3, 5), I32)) == SHAPE
    assert call(table=t((10,), I32)) == SHAPE
    assert call(lengths=t((3,), I32)) == SHAPE
    assert call(lengths=t((2, 1), I32)) == SHAPE
    assert call(counts=t((1,), I32)) == SHAPE
    assert call(kp=t((9, 2, 16, 128))) == SHAPE
    for rows in (8, 24, 2048):
        assert call(kp=t((9, 2, rows, 64))) == UNSUP
    assert call(table=t((2, (1 << 26) + 1), I32)) == UNSUP
    assert call(kp=t((9, 2, 16, 64), data=0)) == NULL
    assert call(vp=t((9, 2, 16, 64), data=0)) == NULL
    assert call(table=t((2, 5), I32, data=0)) == NULL
    assert call(lengths=t((2,), I32, data=0)) == NULL
    assert call(counts=t((2,), I32, data=0)) == NULL
    assert call(kp=t((9, 2, 16, 64), data=FAKE + 8)) == LAYOUT
    assert call(kp=t((9, 2, 16, 64), stride=(0, 1024, 64, 1))) == LAYOUT
    assert call(kp=t((9, 2, 16, 64), stride=(2176, 1088, 68, 1))) == LAYOUT
    assert call(table=t((2, 5), I32, stride=(10, 2))) == LAYOUT
    assert call(table=t((2, 5), I32, stride=(-5, 1))) == LAYOUT
    assert call(table=t((2, 5), I32, data=FAKE + 2)) == LAYOUT
    assert call(lengths=t((2,), I32, stride=(2,))) == LAYOUT
    assert call(counts=t((2,), I32, data=FAKE + 2)) == LAYOUT


def test_append_validation():
    lib = cp.load_library()
    q = t((2, 4, 3, 64))
    assert lib.cpattn_cache_append(None, None, K, None, None, 0.0, None, 0, None, 0.0, 0, PAGES, PAGES, TABLE, LEN, None, None,
                                   None) == NULL
    assert lib.cpattn_cache_append(q, K, K, None, None, 0.0, None, 0, None, 0.0, 0, PAGES, PAGES, TABLE, LEN, None, None,
                                   None) == NULL
    assert append(v=t((2, 2, 3, 64), F32)) == DTYPE
    assert append(v=t((2, 1, 3, 64))) == SHAPE
    assert append(v=t((2, 2, 4, 64))) == SHAPE
    assert append(k=t((2, 3, 3, 64))) == SHAPE                     # the pages have 2 heads
    assert append(q=t((2, 4, 4, 64))) == SHAPE
    assert append(q=t((1, 4, 3, 64))) == SHAPE
    assert append(q=t((2, 4, 3, 64), F32)) == DTYPE
    assert append(q=q, q_out=t((2, 4, 3, 64), F32)) == DTYPE
    assert append(q=q, q_out=t((2, 5, 3, 64))) == SHAPE
    assert append(q=q, q_out=t((2, 4, 3, 64), stride=(768, 64, 256, 1))) == LAYOUT   # in place, other strides
    assert append(q=t((2, 4, 3, 64), data=0)) == NULL
    assert append(k=t((2, 2, 3, 64), data=0)) == NULL
    assert append(kw=t((32,))) == SHAPE
    assert append(kw=t((64,), I32)) == DTYPE
    assert append(kw=t((64,), stride=(2,))) == LAYOUT
    assert append(q=q, kw=t((64,)), qw=t((64,), F32)) == DTYPE
    assert append(pos=t((3, 1))) == DTYPE
    assert append(pos=t((4, 1), F32)) == SHAPE
    assert append(pos=t((3, 1), F32), axes=(66,)) == SHAPE
    assert append(pos=t((3, 1), F32), axes=(63,)) == SHAPE
    assert append(pos=t((3, 1), F32), axes=()) == SHAPE
    assert append(k=t((2, 2, 3, 12)), kp=t((9, 2, 16, 12))) == UNSUP
    assert append(vp=t((9, 2, 16, 64))) == LAYOUT                  # keys and values in one place
    e = t((2, 2, 0, 64), data=0)
    assert append(k=e, v=e) == OK


def test_attention_validation():
    lib = cp.load_library()
    q = t((2, 4, 3, 64))
    assert lib.cpattn_cache_attention(None, PAGES, PAGES, TABLE, LEN, None, None, 0.0, q, LEN, None, 0, None) == NULL
    assert lib.cpattn_cache_attention(q, PAGES, PAGES, TABLE, LEN, None, None, 0.0, q, None, None, 0, None) == NULL
    assert attend(out=t((2, 4, 3, 64), F32)) == DTYPE
    assert attend(lse=t((2, 4, 3))) == DTYPE
    assert attend(out=t((2, 4, 4, 64))) == SHAPE
    assert attend(lse=t((2, 4, 4), F32)) == SHAPE
    assert attend(q=t((2, 5, 3, 64))) == DIV
    assert attend(q=t((2, 4, 3, 96)), kp=t((9, 2, 16, 96))) == UNSUP
    assert attend(q=t((2, 4, (1 << 24) + 1, 64))) == UNSUP
    assert attend(q=t((2, 4, 3, 64), data=FAKE + 8)) == LAYOUT
    assert attend(q=t((2, 4, 3, 64), stride=(0, 192, 64, 1))) == LAYOUT
    assert attend(out=t((2, 4, 3, 64), stride=(0, 192, 64, 1))) == LAYOUT
    assert attend(lse=t((2, 4, 3), F32, stride=(24, 1, 8))) == LAYOUT
    assert attend(q=t((2, 4, 3, 64), data=0)) == NULL
    assert attend(parents=t((2, 3), F32)) == DTYPE
    assert attend(parents=t((2, 4), I32)) == SHAPE
    assert attend(parents=t((1, 3), I32)) == SHAPE
    assert attend(q=t((2, 4, 257, 64)), parents=t((2, 257), I32)) == UNSUP
    assert attend(parents=t((2, 3), I32, data=0)) == NULL
    assert attend(parents=t((2, 3), I32, stride=(6, 2))) == LAYOUT
    big = t((2, 4096), I32)
    need = lib.cpattn_cache_attention_workspace_bytes(q, PAGES, big)
    assert need > 0 and need % 16 == 0
    assert attend(table=big, ws=None, ws_bytes=need) == WS
    assert attend(table=big, ws_bytes=need - 4) == WS
    assert attend(table=big, ws=FAKE + 4, ws_bytes=need) == WS
    assert lib.cpattn_cache_attention_workspace_bytes(None, PAGES, big) == 0
    assert lib.cpattn_cache_attention_workspace_bytes(t((2, 5, 3, 64)), PAGES, big) == 0
    z = t((2, 4, 0, 64), data=0)
    assert attend(q=z, out=z, lse=t((2, 4, 0), F32, data=0), ws=None, ws_bytes=0) == OK


def test_python_refusals():
    x, w, pos, i = torch.zeros(1, 1, 4, 64), torch.ones(64), torch.zeros(4, 1), torch.zeros(1, 2, dtype=torch.int32)
    pages, n = torch.zeros(2, 1, 16, 64), torch.zeros(1, dtype=torch.int32)
    for call in (lambda: cp.norm_rotary(x, w, pos, (64,)), lambda: cp.norm_rotary_backward(x, w, pos, (64,), x),
                 lambda: cp.cache_append(x, x, pages, pages, i, n), lambda: cp.cache_attention(x, pages, pages, i, n)):
        with pytest.raises(ValueError, match="CUDA tensors only"):
            call()
    with pytest.raises(ValueError, match="2 tensors but 1 weights"):
        cp.norm_rotary([x, x], [w], pos, (64,))
    with pytest.raises(ValueError, match="1 tensors but 2 gradients"):
        cp.norm_rotary_backward([x], None, pos, (64,), [x, x])
    with pytest.raises(ValueError, match="1 tensors but 2 outputs"):
        cp.norm_rotary([x], None, pos, (64,), outs=[x, x])
    with pytest.raises(cp.CpattnError):
        cp.norm_rotary([x] * 5, None, pos, (64,))
    with pytest.raises(cp.CpattnError):
        cp.norm_rotary(x, w, pos, (8,) * 5)
    with pytest.raises(TypeError):
        cp.norm_rotary(x, w, pos, 64)


def test_workspace_sizes_without_a_device():
    x = torch.zeros(1, 2, 100, 64)
    assert cp.norm_rotary_backward_workspace_bytes([x, x]) > 0
    q, pages, table = torch.zeros(1, 2, 1, 64), torch.zeros(9, 1, 16, 64), torch.zeros(1, 500, dtype=torch.int32)
    assert cp.cache_attention_workspace_bytes(q, pages, table) > 0
    assert cp.cache_attention_workspace_bytes(q, pages, table[:, :1]) == 0


def walk(tiles, kv_heads, blocks, cost, min_tiles=3):
    """The split of the key tiles over blocks as the kernels do it: per block its pieces
    (unit, first tile, last tile, tiles of the unit).  A unit's place in the line is its
    tiles and `cost` that stand for its beginning and end."""
    line = [n for n in tiles for _ in range(kv_heads)]
    total = sum(n + cost for n in line if n)
    used = min(blocks, -(-total // min_tiles))
    pieces = []
    for c in range(used):
        each, more = total // used, total % used
        pos = c * each + min(c, more)
        end, mine, base = pos + each + (c < more), [], 0
        for u, n in enumerate(line):
            lo, hi = max(pos, base), min(end, base + n)
            if lo < hi:
                mine.append((u, lo - base, hi - base, n))
            base += n + cost if n else 0
        pieces.append(mine)
    return pieces


@pytest.mark.parametrize("cost", [0, 1, 3])
@pytest.mark.parametrize("tiles,kv_heads,blocks", [([5], 1, 304), ([1000], 1, 304), ([7, 0, 300, 1], 3, 304),
                                                   ([0, 0], 2, 10), ([64] * 20, 8, 304), ([1, 2, 3], 5, 4), ([1] * 40, 2, 30)])
def test_parts_of_a_unit_have_slots_of_their_own(tiles, kv_heads, blocks, cost):
    """Every tile is taken once, a block has at most one piece for each of its two slots, and a
    unit's parts are slot 1 of the block that begins it and slot 0 of all behind it up to the
    one that ends it, as the join takes them."""
    pieces = walk(tiles, kv_heads, blocks, cost)
    line = [n for n in tiles for _ in range(kv_heads)]
    taken = [[0] * n for n in line]
    first, last, parts = {}, {}, {}
    for c, mine in enumerate(pieces):
        slots = []
        for u, lo, hi, n in mine:
            for i in range(lo, hi):
                taken[u][i] += 1
            if lo == 0:
                first[u] = c
            if hi == n:
                last[u] = c
            if (lo, hi) != (0, n):
                slots.append(0 if lo > 0 else 1)
                parts.setdefault(u, []).append((c, slots[-1]))
        assert len(slots) == len(set(slots))
    assert all(x == 1 for unit in taken for x in unit)
    for u, n in enumerate(line):
        if n and first[u] != last[u]:
            assert parts[u] == [(c, 1 if c == first[u] else 0) for c in range(first[u], last[u] + 1)]
        else:
            assert u not in parts
