"""The rotary and cross-attention entry points through the bounds-checking
build: nothing is reported, the normal build's results are bit-equal, and
with every output's extent 16 bytes short the writes to those bytes are
reported and skipped."""
import pytest
import torch

import context_attention_partial_gb300 as cp
from context_attention_partial_gb300 import _lib, api
from context_attention_partial_gb300 import build as _build

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
OK, BOUNDS = 0, 10
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def chk():
    lib = _lib.bind(_build.build(check=True))
    assert lib.cpattn_is_check_build() == 1
    yield lib
    lib.cpattn_set_check_shrink(0)


@pytest.fixture
def through(monkeypatch):
    """Routes the Python binding's calls to another build of the library."""
    def use(lib):
        monkeypatch.setattr(_lib, "load", lambda: lib)
    return use


def status(lib):
    return lib.cpattn_last_device_status(torch.cuda.current_stream().cuda_stream)


def inputs(B, H, Hk, M, N, D, dtype, lengths):
    g = torch.Generator("cpu").manual_seed(61)
    q, k, v, dout = (torch.randn(B, h, s, D, generator=g).to(dtype).to(DEV)
                     for h, s in ((H, M), (Hk, N), (Hk, N), (H, M)))
    return q, k, v, dout, None if lengths is None else torch.tensor(lengths, dtype=torch.int32, device=DEV)


def cross(q, k, v, dout, n):
    out, lse = cp.cross_attention(q, k, v, kv_lengths=n)
    return out, lse, *cp.cross_attention_backward(q, k, v, out, lse, dout, kv_lengths=n)


CASES = [
    (1, 1, 1, 1, 1, 64, None),
    (2, 4, 2, 3, 130, 128, (130, 7)),
    (1, 4, 1, 77, 129, 64, None),
    (4, 2, 2, 130, 200, 128, (0, 1, 128, 200)),
    (1, 2, 2, 257, 513, 128, (500,)),
    (2, 8, 2, 1, 5001, 128, (5001, 3000)),
    (1, 24, 24, 1000, 301, 64, None),
    (2, 8, 2, 900, 333, 128, (333, 70)),
    (2, 2, 2, 100, 2500, 128, (2500, 1030)),
    (1, 3, 3, 1500, 1030, 64, None),
]


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "x".join(map(str, c[:6])))
def test_cross_check_build_clean_and_equal(chk, through, case, dtype):
    t = inputs(*case[:6], dtype, case[6])
    normal = cp.load_library()
    through(chk)
    got = cross(*t)
    assert status(chk) == OK
    through(normal)
    want = cross(*t)
    for a, b in zip(got, want):
        assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("interleaved", [True, False])
def test_rotary_check_build_clean_and_equal(chk, through, interleaved, dtype):
    normal = cp.load_library()
    for B, H, Hk, S, D, axes in ((1, 3, 1, 33, 128, (16, 56, 56)), (2, 2, 2, 1, 64, (64,)), (3, 5, 2, 17, 24, (8, 8))):
        g = torch.Generator("cpu").manual_seed(62)
        q, k = (torch.randn(B, h, S, D, generator=g).to(dtype).to(DEV) for h in (H, Hk))
        pos = torch.rand(B, S, len(axes), generator=g).to(DEV) * 100
        through(chk)
        got = cp.rotary([q, k], pos, axes, interleaved=interleaved)
        assert status(chk) == OK
        through(normal)
        want = cp.rotary([q, k], pos, axes, interleaved=interleaved)
        assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("M", [1, 77, 300])
def test_check_build_reports_short_outputs(chk, through, M, dtype):
    q, k, v, dout, n = inputs(1, 4, 2, M, 1300, 64, dtype, None)
    normal = cp.load_library()
    want = cross(q, k, v, dout, n)
    through(chk)

    def short(call, outs):
        for o in outs:
            o.fill_(3.0)
        torch.cuda.synchronize()
        chk.cpattn_set_check_shrink(16)
        call()
        chk.cpattn_set_check_shrink(0)
        assert status(chk) == BOUNDS
        for o in outs:
            assert torch.all(o.flatten()[-(16 // o.element_size()):] == 3.0)

    out, lse = torch.empty_like(want[0]), torch.empty_like(want[1])
    short(lambda: cp.cross_attention(q, k, v, out=out), (out,))
    short(lambda: cp.cross_attention(q, k, v, lse=lse), (lse,))
    dq, dk, dv = (torch.empty_like(t) for t in want[2:])
    short(lambda: cp.cross_attention_backward(q, k, v, want[0], want[1], dout, dq=dq, dk=dk, dv=dv), (dq, dk, dv))
    y = torch.empty_like(q)
    pos = torch.zeros(M, 1, device=DEV)
    short(lambda: cp.rotary(q, pos, (64,), outs=y), (y,))
    through(normal)
    got = cross(q, k, v, dout, n)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
