"""Rotary and cross attention on tensors past 2^31 elements: the 64-bit index
paths, each call first through the bounds-checking build, which must report
nothing; samples at the start, the middle and the far end against 64 bits."""
import pytest
import torch

import context_attention_partial_gb300 as cp
import plain_operators as plain
from context_attention_partial_gb300 import _lib
from context_attention_partial_gb300 import build as _build

pytestmark = [pytest.mark.gpu, pytest.mark.slow]
DEV = "cuda:0"
BF = torch.bfloat16


@pytest.fixture
def both(monkeypatch):
    """Runs a call through the check build, then through the normal one."""
    chk, normal = _lib.bind(_build.build(check=True)), cp.load_library()

    def run(call):
        monkeypatch.setattr(_lib, "load", lambda: chk)
        call()
        assert chk.cpattn_last_device_status(torch.cuda.current_stream().cuda_stream) == 0
        monkeypatch.setattr(_lib, "load", lambda: normal)
        return call()
    yield run
    torch.cuda.empty_cache()


def normal(seed, *shape):
    g = torch.Generator(DEV).manual_seed(seed)
    return torch.randn(*shape, generator=g, device=DEV, dtype=torch.float32).to(BF) if torch.Size(shape).numel() < 1 << 30 \
        else torch.stack([torch.randn(*shape[1:], generator=g, device=DEV, dtype=BF) for _ in range(shape[0])])


def test_rotary_past_2_31_elements(both):
    S, axes = (1 << 23) + 5, (16, 56, 56)
    x = normal(1, 2, 1, S, 128)
    assert x.numel() > 1 << 31
    pos = torch.stack([torch.arange(S, device=DEV) // 4096, torch.arange(S, device=DEV) % 64,
                       torch.arange(S, device=DEV) // 64 % 64], -1).float()
    for interleaved in (True, False):
        y = both(lambda: cp.rotary(x, pos, axes, interleaved=interleaved))
        for at in (0, S // 2, S - 50):
            rows = slice(at, at + 50)
            want, mag = plain.rotary(x[:, :, rows], pos[rows], axes, interleaved=interleaved)
            assert plain.worst(y[:, :, rows], want, plain.rotary_tolerance(want, mag, BF)) <= 1.0


def test_few_queries_over_states_past_2_31_elements(both):
    S = (1 << 23) + 77
    k, v = normal(2, 1, 2, S, 128), normal(3, 1, 2, S, 128)
    assert k.numel() > 1 << 31
    q = normal(4, 1, 4, 1, 128)
    out, lse = both(lambda: cp.cross_attention(q, k, v))
    for h in (0, 3):
        s = torch.cat([k[0, h // 2, i:i + (1 << 20)].double() @ q[0, h, 0].double()
                       for i in range(0, S, 1 << 20)]) * 128 ** -0.5
        want_lse = torch.logsumexp(s, 0)
        p = torch.exp(s - want_lse)
        want = sum(p[i:i + (1 << 20)] @ v[0, h // 2, i:i + (1 << 20)].double() for i in range(0, S, 1 << 20))
        mag = sum(p[i:i + (1 << 20)] @ v[0, h // 2, i:i + (1 << 20)].double().abs() for i in range(0, S, 1 << 20))
        # bf16: the probabilities' and the output's rounding; fp32: a part's sum
        # of S / splits terms in lanes of 2^14 at most
        tol = 2.0 ** -8 * (want.abs() + mag) + 2.0 ** -10 * mag
        assert float(((out[0, h, 0].double() - want).abs() / tol).max()) <= 1.0
        assert abs(float(lse[0, h, 0].double() - want_lse)) <= 2.0 ** -10


def test_queries_past_2_31_elements(both):
    M, N, D = (1 << 23) + 131, 70, 128
    q, dout = normal(5, 2, 1, M, D), normal(6, 2, 1, M, D)
    assert q.numel() > 1 << 31
    k, v = normal(7, 2, 1, N, D), normal(8, 2, 1, N, D)
    n = torch.tensor((70, 33), dtype=torch.int32, device=DEV)
    out, lse = both(lambda: cp.cross_attention(q, k, v, kv_lengths=n))
    dq, dk, dv = both(lambda: cp.cross_attention_backward(q, k, v, out, lse, dout, kv_lengths=n))
    for at in (0, M // 2, M - 200):
        rows = slice(at, at + 200)
        want = plain.cross(q[:, :, rows], k, v, (70, 33), dout=dout[:, :, rows])
        for name, got in (("out", out), ("lse", lse), ("dq", dq)):
            assert plain.worst(got[:, :, rows], *want[name]) <= 1.0
    for b, keys in enumerate((70, 33)):
        wk, wv, mk, mv = (torch.zeros(keys, D, dtype=torch.float64, device=DEV) for _ in range(4))
        for i in range(0, M, 1 << 20):
            Q, G = q[b, 0, i:i + (1 << 20)].double(), dout[b, 0, i:i + (1 << 20)].double()
            p = torch.exp(Q @ k[b, 0, :keys].double().T * D ** -0.5 - lse[b, 0, i:i + (1 << 20), None].double())
            ds = p * (G @ v[b, 0, :keys].double().T - (G * out[b, 0, i:i + (1 << 20)].double()).sum(-1, keepdim=True))
            wk += ds.T @ Q * D ** -0.5
            wv += p.T @ G
            mk += ds.abs().T @ Q.abs() * D ** -0.5
            mv += p.T @ G.abs()
        # each term rounded to bf16 once (2^-8), the result once; sums of M terms
        # in fp32 drift by some sqrt(M) 2^-24 of the terms' sizes
        for got, want, mag in ((dk, wk, mk), (dv, wv, mv)):
            tol = 2.0 ** -8 * (want.abs() + 1.1 * mag)
            assert float(((got[b, 0, :keys].double() - want).abs() / tol).max()) <= 1.0
        assert torch.all(dk[b, 0, keys:] == 0) and torch.all(dv[b, 0, keys:] == 0)
