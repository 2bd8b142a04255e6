"""The rotary and cross-attention calls at the ends of their ranges: very many
sequences or heads, very many query heads on one key head, threads that call at
once, inference tensors, outputs given in part."""
import threading

import pytest
import torch

import context_attention_partial_gb300 as cp
import plain_operators as plain
from context_attention_partial_gb300 import _lib
from context_attention_partial_gb300 import build as _build

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture
def both(monkeypatch):
    """Runs a call through the check build, then through the normal one: equal bits."""
    chk, normal = _lib.bind(_build.build(check=True)), cp.load_library()

    def run(call):
        monkeypatch.setattr(_lib, "load", lambda: chk)
        checked = call()
        assert chk.cpattn_last_device_status(torch.cuda.current_stream().cuda_stream) == 0
        monkeypatch.setattr(_lib, "load", lambda: normal)
        got = call()
        assert cp.last_device_status() == 0
        assert all(torch.equal(a, b) for a, b in zip(got, checked))
        return got
    return run


def normal(seed, *shape, dtype=BF):
    return torch.randn(*shape, generator=torch.Generator(DEV).manual_seed(seed), device=DEV).to(dtype)


def batched(q, k, v, dout):
    """The 64-bit form over all heads at once (few keys), each result with what its
    terms add up to in magnitude."""
    g, scale = q.shape[1] // k.shape[1], q.shape[3] ** -0.5
    Q, K, V, G = (t.double() for t in (q, k.repeat_interleave(g, 1), v.repeat_interleave(g, 1), dout))
    p = (Q @ K.mT * scale).softmax(-1)
    o = p @ V
    ds = p * (G @ V.mT - (G * o).sum(-1, keepdim=True))
    # ds: p and ds rounded, and delta from the rounded output
    e = 2 * ds.abs() + p * ((G.abs() * (o.abs() + p @ V.abs())).sum(-1, keepdim=True))
    shared = lambda t: t.unflatten(1, (-1, g)).sum(2)
    return {"out": (o, p @ V.abs()), "dq": (ds @ K * scale, e @ K.abs() * scale),
            "dk": (shared(ds.mT @ Q) * scale, shared(e.mT @ Q.abs()) * scale), "dv": (shared(p.mT @ G), shared(p.mT @ G.abs()))}


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("B,H,Hk,M,N", [(65535, 1, 1, 1, 3), (1, 65535, 65535, 2, 5), (2, 30000, 3, 1, 70), (9000, 2, 1, 40, 2),
                                        (1, 4096, 1, 3, 40)])
def test_very_many_sequences_or_heads(both, B, H, Hk, M, N, dtype):
    q, dout = normal(1, B, H, M, 64, dtype=dtype), normal(2, B, H, M, 64, dtype=dtype)
    k, v = normal(3, B, Hk, N, 64, dtype=dtype), normal(4, B, Hk, N, 64, dtype=dtype)

    def call():
        out, lse = cp.cross_attention(q, k, v)
        return (out, *cp.cross_attention_backward(q, k, v, out, lse, dout))

    got = both(call)
    # a rounding of each term and of the result (bf16); fp32: the scores' and the
    # sums' roundings, below 200 + the sum's length
    u = 2.0 ** -8 if dtype == BF else 0.0
    terms = {"out": N, "dq": N, "dk": M * H // Hk, "dv": M * H // Hk}
    for (name, (want, mag)), x in zip(batched(q, k, v, dout).items(), got):
        tol = (u + (300 + terms[name]) * 2.0 ** -24) * (want.abs() + mag) * 1.05 + 1e-30
        assert plain.worst(x, want, tol) <= 1.0, name


def test_rotary_of_very_many_sequences(both):
    x = normal(5, 65535, 2, 1, 64)
    pos = torch.arange(65535, device=DEV).float().view(-1, 1, 1)
    y, = both(lambda: cp.rotary([x], pos, (64,)))
    want, mag = plain.rotary(x, pos, (64,))
    assert plain.worst(y, want, plain.rotary_tolerance(want, mag, BF)) <= 1.0


def test_threads_that_call_at_once():
    """Four threads, each on a stream of its own, many small calls: every result is
    the single call's."""
    def work(seed):
        q, k, v, dout = (normal(seed + i, 1, 4, s, 64) for i, s in enumerate((60, 90, 90, 60)))
        pos = torch.arange(60, device=DEV).float()[:, None]

        def step():
            rq = cp.rotary(q, pos, (64,))
            out, lse = cp.cross_attention(rq, k, v)
            return (rq, out, lse, *cp.cross_attention_backward(rq, k, v, out, lse, dout))
        return step

    steps = [work(10 * i) for i in range(4)]
    want = [s() for s in steps]
    torch.cuda.synchronize()
    bad = []

    def run(i):
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(50):
                got = steps[i]()
                torch.cuda.current_stream().synchronize()
                if not all(torch.equal(a, b) for a, b in zip(got, want[i])):
                    bad.append(i)

    threads = [threading.Thread(target=run, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad and cp.last_device_status() == 0


def test_inference_tensors_parameters_and_outputs_in_part():
    q, k, v, dout = (normal(20 + i, 2, 4, s, 64) for i, s in enumerate((60, 90, 90, 60)))
    pos = torch.arange(60, device=DEV).float()[:, None]
    rq = cp.rotary(q, pos, (64,))
    out, lse = cp.cross_attention(rq, k, v)
    want = cp.cross_attention_backward(rq, k, v, out, lse, dout)
    with torch.inference_mode():
        o, l = cp.cross_attention(cp.rotary(q.clone(), pos, (64,)), k.clone(), v)
        got = cp.cross_attention_backward(rq, k, v, o, l, dout.clone())
    assert torch.equal(o, out) and torch.equal(l, lse) and all(torch.equal(a, b) for a, b in zip(got, want))
    with torch.no_grad():
        o, _ = cp.cross_attention(torch.nn.Parameter(rq), torch.nn.Parameter(k), v)
    assert torch.equal(o, out)
    dk = torch.empty_like(k)
    got = cp.cross_attention_backward(rq, k, v, out, lse, dout, dk=dk)
    assert got[1].data_ptr() == dk.data_ptr() and all(torch.equal(a, b) for a, b in zip(got, want))
    l = torch.empty_like(lse)
    got = cp.cross_attention(rq, k, v, lse=l)
    assert got[1].data_ptr() == l.data_ptr() and torch.equal(got[0], out) and torch.equal(l, lse)
