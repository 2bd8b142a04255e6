"""Failure path of the cross-attention kernels, without faulting the GPU: a
host-set flag makes the TMA producers skip their copies, so every bounded
wait (short limit here) runs out.  The kernels return on their own and the
device error word says so; the next normal calls are correct."""
import pytest
import torch

import context_attention_partial_gb300 as cp
import plain_operators as plain

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
TIMEOUT = 9


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("queries,keys", [(300, 333), (100, 333), (100, 1300)])
def test_stalled_producers_time_out_and_recover(d, queries, keys):
    lib = cp.load_library()
    g = torch.Generator("cpu").manual_seed(71)
    q, k, v, dout = (torch.randn(2, 3, s, d, generator=g).to(torch.bfloat16).to(DEV)
                     for s in (queries, keys, keys, queries))
    lengths = torch.tensor((keys, 140), dtype=torch.int32, device=DEV)
    out, lse = cp.cross_attention(q, k, v, kv_lengths=lengths)
    grads = cp.cross_attention_backward(q, k, v, out, lse, dout, kv_lengths=lengths)
    assert cp.last_device_status() == 0
    try:
        cp.set_wait_timeout_ns(20_000_000)          # 20 ms
        lib.cpattn_set_fault_injection(1)
        cp.cross_attention(q, k, v, kv_lengths=lengths)
        assert cp.last_device_status() == TIMEOUT
        assert cp.last_device_status() == 0          # the word was cleared
        cp.cross_attention_backward(q, k, v, out, lse, dout, kv_lengths=lengths)
        assert cp.last_device_status() == TIMEOUT
        assert cp.last_device_status() == 0
    finally:
        lib.cpattn_set_fault_injection(0)
        cp.set_wait_timeout_ns(2_000_000_000)
    out2, lse2 = cp.cross_attention(q, k, v, kv_lengths=lengths)
    assert torch.equal(out2, out) and torch.equal(lse2, lse)
    for a, b in zip(cp.cross_attention_backward(q, k, v, out, lse, dout, kv_lengths=lengths), grads):
        assert torch.equal(a, b)
    assert cp.last_device_status() == 0
    want = plain.cross(q, k, v, (keys, 140), dout=dout)
    for name, got in zip(("out", "lse", "dq", "dk", "dv"), (out, lse, *grads)):
        assert plain.worst(got, *want[name]) <= 1.0


@pytest.mark.parametrize("d", [64, 128])
def test_waits_do_not_count_the_kernel_before(d):
    """One query tile over a million keys: dq alone takes some 8 ms, and the blocks
    of dk and dv that start beside it wait for its end longer than a wait's limit."""
    g = torch.Generator("cpu").manual_seed(72)
    q, dout = (torch.randn(1, 1, 100, d, generator=g).to(torch.bfloat16).to(DEV) for _ in range(2))
    k, v = (torch.randn(1, 1, 1 << 20, d, device=DEV, generator=torch.Generator(DEV).manual_seed(s)).to(torch.bfloat16)
            for s in (73, 74))
    out, lse = cp.cross_attention(q, k, v)
    want = cp.cross_attention_backward(q, k, v, out, lse, dout)
    assert cp.last_device_status() == 0
    try:
        cp.set_wait_timeout_ns(3_000_000)           # 3 ms
        got = cp.cross_attention_backward(q, k, v, out, lse, dout)
        assert cp.last_device_status() == 0
    finally:
        cp.set_wait_timeout_ns(2_000_000_000)
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    e = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    e[0].record()
    cp.cross_attention_backward(q, k, v, out, lse, dout)
    e[1].record()
    torch.cuda.synchronize()
    assert e[0].elapsed_time(e[1]) > 6               # (dq's walk is longer than the limit)
