"""Memory that a call with stream= takes from PyTorch's allocator: never a block
that the caller's stream has freed and may still read, and never given out again
while the caller's stream still reads a result."""
import gc

import pytest
import torch

import context_attention_partial_gb300 as cp

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF = torch.bfloat16
AXES = (16, 56, 56)


def normal(seed, *shape):
    return torch.randn(*shape, generator=torch.Generator("cpu").manual_seed(seed)).to(BF).to(DEV)


def rotary_call():
    x, pos = normal(1, 1, 8, 2048, 128), torch.rand(2048, 3, generator=torch.Generator("cpu").manual_seed(2)).to(DEV)
    return lambda s: [cp.rotary(x, pos, AXES, stream=s)]


def rotary_call_one_given():
    x, pos = normal(1, 1, 8, 2048, 128), torch.rand(2048, 3, generator=torch.Generator("cpu").manual_seed(2)).to(DEV)
    given = torch.empty_like(x)
    return lambda s: [cp.rotary([x, x], pos, AXES, outs=[given, None], stream=s)[1]]


def cross_call():
    q, k, v = normal(3, 1, 8, 2048, 128), normal(4, 1, 8, 77, 128), normal(5, 1, 8, 77, 128)
    return lambda s: list(cp.cross_attention(q, k, v, stream=s))


def split_call():
    """Key parts, joined by way of the workspace."""
    q, k, v = normal(3, 1, 2, 1, 128), normal(4, 1, 2, 9000, 128), normal(5, 1, 2, 9000, 128)
    assert cp.cross_workspace_bytes(q, k) > 0
    return lambda s: list(cp.cross_attention(q, k, v, stream=s))


def grad_call():
    q, k, v = normal(3, 1, 8, 2048, 128), normal(4, 1, 8, 1024, 128), normal(5, 1, 8, 1024, 128)
    dout = normal(6, 1, 8, 2048, 128)
    out, lse = cp.cross_attention(q, k, v)
    return lambda s: list(cp.cross_attention_backward(q, k, v, out, lse, dout, stream=s))


CALLS = [rotary_call, rotary_call_one_given, cross_call, split_call, grad_call]


def freed_blocks(sizes):
    """Blocks of these sizes that the current stream has just freed, by address."""
    held = [torch.empty(n, dtype=torch.uint8, device=DEV) for n in sizes for _ in range(8)]
    spans = {(t.data_ptr(), t.data_ptr() + t.numel()) for t in held}
    del held
    return spans


@pytest.mark.parametrize("make", CALLS, ids=lambda f: f.__name__)
def test_results_are_not_the_current_streams_freed_blocks(make):
    call, s = make(), torch.cuda.Stream()
    torch.cuda.synchronize()
    sizes = {t.numel() * t.element_size() for t in call(s)}
    gc.collect()
    torch.cuda.synchronize()
    spans = freed_blocks(sizes)
    got = call(s)
    torch.cuda.synchronize()
    for t in got:
        assert not any(a <= t.data_ptr() < b for a, b in spans)


@pytest.mark.parametrize("make", CALLS, ids=lambda f: f.__name__)
def test_a_freed_temporary_is_read_to_its_end(make):
    """Work queued on the current stream still reads a temporary that has been
    released when the call runs on another stream."""
    call, s = make(), torch.cuda.Stream()
    torch.cuda.synchronize()
    want = call(None)
    torch.cuda.synchronize()
    sizes = [t.numel() * t.element_size() for t in want]
    held = [torch.full((n,), 0x5A, dtype=torch.uint8, device=DEV) for n in sizes for _ in range(4)]
    kept = [torch.zeros_like(t) for t in held]
    torch.cuda.synchronize()
    torch.cuda._sleep(100_000_000)
    for a, b in zip(kept, held):
        a.copy_(b)
    del held, b
    got = call(s)
    torch.cuda.synchronize()
    assert all(torch.all(t == 0x5A) for t in kept)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert cp.last_device_status() == 0


@pytest.mark.parametrize("make", CALLS, ids=lambda f: f.__name__)
def test_a_released_result_is_read_to_its_end(make):
    """The caller's stream still reads a result that has been released when the
    next call runs on the other stream."""
    call, s = make(), torch.cuda.Stream()
    torch.cuda.synchronize()
    want = call(None)
    kept = [torch.zeros_like(t) for t in want]
    torch.cuda.synchronize()
    got = call(s)
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda._sleep(100_000_000)
    for a, b in zip(kept, got):
        a.copy_(b)
    del got, b
    again = call(s)
    with torch.cuda.stream(s):
        for t in again:
            t.zero_()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(kept, want))
    assert cp.last_device_status() == 0


@pytest.mark.parametrize("make", CALLS, ids=lambda f: f.__name__)
def test_a_call_leaves_the_current_stream_as_it_was(make):
    call, s, other = make(), torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(other):
        got = call(s)
        assert torch.cuda.current_stream() == other
        same = call(other)                     # the current stream, named
    assert torch.cuda.current_stream() == torch.cuda.default_stream()
    named = call(torch.cuda.default_stream())
    torch.cuda.synchronize()
    for a, b, c in zip(got, same, named):
        assert torch.equal(a, b) and torch.equal(a, c)


def older_calls():
    """The attention, merge and regroup calls by name, each on tensors of its own."""
    q, k, v = (normal(7 + i, 1, 4, 1024, 64) for i in range(3))
    x = normal(10, 1, 1024, 4, 64)
    grouped = cp.ulysses_permute(x, 2, 1)
    uneven = cp.ulysses_anything_permute(x, 3, 1).zero_()
    cp.ulysses_anything_permute(x, 3, 1, out=uneven)

    def prepared(make, s):
        call = make(s)
        call()
        return [call.out]

    return {
        "partial": lambda s: list(cp.partial(q, k, v, stream=s)),
        "ring": lambda s: list(cp.ring(q, k, v, 2, stream=s)),
        "ring_noalloc": lambda s: list(cp.ring_noalloc(q, k, v, 2, stream=s)),
        "prepare_ring": lambda s: prepared(lambda s: cp.prepare_ring(q, k, v, 2, stream=s), s),
        "permute": lambda s: [cp.ulysses_permute(x, 2, 1, stream=s), cp.ulysses_permute(grouped, 2, -1, stream=s)],
        "permute_batch": lambda s: cp.ulysses_permute_batch([x, x], 2, 1, stream=s),
        "unified": lambda s: list(cp.unified_attention(x, x, x, 2, 2, stream=s)),
        "prepare_unified": lambda s: prepared(lambda s: cp.prepare_unified(x, x, x, 2, 2, stream=s), s),
        "anything_permute": lambda s: [cp.ulysses_anything_permute(uneven, 3, -1, heads=4, stream=s)],
        "anything_permute_batch": lambda s: cp.ulysses_anything_permute_batch([uneven, uneven], 3, -1, heads=4, stream=s),
        "anything": lambda s: [cp.ulysses_anything_attention(x, x, x, 3, stream=s)[0]],
        "prepare_anything": lambda s: prepared(lambda s: cp.prepare_ulysses_anything(x, x, x, 3, stream=s), s),
    }


OLDER = ("partial", "ring", "ring_noalloc", "prepare_ring", "permute", "permute_batch", "unified", "prepare_unified",
         "anything_permute", "anything_permute_batch", "anything", "prepare_anything")


@pytest.mark.parametrize("name", OLDER)
def test_older_calls_results_are_not_the_current_streams_freed_blocks(name):
    test_results_are_not_the_current_streams_freed_blocks(lambda: older_calls()[name])


@pytest.mark.parametrize("name", OLDER)
def test_older_calls_read_a_freed_temporary_to_its_end(name):
    test_a_freed_temporary_is_read_to_its_end(lambda: older_calls()[name])


@pytest.mark.parametrize("name", OLDER)
def test_older_calls_read_a_released_result_to_its_end(name):
    test_a_released_result_is_read_to_its_end(lambda: older_calls()[name])


@pytest.mark.parametrize("make", [rotary_call, cross_call, split_call, grad_call], ids=lambda f: f.__name__)
def test_a_named_stream_inside_a_capture(make):
    """A captured graph that forks to the call's stream and joins it again; what the
    call allocates is the graph's own, and results may be released in it."""
    call, side = make(), torch.cuda.Stream()
    want = call(None)
    call(side)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        main = torch.cuda.current_stream()
        side.wait_stream(main)
        call(side)                              # (released at once)
        got = call(side)
        main.wait_stream(side)
        kept = [t.clone() for t in got]
    for _ in range(2):
        for t in kept:
            t.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(kept, want))
    assert cp.last_device_status() == 0
