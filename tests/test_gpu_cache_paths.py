"""The norm and paged-cache calls where they could go wrong: the bounds-checking build,
waits that run out, captured steps whose lengths change, streams and threads, tensors
past 2^31 elements, many sequences, views, and random sizes."""
import math
import os
import random
import subprocess
import sys
import threading

import pytest
import torch

import context_attention_partial_gb300 as cp
import plain_cache as C
import plain_operators as P
import test_gpu_operator_streams as streams
from context_attention_partial_gb300 import _lib
from context_attention_partial_gb300 import build as _build
from test_gpu_cache import bits, check, randn

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32
OK, TIMEOUT, BOUNDS = 0, 9, 10
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def ints(*xs):
    return torch.tensor(xs, dtype=torch.int32, device=DEV)


def attend(cache, q, parents=None, **kw):
    pt = None if parents is None else parents.to(torch.int32).to(DEV)
    return cp.cache_attention(q, cache.key_pages, cache.value_pages, cache.table, cache.lengths_t, parents=pt,
                              counts=cache.counts_t, **kw)


def verify(cache, q, got, parents=None, scale=None):
    want = C.attend(q, cache.k, cache.v, cache.lengths, cache.counts, None if parents is None else parents.tolist(), scale)
    check(got[0], want[0])
    check(got[1], want[1])


# ------------------------------------------------------------- check build
@pytest.fixture(scope="module")
def chk():
    lib = _lib.bind(_build.build(check=True))
    yield lib
    lib.cpattn_set_check_shrink(0)


@pytest.fixture
def through(monkeypatch):
    return lambda lib: monkeypatch.setattr(_lib, "load", lambda: lib)


def status(lib):
    return lib.cpattn_last_device_status(torch.cuda.current_stream().cuda_stream)


ATTEND = [(4, 4, 1, 128, 16, (0, 5), None), (8, 2, 1, 64, 64, (700, 3), (1, 0)), (8, 1, 4, 128, 32, (1000, 130), (4, 2)),
          (4, 2, 27, 128, 16, (2100, 40, 127), (27, 1, 20)), (2, 1, 200, 64, 256, (300, 0), (200, 131)),
          (160, 1, 2, 64, 16, (90,), None), (12, 4, 70, 128, 64, (130, 500), (70, 66))]


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("case", ATTEND, ids=lambda c: "x".join(map(str, c[:5])))
def test_attention_check_build_clean_and_equal(chk, through, case, dtype):
    H, Hk, S, D, page, lengths, counts = case
    cache = C.Cache(lengths, counts, S, Hk, D, page, dtype, DEV, 1)
    q = randn(len(lengths), H, S, D, dtype=dtype, seed=2)
    normal = cp.load_library()
    for parents in (None, C.tree(S, len(lengths))):
        through(chk)
        got = attend(cache, q, parents)
        assert status(chk) == OK
        through(normal)
        want = attend(cache, q, parents)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        verify(cache, q, got, parents)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("interleaved", [True, False])
def test_norm_and_append_check_build_clean_and_equal(chk, through, interleaved, dtype):
    normal = cp.load_library()
    for B, H, Hk, S, D, axes in ((1, 3, 1, 33, 128, (16, 56, 56)), (2, 2, 2, 1, 64, (64,)), (3, 5, 2, 17, 24, (8, 8)),
                                 (1, 9, 1, 5, 256, (256,))):
        q, k = randn(B, H, S, D, dtype=dtype, seed=3), randn(B, Hk, S, D, dtype=dtype, seed=4)
        w = [1 + 0.1 * randn(D, dtype=F32, seed=5)] * 2
        pos = torch.rand(B, S, len(axes), generator=torch.Generator().manual_seed(6)).to(DEV) * 100
        cache = C.Cache([7] * B, None, S, Hk, D, 16, dtype, DEV, 7)

        def call():
            y = cp.norm_rotary([q, k], w, pos, axes, interleaved=interleaved)
            dx, dw = cp.norm_rotary_backward([q, k], w, pos, axes, y, interleaved=interleaved)
            r = cp.cache_append(k, k, cache.key_pages, cache.value_pages, cache.table, cache.lengths_t, positions=pos,
                                axes_dims=axes, q=q, weight=w[0], q_weight=w[1], interleaved=interleaved)
            return [*y, *dx, *dw, r, bits(cache.key_pages).clone(), bits(cache.value_pages).clone()]

        through(chk)
        got = call()
        assert status(chk) == OK
        through(normal)
        assert all(torch.equal(a, b) for a, b in zip(got, call()))


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("S", [1, 30, 300])
def test_check_build_reports_short_outputs(chk, through, S, dtype):
    cache = C.Cache([400], None, S, 2, 64, 16, dtype, DEV, 1, extra=0)
    q, k = randn(1, 4, S, 64, dtype=dtype, seed=2), randn(1, 2, S, 64, dtype=dtype, seed=3)
    pos, w = torch.zeros(S, 1, device=DEV), torch.ones(64, device=DEV)
    normal = cp.load_library()
    want = attend(cache, q)
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
    short(lambda: attend(cache, q, out=out), (out,))
    short(lambda: attend(cache, q, lse=lse), (lse,))
    y, dw = torch.empty_like(q), torch.empty(64, device=DEV)
    short(lambda: cp.norm_rotary(q, w, pos, (64,), outs=y), (y,))
    short(lambda: cp.norm_rotary_backward(q, w, pos, (64,), q, dxs=y, dweights=dw), (y, dw))
    short(lambda: cp.cache_append(k, k, cache.key_pages, cache.value_pages, cache.table, cache.lengths_t, q=q, q_out=y), (y,))
    # a pool of one page, whose last row is written
    pages = torch.empty(1, 2, 16, 64, dtype=dtype, device=DEV), torch.empty(1, 2, 16, 64, dtype=dtype, device=DEV)
    short(lambda: cp.cache_append(k[:, :, :1], k[:, :, :1], *pages, ints(0).view(1, 1), ints(15)), pages)
    through(normal)
    cache.write(0, 0, cache.k[0], cache.v[0])   # (k went to the cache)
    assert all(torch.equal(a, b) for a, b in zip(attend(cache, q), want))


# ------------------------------------------------------------------- waits
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("H,S,tree", [(4, 20, True), (8, 60, False), (8, 300, False)])
def test_stalled_producers_time_out_and_recover(H, S, tree, d):
    lib = cp.load_library()
    cache = C.Cache([1300, 20, 0], [S, S, 3], S, 2, d, 32, BF, DEV, 4)
    q = randn(3, H, S, d, dtype=BF, seed=5)
    parents = C.tree(S, 3) if tree else None
    want = attend(cache, q, parents)
    assert cp.last_device_status() == OK
    try:
        cp.set_wait_timeout_ns(20_000_000)          # 20 ms
        lib.cpattn_set_fault_injection(1)
        attend(cache, q, parents)
        assert cp.last_device_status() == TIMEOUT
        assert cp.last_device_status() == OK
    finally:
        lib.cpattn_set_fault_injection(0)
        cp.set_wait_timeout_ns(2_000_000_000)
    got = attend(cache, q, parents)
    assert cp.last_device_status() == OK
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    verify(cache, q, got, parents)


# ------------------------------------------- graphs, streams, threads
@pytest.mark.parametrize("S", [1, 12])
@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_a_captured_step_follows_the_lengths(dtype, S):
    """One captured step (append, attend) replayed as the sequences grow over tiles and pages."""
    B, H, Hk, D, page = 2, 8, 2, 64, 16
    table = torch.arange(2 * 40, device=DEV).to(torch.int32).view(2, 40)
    pools = [torch.full((80, Hk, page, D), math.nan, dtype=dtype, device=DEV) for _ in range(2)]
    lengths, pos = ints(0, 100), torch.zeros(B, S, 1, device=DEV)
    q, k, v = (torch.zeros(B, h, S, D, dtype=dtype, device=DEV) for h in (H, Hk, Hk))
    first = randn(1, Hk, 100, D, dtype=dtype, seed=1)
    cp.cache_append(first, first, *pools, table[1:], ints(0))

    def step():
        r = cp.cache_append(k, v, *pools, table, lengths, positions=pos, axes_dims=(D,), q=q)
        out = cp.cache_attention(r, *pools, table, lengths)
        lengths.add_(S)
        return (r, *out)

    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r, out, lse = step()
    keys = [torch.zeros(Hk, 0, D, dtype=dtype, device=DEV), first[0]]
    values = [torch.zeros(Hk, 0, D, dtype=dtype, device=DEV), first[0]]
    for i in range(20):
        for t, h, seed in ((q, H, 10), (k, Hk, 11), (v, Hk, 12)):
            t.copy_(randn(B, h, S, D, dtype=dtype, seed=seed + 100 * i))
        pos.copy_((lengths[:, None] + torch.arange(S, device=DEV)).float().unsqueeze(-1))
        before = lengths.tolist()
        graph.replay()
        torch.cuda.synchronize()
        new = []
        for b in range(B):   # (as the pages hold them)
            at = torch.arange(before[b], before[b] + S, device=DEV)
            new.append(pools[0][table[b].long()[at // page], :, at % page].transpose(0, 1))
        check(torch.stack(new), C.norm_rotary(k, None, pos, (D,), norm=False))
        check(r, C.norm_rotary(q, None, pos, (D,), norm=False))
        keys = [torch.cat([keys[b], new[b]], 1) for b in range(B)]
        values = [torch.cat([values[b], v[b]], 1) for b in range(B)]
        want = C.attend(r, keys, values, before, [S, S])
        check(out, want[0])
        check(lse, want[1])
    assert cp.last_device_status() == OK


def norm_call():
    x, pos = streams.normal(1, 1, 8, 2048, 128), torch.rand(2048, 3, generator=torch.Generator("cpu").manual_seed(2)).to(DEV)
    w = torch.ones(128, device=DEV)
    return lambda s: [cp.norm_rotary(x, w, pos, streams.AXES, stream=s)]


def norm_grad_call():
    x, pos = streams.normal(1, 1, 8, 2048, 128), torch.rand(2048, 3, generator=torch.Generator("cpu").manual_seed(2)).to(DEV)
    w = torch.ones(128, device=DEV)

    def call(s):
        dx, dw = cp.norm_rotary_backward(x, w, pos, streams.AXES, x, stream=s)
        return [dx, dw]
    return call


def append_call():
    cache = C.Cache([5], None, 200, 8, 128, 16, BF, DEV, 1)
    k, q = streams.normal(3, 1, 8, 200, 128), streams.normal(4, 1, 32, 200, 128)
    return lambda s: [cp.cache_append(k, k, cache.key_pages, cache.value_pages, cache.table, cache.lengths_t, q=q, stream=s)]


def split_call():
    """Key parts, joined by way of the workspace."""
    cache = C.Cache([9000], None, 1, 2, 128, 16, BF, DEV, 1)
    q = streams.normal(3, 1, 4, 1, 128)
    assert cp.cache_attention_workspace_bytes(q, cache.key_pages, cache.table) > 0
    return lambda s: list(attend(cache, q, stream=s))


def rows_call():
    cache = C.Cache([900, 20], None, 64, 2, 128, 16, BF, DEV, 1)
    q = streams.normal(3, 2, 8, 64, 128)
    return lambda s: list(attend(cache, q, stream=s))


CALLS = [norm_call, norm_grad_call, append_call, split_call, rows_call]


@pytest.mark.parametrize("make", CALLS, ids=lambda f: f.__name__)
@pytest.mark.parametrize("test", [streams.test_results_are_not_the_current_streams_freed_blocks,
                                  streams.test_a_freed_temporary_is_read_to_its_end,
                                  streams.test_a_released_result_is_read_to_its_end], ids=lambda f: f.__name__[5:])
def test_memory_of_a_given_stream(test, make):
    test(make)


def test_two_streams_at_once():
    """Calls of every kernel on two streams, each with a workspace of its own."""
    side = [torch.cuda.Stream() for _ in range(2)]
    jobs = []
    for i, (H, S, D, dtype) in enumerate(((8, 1, 128, BF), (8, 40, 64, BF), (8, 300, 128, BF), (4, 3, 64, F32))):
        cache = C.Cache([3000, 77], None, S, 2, D, 32, dtype, DEV, i)
        q = randn(2, H, S, D, dtype=dtype, seed=i)
        jobs.append((cache, q, attend(cache, q)))
    torch.cuda.synchronize()
    for _ in range(5):
        got = [[attend(c, q, stream=s) for c, q, _ in jobs] for s in side]
        torch.cuda.synchronize()
        for each in got:
            for a, (_, _, b) in zip(each, jobs):
                assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    assert cp.last_device_status() == OK


def test_threads():
    errors = []

    def work(seed):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                cache = C.Cache([500 + seed], None, 9, 2, 64, 16, BF, DEV, seed)
                q, w = randn(1, 8, 9, 64, dtype=BF, seed=seed), torch.ones(64, device=DEV)
                pos = torch.arange(9, device=DEV).float()[:, None]
                first = None
                for _ in range(30):
                    y = cp.norm_rotary(q, w, pos, (64,))
                    got = (*attend(cache, y), *cp.norm_rotary_backward(q, w, pos, (64,), y))
                    torch.cuda.current_stream().synchronize()
                    if first is None:
                        first = got
                        verify(cache, y, got[:2])
                    assert all(torch.equal(a, b) for a, b in zip(got, first))
        except Exception as e:   # (reported by the test's own thread)
            errors.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors


PROGRAM = """
import sys
import torch
sys.path.insert(0, "tests")
import context_attention_partial_gb300 as cp
import plain_cache as C
what, dtype = sys.argv[1], {"bf16": torch.bfloat16, "f32": torch.float32}[sys.argv[2]]
S, n = {"few": (1, 3000), "rows": (40, 300), "many": (200, 900)}[what]
cache = C.Cache([n], None, S, 2, 64, 16, dtype, "cuda:0")
q = torch.randn(1, 4, S, 64, generator=torch.Generator().manual_seed(1)).to(dtype).cuda()
pos, w = torch.arange(S, dtype=torch.float32, device="cuda")[:, None], torch.ones(64, device="cuda")

def step():
    k, v = q[:, :2], q[:, 2:]
    r = cp.cache_append(k, v, cache.key_pages, cache.value_pages, cache.table, cache.lengths_t, positions=pos,
                        axes_dims=(64,), q=q, weight=w, q_weight=w)
    out, lse = cp.cache_attention(r, cache.key_pages, cache.value_pages, cache.table, cache.lengths_t)
    return [r, out, lse, cp.norm_rotary(q, w, pos, (64,), interleaved=False), *cp.norm_rotary_backward(q, w, pos, (64,), out)]

torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    got = step()
graph.replay()
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(got, step()))
assert cp.last_device_status() == 0
"""


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("what", ["few", "rows", "many"])
def test_first_call_in_a_capture(what, dtype):
    p = subprocess.run([sys.executable, "-c", PROGRAM, what, dtype], cwd=ROOT, capture_output=True, text=True, timeout=120)
    assert p.returncode == 0, p.stderr[-2000:]


# ---------------------------------------------------------- sizes, views
@pytest.mark.slow
@pytest.mark.parametrize("layout", ["phrd", "prhd"])
def test_pool_past_2_31_elements(layout):
    """Tokens in pages far apart in a pool of more than 2^31 elements."""
    Hk, R, D, pages = 8, 128, 128, (1 << 14) + 3
    shape = (pages, Hk, R, D) if layout == "phrd" else (pages, R, Hk, D)
    pools = [torch.zeros(shape, dtype=BF, device=DEV) for _ in range(2)]
    assert pools[0].numel() > 1 << 31
    if layout != "phrd":
        pools = [x.transpose(1, 2) for x in pools]
    far = [pages - 1, 5, pages - 2, pages // 2]
    table = torch.tensor([far], dtype=torch.int32, device=DEV)
    k, v = randn(1, Hk, 400, D, dtype=BF, seed=1), randn(1, Hk, 400, D, dtype=BF, seed=2)
    cp.cache_append(k, v, *pools, table, ints(0))
    assert cp.last_device_status() == OK
    for i, x in ((0, k), (1, v)):
        got = pools[i][table[0].long()].transpose(0, 1).reshape(Hk, -1, D)[:, :400]
        assert torch.equal(got, x[0])
    for H, S in ((8, 1), (32, 30), (16, 200)):
        q = randn(1, H, S, D, dtype=BF, seed=3)
        got = cp.cache_attention(q, *pools, table, ints(400 - S))
        want = C.attend(q, [k[0]], [v[0]], [400 - S], [S])
        check(got[0], want[0])
        check(got[1], want[1])
    assert cp.last_device_status() == OK
    del pools
    torch.cuda.empty_cache()


@pytest.mark.slow
def test_norm_past_2_31_elements():
    S, axes = (1 << 23) + 5, (16, 56, 56)
    x = torch.cat([torch.randn(2, 1, 1 << 20, 128, device=DEV, generator=torch.Generator(DEV).manual_seed(i)).to(BF)
                   for i in range(9)], 2)[:, :, :S]
    assert x.numel() > 1 << 31
    at = torch.arange(S, device=DEV)
    pos = torch.stack([at // 4096, at % 64, at // 64 % 64], -1).float()
    w = 1 + 0.1 * randn(128, dtype=F32, seed=1)
    y = cp.norm_rotary(x, w, pos, axes)
    dx, dw = cp.norm_rotary_backward(x, w, pos, axes, y)
    for first in (0, S // 2, S - 50):
        rows = slice(first, first + 50)
        check(y[:, :, rows], C.norm_rotary(x[:, :, rows], w, pos[rows], axes))
        check(dx[:, :, rows], C.norm_rotary_backward(x[:, :, rows], w, pos[rows], axes, y[:, :, rows])[0])
    # dy = y: a row's dz is w n up to y's rounding, so dw = sum of w n^2, of 2^24 rows, each
    # term off by 2^-8; fp32 sums of 2^14 rows a thread at most
    want = sum((x[:, :, i:i + (1 << 20)].double().square() / x[:, :, i:i + (1 << 20)].double().square().mean(-1, keepdim=True))
               .sum((0, 1, 2)) for i in range(0, S, 1 << 20)) * w.double()
    assert float(((dw.double() - want).abs() / want.abs()).max()) <= 2.0 ** -8
    del x, y, dx
    torch.cuda.empty_cache()


@pytest.mark.parametrize("H,S,dtype", [(2, 1, BF), (4, 20, BF), (2, 140, BF), (2, 2, F32)])
def test_many_sequences(H, S, dtype):
    """More units than are split, with empty ones among them, and a few long ones."""
    B = 1500
    rng = random.Random(1)
    lengths = [rng.randint(0, 40) if i % 300 else 700 for i in range(B)]
    counts = [0 if i % 7 == 3 else rng.randint(1, S) for i in range(B)]
    cache = C.Cache(lengths, counts, S, 2, 64, 16, dtype, DEV, 2)
    q = randn(B, H, S, 64, dtype=dtype, seed=3)
    out, lse = attend(cache, q)
    assert cp.last_device_status() == OK
    pick = list(range(0, B, 97)) + [300, 600, 3, 10]
    want = C.attend(q[pick], [cache.k[b] for b in pick], [cache.v[b] for b in pick], [lengths[b] for b in pick],
                    [counts[b] for b in pick])
    check(out[pick], want[0])
    check(lse[pick], want[1])
    for b in range(3, B, 7):
        assert counts[b] == 0
    none = torch.tensor([c == 0 for c in counts], device=DEV)
    assert torch.all(out[none] == 0) and torch.all(lse[none] == -math.inf)


@pytest.mark.parametrize("interleaved", [True, False])
@pytest.mark.parametrize("S", [1, 3])
def test_norm_and_append_of_many_sequences(S, interleaved):
    """Sequences shorter than a block's tokens: one token each, and three."""
    B, D = 5000, 64
    x, k = randn(B, 2, S, D, dtype=BF, seed=1), randn(B, 1, S, D, dtype=BF, seed=2)
    pos = torch.randint(0, 4000, (B, S, 1), generator=torch.Generator().manual_seed(3)).float().to(DEV)
    w = 1 + 0.1 * randn(D, dtype=BF, seed=4)
    kw = dict(interleaved=interleaved)
    check(cp.norm_rotary(x, w, pos, (D,), **kw), C.norm_rotary(x, w, pos, (D,), **kw))
    dx, dw = cp.norm_rotary_backward(x, w, pos, (D,), x, **kw)
    a, b = C.norm_rotary_backward(x, w, pos, (D,), x, **kw)
    check(dx, a)
    check(dw, b)
    pools = [torch.zeros(B, 1, 16, D, dtype=BF, device=DEV) for _ in range(2)]
    table = torch.randperm(B, generator=torch.Generator().manual_seed(5)).view(B, 1).to(torch.int32).to(DEV)
    at = torch.randint(0, 13, (B,), generator=torch.Generator().manual_seed(6)).to(torch.int32).to(DEV)
    q = cp.cache_append(k, k, *pools, table, at, positions=pos, axes_dims=(D,), q=x, weight=w, q_weight=w, **kw)
    check(q, C.norm_rotary(x, w, pos, (D,), **kw))
    rows = at.long()[:, None] + torch.arange(S, device=DEV)
    got = [p[table.long(), 0, rows].unsqueeze(1) for p in pools]
    check(got[0], C.norm_rotary(k, w, pos, (D,), **kw))
    assert torch.equal(got[1], k)
    for p in pools:
        p[table.long(), 0, rows] = 0
        assert torch.all(p == 0)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("S", [1, 33, 150])
def test_views_of_fused_projections(S, dtype):
    B, H, Hk, D = 2, 8, 2, 64
    fused = randn(B, S, (H + 2 * Hk), D, dtype=dtype, seed=1)
    q, k, v = (fused[:, :, a:b].transpose(1, 2) for a, b in ((0, H), (H, H + Hk), (H + Hk, H + 2 * Hk)))
    both = torch.full((60, 2, Hk, 16, D), math.nan, dtype=dtype, device=DEV)   # keys and values of a page together
    pools = both[:, 0], both[:, 1]
    table = torch.randperm(60, generator=torch.Generator().manual_seed(1)).view(2, 30).to(torch.int32).to(DEV)
    first = randn(B, Hk, 170, D, dtype=dtype, seed=2)
    cp.cache_append(first, first, *pools, table, ints(0, 0))
    r = cp.cache_append(k, v, *pools, table, ints(170, 170), q=q)
    assert torch.equal(r, q)
    out = torch.empty(B, S, H, D, dtype=dtype, device=DEV).transpose(1, 2)
    got, lse = cp.cache_attention(q, *pools, table, ints(170, 170), out=out)
    assert got is out
    want = C.attend(q, [torch.cat([first[b], k[b]], 1) for b in range(B)], [torch.cat([first[b], v[b]], 1) for b in range(B)],
                    [170, 170], [S, S])
    check(out, want[0])
    check(lse, want[1])


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("H,S", [(1, 1), (8, 30), (8, 100)])
def test_large_scores(H, S, dtype):
    """Scores of some hundreds, rising from tile to tile: sums are carried over by their maximum."""
    cache = C.Cache([900], None, S, 1, 64, 16, dtype, DEV, 3)
    ramp = torch.linspace(0.1, 8, 900 + S, device=DEV)[None, :, None]
    cache.k = [(cache.k[0].double() * ramp).to(dtype)]
    cache.write(0, 0, cache.k[0], cache.v[0])
    q = 8 * randn(1, H, S, 64, dtype=dtype, seed=4)
    verify(cache, q, attend(cache, q))


def test_nothing_cached_and_nothing_new():
    q = randn(2, 4, 3, 64, dtype=BF, seed=1)
    empty = torch.empty(0, 2, 16, 64, dtype=BF, device=DEV)
    table = torch.empty(2, 0, dtype=torch.int32, device=DEV)
    for S in (3, 1):
        out, lse = cp.cache_attention(q[:, :, :S], empty, empty, table, ints(0, 0), counts=ints(0, 0))
        assert torch.all(out == 0) and torch.all(lse == -math.inf)
    out, lse = cp.cache_attention(randn(2, 40, 3, 64, dtype=BF, seed=1), empty, empty, table, ints(5, 5), counts=ints(0, 0))
    assert torch.all(out == 0) and torch.all(lse == -math.inf) and cp.last_device_status() == OK
    # tokens without a place: zeros for keys, so the mean of zeros, and reported
    out, lse = cp.cache_attention(q, empty, empty, table, ints(0, 0))
    assert cp.last_device_status() == BOUNDS
    assert torch.all(out == 0)
    cp.cache_append(q[:, :2], q[:, :2], empty, empty, table, ints(0, 0))
    assert cp.last_device_status() == BOUNDS


@pytest.mark.parametrize("seed", range(60))
def test_random_sizes(seed):
    rng = random.Random(seed)
    dtype = rng.choice([BF, BF, BF, F32])
    D, page, Hk = rng.choice([64, 128]), rng.choice([16, 32, 64, 128, 256]), rng.randint(1, 4)
    share = rng.choice([1, 1, 2, 3, 4, 5, 7, 8, 16, 33])
    S = rng.choice([1, 1, 2, rng.randint(1, 12), rng.randint(1, 64), rng.randint(1, 256)])
    B = rng.randint(1, 5)
    while B * Hk * share * S > 6000:
        S = max(1, S // 2)
    most = rng.choice([0, 5, 100, 700, 2500])
    lengths = [rng.randint(0, most) for _ in range(B)]
    counts = None if rng.random() < 0.4 else [rng.choice([0, S, rng.randint(0, S)]) for _ in range(B)]
    parents = C.tree(S, B, seed, back=rng.choice([1, 3, 40])) if rng.random() < 0.5 else None
    cache = C.Cache(lengths, counts, S, Hk, D, page, dtype, DEV, seed, rng.choice(["phrd", "prhd"]))
    q = randn(B, Hk * share, S, D, dtype=dtype, seed=seed, layout=rng.choice(["bhsd", "bshd"]))
    got = attend(cache, q, parents)
    assert cp.last_device_status() == OK
    verify(cache, q, got, parents)
