"""Cross attention around the borders where another kernel, another number of key
parts or another way of joining them takes over.

Seeded random calls draw sizes beside those borders -- query rows a key head (32,
64), queries (128, 256), keys (a tile, 192 a part, 1024, 8192), heads that leave
few or many parts -- and go through the bounds-checking build and the normal one:
nothing reported, equal bits, and within the tolerances that count roundings."""
import random

import pytest
import torch

import context_attention_partial_gb300 as cp
import plain_operators as plain
from context_attention_partial_gb300 import _lib
from context_attention_partial_gb300 import build as _build

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def chk():
    return _lib.bind(_build.build(check=True))


@pytest.fixture
def through(monkeypatch):
    def use(lib):
        monkeypatch.setattr(_lib, "load", lambda: lib)
    return use


def inputs(seed, B, H, Hk, M, N, D, dtype, lengths, layout):
    g = torch.Generator(DEV).manual_seed(seed)

    def normal(heads, length):
        shape = (B, heads, length, D) if layout == "bhsd" else (B, length, heads, D)
        x = torch.randn(shape, generator=g, device=DEV).to(dtype)
        return x if layout == "bhsd" else x.transpose(1, 2)

    q, k, v, dout = normal(H, M), normal(Hk, N), normal(Hk, N), normal(H, M)
    n = None
    if lengths is not None:
        n = torch.tensor(lengths, dtype=torch.int32, device=DEV)
        for b in range(B):   # what lies past a length is never used
            k[b, :, max(0, lengths[b]):] = float("nan")
            v[b, :, max(0, lengths[b]):] = float("inf")
    return q, k, v, dout, n


def step(q, k, v, dout, n, grad):
    out, lse = cp.cross_attention(q, k, v, kv_lengths=n)
    got = [("out", out), ("lse", lse)]
    if grad:
        got += zip(("dq", "dk", "dv"), cp.cross_attention_backward(q, k, v, out, lse, dout, kv_lengths=n))
    return got


def compare(chk, through, seed, case, dtype, layout="bhsd", grad=True):
    B, H, Hk, M, N, D, lengths = case
    t = inputs(seed, B, H, Hk, M, N, D, dtype, lengths, layout)
    normal = cp.load_library()
    through(chk)
    checked = step(*t, grad)
    assert chk.cpattn_last_device_status(torch.cuda.current_stream().cuda_stream) == 0
    through(normal)
    got = step(*t, grad)
    assert cp.last_device_status() == 0
    want = plain.cross(*t[:3], lengths, None, t[3] if grad else None)
    for (name, a), (_, b) in zip(got, checked):
        assert torch.equal(a, b), f"{name} of {case}"
        value, tol = want[name]
        assert plain.worst(a, value, tol) <= 1.0, f"{name} of {case}: {plain.worst(a, value, tol):.3g}"


def parts_to_join(q, k):
    rows = q.shape[0] * q.shape[1] * q.shape[2]
    return cp.cross_workspace_bytes(q, k) // (rows * (q.shape[3] + 1) * 4)


# more key parts than a cluster holds: the clusters' results meet in the workspace
CLUSTERS = [
    (1, 4, 4, 77, 16384, 64, None),              # one query tile, two chains
    (1, 4, 4, 77, 16384, 128, (16001,)),
    (1, 2, 1, 128, 9000, 128, (9000,)),
    (1, 2, 2, 129, 9001, 64, None),              # two query tiles
    (1, 1, 1, 250, 20000, 128, (19999,)),
    (2, 2, 1, 100, 12000, 64, (12000, 300)),     # a sequence that leaves most parts without keys
    (3, 1, 1, 200, 10000, 128, (0, 1, 10000)),
]


@pytest.mark.parametrize("case", CLUSTERS, ids=lambda c: "x".join(map(str, c[:6])) + ("r" if c[6] else ""))
def test_more_parts_than_a_cluster(chk, through, case):
    q, k, *_ = inputs(1, *case[:6], BF, None, "bhsd")
    assert parts_to_join(q, k) > 1 and q.shape[2] * q.shape[1] // k.shape[1] > 64
    compare(chk, through, 2, case, BF, "bshd", grad=False)


def test_more_parts_than_a_cluster_captured():
    """Two graphs with workspaces of their own, replayed at once."""
    sets = [inputs(3 + i, 1, 4, 4, 77, 16384, 64, BF, (16384 - i,), "bhsd") for i in range(2)]
    want = [cp.cross_attention(q, k, v, kv_lengths=n) for q, k, v, _, n in sets]
    graphs, got = [], []
    for q, k, v, _, n in sets:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got.append(cp.cross_attention(q, k, v, kv_lengths=n))
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in graphs]
    for _ in range(3):
        for s, g in zip(streams, graphs):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def near(rng, *borders):
    return max(1, rng.choice(borders) + rng.choice([-1, 0, 0, 1]))


def draw(rng, dtype):
    """Sizes beside a border, at a cost that a 64-bit walk head by head can take."""
    B, D = rng.randint(1, 3), rng.choice([64, 128])
    share = rng.choice([1, 1, 2, 3, 8])
    kv_heads = rng.randint(1, 4)
    form = rng.choice(["rows", "queries", "keys", "many"])
    if form == "rows":               # rows a key head: 16, 32, 64
        M = max(1, near(rng, 16, 32, 64) // share)
        N = near(rng, 64, 192, 384, 1024, 1536)
    elif form == "queries":          # query tiles: 64, 128, 256
        M, share = near(rng, 64, 128, 256), min(share, 2)
        N = near(rng, 32, 128, 256, 1024, 2048)
    elif form == "keys":             # parts and clusters
        B, kv_heads, share = 1, rng.randint(1, 2), min(share, 2)
        M = rng.choice([1, 3, 30, 77, 130])
        N = near(rng, 1024, 1536, 4096, 8192)
    else:                            # blocks that fill the GPU
        M, N, kv_heads = near(rng, 128, 384, 640), near(rng, 8, 64, 128, 300), rng.randint(4, 8)
        share = min(share, 2)
    lengths = None if rng.random() < 0.5 else tuple(rng.choice([0, 1, N, max(1, N - 1), rng.randint(1, N)])
                                                    for _ in range(B))
    return B, kv_heads * share, kv_heads, M, N, D, lengths


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("seed", range(24))
def test_random_sizes_beside_the_borders(chk, through, seed, dtype):
    rng = random.Random(1000 * seed + (dtype == F32))
    for i in range(8):
        case = draw(rng, dtype)
        compare(chk, through, rng.randrange(1 << 30), case, dtype, rng.choice(["bhsd", "bshd"]))
