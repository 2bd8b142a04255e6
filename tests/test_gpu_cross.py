"""Cross attention and its gradient against a plain 64-bit form; tolerances
count roundings (plain_operators.py)."""
import math

import pytest
import torch

import context_attention_partial_gb300 as cp
import plain_operators as plain

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32


def normal(g, layout, B, H, S, D, dtype):
    shape = (B, S, H, D) if layout == "bshd" else (B, H, S, D)
    x = torch.randn(*shape, generator=g).to(dtype).to(DEV)
    return x.transpose(1, 2) if layout == "bshd" else x


def make(B, H, Hk, M, N, D, dtype, lengths=None, seed=0, layout="bhsd", poison=True):
    g = torch.Generator("cpu").manual_seed(seed)
    q = normal(g, layout, B, H, M, D, dtype)
    k, v = (normal(g, layout, B, Hk, N, D, dtype) for _ in range(2))
    dout = normal(g, layout, B, H, M, D, dtype)
    if lengths is None:
        return q, k, v, dout, None
    n = torch.tensor(lengths, dtype=torch.int32, device=DEV)
    if poison:   # what lies past a length is never used
        for b in range(B):
            k[b, :, max(0, lengths[b]):] = float("nan")
            v[b, :, max(0, lengths[b]):] = float("inf")
    return q, k, v, dout, n


def check(name, got, want):
    value, tol = want[name]
    assert got.shape == value.shape
    ratio = plain.worst(got, value, tol)
    assert ratio <= 1.0, f"{name}: {ratio:.3g} of its tolerance"


def run(case, dtype, layout="bhsd", scale=None, seed=0):
    B, H, Hk, M, N, D, lengths = case
    q, k, v, dout, n = make(B, H, Hk, M, N, D, dtype, lengths, seed=seed, layout=layout)
    want = plain.cross(q, k, v, lengths, scale, dout)
    out, lse = cp.cross_attention(q, k, v, kv_lengths=n, scale=scale)
    assert cp.last_device_status() == 0
    check("out", out, want)
    check("lse", lse, want)
    grads = cp.cross_attention_backward(q, k, v, out, lse, dout, kv_lengths=n, scale=scale)
    assert cp.last_device_status() == 0
    for name, got in zip(("dq", "dk", "dv"), grads):
        assert got.dtype == dtype
        check(name, got, want)


CASES = [
    # (B, H, H_kv, S_q, S_kv, D, lengths)
    (1, 1, 1, 1, 1, 64, None),
    (1, 1, 1, 1, 1, 128, None),
    (1, 2, 2, 5, 3, 128, None),
    (2, 3, 3, 127, 129, 64, None),
    (2, 3, 3, 129, 127, 128, None),
    (1, 2, 2, 300, 77, 128, None),
    (1, 1, 1, 513, 512, 64, None),
    (1, 1, 1, 255, 640, 128, None),
    (4, 2, 2, 130, 200, 128, (0, 1, 128, 200)),       # no key, one key, a whole tile, all
    (4, 4, 2, 33, 257, 64, (129, 0, 256, 257)),
    (3, 2, 1, 257, 300, 64, (-5, 1000, 63)),          # brought into [0, S_kv]
    (2, 8, 2, 1, 1000, 128, (999, 3)),                # single tokens, shared heads
    (2, 8, 1, 3, 700, 64, (0, 640)),
    (1, 12, 4, 20, 333, 128, None),
    (1, 4, 4, 16, 2100, 64, None),
    (2, 2, 2, 65, 4481, 64, (4481, 1500)),            # few queries, long states
    (3, 5, 5, 1, 9001, 128, (9001, 0, 4096)),
    (1, 32, 2, 4, 5000, 128, None),                   # 64 rows share a key head
    (1, 6, 1, 11, 3001, 64, (2050,)),                 # 66 rows
    (2, 16, 2, 7, 2500, 128, (2500, 1200)),           # 56 rows, many query heads a key head
    (2, 3, 3, 31, 1500, 128, None),                   # 31 rows of one head
]


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "x".join(map(str, c[:6])) + ("r" if c[6] else ""))
def test_cross_matches_plain(case, dtype):
    run(case, dtype)


MANY = [
    (2, 12, 4, 515, 300, 128, (300, 161)),            # rows that fill the GPU, shared heads
    (4, 16, 16, 190, 257, 64, (0, 1, 128, 257)),
    (3, 20, 5, 200, 64, 128, (64, 33, 5)),
    (1, 40, 40, 256, 129, 64, (-3,)),
    (1, 3, 3, 1500, 1030, 64, None),                  # few key tiles: dk, dv in parts
    (3, 2, 2, 100, 1100, 128, (1100, 130, 0)),        # one query tile, its keys in parts of 1 to 5 tiles
    (1, 4, 2, 128, 2049, 64, (2049,)),
    (2, 3, 1, 77, 4481, 128, (4481, 3000)),
]


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("case", MANY, ids=lambda c: "x".join(map(str, c[:6])) + ("r" if c[6] else ""))
def test_cross_many_rows(case, dtype):
    run(case, dtype, layout="bshd", seed=2)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_cross_layouts_and_scale(dtype):
    run((2, 6, 3, 70, 150, 64, (150, 90)), dtype, layout="bshd", scale=0.3, seed=3)
    run((2, 4, 2, 2, 600, 128, (0, 600)), dtype, layout="bshd", scale=0.02, seed=4)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_cross_views_of_fused_projections(dtype):
    """k, v as views of one [B,S,2,H,D] projection, dk, dv into such a buffer; what
    lies around the views stays as it was."""
    B, H, M, N, D = 2, 3, 140, 131, 64
    g = torch.Generator("cpu").manual_seed(11)
    kv = torch.randn(B, N, 2, H, D, generator=g).to(dtype).to(DEV)
    k, v = (kv[:, :, i].transpose(1, 2) for i in range(2))
    q = torch.randn(B, H, M, D, generator=g).to(dtype).to(DEV)
    dout = torch.randn(B, H, M, D, generator=g).to(dtype).to(DEV)
    want = plain.cross(q, k, v, dout=dout)
    big = torch.full((B, H, M + 4, D + 8), 5.0, device=DEV, dtype=dtype)
    o = big[:, :, 2:-2, :D]
    out, lse = cp.cross_attention(q, k, v, out=o)
    assert out.data_ptr() == o.data_ptr()
    check("out", out, want)
    big_dq = torch.full((B, H, M + 4, D + 8), 5.0, device=DEV, dtype=dtype)
    dkv = torch.full((B, N + 2, 3, H, D), 5.0, device=DEV, dtype=dtype)
    dk, dv = (dkv[:, 1:-1, i].transpose(1, 2) for i in range(2))
    grads = cp.cross_attention_backward(q, k, v, out, lse, dout, dq=big_dq[:, :, 2:-2, :D], dk=dk, dv=dv)
    for name, got in zip(("dq", "dk", "dv"), grads):
        check(name, got, want)
    for t, inner in ((big, (slice(None), slice(None), slice(2, -2), slice(0, D))),
                     (big_dq, (slice(None), slice(None), slice(2, -2), slice(0, D))),
                     (dkv, (slice(None), slice(1, -1), slice(0, 2)))):
        mask = torch.ones_like(t, dtype=torch.bool)
        mask[inner] = False
        assert torch.all(t[mask] == 5.0)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_cross_large_scores(dtype):
    """Scores of some hundreds: one key takes each row, nothing overflows."""
    q, k, v, dout, _ = make(1, 2, 2, 96, 260, 64, dtype, seed=5)
    q, k = q * 8, k * 8
    want = plain.cross(q, k, v, dout=dout)
    out, lse = cp.cross_attention(q, k, v)
    check("out", out, want)
    check("lse", lse, want)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_cross_empty_axes(dtype):
    q, k, v, dout, _ = make(2, 4, 2, 5, 9, 64, dtype)
    out, lse = cp.cross_attention(q, k[:, :, :0], v[:, :, :0])
    assert torch.all(out == 0) and torch.all(lse == -math.inf)
    dq, dk, dv = cp.cross_attention_backward(q, k[:, :, :0], v[:, :, :0], out, lse, dout)
    assert torch.all(dq == 0) and dk.shape == (2, 2, 0, 64) and dv.shape == (2, 2, 0, 64)
    e, el = cp.cross_attention(q[:, :, :0], k, v)
    assert e.shape == (2, 4, 0, 64) and el.shape == (2, 4, 0)
    dq, dk, dv = cp.cross_attention_backward(q[:, :, :0], k, v, e, el, dout[:, :, :0])
    assert dq.shape == (2, 4, 0, 64) and torch.all(dk == 0) and torch.all(dv == 0)
    n = torch.zeros(2, dtype=torch.int32, device=DEV)      # every sequence without keys
    out, lse = cp.cross_attention(q, k, v, kv_lengths=n)
    assert torch.all(out == 0) and torch.all(lse == -math.inf)
    for t in cp.cross_attention_backward(q, k, v, out, lse, dout, kv_lengths=n):
        assert torch.all(t == 0)
    assert cp.last_device_status() == 0


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("M", [1, 150])
def test_cross_single_key_has_no_score_gradient(dtype, M):
    """One key takes all the weight whatever q and k are: dq and dk are 0, to the bit."""
    for keys, lengths in ((1, None), (200, (1, 1)), (1, (1, 0))):
        q, k, v, dout, n = make(2, 4, 2, M, keys, 128, dtype, lengths, seed=9)
        out, lse = cp.cross_attention(q, k, v, kv_lengths=n)
        dq, dk, dv = cp.cross_attention_backward(q, k, v, out, lse, dout, kv_lengths=n)
        assert torch.all(dq == 0) and torch.all(dk == 0)
        want = plain.cross(q, k, v, lengths, dout=dout)
        check("out", out, want)
        check("dv", dv, want)


def test_cross_gradient_against_differences():
    """fp32 central differences of sum(dout out) in a few directions."""
    B, H, Hk, M, N, D = 2, 4, 2, 9, 21, 64
    q, k, v, dout, n = make(B, H, Hk, M, N, D, F32, (21, 13), seed=6, poison=False)
    out, lse = cp.cross_attention(q, k, v, kv_lengths=n)
    grads = cp.cross_attention_backward(q, k, v, out, lse, dout, kv_lengths=n)
    f = lambda *t: (cp.cross_attention(*t, kv_lengths=n)[0].double() * dout.double()).sum()
    step = 2.0 ** -7
    for i, grad in enumerate(grads):
        for seed in range(3):
            d = torch.randn(grad.shape, generator=torch.Generator("cpu").manual_seed(20 + seed)).to(DEV)
            d = d / d.norm()
            plus, minus = [q, k, v], [q, k, v]
            plus[i], minus[i] = plus[i] + step * d, minus[i] - step * d
            num = (f(*plus) - f(*minus)) / (2 * step)
            ana = (grad.double() * d.double()).sum()
            # the differences: fp32 outputs (4 u each, |dout| |out| summed as a walk) over the step,
            # and the cubic term step^2 of a function whose derivatives are of the order of |dout| |v|
            size = float((dout.double().norm() * v.double().abs().max()))
            assert abs(float(num - ana)) <= size * (8 * 2 ** -24 / step + step ** 2)


def test_cross_backward_is_repeatable_and_shares_heads():
    """Equal calls give equal bits; dk, dv of a shared head are the sums over repeated heads."""
    q, k, v, dout, n = make(2, 8, 2, 200, 300, 128, BF, (300, 170), seed=7, poison=False)
    out, lse = cp.cross_attention(q, k, v, kv_lengths=n)
    a = cp.cross_attention_backward(q, k, v, out, lse, dout, kv_lengths=n)
    b = cp.cross_attention_backward(q, k, v, out, lse, dout, kv_lengths=n)
    for x, y in zip(a, b):
        assert torch.equal(x, y)
    kr, vr = (t.repeat_interleave(4, 1) for t in (k, v))
    out_r, lse_r = cp.cross_attention(q, kr, vr, kv_lengths=n)
    dq, dk, dv = cp.cross_attention_backward(q, kr, vr, out_r, lse_r, dout, kv_lengths=n)
    want = plain.cross(q, k, v, (300, 170), dout=dout)
    for name, got in (("dk", dk), ("dv", dv)):
        value, tol = want[name]
        # four roundings to bf16 more
        got = got.double().view(2, 2, 4, 300, 128)
        extra = 2 ** -8 * got.abs().sum(2)
        assert plain.worst(got.sum(2), value, tol + extra + 1e-30) <= 1.0


@pytest.mark.parametrize("M", [1, 300])
def test_cross_streams_and_graphs(M):
    """Two calls at once on two streams, and two captured graphs replayed at
    once, give what the single calls give."""
    sets = [make(2, 8, 2, M, 2000, 128, BF, (2000, 1111), seed=30 + i, poison=False) for i in range(2)]
    want = []
    for q, k, v, dout, n in sets:
        out, lse = cp.cross_attention(q, k, v, kv_lengths=n)
        want.append((out, lse, *cp.cross_attention_backward(q, k, v, out, lse, dout, kv_lengths=n)))
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = []
    for s, (q, k, v, dout, n) in zip(streams, sets):
        out, lse = cp.cross_attention(q, k, v, kv_lengths=n, stream=s)
        got.append((out, lse, *cp.cross_attention_backward(q, k, v, out, lse, dout, kv_lengths=n, stream=s)))
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        for x, y in zip(a, b):
            assert torch.equal(x, y)
    graphs, outs = [], []
    for q, k, v, dout, n in sets:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out, lse = cp.cross_attention(q, k, v, kv_lengths=n)
            outs.append((out, lse, *cp.cross_attention_backward(q, k, v, out, lse, dout, kv_lengths=n)))
        graphs.append(g)
    for rep in range(3):
        for s, g in zip(streams, graphs):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for a, b in zip(outs, want):
            for x, y in zip(a, b):
                assert torch.equal(x, y)
    # lengths are read when the graph runs
    sets[0][4].zero_()
    graphs[0].replay()
    torch.cuda.synchronize()
    assert torch.all(outs[0][0] == 0) and all(torch.all(t == 0) for t in outs[0][2:])
    assert cp.last_device_status() == 0


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_cross_captured_across_two_streams(dtype):
    """A captured graph that forks (a key side and a query side on two streams)
    and joins: every kernel waits for both of the kernels it depends on."""
    q, k, v, dout, n = make(2, 8, 2, 200, 700, 128, dtype, (700, 333), seed=35, poison=False)
    pos = torch.arange(700, device=DEV).float()[:, None]

    def step(side):
        main = torch.cuda.current_stream()
        side.wait_stream(main)
        with torch.cuda.stream(side):
            rk = cp.rotary(k * 2, pos, (128,))
        rq = cp.rotary(q * 2, pos[:200], (128,))
        main.wait_stream(side)
        out, lse = cp.cross_attention(rq, rk, v, kv_lengths=n)
        side.wait_stream(main)
        with torch.cuda.stream(side):
            grads = cp.cross_attention_backward(rq, rk, v, out, lse, dout, kv_lengths=n)
        y = cp.rotary(out, pos[:200], (128,))
        main.wait_stream(side)
        return (rk, out, lse, y, *grads, cp.rotary(grads[0], pos[:200], (128,), inverse=True))

    side = torch.cuda.Stream()
    want = step(side)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = step(side)
    for _ in range(3):
        for t in got:
            t.fill_(7.0)
        g.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)
    assert cp.last_device_status() == 0


def test_cross_workspace_given_and_refused():
    q, k, v, dout, _ = make(1, 2, 2, 1, 6000, 128, BF)
    need = cp.cross_workspace_bytes(q, k)
    assert need > 0                                        # the keys are split
    want = cp.cross_attention(q, k, v)
    guard = torch.full((need + 64,), 0x5A, dtype=torch.uint8, device=DEV)
    got = cp.cross_attention(q, k, v, workspace=guard[:need])
    assert torch.equal(got[0], want[0]) and torch.all(guard[need:] == 0x5A)
    with pytest.raises(cp.CpattnError) as e:
        cp.cross_attention(q, k, v, workspace=guard[: need - 16])
    assert e.value.name == "CPATTN_ERR_WORKSPACE"
    with pytest.raises(ValueError, match="contiguous"):    # fewer bytes than it seems to have
        cp.cross_attention(q, k, v, workspace=torch.zeros(1, dtype=torch.uint8, device=DEV).expand(need))
    need = cp.cross_backward_workspace_bytes(q, k)
    guard = torch.full((need + 64,), 0x5A, dtype=torch.uint8, device=DEV)
    cp.cross_attention_backward(q, k, v, *want, dout, workspace=guard[:need])
    torch.cuda.synchronize()
    assert torch.all(guard[need:] == 0x5A)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_block_of_rotary_ring_and_cross_attention(dtype):
    """A transformer block's attentions as they run together: rotary positions,
    ring self-attention, cross attention, and the gradients back through the
    cross attention and the positions."""
    B, H, D, axes, N = 2, 4, 64, (16, 24, 24), 77
    g = torch.meshgrid(torch.arange(2), torch.arange(9), torch.arange(10), indexing="ij")
    pos = torch.stack(g, -1).reshape(-1, 3).float().to(DEV)
    S = pos.shape[0]
    q, k, v, dout, _ = make(B, H, H, S, S, D, dtype, seed=40)
    ek, ev = (t[:, :, :N] for t in make(B, H, H, S, 128, D, dtype, seed=41)[1:3])
    lengths = torch.tensor((N, 20), dtype=torch.int32, device=DEV)
    rq, rk = cp.rotary([q, k], pos, axes)
    out, lse = cp.ring(rq, rk, v, ring_degree=4)
    x, xl = cp.cross_attention(out, ek, ev, kv_lengths=lengths)
    dq, dk, dv = cp.cross_attention_backward(out, ek, ev, x, xl, dout, kv_lengths=lengths)
    back = cp.rotary(dq, pos, axes, inverse=True)
    assert cp.last_device_status() == 0
    for got, t in ((rq, q), (rk, k)):
        y, mag = plain.rotary(t, pos, axes)
        assert plain.worst(got, y, plain.rotary_tolerance(y, mag, dtype)) <= 1.0
    ref = plain.cross(rq, rk, v)["out"][0]
    assert float((out.double() - ref).abs().max()) <= (1e-2 if dtype == BF else 2e-3)
    want = plain.cross(out, ek, ev, (N, 20), dout=dout)
    for name, got in (("out", x), ("lse", xl), ("dq", dq), ("dk", dk), ("dv", dv)):
        check(name, got, want)
    y, mag = plain.rotary(dq, pos, axes, inverse=True)
    assert plain.worst(back, y, plain.rotary_tolerance(y, mag, dtype)) <= 1.0


def test_cross_attention_merges_with_other_partials():
    """Attention over the text states merged with attention over image states
    equals attention over both (an empty text is the merge's identity)."""
    q, k, v, _, _ = make(2, 2, 2, 64, 300, 64, F32, seed=50)
    n = torch.tensor((90, 0), dtype=torch.int32, device=DEV)
    a, la = cp.cross_attention(q, k[:, :, :100], v[:, :, :100], kv_lengths=n)
    b, lb = cp.cross_attention(q, k[:, :, 100:], v[:, :, 100:])
    cp.merge(a, la, b, lb)
    for i, cut in enumerate((90, 0)):
        kk = torch.cat([k[i:i + 1, :, :cut], k[i:i + 1, :, 100:]], 2)
        vv = torch.cat([v[i:i + 1, :, :cut], v[i:i + 1, :, 100:]], 2)
        value, tol = plain.cross(q[i:i + 1], kk, vv)["out"]
        assert plain.worst(a[i:i + 1], value, 3 * tol) <= 1.0


def broadcast_inputs(dtype, B, H, Hk, M, N, D):
    """q, k, v, dout with extents that walk on the spot, and their dense copies."""
    g = torch.Generator("cpu").manual_seed(60)
    q = torch.randn(1, H, M, D, generator=g).to(dtype).to(DEV).expand(B, H, M, D)            # one query block
    k = torch.randn(1, Hk, N, D, generator=g).to(dtype).to(DEV).expand(B, Hk, N, D)          # one prompt for all
    v = torch.randn(B, 1, N, D, generator=g).to(dtype).to(DEV).expand(B, Hk, N, D)
    dout = torch.full((), 0.5, dtype=dtype, device=DEV).expand(B, H, M, D)                   # of (out / 2).sum()
    return (q, k, v, dout), tuple(t.contiguous() for t in (q, k, v, dout))


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("sizes", [(2, 4, 2, 150, 77, 64), (3, 2, 2, 1, 700, 128), (2, 4, 4, 90, 3000, 64)],
                         ids=lambda s: "x".join(map(str, s)))
def test_cross_broadcast_inputs(sizes, dtype):
    """Broadcast inputs give what their dense copies give, also on another stream
    and captured; a broadcast output is refused."""
    B = sizes[0]
    views, dense = broadcast_inputs(dtype, *sizes)
    n = torch.full((1,), sizes[4] - 3, dtype=torch.int32, device=DEV)
    out, lse = cp.cross_attention(*dense[:3], kv_lengths=n.expand(B).contiguous())
    want = (out, lse, *cp.cross_attention_backward(*dense[:3], out, lse, dense[3], kv_lengths=n.expand(B).contiguous()))

    def step(stream=None):
        o, l = cp.cross_attention(*views[:3], kv_lengths=n.expand(B), stream=stream)
        return (o, l, *cp.cross_attention_backward(*views[:3], o, l, views[3], kv_lengths=n.expand(B), stream=stream))

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = [step(), step(s)]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got.append(step())
    graph.replay()
    torch.cuda.synchronize()
    for result in got:
        for a, b in zip(result, want):
            assert a.shape == b.shape and torch.equal(a, b)
    with pytest.raises(cp.CpattnError) as e:
        cp.cross_attention(*dense[:3], out=dense[0][:1].expand_as(dense[0]))
    assert e.value.name == "CPATTN_ERR_LAYOUT"
    assert cp.last_device_status() == 0
