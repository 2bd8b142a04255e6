"""The measured cases of the rotary and cross-attention operators.

Every case is one call of the kind a transformer over image or video tokens makes: positions put on q and
k before self-attention (``rotary``), the latent tokens' attention to a text encoder's states
(``cross_attention``), and the gradients of both.  ``run`` holds the plain form of each operator (elementary
torch operations in 32 bits, angles in 64) and the framework's own calls side by side.
"""
import math

import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # q and k of a 1024 x 1024 image's block: 512 text tokens (position 0) and 64 x 64 image tokens,
        # tensors as the projections leave them ([B, S, H, D])
        dict(name="rotary_image", op="rotary", batch=1, heads=24, kv_heads=24, text=512, t=1, h=64, w=64, start=0,
             axes="16,56,56", dim=128, pairs="interleaved", inverse=False, layout="bshd", dtype="bf16", per_batch=False),
        # gradients of q and k of a video block, 8 frames of 64 x 64 tokens, ring layout [B, H, S, D]
        dict(name="rotary_video_grad", op="rotary", batch=1, heads=24, kv_heads=24, text=0, t=8, h=64, w=64, start=0,
             axes="44,42,42", dim=128, pairs="interleaved", inverse=True, layout="bhsd", dtype="bf16", per_batch=False),
        # fp32, shared key heads, halves, an odd token count and positions of each sequence's own
        dict(name="rotary_f32_halves", op="rotary", batch=2, heads=8, kv_heads=2, text=17, t=3, h=15, w=13, start=5,
             axes="16,24,24", dim=64, pairs="halves", inverse=False, layout="bhsd", dtype="f32", per_batch=True),
        # one new token at a far position for a batch of sequences: latency
        dict(name="rotary_token", op="rotary", batch=8, heads=24, kv_heads=8, text=0, t=1, h=1, w=1, start=100003,
             axes="128", dim=128, pairs="halves", inverse=False, layout="bshd", dtype="bf16", per_batch=True),
        # image tokens against 512 text states
        dict(name="cross_image", op="cross", batch=1, heads=24, kv_heads=24, queries=4608, keys=512, dim=128,
             ragged=False, layout="bhsd", dtype="bf16"),
        # video tokens of a guided pair (prompt and negative prompt) against prompts of their own lengths
        dict(name="cross_video", op="cross", batch=2, heads=24, kv_heads=24, queries=32768, keys=512, dim=128,
             ragged=True, layout="bshd", dtype="bf16"),
        # one new token of eight sequences against long encoder states, shared key heads: the keys are split
        dict(name="cross_token", op="cross", batch=8, heads=32, kv_heads=8, queries=1, keys=16384, dim=128,
             ragged=True, layout="bhsd", dtype="bf16"),
        # a short caption's queries against image states of odd length, head size 64
        dict(name="cross_caption", op="cross", batch=2, heads=16, kv_heads=16, queries=77, keys=4481, dim=64,
             ragged=False, layout="bhsd", dtype="bf16"),
        # the fp32 size of the framework's own smallest workload
        dict(name="cross_f32", op="cross", batch=2, heads=2, kv_heads=2, queries=256, keys=77, dim=64,
             ragged=True, layout="bhsd", dtype="f32"),
        # training step of the image block's cross attention
        dict(name="cross_image_grad", op="cross_grad", batch=1, heads=24, kv_heads=24, queries=4608, keys=512, dim=128,
             ragged=False, layout="bhsd", dtype="bf16"),
        # training step of the video block's: the largest case
        dict(name="cross_video_grad", op="cross_grad", batch=2, heads=24, kv_heads=24, queries=32768, keys=512, dim=128,
             ragged=True, layout="bhsd", dtype="bf16"),
        # a ragged batch with shared key heads and head size 64, odd sizes
        dict(name="cross_shared_grad", op="cross_grad", batch=4, heads=16, kv_heads=4, queries=1000, keys=333, dim=64,
             ragged=True, layout="bshd", dtype="bf16"),
    ]


def _log(rng, lo, hi):
    """A whole number spread over [lo, hi] by its logarithm."""
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    op = rng.choice(["rotary", "cross", "cross", "cross_grad"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    dim = rng.choice([64, 128])
    layout = rng.choice(["bhsd", "bshd"])
    batch = rng.randint(1, 4)
    kv_heads = rng.randint(1, 12)
    heads = kv_heads * rng.choice([1, 1, 2, 4])
    if heads > 32:
        heads = kv_heads
    if op == "rotary":
        grid = rng.choice(["token", "line", "image", "video"])
        t, h, w, text = 1, 1, 1, rng.choice([0, 0, 77, 512])
        if grid == "line":
            w = _log(rng, 1, 8192)
        elif grid == "image":
            h, w = rng.randint(1, 96), rng.randint(1, 96)
        elif grid == "video":
            t, h, w = rng.randint(1, 16), rng.randint(1, 48), rng.randint(1, 48)
        if grid in ("token", "line"):
            axes, text = [dim], 0
        else:
            a = 2 * rng.randint(1, dim // 4)
            b = 2 * rng.randint(1, (dim - a) // 2 - 1) if dim - a > 4 else 2
            axes = [a, b, dim - a - b]
        return dict(op=op, batch=batch, heads=heads, kv_heads=kv_heads, text=text, t=t, h=h, w=w,
                    start=_log(rng, 1, 1000000) if grid in ("token", "line") else rng.randint(0, 64),
                    axes=",".join(map(str, axes)), dim=dim, pairs=rng.choice(["interleaved", "halves"]),
                    inverse=rng.random() < 0.5, layout=layout, dtype=dtype, per_batch=rng.random() < 0.5)
    if dtype == "f32":
        queries, keys = _log(rng, 1, 1024), _log(rng, 1, 512)
    elif op == "cross" and rng.random() < 0.5:
        queries, keys = rng.randint(1, 16), _log(rng, 1, 32768)
    else:
        queries, keys = _log(rng, 1, 16384), _log(rng, 1, 2048)
    return dict(op=op, batch=batch, heads=heads, kv_heads=kv_heads, queries=queries, keys=keys, dim=dim,
                ragged=rng.random() < 0.5, layout=layout, dtype=dtype)


def _axes(case):
    return [int(a) for a in case["axes"].split(",")]


def _seq(case):
    return case["text"] + case["t"] * case["h"] * case["w"]


def _normal(gen, case, heads, length, dtype=None):
    """N(0, 1) in the case's type as a [B, H, S, D] view of its layout."""
    b, d = case["batch"], case["dim"]
    shape = (b, heads, length, d) if case["layout"] == "bhsd" else (b, length, heads, d)
    x = torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32).to(dtype or _TYPES[case["dtype"]])
    return x if case["layout"] == "bhsd" else x.transpose(1, 2)


def _lengths(gen, case):
    """A batch's valid key counts: from half the keys to all of them, one sequence in four has none."""
    keys, b = case["keys"], case["batch"]
    n = torch.randint(keys // 2, keys + 1, (b,), generator=gen, device="cuda", dtype=torch.int32)
    n[3::4] = 0
    return n


def prepare(case, seed):
    gen = torch.Generator("cuda").manual_seed(seed)
    s = {"case": case, "scale": case["dim"] ** -0.5}
    if case["op"] == "rotary":
        axes, n = _axes(case), _seq(case)
        t, h, w = torch.meshgrid(*(torch.arange(case[a], device="cuda") for a in "thw"), indexing="ij")
        ids = torch.stack([t, h, w], -1).reshape(-1, 3)[:, 3 - len(axes):] + case["start"]
        pos = torch.cat([torch.zeros(case["text"], len(axes), device="cuda", dtype=ids.dtype), ids]).float()
        if case["per_batch"]:   # sequences that began earlier or later
            pos = pos + torch.arange(case["batch"], device="cuda").view(-1, 1, 1).float()
        s.update(x=[_normal(gen, case, case["heads"], n), _normal(gen, case, case["kv_heads"], n)], pos=pos, axes=axes,
                 theta=10000.0)
        return s
    q = _normal(gen, case, case["heads"], case["queries"])
    k = _normal(gen, case, case["kv_heads"], case["keys"])
    v = _normal(gen, case, case["kv_heads"], case["keys"])
    lengths = _lengths(gen, case) if case["ragged"] else None
    s.update(q=q, k=k, v=v, lengths=lengths)
    if case["op"] == "cross_grad":   # what a training step's forward pass has left
        out, lse = _cross(q, k, v, lengths, s["scale"])
        s.update(out=out, lse=lse, dout=_normal(gen, case, case["heads"], case["queries"]))
    return s


def _angles(pos, axes, theta):
    """[..., S, sum(axes) / 2] angles in 64 bits."""
    return torch.cat([pos[..., a, None].double()
                      * theta ** (-torch.arange(0, d, 2, device=pos.device, dtype=torch.float64) / d)
                      for a, d in enumerate(axes)], -1)


def _pair_index(axes, pairs, device):
    """Feature numbers of the first and second member of every pair."""
    base = torch.cat([torch.zeros(d // 2, dtype=torch.int64) + sum(axes[:a]) for a, d in enumerate(axes)])
    i = torch.cat([torch.arange(d // 2) for d in axes])
    half = torch.cat([torch.full((d // 2,), d // 2) for d in axes])
    first, second = (base + 2 * i, base + 2 * i + 1) if pairs == "interleaved" else (base + i, base + i + half)
    return first.to(device), second.to(device)


def _rotary(x, cos, sin, first, second):
    y = x.float()
    a, b = y[..., first], y[..., second]
    z = y.clone()
    z[..., first] = a * cos - b * sin
    z[..., second] = a * sin + b * cos
    return z.to(x.dtype)


def _shared(x, heads):
    """Key heads repeated for the query heads that share them, in 32 bits."""
    return x.float().repeat_interleave(heads // x.shape[1], dim=1)


def _probabilities(q, k, lengths, scale):
    """exp(s - lse) and lse over each sequence's keys; rows without keys: 0 and -inf."""
    s = torch.matmul(q.float() * scale, _shared(k, q.shape[1]).transpose(-1, -2))
    if lengths is not None:
        s = s.masked_fill(torch.arange(k.shape[2], device=k.device) >= lengths.view(-1, 1, 1, 1), -math.inf)
    top = s.amax(-1, keepdim=True).clamp_min(torch.finfo(torch.float32).min)
    e = torch.exp(s - top)
    total = e.sum(-1, keepdim=True)
    return e / total.clamp_min(torch.finfo(torch.float32).tiny), (top + torch.log(total)).squeeze(-1)


def _cross(q, k, v, lengths, scale):
    p, lse = _probabilities(q, k, lengths, scale)
    return torch.matmul(p, _shared(v, q.shape[1])).to(q.dtype), lse


def _cross_grad(q, k, v, dout, lengths, scale):
    b, h, m, d = q.shape
    kv = k.shape[1]
    p, _ = _probabilities(q, k, lengths, scale)
    g = dout.float()
    dp = torch.matmul(g, _shared(v, h).transpose(-1, -2))
    ds = p * (dp - (p * dp).sum(-1, keepdim=True)) * scale
    dq = torch.matmul(ds, _shared(k, h))
    dk = torch.matmul(ds.transpose(-1, -2), q.float()).view(b, kv, h // kv, -1, d).sum(2)
    dv = torch.matmul(p.transpose(-1, -2), g).view(b, kv, h // kv, -1, d).sum(2)
    return dq.to(q.dtype), dk.to(q.dtype), dv.to(q.dtype)


def run(state):
    case = state["case"]
    if own:
        import context_attention_partial_gb300 as cp
        if case["op"] == "rotary":
            return cp.rotary(state["x"], state["pos"], state["axes"], theta=state["theta"],
                             interleaved=case["pairs"] == "interleaved", inverse=case["inverse"])
        if case["op"] == "cross":
            return cp.cross_attention(state["q"], state["k"], state["v"], kv_lengths=state["lengths"], scale=state["scale"])
        return cp.cross_attention_backward(state["q"], state["k"], state["v"], state["out"], state["lse"], state["dout"],
                                           kv_lengths=state["lengths"], scale=state["scale"])
    if case["op"] == "rotary":
        angle = _angles(state["pos"], state["axes"], state["theta"])
        cos, sin = angle.cos().float(), angle.sin().float()
        if case["per_batch"]:
            cos, sin = cos[:, None], sin[:, None]
        first, second = _pair_index(state["axes"], case["pairs"], cos.device)
        return [_rotary(x, cos, -sin if case["inverse"] else sin, first, second) for x in state["x"]]
    if case["op"] == "cross":
        return _cross(state["q"], state["k"], state["v"], state["lengths"], state["scale"])
    return _cross_grad(state["q"], state["k"], state["v"], state["dout"], state["lengths"], state["scale"])


def exact(case, seed):
    """The definitions in 64 bits: a pair as a complex number times e^(i angle), attention head by head."""
    s = prepare(case, seed)
    if case["op"] == "rotary":
        outs = []
        for x in s["x"]:
            y = x.double().clone()
            at = 0
            for a, d in enumerate(s["axes"]):
                for i in range(d // 2):
                    u, w = (at + 2 * i, at + 2 * i + 1) if case["pairs"] == "interleaved" else (at + i, at + d // 2 + i)
                    angle = s["pos"][..., a].double() * s["theta"] ** (-2.0 * i / d) * (-1 if case["inverse"] else 1)
                    turn = torch.polar(torch.ones_like(angle), angle)
                    turn = turn[:, None] if case["per_batch"] else turn
                    z = torch.complex(x[..., u].double(), x[..., w].double()) * turn
                    y[..., u], y[..., w] = z.real, z.imag
                at += d
            outs.append(y)
        return outs
    q, k, v, scale = s["q"], s["k"], s["v"], s["scale"]
    b, h, m, d = q.shape
    group = h // k.shape[1]
    zero = dict(dtype=torch.float64, device=q.device)
    out, lse = torch.zeros(b, h, m, d, **zero), torch.full((b, h, m), -math.inf, **zero)
    dq, dk, dv = torch.zeros(b, h, m, d, **zero), torch.zeros(k.shape, **zero), torch.zeros(k.shape, **zero)
    for i in range(b):
        n = case["keys"] if s["lengths"] is None else int(s["lengths"][i])
        if n == 0:
            continue
        for j in range(h):
            qq, kk, vv = q[i, j].double(), k[i, j // group, :n].double(), v[i, j // group, :n].double()
            z = qq @ kk.T * scale
            lse[i, j] = torch.logsumexp(z, -1)
            p = torch.exp(z - lse[i, j][:, None])
            if case["op"] == "cross":
                out[i, j] = p @ vv
                continue
            g = s["dout"][i, j].double()
            dz = torch.mul(p, g @ vv.T - (g * (p @ vv)).sum(-1, keepdim=True))
            dq[i, j] = dz @ kk * scale
            dk[i, j // group, :n] += dz.T @ qq * scale
            dv[i, j // group, :n] += p.T @ g
    return (out, lse) if case["op"] == "cross" else (dq, dk, dv)


def work(case):
    """Each input read once, each output written once; the products of the definition."""
    es, b, d, h, kv = 4 if case["dtype"] == "f32" else 2, case["batch"], case["dim"], case["heads"], case["kv_heads"]
    if case["op"] == "rotary":
        n = _seq(case)
        values = b * n * (h + kv) * d
        return {"bytes": 2 * values * es + 4 * n * len(_axes(case)) * (b if case["per_batch"] else 1), "flops": 3 * values}
    m, n = case["queries"], case["keys"]
    # ragged: three quarters of the keys on average, one sequence in four has none
    share = 0.75 * (b - b // 4) / b if case["ragged"] else 1.0
    rows, keys, pairs = b * h * m, b * kv * n * share, b * h * m * n * share
    if case["op"] == "cross":
        return {"bytes": es * d * (2 * rows + 2 * keys) + 4 * rows, "flops": 4 * d * pairs}
    return {"bytes": es * d * (4 * rows + 2 * keys + 2 * b * kv * n) + 4 * rows, "flops": 10 * d * pairs}
