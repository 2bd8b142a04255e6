"""The measured cases of the per-head norms with rotary positions and of the paged key / value cache.

Every case is one call of the kind a transformer makes next to its attentions: queries and keys normed for each
head and turned to their positions in one pass (``norm_rotary``) and the gradient of that (``norm_grad``); new
tokens' keys and values brought to a paged cache on the same way (``append``); and the attention of new tokens,
a chain or a tree of drafts, to such a cache (``attend``).  ``run`` holds the plain form of each operator
(elementary torch operations in 32 bits, angles in 64) and the framework's own calls side by side.
"""
import math

import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
_EPS = 1e-6
_THETA = 10000.0


def listed():
    return [
        # q and k of a 1024 x 1024 image's block: 512 text tokens (position 0) and 64 x 64 image tokens,
        # tensors as the projections leave them ([B, S, H, D])
        dict(name="norm_image", op="norm_rotary", batch=1, heads=24, kv_heads=24, text=512, t=1, h=64, w=64,
             axes="16,56,56", dim=128, pairs="interleaved", layout="bshd", dtype="bf16", weights="bf16"),
        # fp32, shared key heads, halves, an odd token count
        dict(name="norm_f32_halves", op="norm_rotary", batch=2, heads=8, kv_heads=2, text=17, t=3, h=15, w=13,
             axes="16,24,24", dim=64, pairs="halves", layout="bhsd", dtype="f32", weights="f32"),
        # training step of a video block, 8 frames of 64 x 64 tokens, weights kept in fp32
        dict(name="norm_video_grad", op="norm_grad", batch=1, heads=24, kv_heads=24, text=0, t=8, h=64, w=64,
             axes="44,42,42", dim=128, pairs="interleaved", layout="bhsd", dtype="bf16", weights="f32"),
        # training step of a guided pair's small image, shared key heads, halves, head size 64
        dict(name="norm_small_grad", op="norm_grad", batch=2, heads=16, kv_heads=4, text=77, t=1, h=15, w=17,
             axes="32,32", dim=64, pairs="halves", layout="bshd", dtype="bf16", weights="bf16"),
        # one new token of eight sequences, queries turned in the same call: latency
        dict(name="append_token", op="append", batch=8, heads=32, kv_heads=8, tokens=1, context=4096, page=64,
             ragged=True, tree=False, pages="phsd", norm=True, queries=True, axes="128", dim=128, pairs="halves",
             layout="bshd", dtype="bf16"),
        # four prompts of their own lengths to an empty cache with small pages, no norm
        dict(name="append_prompt", op="append", batch=4, heads=32, kv_heads=8, tokens=4001, context=0, page=16,
             ragged=True, tree=False, pages="pshd", norm=False, queries=True, axes="128", dim=128, pairs="halves",
             layout="bshd", dtype="bf16"),
        # a few fp32 tokens of a small model
        dict(name="append_f32", op="append", batch=3, heads=8, kv_heads=2, tokens=13, context=700, page=16,
             ragged=True, tree=True, pages="phsd", norm=True, queries=True, axes="64", dim=64, pairs="interleaved",
             layout="bhsd", dtype="f32"),
        # one new token of eight sequences against long caches
        dict(name="attend_token", op="attend", batch=8, heads=32, kv_heads=8, tokens=1, context=16384, page=64,
             ragged=True, tree=False, pages="phsd", dim=128, layout="bshd", dtype="bf16"),
        # trees of 27 drafted tokens, one step of speculative decoding
        dict(name="attend_tree", op="attend", batch=8, heads=32, kv_heads=8, tokens=27, context=8192, page=32,
             ragged=True, tree=True, pages="pshd", dim=128, layout="bshd", dtype="bf16"),
        # wide trees at long caches, keys not shared, head size 64
        dict(name="attend_wide", op="attend", batch=4, heads=24, kv_heads=24, tokens=64, context=16384, page=128,
             ragged=False, tree=True, pages="phsd", dim=64, layout="bhsd", dtype="bf16"),
        # the next piece of a long prompt: the largest case
        dict(name="attend_prompt", op="attend", batch=1, heads=32, kv_heads=8, tokens=1024, context=16384, page=64,
             ragged=False, tree=False, pages="phsd", dim=128, layout="bshd", dtype="bf16"),
        # drafts of a small model in fp32
        dict(name="attend_f32", op="attend", batch=3, heads=8, kv_heads=2, tokens=13, context=700, page=16,
             ragged=True, tree=True, pages="phsd", dim=64, layout="bhsd", dtype="f32"),
    ]


def _log(rng, lo, hi):
    """A whole number spread over [lo, hi] by its logarithm."""
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    op = rng.choice(["norm_rotary", "norm_grad", "append", "attend", "attend", "attend"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    dim = rng.choice([64, 128])
    layout = rng.choice(["bhsd", "bshd"])
    pairs = rng.choice(["interleaved", "halves"])
    kv_heads = rng.randint(1, 12)
    heads = kv_heads * rng.choice([1, 1, 2, 4])
    if heads > 32:
        heads = kv_heads
    if op in ("norm_rotary", "norm_grad"):
        grid = rng.choice(["line", "image", "video"])
        t, h, w, text = 1, 1, 1, rng.choice([0, 0, 77, 512])
        if grid == "line":
            w, text, axes = _log(rng, 1, 8192), 0, [dim]
        else:
            if grid == "image":
                h, w = rng.randint(1, 96), rng.randint(1, 96)
            else:
                t, h, w = rng.randint(1, 12), rng.randint(1, 48), rng.randint(1, 48)
            a = 2 * rng.randint(1, dim // 4)
            b = 2 * rng.randint(1, (dim - a) // 2 - 1) if dim - a > 4 else 2
            axes = [a, b, dim - a - b]
        batch = rng.randint(1, 2)
        return dict(op=op, batch=batch, heads=heads, kv_heads=kv_heads, text=text, t=t, h=h, w=w,
                    axes=",".join(map(str, axes)), dim=dim, pairs=pairs, layout=layout, dtype=dtype,
                    weights=rng.choice([dtype, "f32"]))
    case = dict(op=op, batch=rng.randint(1, 8), heads=heads, kv_heads=kv_heads, page=rng.choice([16, 32, 64, 128]),
                ragged=rng.random() < 0.7, pages=rng.choice(["phsd", "pshd"]), dim=dim, layout=layout, dtype=dtype)
    if op == "append":
        case.update(tree=False, tokens=_log(rng, 1, 2048), context=_log(rng, 1, 2048), norm=rng.random() < 0.5,
                    queries=rng.random() < 0.7, axes=str(dim), pairs=pairs)
        return case
    tree = rng.random() < 0.6
    if dtype == "f32":
        case.update(tree=tree, tokens=_log(rng, 1, 32), context=_log(rng, 1, 1024), batch=rng.randint(1, 4))
    elif rng.random() < 0.2:
        case.update(tree=False, tokens=_log(rng, 64, 1024), context=_log(rng, 1, 4096), batch=rng.randint(1, 2))
    else:
        case.update(tree=tree, tokens=_log(rng, 1, 64), context=_log(rng, 1, 16384))
    return case


def _axes(case):
    return [int(a) for a in case["axes"].split(",")]


def _normal(gen, case, heads, length):
    """N(0, 1) in the case's type as a [B, H, S, D] view of its layout."""
    b, d = case["batch"], case["dim"]
    shape = (b, heads, length, d) if case["layout"] == "bhsd" else (b, length, heads, d)
    x = torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32).to(_TYPES[case["dtype"]])
    return x if case["layout"] == "bhsd" else x.transpose(1, 2)


def _weight(gen, case, dtype):
    return (1 + 0.2 * torch.randn(case["dim"], generator=gen, device="cuda")).to(_TYPES[dtype])


def _width(case):
    """Pages of a sequence's row in the page table."""
    return -(-(case["context"] + case["tokens"]) // case["page"])


def _cache(gen, case, s):
    """A pool of pages in random order, each sequence's page numbers, cached and new token counts, and drafts."""
    b, n, page, context = case["batch"], case["tokens"], case["page"], case["context"]
    width = _width(case)
    count = b * width + 3   # (a pool has pages of nobody)
    shape = (count, case["kv_heads"], page, case["dim"])
    if case["pages"] == "pshd":
        shape = (count, page, case["kv_heads"], case["dim"])
    for name in ("key_pages", "value_pages"):
        x = torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32).to(_TYPES[case["dtype"]])
        s[name] = x if case["pages"] == "phsd" else x.transpose(1, 2)
    order = torch.randperm(count, generator=gen, device="cuda")[:b * width].view(b, width).to(torch.int32)
    lengths = torch.full((b,), context, device="cuda", dtype=torch.int32)
    counts = None
    if case["ragged"]:   # half the cache to all of it; half the new tokens to all of them, one sequence in four has none
        lengths = torch.randint(context // 2, context + 1, (b,), generator=gen, device="cuda", dtype=torch.int32)
        counts = torch.randint((n + 1) // 2, n + 1, (b,), generator=gen, device="cuda", dtype=torch.int32)
        counts[3::4] = 0
    # rows of the table behind a sequence's pages are not filled in
    used = (lengths + n + page - 1) // page
    table = torch.where(torch.arange(width, device="cuda") < used.view(-1, 1), order, torch.full_like(order, -1))
    s.update(page_table=table, lengths=lengths, counts=counts, parents=None)
    if case["tree"]:   # a draft's parent is one of the eight before it, or the last cached token
        back = torch.randint(1, 9, (b, n), generator=gen, device="cuda")
        s["parents"] = (torch.arange(n, device="cuda") - back).clamp_min(-1).to(torch.int32)


def _depths(parents):
    """Drafts above each draft, [B, N] (a tree's positions behind the cache)."""
    return _ancestors(parents).sum(-1) - 1


def prepare(case, seed):
    gen = torch.Generator("cuda").manual_seed(seed)
    s = {"case": case}
    op = case["op"]
    if op in ("norm_rotary", "norm_grad"):
        axes = _axes(case)
        t, h, w = torch.meshgrid(*(torch.arange(case[a], device="cuda") for a in "thw"), indexing="ij")
        ids = torch.stack([t, h, w], -1).reshape(-1, 3)[:, 3 - len(axes):]
        pos = torch.cat([torch.zeros(case["text"], len(axes), device="cuda", dtype=ids.dtype), ids]).float()
        n = pos.shape[0]
        s.update(x=[_normal(gen, case, case["heads"], n), _normal(gen, case, case["kv_heads"], n)], axes=axes, pos=pos,
                 w=[_weight(gen, case, case["weights"]) for _ in range(2)])
        if op == "norm_grad":
            s["dy"] = [_normal(gen, case, case["heads"], n), _normal(gen, case, case["kv_heads"], n)]
        return s
    _cache(gen, case, s)
    if op == "attend":
        s.update(q=_normal(gen, case, case["heads"], case["tokens"]), scale=case["dim"] ** -0.5)
        return s
    s.update(k=_normal(gen, case, case["kv_heads"], case["tokens"]), v=_normal(gen, case, case["kv_heads"], case["tokens"]),
             q=_normal(gen, case, case["heads"], case["tokens"]) if case["queries"] else None, axes=_axes(case),
             wk=_weight(gen, case, case["dtype"]) if case["norm"] else None,
             wq=_weight(gen, case, case["dtype"]) if case["norm"] and case["queries"] else None)
    steps = torch.arange(case["tokens"], device="cuda") if s["parents"] is None else _depths(s["parents"])
    s["pos"] = (s["lengths"].view(-1, 1) + steps).float().unsqueeze(-1)
    return s


def _angles(pos, axes):
    """[..., S, sum(axes) / 2] angles in 64 bits."""
    return torch.cat([pos[..., a, None].double()
                      * _THETA ** (-torch.arange(0, d, 2, device=pos.device, dtype=torch.float64) / d)
                      for a, d in enumerate(axes)], -1)


def _pair_index(axes, pairs, device):
    """Feature numbers of the first and second member of every pair."""
    base = torch.cat([torch.zeros(d // 2, dtype=torch.int64) + sum(axes[:a]) for a, d in enumerate(axes)])
    i = torch.cat([torch.arange(d // 2) for d in axes])
    half = torch.cat([torch.full((d // 2,), d // 2) for d in axes])
    first, second = (base + 2 * i, base + 2 * i + 1) if pairs == "interleaved" else (base + i, base + i + half)
    return first.to(device), second.to(device)


def _turn(x, cos, sin, first, second):
    a, b = x[..., first], x[..., second]
    y = x.clone()
    y[..., first] = a * cos - b * sin
    y[..., second] = a * sin + b * cos
    return y


def _normed(x, w):
    """x / rms(x) * w in 32 bits (w None: x)."""
    x = x.float()
    return x if w is None else x * torch.rsqrt((x * x).mean(-1, keepdim=True) + _EPS) * w.float()


def _norm_grad(x, w, dy, cos, sin, first, second):
    x = x.float()
    dz = _turn(dy.float(), cos, -sin, first, second)
    r = torch.rsqrt((x * x).mean(-1, keepdim=True) + _EPS)
    n = x * r
    g = dz * w.float()
    return r * (g - n * (g * n).mean(-1, keepdim=True)), (dz * n).sum((0, 1, 2))


def _ancestors(parents):
    """[B, N, N]: whether draft j is draft i or above it (the paths of the tree, by squaring)."""
    n = parents.shape[1]
    a = torch.eye(n, device=parents.device) + (parents.unsqueeze(-1) == torch.arange(n, device=parents.device)).float()
    for _ in range(max(1, n - 1).bit_length()):
        a = (torch.matmul(a, a) > 0).float()
    return a > 0


def _seen(state, keys):
    """[B, N, keys]: whether new token i sees the key at place j of its sequence's cache."""
    case, lengths, counts = state["case"], state["lengths"].long().view(-1, 1, 1), state["counts"]
    n = case["tokens"]
    i = torch.arange(n, device="cuda").view(1, -1, 1)
    j = torch.arange(keys, device="cuda").view(1, 1, -1) - lengths
    if state["parents"] is None:
        seen = j <= i
    else:
        tree = _ancestors(state["parents"])
        above = torch.gather(tree, 2, j.clamp(0, n - 1).expand(-1, n, -1))
        seen = (j < 0) | ((j < n) & above)
    return seen if counts is None else seen & (i < counts.view(-1, 1, 1))


def _attend(state):
    case, q, scale = state["case"], state["q"], state["scale"]
    b, h, n, d = q.shape
    kv = case["kv_heads"]
    table = state["page_table"].long().clamp_min(0)

    def gathered(pages):   # [B, H_kv, keys, D]
        return pages[table].float().transpose(1, 2).reshape(b, kv, -1, d)

    x = q.float().reshape(b, kv, -1, d)
    s = torch.matmul(x * scale, gathered(state["key_pages"]).transpose(-1, -2)).view(b, h, n, -1)
    s = s.masked_fill(~_seen(state, s.shape[-1]).unsqueeze(1), -math.inf)
    top = s.amax(-1, keepdim=True).clamp_min(torch.finfo(torch.float32).min)
    e = torch.exp(s - top)
    total = e.sum(-1, keepdim=True)
    p = e / total.clamp_min(torch.finfo(torch.float32).tiny)
    out = torch.matmul(p.view(b, kv, -1, p.shape[-1]), gathered(state["value_pages"])).view(b, h, n, d)
    return out.to(q.dtype), (top + torch.log(total)).squeeze(-1)


def _append(state):
    case = state["case"]
    angle = _angles(state["pos"], state["axes"])
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    first, second = _pair_index(state["axes"], case["pairs"], cos.device)
    i = torch.arange(case["tokens"], device="cuda")
    at = state["lengths"].long().view(-1, 1) + i
    page, slot = torch.gather(state["page_table"].long(), 1, at // case["page"]), at % case["page"]
    k = _turn(_normed(state["k"], state["wk"]), cos, sin, first, second)
    for new, pages in ((k, state["key_pages"]), (state["v"], state["value_pages"])):
        new = new.transpose(1, 2).to(pages.dtype)   # [B, N, H, D]
        if state["counts"] is not None:   # a token behind a sequence's last leaves its place as it was
            new = torch.where((i < state["counts"].view(-1, 1))[..., None, None], new, pages[page, :, slot])
        pages[page, :, slot] = new
    q = state["q"]
    if q is not None:
        q = _turn(_normed(q, state["wq"]), cos, sin, first, second).to(q.dtype)
    return [state["key_pages"], state["value_pages"]] + ([] if q is None else [q])


def run(state):
    case = state["case"]
    op = case["op"]
    if own:
        import context_attention_partial_gb300 as cp
        pairs = dict(theta=_THETA, interleaved=case.get("pairs") == "interleaved")
        if op == "norm_rotary":
            return cp.norm_rotary(state["x"], state["w"], state["pos"], state["axes"], eps=_EPS, **pairs)
        if op == "norm_grad":
            dx, dw = cp.norm_rotary_backward(state["x"], state["w"], state["pos"], state["axes"], state["dy"], eps=_EPS,
                                             **pairs)
            return [*dx, *dw]
        if op == "append":
            q = cp.cache_append(state["k"], state["v"], state["key_pages"], state["value_pages"], state["page_table"],
                                state["lengths"], positions=state["pos"], axes_dims=state["axes"], q=state["q"],
                                counts=state["counts"], weight=state["wk"], q_weight=state["wq"], eps=_EPS, **pairs)
            return [state["key_pages"], state["value_pages"]] + ([] if q is None else [q])
        return cp.cache_attention(state["q"], state["key_pages"], state["value_pages"], state["page_table"],
                                  state["lengths"], parents=state["parents"], counts=state["counts"], scale=state["scale"])
    if op == "append":
        return _append(state)
    if op == "attend":
        return _attend(state)
    angle = _angles(state["pos"], state["axes"])
    cos, sin = angle.cos().float(), angle.sin().float()
    first, second = _pair_index(state["axes"], case["pairs"], cos.device)
    if op == "norm_rotary":
        return [_turn(_normed(x, w), cos, sin, first, second).to(x.dtype) for x, w in zip(state["x"], state["w"])]
    grads = [_norm_grad(x, w, dy, cos, sin, first, second) for x, w, dy in zip(state["x"], state["w"], state["dy"])]
    return [dx.to(x.dtype) for (dx, _), x in zip(grads, state["x"])] + \
        [dw.to(w.dtype) for (_, dw), w in zip(grads, state["w"])]


def _exact_turn(x, pos, axes, pairs, sign=1):
    """Each pair as a complex number times e^(i angle); x [B, H, S, D] in 64 bits, pos [S, A] or [B, S, A]."""
    y = x.clone()
    at = 0
    for a, d in enumerate(axes):
        for i in range(d // 2):
            u, w = (at + 2 * i, at + 2 * i + 1) if pairs == "interleaved" else (at + i, at + d // 2 + i)
            angle = pos[..., a].double() * _THETA ** (-2.0 * i / d) * sign
            angle = angle[:, None] if angle.dim() == 2 else angle
            z = torch.complex(x[..., u], x[..., w]) * torch.polar(torch.ones_like(angle), angle)
            y[..., u], y[..., w] = z.real, z.imag
        at += d
    return y


def _exact_normed(x, w):
    return x if w is None else x / torch.sqrt(x.square().mean(-1, keepdim=True) + _EPS) * w.double()


def exact(case, seed):
    """The definitions in 64 bits: sequence by sequence, paths of a tree by their parents, gradients by the chain rule
    through the norm's quotient."""
    s = prepare(case, seed)
    op = case["op"]
    if op == "norm_rotary":
        return [_exact_turn(_exact_normed(x.double(), w), s["pos"], s["axes"], case["pairs"])
                for x, w in zip(s["x"], s["w"])]
    if op == "norm_grad":
        dxs, dws = [], []
        for x, w, dy in zip(s["x"], s["w"], s["dy"]):
            dx, dw = torch.empty(x.shape, dtype=torch.float64, device="cuda"), 0.0
            for h in range(x.shape[1]):   # (a head at a time: memory)
                xx = x[:, h:h + 1].double()
                dz = _exact_turn(dy[:, h:h + 1].double(), s["pos"], s["axes"], case["pairs"], -1)
                rms = torch.sqrt(xx.square().mean(-1, keepdim=True) + _EPS)
                dw = dw + (dz * xx / rms).sum((0, 1, 2))
                u = dz * w.double()
                dx[:, h:h + 1] = (u * rms.square() - xx * (u * xx).mean(-1, keepdim=True)) / rms ** 3
            dxs.append(dx)
            dws.append(dw)
        return dxs + dws
    table, lengths = s["page_table"].tolist(), s["lengths"].tolist()
    counts = [case["tokens"]] * case["batch"] if s["counts"] is None else s["counts"].tolist()
    page = case["page"]
    if op == "append":
        keys, values = s["key_pages"].double(), s["value_pages"].double()
        new = _exact_turn(_exact_normed(s["k"].double(), s["wk"]), s["pos"], s["axes"], case["pairs"])
        for b, (first, n) in enumerate(zip(lengths, counts)):
            done = 0
            while done < n:   # a page's part at a time
                slot = (first + done) % page
                m = min(page - slot, n - done)
                number = table[b][(first + done) // page]
                keys[number, :, slot:slot + m] = new[b, :, done:done + m]
                values[number, :, slot:slot + m] = s["v"][b, :, done:done + m].double()
                done += m
        q = [] if s["q"] is None else [_exact_turn(_exact_normed(s["q"].double(), s["wq"]), s["pos"], s["axes"], case["pairs"])]
        return [keys, values, *q]
    q, scale = s["q"], s["scale"]
    b, h, n, d = q.shape
    group = h // case["kv_heads"]
    zero = dict(dtype=torch.float64, device="cuda")
    out, lse = torch.zeros(b, h, n, d, **zero), torch.full((b, h, n), -math.inf, **zero)
    for i in range(b):
        m, first = counts[i], lengths[i]
        if m == 0:
            continue
        numbers = torch.tensor(table[i][:-(-(first + m) // page)], device="cuda")
        hidden = torch.triu(torch.ones(m, m, dtype=torch.bool, device="cuda"), 1)
        if s["parents"] is not None:
            parents = s["parents"][i].tolist()
            paths = [[False] * m for _ in range(m)]
            for x in range(m):
                y = x
                while y >= 0:
                    paths[x][y] = True
                    y = parents[y]
            hidden = ~torch.tensor(paths, device="cuda")
        for j in range(case["kv_heads"]):
            k = s["key_pages"][numbers, j].double().reshape(-1, d)[:first + m]
            v = s["value_pages"][numbers, j].double().reshape(-1, d)[:first + m]
            for g in range(j * group, (j + 1) * group):
                z = q[i, g, :m].double() @ k.T * scale
                z[:, first:] = z[:, first:].masked_fill(hidden, -math.inf)
                lse[i, g, :m] = torch.logsumexp(z, -1)
                out[i, g, :m] = torch.exp(z - lse[i, g, :m, None]) @ v
    return out, lse


def work(case):
    """Each input read once, each output written once; the products of the definition."""
    es, b, d, h, kv = 4 if case["dtype"] == "f32" else 2, case["batch"], case["dim"], case["heads"], case["kv_heads"]
    op = case["op"]
    if op in ("norm_rotary", "norm_grad"):
        n = case["text"] + case["t"] * case["h"] * case["w"]
        values = b * n * (h + kv) * d
        tensors, flops = (2, 8) if op == "norm_rotary" else (3, 18)
        return {"bytes": tensors * values * es + 4 * n * len(_axes(case)), "flops": flops * values}
    n, context = case["tokens"], case["context"]
    # ragged: three quarters of the cache and of the new tokens on average, one sequence in four has none of these
    rows = b * n * (0.75 * (b - b // 4) / b if case["ragged"] else 1.0)
    if op == "append":
        values = 2 * rows * kv * d + (b * n * h * d if case["queries"] else 0)
        return {"bytes": 2 * values * es + 4 * b * n, "flops": (8 if case["norm"] else 3) * values}
    sequences = b - b // 4 if case["ragged"] else b
    cached = context * (0.75 if case["ragged"] else 1.0)
    new = rows / sequences
    seen = cached + (new / 2 if not case["tree"] else min(new, 8))   # keys that a row sees
    keys = sequences * (cached + new)
    return {"bytes": es * d * (2 * b * n * h + 2 * keys * kv) + 4 * b * n * h, "flops": 4 * d * rows * h * seen}
