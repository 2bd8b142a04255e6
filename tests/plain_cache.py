"""Plain 64-bit forms of the per-head norms with rotary positions, their gradient, and
of a paged cache, and how far a kernel's fp32 (or bf16) result may be from them.

Tolerances count roundings; u = 2^-24 is half a step of fp32 relative to the value.
A row's sum of squares: at most 8 products in a lane, 5 additions over the lanes, the
factor 1 / D and eps, all of one sign, 16 u; its inverse root half of that and two
steps of its own (4 u): r is within 12 u.  A turned value: 16 u of the magnitudes that
make it up (``plain_operators.rotary_tolerance``), and 2 u for its two factors.
"""
import math

import torch

import plain_operators as P

U = P.U
F32 = P.F32


def norm_rotary(x, w, pos, axes, eps=1e-6, theta=10000.0, interleaved=True, norm=True):
    """fp64 result and tolerance.  w None: ones.  pos None: not turned."""
    dtype = x.dtype
    z = x.double()
    if norm:
        z = z * torch.rsqrt(z.square().mean(-1, keepdim=True) + eps)
        if w is not None:
            z = z * w.double()
    if pos is None:
        y, mag = z, z.abs()
    else:
        y, mag = P.rotary(z, pos, axes, theta, interleaved)
    u = U[dtype] * 1.001 if dtype == torch.bfloat16 else 0.0
    return y, u * y.abs() + 32 * F32 * mag


def norm_rotary_backward(x, w, pos, axes, dy, eps=1e-6, theta=10000.0, interleaved=True):
    """fp64 (dx, dw) and their tolerances."""
    u = U[x.dtype] * 1.001 if x.dtype == torch.bfloat16 else 0.0
    D = x.shape[-1]
    z = x.double()
    wd = torch.ones(D, dtype=torch.float64, device=x.device) if w is None else w.double()
    dz, mag = P.rotary(dy, pos, axes, theta, interleaved, inverse=True)     # dz within 16 u of mag
    r = torch.rsqrt(z.square().mean(-1, keepdim=True) + eps)
    g = dz * wd
    s = (g * z).sum(-1, keepdim=True)
    s_abs = (wd.abs() * mag * z.abs()).sum(-1, keepdim=True)
    dx = r * (g - z * r * r * s / D)
    # s: its terms 16 + 3 u, sums of 8 and over 5 lanes; x r^2 s / D: r twice (24 u) and
    # four products; the whole: r (12 u), a difference and a product
    dx_tol = u * dx.abs() + r * (32 * F32 * wd.abs() * mag + z.abs() * r * r / D * (32 + 32 + 16) * F32 * s_abs)
    terms = dz * z * r
    n = terms[..., 0].numel()
    dw = terms.sum((0, 1, 2))
    uw = 0.0 if w is None or w.dtype != torch.bfloat16 else U[w.dtype] * 1.001
    # a term: 16 u of its magnitude, r and three products; n additions at most in a row
    dw_tol = uw * dw.abs() + (32 + n) * F32 * (mag * z.abs() * r).sum((0, 1, 2)) + F32 * dw.abs()
    return (dx, dx_tol), (dw, dw_tol)


def ancestors(parents, n):
    """[n][n] booleans of one sequence: whether draft j is draft i or above it."""
    seen = torch.zeros(n, n, dtype=torch.bool)
    for i in range(n):
        j = i
        while j >= 0:
            seen[i, j] = True
            up = int(parents[j])
            j = up if up < j else -1
    return seen


class Cache:
    """A pool of pages in random order with sequences of given lengths.  Rows of the pool
    that hold no token of a sequence are NaN, and so are pages of nobody; table entries
    behind a sequence's pages are -1."""

    def __init__(self, lengths, counts, S, kv_heads, D, page, dtype, device, seed=0, layout="phrd", extra=2):
        g = torch.Generator("cpu").manual_seed(seed)
        B = len(lengths)
        self.lengths, self.S, self.page = list(lengths), S, page
        self.counts = [S] * B if counts is None else list(counts)
        used = [-(-(n + c) // page) for n, c in zip(lengths, self.counts)]
        width = max(used + [1]) + 1
        total = sum(used) + extra
        order = torch.randperm(total, generator=g).tolist()
        table = torch.full((B, width), -1, dtype=torch.int32)
        for b in range(B):
            for i in range(used[b]):
                table[b, i] = order.pop()
        shape = (total, kv_heads, page, D) if layout == "phrd" else (total, page, kv_heads, D)
        self.key_pages, self.value_pages = (torch.full(shape, math.nan).to(dtype).to(device) for _ in range(2))
        if layout != "phrd":
            self.key_pages, self.value_pages = self.key_pages.transpose(1, 2), self.value_pages.transpose(1, 2)
        self.k, self.v = [], []          # per sequence [H_kv, keys, D]
        for b in range(B):
            n = self.lengths[b] + self.counts[b]
            self.k.append(torch.randn(kv_heads, n, D, generator=g).to(dtype).to(device))
            self.v.append(torch.randn(kv_heads, n, D, generator=g).to(dtype).to(device))
        self.table = table.to(device)
        self.lengths_t = torch.tensor(lengths, dtype=torch.int32, device=device)
        self.counts_t = None if counts is None else torch.tensor(counts, dtype=torch.int32, device=device)
        for b in range(B):
            self.write(b, 0, self.k[b], self.v[b])

    def places(self, b, first, n):
        at = torch.arange(first, first + n, device=self.table.device)
        return self.table[b].long()[at // self.page], at % self.page

    def write(self, b, first, k, v):
        page, row = self.places(b, first, k.shape[1])
        self.key_pages[page, :, row] = k.transpose(0, 1)
        self.value_pages[page, :, row] = v.transpose(0, 1)

    def read(self, b, n):
        page, row = self.places(b, 0, n)
        return (self.key_pages[page, :, row].transpose(0, 1), self.value_pages[page, :, row].transpose(0, 1))


def attend(q, k, v, lengths, counts, parents=None, scale=None):
    """fp64 attention of q [B,H,S,D]; k, v: per sequence [H_kv, keys, D]; parents: per
    sequence lists, or None.  Returns ((out, tolerance), (lse, tolerance)), tolerances
    as plain_operators.cross derives them."""
    B, H, S, D = q.shape
    u = U[q.dtype] if q.dtype == torch.bfloat16 else 0.0
    scale = D ** -0.5 if scale is None else scale
    z = lambda *s: torch.zeros(*s, dtype=torch.float64, device=q.device)
    out, out_tol, lse, lse_tol = z(B, H, S, D), z(B, H, S, D), z(B, H, S) - math.inf, z(B, H, S)
    for b in range(B):
        n, c = lengths[b], counts[b]
        if c == 0:
            continue
        tree = torch.ones(c, c, dtype=torch.bool).tril() if parents is None else ancestors(parents[b], c)
        seen = torch.cat([torch.ones(c, n, dtype=torch.bool), tree], 1).to(q.device)
        group = H // k[b].shape[0]
        for h in range(H):
            Q, K, V = q[b, h, :c].double(), k[b][h // group].double(), v[b][h // group].double()
            V = torch.where(seen.any(0)[:, None], V, 0.0)
            s = Q @ K.T * scale
            s_err = (D + 4) * F32 * (Q.norm(dim=-1)[:, None] * K.norm(dim=-1)[None] * scale)
            s = s.masked_fill(~seen, -math.inf)
            L = torch.logsumexp(s, -1)
            p = torch.exp(s - L[:, None])
            s_err = torch.where(seen, s_err + 4 * F32 * (s.abs() + L.abs()[:, None] + 1), 0.0)
            rel = 2 * s_err.amax(-1, keepdim=True) + (n + c + 8) * F32
            o = p @ V
            out[b, h, :c] = o
            out_tol[b, h, :c] = u * o.abs() + (u + rel) * (p @ V.abs()) * 1.01 + 2 * F32 * o.abs()
            lse[b, h, :c] = L
            lse_tol[b, h, :c] = s_err.amax(-1) + (n + c + 8) * F32 + 4 * F32 * L.abs()
    return (out, out_tol), (lse, lse_tol)


def tree(S, B, seed=0, back=8):
    """Parents [B][S]: one of the `back` drafts before, or none."""
    g = torch.Generator("cpu").manual_seed(seed)
    step = torch.randint(1, back + 1, (B, S), generator=g)
    return (torch.arange(S) - step).clamp_min(-1)
