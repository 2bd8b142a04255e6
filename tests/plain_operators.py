"""Plain 64-bit forms of the rotary and cross-attention operators, and how far
a kernel's fp32 (or bf16) result may be from them.

Tolerances count roundings.  u is half a step of the type relative to the
value (bf16 2^-8, fp32 2^-24).  A bf16 attention rounds each probability (and
each ds) once to bf16 before its product and each output once, so an output
o = sum_j p_j v_j is within u (|o| + sum_j p_j |v_j|) of the exact one, plus
what fp32 arithmetic adds: scores off by at most (D + 4) 2^-24 |q| |k| scale,
probabilities by twice that relatively, sums by n 2^-24.
"""
import math

import torch

U = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
F32 = 2.0 ** -24


def rotary(x, pos, axes, theta=10000.0, interleaved=True, inverse=False):
    """x [B,H,S,D], pos [S,A] or [B,S,A] -> fp64, and sum of the magnitudes that make up each value."""
    y = x.double()
    out, mag = y.clone(), y.abs().clone()
    base = 0
    for a, d in enumerate(axes):
        for i in range(d // 2):
            u, w = (base + 2 * i, base + 2 * i + 1) if interleaved else (base + i, base + d // 2 + i)
            angle = pos[..., a].double() * math.exp(-2.0 * i / d * math.log(theta))
            angle = angle[:, None] if pos.dim() == 3 else angle
            c, s = angle.cos(), angle.sin() * (-1 if inverse else 1)
            out[..., u], out[..., w] = y[..., u] * c - y[..., w] * s, y[..., u] * s + y[..., w] * c
            mag[..., u] = mag[..., w] = y[..., u].abs() + y[..., w].abs()
        base += d
    return out, mag


def rotary_tolerance(out, mag, dtype):
    # the type's rounding (bf16; fp32's is among the eight), and in fp32: two
    # products and a sum, cos and sin off by 2^-22 (the angle by 2^-24 turns,
    # the functions by 2 steps)
    return U[dtype] * out.abs() * 1.001 * (dtype == torch.bfloat16) + 8 * 2 * F32 * mag


def cross(q, k, v, lengths=None, scale=None, dout=None):
    """fp64 attention of each sequence's first lengths[b] keys and, with dout,
    its gradients, with each result's tolerance: a dict name -> (value, tolerance)."""
    dtype = q.dtype
    u = U[dtype] if dtype == torch.bfloat16 else 0.0
    B, H, M, D = q.shape
    N, g = k.shape[2], H // k.shape[1] if k.shape[1] else 1
    scale = D ** -0.5 if scale is None else scale
    z = lambda *s: torch.zeros(*s, dtype=torch.float64, device=q.device)
    r = {n: z(B, H, M, D) for n in ("out", "out_tol", "dq", "dq_tol")}
    r.update({n: z(*k.shape) for n in ("dk", "dk_tol", "dv", "dv_tol")})
    r["lse"], r["lse_tol"] = z(B, H, M) - math.inf, z(B, H, M)
    for b in range(B):
        n = N if lengths is None else max(0, min(N, int(lengths[b])))
        if n == 0:
            continue
        for h in range(H):
            Q, K, V = q[b, h].double(), k[b, h // g, :n].double(), v[b, h // g, :n].double()
            s = Q @ K.T * scale
            lse = torch.logsumexp(s, -1)
            p = torch.exp(s - lse[:, None])
            # scores in fp32, base-2 exponents of up to |s| log2 e: their rounding too
            s_err = (D + 4) * F32 * (Q.norm(dim=-1)[:, None] * K.norm(dim=-1)[None] * scale) \
                + 4 * F32 * (s.abs() + lse.abs()[:, None] + 1)
            rel = 2 * s_err.amax(-1, keepdim=True) + (n + 8) * F32          # of every probability
            r["out"][b, h] = o = p @ V
            r["out_tol"][b, h] = u * o.abs() + (u + rel) * (p @ V.abs()) * 1.01
            r["lse"][b, h] = lse
            r["lse_tol"][b, h] = s_err.amax(-1) + (n + 8) * F32 + 4 * F32 * lse.abs()
            if dout is None:
                continue
            G = dout[b, h].double()
            dp = G @ V.T
            # delta comes from the output as the forward call rounded it
            delta = (G * o).sum(-1, keepdim=True)
            d_err = (G.abs() * (r["out_tol"][b, h] + (D + 4) * F32 * o.abs())).sum(-1, keepdim=True)
            dp_err = (D + 4) * F32 * (G.norm(dim=-1)[:, None] * V.norm(dim=-1)[None])
            ds = p * (dp - delta)
            # ds rounded to bf16 from a p that may itself have been rounded
            ds_err = (2 * u + rel + 4 * F32) * ds.abs() + p * (d_err + dp_err)
            r["dq"][b, h] = x = ds @ K * scale
            r["dq_tol"][b, h] = u * x.abs() + (ds_err + n * F32 * ds.abs()) @ K.abs() * scale * 1.01
            m = M * g
            r["dk"][b, h // g, :n] += ds.T @ Q * scale
            r["dk_tol"][b, h // g, :n] += (ds_err + m * F32 * ds.abs()).T @ Q.abs() * scale * 1.01
            r["dv"][b, h // g, :n] += p.T @ G
            r["dv_tol"][b, h // g, :n] += ((u + rel + m * F32) * p).T @ G.abs() * 1.01
    for name in ("dk", "dv"):
        r[name + "_tol"] += u * r[name].abs() + 2 * F32 * r[name].abs()
    for name in ("out", "dq"):
        r[name + "_tol"] += 2 * F32 * r[name].abs()
    return {n: (r[n], r[n + "_tol"]) for n in ("out", "lse", "dq", "dk", "dv")}


def worst(got, want, tol):
    """Largest |got - want| / tol (tol 0: equal, or infinite); equal infinities count as 0."""
    got = got.double()
    same = got == want
    ratio = torch.where(same, torch.zeros_like(want), (got - want).abs() / tol)
    return float(torch.nan_to_num(ratio, nan=math.inf).max()) if ratio.numel() else 0.0
