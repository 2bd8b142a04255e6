"""Cross attention and its gradient on tensors past 2^31 elements, with results
that come from a few rows or keys at the start, in the middle and at the far end:
what one of those places adds is large against the tolerance, so a result that
leaves it out, or a zero, fails (and is asserted to)."""
import pytest
import torch

import context_attention_partial_gb300 as cp
import plain_operators as plain
from context_attention_partial_gb300 import _lib
from context_attention_partial_gb300 import build as _build

pytestmark = [pytest.mark.gpu, pytest.mark.slow]
DEV = "cuda:0"
BF = torch.bfloat16
F32 = 2.0 ** -24


@pytest.fixture
def both(monkeypatch):
    """Runs a call through the check build, then through the normal one."""
    chk, normal = _lib.bind(_build.build(check=True)), cp.load_library()

    def run(call):
        monkeypatch.setattr(_lib, "load", lambda: chk)
        call()
        assert chk.cpattn_last_device_status(torch.cuda.current_stream().cuda_stream) == 0
        monkeypatch.setattr(_lib, "load", lambda: normal)
        got = call()
        assert cp.last_device_status() == 0
        return got
    yield run
    torch.cuda.empty_cache()


def normal(seed, *shape):
    g = torch.Generator(DEV).manual_seed(seed)
    return torch.cat([torch.randn(*shape[:2], min(1 << 20, shape[2] - i), shape[3], generator=g, device=DEV).to(BF)
                      for i in range(0, shape[2], 1 << 20)], 2)


def windows(n, width):
    return [slice(0, width), slice(n // 2, n // 2 + width), slice(n - width, n)]


def check(got, want, tol, without):
    """Within the tolerance, which neither a zero nor `without` (a window left out)
    would be."""
    assert plain.worst(got, want, tol) <= 1.0
    assert plain.worst(torch.zeros_like(want), want, tol) > 4
    for other in without:
        assert plain.worst(other, want, tol) > 4


def test_gradients_of_query_rows_far_apart(both):
    """dout is 0 but for 100 rows in each of three places, so dk and dv are sums
    over those rows: the others add exact zeros."""
    M, D, keys = (1 << 23) + 131, 128, (70, 33)
    q, k, v = normal(1, 2, 1, M, D), normal(2, 2, 1, 70, D), normal(3, 2, 1, 70, D)
    assert q.numel() > 1 << 31
    n = torch.tensor(keys, dtype=torch.int32, device=DEV)
    dout = torch.zeros_like(q)
    places = windows(M, 100)
    for i, w in enumerate(places):
        # (a common offset: what the places add to dv does not cancel)
        dout[:, :, w] = (normal(4 + i, 2, 1, 100, D).float() + 1).to(BF)
    out, lse = both(lambda: cp.cross_attention(q, k, v, kv_lengths=n))
    dq, dk, dv = both(lambda: cp.cross_attention_backward(q, k, v, out, lse, dout, kv_lengths=n))
    take = lambda ws: [torch.cat([t[:, :, w] for w in ws], 2) for t in (q, dout)]
    rows = take(places)
    want = plain.cross(rows[0], k, v, keys, dout=rows[1])
    fewer = []
    for left in range(3):
        r = take([w for i, w in enumerate(places) if i != left])
        fewer.append(plain.cross(r[0], k, v, keys, dout=r[1]))
    for name, got in (("dk", dk), ("dv", dv)):
        check(got, *want[name], [f[name][0] for f in fewer])
    check(torch.cat([dq[:, :, w] for w in places], 2), *want["dq"], [])
    quiet = torch.ones(M, dtype=torch.bool, device=DEV)
    for w in places:
        quiet[w] = False
    for at in range(0, M, 1 << 20):
        some = quiet[at:at + (1 << 20)]
        assert torch.all(dq[:, :, at:at + (1 << 20)][:, :, some] == 0)


def test_weight_on_keys_far_apart(both):
    """Keys along the queries' direction in three places hold nearly all weight:
    output, lse, dq, dk and dv come from them."""
    N, D, H, Hk, width = (1 << 23) + 77, 128, 4, 2, 40
    g = torch.Generator(DEV).manual_seed(10)
    c = 1.4 * (torch.randint(0, 2, (D,), generator=g, device=DEV) * 2 - 1).float()   # |c|^2 / sqrt(D) = 22
    q = (c + 0.1 * torch.randn(1, H, 1, D, generator=g, device=DEV)).to(BF)
    dout = (1 + 0.3 * torch.randn(1, H, 1, D, generator=g, device=DEV)).to(BF)
    k, v = normal(11, 1, Hk, N, D), normal(12, 1, Hk, N, D)
    k *= 0.25
    places = windows(N, width)
    for w, offset in zip(places, (2.0, -1.0, -1.0)):   # (values of their own: dp tells the places apart)
        k[:, :, w] = (c + 0.3 * torch.randn(1, Hk, width, D, generator=g, device=DEV)).to(BF)
        v[:, :, w] = (v[:, :, w].float() + offset).to(BF)
    assert k.numel() > 1 << 31
    out, lse = both(lambda: cp.cross_attention(q, k, v))
    dq, dk, dv = both(lambda: cp.cross_attention_backward(q, k, v, out, lse, dout))
    share, scale, u = H // Hk, D ** -0.5, 2.0 ** -8
    heavy = torch.zeros(N, dtype=torch.bool, device=DEV)
    for w in places:
        heavy[w] = True
    # fp32 sums of N terms by lanes and parts: at most 2^16 additions each
    rel = 2.0 ** 16 * F32
    for h in range(H):
        K = [k[0, h // share, i:i + (1 << 20)].double() for i in range(0, N, 1 << 20)]
        V = [v[0, h // share, i:i + (1 << 20)].double() for i in range(0, N, 1 << 20)]
        Q, G = q[0, h, 0].double(), dout[0, h, 0].double()
        s = torch.cat([x @ Q for x in K]) * scale
        L = torch.logsumexp(s, 0)
        p = torch.exp(s - L)
        assert float(p[heavy].sum()) > 0.9
        p_of = torch.split(p, 1 << 20)
        dp = torch.cat([x @ G for x in V])

        def attend(weights):
            return sum(a @ x for a, x in zip(torch.split(weights, 1 << 20), V))

        o, mag = attend(p), sum(a @ x.abs() for a, x in zip(p_of, V))
        # scores: D + 4 roundings of |q| |k|, and 4 of their size, as in plain_operators
        p_rel = 2 * ((D + 4) * F32 * float(Q.norm() * 1.5 * c.norm()) * scale + 4 * F32 * 60) + rel
        tol_o = u * o.abs() + (u + p_rel) * mag * 1.01 + 2 * F32 * o.abs()
        without = []
        for w in places:
            part = p.clone()
            part[w] = 0
            without.append(attend(part))
        check(out[0, h, 0], o, tol_o, without)
        assert abs(float(lse[0, h, 0].double() - L)) <= p_rel + 4 * F32 * abs(float(L))
        delta = float(G @ o)
        d_err = float((G.abs() * (tol_o + (D + 4) * F32 * o.abs())).sum())
        ds = p * (dp - delta)
        dp_err = (D + 4) * F32 * float(G.norm() * max(x.norm(dim=-1).max() for x in V))
        ds_err = (2 * u + p_rel + 4 * F32) * ds.abs() + p * (d_err + dp_err)
        spread = lambda w, f=lambda x: x: sum(a @ f(x) for a, x in zip(torch.split(w, 1 << 20), K))
        x = spread(ds) * scale
        tol_q = u * x.abs() + spread(ds_err + rel * ds.abs(), torch.abs) * scale * 1.01 + 2 * F32 * x.abs()
        without = []
        for w in places:
            part = ds.clone()
            part[w] = 0
            without.append(spread(part) * scale)
        assert plain.worst(dq[0, h, 0], x, tol_q) <= 1.0
        assert all(plain.worst(y, x, tol_q) > 4 for y in without)
        if h % share == 0:
            want_k = torch.zeros(N, dtype=torch.float64, device=DEV)
            sums = {name: [torch.zeros(3 * width, D, dtype=torch.float64, device=DEV) for _ in range(2)] for name in ("dk", "dv")}
        for name, w, e, vec in (("dk", ds, ds_err, Q * scale), ("dv", p, (u + p_rel) * p, G)):
            sums[name][0] += w[heavy][:, None] * vec
            sums[name][1] += e[heavy][:, None] * vec.abs() * 1.01
        want_k += p
        if h % share == share - 1:
            for name, got in (("dk", dk), ("dv", dv)):
                value, tol = sums[name]
                tol = tol + (u + 4 * F32) * value.abs()
                check(got[0, h // share][heavy], value, tol, [])
            # ordinary keys between the places: dv is small there, and not 0
            for at in (width + 5, N // 4, N - width - 5):
                got = dv[0, h // share, at].double()
                assert 0 < float(got.norm()) <= float(want_k[at]) * 2 * float(dout[0].double().norm(dim=-1).max())
