"""The paged cache: new tokens' way to it, and the attention of chains and trees to it,
against the definitions in 64 bits."""
import math

import pytest
import torch

import context_attention_partial_gb300 as cp
import plain_cache as C
import plain_operators as P

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32
OK, BOUNDS = 0, 10


def randn(*shape, dtype, seed, layout="bhsd"):
    g = torch.Generator("cpu").manual_seed(seed)
    if layout == "bshd":
        b, h, s, d = shape
        return torch.randn(b, s, h, d, generator=g).to(dtype).to(DEV).transpose(1, 2)
    return torch.randn(*shape, generator=g).to(dtype).to(DEV)


def check(got, want_tol):
    want, tol = want_tol
    assert got.shape == want.shape
    assert P.worst(got, want, tol) <= 1


def bits(t):
    return t.contiguous().view(torch.int16 if t.dtype == BF else torch.int32)


# ------------------------------------------------------------------- append
# (B, H, Hk, S, D, page, lengths, counts, axes)
APPEND = [
    (1, 4, 4, 1, 128, 16, (0,), None, (128,)),
    (2, 8, 2, 1, 128, 64, (63, 64), None, (128,)),
    (3, 6, 2, 7, 64, 16, (9, 0, 700), (7, 3, 0), (64,)),
    (2, 4, 1, 130, 64, 32, (31, 5), (130, 1), (16, 24, 24)),
    (1, 2, 2, 40, 24, 1024, (1000,), None, (8, 8)),
    (4, 32, 8, 5, 128, 128, (1, 2, 126, 127), (5, 4, 2, 1), (128,)),
]


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("interleaved", [True, False])
@pytest.mark.parametrize("case", APPEND, ids=lambda c: "x".join(map(str, c[:6])))
def test_append(case, interleaved, dtype):
    B, H, Hk, S, D, page, lengths, counts, axes = case
    for seed, (layout, pages, with_q, normed, turned) in enumerate((("bhsd", "phrd", True, True, True),
                                                                    ("bshd", "prhd", False, True, False),
                                                                    ("bshd", "phrd", True, False, True),
                                                                    ("bhsd", "prhd", True, False, False))):
        cache = C.Cache(lengths, counts, S, Hk, D, page, dtype, DEV, seed, pages)
        k, v = randn(B, Hk, S, D, dtype=dtype, seed=1, layout=layout), randn(B, Hk, S, D, dtype=dtype, seed=2, layout=layout)
        q = randn(B, H, S, D, dtype=dtype, seed=3, layout=layout) if with_q else None
        w = [1 + 0.2 * randn(D, dtype=dtype, seed=s) for s in (4, 5)] if normed else [None, None]
        pos = (cache.lengths_t[:, None, None] + torch.arange(S, device=DEV)[:, None]).float().expand(B, S, len(axes))
        pos = pos if turned else None
        before = [bits(t).clone() for t in (cache.key_pages, cache.value_pages)]
        got = cp.cache_append(k, v, cache.key_pages, cache.value_pages, cache.table, cache.lengths_t, positions=pos,
                              axes_dims=axes if turned else (), q=q, counts=cache.counts_t, weight=w[0],
                              q_weight=w[1] if with_q else None, interleaved=interleaved)
        assert cp.last_device_status() == OK
        want_k, tol_k = C.norm_rotary(k, w[0], pos, axes, interleaved=interleaved, norm=normed)
        if with_q:
            check(got, C.norm_rotary(q, w[1], pos, axes, interleaved=interleaved, norm=normed))
        else:
            assert got is None
        after = [bits(t).clone() for t in (cache.key_pages, cache.value_pages)]
        for b in range(B):
            n = cache.counts[b]
            page_no, row = cache.places(b, lengths[b], n)
            new_k = cache.key_pages[page_no, :, row].transpose(0, 1)
            new_v = cache.value_pages[page_no, :, row].transpose(0, 1)
            if normed or turned:
                assert P.worst(new_k, want_k[b, :, :n], tol_k[b, :, :n]) <= 1
            else:
                assert torch.equal(new_k, k[b, :, :n])
            assert torch.equal(new_v, v[b, :, :n])
            for new, old in zip(after, before):   # everything else as it was
                new[page_no, :, row] = old[page_no, :, row]
        assert all(torch.equal(a, b) for a, b in zip(after, before))


def test_append_values_keep_their_bits():
    cache = C.Cache((3,), None, 2, 1, 64, 16, BF, DEV)
    v = torch.randint(-2 ** 15, 2 ** 15, (1, 1, 2, 64), dtype=torch.int16).view(BF).to(DEV)   # NaNs among them
    cp.cache_append(v, v, cache.key_pages, cache.value_pages, cache.table, cache.lengths_t)
    page, row = cache.places(0, 3, 2)
    for pages in (cache.key_pages, cache.value_pages):
        assert torch.equal(bits(pages[page, :, row].transpose(0, 1)), bits(v[0]))


def test_append_queries_in_place():
    cache = C.Cache((3, 8), None, 5, 2, 64, 16, BF, DEV)
    k, q = randn(2, 2, 5, 64, dtype=BF, seed=1), randn(2, 4, 5, 64, dtype=BF, seed=2)
    pos = torch.arange(5, device=DEV).float()[:, None]
    args = (k, k, cache.key_pages, cache.value_pages, cache.table, cache.lengths_t)
    for interleaved in (True, False):
        kw = dict(positions=pos, axes_dims=(64,), interleaved=interleaved)
        want = cp.cache_append(*args, q=q, **kw)
        mine = q.clone()
        assert cp.cache_append(*args, q=mine, q_out=mine, **kw) is mine and torch.equal(mine, want)


def test_append_to_bad_places():
    """Tokens whose page is not in the pool, or past the table, are not written; the others are."""
    cache = C.Cache((14, 14, 14, -3), None, 4, 2, 64, 16, BF, DEV)
    cache.lengths_t = torch.tensor([14, 14, 46, -3], dtype=torch.int32, device=DEV)
    P_ = cache.key_pages.shape[0]
    table = cache.table.clone()
    assert table.shape[1] == 3 and 46 // 16 == 2
    table[0, 1], table[1, 1], table[2, 2] = P_, -7, cache.table[2, 0]
    k = randn(4, 2, 4, 64, dtype=BF, seed=1)
    before = [bits(t).clone() for t in (cache.key_pages, cache.value_pages)]
    assert cp.last_device_status() == OK
    cp.cache_append(k, k, cache.key_pages, cache.value_pages, table, cache.lengths_t)
    assert cp.last_device_status() == BOUNDS and cp.last_device_status() == OK
    kb = bits(k)
    for b, i, page, row in ((0, 0, cache.table[0, 0], 14), (0, 1, cache.table[0, 0], 15), (1, 0, cache.table[1, 0], 14),
                            (1, 1, cache.table[1, 0], 15), (2, 0, cache.table[2, 0], 14), (2, 1, cache.table[2, 0], 15),
                            (3, 0, cache.table[3, 0], 0), (3, 1, cache.table[3, 0], 1), (3, 2, cache.table[3, 0], 2),
                            (3, 3, cache.table[3, 0], 3)):
        for want in before:
            want[int(page), :, row] = kb[b, :, i]
    assert torch.equal(bits(cache.key_pages), before[0]) and torch.equal(bits(cache.value_pages), before[1])


# ---------------------------------------------------------------- attention
# (H, Hk, S, D, page, lengths, counts)
ATTEND = [
    (4, 4, 1, 128, 16, (0,), None),                       # a first token sees itself
    (8, 2, 1, 128, 64, (63, 64, 65), None),
    (8, 8, 1, 64, 32, (5000, 17, 0, 300), (1, 1, 0, 1)),
    (32, 8, 1, 128, 64, (9000, 4000), None),
    (6, 2, 7, 64, 16, (9, 0, 700), (7, 3, 0)),            # (21 rows a key head)
    (8, 1, 4, 128, 128, (1000, 130), (4, 2)),             # 32 rows
    (4, 2, 27, 128, 32, (2100, 40, 127), (27, 1, 20)),    # 54 rows
    (3, 1, 30, 64, 16, (777,), None),                     # 90 rows
    (8, 2, 64, 128, 64, (1500, 64), (64, 33)),            # 256 rows
    (2, 2, 200, 64, 256, (300, 0), (200, 131)),           # 200 rows
    (2, 1, 256, 128, 1024, (1030,), None),                # 512 rows
    (16, 1, 17, 128, 16, (5, 40), (17, 9)),               # 272 rows
    (1, 1, 5, 64, 16, (40000,), None),                    # one unit over many blocks
    (12, 4, 70, 128, 64, (130, 500), (70, 66)),           # 210 rows, not a divisor of the tile
]


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("kind", ["chain", "tree"])
@pytest.mark.parametrize("case", ATTEND, ids=lambda c: "x".join(map(str, c[:5])))
def test_attention(case, kind, dtype):
    H, Hk, S, D, page, lengths, counts = case
    B = len(lengths)
    layout, pages = ("bshd", "prhd") if S % 2 else ("bhsd", "phrd")
    cache = C.Cache(lengths, counts, S, Hk, D, page, dtype, DEV, S + H, pages)
    q = randn(B, H, S, D, dtype=dtype, seed=9, layout=layout)
    parents = C.tree(S, B, S) if kind == "tree" else None
    pt = None if parents is None else parents.to(torch.int32).to(DEV)
    kw = dict(parents=pt, counts=cache.counts_t, scale=0.11)
    out, lse = cp.cache_attention(q, cache.key_pages, cache.value_pages, cache.table, cache.lengths_t, **kw)
    assert cp.last_device_status() == OK
    assert out.dtype == dtype and out.stride() == q.stride() and lse.dtype == F32
    want = C.attend(q, cache.k, cache.v, cache.lengths, cache.counts, None if parents is None else parents.tolist(), 0.11)
    check(out, want[0])
    check(lse, want[1])
    again = cp.cache_attention(q, cache.key_pages, cache.value_pages, cache.table, cache.lengths_t, **kw)
    assert torch.equal(again[0], out) and torch.equal(again[1], lse)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("case", [(16, 8, 700, 128, 64, (900, 35), (700, 641)), (24, 8, 900, 64, 32, (33, 2000), None)],
                         ids=lambda c: "x".join(map(str, c[:5])))
def test_attention_of_many_units_over_many_blocks(case, dtype):
    """So many rows, of units that blocks share, that one thread joins all parts of an item."""
    test_attention(case, "chain", dtype)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("S", [1, 2, 31, 100])
@pytest.mark.parametrize("H,Hk", [(4, 4), (8, 2), (5, 1)])
def test_attention_at_tile_borders(H, Hk, S, dtype):
    """Cached tokens around the sizes of tiles and pages, in one ragged batch."""
    lengths = [0, 1, 15, 16, 17, 31, 33, 63, 64, 65, 127, 128, 129, 191, 192, 193, 255, 257]
    counts = [S if i % 3 else (S + 1) // 2 for i in range(len(lengths))]
    cache = C.Cache(lengths, counts, S, Hk, 64, 16, dtype, DEV, S)
    q = randn(len(lengths), H, S, 64, dtype=dtype, seed=10)
    parents = C.tree(S, len(lengths), S + 1, back=3)
    for par in (None, parents):
        pt = None if par is None else par.to(torch.int32).to(DEV)
        out, lse = cp.cache_attention(q, cache.key_pages, cache.value_pages, cache.table, cache.lengths_t, parents=pt,
                                      counts=cache.counts_t)
        want = C.attend(q, cache.k, cache.v, lengths, counts, None if par is None else par.tolist())
        check(out, want[0])
        check(lse, want[1])


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("H,S", [(2, 9), (8, 30)])
def test_drafts_beside_a_query_have_no_part(H, S, dtype):
    """Keys and values of drafts that a query does not see may hold anything; those that it
    sees reach its result, infinities included."""
    lengths, bad = [50, 3], 4
    parents = torch.tensor([[-1, 0, 0, 1, 0, 4, 2, 5, 3] + [8] * (S - 9)] * 2)
    cache = C.Cache(lengths, None, S, 1, 64, 16, dtype, DEV, 3)
    q = randn(2, H, S, 64, dtype=dtype, seed=11)
    pt = parents.to(torch.int32).to(DEV)
    run = lambda: cp.cache_attention(q, cache.key_pages, cache.value_pages, cache.table, cache.lengths_t, parents=pt)
    out, lse = run()
    below = [i for i in range(S) if bool(C.ancestors(parents[0], S)[i, bad])]
    rest = [i for i in range(S) if i not in below]
    assert below[:3] == [4, 5, 7]
    page, row = cache.places(0, lengths[0] + bad, 1)
    clean_v = cache.value_pages[page, :, row].clone()
    for value in (math.nan, math.inf, -math.inf):
        cache.value_pages[page, :, row, 7] = value
        o, l = run()
        assert torch.equal(l, lse) and torch.equal(o[1], out[1])
        assert torch.equal(o[0][:, rest], out[0][:, rest])
        other = torch.arange(64, device=DEV) != 7
        assert torch.equal(o[0][:, below][..., other], out[0][:, below][..., other])
        x = o[0][:, below][..., 7]
        assert bool(x.isnan().all() if math.isnan(value) else (x == value).all())
    cache.value_pages[page, :, row] = clean_v
    cache.key_pages[page, :, row, 5] = math.nan
    o, l = run()
    assert torch.equal(o[0][:, rest], out[0][:, rest]) and torch.equal(l[0][:, rest], lse[0][:, rest])
    assert bool(o[0][:, below].isnan().all()) and torch.equal(o[1], out[1])
    cache.key_pages[page, :, row] = -math.inf * q[0, 0, 0].sign().unsqueeze(0)
    o, l = run()
    assert torch.equal(o[0][:, rest], out[0][:, rest])


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_scores_of_minus_infinity(dtype):
    """A row whose scores are all -inf is (0, -inf); keys of score -inf have no part."""
    cache = C.Cache([40], None, 3, 1, 64, 16, dtype, DEV, 5)
    q = randn(1, 2, 3, 64, dtype=dtype, seed=12).abs() + 0.1
    want = cp.cache_attention(q, cache.key_pages, cache.value_pages, cache.table, cache.lengths_t)
    page, row = cache.places(0, 0, 43)
    cache.key_pages[page, :, row] = -math.inf
    out, lse = cp.cache_attention(q, cache.key_pages, cache.value_pages, cache.table, cache.lengths_t)
    assert torch.all(out == 0) and torch.all(lse == -math.inf)
    cache.write(0, 0, cache.k[0], cache.v[0])
    cache.key_pages[page[:20], :, row[:20]] = -math.inf
    out, lse = cp.cache_attention(q, cache.key_pages, cache.value_pages, cache.table, cache.lengths_t)
    keep = [cache.k[0][:, 20:]], [cache.v[0][:, 20:]]
    ref = C.attend(q, *keep, [20], [3])
    check(out, ref[0])
    check(lse, ref[1])
    assert not torch.equal(out, want[0])


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("H", [2, 40])
def test_bad_pages(H, dtype):
    """Page numbers outside the pool: reported, their tokens read as zeros, other sequences unharmed."""
    S = 4
    cache = C.Cache([100, 100, 100], None, S, 1, 64, 16, dtype, DEV, 6)
    q = randn(3, H, S, 64, dtype=dtype, seed=13)
    good = cp.cache_attention(q, cache.key_pages, cache.value_pages, cache.table, cache.lengths_t)
    assert cp.last_device_status() == OK
    table = cache.table.clone()
    table[0, 2], table[1, 5] = cache.key_pages.shape[0], -5
    out, lse = cp.cache_attention(q, cache.key_pages, cache.value_pages, table, cache.lengths_t)
    assert cp.last_device_status() == BOUNDS and cp.last_device_status() == OK
    k, v = [x.clone() for x in cache.k], [x.clone() for x in cache.v]
    for b, i in ((0, 2), (1, 5)):
        k[b][:, 16 * i:16 * i + 16] = 0
        v[b][:, 16 * i:16 * i + 16] = 0
    want = C.attend(q, k, v, cache.lengths, cache.counts)
    check(out, want[0])
    check(lse, want[1])
    assert torch.equal(out[2], good[0][2])
    # cached tokens past the table
    short = cache.table[:, :6].contiguous()
    out, lse = cp.cache_attention(q, cache.key_pages, cache.value_pages, short, cache.lengths_t)
    assert cp.last_device_status() == BOUNDS
    # (lengths are brought into the table's 96 places, the drafts lie behind it)
    zeros = [torch.cat([x[:, :96], torch.zeros_like(x[:, :S])], 1) for x in cache.k], \
            [torch.cat([x[:, :96], torch.zeros_like(x[:, :S])], 1) for x in cache.v]
    want = C.attend(q, *zeros, [96] * 3, cache.counts)
    check(out, want[0])
    check(lse, want[1])


@pytest.mark.parametrize("page", [16, 32, 256])
@pytest.mark.parametrize("H,Hk,S,D", [(24, 24, 40, 64), (32, 16, 30, 128), (24, 24, 3, 64), (16, 16, 2, 128)])
def test_pieces_of_many_pages(H, Hk, S, D, page):
    """A block walks more pages than it holds numbers of; one of them, far from the piece's
    beginning, is not in the pool."""
    lengths = [2500, 1, 2047, 1300, 2300, 700, 1900, 2222]
    cache = C.Cache(lengths, None, S, Hk, D, page, BF, DEV, 21, "prhd")
    q = randn(len(lengths), H, S, D, dtype=BF, seed=22)
    out, lse = cp.cache_attention(q, cache.key_pages, cache.value_pages, cache.table, cache.lengths_t)
    assert cp.last_device_status() == OK
    want = C.attend(q, cache.k, cache.v, cache.lengths, cache.counts)
    check(out, want[0])
    check(lse, want[1])
    table = cache.table.clone()
    bad = ((0, 2100 // page), (4, 1200 // page))
    for b, i in bad:
        table[b, i] = cache.key_pages.shape[0] + b
    out, lse = cp.cache_attention(q, cache.key_pages, cache.value_pages, table, cache.lengths_t)
    assert cp.last_device_status() == BOUNDS and cp.last_device_status() == OK
    k, v = [x.clone() for x in cache.k], [x.clone() for x in cache.v]
    for b, i in bad:
        k[b][:, page * i:page * (i + 1)] = 0
        v[b][:, page * i:page * (i + 1)] = 0
    want = C.attend(q, k, v, cache.lengths, cache.counts)
    check(out, want[0])
    check(lse, want[1])


def test_counts_and_lengths_out_of_range():
    cache = C.Cache([20, 20], None, 4, 2, 64, 16, BF, DEV, 7)
    q = randn(2, 4, 4, 64, dtype=BF, seed=14)
    args = (q, cache.key_pages, cache.value_pages, cache.table)
    want = cp.cache_attention(*args, cache.lengths_t)
    got = cp.cache_attention(*args, cache.lengths_t, counts=torch.tensor([9, -1], dtype=torch.int32, device=DEV))
    assert torch.equal(got[0][0], want[0][0]) and torch.all(got[0][1] == 0) and torch.all(got[1][1] == -math.inf)
    low = cp.cache_attention(*args, torch.tensor([-9, 0], dtype=torch.int32, device=DEV))
    zero = cp.cache_attention(*args, torch.tensor([0, 0], dtype=torch.int32, device=DEV))
    assert torch.equal(low[0], zero[0]) and torch.equal(low[1], zero[1])


def test_parents_that_are_none():
    """A parent that is not before its draft is none."""
    cache = C.Cache([20], None, 6, 1, 64, 16, BF, DEV, 8)
    q = randn(1, 2, 6, 64, dtype=BF, seed=15)
    run = lambda par: cp.cache_attention(q, cache.key_pages, cache.value_pages, cache.table, cache.lengths_t,
                                         parents=torch.tensor([par], dtype=torch.int32, device=DEV))
    a, b = run([-1, 0, -1, 2, -1, 4]), run([0, 0, 2 ** 31 - 1, 2, 5, 4])
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    c = run([-2 ** 31, 0, -5, 2, -1, 4])
    assert torch.equal(a[0], c[0])


def test_shared_pages_and_table_views():
    """Two sequences with one prefix, a table that is a view of a wider one, and a broadcast row."""
    cache = C.Cache([64, 64], None, 1, 2, 64, 32, BF, DEV, 9)
    wide = torch.full((2, 9), -1, dtype=torch.int32, device=DEV)
    wide[:, :cache.table.shape[1]] = cache.table
    wide[1, :2] = wide[0, :2]
    view = wide[:, :3]
    q = randn(1, 4, 1, 64, dtype=BF, seed=16).expand(2, 4, 1, 64)
    out, lse = cp.cache_attention(q, cache.key_pages, cache.value_pages, view, cache.lengths_t)
    k = [cache.k[0], torch.cat([cache.k[0][:, :64], cache.k[1][:, 64:]], 1)]
    v = [cache.v[0], torch.cat([cache.v[0][:, :64], cache.v[1][:, 64:]], 1)]
    want = C.attend(q, k, v, cache.lengths, cache.counts)
    check(out, want[0])
    check(lse, want[1])
    one = cp.cache_attention(q, cache.key_pages, cache.value_pages, view[:1].expand(2, 3), cache.lengths_t[:1].expand(2))
    assert torch.equal(one[0][0], out[0]) and torch.equal(one[0][1], out[0])


def test_no_queries():
    cache = C.Cache([20], None, 1, 2, 64, 16, BF, DEV, 8)
    for shape in ((1, 0, 1, 64), (1, 2, 0, 64)):
        q = torch.empty(shape, dtype=BF, device=DEV)
        out, lse = cp.cache_attention(q, cache.key_pages, cache.value_pages, cache.table, cache.lengths_t)
        assert out.shape == shape and lse.shape == shape[:3]


@pytest.mark.parametrize("tree", [False, True])
@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_steps_of_a_transformer(dtype, tree):
    """Prompts, then single tokens or trees of drafts of which the longest path is kept:
    append and attend, step by step, equal to attention over the whole sequence."""
    B, H, Hk, D, page = 2, 4, 2, 64, 16
    prompts = [37, 12]
    pages = torch.zeros(24, Hk, page, D, dtype=dtype, device=DEV)
    key_pages, value_pages = pages, pages.clone()
    table = torch.randperm(24, generator=torch.Generator().manual_seed(0))[:24].view(2, 12).to(torch.int32).to(DEV)
    w = [1 + 0.2 * randn(D, dtype=dtype, seed=s) for s in (1, 2)]
    lengths = torch.zeros(B, dtype=torch.int32, device=DEV)
    ks, vs = [torch.zeros(Hk, 0, D, dtype=torch.float64, device=DEV) for _ in range(B)], \
             [torch.zeros(Hk, 0, D, dtype=torch.float64, device=DEV) for _ in range(B)]

    def step(S, counts, parents, seed):
        q, k, v = (randn(B, h, S, D, dtype=dtype, seed=seed + i, layout="bshd") for i, h in enumerate((H, Hk, Hk)))
        depth = torch.arange(S).expand(B, S) if parents is None else \
            torch.stack([C.ancestors(parents[b], S).sum(1) - 1 for b in range(B)])
        pos = (lengths[:, None] + depth.to(DEV)).float().unsqueeze(-1)
        ct = torch.tensor(counts, dtype=torch.int32, device=DEV)
        rq = cp.cache_append(k, v, key_pages, value_pages, table, lengths, positions=pos, axes_dims=(D,), q=q, counts=ct,
                             weight=w[0], q_weight=w[1], interleaved=False)
        pt = None if parents is None else parents.to(torch.int32).to(DEV)
        out, lse = cp.cache_attention(rq, key_pages, value_pages, table, lengths, parents=pt, counts=ct)
        rk = C.norm_rotary(k, w[0], pos, (D,), interleaved=False)[0].to(dtype)   # (as the pages hold them)
        kk = [torch.cat([ks[b], rk[b, :, :counts[b]].double()], 1) for b in range(B)]
        vv = [torch.cat([vs[b], v[b, :, :counts[b]].double()], 1) for b in range(B)]
        want = C.attend(rq, kk, vv, lengths.tolist(), counts, None if parents is None else parents.tolist())
        # a key's rounding may fall the other way: half a step more of each key
        slack = 2 * P.U[dtype] * D ** -0.5 * float(rq.double().norm(dim=-1).max() * max(x.norm(dim=-1).max() for x in kk))
        for got, (ref, tol) in zip((out, lse), want):
            big = max(float(x.abs().max()) for x in vv) if got.dim() == 4 else 1.0
            assert P.worst(got, ref, tol + slack * big) <= 1
        return kk, vv

    ks, vs = step(40, prompts, None, 100)
    lengths += torch.tensor(prompts, dtype=torch.int32, device=DEV)
    for i in range(4):
        if not tree:
            ks, vs = step(1, [1, 1], None, 200 + 10 * i)
            lengths += 1
            continue
        parents = C.tree(9, B, i, back=3)
        kk, vv = step(9, [9, 9], parents, 200 + 10 * i)
        for b in range(B):   # keep the first draft: the others' places are written again
            n = int(lengths[b]) + 1
            ks[b], vs[b] = kk[b][:, :n], vv[b][:, :n]
        lengths += 1
    assert cp.last_device_status() == OK
