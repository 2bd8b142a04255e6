"""Infinite values of drafts that a row sees reach its result, whether or not several blocks
share the sequence: an attention's parts may have maxima far apart, or no weight at all."""
import math

import pytest
import torch

import context_attention_partial_gb300 as cp
import plain_cache as C

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32
D, N = 64, 4096
# (query heads, tokens, dtype): 16 rows or fewer, one query tile, two, fp32 of 16 and of 64 rows
FORMS = [(2, 5, BF), (4, 30, BF), (4, 60, BF), (2, 5, F32), (4, 30, F32)]


def one_sequence(H, S, dtype):
    """A query's score is 256 with the first key and 0 with all others, so only the first value has weight."""
    cache = C.Cache([N], None, S, 1, D, 16, dtype, DEV, 1)
    page, row = cache.places(0, 0, N + S)
    cache.key_pages[page, :, row] = 0
    cache.key_pages[page[0], :, row[0], 3] = 16
    q = torch.zeros(1, H, S, D, dtype=dtype, device=DEV)
    q[..., 3] = 16
    return cache, q, page, row


def attend(cache, q, batch, parents=None):
    """The sequence `batch` times over: few of them are split over blocks, many are not."""
    S = q.shape[2]
    many = [t.expand(batch, *t.shape[1:]).contiguous() for t in (q, cache.table, cache.lengths_t)]
    pt = None if parents is None else torch.tensor([parents] * batch, dtype=torch.int32, device=DEV)
    out, lse = cp.cache_attention(many[0], cache.key_pages, cache.value_pages, many[1], many[2], parents=pt, scale=1.0)
    assert cp.last_device_status() == 0
    assert (cp.cache_attention_workspace_bytes(many[0], cache.key_pages, many[1]) > 0) == (batch == 1)
    assert out.shape[2] == S
    return out, lse


def expected(cache, q, draft, features, parents):
    """The first value (its weight is 1, the others' are below 2^-368), and what the draft's
    values that are not finite make of their features in the rows that see it."""
    S = q.shape[2]
    seen = C.ancestors(list(range(-1, S - 1)) if parents is None else parents, S)[:, draft].to(DEV)
    want = cache.v[0][0, 0].expand(1, q.shape[1], S, D).clone()
    for f, value in features.items():
        want[:, :, seen, f] = value
    return want


def same(got, want, tree=False):
    """Equal, but that in a chain's rows from token 16 on an infinity may be NaN:
    a row tile of fp32 has 64 rows, 16 tokens of 4 heads, so all rows of a later one see the draft, and its values
    are multiplied as a cached token's are: by a weight of 2^-369 or less, which is 0 in fp32, and 0 times an
    infinity is NaN."""
    nan = got.isnan()
    if not tree:
        nan[:, :, 16:] &= ~want[:, :, 16:].isinf()
        got = torch.where(got.isnan() & ~nan, want, got)
    return torch.equal(nan, want.isnan()) and torch.equal(got.nan_to_num(nan=0.0), want.nan_to_num(nan=0.0))


@pytest.mark.parametrize("batch", [1, 4000], ids=["split", "whole"])
@pytest.mark.parametrize("tree", [False, True], ids=["chain", "tree"])
@pytest.mark.parametrize("H,S,dtype", FORMS, ids=lambda x: str(x).split(".")[-1])
def test_a_seen_draft_of_a_small_weight(H, S, dtype, tree, batch):
    cache, q, page, row = one_sequence(H, S, dtype)
    parents = [-1, 0, 0] + [1 + i % 2 for i in range(S - 3)] if tree else None
    features = {5: math.inf, 17: -math.inf, 40: math.nan}
    for f, value in features.items():
        cache.value_pages[page[N + 1], :, row[N + 1], f] = value
    out, lse = attend(cache, q, batch, parents)
    want = expected(cache, q, 1, features, parents)
    for b in {0, batch // 2, batch - 1}:
        assert same(out[b:b + 1], want, tree)
    # 256, its product with log2 e and back: four roundings of fp32
    assert float((lse - 256).abs().max()) <= 256 * 4 * 2.0 ** -24


@pytest.mark.parametrize("batch", [1, 4000], ids=["split", "whole"])
@pytest.mark.parametrize("H,S,dtype", FORMS, ids=lambda x: str(x).split(".")[-1])
def test_a_seen_draft_among_scores_of_minus_infinity(H, S, dtype, batch):
    """The second half of the keys, drafts included, has scores of -inf: blocks that read
    nothing else have no weight at all, and the draft's infinities are theirs."""
    cache, q, page, row = one_sequence(H, S, dtype)
    cache.key_pages[page[N // 2:], :, row[N // 2:], 3] = -math.inf
    features = {5: math.inf, 17: -math.inf}
    for f, value in features.items():
        cache.value_pages[page[N + 1], :, row[N + 1], f] = value
    out, lse = attend(cache, q, batch)
    want = expected(cache, q, 1, features, None)
    for b in {0, batch // 2, batch - 1}:
        assert same(out[b:b + 1], want)
    # all scores -inf: nothing has weight, and nothing reaches the result
    cache.key_pages[page, :, row, 3] = -math.inf
    out, lse = attend(cache, q, batch)
    assert torch.all(out == 0) and torch.all(lse == -math.inf)
