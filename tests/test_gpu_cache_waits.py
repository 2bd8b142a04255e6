"""A limit for waits that is far below the time of a piece of work: roles of the tensor-core
kernel that have nothing to do in some pieces run ahead of the others, and then wait for whole
pieces, which is no fault."""
import pytest
import torch

import context_attention_partial_gb300 as cp

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF = torch.bfloat16
OK = 0
PAGE, PAGES, D = 64, 1024, 128
LIMIT_NS = 100_000      # a piece of 65536 keys takes two to three times that


@pytest.fixture(scope="module")
def pools():
    g = torch.Generator(DEV).manual_seed(1)
    return [torch.randn(PAGES + 8, 8, PAGE, D, generator=g, dtype=BF, device=DEV) for _ in range(2)]


def run(pools, H, kv_heads, S, lengths, counts):
    """Sequences of the same pages, as many as leave each unit whole; with the default limit and a short one."""
    B = len(lengths)
    q = torch.randn(B, H, S, D, generator=torch.Generator(DEV).manual_seed(2), dtype=BF, device=DEV)
    table = torch.arange(PAGES + 8, dtype=torch.int32, device=DEV).expand(B, PAGES + 8)
    ints = [torch.tensor(x, dtype=torch.int32, device=DEV) for x in (lengths, counts)]
    pages = [p[:, :kv_heads] for p in pools]
    assert cp.cache_attention_workspace_bytes(q, pages[0], table) == 0

    def call():
        out, lse = cp.cache_attention(q, *pages, table, ints[0], counts=ints[1])
        return out, lse, cp.last_device_status()

    *want, status = call()
    assert status == OK
    try:
        cp.set_wait_timeout_ns(LIMIT_NS)
        *got, status = call()
    finally:
        cp.set_wait_timeout_ns(2_000_000_000)
    assert status == OK
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def blocks():
    return torch.cuda.get_device_properties(0).multi_processor_count


def test_a_group_without_rows_runs_ahead(pools):
    """Two query tiles a unit, of which the second has no tokens anywhere."""
    B = blocks()
    run(pools, 32, 8, 40, [PAGES * PAGE] * B, [20] * B)


def test_a_group_whose_rows_come_after_pieces_without(pools):
    """Every fourth piece of a block has rows in its second query tile."""
    n = blocks()
    B = 8 * n
    run(pools, 4, 1, 40, [PAGES * PAGE] * B, [40 if b // n % 4 == 3 else 20 for b in range(B)])


def test_values_without_drafts_keep_the_cleaner_waiting(pools):
    """Single tokens whose keys end with a key tile: no tile of values is cleaned."""
    B = 8 * blocks()
    run(pools, 32, 1, 1, [PAGES * PAGE - 1] * B, [1] * B)


def test_a_short_piece_behind_long_ones(pools):
    """Every fourth piece of a block is a few keys with drafts among them, which the cleaner waits for
    while the three long ones before it run."""
    n = blocks()
    B = 8 * n
    run(pools, 32, 1, 1, [5 if b // n % 4 == 3 else PAGES * PAGE - 1 for b in range(B)], [1] * B)
