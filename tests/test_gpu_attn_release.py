"""GPU test of a release that names rows more than once."""

import pytest
import torch

import bitwise_invariant_gated_amd as gdn
from gpu_util import note

pytestmark = pytest.mark.gpu

I32 = dict(dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("rows", [[2, 2], [0, 2, 1, 2, -1, 0], list(range(40)) * 30])  # the last over two rounds of 1,024
def test_a_row_named_twice_gives_its_blocks_back_once(rows):
    note(f"release twice {rows[:6]} {len(rows)}")
    slots, width, blocks = 40, 9, 400
    pool = gdn.alloc_attn_pool(slots, width, blocks)
    lens = [64 * (1 + i % 8) - 3 for i in range(slots)]
    cu = torch.tensor([0] + lens, device="cuda").cumsum(0).to(torch.int32)
    gdn.gdn_attn_plan(pool, cu, gdn.alloc_attn_plan(pool, slots, sum(lens)))
    held, table, before = pool.blocks_held.tolist(), pool.block_table.tolist(), int(pool.free_count)
    assert before == blocks - sum(held)
    gdn.gdn_attn_release(pool, torch.tensor(rows, **I32))
    gone = {r for r in rows if r >= 0}
    count = int(pool.free_count)
    assert count == before + sum(held[r] for r in gone)
    free = pool.free_blocks[:count].tolist()
    back = [x for r in gone for x in table[r] if x >= 0]
    assert len(set(free)) == count and sorted(free[before:]) == sorted(back)
    assert pool.blocks_held.tolist() == [0 if r in gone else held[r] for r in range(slots)]
    assert pool.seq_len.tolist() == [0 if r in gone else lens[r] for r in range(slots)]
    assert pool.block_table.tolist() == [[-1] * width if r in gone else table[r] for r in range(slots)]
