"""GPU tests of the block plan and the release against the oracle's pool: whole numbers, so equal."""

import numpy as np
import pytest
import torch

import bitwise_invariant_gated_amd as gdn
from gpu_util import note
from oracle import attention as ref

pytestmark = pytest.mark.gpu

DEV = "cuda"


def i32(x):
    return torch.tensor(list(x), dtype=torch.int32, device=DEV)


def check_pool(pool, want):
    assert pool.block_table.cpu().numpy().tolist() == want.table.tolist()
    assert pool.blocks_held.tolist() == want.held
    assert pool.seq_len.tolist() == want.len
    n = int(pool.free_count)
    assert pool.free_blocks[:n].tolist() == want.free


def step(pool, want, rows, news, advance=True):
    cu = i32(np.concatenate([[0], np.cumsum(news)]))
    plan = gdn.alloc_attn_plan(pool, len(rows), sum(news), i32(rows))
    gdn.gdn_attn_plan(pool, cu, plan, advance=advance)
    ctx, pos, place, refused = want.plan(rows, news, advance)
    assert plan.ctx_len.tolist() == ctx
    assert plan.positions.tolist() == pos
    assert plan.slot_map.tolist() == [int(x) for x in place]
    assert int(plan.status) == refused
    check_pool(pool, want)


@pytest.mark.parametrize("seed,n,most", [(1, 1, 1), (2, 5, 300), (3, 64, 200), (4, 300, 40), (5, 1500, 9), (6, 3, 9000)])
def test_steps_and_releases(seed, n, most):
    note(f"plan seed={seed} n={n} most={most}")
    rng = np.random.default_rng(seed)
    slots, width = n + 4, most * 4 // 64 + 3
    blocks = int(n * most * 1.2 / 64) + n
    pool, want = gdn.alloc_attn_pool(slots, width, blocks, DEV), ref.Pool(slots, width, blocks)
    for _ in range(5):
        m = int(rng.integers(1, n + 1))
        rows = rng.permutation(slots)[:m]
        rows = np.where(rng.random(m) < 0.1, -1, rows).tolist()
        news = rng.integers(0, most + 1, m).tolist()
        step(pool, want, rows, news, advance=bool(rng.random() < 0.8))
        gone = [r for r in rng.permutation(slots)[: m // 2].tolist()]
        if gone:
            gdn.gdn_attn_release(pool, i32(gone))
            want.release(gone)
            check_pool(pool, want)


def test_refusal_leaves_the_row_and_later_small_needs_go_on():
    note("plan refusal")
    pool, want = gdn.alloc_attn_pool(4, 8, 5, DEV), ref.Pool(4, 8, 5)
    step(pool, want, [0, 1], [100, 60])
    # row 2 wants more than is free; row 0 fits in the block that it holds; row 1 needs one more
    step(pool, want, [2, 0, 1], [300, 20, 30])
    step(pool, want, [1, 0], [30, 1])
    step(pool, want, [3], [8 * 64 + 1])  # wider than the table


def test_the_same_lengths_again_take_nothing():
    note("plan again")
    pool, want = gdn.alloc_attn_pool(3, 8, 20, DEV), ref.Pool(3, 8, 20)
    for _ in range(3):
        step(pool, want, [2, 0], [130, 64], advance=False)


def test_no_requests():
    note("plan empty")
    pool = gdn.alloc_attn_pool(3, 8, 20, DEV)
    plan = gdn.alloc_attn_plan(pool, 0, 0)
    gdn.gdn_attn_plan(pool, i32([0]), plan)
    assert int(plan.status) == 0 and int(pool.free_count) == 20
    gdn.gdn_attn_release(pool, i32([]))


def test_graph_replay_advances():
    note("plan graph")
    pool, want = gdn.alloc_attn_pool(3, 8, 20, DEV), ref.Pool(3, 8, 20)
    step(pool, want, [0, 1, 2], [60, 1, 127])
    plan = gdn.alloc_attn_plan(pool, 3, 3, i32([0, 1, 2]))
    cu = i32([0, 1, 2, 3])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gdn.gdn_attn_plan(pool, cu, plan)
    for _ in range(6):
        graph.replay()
        ctx, pos, place, _ = want.plan([0, 1, 2], [1, 1, 1])
        torch.cuda.synchronize()
        assert plan.ctx_len.tolist() == ctx and plan.slot_map.tolist() == [int(x) for x in place]
        check_pool(pool, want)
