"""Refusals and copies of the attention layer's binding that need no GPU."""

import copy
import os
import pickle

import pytest
import torch

import bitwise_invariant_gated_amd as gdn
from bitwise_invariant_gated_amd import _lib


@pytest.fixture
def lib():
    if not os.path.exists(_lib.LIB_PATH):
        pytest.skip("library not built")
    return _lib.load()


def test_plan_refuses_a_step_of_another_pool(lib):
    """The step's table is what attention reads: one that is not the pool's would go unplanned."""
    import ctypes

    fake = 0x10000  # never dereferenced: validation fails first
    pool = _lib.AttnPoolC(fake, fake, fake, fake, fake, 4, 8, 16)
    for table, width, slots, name in ((2 * fake, 8, 4, "block_table"), (None, 8, 4, "block_table"), (fake, 9, 4, "max_blocks"),
                                      (fake, 8, 5, "num_slots")):
        step = _lib.AttnStepC(fake, fake, fake, fake, table, None, width, slots)
        got = lib.gdn_attn_plan(ctypes.byref(pool), 2, 10, fake, 1, ctypes.byref(step), None)
        assert got == _lib.GDN_ERR_INVALID_ARG and name in lib.gdn_cpr_last_error().decode(), name


def equal(a, b):
    return a is None and b is None or torch.equal(a, b) and a.data_ptr() != b.data_ptr()


@pytest.mark.parametrize("how", [copy.deepcopy, lambda x: pickle.loads(pickle.dumps(x))])
def test_caches_pools_and_plans_can_be_copied(how):
    """A request's state is snapshot and kept: the copy holds arrays of its own, and its
    handle is of those."""
    shape = gdn.AttnShape(4, 2, 64)
    pool = gdn.alloc_attn_pool(3, 4, 8, "cpu")
    cache = gdn.alloc_attn_cache(shape, 8, 3, "cpu")
    cache.tail_k.normal_()
    plan = gdn.alloc_attn_plan(pool, 2, 5, torch.tensor([2, 0], dtype=torch.int32))
    bare = gdn.alloc_attn_plan(pool, 2, 5)
    for x in (pool, cache, plan, bare):
        y = how(x)
        for f in x.__dataclass_fields__:
            assert equal(getattr(x, f), getattr(y, f)), f
        first = next(iter(x.__dataclass_fields__))
        assert getattr(y._ref._obj, first) == getattr(y, first).data_ptr()
        assert {n: getattr(x._ref._obj, n) for n, _ in x._ref._obj._fields_ if n.startswith(("num", "max"))} == \
               {n: getattr(y._ref._obj, n) for n, _ in y._ref._obj._fields_ if n.startswith(("num", "max"))}
    pool2, plan2 = how((pool, plan))
    assert plan2.block_table is pool2.block_table  # what they share stays shared
    assert copy.copy(cache).k8 is cache.k8
