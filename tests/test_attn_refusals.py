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
