"""CPU checks of the build's spill check for the attention kernels: those that do not
spill must not begin to, those that do may not spill more."""

import pytest

from bitwise_invariant_gated_amd.build import MAY_SPILL, check_spills


def meta(name, spills):
    return f"""    .name:           _ZN4attn{name}EEvNS_8RowsArgsE
    .vgpr_count:     256
    .vgpr_spill_count: {spills}
    .wavefront_size: 64
"""


@pytest.mark.parametrize("name", ["11k_attn_rowsILi64ELi1ELb0ELb1", "11k_attn_rowsILi128ELi1ELb0ELb1",
                                  "11k_attn_rowsILi256ELi1ELb0ELb0", "11k_attn_rowsILi256ELi1ELb1ELb1",
                                  "11k_attn_rowsILi64ELi2ELb1ELb0", "11k_attn_rowsILi128ELi1ELb1ELb1", "14k_attn_prefillILi64",
                                  "17k_attn_cache_readILi128"])
def test_attention_kernels_that_do_not_spill(name):
    assert check_spills(meta(name, 0)) == []
    assert [k for _, k in check_spills(meta(name, 1))] == [1]


@pytest.mark.parametrize("name", ["11k_attn_rowsILi128ELi2ELb1ELb1", "11k_attn_rowsILi128ELi2ELb1ELb0", "14k_attn_prefillILi128",
                                  "14k_attn_prefillILi256"])
def test_attention_kernels_that_spill_have_a_ceiling(name):
    most = [n for frag, n in MAY_SPILL.items() if frag in meta(name, 0)]
    assert len(most) == 1 and 0 < most[0] < 100
    assert check_spills(meta(name, most[0])) == []
    assert [k for _, k in check_spills(meta(name, most[0] + 1))] == [most[0] + 1]
