"""Check of the built library that needs no GPU: which kernels there are for rows of one part (up to 2,048
columns), which one launch answers.  The entropy's sum is to be formed only where the entropy is asked for, as
in longer rows, so each of them comes in two forms, and the divergence's in the one without."""

import os
import re

import pytest

from bitwise_invariant_gated_amd import _lib


def test_forms_without_the_entropys_sum():
    if not os.path.exists(_lib.LIB_PATH):
        pytest.skip("library not built")
    with open(_lib.LIB_PATH, "rb") as f:
        names = f.read()
    join, make, entropy = b"0", b"1", b"2"
    for e in (b"3B16", b"3F32"):
        rows = set(re.findall(rb"k_stack_logprobsINS_" + e + rb"ELi(\d)ELNS_7RowFormE(\d)EE", names))
        # no alternatives, among the columns themselves, through groups of 8 (also where rows are longer), of 128
        want = {*((m, f) for m in (b"0", b"1", b"2") for f in (make, entropy)), *((m, join) for m in (b"0", b"2", b"3"))}
        assert rows == want
        assert set(re.findall(rb"k_stack_distillINS_" + e + rb"ELNS_7RowFormE(\d)EE", names)) == {join, make}
