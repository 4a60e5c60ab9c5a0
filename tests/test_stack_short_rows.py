"""Check of the built library that needs no GPU: which kernels there are for rows of one part (up to 2,048
columns), which one launch answers.  The entropy's sum is to be formed only where the entropy is asked for, as
in longer rows, so each of them comes in two forms, and the divergence's in the one without."""

import os
import re
import subprocess

import pytest

from bitwise_invariant_gated_amd import _lib


def test_forms_without_the_entropys_sum():
    if not os.path.exists(_lib.LIB_PATH):
        pytest.skip("library not built")
    names = subprocess.run(["nm", "-C", _lib.LIB_PATH], capture_output=True, text=True, check=True).stdout
    join, make, entropy = "(stack::RowForm)0", "(stack::RowForm)1", "(stack::RowForm)2"
    for e in ("B16", "F32"):
        rows = set(re.findall(rf"__device_stub__k_stack_logprobs<stack::{e}, (\d), ([^>]*)>", names))
        # no alternatives, among the columns themselves, through groups of 8 (also where rows are longer), of 128
        assert rows == {*((m, f) for m in "012" for f in (make, entropy)), *((m, join) for m in "023")}
        assert set(re.findall(rf"__device_stub__k_stack_distill<stack::{e}, ([^>]*)>", names)) == {join, make}
