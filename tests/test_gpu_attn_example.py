"""GPU test of the hybrid stack in examples/: all operators together, through the
public entry points; decode and prefill agree in every bit."""

import importlib.util
import os

import pytest

from gpu_util import note

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "hybrid_generate.py")


@pytest.mark.parametrize("kw", [dict(layers=4), dict(layers=4, attn_heads=8, kv_heads=1, attn_d=64),
                                dict(layers=4, attn_heads=2, kv_heads=2, attn_d=256)])
def test_generation_equals_prefill(kw):
    note(f"hybrid example {kw}")
    spec = importlib.util.spec_from_file_location("hybrid_generate", PATH)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    tokens = example.main(lens=(3, 64, 130), steps=66, **kw)
    assert tokens.shape == (67, 3)
