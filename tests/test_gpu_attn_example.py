"""examples/hybrid_decode.py: the attention layer's operators and a Gated
DeltaNet decode step together, as one CUDA graph, against plain attention."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_hybrid_decode_example():
    from gated_deltanet_linear_04_gb300.build import build_library
    build_library()
    spec = importlib.util.spec_from_file_location("hybrid_decode", os.path.join(ROOT, "examples", "hybrid_decode.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    # one bf16 rounding of the result (2^-8), and of the weights before the product with V
    assert m.main(rows=5, prompt=150, steps=6) <= 2.0 ** -7
