"""The example of the expert block: its outputs against fp32 products on the
same 4-bit weights. Each compared output is one bf16 rounding (2^-9 relative at
most, h another in front of it) away, so a relative error of 2^-7 in the norm
holds with room; the 4-bit projection starts from the same quantized input."""

import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


def test_moe_block():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "moe_block.py")
    spec = importlib.util.spec_from_file_location("moe_block", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    assert all(e < 2.0 ** -7 for e in m.main(tokens=70, steps=2, D=256, F=96, E=8, k=2))
