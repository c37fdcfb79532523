"""The 8-bit example runs the projection, the scored routing and the 8-bit experts together."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T", [1, 7, 200])
def test_fp8_layer_example(T):
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "fp8_layer.py")
    spec = importlib.util.spec_from_file_location("fp8_layer_example", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    err, bits = m.main(T)
    # e4m3 rounding of x, y and h: 2^-4 / sqrt(3) of a value's spacing at most, about 3 percent each
    assert 0 < err < 0.08 and bits == 0
