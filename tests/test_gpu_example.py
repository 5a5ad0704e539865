"""The served attention layer of examples/cached_layer.py runs, and its outputs are as near
to the unquantised fp64 layer as the steps' roundings allow: an int8 code is off by at most
half of 1/127 of its block's largest value, about 1/60 of a normal value's size for blocks of
a few thousand values (maximum about 3.7 sizes: 3.7 / 254, uniform error: / sqrt(3) = 0.0084
of a value), for keys and for values; the bf16 projections add about 0.004 each."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():   # pragma: no cover - CPU machine
    pytest.skip("needs a GPU", allow_module_level=True)


def test_cached_layer_example():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "cached_layer.py")
    spec = importlib.util.spec_from_file_location("cached_layer", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    assert m.main() < 0.03
