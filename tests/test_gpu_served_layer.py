"""The served attention layer of examples/cached_layer.py over the 4-bit cache: projections, norms
and rotation, append, attention and output projection together, prompts and then single tokens.

A code is off by at most half a step, evenly; the step is a seventh of the largest of 16 values, 1.77
of a normal value's size on average, and its e4m3 rounding moves it by 2% on average: 0.26 / sqrt(12)
= 0.075 of a value.  That reaches the output once through the values and once, where scores
have about a normal value's size, through the weights: 0.106 together.  The worst of 36 sequences'
steps, some of them of a handful of tokens, is allowed half as much again."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():   # pragma: no cover - CPU machine
    pytest.skip("needs a GPU", allow_module_level=True)


def test_cached_layer_in_4_bits():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "cached_layer.py")
    spec = importlib.util.spec_from_file_location("cached_layer", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    assert m.main(bits=4) < 0.16


@pytest.mark.parametrize("bits", [8, 4])
def test_a_decode_step_in_a_graph(bits):
    """One captured step, replayed for token after token with the lengths counted up between, against
    the same steps one by one."""
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "cached_layer.py")
    spec = importlib.util.spec_from_file_location("cached_layer", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    layers = [m.Layer(bits=bits) for _ in range(2)]
    i32 = dict(dtype=torch.int32, device="cuda")
    gen = torch.Generator(device="cuda")
    gen.manual_seed(3)
    prompt = torch.randn((90, 1024), device="cuda", generator=gen).bfloat16()
    adapters = torch.tensor([0] * 60 + [2] * 30, **i32)
    for layer in layers:
        layer.step(prompt, adapters, torch.tensor([60, 30], **i32), offsets=torch.tensor([0, 60, 90], **i32), max_new=60)
    X, lengths, ids = torch.zeros((2, 1024), dtype=torch.bfloat16, device="cuda"), torch.tensor([60, 30], **i32), torch.tensor([0, 2], **i32)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):       # (torch's buffers: one step ahead of the capture, over the last token)
        layers[1].step(X, ids, lengths)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = layers[1].step(X, ids, lengths)
    layers[1].step(prompt, adapters, torch.tensor([60, 30], **i32), offsets=torch.tensor([0, 60, 90], **i32), max_new=60)
    for k in range(1, 6):
        x = torch.randn((2, 1024), device="cuda", generator=gen).bfloat16()
        now = torch.tensor([60 + k, 30 + k], **i32)
        want = layers[0].step(x, ids, now)
        X.copy_(x)
        lengths.copy_(now)
        graph.replay()
        assert torch.equal(out, want)
    for layer in layers:
        assert layer.cache.status() == layer.rotary.status() == 0
