"""A decoder layer of the library's operators together: chunks of prompts and
single tokens over one paged cache, eager and captured."""
import os
import sys

import pytest
import torch

from gpu_util import DEV, say

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ex():
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    import decoder_layer
    return decoder_layer


@pytest.mark.parametrize("window,sinks", [(0, 0), (40, 3)])
@pytest.mark.parametrize("heads,kv,dim", [(8, 2, 128), (6, 3, 64)])
def test_layer_against_fp32(ex, window, sinks, heads, kv, dim):
    """Codes of an activation are off by a uniform half step of amax / 127, with amax about
    4 sigma for normal values: 0.9% of the row's norm, and of a weight row's likewise.  Six
    such errors a way through the layer (two products, each of activation and weight, after
    two more behind the softmax) stay below 5%."""
    say("layer", window, sinks, heads, kv, dim)
    layer = ex.Layer(512, heads, kv, dim, 1408, window, sinks)
    x, y = ex.run(layer, [150, 7, 83], chunk=64, single=5)
    for a, b in zip(x, y):
        ref = layer.plain(a)
        assert float((b - ref).norm() / (ref - a).norm()) < 0.05


def test_chunks_do_not_matter(ex):
    """The same tokens in other chunks: weights are rounded in other tiles (half a bf16 step
    of attention's output each way) and may move codes by one: under 2% of the change."""
    layer = ex.Layer(512, 8, 2, 64, 1408)
    x, a = ex.run(layer, [140, 33], chunk=140, single=0)
    _, b = ex.run(layer, [140, 33], chunk=31, single=20)
    for t, p, q in zip(x, a, b):
        assert float((p - q).norm() / (p - t).norm()) < 0.02


def test_a_captured_step_replays(ex):
    """Append, attention and products of a step in one graph: every replay, with eager work
    between, is the eager step on the same inputs bit for bit."""
    layer = ex.Layer(512, 8, 2, 64, 1408)
    cache = ex.Cache(64, 16, 3, 2, 64, 200)
    g = torch.Generator(device=DEV).manual_seed(3)
    first = torch.randn(150 + 40 + 9, 512, generator=g, device=DEV)
    layer.forward(cache, ex.Batch(cache, [150, 40, 9]), first)
    b = ex.Batch(cache, [1, 1, 1])
    x = torch.zeros(3, 512, device=DEV)
    h, n = 8 * 64, 2 * 64

    def step():
        qkv = layer.product("qkv", x)
        return layer.product("o", layer.attention(cache, b, qkv))

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for i in range(4):
        say("layer replay", i)
        x.copy_(torch.randn(3, 512, generator=g, device=DEV))
        graph.replay()
        got = out.clone()
        want = step()
        torch.cuda.synchronize()
        assert torch.equal(got, want) and got.abs().max() > 0
    assert h + 2 * n == layer.w["qkv"].N
