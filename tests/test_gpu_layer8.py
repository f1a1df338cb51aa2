"""The 8-bit cache's operators and the verification of drafts as they are used together: a
decoder layer over the cache, eager and captured, and decoding with drafts."""
import os
import sys

import numpy as np
import pytest
import torch

from cache8_ref import verify
from gpu_util import DEV, say
from layer_ref import f64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ex():
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    import decoder_layer
    return decoder_layer


@pytest.mark.parametrize("window,sinks", [(0, 0), (40, 3)])
@pytest.mark.parametrize("heads,kv,dim", [(8, 2, 128), (6, 3, 64), (4, 1, 80)])
def test_layer_against_fp32(ex, window, sinks, heads, kv, dim):
    """Codes of a row are off by a uniform half step of amax / 127, with amax about 4 sigma for
    normal values: 0.9% of the row's norm, for keys and values as for the products' activations and
    weights.  Eight such errors a way through the layer stay below 5%."""
    say("layer8", window, sinks, heads, kv, dim)
    layer = ex.Layer(512, heads, kv, dim, 1408, window, sinks)
    x, y = ex.run(layer, [150, 7, 83], chunk=64, single=5, bits=8)
    for a, b in zip(x, y):
        ref = layer.plain(a)
        assert float((b - ref).norm() / (ref - a).norm()) < 0.05


def drafts_of(plain, wrong):
    """Four drafts that are right but for every `wrong`-th token."""
    return lambda s, t: [(v + 1) % 500 if wrong and i % wrong == wrong - 1 else v for i, v in enumerate(plain[s])][len(t):len(t) + 4]


@pytest.mark.parametrize("bits", [8, 16])
@pytest.mark.parametrize("wrong", [0, 2, 5])
def test_decoding_with_drafts_is_decoding(ex, bits, wrong):
    """At temperature 0 the tokens are those of single steps, in fewer steps; refused tokens' places are written again."""
    say("drafts", bits, wrong)
    layer = ex.Layer(256, 4, 2, 64, 512)
    prompts = [[1, 2, 3], [40, 50, 60, 70, 80], [7, 8]]
    plain, steps = ex.generate(ex.Model(layer, 500, 3, 120, bits=bits), prompts, 40, lambda s, t: [])
    assert steps == 40
    model = ex.Model(layer, 500, 3, 120, bits=bits)
    text, fewer = ex.generate(model, prompts, 30, drafts_of(plain, wrong))
    assert fewer < 30 and (wrong or fewer <= 7)
    for a, b, p in zip(text, plain, prompts):
        assert a[:len(p) + 30] == b[:len(p) + 30]
    assert sum(-(-n // 16) for n in model.cache.lengths) + len(model.cache.free) == model.cache.table.numel()


def test_a_captured_step_with_drafts_replays(ex):
    """Append, attention, products and verification of a step in one graph: every replay, with eager
    work between, is the eager step on the same inputs, and the definition's tokens for its logits."""
    layer = ex.Layer(256, 4, 2, 64, 512)
    model = ex.Model(layer, 700, 3, 120)
    g = torch.Generator(device=DEV).manual_seed(5)
    model.step([list(range(50)), list(range(20)), [9]])
    b = ex.Batch(model.cache, [4, 1, 3])
    x, ids = torch.zeros(8, 256, device=DEV), torch.zeros(8, dtype=torch.int32, device=DEV)
    u, warm = torch.zeros(8, device=DEV), torch.full((3,), 0.8, device=DEV)
    out = torch.zeros(2, 3, dtype=torch.int32, device=DEV)

    def step():
        logits = layer.forward(model.cache, b, x) @ model.head.t()
        ex.qg.qgemv_verify_draft(logits, 0, 8, 700, 700, b.start, 3, 4, ids, None, 0, u, warm, out[0], out[1], layer.ws, ex.qg.QGEMV_WS_BYTES)
        return logits

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        logits = step()
    for i in range(4):
        say("layer8 replay", i)
        x.copy_(torch.randn(8, 256, generator=g, device=DEV))
        ids.copy_(torch.randint(700, (8,), generator=g, device=DEV))
        u.copy_(torch.rand(8, generator=g, device=DEV) * 0.01)
        graph.replay()
        got, tokens = logits.clone(), out.cpu().numpy().copy()
        want = step()
        torch.cuda.synchronize()
        assert torch.equal(got, want) and np.array_equal(tokens, out.cpu().numpy())
        assert np.array_equal(tokens, verify(f64(got), f64(b.start).astype(int), 4, f64(ids).astype(int), None, f64(u).astype(np.float32), f64(warm)))


def test_two_streams_at_once(ex):
    """Two steps over caches and workspaces of their own on two streams: the bits of each alone."""
    def work(model):
        return model.step([list(range(60)), [5] * 7])[0]

    alone, streams, got = [], [torch.cuda.Stream() for _ in range(2)], []
    layers = [ex.Layer(256, 4, 2, 64, 512, seed=s) for s in range(2)]
    for layer in layers:
        alone.append(work(ex.Model(layer, 300, 2, 80)))
    models = [ex.Model(layer, 300, 2, 80) for layer in layers]
    torch.cuda.synchronize()
    say("layer8 two streams")
    for stream, model in zip(streams, models):
        with torch.cuda.stream(stream):
            got.append(work(model))
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(alone, got))
