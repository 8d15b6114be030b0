"""The example layer on a stream that is not torch's current one: positions, lengths and starts are
written there too, and nothing of a chunk comes from the host."""
import importlib.util
import os

import pytest
import torch

import seeded_inputs as si
from conftest import ROOT

pytestmark = pytest.mark.gpu

SPEC = si.LayerSpec(hidden=512, inter=256, n_experts=32, top_k=8)
CHUNKS = (19, 1, 33)


@pytest.fixture(scope="module")
def example():
    from quantized_routed_expert_moe_gb300 import build
    build.build()
    spec = importlib.util.spec_from_file_location("decoder_layer", os.path.join(ROOT, "examples", "decoder_layer.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def layer(example):
    return example.DecoderLayer(si.gen_layer(3, 0, SPEC), 8, 2, 64, sum(CHUNKS) + 4, seed=4, head_norm=True, max_chunk=40)


def inputs():
    g = torch.Generator("cuda").manual_seed(5)
    return torch.randn(sum(CHUNKS), 512, device="cuda", generator=g), torch.randn(4, 512, device="cuda", generator=g)


def walk(example, busy=None, stream=None):
    """A prompt in chunks and four steps: what they return, and the residual stream."""
    L = layer(example)
    x, steps = inputs()
    torch.cuda.synchronize()
    got = []
    with torch.cuda.stream(busy):   # (None: as it is)
        for part in x.split(CHUNKS):
            if busy is not None:
                torch.cuda._sleep(20_000_000)   # about 10 ms: what the current stream gets now comes too late
            got.append(L.prefill(part, stream=stream))
        for t in range(len(steps)):
            if busy is not None:
                torch.cuda._sleep(20_000_000)
            got.append(L.step(steps[t:t + 1], stream=stream))
            with torch.cuda.stream(stream):
                got[-1] = got[-1].clone()   # (the steps return one buffer)
    torch.cuda.synchronize()
    assert L.kv.health() == (0, 0)
    assert int(L.position) == int(L.length) == sum(CHUNKS) + len(steps)
    L.close()
    return torch.cat(got), x, steps


def test_a_stream_of_its_own_beside_a_busy_one(example):
    plain = walk(example)
    other = walk(example, busy=torch.cuda.Stream(), stream=torch.cuda.Stream())
    for a, b in zip(plain, other):
        assert torch.equal(a, b)


def test_a_chunk_reads_nothing_from_the_host(example):
    """A blocking copy is an error while a graph is captured: a chunk can be captured, and replayed."""
    L, M = layer(example), layer(example)
    x, _ = inputs()
    y = x.clone()
    want = [L.prefill(p).clone() for p in (x[:19], x[19:38])]
    M.prefill(y[:19])
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = M.prefill(y[19:38])
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(got, want[1]) and torch.equal(x, y)
    assert M.kv.health() == (0, 0)
    L.close()
    M.close()
