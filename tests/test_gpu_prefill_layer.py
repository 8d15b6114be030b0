"""A prompt in chunks through the whole example layer (norm, projection, head norms and
rotation in the append, chunk attention, projection, norms, routed experts), stage by stage
against the 64-bit forms, then decode steps that continue it."""
import importlib.util
import os

import numpy as np
import pytest
import torch

import oracle
import seeded_inputs as si
from _chunk_ref import attend_chunk, head_norm, linear, rotate64
from _decoder_ref import assert_close, block_norm, f64, rounded
from _parity import REL_TOL
from conftest import ROOT

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


@pytest.fixture(scope="module")
def example():
    from quantized_routed_expert_moe_gb300 import build
    build.build()
    spec = importlib.util.spec_from_file_location("decoder_layer", os.path.join(ROOT, "examples", "decoder_layer.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


SPEC = si.LayerSpec(hidden=512, inter=256, n_experts=32, top_k=8)


@pytest.mark.parametrize("cache", [BF16, torch.float8_e4m3fn])
@pytest.mark.parametrize("norms", [False, True])
def test_chunks_stage_by_stage(example, cache, norms):
    lay = si.gen_layer(3, 0, SPEC)
    d, chunks = 64, (19, 1, 33, 16)
    L = example.DecoderLayer(lay, 8, 2, d, sum(chunks) + 3, cache=cache, seed=4, head_norm=norms, max_chunk=40)
    inv = np.array([10000.0 ** (-2.0 * i / d) for i in range(d // 2)])
    scale = None if cache is BF16 else np.full(2, 8 / 448, np.float32)
    x = torch.randn(sum(chunks), 512, device="cuda", generator=torch.Generator("cuda").manual_seed(5))
    done = 0
    for n in chunks:
        part = x[done:done + n]
        x0 = part.clone()
        h_next = L.prefill(part)
        torch.cuda.synchronize()
        c = L.chunk
        _, _, h, eh = block_norm(x0, None, None, None, L.first.w_pre, 1e-6, 1.0, 0.0)
        assert_close(c["h"], h, rounded(h, eh, BF16), "h")
        got = torch.cat([c[k].reshape(n, -1) for k in "qkv"], 1)
        v, e = linear(c["h"], L.w_qkv, None, "none", None)
        assert_close(got, v, rounded(v, e, BF16), "qkv")
        pos = np.arange(done, done + n)
        q, rel = head_norm(c["q"], L.q_norm, 1e-6, 0.0)
        turned = rotate64(q, pos, inv, False)
        # the norm's error and the rotation's (2^-20), of a pair's both channels
        bound = (2 * rel + 2.0 ** -20) * (q.abs() + q.abs().roll(d // 2, -1) + turned.abs())
        assert_close(c["q_rot"], turned, rounded(turned, bound, BF16), "q")
        done += n
        table = L.table.cpu()
        vo, eo, _, _ = attend_chunk(c["q_rot"], L.kv.k_pages, L.kv.v_pages, table, [0, n], [done], d ** -0.5, 0.0, 0, scale, scale)
        assert_close(c["o"], vo, rounded(vo, eo, BF16), "attention")
        v, e = linear(c["o"].view(n, -1), L.w_o, None, "none", None)
        assert_close(c["attn"], v, rounded(v, e, BF16), "output projection")
        r1, e1, hm, em = block_norm(x0, c["attn"], None, L.after_attention.w_post, L.after_attention.w_pre, 1e-6, 1.0, 0.0)
        assert_close(c["h_mid"], hm, rounded(hm, em, BF16), "h_mid")
        for t in {0, n - 1}:
            y, _ = oracle.moe_token(lay, c["h_mid"][t].cpu().view(torch.int16).numpy().view(np.uint16))
            assert float((f64(c["y"][t]) - torch.from_numpy(y)).abs().max() / np.abs(y).max()) <= REL_TOL + 2.0 ** -8
        r2, e2, _, _ = block_norm(r1, c["y"], None, L.after_experts.w_post, L.after_experts.w_pre, 1e-6, 1.0, 0.0)
        assert_close(part, r2, rounded(r2, e2 + e1 + 2.0 ** -24 * r1.abs(), torch.float32), "x")
        assert h_next.shape == (n, 512) and torch.isfinite(h_next.float()).all()
    # the steps that follow see the prompt: the cache holds what a chunk of one token would read
    for _ in range(3):
        step = torch.randn(1, 512, device="cuda")
        L.step(step)
        done += 1
        torch.cuda.synchronize()
        vo, eo, _, _ = attend_chunk(L.q_rot, L.kv.k_pages, L.kv.v_pages, table, [0, 1], [done], d ** -0.5, 0.0, 0, scale, scale)
        assert_close(L.o, vo, rounded(vo, eo, BF16), "step")
    assert L.kv.health() == (0, 0)
    L.close()


def test_chunks_of_any_size_agree(example):
    """The same prompt as one chunk and as several: the cache and the outputs agree to their types'
    rounding, carried through the layer."""
    lay = si.gen_layer(3, 0, SPEC)
    x0 = torch.randn(40, 512, device="cuda", generator=torch.Generator("cuda").manual_seed(6))
    outs = []
    for sizes in ((40,), (1, 17, 22), (8,) * 5):
        L = example.DecoderLayer(lay, 8, 2, 64, 40, seed=7, head_norm=True, max_chunk=40)
        x = x0.clone()
        outs.append((torch.cat([L.prefill(p).float() for p in x.split(sizes)]), x))
        torch.cuda.synchronize()
        assert L.kv.health() == (0, 0)
        L.close()
    for h, x in outs[1:]:
        assert float((h - outs[0][0]).abs().max()) <= 2.0 ** -4 * float(outs[0][0].abs().max())
        assert float((x - outs[0][1]).abs().max()) <= 2.0 ** -4 * float(outs[0][1].abs().max())
