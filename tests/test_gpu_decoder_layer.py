"""The example layer (norms, cache append, paged attention, routed experts) step by
step: every stage against its 64-bit form on the inputs that the GPU gave it."""
import importlib.util
import os

import numpy as np
import pytest
import torch

import oracle
import seeded_inputs as si
from _decoder_ref import assert_close, attend, block_norm, f64, rotate, rounded
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


@pytest.mark.parametrize("cache", [BF16, torch.float8_e4m3fn])
def test_decoder_layer_step_by_step(example, cache):
    spec = si.LayerSpec(hidden=512, inter=256, n_experts=32, top_k=8)
    lay = si.gen_layer(3, 0, spec)
    tokens, d = 19, 64
    L = example.DecoderLayer(lay, 8, 2, d, tokens, cache=cache, seed=4)
    inv = np.array([10000.0 ** (-2.0 * i / d) for i in range(d // 2)])
    scale = None if cache is BF16 else np.full(2, 8 / 448, np.float32)
    x = torch.randn(1, 512, device="cuda", generator=torch.Generator("cuda").manual_seed(5))
    side = torch.cuda.Stream()
    for t in range(tokens):
        x0 = x.clone()
        if t % 2:
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(side):
                L.step(x)
            torch.cuda.current_stream().wait_stream(side)
        else:
            L.step(x)
        torch.cuda.synchronize()
        if t not in (0, 1, 15, 16, 18):
            continue
        _, _, h, eh = block_norm(x0, None, None, None, L.first.w_pre, 1e-6, 1.0, 0.0)
        assert_close(L.h, h, rounded(h, eh, BF16), "h")
        q, eq = rotate(L.q, [t], inv, False)
        assert_close(L.q_rot, q, rounded(q, eq, BF16), "q")
        k, ek = rotate(L.k, [t], inv, False)
        if scale is not None:
            k, ek = k / float(scale[0]), ek / float(scale[0]) + 2.0 ** -23 * (k / float(scale[0])).abs()
        table = L.table.cpu()
        got = L.kv.k_pages[int(table[0, t // 16]), :, t % 16]
        assert_close(got, k[0], rounded(k, ek, cache)[0], "cached k")
        o, eo, _, _ = attend(L.q_rot, L.kv.k_pages, L.kv.v_pages, table, [t + 1], d ** -0.5, 0.0, 0, scale, scale)
        assert_close(L.o, o, rounded(o, eo, BF16), "attention")
        r1, e1, hm, em = block_norm(x0, L.attn, None, L.after_attention.w_post, L.after_attention.w_pre, 1e-6, 1.0, 0.0)
        assert_close(L.h_mid, hm, rounded(hm, em, BF16), "h_mid")
        y, _ = oracle.moe_token(lay, L.h_mid[0].cpu().view(torch.int16).numpy().view(np.uint16))
        assert float((f64(L.y) - torch.from_numpy(y)).abs().max() / np.abs(y).max()) <= REL_TOL + 2.0 ** -8
        r2, e2, hn, en = block_norm(r1, L.y[None], None, L.after_experts.w_post, L.after_experts.w_pre, 1e-6, 1.0, 0.0)
        # the residual stream between the two norms is itself off by e1, which the second norm passes on
        assert_close(x, r2, rounded(r2, e2 + e1 + 2.0 ** -24 * r1.abs(), torch.float32), "x")
        w = f64(L.after_experts.w_pre).abs() / torch.sqrt((r2 * r2).mean(1, keepdim=True))
        assert_close(L.h_next, hn, rounded(hn, en + 2 * w * (e1 + 2.0 ** -24 * r1.abs()), BF16), "h_next")
    assert L.kv.health() == (0, 0)
    L.close()


def test_the_step_in_a_graph(example):
    """One step captured once and replayed: positions and lengths are read on the device."""
    spec = si.LayerSpec(hidden=512, inter=256, n_experts=32, top_k=8)
    lay = si.gen_layer(3, 0, spec)
    x0 = torch.randn(1, 512, device="cuda", generator=torch.Generator("cuda").manual_seed(6))
    a = example.DecoderLayer(lay, 8, 2, 64, 24, seed=7)
    xa, plain = x0.clone(), []
    for _ in range(20):
        plain.append(a.step(xa).clone())
    torch.cuda.synchronize()
    b = example.DecoderLayer(lay, 8, 2, 64, 24, seed=7)
    xb = x0.clone()
    got = [b.step(xb).clone() for _ in range(2)]   # first uses outside the capture
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        b.step(xb)
    for _ in range(18):
        g.replay()
        got.append(b.h_next.clone())
    torch.cuda.synchronize()
    for t, (p, q) in enumerate(zip(plain, got)):
        assert torch.equal(p, q), t
    assert torch.equal(xa, xb) and b.kv.health() == (0, 0)
    a.close()
    b.close()
