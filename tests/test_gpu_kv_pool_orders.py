"""Pools in every order of pages, heads and slots hold and give the same."""
import itertools

import numpy as np
import pytest
import torch

import quantized_routed_expert_moe_gb300 as moe

pytestmark = pytest.mark.gpu

BF16, E4M3 = torch.bfloat16, torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def built():
    from quantized_routed_expert_moe_gb300 import build
    build.build()
    assert torch.cuda.is_available()


@pytest.mark.parametrize("dt", [BF16, E4M3])
@pytest.mark.parametrize("sizes", [(7, 3, 48), (1, 3, 128), (9, 1, 16), (1, 1, 128)])
@pytest.mark.parametrize("D", [64, 256])
def test_every_order(D, sizes, dt):
    pages, Hk, page = sizes
    n = min(pages * page, 130) - 3
    k, v = (torch.randn(n, Hk, D, generator=torch.Generator("cuda").manual_seed(i), device="cuda").to(BF16) for i in (1, 2))
    q = torch.randn(1, 4 * Hk, D, device="cuda").to(BF16)
    table = torch.randperm(pages, generator=torch.Generator().manual_seed(3))[:-(-n // page)].to(torch.int32)[None].cuda()
    pos = torch.arange(n, dtype=torch.int32, device="cuda")
    lens = torch.full((1,), n, dtype=torch.int32, device="cuda")
    scale = None if dt is BF16 else np.full(Hk, 0.01, np.float32)
    first = None
    for order in itertools.permutations(range(3)):
        back = [order.index(i) for i in range(3)]
        pools = [torch.zeros([sizes[i] for i in order] + [D], device="cuda", dtype=BF16).to(dt).permute(*back, 3)
                 for _ in range(2)]
        assert pools[0].shape == (pages, Hk, page, D)
        out, lse = torch.empty_like(q), torch.empty(1, 4 * Hk, device="cuda")
        with moe.KVCache(*pools, n_heads=4 * Hk, k_scale=scale, v_scale=scale,
                         inv_freq=np.array([10000.0 ** (-i / 16) for i in range(16)])) as kv:
            kv.append(None, k, v, pos, table, seq=torch.zeros_like(pos))
            kv.attend(q, table, lens, out, lse=lse)
            assert kv.health() == (0, 0)
        got = [p.float() for p in pools] + [out, lse]
        first = first or got
        assert all(torch.equal(a, b) for a, b in zip(got, first)), order
    assert torch.isfinite(first[2].float()).all() and first[2].any()
