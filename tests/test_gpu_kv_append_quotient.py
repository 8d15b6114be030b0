"""moe_kv_append into an 8-bit cache divides by the scale: quotients that lie half way between
two e4m3 values, where a product with the rounded reciprocal takes the wrong one."""
import numpy as np
import pytest
import torch

import quantized_routed_expert_moe_gb300 as moe

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from quantized_routed_expert_moe_gb300 import build
    build.build()
    assert torch.cuda.is_available()


def test_ties_go_as_the_quotient_does():
    heads, d = 256, 64
    ties = np.array([17, 19, 23, 34, 250, 1.0625, 2.75, 100], np.float32)
    x = (torch.arange(heads).float() * 0.37 + 0.011).to(torch.bfloat16)
    # each head has a value whose quotient is one of the ties, as nearly as fp32 has it
    scale = (x.float().numpy() / ties[np.arange(heads) % len(ties)]).astype(np.float32)
    k = torch.randn(3, heads, d, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16)
    k[:, :, 0], k[:, :, 9], k[:, :, 40] = x, -x, 2 * x
    k[1, :, 20:25] = torch.tensor([torch.inf, -torch.inf, torch.nan, 3e38, -3e38])
    want = (k.float() / torch.from_numpy(scale)[None, :, None]).clamp(-448, 448).to(torch.float8_e4m3fn)
    product = (k.float() * (1 / torch.from_numpy(scale))[None, :, None]).clamp(-448, 448).to(torch.float8_e4m3fn)
    assert (want.float() != product.float())[~torch.isnan(want.float())].sum() > 30   # the values tell the two apart
    kp, vp = (torch.zeros(1, heads, 16, d, device="cuda", dtype=torch.bfloat16).to(torch.float8_e4m3fn) for _ in range(2))
    pos = torch.tensor([0, 5, 15], dtype=torch.int32, device="cuda")
    with moe.KVCache(kp, vp, n_heads=heads, k_scale=scale, v_scale=scale) as kv:
        kv.append(None, k.cuda(), k.cuda(), pos, torch.zeros(1, 1, dtype=torch.int32, device="cuda"),
                  seq=torch.zeros_like(pos))
        assert kv.health() == (0, 0)
    for pool in (kp, vp):
        got = pool[0, :, [0, 5, 15]].transpose(0, 1).cpu()
        nan = torch.isnan(want.float())
        assert torch.equal(torch.isnan(got.float()), nan) and int(nan.sum()) == heads
        assert torch.equal(got.view(torch.uint8)[~nan], want.view(torch.uint8)[~nan])
