"""Arguments that do not fit their C types are refused: as ValueError by the classes, or (a
float past fp32's range is an infinity to the call) as MoEError by the library."""
import pytest
import torch

import quantized_routed_expert_moe_gb300 as moe

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def built():
    from quantized_routed_expert_moe_gb300 import build
    build.build()
    assert torch.cuda.is_available()


@pytest.mark.parametrize("kw", [dict(window=2 ** 31), dict(window=1.5), dict(scale=1e39), dict(softcap=-1e39),
                                dict(scale="1")])
def test_attend(kw):
    kp, vp = (torch.zeros(2, 2, 16, 64, device="cuda", dtype=BF16) for _ in range(2))
    q = torch.zeros(1, 4, 64, device="cuda", dtype=BF16)
    table, lens = torch.zeros(1, 1, dtype=torch.int32, device="cuda"), torch.ones(1, dtype=torch.int32, device="cuda")
    with moe.KVCache(kp, vp, n_heads=4) as kv:
        with pytest.raises((ValueError, moe.MoEError)):
            kv.attend(q, table, lens, torch.empty_like(q), **kw)


@pytest.mark.parametrize("kw", [dict(eps=1e39), dict(scale=-1e39), dict(weight_offset="1")])
def test_norm_numbers(kw):
    x, h = torch.zeros(2, 256, device="cuda"), torch.empty(2, 256, device="cuda", dtype=BF16)
    with pytest.raises((ValueError, moe.MoEError)):
        moe.BlockNorm(256, None, torch.ones(256, device="cuda"), **kw).run(x, h=h)


def test_norm_gate_of_other_ranks():
    x, o = torch.zeros(2, 256, device="cuda"), torch.zeros(2, 256, device="cuda", dtype=BF16)
    n = moe.BlockNorm(256)
    for gate in (torch.ones((), device="cuda", dtype=BF16), torch.ones(1, 1, 256, device="cuda", dtype=BF16),
                 torch.ones(2, 1, 256, device="cuda", dtype=BF16)):
        with pytest.raises(ValueError):
            n.run(x, o, r=torch.empty_like(x), gate=gate)
