"""moe_kv_health: what one call reports is not taken from the next."""
import pytest
import torch

import quantized_routed_expert_moe_gb300 as moe

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from quantized_routed_expert_moe_gb300 import build
    build.build()
    assert torch.cuda.is_available()


def test_a_bit_set_right_after_a_report_is_kept():
    """The report clears the bits on the legacy stream, and torch's streams do not wait for that one."""
    kp, vp = (torch.zeros(3, 2, 16, 64, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    k = torch.randn(1, 2, 64, device="cuda").bfloat16()
    table = torch.tensor([[7]], dtype=torch.int32, device="cuda")
    pos = torch.zeros(1, dtype=torch.int32, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with moe.KVCache(kp, vp, n_heads=2) as kv:
        for _ in range(300):
            kv.append(None, k, k, pos, table, stream=s)
            assert kv.health() == (6, moe.MOE_KV_BAD_PAGE)
        assert kv.health() == (0, 0)
    assert not kp.any() and not vp.any()
