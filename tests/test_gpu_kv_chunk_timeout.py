"""A bounded wait of moe_kv_attend_chunk that runs out: the copies of one sequence are never
started (MOE_KV_OPT_TEST_STALL), so that no fault is needed for it."""
import time

import pytest
import torch

import quantized_routed_expert_moe_gb300 as moe
from test_gpu_kv_attend_chunk import BF16, E4M3, Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from quantized_routed_expert_moe_gb300 import build
    build.build()
    assert torch.cuda.is_available()


@pytest.mark.parametrize("chunks,stalled", [([(9, 300), (40, 700)], 1), ([(300, 5000), (3, 9)], 0), ([(1, 200)] * 30, 17)])
@pytest.mark.parametrize("D,dt", [(64, BF16), (128, BF16), (128, E4M3), (256, BF16), (256, E4M3)])
def test_a_wait_that_runs_out_is_told(chunks, stalled, D, dt):
    c = Case(chunks, 8, 2, D, 32, dt, seed=31)
    with c.handle() as kv:
        clean, clean_lse = c.run(kv)
        assert kv.health() == (0, 0)
        kv.set_option(moe.MOE_KV_OPT_TEST_STALL, stalled)
        t = time.perf_counter()
        c.run(kv)
        assert time.perf_counter() - t < 10
        assert kv.health() == (5, moe.MOE_KV_TIMEOUT)
        # nothing of it is left for the next call
        kv.set_option(moe.MOE_KV_OPT_TEST_STALL, -1)
        out, lse = c.run(kv)
        assert kv.health() == (0, 0)
    assert torch.equal(out, clean) and torch.equal(lse, clean_lse)
