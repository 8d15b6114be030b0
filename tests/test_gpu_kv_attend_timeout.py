"""A bounded wait of moe_kv_attend that runs out: the copies of one sequence are never
started (MOE_KV_OPT_TEST_STALL), so that no fault is needed for it."""
import time

import pytest
import torch

import quantized_routed_expert_moe_gb300 as moe
from test_gpu_kv_attend import BF16, E4M3, Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from quantized_routed_expert_moe_gb300 import build
    build.build()
    assert torch.cuda.is_available()


# a segment within a warp; cut between warps; between two CTAs; between many
@pytest.mark.parametrize("lens,stalled", [([700, 33, 40, 3000], 1), ([700, 900, 40, 3000], 1), ([9, 5000], 1),
                                          ([40000], 0), ([0, 800] * 40, 41)])
@pytest.mark.parametrize("G,D,dt", [(4, 64, BF16), (12, 128, E4M3), (16, 256, BF16)])
def test_rows_without_their_cache_are_nan(lens, stalled, G, D, dt):
    c = Case(lens, 2 * G, 2, D, 32, dt, seed=31)
    with c.handle() as kv:
        clean, clean_lse = c.run(kv)
        assert kv.health() == (0, 0)
        kv.set_option(moe.MOE_KV_OPT_TEST_STALL, stalled)
        t = time.perf_counter()
        out, lse = c.run(kv)
        assert time.perf_counter() - t < 3
        assert kv.health() == (5, moe.MOE_KV_TIMEOUT)
        assert torch.isnan(out[stalled]).all() and torch.isnan(lse[stalled]).all()
        # the others are right, or shared a CTA with the stalled one and are NaN
        lost = torch.isnan(lse)
        assert torch.equal(torch.isnan(out), lost[..., None].expand_as(out))
        assert torch.equal(out[~lost], clean[~lost]) and torch.equal(lse[~lost], clean_lse[~lost])
        # nothing of it is left for the next call
        kv.set_option(moe.MOE_KV_OPT_TEST_STALL, -1)
        out, lse = c.run(kv)
        assert kv.health() == (0, 0)
    assert torch.equal(out, clean) and torch.equal(lse, clean_lse)


def test_option_refusals():
    c = Case([5, 6], 4, 2, 64, 16)
    with c.handle() as kv:
        for option, value in ((0, 0), (2, 0), (moe.MOE_KV_OPT_TEST_STALL, 2), (moe.MOE_KV_OPT_TEST_STALL, -2)):
            with pytest.raises(moe.MoEError) as ei:
                kv.set_option(option, value)
            assert ei.value.status == 1
