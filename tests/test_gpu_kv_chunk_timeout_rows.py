"""The rows of a moe_kv_attend_chunk call in which a bounded wait ran out: each is right or NaN as a
whole, and those of the sequence whose copies were never started (MOE_KV_OPT_TEST_STALL) are NaN."""
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


@pytest.mark.parametrize("D,dt", [(64, BF16), (64, E4M3), (128, BF16), (128, E4M3), (256, BF16), (256, E4M3)])
@pytest.mark.parametrize("chunks,stalled,alone", [
    ([(1, 200)] * 30, 17, True),                     # whole tiles, one to a CTA
    ([(9, 300), (40, 700)], 1, False),               # cut tiles
    ([(300, 5000), (3, 9)], 0, False),
    ([(3, 9), (1, 20000), (700, 700)], 1, False),    # one tile over many CTAs
    ([(20, 100), (6, 2), (30, 400), (5, 0)], 2, False),   # rows that see nothing
])
def test_rows_are_right_or_nan(chunks, stalled, alone, D, dt):
    c = Case(chunks, 8, 2, D, 32, dt, seed=31, before=2, after=3)
    mine = torch.zeros(c.q.shape[0], dtype=torch.bool, device="cuda")
    mine[c.starts[stalled]:c.starts[stalled + 1]] = True
    for with_lse in (True, False) if alone else (True,):
        with c.handle() as kv:
            clean, clean_lse = c.run(kv, with_lse=with_lse)
            assert kv.health() == (0, 0)
            kv.set_option(moe.MOE_KV_OPT_TEST_STALL, stalled)
            # what the last call left in the workspace is none of this one's
            kv._workspace.fill_(0x40)
            out, lse = c.run(kv, with_lse=with_lse)
            assert kv.health() == (5, moe.MOE_KV_TIMEOUT)
            kv.set_option(moe.MOE_KV_OPT_TEST_STALL, -1)
            again, again_lse = c.run(kv, with_lse=with_lse)
            assert kv.health() == (0, 0)
        assert torch.equal(again, clean)
        nan = torch.isnan(out).all(2)
        right = (out == clean).all(2)
        assert (nan ^ right).all()
        assert nan[mine].all()
        if alone:
            assert not nan[~mine].any()
        assert right[:2].all() and right[-3:].all()   # rows of no sequence
        if with_lse:
            assert torch.equal(again_lse, clean_lse)
            assert torch.equal(torch.isnan(lse), nan) and (lse[right] == clean_lse[right]).all()
