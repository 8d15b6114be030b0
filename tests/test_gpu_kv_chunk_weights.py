"""How far the softmax weights of moe_kv_attend_chunk are rounded: to fp16 over an 8-bit cache (2^-11),
to bf16 over a bf16 one (2^-8). Seen from the outputs' side of the borders between two bf16 numbers."""
import pytest
import torch

from test_gpu_kv_attend_chunk import BF16, E4M3, Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from quantized_routed_expert_moe_gb300 import build
    build.build()
    assert torch.cuda.is_available()


# Outputs that are at least half as large as their row's norm says lie 2^-8 to 2^-7 of themselves from the
# next bf16 number. Weights that are off by 2^-11 each (0.29 of that on average, signs mixed) move them by
# 1.9e-4 of the norm and 2.6% of them over a border; by 2^-8, 1.5e-3 and 23%. (400 positions in 64 bits,
# weights rounded alone.) The limits are between: what falls back to bf16 passes the second only.
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("dt,limit", [(E4M3, 0.08), (BF16, 0.32)])
def test_rounding_of_the_weights(dt, limit, D):
    c = Case([(200, 600), (3, 9000), (40, 400)], 8, 2, D, 64, dt, seed=D, sharp=0.5)
    with c.handle() as kv:
        out, _ = c.run(kv)
        assert kv.health() == (0, 0)
    v = c.want()[0]
    large = v.abs() >= 0.5 * v.square().mean(-1, keepdim=True).sqrt()
    other = out.cpu() != v.bfloat16()
    for rows in (slice(0, 200), slice(200, 203), slice(203, 243)):
        assert float(other[rows][large[rows]].double().mean()) <= limit
