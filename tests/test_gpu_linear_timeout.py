"""A bounded wait of moe_linear that runs out: the copies of one tile are never started
(MOE_LINEAR_OPT_TEST_STALL), so that no fault is needed for it. Its outputs are NaN, as are those of
the tiles that its CTA takes after it; all others are right, and so is the next call."""
import time

import pytest
import torch

import quantized_routed_expert_moe_gb300 as moe

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def built():
    from quantized_routed_expert_moe_gb300 import build
    build.build()
    assert torch.cuda.is_available()


@pytest.mark.parametrize("out", [BF16, F32])
@pytest.mark.parametrize("T,K,N,tile", [
    (1, 6144, 512, 2),        # cut along K over a cluster
    (100, 4096, 1032, 8),     # the same, and the last tile has 8 channels
    (300, 192, 264, 1),       # few products: the copies are done before the first wait
    (1, 72, 128, 0),
    (4000, 256, 2048, 3),     # more tiles than SMs: the CTA's later tiles
    (4000, 256, 2048, 200),
])
@pytest.mark.parametrize("bias", [False, True])
def test_a_wait_that_runs_out_leaves_nan(T, K, N, tile, out, bias):
    g = torch.Generator("cuda").manual_seed(T + tile)
    x = torch.randn(T, K, generator=g, device="cuda").bfloat16()
    w = torch.randn(N, K, generator=g, device="cuda").bfloat16()
    lin = moe.Linear(w, bias=torch.randn(N, generator=g, device="cuda") if bias else None, activation="silu" if bias else "none")
    clean, y, again = (torch.full((T, N), 7.0, dtype=out, device="cuda") for _ in range(3))
    lin.run(x, clean)
    torch.cuda.synchronize()
    moe.moe_linear_set_option(moe.MOE_LINEAR_OPT_TEST_STALL, tile)
    try:
        t = time.perf_counter()
        lin.run(x, y)
        torch.cuda.synchronize()
        assert time.perf_counter() - t < 10
    finally:
        moe.moe_linear_set_option(moe.MOE_LINEAR_OPT_TEST_STALL, -1)
    nan, right = torch.isnan(y), y == clean
    assert (nan ^ right).all()
    # the tile's own outputs, and whole tiles
    rows = -(-N // 128)
    cols = next(b for b in ((16, 32, 64, 128) if out is F32 else (16, 32, 64, 128, 256)) if b >= T or b == (128 if out is F32 else 256))
    lost = 0
    for i in range(rows * -(-T // cols)):
        part = nan[i // rows * cols:(i // rows + 1) * cols, i % rows * 128:(i % rows + 1) * 128]
        assert part.all() or not part.any()
        lost += bool(part.any())
        if i == tile:
            assert part.all()
    assert lost >= 1 and (lost == 1 or rows * -(-T // cols) > torch.cuda.get_device_properties(0).multi_processor_count)
    lin.run(x, again)
    torch.cuda.synchronize()
    assert torch.equal(again, clean)
