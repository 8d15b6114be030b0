"""moe_linear where a CTA takes tile after tile, its accumulators in turn (more tiles than SMs), and the
errors of whole outputs."""
import pytest
import torch

import quantized_routed_expert_moe_gb300 as moe
from _chunk_ref import linear
from test_gpu_linear import BF16, F32, run_case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from quantized_routed_expert_moe_gb300 import build
    build.build()
    assert torch.cuda.is_available()


@pytest.mark.parametrize("out", [BF16, F32])
@pytest.mark.parametrize("T,K,N,act,bias,residual,room", [
    (8191, 136, 1032, "gelu_tanh", True, False, 0),     # 9 x 32 tiles of 256 tokens, the last of 8 channels
    (4097, 64, 2560, "none", False, True, 0),           # one stage to a tile; the last tile of one token
    (5000, 1544, 1288, "silu", True, True, 24),
    (2049, 2816, 4104, "sigmoid", False, False, 8),
])
def test_more_tiles_than_sms(T, K, N, act, bias, residual, room, out):
    y = run_case(T, K, N, out, act, bias, residual, room=room, seed=T)
    assert torch.isfinite(y).all()


def test_more_tiles_than_sms_in_place_and_on_another_stream():
    run_case(5000, 264, 1288, BF16, "none", True, True, inplace=True, seed=3)
    run_case(5000, 264, 1288, F32, "silu", False, True, inplace=True, seed=4, stream=torch.cuda.Stream())


def test_more_tiles_than_sms_same_bits():
    g = torch.Generator("cuda").manual_seed(1)
    x, w = (torch.randn(n, 512, generator=g, device="cuda").bfloat16() for n in (8000, 2048))
    first, again = torch.empty(8000, 2048, dtype=BF16, device="cuda"), torch.empty(8000, 2048, dtype=BF16, device="cuda")
    lin = moe.Linear(w, activation="silu")
    lin.run(x, first)
    for _ in range(5):
        again.zero_()
        lin.run(x, again)
        torch.cuda.synchronize()
        assert torch.equal(first, again)


def outputs(T, K, N, out):
    g = torch.Generator("cuda").manual_seed(K + T)
    x = torch.randn(T, K, generator=g, device="cuda").bfloat16()
    w = (torch.randn(N, K, generator=g, device="cuda") * K ** -0.5).bfloat16()
    y = torch.empty(T, N, dtype=out, device="cuda")
    moe.Linear(w).run(x, y)
    return y.double().cpu(), linear(x, w, None, "none", None)[0]


@pytest.mark.parametrize("T", [1, 64, 128, 600])
@pytest.mark.parametrize("K,N", [(6144, 1032), (2816, 6144)])
def test_fp32_sums(T, K, N):
    """Every step of 16 products in the tensor cores cuts off 1.8e-8 of what the sum then is, always
    towards zero. Over 512 products, 32 steps, of a sum that grows as a root: 32 * 2/3 * 1.8e-8 = 3.8e-7
    of it at most, and of the whole, as such sums add up in squares; what adds them outside rounds, 2^-25
    of the whole a time. Without the sums outside it is 1.5e-6 over 6144 products."""
    y, v = outputs(T, K, N, F32)
    assert float((y - v).norm() / v.norm()) <= 5e-7


@pytest.mark.parametrize("T", [1, 128, 600])
def test_bf16_outputs_are_the_rounded_sums(T):
    """A sum that is off by 1.5e-6 of the norm lies on the other side of a border between two bf16
    numbers, 2^-8 to 2^-7 of them apart, once in 2000 times where it is at least half the norm."""
    y, v = outputs(T, 6144, 1032, BF16)
    large = v.abs() >= 0.5 * v.square().mean().sqrt()
    assert float((y != v.bfloat16().double())[large].double().mean()) <= 2e-3
