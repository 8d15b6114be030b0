"""moe_kv_attend on the GPU within the bounds that its arithmetic gives, where
those of test_gpu_kv_attend.py are wider."""
import pytest
import torch

import _decoder_ref
from _decoder_ref import assert_close, attend, rounded
from test_gpu_kv_attend import BF16, Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from quantized_routed_expert_moe_gb300 import build
    build.build()
    assert torch.cuda.is_available()


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("G", [1, 6, 16])
def test_bf16_weights_are_not_cut_to_bf16(G, D, monkeypatch):
    """A weight enters the product with values as two bf16 numbers, its own rounding (2^-8)
    and what that left, rounded once more: 2^-16 relative."""
    monkeypatch.setattr(_decoder_ref, "UP", 2.0 ** -16)
    Case([1, 16, 77, 300, 1025], 2 * G, 2, D, 32, seed=G).check()
    Case([20000], G, 1, D, 64, seed=G).check()
