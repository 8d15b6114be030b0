"""Options and calls of moe_linear that are refused before anything reaches a device."""
import pytest

import quantized_routed_expert_moe_gb300 as moe


@pytest.fixture(scope="module", autouse=True)
def built():
    from quantized_routed_expert_moe_gb300 import build
    build.build()


def test_options_are_looked_at():
    for option, value in ((2, 0), (0, 0), (moe.MOE_LINEAR_OPT_TEST_STALL, -2), (moe.MOE_LINEAR_OPT_TEST_STALL, 2 ** 31)):
        with pytest.raises(moe.MoEError):
            moe.moe_linear_set_option(option, value)
