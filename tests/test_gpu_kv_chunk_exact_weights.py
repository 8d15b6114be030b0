"""moe_kv_attend_chunk with weights as two bf16 numbers (MOE_KV_OPT_CHUNK_WEIGHTS)."""
import pytest
import torch

import _chunk_ref
import quantized_routed_expert_moe_gb300 as moe
from test_gpu_kv_attend_chunk import BF16, E4M3, FEW, Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from quantized_routed_expert_moe_gb300 import build
    build.build()
    assert torch.cuda.is_available()


@pytest.fixture(autouse=True)
def bound(monkeypatch):
    """The first number is a weight's upper 16 bits; the second what those leave, 2^-7 of the weight at
    most, rounded (2^-8 of it), and 2^-20 of the weight more than it."""
    monkeypatch.setattr(_chunk_ref, "UP", 2.0 ** -15 + 2.0 ** -20)


def check(c, softcap=0.0):
    with c.handle() as kv:
        kv.set_option(moe.MOE_KV_OPT_CHUNK_WEIGHTS, 2)
        out, lse = c.run(kv, softcap)
        again, _ = c.run(kv, softcap)
        assert kv.health() == (0, 0)
        kv.set_option(moe.MOE_KV_OPT_CHUNK_WEIGHTS, 1)
        _, plain = c.run(kv, softcap)
    c.compare(out, lse, softcap)
    assert torch.equal(out.view(torch.int16), again.view(torch.int16))
    assert torch.equal(lse, plain)   # the sums are those of the weights before any rounding
    return out


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("layout", ["hnd", "nhd"])
def test_few_tokens(D, layout):
    check(Case(FEW, 4, 2, D, 16, BF16, layout, seed=D))


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("G,window,cap", [(1, 0, 0.0), (6, 100, 0.0), (17, 0, 30.0), (40, 33, 0.5)])
def test_groups_windows_caps(D, G, window, cap):
    check(Case([(33, 77), (0, 5), (300, 1300), (1, 1), (130, 131)], 2 * G, 2, D, 48, window=window, seed=G), cap)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_long_context_is_split(D):
    check(Case([(3, 20000), (130, 5000)], 6, 1, D, 64, seed=D))


@pytest.mark.parametrize("D", [64, 128, 256])
def test_outputs_are_the_rounded_ones(D):
    """Weights that are off by 2^-15 move an output of at least half its row's norm over a border between
    two bf16 numbers about once in 500 times (2.6% at 2^-11, as signs mix); fp32 scores add 1e-6."""
    c = Case([(200, 600), (3, 9000)], 8, 2, D, 64, seed=D, sharp=0.5)
    out = check(c)
    v = c.want()[0]
    large = v.abs() >= 0.5 * v.square().mean(-1, keepdim=True).sqrt()
    assert float((out.cpu() != v.bfloat16())[large].double().mean()) <= 0.01


@pytest.mark.parametrize("D", [64, 128, 256])
def test_values_that_are_not_finite(D):
    """An infinite value that all rows see stays one: both numbers of a weight have its sign."""
    for bad in (torch.inf, -torch.inf, torch.nan):
        c = Case([(20, 700), (130, 400)], 6, 2, D, 16, seed=3, sharp=0.5)
        for b, p in ((0, 5), (0, 300), (1, 0), (1, 330)):
            c.v[int(c.table[b, p // 16]), :, p % 16, 7 + p % 3] = bad
        check(c)


def test_a_weight_of_one():
    """One position: its two numbers are one and 2^-20, and the output is the value."""
    c = Case([(1, 1)] * 4, 8, 2, 128, 16, seed=1)
    out = check(c)
    for b in range(4):
        for h in range(8):
            assert torch.equal(out[b, h], c.v[int(c.table[b, 0]), h // 4, 0])


def test_eight_bits_are_left_as_they_are():
    c = Case([(33, 77), (300, 900)], 8, 2, 128, 32, E4M3, seed=1)
    with c.handle() as kv:
        a, la = c.run(kv)
        kv.set_option(moe.MOE_KV_OPT_CHUNK_WEIGHTS, 2)
        b, lb = c.run(kv)
        assert torch.equal(a, b) and torch.equal(la, lb)
        for value in (0, 3, -1):
            with pytest.raises(moe.MoEError):
                kv.set_option(moe.MOE_KV_OPT_CHUNK_WEIGHTS, value)


def test_a_wait_that_runs_out():
    for D in (64, 128, 256):
        c = Case([(9, 300), (40, 700), (1, 20000)], 8, 2, D, 32, seed=31)
        with c.handle() as kv:
            kv.set_option(moe.MOE_KV_OPT_CHUNK_WEIGHTS, 2)
            clean, _ = c.run(kv)
            kv.set_option(moe.MOE_KV_OPT_TEST_STALL, 1)
            out, _ = c.run(kv)
            assert kv.health() == (5, moe.MOE_KV_TIMEOUT)
            kv.set_option(moe.MOE_KV_OPT_TEST_STALL, -1)
            again, _ = c.run(kv)
            assert kv.health() == (0, 0)
        nan = torch.isnan(out).all(2)
        assert nan[9:49].all() and (nan | (out == clean).all(2)).all() and torch.equal(clean, again)
