"""moe_block_norm on the GPU against its 64-bit form."""
import numpy as np
import pytest
import torch

import quantized_routed_expert_moe_gb300 as moe
from _decoder_ref import assert_close, block_norm, rounded

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def built():
    from quantized_routed_expert_moe_gb300 import build
    build.build()
    assert torch.cuda.is_available()


def make(T, H, res=F32, blk=BF16, out=BF16, post=True, gate="none", seed=0, pad=0):
    g = torch.Generator("cuda").manual_seed(seed)

    def rows(n, dt, amp=1.0):
        return (torch.randn(n, H + pad, generator=g, device="cuda") * amp).to(dt)[:, :H]
    x, o = rows(T, res, 3.0), rows(T, blk)
    ga = {"none": None, "row": rows(1, blk)[0].contiguous() if gate == "row" else None,
          "full": rows(T, blk) if gate == "full" else None}[gate]
    wp = torch.randn(H, generator=g, device="cuda") if post else None
    wn = torch.randn(H, generator=g, device="cuda")
    r = torch.full((T, H + pad), 7.0, dtype=res, device="cuda")[:, :H]
    h = torch.full((T, H + pad), 7.0, dtype=out, device="cuda")[:, :H]
    return x, o, ga, wp, wn, r, h


def check(x, o, ga, wp, wn, r, h, eps=1e-6, scale=1.0, offset=0.0, stream=None):
    vr, er, vh, eh = block_norm(x, o, ga, wp, wn if h is not None else None, eps, scale, offset)
    moe.BlockNorm(x.shape[1], wp, wn, eps=eps, scale=scale, weight_offset=offset).run(x, o, r, h, gate=ga, stream=stream)
    torch.cuda.synchronize()
    if r is not None:
        assert_close(r, vr, rounded(vr, er, r.dtype), "r")
    if h is not None:
        assert_close(h, vh, rounded(vh, eh, h.dtype), "h")


@pytest.mark.parametrize("H", [64, 128, 192, 704, 1088, 2048, 2816, 4160, 6144, 8192, 12352, 16384])
@pytest.mark.parametrize("T", [1, 5])
def test_sizes(T, H):
    check(*make(T, H, gate="full", seed=H + T), scale=0.5, offset=1.0)


@pytest.mark.parametrize("res", [F32, BF16])
@pytest.mark.parametrize("blk", [F32, BF16])
@pytest.mark.parametrize("out", [F32, BF16])
@pytest.mark.parametrize("post,gate", [(True, "none"), (False, "row"), (True, "full"), (False, "none")])
def test_types(res, blk, out, post, gate):
    check(*make(3, 832, res, blk, out, post, gate, seed=5), scale=-0.7, offset=0.5)


@pytest.mark.parametrize("T", [2, 151, 152, 153, 700, 3001])
def test_many_rows(T):
    check(*make(T, 512, gate="row", seed=T))


# more rows than the device holds at a time, in every layout of a row
@pytest.mark.parametrize("res,blk,out,gate", [(F32, BF16, BF16, "full"), (F32, F32, F32, "row"),
                                              (BF16, BF16, F32, "none"), (BF16, F32, BF16, "full")])
@pytest.mark.parametrize("T,H", [(20001, 64), (20001, 320), (12345, 768), (12345, 1024), (2501, 1088), (2501, 4160),
                                 (2501, 4608), (2501, 5120), (2501, 6144),
                                 (2501, 6208), (1701, 8192), (701, 8256), (701, 11264), (701, 12352), (701, 16384)])
def test_many_rows_of_every_layout(T, H, res, blk, out, gate):
    check(*make(T, H, res, blk, out, True, gate, seed=H), scale=0.75, offset=1.0)


@pytest.mark.parametrize("gate", ["full", "row"])
def test_strided_rows(gate):
    x, o, ga, wp, wn, r, h = make(9, 320, gate=gate, seed=3, pad=24)
    rest = [t._base for t in (r, h)]
    check(x, o, ga, wp, wn, r, h)
    for t in rest:   # what lies between the rows is left alone
        assert torch.all(t[:, 320:] == 7.0)


def test_residual_in_place():
    x, o, ga, wp, wn, r, h = make(33, 1024, seed=8)
    vr, er, vh, eh = block_norm(x, o, ga, wp, wn, 1e-6, 1.0, 0.0)
    moe.BlockNorm(1024, wp, wn).run(x, o, x, h)
    torch.cuda.synchronize()
    assert_close(x, vr, rounded(vr, er, x.dtype), "r")
    assert_close(h, vh, rounded(vh, eh, h.dtype), "h")


def test_norm_only_and_sum_only():
    x, o, ga, wp, wn, r, h = make(6, 640, seed=2)
    check(x, None, None, None, wn, None, h)      # the first norm of a stack
    check(x, None, None, None, wn, r, h)
    check(x, o, None, wp, wn, r, None)           # the last block: no next norm
    check(x, o, None, wp, wn, None, h)


def test_zero_rows_and_empty_batch():
    x, o, ga, wp, wn, r, h = make(4, 256, seed=1)
    x[1], o[1] = 0, 0
    o[2] = 0
    check(x, o, ga, wp, wn, r, h)
    assert torch.all(h[1] == 0)
    r.fill_(3.0)
    moe.BlockNorm(256, wp, wn).run(x[:0], o[:0], r[:0], h[:0])
    torch.cuda.synchronize()
    assert torch.all(r == 3.0)


@pytest.mark.parametrize("amp", [1e-15, 1e15])
def test_magnitudes(amp):
    """The squares stay within fp32: 1e-30 with eps 0, 1e30 * H."""
    x, o, ga, wp, wn, r, h = make(4, 512, F32, F32, F32, seed=4)
    check(x * amp, o * amp, ga, wp, wn, r, h, eps=0.0)


def test_infinity_and_nan_stay_in_their_row():
    x, o, ga, wp, wn, r, h = make(5, 512, seed=6)
    clean = make(5, 512, seed=6)
    moe.BlockNorm(512, wp, wn).run(clean[0], clean[1], clean[5], clean[6])
    x[1, 3] = torch.nan
    o[3, 7] = torch.inf
    moe.BlockNorm(512, wp, wn).run(x, o, r, h)
    torch.cuda.synchronize()
    for t in (0, 2, 4):
        assert torch.equal(r[t], clean[5][t]) and torch.equal(h[t], clean[6][t])
    assert torch.isnan(h[1]).all() and torch.isnan(r[1, 3]) and torch.isfinite(r[1]).sum() == 511
    assert torch.isnan(r[3, 7]) and torch.isnan(h[3]).all()


def test_repeats_bit_for_bit_on_another_stream():
    x, o, ga, wp, wn, r, h = make(300, 2816, BF16, gate="row", seed=9)
    n = moe.BlockNorm(2816, wp, wn, scale=0.3)
    n.run(x, o, r, h, gate=ga)
    torch.cuda.synchronize()
    r2, h2 = torch.empty_like(r), torch.empty_like(h)
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        n.run(x, o, r2, h2, gate=ga, stream=s)
    s.synchronize()
    assert torch.equal(r, r2) and torch.equal(h, h2)


def test_captured_in_a_graph():
    x, o, ga, wp, wn, r, h = make(7, 1024, seed=10)
    n = moe.BlockNorm(1024, wp, wn)
    n.run(x, o, r, h)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        n.run(x, o, r, h, stream=torch.cuda.current_stream())
    x.copy_(x * 2 + 1)
    g.replay()
    torch.cuda.synchronize()
    vr, er, vh, eh = block_norm(x, o, ga, wp, wn, 1e-6, 1.0, 0.0)
    assert_close(r, vr, rounded(vr, er, r.dtype), "r")
    assert_close(h, vh, rounded(vh, eh, h.dtype), "h")


def test_binding_refuses_other_tensors():
    x, o, ga, wp, wn, r, h = make(4, 256, seed=1)
    n = moe.BlockNorm(256, wp, wn)
    for bad in (dict(x=x[:, :128]), dict(o=o[:2]), dict(r=r.to(BF16)), dict(h=h.cpu()), dict(x=x.T.contiguous().T),
                dict(gate=torch.ones(3, 256, device="cuda", dtype=BF16)), dict(gate=torch.ones(256, device="cuda"))):
        a = dict(x=x, o=o, r=r, h=h)
        a.update(bad)
        with pytest.raises((ValueError, TypeError)):
            n.run(**a)
    with pytest.raises(moe.MoEError):
        n.run(x, o, None, None)
