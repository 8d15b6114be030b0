"""moe_linear on the GPU against the product in 64 bits."""
import pytest
import torch

import quantized_routed_expert_moe_gb300 as moe
from _chunk_ref import linear
from _decoder_ref import assert_close, rounded

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def built():
    from quantized_routed_expert_moe_gb300 import build
    build.build()
    assert torch.cuda.is_available()


def run_case(T, K, N, out=BF16, act="none", bias=False, residual=False, inplace=False, room=0, seed=0, stream=None):
    g = torch.Generator("cuda").manual_seed(seed)

    def rows(n, width, dt, scale=1.0):
        """[n, width], with `room` more elements between the rows than a row has."""
        return (torch.randn(n, width + room, generator=g, device="cuda") * scale).to(dt)[:, :width]
    x, w = rows(T, K, BF16), rows(N, K, BF16, K ** -0.5)
    b = torch.randn(N, generator=g, device="cuda") if bias else None
    y = torch.full((T + 1, N + room), 7.0, dtype=out, device="cuda")
    body = y[:T, :N]
    r = rows(T, N, out, 2.0) if residual else None
    if inplace:
        body.copy_(r)
        arg = body
    else:
        arg = r
    value, bound = linear(x, w, b, act, r)
    lin = moe.Linear(w, bias=b, activation=act)
    if stream is not None:
        stream.wait_stream(torch.cuda.current_stream())
    lin.run(x, body, residual=arg, stream=stream)
    torch.cuda.synchronize()
    assert_close(body, value, rounded(value, bound, out), "y")
    assert (y[T:] == 7.0).all() and (y[:, N:] == 7.0).all(), "written outside the rows"
    return body.clone()


@pytest.mark.parametrize("out", [BF16, F32])
@pytest.mark.parametrize("T", [1, 2, 3, 7, 8, 9, 15, 16, 17, 31, 33, 63, 64, 65, 127, 128, 129, 200, 255, 257, 600])
def test_tokens(T, out):
    run_case(T, 256, 392, out, bias=True, residual=T % 2 == 0, seed=T)


@pytest.mark.parametrize("T", [1, 20, 130, 400])
@pytest.mark.parametrize("K,N", [(8, 8), (8, 136), (64, 64), (72, 8), (120, 264), (512, 768), (2824, 520), (1000, 128)])
def test_odd_sizes(T, K, N):
    run_case(T, K, N, BF16 if N % 16 else F32, seed=K + N)


@pytest.mark.parametrize("act", ["none", "silu", "gelu_tanh", "sigmoid"])
@pytest.mark.parametrize("out", [BF16, F32])
@pytest.mark.parametrize("T", [1, 70, 300])
def test_epilogues(T, act, out):
    for bias in (False, True):
        for residual in (False, True):
            run_case(T, 136, 200, out, act, bias, residual, seed=T)


@pytest.mark.parametrize("T,K,N", [(1, 6144, 8192), (4, 6144, 6144), (33, 6144, 2816), (128, 6144, 6144), (1030, 2816, 4096),
                                   (3001, 512, 768), (2500, 6144, 512), (300, 16384, 128)])
def test_layer_sizes(T, K, N):
    run_case(T, K, N, F32, residual=True, seed=1)


@pytest.mark.parametrize("T", [1, 50, 500])
def test_rows_with_gaps_and_in_place(T):
    run_case(T, 264, 328, BF16, "silu", True, True, room=40, seed=2)
    run_case(T, 264, 328, F32, "none", True, True, inplace=True, room=8, seed=3)
    run_case(T, 264, 328, BF16, "none", False, True, inplace=True, seed=4)


def test_no_tokens_and_other_stream():
    lin = moe.Linear(torch.zeros(16, 32, dtype=BF16, device="cuda"))
    lin.run(torch.zeros(0, 32, dtype=BF16, device="cuda"), torch.zeros(0, 16, dtype=BF16, device="cuda"))
    run_case(130, 256, 392, stream=torch.cuda.Stream())
    run_case(3, 256, 392, stream=torch.cuda.Stream())


def test_a_row_does_not_depend_on_the_others():
    """Infinities and NaN stay in their rows, and so do the weights' in their channels."""
    for T in (5, 40, 300):
        x = torch.randn(T, 128, device="cuda").bfloat16()
        w = torch.randn(264, 128, device="cuda").bfloat16()
        y, z = (torch.empty(T, 264, device="cuda") for _ in range(2))
        moe.Linear(w).run(x, y)
        x[1, 5], x[T - 1, 100] = torch.nan, torch.inf
        w[7, 3], w[263, 0] = torch.nan, -torch.inf
        moe.Linear(w).run(x, z)
        rows = torch.ones(T, dtype=torch.bool)
        rows[[1, T - 1]] = False
        cols = torch.ones(264, dtype=torch.bool)
        cols[[7, 263]] = False
        y, z = y.cpu(), z.cpu()
        assert torch.equal(y[rows][:, cols], z[rows][:, cols])
        assert torch.isnan(z[1]).all() and torch.isnan(z[:, 7]).all() and not torch.isfinite(z[T - 1]).any()


def test_large_and_small_values():
    for scale in (1e30, 1e-30):
        x = (torch.randn(30, 64, device="cuda") * scale).bfloat16()
        w = torch.randn(72, 64, device="cuda").bfloat16()
        for act in ("none", "silu", "gelu_tanh", "sigmoid"):
            y = torch.empty(30, 72, device="cuda")
            moe.Linear(w, activation=act).run(x, y)
            v, e = linear(x, w, None, act, None)
            assert torch.isfinite(y).all()
            assert_close(y, v, rounded(v, e, F32) + 2.0 ** -126, act)


@pytest.mark.parametrize("T", [1, 9, 128, 700])
def test_same_bits_every_time_and_in_a_graph(T):
    g = torch.Generator("cuda").manual_seed(T)
    x = torch.randn(T, 2816, generator=g, device="cuda").bfloat16()
    w = torch.randn(1032, 2816, generator=g, device="cuda").bfloat16()
    lin = moe.Linear(w)
    first, again = torch.empty(T, 1032, device="cuda"), torch.empty(T, 1032, device="cuda")
    lin.run(x, first)
    for _ in range(5):
        lin.run(x, again)
        torch.cuda.synchronize()
        assert torch.equal(first, again)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lin.run(x, again)
    again.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(first, again)


def test_two_streams_at_once():
    """No scratch is shared: calls on two streams may overlap."""
    x = torch.randn(64, 4096, device="cuda").bfloat16()
    ws = [torch.randn(2048, 4096, device="cuda").bfloat16() for _ in range(2)]
    want = [torch.empty(64, 2048, device="cuda") for _ in range(2)]
    for w, y in zip(ws, want):
        moe.Linear(w).run(x, y)
    torch.cuda.synchronize()
    lins, streams = [moe.Linear(w) for w in ws], [torch.cuda.Stream() for _ in range(2)]
    got = [[torch.empty(64, 2048, device="cuda") for _ in range(20)] for _ in range(2)]
    torch.cuda.synchronize()
    for i in range(20):
        for j in range(2):
            lins[j].run(x, got[j][i], stream=streams[j])
    torch.cuda.synchronize()
    for j in range(2):
        assert all(torch.equal(y, want[j]) for y in got[j])


def test_moved_weights_are_found():
    m = torch.nn.Linear(64, 72, bias=True)
    w = torch.nn.Parameter(m.weight.detach().bfloat16().cuda())
    lin = moe.Linear(w, bias=m.bias.detach().cuda())
    x = torch.randn(5, 64, device="cuda").bfloat16()
    y = torch.empty(5, 72, device="cuda")
    lin.run(x, y)
    w.data = (w.data * 2).clone()
    lin.run(x, y)
    v, e = linear(x, w, lin.bias, "none", None)
    torch.cuda.synchronize()
    assert_close(y, v, rounded(v, e, F32))


def test_refusals():
    w = torch.zeros(16, 32, dtype=BF16, device="cuda")
    x, y = torch.zeros(3, 32, dtype=BF16, device="cuda"), torch.zeros(3, 16, dtype=BF16, device="cuda")
    lin = moe.Linear(w)
    for args in ((x.float(), y), (x[:, :16], y), (x, y[:2]), (x, y[:, :8]), (x.cpu(), y), (x, y.cpu()),
                 (x, y, y.float()), (x, y, y[:2]), (x[0], y), (x, y.half())):
        with pytest.raises((ValueError, TypeError)):
            lin.run(*args)
    with pytest.raises(ValueError):
        moe.Linear(w, activation="relu6")
    with pytest.raises(ValueError):
        moe.Linear(w.float())
    with pytest.raises(ValueError):
        moe.Linear(w, bias=torch.zeros(16, dtype=BF16, device="cuda"))
    with pytest.raises(ValueError):
        moe.Linear(w.cpu())
    with pytest.raises(moe.MoEError):
        moe.Linear(torch.zeros(12, 32, dtype=BF16, device="cuda")).run(x, torch.zeros(3, 12, dtype=BF16, device="cuda"))
    with pytest.raises(moe.MoEError):   # rows that do not start on 16 bytes
        lin.run(torch.zeros(3, 36, dtype=BF16, device="cuda")[:, :32], y)
