"""BlockNorm and KVCache without stream=: on torch's current stream, behind the producers of
their inputs, also inside torch.cuda.stream()."""
import pytest
import torch

import quantized_routed_expert_moe_gb300 as moe

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def built():
    from quantized_routed_expert_moe_gb300 import build
    build.build()
    assert torch.cuda.is_available()


def late(pairs):
    """Fill tensors on the current stream, some 20 ms from now."""
    torch.cuda._sleep(40_000_000)
    for dst, src in pairs:
        dst.copy_(src)


def test_block_norm():
    x1, o1 = torch.randn(40, 512, device="cuda"), torch.randn(40, 512, device="cuda").to(BF16)
    x, o = torch.zeros_like(x1), torch.zeros_like(o1)
    r, h, want_r, want_h = (torch.empty_like(t) for t in (x, o, x, o))
    w = torch.ones(512, device="cuda")
    n = moe.BlockNorm(512, w, w)
    n.run(x1, o1, want_r, want_h, stream=torch.cuda.current_stream())
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        late(((x, x1), (o, o1)))
        n.run(x, o, r, h)
    s.synchronize()
    assert torch.equal(r, want_r) and torch.equal(h, want_h)


def test_append_and_attend():
    k1, v1 = (torch.randn(20, 2, 64, device="cuda").to(BF16) for _ in range(2))
    q1 = torch.randn(1, 4, 64, device="cuda").to(BF16)
    k, v, q = (torch.zeros_like(t) for t in (k1, v1, q1))
    pos = torch.arange(20, dtype=torch.int32, device="cuda")
    seq, lens = torch.zeros_like(pos), torch.full((1,), 20, dtype=torch.int32, device="cuda")
    table = torch.tensor([[1, 0]], dtype=torch.int32, device="cuda")
    out, want = torch.empty_like(q), torch.empty_like(q)
    pools = [torch.zeros(2, 2, 16, 64, device="cuda", dtype=BF16) for _ in range(4)]
    with moe.KVCache(*pools[:2], n_heads=4) as kv, moe.KVCache(*pools[2:], n_heads=4) as other:
        now = torch.cuda.current_stream()
        other.append(None, k1, v1, pos, table, seq=seq, stream=now)
        other.attend(q1, table, lens, want, stream=now)
        torch.cuda.synchronize()
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            late(((k, k1), (v, v1)))
            kv.append(None, k, v, pos, table, seq=seq)
        s.synchronize()
        assert torch.equal(pools[0], pools[2]) and torch.equal(pools[1], pools[3])
        with torch.cuda.stream(s):
            late(((q, q1),))
            kv.attend(q, table, lens, out)
        s.synchronize()
        assert kv.health() == (0, 0) and other.health() == (0, 0)
    assert torch.equal(out, want)


def test_in_a_capture():
    x = torch.randn(3, 512, device="cuda")
    h = torch.zeros(3, 512, device="cuda", dtype=BF16)
    n = moe.BlockNorm(512, None, torch.ones(512, device="cuda"))
    n.run(x, h=h)
    torch.cuda.synchronize()
    want = h.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        n.run(x, h=h)
    h.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(h, want)
