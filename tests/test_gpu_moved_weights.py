"""Weights and pools that get new memory after an object has been made over them."""
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


def test_the_norm_reads_the_weights_where_they_are():
    x, o = torch.randn(5, 256, device="cuda"), torch.randn(5, 256, device="cuda").to(BF16)
    w, v = (torch.nn.Parameter(torch.randn(256, device="cuda"), requires_grad=False) for _ in range(2))
    n = moe.BlockNorm(256, w, v)
    r, h, want_r, want_h = (torch.empty_like(t) for t in (x, o, x, o))
    n.run(x, o, r, h)
    w.data, v.data = w.data * -2.0, torch.randn(256, device="cuda")   # as moving a module does
    n.run(x, o, r, h)
    moe.BlockNorm(256, w.detach().clone(), v.detach().clone()).run(x, o, want_r, want_h)
    torch.cuda.synchronize()
    assert torch.equal(r, want_r) and torch.equal(h, want_h)


@pytest.mark.parametrize("which", ["w_post", "w_pre"])
@pytest.mark.parametrize("to", [lambda t: t.to(BF16), lambda t: t.cpu(), lambda t: t[:128], lambda t: t.repeat(2)[::2]])
def test_the_norm_refuses_what_they_became(which, to):
    x, o = torch.randn(5, 256, device="cuda"), torch.randn(5, 256, device="cuda").to(BF16)
    n = moe.BlockNorm(256, torch.ones(256, device="cuda"), torch.ones(256, device="cuda"))
    w = getattr(n, which)
    setattr(n, which, to(w))
    with pytest.raises(ValueError, match=which):
        n.run(x, o, torch.empty_like(x), torch.empty_like(o))


def test_the_cache_refuses_pools_with_new_memory():
    kp, vp = (torch.nn.Parameter(torch.zeros(3, 2, 16, 64, device="cuda", dtype=BF16), requires_grad=False)
              for _ in range(2))
    k, q = torch.randn(1, 2, 64, device="cuda").to(BF16), torch.randn(1, 4, 64, device="cuda").to(BF16)
    pos, table = (torch.zeros(n, dtype=torch.int32, device="cuda") for n in ((1,), (1, 1)))
    for pool in (kp, vp):
        with moe.KVCache(kp, vp, n_heads=4) as kv:
            kv.append(None, k, k, pos, table)
            torch.cuda.synchronize()
            old, pool.data = pool.data, torch.zeros_like(pool)
            with pytest.raises(ValueError, match="new memory"):
                kv.append(None, k, k, pos, table)
            with pytest.raises(ValueError, match="new memory"):
                kv.attend(q, table, pos + 1, torch.empty_like(q))
            pool.data = old
            kv.attend(q, table, pos + 1, torch.empty_like(q))
            assert kv.health() == (0, 0)
