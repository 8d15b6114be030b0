"""moe_kv_attend on the GPU within the bounds that its arithmetic gives, where
those of test_gpu_kv_attend.py are wider."""
import numpy as np
import pytest
import torch

import quantized_routed_expert_moe_gb300 as moe
import _decoder_ref
from _decoder_ref import assert_close, attend, rounded
from test_gpu_kv_attend import BF16, E4M3, Case

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


@pytest.mark.parametrize("nats", [8, 13, 16, 18, 24])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_a_flat_tail_beside_a_sink_in_8_bits(D, nats):
    """One position stands far above the rest and has values of zero, so that the output is
    the tail's alone. Weights go into the product as fp16: 2^-11 relative, and those 28
    octaves below the largest within 2^-39 of it."""
    lens, G, page = [20, 64, 700], 4, 16
    n_pages = sum(-(-n // page) for n in lens)
    g = torch.Generator("cuda").manual_seed(D + nats)
    k = torch.randn(n_pages, 1, page, D, generator=g, device="cuda") * 90
    v = torch.randn(n_pages, 1, page, D, generator=g, device="cuda") * 90
    k[..., 0] = 0
    q = torch.zeros(3, G, D, device="cuda")
    q[..., 0] = torch.tensor([1.0, 1.125, 0.5, 1.0], device="cuda")
    table, at = torch.zeros(3, -(-max(lens) // page), dtype=torch.int32), 0
    for b, (n, sink) in enumerate(zip(lens, (19, 0, 333))):
        need = -(-n // page)
        table[b, :need] = torch.arange(at, at + need)
        k[at + sink // page, 0, sink % page, 0] = nats
        v[at + sink // page, 0, sink % page] = 0
        at += need
    k, v, q = k.clamp(-448, 448).to(E4M3), v.clamp(-448, 448).to(E4M3), q.to(BF16)
    one = np.ones(1, np.float32)
    out, lse = torch.empty(3, G, D, dtype=BF16, device="cuda"), torch.empty(3, G, device="cuda")
    with moe.KVCache(k, v, n_heads=G, k_scale=one, v_scale=one, max_batch=3) as kv:
        kv.attend(q, table.cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda"), out, lse=lse, scale=1.0,
                  stream=torch.cuda.current_stream())
        assert kv.health() == (0, 0)
    for b, n in enumerate(lens):
        kk, vv = (_decoder_ref.gather(x, table, b, 0, n, 0) for x in (k, v))
        s = q[b].cpu().double() @ kk.T
        p = torch.softmax(s, 1)
        # the scores are sums of one term that is not zero: two roundings, and those of the
        # base and of the exponential's argument, each of a number up to 1.5 * 24 * 1.44
        rel = 2.0 ** -11 + 2.0 ** -21 + 4 * 52 * 2.0 ** -24 + 2 * n * 2.0 ** -24
        bound = rel * (p @ vv.abs()) + 2.0 ** -39 * vv.abs().sum(0) * p.amax(1, keepdim=True)
        assert_close(out[b], p @ vv, rounded(p @ vv, bound, BF16), f"out {b}")
        L = torch.logsumexp(s, 1)
        assert_close(lse[b], L, torch.full_like(L, 2.0 ** -21 + (n + 8 + 4 * 52) * 2.0 ** -24), f"lse {b}")


@pytest.mark.parametrize("dt", [BF16, E4M3])
@pytest.mark.parametrize("cap", [1e-3, 0.5, 50.0, 1e4, 1e7, 1e12, 3e38])
def test_caps_of_any_size(cap, dt):
    """The capped score is off relative to itself, not to the cap."""
    c = Case([1, 40, 513, 300], 8, 2, 128, 16, dt, seed=21, sharp=3.0)
    with c.handle() as kv:
        out, lse = c.run(kv, softcap=cap)
        assert kv.health() == (0, 0)
    cap32 = float(np.float32(cap))
    for b, n in enumerate(c.lens):
        for h in range(2):
            k, v = (_decoder_ref.gather(x, c.table, b, 0, n, h) * (1.0 if sc is None else float(sc[h]))
                    for x, sc in ((c.k, c.scales[0]), (c.v, c.scales[1])))
            q = c.q[b, 4 * h:4 * h + 4].cpu().double()
            s = cap32 * torch.tanh(q @ k.T * c.scale / cap32)
            # before the cap as without one; then the share of the cap, its tanh and the cap
            es = (128 + 6) * 2.0 ** -24 * (q.abs() @ k.abs().T * c.scale) + 12 * 2.0 ** -24 * s.abs()
            es = torch.minimum(es, torch.tensor(2 * cap32)).amax(1, keepdim=True)   # both are within the cap
            up = 2.0 ** (-16 if dt is BF16 else -11)
            p = torch.softmax(s, 1)
            rel = 2 * es + 2.0 ** -21 + up + 2 * n * 2.0 ** -24
            assert_close(out[b, 4 * h:4 * h + 4], p @ v, rounded(p @ v, rel * (p @ v.abs()), BF16), f"out {b} {h}")
            L = torch.logsumexp(s, 1)
            assert_close(lse[b, 4 * h:4 * h + 4], L, es[:, 0] + 2.0 ** -21 + n * 2.0 ** -24 + 8 * 2.0 ** -24 * L.abs(),
                         f"lse {b} {h}")


@pytest.mark.parametrize("dt", [BF16, E4M3])
@pytest.mark.parametrize("cap,times", [(1e30, 2.0 ** 85), (3e38, 2.0 ** 60), (1e24, 2.0 ** 60)])
def test_caps_above_large_scores(cap, times, dt):
    """Of one token the log-sum-exp is its score."""
    c = Case([1, 1, 1, 1], 4, 2, 64, 16, dt, seed=25)
    c.q *= times
    out, lse = c.check(softcap=0.0)
    with c.handle() as kv:
        out2, lse2 = c.run(kv, softcap=cap)
        assert kv.health() == (0, 0)
    # the scores are below cap / 2^10, the cap takes 2^-20 / 3 off them, in 12 operations more
    assert float(lse.abs().max()) < cap * 2.0 ** -10
    assert torch.all((lse - lse2).abs() <= (2.0 ** -21 + 24 * 2.0 ** -24) * lse.abs()) and torch.equal(out, out2)


@pytest.mark.parametrize("dt", [BF16, E4M3])
@pytest.mark.parametrize("times", [2.0 ** 20, 2.0 ** 40, 2.0 ** 90])
def test_scores_of_any_finite_size(times, dt):
    """Where the distance between two scores is far past the exponential's range, the
    position with the largest takes all."""
    c = Case([1, 90, 513], 4, 2, 64, 16, dt, seed=23)
    c.q *= times
    with c.handle() as kv:
        out, lse = c.run(kv)
        assert kv.health() == (0, 0)
    compared = 0
    for b, n in enumerate(c.lens):
        for h in range(4):
            k, v = (_decoder_ref.gather(x, c.table, b, 0, n, h // 2) * (1.0 if sc is None else float(sc[h // 2]))
                    for x, sc in ((c.k, c.scales[0]), (c.v, c.scales[1])))
            q = c.q[b, h].cpu().double()
            s = k @ q * c.scale
            # fp32 scores of 64 terms, their scale and the conversion to base two
            es = (64 + 6) * 2.0 ** -24 * float((k.abs() @ q.abs()).max() * c.scale)
            assert abs(float(lse[b, h]) - float(s.max())) <= es + 2.0 ** -20 * abs(float(s.max()))
            top = s.sort(descending=True).values
            if n == 1 or float(top[0] - top[1]) > 2 * es + 40:
                one = v[int(s.argmax())]
                assert_close(out[b, h], one, rounded(one, 2.0 ** -10 * one.abs(), BF16), f"out {b} {h}")
                compared += 1
    assert compared >= 10


@pytest.mark.parametrize("dt", [BF16, E4M3])
@pytest.mark.parametrize("n,B,Hk,G,D", [(20011, 1, 1, 16, 256), (30001, 1, 1, 16, 128), (9007, 2, 1, 12, 256),
                                        (24001, 1, 1, 40, 64), (16001, 1, 2, 9, 256)])
def test_long_segments_of_more_than_8_queries(n, B, Hk, G, D, dt, monkeypatch):
    """Two columns of heads: parts of many CTAs, joined in several batches."""
    monkeypatch.setattr(_decoder_ref, "UP", 2.0 ** (-16 if dt is BF16 else -11))
    Case([n - 1000 * b for b in range(B)], Hk * G, Hk, D, 64, dt, seed=n).check()
