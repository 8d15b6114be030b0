"""moe_kv_attend_chunk on caps and scores of any size, within the bounds that its arithmetic gives."""
import numpy as np
import pytest
import torch

import quantized_routed_expert_moe_gb300 as moe
import _decoder_ref
from _decoder_ref import assert_close, rounded
from test_gpu_kv_attend_chunk import BF16, E4M3, Case

pytestmark = pytest.mark.gpu

DS = [(64, BF16), (128, BF16), (256, BF16), (64, E4M3), (128, E4M3), (256, E4M3)]


@pytest.fixture(scope="module", autouse=True)
def built():
    from quantized_routed_expert_moe_gb300 import build
    build.build()
    assert torch.cuda.is_available()


def rows(c):
    """(row, sequence, cached tokens that it sees) of every token."""
    for b, n in enumerate(c.new):
        for i in range(n):
            if c.lens[b] - n + i >= 0:
                yield c.starts[b] + i, b, c.lens[b] - n + i + 1


def cached(c, b, n, h):
    return (_decoder_ref.gather(x, c.table, b, 0, n, h) * (1.0 if sc is None else float(sc[h]))
            for x, sc in ((c.k, c.scales[0]), (c.v, c.scales[1])))


@pytest.mark.parametrize("D,dt", DS)
@pytest.mark.parametrize("cap", [1e-44, 1e-38, 1e-20, 1e-3, 0.5, 50.0, 1e4, 1e7, 1e12, 1e24, 3e38])
def test_caps_of_any_size(cap, D, dt):
    """The capped score is off relative to itself, not to the cap."""
    c = Case([(1, 1), (2, 40), (5, 513), (3, 3)], 8, 2, D, 16, dt, seed=21, sharp=3.0)
    c.q[3] = 0   # scores of zero
    cap32 = float(np.float32(cap))
    with c.handle() as kv:
        out, lse = c.run(kv, softcap=cap32)
        assert kv.health() == (0, 0)
    up = 2.0 ** (-8 if dt is BF16 else -11)
    for t, b, n in rows(c):
        for h in range(2):
            k, v = cached(c, b, n, h)
            q = c.q[t, 4 * h:4 * h + 4].cpu().double()
            s = cap32 * torch.tanh(q @ k.T * c.scale / cap32)
            # before the cap as without one; then the share of the cap, its tanh and the cap (2^-126: the
            # products' own underflow)
            es = (D + 6) * 2.0 ** -24 * (q.abs() @ k.abs().T * c.scale) + 12 * 2.0 ** -24 * s.abs() + 2.0 ** -126
            es = torch.minimum(es, torch.tensor(2 * cap32 + 2.0 ** -126)).amax(1, keepdim=True)   # both are within the cap
            p = torch.softmax(s, 1)
            rel = 2 * es + 2.0 ** -21 + up + 2 * n * 2.0 ** -24
            assert_close(out[t, 4 * h:4 * h + 4], p @ v, rounded(p @ v, rel * (p @ v.abs()), BF16), f"out {t} {h}")
            L = torch.logsumexp(s, 1)
            assert_close(lse[t, 4 * h:4 * h + 4], L, es[:, 0] + 2.0 ** -21 + n * 2.0 ** -24 + 8 * 2.0 ** -24 * L.abs(),
                         f"lse {t} {h}")


@pytest.mark.parametrize("D,dt", DS)
@pytest.mark.parametrize("cap,times,scale", [(1e30, 2.0 ** 85, 0.125), (3e38, 2.0 ** 60, 0.125), (1e24, 2.0 ** 60, 0.125),
                                             (1e22, 2.0 ** 110, 2.0 ** -108), (1e20, 2.0 ** 100, 2.0 ** -80)])
def test_caps_above_large_scores(cap, times, scale, D, dt):
    """Of one position the log-sum-exp is its score."""
    c = Case([(1, 1)] * 4, 4, 2, D, 16, dt, seed=25)
    c.q *= times
    c.scale = scale
    out, lse = c.check(softcap=0.0)
    with c.handle() as kv:
        out2, lse2 = c.run(kv, softcap=cap)
        assert kv.health() == (0, 0)
    # the scores are below cap / 2^10, the cap takes 2^-20 / 3 off them, in 12 operations more
    assert float(lse.abs().max()) < cap * 2.0 ** -10
    assert torch.all((lse - lse2).abs() <= (2.0 ** -21 + 24 * 2.0 ** -24) * lse.abs()) and torch.equal(out, out2)


@pytest.mark.parametrize("D,dt", DS)
@pytest.mark.parametrize("times", [2.0 ** 20, 2.0 ** 40, 2.0 ** 90])
def test_scores_of_any_finite_size(times, D, dt):
    """Where the distance between two scores is far past the exponential's range, the position with
    the largest takes all."""
    c = Case([(1, 1), (3, 90), (4, 513)], 4, 2, D, 16, dt, seed=23)
    c.q *= times
    with c.handle() as kv:
        out, lse = c.run(kv)
        assert kv.health() == (0, 0)
    compared = 0
    for t, b, n in rows(c):
        for h in range(4):
            k, v = cached(c, b, n, h // 2)
            q = c.q[t, h].cpu().double()
            s = k @ q * c.scale
            # fp32 scores of D terms, their scale and the conversion to base two
            es = (D + 6) * 2.0 ** -24 * float((k.abs() @ q.abs()).max() * c.scale)
            assert abs(float(lse[t, h]) - float(s.max())) <= es + 2.0 ** -20 * abs(float(s.max()))
            top = s.sort(descending=True).values
            if n == 1 or float(top[0] - top[1]) > 2 * es + 40:
                one = v[int(s.argmax())]
                assert_close(out[t, h], one, rounded(one, 2.0 ** -8 * one.abs(), BF16), f"out {t} {h}")
                compared += 1
    assert compared >= 20


@pytest.mark.parametrize("nats", [8, 13, 16, 18])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_a_flat_tail_beside_a_sink_in_8_bits(D, nats):
    """One position stands far above the rest and has values of zero, so that the output is the tail's
    alone: weights go into the product as fp16, 2^-11 relative, or 2^-32 of the largest."""
    lens, new, G, page = [20, 64, 700], [1, 3, 2], 4, 16
    n_pages = sum(-(-n // page) for n in lens)
    g = torch.Generator("cuda").manual_seed(D + nats)
    k = torch.randn(n_pages, 1, page, D, generator=g, device="cuda") * 90
    v = torch.randn(n_pages, 1, page, D, generator=g, device="cuda") * 90
    k[..., 0] = 0
    q = torch.zeros(sum(new), G, D, device="cuda")
    q[..., 0] = torch.tensor([1.0, 1.125, 0.5, 1.0], device="cuda")
    table, at = torch.zeros(3, -(-max(lens) // page), dtype=torch.int32), 0
    for b, (n, sink) in enumerate(zip(lens, (9, 0, 333))):
        need = -(-n // page)
        table[b, :need] = torch.arange(at, at + need)
        k[at + sink // page, 0, sink % page, 0] = nats
        v[at + sink // page, 0, sink % page] = 0
        at += need
    k, v, q = k.clamp(-448, 448).to(E4M3), v.clamp(-448, 448).to(E4M3), q.to(BF16)
    one = np.ones(1, np.float32)
    out, lse = torch.empty_like(q), torch.empty(sum(new), G, device="cuda")
    starts = [0, 1, 4, 6]
    with moe.KVCache(k, v, n_heads=G, k_scale=one, v_scale=one, max_batch=3) as kv:
        kv.attend_chunk(q, torch.tensor(starts, dtype=torch.int32, device="cuda"), table.cuda(),
                        torch.tensor(lens, dtype=torch.int32, device="cuda"), out, lse=lse, scale=1.0)
        assert kv.health() == (0, 0)
    for b in range(3):
        for t in range(starts[b], starts[b + 1]):
            n = lens[b] - (starts[b + 1] - t) + 1
            kk, vv = (_decoder_ref.gather(x, table, b, 0, n, 0) for x in (k, v))
            s = q[t].cpu().double() @ kk.T
            p = torch.softmax(s, 1)
            # the scores are sums of one term that is not zero: two roundings, and those of the
            # base and of the exponential's argument, each of a number up to 1.5 * 24 * 1.44
            rel = 2.0 ** -11 + 2.0 ** -21 + 4 * 52 * 2.0 ** -24 + 2 * n * 2.0 ** -24
            bound = rel * (p @ vv.abs()) + 2.0 ** -32 * vv.abs().sum(0) * p.amax(1, keepdim=True)
            assert_close(out[t], p @ vv, rounded(p @ vv, bound, BF16), f"out {t}")
            L = torch.logsumexp(s, 1)
            assert_close(lse[t], L, torch.full_like(L, 2.0 ** -21 + (n + 8 + 4 * 52) * 2.0 ** -24), f"lse {t}")
