"""moe_kv_append_norm on the GPU against the norm and the rotation in 64 bits."""
import numpy as np
import pytest
import torch

import quantized_routed_expert_moe_gb300 as moe
from _chunk_ref import head_norm, rotate64
from _decoder_ref import assert_close, f64, rounded

pytestmark = pytest.mark.gpu

BF16, E4M3 = torch.bfloat16, torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def built():
    from quantized_routed_expert_moe_gb300 import build
    build.build()
    assert torch.cuda.is_available()


def expected(x, w, eps, offset, pos, freq, adjacent):
    v, rel = head_norm(x, w, eps, offset)
    # the norm's error goes through the rotation with both channels of a pair; the rotation's
    # own is 2^-21 of them and 2^-52 of the angle
    turned = rotate64(v, pos, freq, adjacent)
    size = turned.abs() + rotate64(v.abs(), np.zeros_like(pos), freq, adjacent) + v.abs().amax(-1, keepdim=True)
    far = 2.0 ** -52 * float(np.abs(np.asarray(pos)).max(initial=0)) * (float(np.abs(freq).max()) if len(freq) else 0)
    return turned, (2 * rel + 2.0 ** -20 + far) * size


def run_case(T, Hq, Hk, d, page=16, dt=BF16, rot=None, adjacent=False, layout="hnd", which="qk", offset=0.0, eps=1e-6,
             seed=0, inplace=False, size=2.0, far=5000, zero_row=False, with_q=True, stream=None):
    g = torch.Generator("cuda").manual_seed(seed)
    rng = np.random.default_rng(seed)
    rot = d if rot is None else rot
    freq = np.array([10000.0 ** (-2.0 * i / rot) for i in range(rot // 2)])
    pos = rng.choice(max(far, 2 * T), size=T, replace=False)
    if T > 3:
        pos[1] = -1
    width = int(pos.max()) // page + 1
    need = sorted({int(p) // page for p in pos if p >= 0})
    n_pages = len(need) + 1
    table = np.full((1, width), -1, np.int32)
    table[0, need] = rng.permutation(n_pages)[:len(need)]
    shape = (n_pages, Hk, page, d) if layout == "hnd" else (n_pages, page, Hk, d)
    kp, vp = (torch.full(shape, 3.0, device="cuda", dtype=BF16).to(dt) for _ in range(2))
    if layout == "nhd":
        kp, vp = kp.permute(0, 2, 1, 3), vp.permute(0, 2, 1, 3)
    before = [f64(kp), f64(vp)]
    qkv = (torch.randn(T, (Hq + 2 * Hk) * d, generator=g, device="cuda") * size).to(BF16)
    if zero_row:
        qkv[0] = 0
    q, k, v = (qkv[:, a * d:b * d].unflatten(1, (b - a, d)) for a, b in ((0, Hq), (Hq, Hq + Hk), (Hq + Hk, Hq + 2 * Hk)))
    if inplace:
        q = q.contiguous()
    wq, wk = (torch.randn(d, generator=g, device="cuda") * 0.3 + 1 - offset for _ in range(2))
    wq, wk = wq if "q" in which else None, wk if "k" in which else None
    scales = (None, None) if dt == BF16 else (np.linspace(0.005, 0.02, Hk, dtype=np.float32),
                                              np.linspace(0.03, 0.01, Hk, dtype=np.float32))
    q_ref = q.clone()
    q_out = q if inplace else torch.full((T, Hq, d), 9.0, device="cuda", dtype=BF16)
    with moe.KVCache(kp, vp, n_heads=Hq, inv_freq=freq if rot else None, interleaved=adjacent, k_scale=scales[0],
                     v_scale=scales[1]) as kv:
        if stream is not None:
            stream.wait_stream(torch.cuda.current_stream())
        kv.append(q if with_q else None, k, v, torch.tensor(pos, dtype=torch.int32, device="cuda"),
                  torch.from_numpy(table).cuda(), q_out if with_q else None,
                  seq=torch.zeros(T, dtype=torch.int32, device="cuda"), q_norm=wq, k_norm=wk, norm_eps=eps,
                  norm_offset=offset, stream=stream)
        assert kv.health() == (0, 0)
    live = torch.from_numpy(pos >= 0)
    at = np.maximum(pos, 0)
    if with_q:
        vq, eq = expected(q_ref, wq, eps, offset, at, freq, adjacent)
        vq[~live], eq[~live] = 0, 0
        assert_close(q_out, vq, rounded(vq, eq, BF16) * live[:, None, None], "q")
    pg = torch.tensor([table[0, p // page] for p in pos if p >= 0], dtype=torch.long)
    sl = torch.tensor([p % page for p in pos if p >= 0], dtype=torch.long)
    for name, pool, old, (x, e), sc in (("k", kp, before[0], expected(k, wk, eps, offset, at, freq, adjacent), scales[0]),
                                        ("v", vp, before[1], (f64(v), torch.zeros(v.shape, dtype=torch.float64)), scales[1])):
        if dt == E4M3:
            s = torch.from_numpy(np.asarray(sc, np.float64))[None, :, None]
            x, e = x / s, e / s + (x / s).abs() * 2.0 ** -24
            x = x.clamp(-448, 448)
        got = f64(pool)
        assert_close(got[pg, :, sl], x[live], rounded(x, e, dt)[live], name)
        got[pg, :, sl] = old[pg, :, sl]
        assert torch.equal(got, old), f"{name}: slots outside the tokens changed"


@pytest.mark.parametrize("dt", [BF16, E4M3])
@pytest.mark.parametrize("adjacent", [False, True])
@pytest.mark.parametrize("d,rot", [(64, 64), (64, 16), (128, 128), (128, 48), (128, 0), (256, 256), (256, 64)])
def test_head_and_rotary_dims(d, rot, adjacent, dt):
    run_case(5, 4, 2, d, dt=dt, rot=rot, adjacent=adjacent, seed=d + rot)


@pytest.mark.parametrize("T,Hq,Hk", [(1, 1, 1), (1, 48, 8), (3, 6, 3), (17, 16, 1), (130, 8, 8), (401, 5, 5), (1500, 12, 4)])
@pytest.mark.parametrize("which", ["q", "k", "qk"])
def test_shapes(T, Hq, Hk, which):
    run_case(T, Hq, Hk, 64 if T % 2 else 128, 48 if T == 17 else 32, layout="nhd" if T % 2 else "hnd", which=which, seed=T,
             offset=float(T % 3 == 0))


@pytest.mark.parametrize("eps", [0.0, 1e-6, 0.5])
def test_eps_and_sizes(eps):
    for size in (1e-4, 1.0, 300.0):
        run_case(9, 4, 2, 128, eps=eps, size=size, seed=1)


def test_zero_heads():
    """A head of zeros stays zero: eps keeps its quotient finite."""
    run_case(6, 4, 2, 64, zero_row=True, seed=2)


def test_in_place_without_queries_and_other_stream():
    run_case(40, 8, 2, 64, inplace=True, seed=3)
    run_case(40, 8, 2, 64, with_q=False, seed=4)
    run_case(40, 8, 2, 64, seed=5, stream=torch.cuda.Stream())


def test_unit_weights_match_a_norm_before_the_append():
    """Against the append alone on queries normed by torch in 64 bits and rounded: one rounding apart."""
    torch.manual_seed(0)
    q, k, v = (torch.randn(7, h, 128, device="cuda").bfloat16() for h in (4, 2, 2))
    one = torch.ones(128, device="cuda")
    pos, seq = torch.arange(7, dtype=torch.int32, device="cuda"), torch.zeros(7, dtype=torch.int32, device="cuda")
    table = torch.zeros(1, 1, dtype=torch.int32, device="cuda")
    freq = 10000.0 ** (-np.arange(64) / 64)
    outs = []
    for normed in (False, True):
        pools = torch.zeros(2, 1, 2, 16, 128, dtype=BF16, device="cuda")
        out = torch.empty_like(q)
        with moe.KVCache(pools[0], pools[1], n_heads=4, inv_freq=freq) as kv:
            if normed:
                qq, kk = ((x.double() / (x.double().square().mean(-1, keepdim=True) + 1e-6).sqrt()).bfloat16() for x in (q, k))
                kv.append(qq, kk, v, pos, table, out, seq=seq)
            else:
                kv.append(q, k, v, pos, table, out, seq=seq, q_norm=one, k_norm=one)
            torch.cuda.synchronize()
        outs.append((out.double(), pools.double()))
    for a, b in zip(*outs):
        assert float((a - b).abs().max()) <= 2.0 ** -7 * float(b.abs().max())


def test_graph():
    torch.manual_seed(1)
    q, k, v = (torch.randn(3, h, 64, device="cuda").bfloat16() for h in (4, 2, 2))
    w = torch.rand(64, device="cuda")
    pos, seq = torch.arange(3, dtype=torch.int32, device="cuda"), torch.zeros(3, dtype=torch.int32, device="cuda")
    table = torch.zeros(1, 1, dtype=torch.int32, device="cuda")
    pools = torch.zeros(2, 1, 2, 16, 64, dtype=BF16, device="cuda")
    eager, out = torch.empty_like(q), torch.empty_like(q)
    with moe.KVCache(pools[0], pools[1], n_heads=4, inv_freq=np.ones(32)) as kv:
        kv.append(q, k, v, pos, table, eager, seq=seq, q_norm=w, k_norm=w)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            kv.append(q, k, v, pos, table, out, seq=seq, q_norm=w, k_norm=w)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, eager)


def test_refusals():
    pools = torch.zeros(2, 1, 2, 16, 64, dtype=BF16, device="cuda")
    x = torch.zeros(1, 2, 64, dtype=BF16, device="cuda")
    i = torch.zeros(1, dtype=torch.int32, device="cuda")
    w = torch.ones(64, device="cuda")
    with moe.KVCache(pools[0], pools[1], n_heads=2) as kv:
        for bad in (w[:32], w.double(), w.cpu(), torch.ones(128, device="cuda")[::2]):
            with pytest.raises(ValueError):
                kv.append(x, x, x, i, i[None], x.clone(), q_norm=bad)
            with pytest.raises(ValueError):
                kv.append(x, x, x, i, i[None], x.clone(), k_norm=bad)
        with pytest.raises(moe.MoEError):
            kv.append(x, x, x, i, i[None], x.clone(), q_norm=w, norm_eps=-1.0)
        with pytest.raises(ValueError):
            kv.append(x, x, x, i, i[None], x.clone(), q_norm=w, norm_eps="a")
