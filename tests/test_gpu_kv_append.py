"""moe_kv_append on the GPU against the 64-bit rotation and the cache's rounding."""
import numpy as np
import pytest
import torch

import quantized_routed_expert_moe_gb300 as moe
from _decoder_ref import assert_close, f64, rotate, rounded

pytestmark = pytest.mark.gpu

BF16, E4M3 = torch.bfloat16, torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def built():
    from quantized_routed_expert_moe_gb300 import build
    build.build()
    assert torch.cuda.is_available()


def freqs(rot, theta=10000.0):
    return np.array([theta ** (-2.0 * i / rot) for i in range(rot // 2)])


def pool(n, hk, page, d, dt, layout, fill=3.0):
    shape = (n, hk, page, d) if layout == "hnd" else (n, page, hk, d)
    x = torch.full(shape, fill, device="cuda", dtype=BF16).to(dt)
    return x if layout == "hnd" else x.permute(0, 2, 1, 3)


def expect(x, scale, dt):
    """What the cache holds of the values x (64-bit) with their bounds e."""
    v, e = x
    if dt == BF16:
        return v, rounded(v, e, dt)
    s = torch.from_numpy(np.asarray(scale, np.float64))[None, :, None]
    v, e = v / s, e / s + (v / s).abs() * 2.0 ** -24
    v = v.clamp(-448, 448)
    return v, rounded(v, e, dt)


def run_case(T, Hq, Hk, d, page, dt=BF16, rot=None, adjacent=False, layout="hnd", positions=None, seq=None, seed=0,
             split=True, with_q=True, inplace=False, stream=None):
    g = torch.Generator("cuda").manual_seed(seed)
    rot = d if rot is None else rot
    rng = np.random.default_rng(seed)
    if positions is None:
        positions = rng.choice(max(15 * page, 2 * T), size=T, replace=False)
    positions = np.asarray(positions)
    seq_np = np.zeros(T, int) if seq is None else np.asarray(seq)
    n_seqs, width = int(seq_np.max()) + 1, int(max(positions.max(), 0)) // page + 1
    # a page for every (sequence, page index) that is written
    need = sorted({(int(s), int(p) // page) for s, p in zip(seq_np, positions) if p >= 0})
    n_pages = len(need) + 2
    table = np.full((n_seqs, width), -1, np.int32)
    for (s, i), pg in zip(need, rng.permutation(n_pages)):
        table[s, i] = pg
    kp, vp = pool(n_pages, Hk, page, d, dt, layout), pool(n_pages, Hk, page, d, dt, layout)
    kp0, vp0 = f64(kp), f64(vp)
    if split:
        qkv = torch.randn(T, (Hq + 2 * Hk) * d, generator=g, device="cuda").to(BF16)
        q = qkv[:, :Hq * d].unflatten(1, (Hq, d))
        k = qkv[:, Hq * d:(Hq + Hk) * d].unflatten(1, (Hk, d))
        v = qkv[:, (Hq + Hk) * d:].unflatten(1, (Hk, d))
    else:
        q, k, v = (torch.randn(T, n, d, generator=g, device="cuda").to(BF16) for n in (Hq, Hk, Hk))
    scales = (None, None) if dt == BF16 else (np.linspace(0.005, 0.02, Hk, dtype=np.float32),
                                              np.linspace(0.03, 0.004, Hk, dtype=np.float32))
    f = freqs(rot) if rot else np.zeros(0)
    q_ref = q.clone()
    q_out = q if inplace else torch.full((T, Hq, d), 9.0, device="cuda", dtype=BF16)
    with moe.KVCache(kp, vp, n_heads=Hq, inv_freq=f, interleaved=adjacent, k_scale=scales[0], v_scale=scales[1]) as kv:
        kv.append(q if with_q else None, k, v, torch.tensor(positions, dtype=torch.int32, device="cuda"),
                  torch.from_numpy(table).cuda(), q_out if with_q else None,
                  seq=torch.tensor(seq_np, dtype=torch.int32, device="cuda"), stream=stream)
        assert kv.health() == (0, 0)
        offs = [kv.locate(table, int(s), int(p), 0) for s, p in zip(seq_np, positions) if p >= 0]
    live = positions >= 0
    lt = torch.from_numpy(live)
    if with_q:
        vq, eq = rotate(q_ref, np.maximum(positions, 0), f, adjacent)
        vq[~lt], eq[~lt] = 0, 0
        assert_close(q_out, vq, rounded(vq, eq, BF16) * lt[:, None, None], "q")
    pg = torch.tensor([table[s, p // page] for s, p in zip(seq_np, positions) if p >= 0], dtype=torch.long)
    sl = torch.tensor([p % page for p in positions if p >= 0], dtype=torch.long)
    for name, got, before, x, sc in (("k", kp, kp0, rotate(k, np.maximum(positions, 0), f, adjacent), scales[0]),
                                     ("v", vp, vp0, (f64(v), torch.zeros(v.shape, dtype=torch.float64)), scales[1])):
        want, bound = expect(x, sc, dt)
        a = f64(got)
        assert_close(a[pg, :, sl], want[lt], bound[lt], name)
        a[pg, :, sl] = before[pg, :, sl]
        assert torch.equal(a, before), f"{name}: slots outside the tokens changed"
    # moe_kv_locate points at the same rows
    flat = kp.as_strided((n_pages * Hk * page * d,), (1,))
    for o, p, s in list(zip(offs, pg.tolist(), sl.tolist()))[:4]:
        assert torch.equal(f64(flat[o:o + d]), f64(kp[p, 0, s]))


@pytest.mark.parametrize("dt", [BF16, E4M3])
@pytest.mark.parametrize("adjacent", [False, True])
@pytest.mark.parametrize("d,rot", [(64, 64), (64, 16), (128, 128), (128, 48), (128, 0), (256, 256), (256, 64)])
def test_head_and_rotary_dims(d, rot, adjacent, dt):
    run_case(5, 4, 2, d, 16, dt, rot, adjacent, seed=d + rot)


@pytest.mark.parametrize("T,Hq,Hk", [(1, 1, 1), (1, 48, 8), (3, 6, 3), (17, 16, 1), (130, 8, 8), (401, 5, 5)])
@pytest.mark.parametrize("page", [16, 48, 128])
def test_shapes(T, Hq, Hk, page):
    run_case(T, Hq, Hk, 64, page, layout="nhd" if T % 2 else "hnd", seed=T, split=T % 3 != 0)


# enough tokens that a warp has several units, of one round or more of a token
@pytest.mark.parametrize("T,Hq,Hk,d,rot,adjacent", [(700, 32, 8, 128, 128, False), (1333, 16, 4, 64, 32, True),
                                                    (3777, 12, 2, 64, 64, False), (4001, 5, 1, 256, 128, True),
                                                    (8000, 3, 1, 128, 96, False)])
@pytest.mark.parametrize("dt", [BF16, E4M3])
def test_many_tokens(T, Hq, Hk, d, rot, adjacent, dt):
    run_case(T, Hq, Hk, d, 32, dt, rot, adjacent, seed=T)


@pytest.mark.parametrize("dt", [BF16, E4M3])
def test_far_positions(dt):
    """Angles of 10^6 turns and more: the phase may not lose its fraction."""
    pos = [0, 1, 65535, 999999, 1000003, 16777217, 123456789, 2 ** 31 - 4100]
    seq = list(range(8))
    run_case(8, 2, 2, 128, 4096, dt, positions=pos, seq=seq, seed=1)


def test_padding_and_sequences():
    run_case(7, 4, 2, 64, 16, positions=[5, -1, 0, 31, -7, 16, 15], seq=[0, 0, 2, 1, 1, 2, 1], seed=3)


def test_token_t_is_sequence_t_by_default():
    kp, vp = pool(4, 1, 16, 64, BF16, "hnd", 0.0), pool(4, 1, 16, 64, BF16, "hnd", 0.0)
    k = torch.randn(3, 1, 64, device="cuda").to(BF16)
    table = torch.tensor([[2], [0], [3], [1]], dtype=torch.int32, device="cuda")
    with moe.KVCache(kp, vp, n_heads=1) as kv:
        kv.append(None, k, k, torch.tensor([4, 0, 15], dtype=torch.int32, device="cuda"), table)
        assert kv.health() == (0, 0)
    for t, (p, s) in enumerate(((2, 4), (0, 0), (3, 15))):
        assert torch.equal(kp[p, 0, s], k[t, 0]) and torch.equal(vp[p, 0, s], k[t, 0])


def test_without_queries_and_in_place():
    run_case(6, 4, 2, 128, 16, with_q=False)
    run_case(6, 4, 2, 128, 16, inplace=True, split=False)
    run_case(6, 4, 2, 128, 16, rot=64, adjacent=True, inplace=True, split=False)


def test_saturation_nan_and_infinity_in_8_bits():
    kp, vp = pool(1, 1, 16, 64, E4M3, "hnd"), pool(1, 1, 16, 64, E4M3, "hnd")
    k = torch.zeros(1, 1, 64, device="cuda", dtype=BF16)
    k[0, 0, :6] = torch.tensor([1e30, -1e30, float("inf"), float("-inf"), float("nan"), 448.0])
    one = np.ones(1, np.float32)
    with moe.KVCache(kp, vp, n_heads=1, k_scale=one, v_scale=one) as kv:
        kv.append(None, k, k, torch.zeros(1, dtype=torch.int32, device="cuda"),
                  torch.zeros(1, 1, dtype=torch.int32, device="cuda"))
        assert kv.health() == (0, 0)
    got = f64(kp[0, 0, 0])
    assert got[:4].tolist() == [448, -448, 448, -448] and torch.isnan(got[4]) and got[5] == 448


@pytest.mark.parametrize("what,bit", [("page", moe.MOE_KV_BAD_PAGE), ("length", moe.MOE_KV_BAD_LENGTH),
                                      ("seq", moe.MOE_KV_BAD_SEQ)])
def test_refused_tokens_leave_the_cache_alone(what, bit):
    kp, vp = pool(3, 2, 16, 64, BF16, "hnd"), pool(3, 2, 16, 64, BF16, "hnd")
    k = torch.randn(2, 2, 64, device="cuda").to(BF16)
    table = torch.tensor([[1, 7 if what == "page" else 0], [2, -3]], dtype=torch.int32, device="cuda")
    pos = torch.tensor([3, 32 if what == "length" else 20], dtype=torch.int32, device="cuda")
    seq = torch.tensor([0, 2 if what == "seq" else 0], dtype=torch.int32, device="cuda")
    with moe.KVCache(kp, vp, n_heads=2) as kv:
        kv.append(None, k, k, pos, table, seq=seq)
        assert kv.health() == (6, bit)
        assert kv.health() == (0, 0)
    assert torch.equal(kp[1, :, 3], k[0])
    kp[1, :, 3], vp[1, :, 3] = 3.0, 3.0
    assert torch.all(kp == 3.0) and torch.all(vp == 3.0)


def test_on_another_stream():
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    run_case(40, 8, 2, 128, 32, stream=s, seed=12)


def test_binding_refuses_other_tensors():
    kp, vp = pool(3, 2, 16, 64, BF16, "hnd"), pool(3, 2, 16, 64, BF16, "hnd")
    k = torch.zeros(2, 2, 64, device="cuda", dtype=BF16)
    q = torch.zeros(2, 4, 64, device="cuda", dtype=BF16)
    pos = torch.zeros(2, dtype=torch.int32, device="cuda")
    table = torch.zeros(2, 2, dtype=torch.int32, device="cuda")
    with moe.KVCache(kp, vp, n_heads=4) as kv:
        good = dict(q=q, k=k, v=k, positions=pos, block_table=table, q_out=torch.empty_like(q))
        for bad in (dict(q=q[:, :2]), dict(k=k.float()), dict(v=k[:1]), dict(positions=pos.long()),
                    dict(block_table=table.cpu()), dict(q_out=torch.empty(2, 8, 64, device="cuda", dtype=BF16)[:, ::2]),
                    dict(k=k.transpose(1, 2).contiguous().transpose(1, 2)), dict(seq=pos[:1])):
            with pytest.raises(ValueError):
                kv.append(**{**good, **bad})
        with pytest.raises(moe.MoEError):
            kv.append(**{**good, "q": None})
    with pytest.raises(ValueError):
        moe.KVCache(kp, vp[:2], n_heads=4)
    with pytest.raises(ValueError):
        moe.KVCache(kp, vp.permute(0, 1, 3, 2), n_heads=4)
