"""moe_kv_attend on the GPU against attention in 64 bits."""
import numpy as np
import pytest
import torch

import quantized_routed_expert_moe_gb300 as moe
from _decoder_ref import assert_close, attend, f64, rounded

pytestmark = pytest.mark.gpu

BF16, E4M3 = torch.bfloat16, torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def built():
    from quantized_routed_expert_moe_gb300 import build
    build.build()
    assert torch.cuda.is_available()


class Case:
    """Caches whose unattended slots and unowned pages are NaN, shuffled pages,
    and table entries that no call may read as pages set out of range."""

    def __init__(self, lens, Hq, Hk, D, page, dt=BF16, layout="hnd", window=0, seed=0, extra_pages=1, sharp=1.5):
        g = torch.Generator("cuda").manual_seed(seed)
        rng = np.random.default_rng(seed)
        self.lens, self.window, self.dt = list(lens), window, dt
        B = len(self.lens)
        width = max(1, -(-max(self.lens) // page)) + extra_pages
        need = [-(-max(n, 0) // page) for n in self.lens]
        n_pages = sum(need) + 2
        order = rng.permutation(n_pages)
        table = rng.choice([-1, n_pages, 2 ** 31 - 1, -2 ** 31], size=(B, width)).astype(np.int32)
        shape = (n_pages, Hk, page, D) if layout == "hnd" else (n_pages, page, Hk, D)
        pools = []
        live = torch.zeros(n_pages, page, dtype=torch.bool)
        at = 0
        for b, n in enumerate(self.lens):
            lo = max(0, n - window) if window else 0
            for i in range(need[b]):
                if (i + 1) * page > lo:
                    table[b, i] = order[at + i]
                    live[order[at + i], max(0, lo - i * page):min(page, n - i * page)] = True
            at += need[b]
        for _ in range(2):
            x = torch.randn(shape, generator=g, device="cuda")
            if dt == E4M3:
                x = (x * 90).clamp(-448, 448)
            m = live.cuda()[:, None, :, None] if layout == "hnd" else live.cuda()[:, :, None, None]
            x = torch.where(m, x, torch.nan).to(dt)
            pools.append(x if layout == "hnd" else x.permute(0, 2, 1, 3))
        self.k, self.v = pools
        self.scales = (None, None) if dt == BF16 else (np.linspace(0.008, 0.015, Hk, dtype=np.float32),
                                                       np.linspace(0.02, 0.006, Hk, dtype=np.float32))
        self.table = torch.from_numpy(table)
        self.q = (torch.randn(B, Hq, D, generator=g, device="cuda") * sharp).to(BF16)
        self.scale = D ** -0.5

    def handle(self, max_batch=None):
        return moe.KVCache(self.k, self.v, n_heads=self.q.shape[1], k_scale=self.scales[0], v_scale=self.scales[1],
                           max_batch=max_batch or len(self.lens))

    def run(self, kv, softcap=0.0, with_lse=True, stream=None, q=None):
        q = self.q if q is None else q
        out = torch.full(self.q.shape, 7.0, dtype=BF16, device="cuda")
        lse = torch.full(self.q.shape[:2], 7.0, device="cuda") if with_lse else None
        table, lens = self.table.cuda(), torch.tensor(self.lens, dtype=torch.int32, device="cuda")
        if stream is not None:
            stream.wait_stream(torch.cuda.current_stream())
        kv.attend(q, table, lens, out, lse=lse, scale=self.scale, softcap=softcap, window=self.window, stream=stream)
        torch.cuda.synchronize()
        return out, lse

    def check(self, softcap=0.0, health=(0, 0), **kw):
        with self.handle() as kv:
            out, lse = self.run(kv, softcap, **kw)
            assert kv.health() == health
        vo, eo, vl, el = attend(self.q, self.k, self.v, self.table, self.lens, self.scale, softcap, self.window,
                                *self.scales)
        assert_close(out, vo, rounded(vo, eo, BF16), "out")
        if lse is not None:
            assert_close(lse, vl, el + 2.0 ** -24 * torch.nan_to_num(vl, neginf=0.0).abs(), "lse")
        return out, lse


LENGTHS = [0, 1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 257, 1000]


@pytest.mark.parametrize("dt", [BF16, E4M3])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("layout", ["hnd", "nhd"])
def test_lengths(D, dt, layout):
    Case(LENGTHS, 4, 2, D, 16, dt, layout, seed=D).check()


@pytest.mark.parametrize("dt", [BF16, E4M3])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("G", [1, 3, 6, 8, 9, 16, 17, 40])
def test_query_groups(G, D, dt):
    Case([77, 0, 300, 1], 2 * G, 2, D, 32, dt, seed=G).check()


@pytest.mark.parametrize("page", [16, 32, 48, 64, 80, 128, 256, 4096])
@pytest.mark.parametrize("dt", [BF16, E4M3])
def test_page_sizes(page, dt):
    Case([5, page - 1, page, page + 1, 3 * page + 7], 6, 3, 128, page, dt, "nhd" if page % 32 else "hnd",
         seed=page).check()


@pytest.mark.parametrize("window", [1, 2, 15, 16, 17, 64, 100, 129, 5000])
@pytest.mark.parametrize("D,dt", [(64, BF16), (128, E4M3), (256, BF16)])
def test_windows(window, D, dt):
    Case([0, 1, 16, 17, 100, 129, 700], 8, 2, D, 16, dt, window=window, seed=window).check()


@pytest.mark.parametrize("dt", [BF16, E4M3])
@pytest.mark.parametrize("cap", [0.5, 30.0])
def test_softcap(dt, cap):
    Case([1, 40, 513], 8, 2, 128, 16, dt, seed=4, sharp=6.0).check(softcap=cap)


@pytest.mark.parametrize("n,Hk,G,D,dt", [(20000, 1, 8, 128, BF16), (50001, 2, 4, 64, E4M3), (9999, 1, 1, 256, BF16),
                                         (131072, 1, 2, 128, E4M3), (4097, 8, 6, 128, BF16)])
def test_one_long_sequence(n, Hk, G, D, dt):
    Case([n], Hk * G, Hk, D, 64, dt, seed=7).check()


def test_one_long_among_many_short():
    lens = [3] * 40 + [30000] + [0] * 5 + [17] * 50 + [800] * 3
    Case(lens, 8, 4, 64, 16, seed=11).check()


@pytest.mark.parametrize("B", [1, 7, 129, 1024])
def test_batches(B):
    rng = np.random.default_rng(B)
    Case(rng.integers(0, 90, B).tolist() if B > 1 else [1], 2, 1, 64, 16, seed=B).check()


def test_all_empty():
    out, lse = Case([0, -5, 0], 4, 2, 64, 16).check()
    assert torch.all(out == 0) and torch.all(lse == -torch.inf)


def test_sharp_and_flat_scores():
    """One position takes all the weight; all positions alike; scores of +-1e4."""
    Case([500, 33], 8, 2, 128, 16, seed=3, sharp=100.0).check()
    Case([500, 33], 8, 2, 128, 16, seed=3, sharp=0.0).check()
    c = Case([500, 33], 8, 2, 128, 16, E4M3, seed=3, sharp=1.0)
    c.q *= 2.0 ** 10
    c.check()
    c.q *= 2.0 ** -60
    c.check()


@pytest.mark.parametrize("dt", [BF16, E4M3])
@pytest.mark.parametrize("scale,cap", [(0.0, 0.0), (-0.09, 0.0), (0.0, 5.0), (-0.2, 3.0)])
def test_scales_of_zero_and_below(scale, cap, dt):
    c = Case([1, 100, 77], 4, 2, 64, 16, dt, seed=13)
    c.scale = scale
    c.check(softcap=cap)


def test_strided_queries():
    c = Case([200, 31, 64], 8, 2, 64, 16, seed=5)
    wide = torch.full((3, 8 * 64 + 192), torch.nan, dtype=BF16, device="cuda")
    q = wide[:, 64:64 + 512].unflatten(1, (8, 64))
    q.copy_(c.q)
    with c.handle() as kv:
        a, la = c.run(kv, q=q)
        b, lb = c.run(kv)
    assert torch.equal(a, b) and torch.equal(la, lb)


def test_without_lse_and_repeated_bit_for_bit():
    c = Case([3000, 0, 77, 1], 16, 2, 128, 16, seed=6)
    with c.handle(max_batch=9) as kv:
        a, la = c.run(kv)
        for _ in range(5):
            b, lb = c.run(kv)
            assert torch.equal(a, b) and torch.equal(la, lb)
        b, _ = c.run(kv, with_lse=False)
        assert torch.equal(a, b)
        s = torch.cuda.Stream()
        b, lb = c.run(kv, stream=s)
        assert torch.equal(a, b) and torch.equal(la, lb)


def test_nan_and_infinity_of_live_slots_stay_in_their_head():
    c = Case([100, 100, 100], 4, 2, 64, 16, seed=8)
    with c.handle() as kv:
        clean, _ = c.run(kv)
        page = int(c.table[1, 2])
        c.k[page, 0, 5, 3] = torch.nan       # sequence 1, head 0
        c.v[int(c.table[2, 0]), 1, 0, 7] = torch.inf   # sequence 2, head 1, one channel
        out, lse = c.run(kv)
    want = torch.zeros(3, 4, 64, dtype=torch.bool, device="cuda")
    want[1, :2] = True
    assert torch.isnan(out[1, :2]).all() and torch.isnan(lse[1, :2]).all()
    assert torch.isinf(out[2, 2:, 7]).all()
    want[2, 2:, 7] = True
    assert torch.equal(out[~want], clean[~want])


@pytest.mark.parametrize("bad", [-1, 10 ** 6])
def test_bad_pages_are_skipped(bad):
    """A page id outside the pool inside the length: its tokens are left out."""
    c = Case([64, 40], 4, 2, 64, 16, seed=9)
    c.table[0, 1] = bad
    with c.handle() as kv:
        out, lse = c.run(kv)
        assert kv.health() == (6, moe.MOE_KV_BAD_PAGE)
        assert kv.health() == (0, 0)
    # the same as a shorter sequence over the other pages
    d = Case([48, 40], 4, 2, 64, 16, seed=9)
    d.k, d.v, d.q = c.k, c.v, c.q
    d.table = c.table.clone()
    d.table[0, 1:3] = c.table[0, 2:4]
    vo, eo, vl, el = attend(d.q, d.k, d.v, d.table, d.lens, d.scale)
    assert_close(out, vo, rounded(vo, eo, BF16), "out")
    assert_close(lse, vl, el + 2.0 ** -24 * vl.abs(), "lse")


def test_length_past_the_table_is_cut():
    c = Case([48, 20], 4, 2, 64, 16, seed=10, extra_pages=0)
    c.lens[0] = 2 ** 31 - 1
    with c.handle() as kv:
        out, lse = c.run(kv)
        assert kv.health() == (6, moe.MOE_KV_BAD_LENGTH)
    vo, eo, vl, el = attend(c.q, c.k, c.v, c.table, [48, 20], c.scale)
    assert_close(out, vo, rounded(vo, eo, BF16), "out")


def test_rows_past_32_bits_of_offset():
    """Pages beyond 2^32 bytes and 2^31 elements of a pool."""
    n_pages, page, D = 70000, 256, 128          # 2.3e9 elements per pool, one byte each
    k = torch.zeros(n_pages, 1, page, D, dtype=torch.uint8, device="cuda").view(E4M3)
    v = torch.zeros_like(k.view(torch.uint8)).view(E4M3)
    pages = [n_pages - 1, 0, 66000, 69999 - 7]
    x = torch.randn(2, 4, page, D, device="cuda", generator=torch.Generator("cuda").manual_seed(1)) * 50
    for i, p in enumerate(pages):
        k[p, 0], v[p, 0] = x[0, i].to(E4M3), x[1, i].to(E4M3)
    one = np.full(1, 0.02, np.float32)
    q = torch.randn(1, 4, D, device="cuda").to(BF16)
    table = torch.tensor([pages], dtype=torch.int32)
    out = torch.empty(1, 4, D, dtype=BF16, device="cuda")
    with moe.KVCache(k, v, n_heads=4, k_scale=one, v_scale=one) as kv:
        kv.attend(q, table.cuda(), torch.tensor([1000], dtype=torch.int32, device="cuda"), out)
        assert kv.health() == (0, 0)
    vo, eo, _, _ = attend(q, k, v, table, [1000], D ** -0.5, 0.0, 0, one, one)
    assert_close(out, vo, rounded(vo, eo, BF16), "out")


def test_captured_in_a_graph_with_lengths_that_grow():
    """One captured append and attention, replayed as a sequence grows: the
    lengths and positions are read on the device."""
    D, page, Hq, Hk = 64, 16, 4, 2
    g = torch.Generator("cuda").manual_seed(2)
    kp = torch.full((8, Hk, page, D), torch.nan, dtype=BF16, device="cuda")
    vp = torch.full_like(kp, torch.nan)
    table = torch.tensor([[5, 0, 7]], dtype=torch.int32, device="cuda")
    q, k, v = (torch.empty(1, n, D, dtype=BF16, device="cuda") for n in (Hq, Hk, Hk))
    pos, lens = (torch.zeros(1, dtype=torch.int32, device="cuda") for _ in range(2))
    qr, out = torch.empty_like(q), torch.empty_like(q)
    with moe.KVCache(kp, vp, n_heads=Hq, inv_freq=np.array([10000.0 ** (-i / 32) for i in range(32)])) as kv:
        kv.attend(q.zero_(), table, lens, out)     # first use outside the capture
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            s = torch.cuda.current_stream()
            kv.append(q, k, v, pos, table, qr, stream=s)
            kv.attend(qr, table, lens, out, stream=s)
        for t in range(40):
            for x in (q, k, v):
                x.copy_(torch.randn(x.shape, generator=g, device="cuda"))
            pos.fill_(t)
            lens.fill_(t + 1)
            graph.replay()
            if t in (0, 1, 15, 16, 39):
                torch.cuda.synchronize()
                vo, eo, _, _ = attend(qr, kp, vp, table.cpu(), [t + 1], D ** -0.5)
                assert_close(out, vo, rounded(vo, eo, BF16), f"token {t}")
        assert kv.health() == (0, 0)


def test_empty_batch_and_refusals():
    c = Case([5, 6], 4, 2, 64, 16)
    lens = torch.tensor(c.lens, dtype=torch.int32, device="cuda")
    out = torch.full((2, 4, 64), 7.0, dtype=BF16, device="cuda")
    with c.handle(max_batch=1) as kv:
        kv.attend(c.q[:0], c.table[:0].cuda(), lens[:0], out[:0])
        with pytest.raises(moe.MoEError) as ei:
            kv.attend(c.q, c.table.cuda(), lens, out)
        assert ei.value.status == 1
        for bad in (dict(q=c.q.float()), dict(lens=lens.long()), dict(out=out[:1]), dict(block_table=c.table),
                    dict(lse=torch.empty(2, 4, device="cuda", dtype=torch.float64))):
            with pytest.raises(ValueError):
                kv.attend(**{**dict(q=c.q, block_table=c.table.cuda(), lens=lens, out=out), **bad})
        torch.cuda.synchronize()
        assert kv.health() == (0, 0)
    assert torch.all(out == 7.0)
