"""moe_kv_attend_chunk on the GPU against attention in 64 bits."""
import numpy as np
import pytest
import torch

import quantized_routed_expert_moe_gb300 as moe
from _chunk_ref import attend_chunk
from _decoder_ref import assert_close, rounded

pytestmark = pytest.mark.gpu

BF16, E4M3 = torch.bfloat16, torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def built():
    from quantized_routed_expert_moe_gb300 import build
    build.build()
    assert torch.cuda.is_available()


class Case:
    """Chunks (new tokens, cached tokens) over caches whose unattended slots and unowned pages
    are NaN, with shuffled pages and table entries out of range where no call may read them.
    `before` and `after` rows of q and out belong to no sequence."""

    def __init__(self, chunks, Hq, Hk, D, page, dt=BF16, layout="hnd", window=0, seed=0, sharp=1.5, extra_pages=1,
                 before=0, after=0, room=0):
        g = torch.Generator("cuda").manual_seed(seed)
        rng = np.random.default_rng(seed)
        self.new, self.lens = [n for n, _ in chunks], [m for _, m in chunks]
        self.window, self.dt, B = window, dt, len(chunks)
        self.starts = [before + sum(self.new[:b]) for b in range(B + 1)]
        T = self.starts[-1] + after
        width = max(1, -(-max(self.lens) // page)) + extra_pages
        need = [-(-max(n, 0) // page) for n in self.lens]
        n_pages = sum(need) + 2
        order = rng.permutation(n_pages)
        table = rng.choice([-1, n_pages, 2 ** 31 - 1, -2 ** 31], size=(B, width)).astype(np.int32)
        live = torch.zeros(n_pages, page, dtype=torch.bool)
        at = 0
        for b, (n, total) in enumerate(chunks):
            lo = max(0, total - n + 1 - window) if window else 0
            for i in range(need[b] if n else 0):
                if (i + 1) * page > lo:
                    table[b, i] = order[at + i]
                    live[order[at + i], max(0, lo - i * page):min(page, total - i * page)] = True
            at += need[b]
        shape = (n_pages, Hk, page, D) if layout == "hnd" else (n_pages, page, Hk, D)
        pools = []
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
        q = (torch.randn(T, Hq * D + room, generator=g, device="cuda") * sharp).to(BF16)
        self.q = q[:, :Hq * D].unflatten(1, (Hq, D))
        self.scale = D ** -0.5

    def handle(self, max_batch=None):
        return moe.KVCache(self.k, self.v, n_heads=self.q.shape[1], k_scale=self.scales[0], v_scale=self.scales[1],
                           max_batch=max_batch or len(self.lens))

    def args(self):
        return (self.table.cuda(), torch.tensor(self.starts, dtype=torch.int32, device="cuda"),
                torch.tensor(self.lens, dtype=torch.int32, device="cuda"))

    def run(self, kv, softcap=0.0, with_lse=True, stream=None, workspace=None):
        out = torch.full(self.q.shape, 7.0, dtype=BF16, device="cuda")
        lse = torch.full(self.q.shape[:2], 7.0, device="cuda") if with_lse else None
        table, starts, lens = self.args()
        if stream is not None:
            stream.wait_stream(torch.cuda.current_stream())
        kv.attend_chunk(self.q, starts, table, lens, out, lse=lse, scale=self.scale, softcap=softcap,
                        window=self.window, stream=stream, workspace=workspace)
        torch.cuda.synchronize()
        return out, lse

    def want(self, softcap=0.0):
        return attend_chunk(self.q, self.k, self.v, self.table, self.starts, self.lens, self.scale, softcap,
                            self.window, *self.scales)

    def compare(self, out, lse, softcap=0.0):
        vo, eo, vl, el = self.want(softcap)
        rows = slice(self.starts[0], self.starts[-1])
        assert_close(out[rows], vo[rows], rounded(vo, eo, BF16)[rows], "out")
        others = torch.ones(out.shape[0], dtype=torch.bool)
        others[rows] = False
        assert (out.cpu()[others] == 7.0).all(), "rows of no sequence changed"
        if lse is not None:
            assert_close(lse[rows], vl[rows], (el + 2.0 ** -24 * torch.nan_to_num(vl, neginf=0.0).abs())[rows], "lse")
            assert (lse.cpu()[others] == 7.0).all()

    def check(self, softcap=0.0, health=(0, 0), **kw):
        with self.handle() as kv:
            out, lse = self.run(kv, softcap, **kw)
            assert kv.health() == health
        self.compare(out, lse, softcap)
        return out, lse


FEW = [(1, 1), (2, 2), (3, 17), (0, 40), (16, 16), (17, 33), (1, 130), (5, 127), (7, 128), (4, 129)]


@pytest.mark.parametrize("dt", [BF16, E4M3])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("layout", ["hnd", "nhd"])
def test_few_tokens(D, dt, layout):
    Case(FEW, 4, 2, D, 16, dt, layout, seed=D).check()


@pytest.mark.parametrize("dt", [BF16, E4M3])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("chunks", [[(127, 127)], [(128, 128), (129, 129)], [(255, 255), (1, 300)], [(256, 257)],
                                    [(300, 300), (61, 400), (130, 1000)], [(513, 900)]])
def test_longer_chunks(chunks, D, dt):
    Case(chunks, 2, 2, D, 64, dt, seed=len(chunks)).check()


@pytest.mark.parametrize("dt", [BF16, E4M3])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("G", [1, 3, 5, 6, 8, 12, 16, 17, 40, 130])
def test_query_groups(G, D, dt):
    Case([(33, 77), (0, 5), (20, 300), (1, 1)], 2 * G, 2, D, 32, dt, seed=G).check()


@pytest.mark.parametrize("page", [16, 32, 48, 64, 80, 96, 128, 256, 4096])
@pytest.mark.parametrize("dt", [BF16, E4M3])
@pytest.mark.parametrize("D", [128, 256])
def test_page_sizes(page, dt, D):
    Case([(5, 5), (3, page - 1), (page % 100, page), (9, page + 1), (70, 3 * page + 77)], 6, 3, D, page, dt,
         "nhd" if page % 32 else "hnd", seed=page).check()


@pytest.mark.parametrize("window", [1, 2, 15, 16, 17, 64, 100, 128, 129, 5000])
@pytest.mark.parametrize("D,dt", [(64, BF16), (128, E4M3), (128, BF16), (256, BF16), (256, E4M3)])
def test_windows(window, D, dt):
    Case([(1, 1), (16, 16), (17, 100), (100, 129), (130, 700), (3, 1000)], 8, 2, D, 16, dt, window=window,
         seed=window).check()


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("dt", [BF16, E4M3])
@pytest.mark.parametrize("cap", [0.5, 30.0])
def test_softcap(dt, cap, D):
    Case([(1, 1), (40, 40), (150, 513)], 8, 2, D, 16, dt, seed=4, sharp=6.0).check(softcap=cap)


@pytest.mark.parametrize("dt", [BF16, E4M3])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("n,far", [(1, 20000), (16, 9000), (130, 5000)])
def test_long_context_is_split(n, far, D, dt):
    """One sequence: its blocks go to many CTAs and are joined."""
    Case([(n, far)], 6, 1, D, 64, dt, seed=n).check()


@pytest.mark.parametrize("dt", [BF16, E4M3])
def test_many_sequences(dt):
    rng = np.random.default_rng(3)
    chunks = [(int(n), int(n + m)) for n, m in zip(rng.integers(0, 40, 300), rng.integers(0, 400, 300))]
    Case(chunks, 4, 1, 64, 16, dt, seed=9).check()


@pytest.mark.parametrize("D,dt", [(64, BF16), (128, BF16), (128, E4M3), (256, BF16)])
def test_whole_prompts(D, dt):
    """Nothing cached before, lengths of their own, more tiles than SMs."""
    Case([(700, 700), (1, 1), (1500, 1500), (333, 333)], 12, 4, D, 64, dt, seed=D).check()


def test_rows_of_no_sequence_stay():
    Case([(5, 9), (0, 3), (4, 4)], 4, 2, 64, 16, before=3, after=6, seed=1).check()


def test_padded_queries():
    Case([(5, 9), (40, 40)], 4, 2, 128, 16, room=72, seed=2).check()


def test_without_lse():
    Case([(5, 9), (40, 40)], 4, 2, 128, 16, seed=2).check(with_lse=False)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("dt", [BF16, E4M3])
def test_chunk_longer_than_its_sequence(D, dt):
    """Tokens at negative positions see nothing: zeros and -inf."""
    Case([(9, 4), (5, 0), (3, -7), (200, 130)], 4, 2, D, 16, dt, seed=3).check()


def test_later_values_that_are_not_finite():
    """A value only later tokens of the chunk (or those whose window still holds it) attend to
    changes the others' result by nothing."""
    for D, dt, window, at in ((128, BF16, 0, (300, 350, 399)), (64, BF16, 40, (305, 340)), (256, BF16, 0, (310,)),
                              (128, E4M3, 33, (290, 333)), (256, E4M3, 0, (399,))):
        c = Case([(10, 30), (130, 400), (5, 50)], 6, 2, D, 16, dt, window=window, seed=at[0])
        pool = c.v.view(torch.uint8) if dt == E4M3 else c.v
        for i, p in enumerate(at):
            page, slot = int(c.table[1, p // 16]), p % 16
            bad = 0x7f if dt == E4M3 else (torch.inf, -torch.inf, torch.nan)[i % 3]
            pool[page, 0, slot, 3 + i] = bad
            pool[page, 1, slot, D - 1 - i] = bad
        c.check()


@pytest.mark.parametrize("window", [0, 40, 200])
@pytest.mark.parametrize("D,dt", [(64, BF16), (128, BF16), (256, BF16), (64, E4M3), (128, E4M3), (256, E4M3)])
def test_values_that_are_not_finite_on_either_side_of_groups(D, dt, window):
    """The same at the ends of groups of 16 positions, of which some are seen by all rows of a tile,
    some by a part of them and some by none, and with pages that end inside them."""
    c = Case([(130, 400), (17, 33)], 6, 2, D, 48, dt, window=window, seed=D + window)
    pool = c.v.view(torch.uint8) if dt == E4M3 else c.v
    for i, p in enumerate((255, 256, 271, 272, 287, 288, 303, 319, 320, 335, 336, 352, 383, 384, 399)):
        page, slot = int(c.table[0, p // 48]), p % 48
        if window and p <= 400 - 130 - window:
            continue   # no token sees it, its page may be none
        pool[page, i % 2, slot, (7 * i) % D] = 0x7f if dt == E4M3 else (torch.inf, -torch.inf, torch.nan)[i % 3]
    c.check()


def test_later_keys_that_are_not_finite():
    for D, dt in ((128, BF16), (256, BF16), (64, E4M3)):
        c = Case([(10, 30), (130, 400)], 6, 2, D, 16, dt, seed=D)
        page, slot = int(c.table[1, 399 // 16]), 399 % 16
        (c.k.view(torch.uint8) if dt == E4M3 else c.k)[page, :, slot] = 0x7f if dt == E4M3 else torch.nan
        with c.handle() as kv:
            out, lse = c.run(kv)
        assert torch.isnan(out[139].float()).all() and torch.isnan(lse[139]).all()   # the one token that sees it
        vo, eo, vl, el = c.want()
        assert_close(out[:139], vo[:139], rounded(vo, eo, BF16)[:139], "out")
        assert_close(lse[:139], vl[:139], el[:139] + 2.0 ** -24 * vl[:139].abs(), "lse")


@pytest.mark.parametrize("scale", [0.0, -0.2, 1e-30, 30.0])
def test_scales(scale):
    c = Case([(70, 200), (3, 3)], 4, 2, 64, 16, seed=8)
    c.scale = scale
    c.check()


@pytest.mark.parametrize("dt,D", [(BF16, 128), (BF16, 256), (E4M3, 128)])
@pytest.mark.parametrize("scale", [0.0, 2.0 ** -104, -2.0 ** -107])
def test_small_scales_of_large_products(dt, D, scale):
    """Products of 2^100 and more: a scale that is as small still counts by its value."""
    c = Case([(70, 200), (3, 3), (1, 40)], 4, 2, D, 16, dt, seed=9)
    c.q = c.q * 2.0 ** (60 if dt == BF16 else 100)
    if dt == BF16:
        c.k = c.k * 2.0 ** 40
    c.scale = scale
    c.check()


@pytest.mark.parametrize("dt", [BF16, E4M3])
def test_large_scores(dt):
    """Scores of 10^8 and more: all weight on the largest, no NaN and no zero."""
    c = Case([(70, 500), (1, 7)], 4, 2, 128, 16, dt, seed=12, sharp=64.0)
    c.scale = 2.0 ** 26
    with c.handle() as kv:
        out, lse = c.run(kv)
        assert kv.health() == (0, 0)
    assert torch.isfinite(out.float()).all() and torch.isfinite(lse).all()
    _, _, vl, _ = c.want()
    assert float(((lse.cpu().double() - vl) / vl).abs().max()) < 2.0 ** -15
    q, v = c.q.double().cpu(), c.v
    # the row of the largest score, where it stands out
    for t in (0, 69, 70):
        b = 0 if t < 70 else 1
        pos = c.lens[b] - (c.starts[b + 1] - t)
        from _decoder_ref import gather
        for h in range(4):
            k = gather(c.k, c.table, b, 0, pos + 1, h // 2)
            s = torch.sort(k @ q[t, h], descending=True)
            if len(s.values) > 1 and float(s.values[0] - s.values[1]) < 1e-2 * float(s.values[0].abs()):
                continue
            want = gather(v, c.table, b, 0, pos + 1, h // 2)[s.indices[0]] * (1.0 if c.scales[1] is None else float(c.scales[1][h // 2]))
            got = out[t, h].cpu().double()
            assert float((got - want).abs().max()) <= 2.0 ** -7 * float(want.abs().max())


def test_bad_pages_and_lengths():
    """An attended page outside the pool is skipped, a length past the table is cut; both are told."""
    for D, dt in ((64, BF16), (128, BF16), (128, E4M3), (256, BF16)):
        c = Case([(3, 100), (140, 150)], 4, 2, D, 16, dt, seed=5, extra_pages=0)
        table = c.table.clone()
        for b, page in ((0, 2), (1, 0), (1, 9)):
            c.table[b, page] = 10 ** 6
        with c.handle() as kv:
            out, lse = c.run(kv)
            assert kv.health() == (6, moe.MOE_KV_BAD_PAGE)
            assert kv.health() == (0, 0)
        # the same tokens without those positions: keys of -inf scores are as good as absent
        q = c.q.double().cpu()
        from _decoder_ref import gather
        for t in (0, 2, 3, 60, 142):
            b = 0 if t < 3 else 1
            pos = c.lens[b] - (c.starts[b + 1] - t)
            j = torch.arange(pos + 1)
            keep = torch.ones(pos + 1, dtype=torch.bool)
            for bb, page in ((0, 2), (1, 0), (1, 9)):
                if bb == b:
                    keep &= j // 16 != page
            for h in (0, 3):
                sc = [1.0 if x is None else float(x[h // 2]) for x in c.scales]
                k, v = (gather(x, table, b, 0, pos + 1, h // 2)[keep] * f for x, f in zip((c.k, c.v), sc))
                if not keep.any():
                    assert (out[t, h] == 0).all() and lse[t, h] == -torch.inf
                    continue
                p = torch.softmax(k @ q[t, h] * c.scale, 0)
                assert float((out[t, h].cpu().double() - p @ v).abs().max()) <= 2.0 ** -6 * float(v.abs().max())
        c.table = table
        c.lens[1] = 16 * table.shape[1] + 5
        with c.handle() as kv:
            c.run(kv)
            assert kv.health()[1] & moe.MOE_KV_BAD_LENGTH


@pytest.mark.parametrize("starts", [[0, 5, 3, 9], [-1, 2, 3, 9], [0, 2, 3, 10], [4, 2, 1, 0]])
def test_bad_starts(starts):
    c = Case([(3, 10), (3, 10), (3, 10)], 4, 2, 64, 16, seed=6)
    c.starts = starts
    with c.handle() as kv:
        out, lse = c.run(kv)
        assert kv.health() == (6, moe.MOE_KV_BAD_START)
    assert (out == 7.0).all() and (lse == 7.0).all()


def test_no_tokens():
    c = Case([(0, 10), (0, 0)], 4, 2, 64, 16, seed=6)
    with c.handle() as kv:
        c.run(kv)
        kv.attend_chunk(c.q[:0], torch.zeros(1, dtype=torch.int32, device="cuda"), c.table[:0].cuda(),
                        torch.zeros(0, dtype=torch.int32, device="cuda"), c.q[:0].contiguous())
        torch.cuda.synchronize()
        assert kv.health() == (0, 0)


def test_same_bits_every_time():
    for D, dt in ((128, BF16), (128, E4M3), (256, BF16)):
        c = Case([(40, 9000), (3, 100), (200, 200)], 6, 1, D, 64, dt, seed=7)
        with c.handle() as kv:
            first = c.run(kv)
            for _ in range(5):
                again = c.run(kv)
                assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


def test_one_token_agrees_with_attend():
    """A chunk of one token is what attend gives, up to the weights' rounding."""
    c = Case([(1, 77), (1, 1), (1, 3000)], 8, 2, 128, 16, seed=3)
    with c.handle() as kv:
        out, lse = c.run(kv)
        o1, l1 = torch.empty_like(out), torch.empty_like(lse)
        table, _, lens = c.args()
        kv.attend(c.q.contiguous(), table, lens, o1, lse=l1, scale=c.scale)
        torch.cuda.synchronize()
    assert float((l1 - lse).abs().max()) <= 1e-5
    assert float((o1.float() - out.float()).abs().max()) <= 2.0 ** -7 * float(o1.float().abs().max())


def test_stream_workspace_and_graph():
    c = Case([(40, 900), (3, 100), (200, 200)], 6, 2, 128, 64, seed=17)
    with c.handle() as kv:
        ws = torch.full((kv.chunk_workspace_bytes,), 255, dtype=torch.uint8, device="cuda")
        c.compare(*c.run(kv, stream=torch.cuda.Stream(), workspace=ws))
        table, starts, lens = c.args()
        out, lse = torch.full_like(c.q, 7.0), torch.full(c.q.shape[:2], 7.0, device="cuda")
        with pytest.raises(RuntimeError):   # no workspace yet, none given
            with torch.cuda.graph(torch.cuda.CUDAGraph()):
                kv.attend_chunk(c.q, starts, table, lens, out)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            for _ in range(2):
                kv.attend_chunk(c.q, starts, table, lens, out, lse=lse, scale=c.scale, workspace=ws)
        g.replay()
        torch.cuda.synchronize()
        c.compare(out, lse)
        # the lengths are read when the graph runs
        lens.copy_(torch.tensor([39, 50, 200], dtype=torch.int32))
        c.lens = [39, 50, 200]
        g.replay()
        torch.cuda.synchronize()
        c.compare(out, lse)
        with pytest.raises(moe.MoEError):
            kv.attend_chunk(c.q, starts, table, lens, out, workspace=ws[:-16])
        assert kv.health() == (0, 0)


def test_handles_share_a_workspace():
    a, b = Case([(40, 5000)], 6, 2, 128, 64, seed=1), Case([(90, 700), (4, 4)], 4, 2, 128, 32, E4M3, seed=2)
    with a.handle() as ka, b.handle() as kb:
        ws = torch.empty(max(ka.chunk_workspace_bytes, kb.chunk_workspace_bytes), dtype=torch.uint8, device="cuda")
        for _ in range(3):
            a.compare(*a.run(ka, workspace=ws))
            b.compare(*b.run(kb, workspace=ws))


def test_far_pages():
    """Pages past 2^31 elements into the pool."""
    D, Hk, page = 128, 2, 16
    n_pages = (2 ** 31 + 2 ** 24) // (Hk * page * D)
    k = torch.zeros(n_pages, Hk, page, D, dtype=BF16, device="cuda")
    v = torch.zeros_like(k)
    c = Case([(20, 60)], 4, Hk, D, page, seed=3)
    table = c.table.clone()
    for i in range(4):
        p = n_pages - 1 - i
        k[p], v[p] = c.k[int(table[0, i])], c.v[int(table[0, i])]
        table[0, i] = p
    want = c.want()
    c.k, c.v, c.table = k, v, table
    with c.handle() as kv:
        out, lse = c.run(kv)
        assert kv.health() == (0, 0)
    assert_close(out, want[0], rounded(want[0], want[1], BF16), "out")
