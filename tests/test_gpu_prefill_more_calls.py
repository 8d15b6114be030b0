"""Calls of the operators of a prompt's chunk that the other files do not make: first calls inside a
capture, several host threads, every order of a pool, many queries to a key-value head."""
import itertools
import os
import subprocess
import sys
import threading

import numpy as np
import pytest
import torch

import quantized_routed_expert_moe_gb300 as moe
from conftest import ROOT
from test_gpu_kv_attend_chunk import BF16, E4M3, Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from quantized_routed_expert_moe_gb300 import build
    build.build()
    assert torch.cuda.is_available()


FIRST_IN_A_CAPTURE = """
import numpy as np, torch
import quantized_routed_expert_moe_gb300 as moe
torch.manual_seed(0)
x, w = torch.randn(40, 512, device="cuda").bfloat16(), torch.randn(768, 512, device="cuda").bfloat16()
pools = torch.zeros(2, 4, 2, 16, 64, dtype=torch.bfloat16, device="cuda")
kv = moe.KVCache(pools[0], pools[1], n_heads=8, inv_freq=np.ones(32))
lin = moe.Linear(w)
ws = torch.empty(kv.chunk_workspace_bytes, dtype=torch.uint8, device="cuda")
one = torch.ones(64, device="cuda")
pos = torch.arange(40, dtype=torch.int32, device="cuda")
table = torch.arange(4, dtype=torch.int32, device="cuda")[None]
starts, lens = (torch.tensor(a, dtype=torch.int32, device="cuda") for a in ([0, 40], [40]))
qkv, seq = torch.empty(40, 768, dtype=torch.bfloat16, device="cuda"), torch.zeros_like(pos)
q_rot, out = (torch.empty(40, 8, 64, dtype=torch.bfloat16, device="cuda") for _ in range(2))
wide = torch.zeros(1, 64, dtype=torch.int32, device="cuda")   # more than four blocks: two launches
wide[:, :4] = table
def step():
    lin.run(x, qkv)
    q, k, v = qkv.view(40, -1, 64).split([8, 2, 2], 1)
    kv.append(q, k, v, pos, table, q_rot, seq=seq, q_norm=one, k_norm=one)
    kv.attend_chunk(q_rot, starts, wide, lens, out, workspace=ws)
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    step()
g.replay()
torch.cuda.synchronize()
got = out.clone()
assert kv.health() == (0, 0)
step()
torch.cuda.synchronize()
assert torch.equal(got, out) and torch.isfinite(got.float()).all() and got.any()
"""


def test_first_calls_of_a_process_inside_a_capture():
    r = subprocess.run([sys.executable, "-c", FIRST_IN_A_CAPTURE], cwd=ROOT, env=dict(os.environ, PYTHONPATH=ROOT),
                       capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stderr[-2000:]


def test_threads_get_what_one_thread_gets():
    """Each with objects and a stream of its own."""
    cases = [Case([(40, 900), (3, 100), (200, 200)], 6, 2, D, 64, dt, seed=D) for D, dt in ((64, BF16), (128, E4M3), (256, BF16))]
    g = torch.Generator("cuda").manual_seed(0)
    sizes = [(1, 512, 768), (1, 2816, 1032), (60, 512, 768), (300, 136, 264), (3000, 512, 1288)]
    mats = [(torch.randn(T, K, generator=g, device="cuda").bfloat16(), torch.randn(N, K, generator=g, device="cuda").bfloat16())
            for T, K, N in sizes]
    got, errors, start = {}, [], threading.Barrier(4)

    def work(me):
        try:
            stream = torch.cuda.Stream()
            stream.wait_stream(torch.cuda.default_stream())
            start.wait()
            with torch.cuda.stream(stream):
                for n in range(3):
                    for i, (x, w) in enumerate(mats):
                        for dt in (BF16, torch.float32):
                            y = torch.empty(x.shape[0], w.shape[0], dtype=dt, device="cuda")
                            moe.Linear(w).run(x, y)
                            got[me, n, "linear", i, dt] = (y,)
                    for i, c in enumerate(cases):
                        with c.handle() as kv:
                            out, lse = torch.empty_like(c.q), torch.empty(c.q.shape[:2], device="cuda")
                            table, starts, lens = c.args()
                            kv.attend_chunk(c.q, starts, table, lens, out, lse=lse, scale=c.scale)
                            stream.synchronize()
                        got[me, n, "chunk", i, None] = (out, lse)
                stream.synchronize()
        except Exception as e:  # noqa: BLE001 - reported by the test's thread
            errors.append(e)

    torch.cuda.synchronize()
    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors
    torch.cuda.synchronize()
    for (me, n, *key), values in got.items():
        assert all(torch.equal(a, b) for a, b in zip(values, got[0, 0, *key])), (me, n, key)
    for i, c in enumerate(cases):
        c.compare(*got[0, 0, "chunk", i, None])


@pytest.mark.parametrize("dt", [BF16, E4M3])
@pytest.mark.parametrize("sizes", [(7, 3, 48), (1, 3, 128), (9, 1, 16), (1, 1, 128)])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_every_order_of_a_pool(D, sizes, dt):
    pages, Hk, page = sizes
    n, new = min(pages * page, 130) - 3, 21
    k, v = (torch.randn(n, Hk, D, generator=torch.Generator("cuda").manual_seed(i), device="cuda").to(BF16) for i in (1, 2))
    q = torch.randn(new, 4 * Hk, D, device="cuda").to(BF16)
    table = torch.randperm(pages, generator=torch.Generator().manual_seed(3))[:-(-n // page)].to(torch.int32)[None].cuda()
    pos = torch.arange(n, dtype=torch.int32, device="cuda")
    starts, lens = (torch.tensor(a, dtype=torch.int32, device="cuda") for a in ([0, new], [n]))
    scale = None if dt is BF16 else np.full(Hk, 0.01, np.float32)
    one, first = torch.ones(D, device="cuda"), None
    for order in itertools.permutations(range(3)):
        back = [order.index(i) for i in range(3)]
        pools = [torch.zeros([sizes[i] for i in order] + [D], device="cuda", dtype=BF16).to(dt).permute(*back, 3)
                 for _ in range(2)]
        out, lse = torch.empty_like(q), torch.empty(new, 4 * Hk, device="cuda")
        with moe.KVCache(*pools, n_heads=4 * Hk, k_scale=scale, v_scale=scale,
                         inv_freq=np.array([10000.0 ** (-i / 16) for i in range(16)])) as kv:
            kv.append(None, k, v, pos, table, seq=torch.zeros_like(pos), k_norm=one)
            kv.attend_chunk(q, starts, table, lens, out, lse=lse)
            assert kv.health() == (0, 0)
        got = [p.float() for p in pools] + [out, lse]
        first = first or got
        assert all(torch.equal(a, b) for a, b in zip(got, first)), order
    assert torch.isfinite(first[2].float()).all() and first[2].any()


@pytest.mark.parametrize("D,dt,G", [(64, BF16, 300), (128, BF16, 257), (256, BF16, 300), (128, E4M3, 512), (64, E4M3, 1000)])
def test_a_token_of_several_tiles(D, dt, G):
    Case([(1, 1), (3, 40), (2, 1000), (0, 9)], G, 1, D, 32, dt, seed=G).check()
    Case([(2, 7), (1, 600)], 2 * G, 2, D, 16, dt, window=5, seed=G).check()


def test_sequences_that_share_pages():
    """Several sequences over the same pages, as after a common prompt."""
    c = Case([(5, 300), (5, 300), (9, 290), (1, 300)], 8, 2, 128, 16, seed=5)
    c.table[1:] = c.table[0]
    c.check()
