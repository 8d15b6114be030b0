"""moe_kv_attend_chunk with more row tiles and more sequences than a CTA has threads."""
import numpy as np
import pytest
import torch

from _chunk_ref import attend_chunk
from _decoder_ref import assert_close, rounded
from test_gpu_kv_attend_chunk import BF16, E4M3, Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from quantized_routed_expert_moe_gb300 import build
    build.build()
    assert torch.cuda.is_available()


@pytest.mark.parametrize("dt", [BF16, E4M3])
@pytest.mark.parametrize("B,wide", [(513, 1), (1000, 1), (1024, 40)])
def test_many_sequences(B, wide, dt):
    """Whole tiles where the table is narrow, cut ones where it is wide; sequences without tokens
    at either end and in between."""
    rng = np.random.default_rng(B)
    new = rng.integers(0, 24, B)
    new[[0, 1, 512, B - 1]] = 0
    chunks = [(int(n), int(n + m)) for n, m in zip(new, rng.integers(0, 90, B))]
    Case(chunks, 16, 1, 64, 16, dt, seed=B, extra_pages=wide, before=1, after=2).check()


@pytest.mark.parametrize("D,dt,G", [(64, BF16, 16), (128, BF16, 17), (128, E4M3, 16), (256, BF16, 8)])
def test_many_tiles_of_one_sequence(D, dt, G):
    """From 512 tiles on the walk adds them up in turns. A window keeps the plain form small: it
    takes the same tokens by the hundred, each as a chunk that ends where it ends."""
    n, before, window = 9001, 700, 50
    c = Case([(3, 40), (n, n + before), (5, 5)], G, 1, D, 64, dt, window=window, seed=D)
    with c.handle() as kv:
        out, lse = c.run(kv)
        assert kv.health() == (0, 0)
        again, _ = c.run(kv)
    assert torch.equal(out, again)
    starts, lens, rows = [0, 3], [40], [0]
    for at in range(0, n, 200):
        step = min(200, n - at)
        starts.append(starts[-1] + step)
        lens.append(before + at + step)
        rows.append(1)
    starts.append(starts[-1] + 5)
    lens.append(5)
    rows.append(2)
    vo, eo, vl, el = attend_chunk(c.q, c.k, c.v, c.table[rows], starts, lens, c.scale, 0.0, window, *c.scales)
    assert_close(out, vo, rounded(vo, eo, BF16), "out")
    assert_close(lse, vl, el + 2.0 ** -24 * vl.abs(), "lse")
