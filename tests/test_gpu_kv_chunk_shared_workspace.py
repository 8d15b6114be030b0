"""Two calls of moe_kv_attend_chunk on one workspace at the same time, which the header rules out: what
they give is undefined, but each stays within its own rows (the join follows no record past them)."""
import pytest
import torch

from test_gpu_kv_attend_chunk import BF16, Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from quantized_routed_expert_moe_gb300 import build
    build.build()
    assert torch.cuda.is_available()


def test_no_row_outside_either_call_is_written():
    # many rows and few, both cut between CTAs
    cases = [Case([(700, 9000), (300, 4000)], 12, 2, 64, 64, seed=1), Case([(5, 30000)], 2, 1, 64, 64, seed=2)]
    kvs = [c.handle() for c in cases]
    ws = torch.zeros(max(kv.chunk_workspace_bytes for kv in kvs), dtype=torch.uint8, device="cuda")
    streams = [torch.cuda.Stream() for _ in cases]
    bufs, calls = [], []
    for c, kv in zip(cases, kvs):
        n = c.q.numel()
        room = torch.full((n + 2 * (1 << 20),), 7.0, dtype=BF16, device="cuda")
        bufs.append((room, n))
        calls.append((kv, c, *c.args(), room[1 << 20:(1 << 20) + n].view(c.q.shape)))
    torch.cuda.synchronize()
    for _ in range(40):
        for s, (kv, c, table, starts, lens, out) in zip(streams, calls):
            kv.attend_chunk(c.q, starts, table, lens, out, scale=c.scale, workspace=ws, stream=s)
    torch.cuda.synchronize()
    for room, n in bufs:
        assert (room[:1 << 20] == 7.0).all() and (room[(1 << 20) + n:] == 7.0).all()
    # one after the other they give what they should
    for c, kv in zip(cases, kvs):
        assert kv.health() == (0, 0)
        c.compare(*c.run(kv, workspace=ws))
        kv.close()
