"""The workspace that KVCache.attend_chunk makes at its first call: on the stream of that call."""
import pytest
import torch

from test_gpu_kv_attend_chunk import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from quantized_routed_expert_moe_gb300 import build
    build.build()
    assert torch.cuda.is_available()


def case():
    """A tile that is cut between many CTAs."""
    return Case([(40, 9000)], 6, 2, 128, 64, seed=17)


@pytest.mark.parametrize("handle", [False, True])
def test_memory_that_another_stream_still_uses_is_not_taken(handle):
    """A tensor of the workspace's size, freed while the current stream has work on it to do: the
    memory is the next allocation's there, and not that of a call on another stream."""
    c = case()
    side = torch.cuda.Stream()
    with c.handle() as kv:
        torch.cuda.synchronize()
        torch.cuda.empty_cache()
        old = torch.empty(kv.chunk_workspace_bytes, dtype=torch.uint8, device="cuda")
        at = old.data_ptr()
        torch.cuda._sleep(20_000_000)
        for _ in range(20):
            old.fill_(255)
        del old
        out, lse = torch.full(c.q.shape, 7.0, dtype=c.q.dtype, device="cuda"), torch.full(c.q.shape[:2], 7.0, device="cuda")
        table, starts, lens = c.args()
        torch.cuda._sleep(20_000_000)
        side.wait_stream(torch.cuda.current_stream())
        kv.attend_chunk(c.q, starts, table, lens, out, lse=lse, scale=c.scale, stream=side.cuda_stream if handle else side)
        new = kv._workspace
        assert new.data_ptr() + new.nbytes <= at or at + new.nbytes <= new.data_ptr()
        torch.cuda.synchronize()
        assert kv.health() == (0, 0)
        c.compare(out, lse)
        # and the same workspace on the current stream
        c.compare(*c.run(kv))
        assert kv._workspace is new


def test_the_workspace_of_the_current_stream():
    c = case()
    with c.handle() as kv:
        c.compare(*c.run(kv))
        assert kv._workspace.nbytes == kv.chunk_workspace_bytes


@pytest.mark.parametrize("captured", ["call", "current"])
def test_no_first_call_while_either_stream_is_captured(captured):
    """The stream of the call is captured and the current one is not, or the other way round."""
    c = case()
    table, starts, lens = c.args()
    out = torch.empty_like(c.q)
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    with c.handle() as kv:
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=a):
            if captured == "call":
                with torch.cuda.stream(b), pytest.raises(RuntimeError, match="workspace"):
                    kv.attend_chunk(c.q, starts, table, lens, out, stream=a)
            else:
                with pytest.raises(RuntimeError, match="workspace"):
                    kv.attend_chunk(c.q, starts, table, lens, out, stream=b)
            out.zero_()   # (a graph of nothing is not made)
        assert kv._workspace is None
        torch.cuda.synchronize()
        c.compare(*c.run(kv))
