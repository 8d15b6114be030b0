"""Block norm and paged attention from several host threads at a time, each with objects
and a stream of its own, first uses of the kernels among them."""
import threading

import pytest
import torch

import quantized_routed_expert_moe_gb300 as moe
from test_gpu_block_norm import make
from test_gpu_kv_attend import BF16, Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from quantized_routed_expert_moe_gb300 import build
    build.build()
    assert torch.cuda.is_available()


def test_threads_get_what_one_thread_gets():
    layouts = [(1, 6144), (3001, 64), (3001, 448), (1501, 2816), (701, 6144), (301, 12352)]
    norms = [make(T, H, res, gate="full", seed=H) for T, H in layouts for res in (torch.float32, BF16)]
    cases = [Case([700, 3, 90], 8, 2, D, 16, seed=D) for D in (64, 128, 256)]
    got, errors = {}, []
    start = threading.Barrier(4)

    def work(me):
        try:
            stream = torch.cuda.Stream()
            stream.wait_stream(torch.cuda.default_stream())
            start.wait()
            for n in range(3):
                for i, (x, o, ga, wp, wn, r, h) in enumerate(norms):
                    with torch.cuda.stream(stream):
                        r, h = torch.empty_like(r), torch.empty_like(h)
                    moe.BlockNorm(x.shape[1], wp, wn).run(x, o, r, h, gate=ga, stream=stream)
                    got[me, n, "norm", i] = (r, h)
                for i, c in enumerate(cases):
                    with c.handle() as kv, torch.cuda.stream(stream):
                        out = torch.empty_like(c.q)
                        table = c.table.cuda()
                        lens = torch.tensor(c.lens, dtype=torch.int32, device="cuda")
                        kv.attend(c.q, table, lens, out, stream=stream)
                        stream.synchronize()
                    got[me, n, "attend", i] = (out,)
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
    for i, (x, o, ga, wp, wn, r, h) in enumerate(norms):
        moe.BlockNorm(x.shape[1], wp, wn).run(x, o, r, h, gate=ga, stream=torch.cuda.current_stream())
    torch.cuda.synchronize()
    assert len(got) == 4 * 3 * (len(norms) + len(cases))
    for (me, n, kind, i), tensors in got.items():
        want = norms[i][5:] if kind == "norm" else got[0, 0, "attend", i]
        assert all(torch.equal(a, b) for a, b in zip(tensors, want)), (me, n, kind, i)
