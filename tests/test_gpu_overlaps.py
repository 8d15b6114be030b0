"""Outputs that lie on an input are refused; outputs beside one in the same buffer are not."""
import pytest
import torch

import quantized_routed_expert_moe_gb300 as moe
from _chunk_ref import linear
from _decoder_ref import assert_close, rounded
from test_gpu_kv_attend_chunk import BF16, Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from quantized_routed_expert_moe_gb300 import build
    build.build()
    assert torch.cuda.is_available()


@pytest.mark.parametrize("T", [3, 200])
def test_linear(T):
    w = torch.randn(64, 64, device="cuda").bfloat16()
    lin = moe.Linear(w)
    buf = torch.randn(T, 192, device="cuda").bfloat16()
    before = buf.clone()
    for x, y, r in ((buf[:, :64], buf[:, :64], None), (buf[:, :64], buf[:, 56:120], None),
                    (buf[:, :64], buf[:, 128:], buf[:, 120:184]), (buf[1:, :64], buf[:-1, :64], None)):
        with pytest.raises(moe.MoEError, match="overlap"):
            lin.run(x, y, residual=r)
    wide = torch.randn(264, 64, device="cuda").bfloat16()
    with pytest.raises(moe.MoEError, match="overlap"):
        moe.Linear(wide[:64]).run(buf[:, :64], wide[60:60 + T])   # on the weight's last rows
    torch.cuda.synchronize()
    assert torch.equal(buf, before)
    # columns of one buffer, and the residual in place
    lin.run(buf[:, :64], buf[:, 64:128])
    lin.run(buf[:, :64], buf[:, 128:], residual=buf[:, 128:])
    torch.cuda.synchronize()
    v, e = linear(before[:, :64], w, None, "none", None)
    assert_close(buf[:, 64:128], v, rounded(v, e, BF16), "beside")
    v, e = linear(before[:, :64], w, None, "none", before[:, 128:])
    assert_close(buf[:, 128:], v, rounded(v, e, BF16), "in place")


def test_chunk():
    c = Case([(40, 900), (3, 100)], 4, 2, 64, 16, seed=5)
    table, starts, lens = c.args()
    T = c.q.shape[0]
    with c.handle() as kv:
        n = kv.chunk_workspace_bytes
        ws = torch.zeros(n + 4096, dtype=torch.uint8, device="cuda")
        out = torch.empty_like(c.q)
        both = torch.randn(T, 2, 4, 64, device="cuda").bfloat16()
        inside = ws[-c.q.nbytes - 4096:-4096].view(BF16).view(c.q.shape)
        for q, o, kw in ((c.q, c.q, {}), (both[:, 0], both.view(-1)[256:256 + c.q.numel()].view(c.q.shape), {}),
                         (c.q, inside, {}), (inside, out, {}),
                         (c.q, out, dict(lse=out.view(-1)[:T * 8].view(torch.float32).view(T, 4)))):
            with pytest.raises(moe.MoEError, match="overlap"):
                kv.attend_chunk(q, starts, table, lens, o, workspace=ws, scale=c.scale, **kw)
        # queries beside the rest of a token's projections, and the workspace before something else
        c.q = both[:, 1]
        tail = ws[n:].view(torch.int32)[:2]
        tail.copy_(lens)
        kv.attend_chunk(c.q, starts, table, tail, out, workspace=ws, scale=c.scale)
        assert kv.health() == (0, 0)
    c.compare(out, None)
