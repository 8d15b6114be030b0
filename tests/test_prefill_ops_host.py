"""Projections, head norms and chunk attention without a GPU: refusals of bad arguments."""
import ctypes

import pytest
import torch

import quantized_routed_expert_moe_gb300 as moe
from test_decoder_ops_host import P, append_args, kv_desc, refused


@pytest.fixture(scope="module", autouse=True)
def built():
    from quantized_routed_expert_moe_gb300 import build
    build.build()


def linear_desc(**kw):
    d = dict(abi_version=moe.MOE_ABI_VERSION, in_features=64, out_features=128, out_dtype=moe.MOE_BF16,
             activation=moe.MOE_ACT_NONE, x_stride=64, w_stride=64, y_stride=128, residual_stride=128)
    d.update(kw)
    return moe.moe_linear_desc(**d)


def chunk_args(**kw):
    a = dict(q=P, q_stride=512, starts=P, block_table=P, lens=P, T=7, B=4, max_pages=5, scale=0.1, softcap=0.0,
             window=0, out=P, lse=None, workspace=P, workspace_bytes=1 << 30)
    a.update(kw)
    return moe.moe_kv_chunk_args(**a)


def head_norm(**kw):
    a = dict(q_weight=P, k_weight=P, eps=1e-6, weight_offset=0.0)
    a.update(kw)
    return moe.moe_kv_head_norm(**a)


def test_packed_structures_match_the_ctypes_ones():
    for packed, c in ((moe.Linear._desc, moe.moe_linear_desc), (moe.KVCache._chunk_args, moe.moe_kv_chunk_args),
                      (moe.KVCache._head_norm, moe.moe_kv_head_norm)):
        assert len(packed.unpack(bytes(packed.size))) == len(c._fields_)
        buf = bytearray(ctypes.sizeof(c))
        packed.pack_into(buf, 0, *range(1, len(c._fields_) + 1))
        got = c.from_buffer(buf)
        assert [getattr(got, n) for n, _ in c._fields_] == list(range(1, len(c._fields_) + 1))


def test_good_arguments_pass():
    moe.moe_linear_check(linear_desc(), P, P, None, None, P, 3)
    moe.moe_linear_check(linear_desc(), P, P, P, P, P, 3)
    moe.moe_linear_check(linear_desc(), None, None, None, None, None, 0)
    moe.moe_linear_check(linear_desc(out_dtype=moe.MOE_F32, y_stride=132), P, P, None, None, P, 1 << 24)
    moe.moe_kv_attend_chunk_check(kv_desc(), chunk_args())
    moe.moe_kv_attend_chunk_check(kv_desc(), chunk_args(B=0, q=None, starts=None, workspace=None))
    moe.moe_kv_attend_chunk_check(kv_desc(), chunk_args(T=0, q=None, starts=None, workspace=None))
    moe.moe_kv_append_norm_check(kv_desc(), append_args(), head_norm())
    moe.moe_kv_append_norm_check(kv_desc(), append_args(), head_norm(q_weight=None, k_weight=None))


@pytest.mark.parametrize("kw,status", [
    (dict(abi_version=2), 1), (dict(in_features=0), 1), (dict(in_features=60), 1), (dict(out_features=12), 1),
    (dict(out_features=-8), 1), (dict(in_features=(1 << 20) + 8, x_stride=1 << 21, w_stride=1 << 21), 2),
    (dict(out_dtype=moe.MOE_E4M3), 1), (dict(activation=4), 1), (dict(activation=-1), 1), (dict(x_stride=56), 1),
    (dict(x_stride=68), 1), (dict(w_stride=0), 1), (dict(y_stride=120), 1), (dict(y_stride=132), 1),
    (dict(residual_stride=64), 1), (dict(x_stride=(1 << 38) + 8), 1)])
def test_linear_descriptors_are_refused(kw, status):
    refused(moe.moe_linear_check, linear_desc(**kw), P, P, P, P, P + 16, 3, status=status)


def test_linear_arguments_are_refused():
    for at in (0, 1, 4):
        args = [P, P, P, P, P, 3]
        args[at] = None
        refused(moe.moe_linear_check, linear_desc(), *args)
    for at in range(5):
        args = [P, P, P, P, P + 32, 3]
        args[at] = P + 8
        refused(moe.moe_linear_check, linear_desc(), *args)
    refused(moe.moe_linear_check, linear_desc(), P, P, P, P, P, -1)
    refused(moe.moe_linear_check, linear_desc(), P, P, P, P, P, (1 << 24) + 1, status=2)
    refused(moe.moe_linear_check, linear_desc(residual_stride=136), P, P, P, P, P, 3)
    with pytest.raises(moe.MoEError):
        moe._check(moe.lib().moe_linear_check(None, P, P, P, P, P, 3), "moe_linear_check")


@pytest.mark.parametrize("kw,status", [
    (dict(B=-1), 1), (dict(B=5), 1), (dict(T=-1), 1), (dict(scale=float("nan")), 1), (dict(scale=float("inf")), 1),
    (dict(softcap=-1.0), 1), (dict(softcap=float("inf")), 1), (dict(window=-1), 1), (dict(q=None), 1),
    (dict(starts=None), 1), (dict(lens=None), 1), (dict(out=None), 1), (dict(block_table=None), 1),
    (dict(max_pages=0), 1), (dict(max_pages=1 << 28), 1), (dict(workspace=None), 1), (dict(workspace=P + 8), 1),
    (dict(q=P + 8), 1), (dict(out=P + 2), 1), (dict(q_stride=504), 1), (dict(q_stride=516), 1),
    (dict(T=1 << 28), 2)])
def test_chunk_arguments_are_refused(kw, status):
    refused(moe.moe_kv_attend_chunk_check, kv_desc(), chunk_args(**kw), status=status)


@pytest.mark.parametrize("kw", [dict(eps=-1e-6), dict(eps=float("nan")), dict(weight_offset=float("inf")),
                                dict(q_weight=P + 4), dict(k_weight=P + 8)])
def test_head_norms_are_refused(kw):
    refused(moe.moe_kv_append_norm_check, kv_desc(), append_args(), head_norm(**kw))


def test_append_arguments_are_looked_at_with_norms_too():
    refused(moe.moe_kv_append_norm_check, kv_desc(), append_args(k=None), head_norm())
    refused(moe.moe_kv_append_norm_check, kv_desc(head_dim=80), append_args(), head_norm(), status=2)


def test_null_handles():
    L = moe.lib()
    assert L.moe_kv_attend_chunk(None, ctypes.byref(chunk_args()), None) == 1
    assert L.moe_kv_append_norm(None, ctypes.byref(append_args()), ctypes.byref(head_norm()), None) == 1
    assert L.moe_kv_chunk_workspace(None) == 0


def test_linear_wants_its_weight_on_a_gpu():
    for w, kw in ((torch.zeros(16, 32, dtype=torch.bfloat16), {}), (torch.zeros(16), {}),
                  (torch.zeros(16, 32), dict(activation="relu"))):
        with pytest.raises(ValueError):
            moe.Linear(w, **kw)
