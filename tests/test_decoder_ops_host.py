"""Block norm and paged cache without a GPU: refusals of bad arguments, and the
block-table arithmetic that the kernels share (moe_kv_locate)."""
import ctypes

import numpy as np
import pytest

import quantized_routed_expert_moe_gb300 as moe

P = 0x10000  # any 16-byte aligned address: the checks never read it


@pytest.fixture(scope="module", autouse=True)
def built():
    from quantized_routed_expert_moe_gb300 import build
    build.build()


def kv_desc(**kw):
    d = dict(abi_version=moe.MOE_ABI_VERSION, n_heads=8, n_kv_heads=2, head_dim=64, page_size=16, n_pages=10,
             cache_dtype=moe.MOE_BF16, rotary_dim=64, rotary_adjacent=0, max_batch=4, page_stride=2 * 16 * 64,
             head_stride=16 * 64, token_stride=64)
    d.update(kw)
    return moe.moe_kv_desc(**d)


def append_args(**kw):
    a = dict(q=P, k=P, v=P, q_stride=512, k_stride=128, v_stride=128, positions=P, seq=P, block_table=P, T=3, n_seqs=4,
             max_pages=5, q_out=P + 4096)
    a.update(kw)
    return moe.moe_kv_append_args(**a)


def attend_args(**kw):
    a = dict(q=P, q_stride=512, block_table=P, lens=P, B=4, max_pages=5, scale=0.1, softcap=0.0, window=0, out=P,
             lse=None)
    a.update(kw)
    return moe.moe_kv_attend_args(**a)


def refused(fn, *args, status=1):
    with pytest.raises(moe.MoEError) as ei:
        fn(*args)
    assert ei.value.status == status, str(ei.value)
    return str(ei.value)


def test_packed_structures_match_the_ctypes_ones():
    """The classes pack their arguments with struct; the layouts are those of the header's types."""
    for packed, c in ((moe.KVCache._append_args, moe.moe_kv_append_args),
                      (moe.KVCache._attend_args, moe.moe_kv_attend_args), (moe.BlockNorm._desc, moe.moe_block_norm_desc)):
        assert len(packed.unpack(bytes(packed.size))) == len(c._fields_)
        buf = bytearray(ctypes.sizeof(c))
        packed.pack_into(buf, 0, *range(1, len(c._fields_) + 1))
        got = c.from_buffer(buf)
        assert [getattr(got, n) for n, _ in c._fields_] == list(range(1, len(c._fields_) + 1))


def test_good_arguments_pass():
    moe.moe_kv_append_check(kv_desc(), append_args())
    moe.moe_kv_append_check(kv_desc(), append_args(q=None, q_out=None, q_stride=0))
    moe.moe_kv_append_check(kv_desc(), append_args(q_out=P))
    moe.moe_kv_append_check(kv_desc(), append_args(T=0, k=None, v=None, positions=None))
    moe.moe_kv_append_check(kv_desc(), append_args(seq=None, T=4))
    moe.moe_kv_attend_check(kv_desc(), attend_args())
    moe.moe_kv_attend_check(kv_desc(), attend_args(B=0, q=None, lens=None))
    # token-major pages, and pages with room between their rows
    moe.moe_kv_attend_check(kv_desc(head_stride=64, token_stride=128), attend_args())
    moe.moe_kv_attend_check(kv_desc(head_stride=2048, token_stride=72, page_stride=8192), attend_args())
    moe.moe_kv_attend_check(kv_desc(n_heads=3, n_kv_heads=1, head_stride=64, token_stride=64, page_stride=1024),
                            attend_args())


@pytest.mark.parametrize("kw,status", [
    (dict(abi_version=9), 1), (dict(n_heads=7), 1), (dict(n_kv_heads=0), 1), (dict(n_heads=0), 1),
    (dict(n_heads=514, n_kv_heads=257), 1), (dict(head_dim=80), 2), (dict(head_dim=0), 2), (dict(page_size=8), 2),
    (dict(page_size=24), 2), (dict(page_size=8192), 2), (dict(n_pages=0), 1), (dict(cache_dtype=moe.MOE_F32), 2),
    (dict(rotary_dim=8), 1), (dict(rotary_dim=80), 1), (dict(rotary_dim=-16), 1), (dict(rotary_adjacent=2), 1),
    (dict(max_batch=0), 1), (dict(max_batch=1025), 1), (dict(token_stride=60), 1), (dict(token_stride=68), 1),
    (dict(head_stride=512), 1), (dict(page_stride=1024), 1), (dict(cache_dtype=moe.MOE_E4M3, token_stride=72), 1),
    (dict(page_stride=1 << 40), 1)])
def test_bad_cache_descriptors(kw, status):
    refused(moe.moe_kv_attend_check, kv_desc(**kw), attend_args(), status=status)
    refused(moe.moe_kv_append_check, kv_desc(**kw), append_args(), status=status)
    refused(moe.moe_kv_create, kv_desc(**kw), P, P, np.ones(32), status=status)


@pytest.mark.parametrize("kw", [
    dict(T=-1), dict(k=None), dict(v=None), dict(positions=None), dict(q=None), dict(q_out=None),
    dict(block_table=None), dict(n_seqs=0), dict(max_pages=0), dict(max_pages=1 << 27), dict(seq=None, T=5),
    dict(q=P + 8), dict(k=P + 2), dict(q_out=P + 4), dict(q_stride=504), dict(k_stride=132), dict(v_stride=64),
    dict(q_out=P, q_stride=520)])
def test_bad_append_arguments(kw):
    refused(moe.moe_kv_append_check, kv_desc(), append_args(**kw))


@pytest.mark.parametrize("kw", [
    dict(B=-1), dict(B=5), dict(q=None), dict(lens=None), dict(out=None), dict(block_table=None), dict(max_pages=0),
    dict(scale=float("nan")), dict(scale=float("inf")), dict(softcap=-1.0), dict(softcap=float("inf")),
    dict(window=-1), dict(q=P + 2), dict(out=P + 8), dict(q_stride=500), dict(q_stride=256)])
def test_bad_attend_arguments(kw):
    refused(moe.moe_kv_attend_check, kv_desc(), attend_args(**kw))


def test_bad_create_arguments():
    f = np.ones(32)
    one = np.ones(2, np.float32)
    refused(moe.moe_kv_create, kv_desc(), None, P, f)
    refused(moe.moe_kv_create, kv_desc(), P, P + 8, f)
    refused(moe.moe_kv_create, kv_desc(), P, P, None)
    refused(moe.moe_kv_create, kv_desc(), P, P, np.array([np.nan] * 32))
    refused(moe.moe_kv_create, kv_desc(), P, P, f, one, one)      # scales on a bf16 cache
    e = kv_desc(cache_dtype=moe.MOE_E4M3)
    refused(moe.moe_kv_create, e, P, P, f)
    refused(moe.moe_kv_create, e, P, P, f, one, None)
    refused(moe.moe_kv_create, e, P, P, f, one, np.array([1, 0], np.float32))
    refused(moe.moe_kv_create, e, P, P, f, np.array([np.inf, 1], np.float32), one)


@pytest.mark.parametrize("bad", [1e-39, -1.0, np.nan, -0.0])
def test_scales_without_a_finite_reciprocal_are_refused(bad):
    e, one, two = kv_desc(cache_dtype=moe.MOE_E4M3), np.ones(2, np.float32), np.array([1, bad], np.float32)
    refused(moe.moe_kv_create, e, P, P, np.ones(32), two, one)
    refused(moe.moe_kv_create, e, P, P, np.ones(32), one, two)


def test_null_handles():
    refused(moe.moe_kv_append, None, append_args())
    refused(moe.moe_kv_attend, None, attend_args())
    assert moe.moe_kv_health(None)[0] == 1
    assert moe.moe_kv_device_bytes(None) == 0
    moe.moe_kv_destroy(None)


def test_create_fails_without_gpu():
    import torch
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    refused(moe.moe_kv_create, kv_desc(), P, P, np.ones(32), status=4)
    d = norm_desc()
    with pytest.raises(moe.MoEError) as ei:
        moe.moe_block_norm(d, P, P, None, P, P, P, P + 65536, 4)
    assert ei.value.status == 4


TABLE = np.array([[3, 0, 9, -1], [1, 10, 2 ** 31 - 1, 5]], np.int32)


@pytest.mark.parametrize("seq,pos,want", [
    (0, 0, 3), (0, 15, 3), (0, 16, 0), (0, 47, 9), (1, 63, 5),
    (0, 48, "page"), (1, 16, "page"), (1, 47, "page"), (0, 64, "length"), (0, -1, "length"), (0, 2 ** 31 - 1, "length"),
    (2, 0, "seq"), (-1, 0, "seq"), (2 ** 31 - 1, 0, "seq")])
def test_locate(seq, pos, want):
    d = kv_desc()
    if not isinstance(want, str):
        got = moe.moe_kv_locate(d, TABLE, seq, pos, 1)
        assert got == want * d.page_stride + d.head_stride + (pos % 16) * d.token_stride
        return
    off, bits = ctypes.c_int64(-5), ctypes.c_uint32()
    st = moe.lib().moe_kv_locate(ctypes.byref(d), TABLE.ctypes.data, 2, 4, seq, pos, 1, ctypes.byref(off),
                                 ctypes.byref(bits))
    assert st == 6 and off.value == -5
    assert bits.value == {"seq": moe.MOE_KV_BAD_SEQ, "length": moe.MOE_KV_BAD_LENGTH,
                          "page": moe.MOE_KV_BAD_PAGE}[want]


def test_locate_past_32_bits():
    d = kv_desc(n_pages=2 ** 31 - 1, n_kv_heads=8, head_dim=256, page_size=4096, head_stride=4096 * 256,
                token_stride=256, page_stride=8 * 4096 * 256)
    t = np.array([[2 ** 31 - 2]], np.int32)
    assert moe.moe_kv_locate(d, t, 0, 4095, 7) == (2 ** 31 - 2) * 8 * 4096 * 256 + 7 * 4096 * 256 + 4095 * 256


def test_locate_refusals():
    d, off = kv_desc(), ctypes.c_int64()
    L = moe.lib()
    for args in ((None, 2, 4, 0, 0, 0), (TABLE.ctypes.data, 0, 4, 0, 0, 0), (TABLE.ctypes.data, 2, 4, 0, 0, 2),
                 (TABLE.ctypes.data, 2, 4, 0, 0, -1)):
        assert L.moe_kv_locate(ctypes.byref(d), *args, ctypes.byref(off), None) == 1
    assert L.moe_kv_locate(ctypes.byref(d), TABLE.ctypes.data, 2, 4, 0, 0, 0, None, None) == 1


# ---- block norm -------------------------------------------------------------------

def norm_desc(**kw):
    d = dict(abi_version=moe.MOE_ABI_VERSION, hidden=128, res_dtype=moe.MOE_F32, block_dtype=moe.MOE_BF16,
             out_dtype=moe.MOE_BF16, eps=1e-6, res_scale=1.0, weight_offset=0.0, x_stride=128, o_stride=136,
             gate_stride=0, r_stride=128, h_stride=128)
    d.update(kw)
    return moe.moe_block_norm_desc(**d)


def norm_args(**kw):
    a = dict(x=P, o=P, gate=P, w_post=P, w_pre=P, r=P, h=P + 65536, T=4)
    a.update(kw)
    return list(a.values())


def test_good_norm_arguments_pass():
    moe.moe_block_norm_check(norm_desc(), *norm_args())
    moe.moe_block_norm_check(norm_desc(), *norm_args(o=None, gate=None, w_post=None))
    moe.moe_block_norm_check(norm_desc(), *norm_args(h=None, w_pre=None))
    moe.moe_block_norm_check(norm_desc(), *norm_args(r=None))
    moe.moe_block_norm_check(norm_desc(), *norm_args(T=0, x=None))
    moe.moe_block_norm_check(norm_desc(hidden=16384, x_stride=16384, o_stride=16384, r_stride=16384, h_stride=16384),
                             *norm_args())


@pytest.mark.parametrize("kw,status", [
    (dict(abi_version=0), 1), (dict(hidden=0), 1), (dict(hidden=100), 1), (dict(hidden=16448), 2),
    (dict(res_dtype=2), 1), (dict(block_dtype=5), 1), (dict(out_dtype=-1), 1), (dict(eps=-1.0), 1),
    (dict(eps=float("nan")), 1), (dict(res_scale=float("inf")), 1), (dict(weight_offset=float("nan")), 1),
    (dict(x_stride=64), 1), (dict(o_stride=132), 1), (dict(gate_stride=64), 1), (dict(gate_stride=-128), 1),
    (dict(r_stride=0), 1), (dict(h_stride=1), 1), (dict(r_stride=136), 1)])
def test_bad_norm_descriptors(kw, status):
    refused(moe.moe_block_norm_check, norm_desc(**kw), *norm_args(), status=status)


@pytest.mark.parametrize("kw", [
    dict(T=-1), dict(x=None), dict(r=None, h=None), dict(o=None), dict(o=None, gate=None), dict(h=None),
    dict(w_pre=None), dict(x=P + 8), dict(o=P + 2), dict(gate=P + 4), dict(w_post=P + 4), dict(w_pre=P + 12),
    dict(r=P + 8), dict(h=P + 1)])
def test_bad_norm_arguments(kw):
    refused(moe.moe_block_norm_check, norm_desc(), *norm_args(**kw))


def test_options_need_a_handle():
    refused(moe.moe_kv_set_option, None, moe.MOE_KV_OPT_TEST_STALL, 0)


# 256 key-value heads of 256 in bf16 (16 tokens to a chunk), 1024 sequences: 8192 chunks each are one too many
@pytest.mark.parametrize("kw,pages,fits", [
    (dict(n_heads=256, n_kv_heads=256, head_dim=256, head_stride=16 * 256, token_stride=256, page_stride=2 ** 20), 8190, True),
    (dict(n_heads=256, n_kv_heads=256, head_dim=256, head_stride=16 * 256, token_stride=256, page_stride=2 ** 20), 8191, False),
    (dict(n_heads=4096, n_kv_heads=1, head_dim=64, head_stride=16 * 64, token_stride=64, page_stride=1024), 4 * 8190, True),
    (dict(n_heads=4096, n_kv_heads=1, head_dim=64, head_stride=16 * 64, token_stride=64, page_stride=1024), 4 * 8191, False)])
def test_tables_of_more_chunks_than_the_kernel_counts(kw, pages, fits):
    d = kv_desc(rotary_dim=0, max_batch=1024, n_pages=4, **kw)
    a = attend_args(B=1024, max_pages=pages, q_stride=kw["n_heads"] * kw["head_dim"])
    if fits:
        moe.moe_kv_attend_check(d, a)
    else:
        refused(moe.moe_kv_attend_check, d, a, status=2)


@pytest.mark.parametrize("kw", [
    dict(page_stride=16 * 64, head_stride=10 * 16 * 64),                                  # heads outermost
    dict(page_stride=2 * 64, head_stride=64, token_stride=10 * 2 * 64),                   # slots outermost
    dict(page_stride=64, head_stride=10 * 64, token_stride=2 * 10 * 64),
    dict(page_stride=80, head_stride=16 * 1000, token_stride=1000),                       # with gaps
    dict(n_pages=1, page_stride=0), dict(n_kv_heads=1, head_stride=0, page_stride=16 * 64)])
def test_pools_in_any_order(kw):
    d = kv_desc(**kw)
    moe.moe_kv_attend_check(d, attend_args())
    moe.moe_kv_append_check(d, append_args(k_stride=128, v_stride=128))
    if d.n_pages > 1 and d.n_kv_heads > 1:
        t = np.array([[7]], np.int32)
        assert moe.moe_kv_locate(d, t, 0, 5, 1) == 7 * d.page_stride + d.head_stride + 5 * d.token_stride


@pytest.mark.parametrize("kw", [
    dict(page_stride=16 * 64, head_stride=9 * 16 * 64), dict(page_stride=64, head_stride=64, token_stride=2048),
    dict(page_stride=2 * 64, head_stride=64, token_stride=9 * 2 * 64), dict(page_stride=56, head_stride=640, token_stride=1280),
    dict(page_stride=0, head_stride=640, token_stride=1280), dict(page_stride=-2048), dict(token_stride=0),
    dict(page_stride=68, head_stride=680, token_stride=1360), dict(head_stride=1 << 39)])
def test_pools_whose_rows_overlap(kw):
    refused(moe.moe_kv_attend_check, kv_desc(**kw), attend_args())
