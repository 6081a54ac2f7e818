"""CPU-only: the attention side refuses what it does not take, before anything
reaches the GPU (fake aligned addresses, never dereferenced) -- and the torch
helpers refuse wrong types, shapes and devices."""
import ctypes
import os

import pytest
import torch

from quant_dequant_gemv_amd import binding as b

pytestmark = pytest.mark.skipif(not os.path.exists(b.LIB_PATH),
                                reason="libqkgemv.so not built (run __graft_entry__.build())")

M = 1 << 28  # fake regions M apart
TYPE, SHAPE, PTR, FLAGS = b.QK_EINVAL_TYPE, b.QK_EINVAL_SHAPE, b.QK_EINVAL_PTR, b.QK_EINVAL_FLAGS


def heads(at, row=512, head=128, elem=1, f16=0):
    return b.qk_heads(at * M, row, head, elem, f16)


def cache(**kw):
    a = dict(pool=10 * M, num_pages=8, n_kv_heads=2, head_dim=128, page_size=64)
    return b.qk_kv_cache(*{**a, **kw}.values())


def seqs(**kw):
    a = dict(rows=4, nseq=2, max_pages=4, q_start=11 * M, kv_len=12 * M, pages=13 * M)
    return b.qk_kv_seqs(*{**a, **kw}.values())


def rope(**kw):
    a = dict(q_norm=14 * M, k_norm=15 * M, inv_freq=16 * M, positions=17 * M, eps=1e-6, rot_dim=64, interleaved=0)
    return b.qk_rope(*{**a, **kw}.values())


def test_page_bytes():
    assert b.qk_kv_page_bytes(256, 4, 64) == 2 * 4 * 64 * 160
    assert b.qk_kv_page_bytes(64, 1, 32) == 2 * 32 * 40
    for bad in ((96, 1, 64), (128, 0, 64), (128, 4097, 64), (128, 1, 16), (128, 1, 48), (128, 1, 2048), (0, 1, 32)):
        assert b.qk_kv_page_bytes(*bad) == -1


@pytest.mark.parametrize("c,s,code", [
    (dict(head_dim=80), {}, SHAPE), (dict(page_size=33), {}, SHAPE), (dict(n_kv_heads=0), {}, SHAPE),
    (dict(num_pages=0), {}, SHAPE), (dict(num_pages=1 << 31), {}, SHAPE), (dict(pool=None), {}, PTR),
    (dict(pool=10 * M + 8), {}, PTR),
    ({}, dict(rows=-1), SHAPE), ({}, dict(rows=(1 << 22) + 1), SHAPE), ({}, dict(nseq=0), SHAPE),
    ({}, dict(nseq=65537), SHAPE), ({}, dict(max_pages=0), SHAPE), ({}, dict(max_pages=(1 << 24) + 1), SHAPE),
    ({}, dict(q_start=None, rows=5), SHAPE), ({}, dict(kv_len=None), PTR), ({}, dict(pages=None), PTR),
    ({}, dict(pages=13 * M + 2), PTR), ({}, dict(q_start=11 * M + 1), PTR),
])
def test_every_call_checks_cache_and_sequences(c, s, code):
    c, s = cache(**c), seqs(**s)
    assert b.qk_kv_append(c, s, None, heads(1), heads(2), 0, None, None) == code
    assert b.qk_kv_read(c, s, heads(1), heads(2)) == code
    assert b.qk_kv_attn(c, s, 4, heads(1, f16=1), heads(2), 1.0, 0, 20 * M, 1 << 40) == code
    if code == SHAPE:
        assert b.qk_kv_attn_workspace_bytes(c, s, 4) == -1


def test_null_structs():
    assert b.qk_kv_append(None, seqs(), None, heads(1), heads(2), 0, None, None) == PTR
    assert b.qk_kv_append(cache(), None, None, heads(1), heads(2), 0, None, None) == PTR
    assert b.qk_kv_append(cache(), seqs(), None, None, heads(2), 0, None, None) == PTR
    assert b.qk_kv_append(cache(), seqs(), None, heads(1), heads(2), 4, heads(3), None) == PTR
    assert b.qk_kv_read(cache(), seqs(), None, None) == PTR
    assert b.qk_kv_attn(cache(), seqs(), 4, None, heads(2), 1.0, 0, 20 * M, 1 << 40) == PTR
    assert b.qk_kv_attn(cache(), seqs(), 4, heads(1, f16=1), None, 1.0, 0, 20 * M, 1 << 40) == PTR
    assert b.qk_norm_rope(None, 4, 128, 4, heads(1), heads(2), 0, None, None) == PTR
    assert b.qk_norm_rope(rope(), 4, 128, 4, None, None, 0, None, None) == PTR
    assert b.qk_norm_rope(rope(), 4, 128, 4, heads(1), None, 0, None, None) == PTR


def test_no_rows_is_no_work():
    assert b.qk_kv_append(cache(), seqs(rows=0), None, heads(1), heads(2), 0, None, None) == b.QK_OK
    assert b.qk_kv_read(cache(), seqs(rows=0), heads(1), None) == b.QK_OK
    assert b.qk_kv_attn(cache(), seqs(rows=0), 4, heads(1, f16=1), heads(2), 1.0, 0, None, 0) == b.QK_OK
    assert b.qk_kv_attn_workspace_bytes(cache(), seqs(rows=0), 4) == 0
    assert b.qk_norm_rope(rope(), 0, 128, 4, heads(1), heads(2), 0, None, None) == b.QK_OK


@pytest.mark.parametrize("h,code", [
    (heads(0), PTR), (b.qk_heads(M + 2, 512, 128, 1, 0), PTR), (b.qk_heads(M + 1, 512, 128, 1, 1), PTR),
    (heads(1, f16=2), TYPE), (heads(1, row=-1), SHAPE), (heads(1, row=1 << 62), SHAPE), (heads(1, head=1 << 60), SHAPE),
])
def test_views(h, code):
    c, s = cache(), seqs()
    assert b.qk_kv_append(c, s, None, h, heads(2), 0, None, None) == code
    assert b.qk_kv_append(c, s, None, heads(2), h, 0, None, None) == code
    assert b.qk_kv_append(c, s, None, heads(2), heads(3), 4, h, heads(4)) == code
    assert b.qk_kv_append(c, s, None, heads(2), heads(3), 4, heads(4), h) == code
    assert b.qk_kv_read(c, s, h, None) == code and b.qk_kv_read(c, s, None, h) == code
    assert b.qk_kv_attn(c, s, 4, heads(1, f16=1), h, 1.0, 0, 20 * M, 1 << 40) == code
    assert b.qk_norm_rope(rope(), 4, 128, 4, h, heads(4), 0, None, None) == code


@pytest.mark.parametrize("strides", [(0, 128, 1), (512, 0, 1), (512, 128, 0), (512, 100, 1), (511, 128, 1), (1, 1, 4)])
def test_outputs_have_elements_of_their_own(strides):
    h = heads(1, *strides)
    if strides != (511, 128, 1):  # too close for 4 heads, far enough for the cache's 2
        assert b.qk_kv_read(cache(), seqs(), h, None) == SHAPE
    assert b.qk_kv_attn(cache(), seqs(), 4, heads(2, f16=1), h, 1.0, 0, 20 * M, 1 << 40) == SHAPE
    assert b.qk_kv_append(cache(), seqs(), None, heads(2), heads(3), 4, heads(4), h) == SHAPE


def test_attn_arguments():
    c, s, q, o = cache(), seqs(), heads(1, f16=1), heads(2)
    assert b.qk_kv_attn(c, s, 4, heads(1), o, 1.0, 0, 20 * M, 1 << 40) == TYPE  # fp32 queries
    for n in (0, -2, 3, 4098):
        assert b.qk_kv_attn(c, s, n, q, o, 1.0, 0, 20 * M, 1 << 40) == SHAPE
        assert b.qk_kv_attn_workspace_bytes(c, s, n) == -1
    assert b.qk_kv_attn(c, s, 4, q, o, float("inf"), 0, 20 * M, 1 << 40) == SHAPE
    assert b.qk_kv_attn(c, s, 4, q, o, float("nan"), 0, 20 * M, 1 << 40) == SHAPE
    assert b.qk_kv_attn(c, s, 4, q, o, -2.0 ** 65, 0, 20 * M, 1 << 40) == SHAPE
    big = seqs(rows=1 << 22, nseq=1, q_start=None)
    assert b.qk_kv_attn(c, big, 16, heads(1, 2048, 128, 1, 1), heads(8, 2048, 128), 1.0, 0, 200 * M, 1 << 40) == SHAPE
    assert b.qk_kv_attn(c, s, 4, q, o, 1.0, -1, 20 * M, 1 << 40) == SHAPE
    # a row each for 65536 sequences: 2^21 sequences x KV heads pass, a KV head more does not
    for hk, ok in ((32, True), (33, False), (512, False)):
        wide = b.qk_kv_cache(c.pool, c.num_pages, hk, c.head_dim, c.page_size)
        assert (b.qk_kv_attn_workspace_bytes(wide, seqs(rows=65536, nseq=65536, q_start=None), hk) >= 0) == ok
    # out over the queries, the pool, the tables
    for at in (1 * M + 4, 10 * M + 64, 11 * M, 12 * M + 4, 13 * M + 28):
        assert b.qk_kv_attn(c, s, 4, q, b.qk_heads(at, 512, 128, 1, 0), 1.0, 0, 20 * M, 1 << 40) == PTR
    big = seqs(rows=1, nseq=1, q_start=None, max_pages=1 << 16)
    need = b.qk_kv_attn_workspace_bytes(c, big, 4)
    assert need >= 0
    if need:
        assert b.qk_kv_attn(c, big, 4, q, o, 1.0, 0, 20 * M, need - 1) == SHAPE
        for ws in (None, 20 * M + 8, 1 * M, 2 * M, 10 * M + 16, 12 * M, 13 * M):
            assert b.qk_kv_attn(c, big, 4, q, o, 1.0, 0, ws, need) == PTR


def test_rope_arguments():
    def call(r, q_out=None):
        return b.qk_norm_rope(r, 4, 128, 4, heads(1), q_out or heads(2), 2, heads(3), heads(4))

    for kw, code in ((dict(rot_dim=3), SHAPE), (dict(rot_dim=-2), SHAPE), (dict(rot_dim=130), SHAPE),
                     (dict(eps=-1.0), SHAPE), (dict(eps=float("nan")), SHAPE), (dict(eps=float("inf")), SHAPE),
                     (dict(interleaved=2), FLAGS), (dict(inv_freq=None), PTR), (dict(positions=None), PTR),
                     (dict(q_norm=14 * M + 2), PTR)):
        assert call(rope(**kw)) == code
    for at in (14 * M, 15 * M + 508, 16 * M, 17 * M + 8, 3 * M, 4 * M + 4, 1 * M + 4):
        assert call(rope(), b.qk_heads(at, 512, 128, 1, 0)) == PTR
    assert call(rope(), b.qk_heads(M, 512, 128, 1, 1)) == PTR  # over its input in another type
    assert b.qk_norm_rope(rope(), 4, 96, 4, heads(1), heads(2), 0, None, None) == SHAPE
    assert b.qk_norm_rope(rope(), -1, 128, 4, heads(1), heads(2), 0, None, None) == SHAPE
    assert b.qk_norm_rope(rope(), 4, 128, 0, heads(1), heads(2), 0, None, None) == SHAPE
    assert b.qk_norm_rope(rope(), 1 << 22, 128, 4096, heads(1), heads(2), 0, None, None) == SHAPE


def test_append_overlaps():
    c, s = cache(), seqs()
    for bad in (10 * M, 11 * M, 13 * M):  # q_out over the pool and the tables
        assert b.qk_kv_append(c, s, None, heads(1), heads(2), 4, heads(3), b.qk_heads(bad, 512, 128, 1, 0)) == PTR
    assert b.qk_kv_append(c, s, None, b.qk_heads(10 * M, 512, 128, 1, 0), heads(2), 0, None, None) == PTR
    assert b.qk_kv_append(c, s, None, heads(1), heads(2), 4, heads(3), b.qk_heads(M + 8, 512, 128, 1, 0)) == PTR
    assert b.qk_kv_append(c, s, rope(inv_freq=10 * M), heads(1), heads(2), 0, None, None) == PTR
    assert b.qk_kv_append(c, seqs(kv_len=10 * M + 4), None, heads(1), heads(2), 0, None, None) == PTR
    assert b.qk_kv_read(c, s, heads(1), heads(1)) == PTR


# ------------------------------------------------------------------ the torch helpers

def z(*shape, dtype=torch.float32):
    return torch.zeros(shape, dtype=dtype)


def test_helpers_refuse():
    pool = z(4 * 2 * 2 * 32 * 80, dtype=torch.uint8)
    c = b.KVCache(4, 2, 128, 32, pool=pool)
    pages, kv_len = z(2, 3, dtype=torch.int32), z(2, dtype=torch.int32)
    k = z(4, 2, 128)
    with pytest.raises(ValueError, match="elements"):
        b.KVCache(4, 2, 128, 32, pool=pool[:-1])
    with pytest.raises(b.QKError):
        b.KVCache(4, 2, 100, 32)
    with pytest.raises(TypeError):
        b.kv_append(c, k.double(), k, pages, kv_len)
    with pytest.raises(ValueError, match="shape"):
        b.kv_append(c, z(4, 3, 128), k, pages, kv_len)
    with pytest.raises(ValueError, match="shape"):
        b.kv_append(c, k, z(5, 2, 128), pages, kv_len)
    with pytest.raises(ValueError, match="shape"):
        b.kv_append(c, k, k, pages[:1], kv_len)
    with pytest.raises(TypeError, match="int32"):
        b.kv_append(c, k, k, pages.long(), kv_len)
    with pytest.raises(ValueError, match="contiguous"):
        b.kv_append(c, k, k, z(3, 2, dtype=torch.int32).t(), kv_len)
    with pytest.raises(ValueError, match="q_start"):
        b.kv_append(c, k, k, pages, kv_len, q_start=z(2, dtype=torch.int32))
    with pytest.raises(ValueError, match="rope"):
        b.kv_append(c, k, k, pages, kv_len, positions=z(4, dtype=torch.int32))
    r = b.Rope(z(32), q_norm=z(64))
    with pytest.raises(ValueError, match="q_norm"):
        b.kv_append(c, k, k, pages, kv_len, rope=r)
    with pytest.raises(TypeError):
        b.Rope(z(32).half())
    with pytest.raises(TypeError, match="float16"):
        b.kv_attn(c, z(4, 4, 128), pages, kv_len)
    with pytest.raises(ValueError, match="positions"):
        b.norm_rope(b.Rope(z(32)), z(3, dtype=torch.int32), z(4, 4, 128))
    # sizes right, tensors on the host
    for call in (lambda: b.kv_append(c, k, k, pages, kv_len), lambda: b.kv_read(c, 4, pages, kv_len),
                 lambda: b.kv_attn(c, z(4, 4, 128, dtype=torch.float16), pages, kv_len),
                 lambda: b.norm_rope(b.Rope(z(32)), z(4, dtype=torch.int32), z(4, 4, 128))):
        with pytest.raises(ValueError, match="CUDA"):
            call()


def test_helpers_refuse_sizes_past_32_bits():
    """Not their low 32 bits."""
    pool = z(4 * 2 * 2 * 32 * 80, dtype=torch.uint8)
    for sizes in ((4, 2 + 2 ** 32, 128, 32), (4, 2, 128 + 2 ** 32, 32), (4, 2, 128, 32 + 2 ** 32), (4 + 2 ** 32, 2, 128, 32)):
        with pytest.raises(b.QKError):
            b.KVCache(*sizes, pool=pool)
    c = b.KVCache(4, 2, 128, 32, pool=pool)
    pages, kv_len = z(1, 3, dtype=torch.int32), z(1, dtype=torch.int32)
    with pytest.raises(b.QKError):
        b.kv_read(c, 2 ** 32 + 1, pages, kv_len)
    with pytest.raises(b.QKError):
        b.kv_read(c, 1, z(1, 1, dtype=torch.int32).expand(1, 2 ** 32 + 3), kv_len)


def test_struct_layouts():
    assert ctypes.sizeof(b.qk_heads) == 40 and ctypes.sizeof(b.qk_rope) == 48
    assert ctypes.sizeof(b.qk_kv_cache) == 32 and ctypes.sizeof(b.qk_kv_seqs) == 40
