"""Sizes of the INT4 prefill's workspace, on the host."""
import ctypes as C

import pytest
import torch

import paged_kv_decode_29_b200 as da


@pytest.fixture(scope="module")
def lib():
    from paged_kv_decode_29_b200 import build
    build.build()
    return da.load_library()


def test_prefill_workspace_with_a_bound_on_the_lengths(lib):
    k = torch.empty((9, 2, 16, 64), dtype=torch.uint8)
    wide, tight = torch.empty((4, 4000), dtype=torch.int32), torch.empty((4, 7), dtype=torch.int32)

    def size(tab, **kw):
        return da.prefill_int4_workspace_bytes((4, 600, 592, 128), k, tab, **kw)
    assert size(wide, max_kv_len=112) == size(wide, max_kv_len=97) == size(tight) == size(tight, max_kv_len=10 ** 6)
    assert size(wide, max_kv_len=113) > size(tight) and size(wide, max_kv_len=0) == size(tight[:, :1], max_kv_len=16)
    assert size(wide) == size(wide, max_kv_len=64000)
    with pytest.raises(ValueError):
        size(wide, max_kv_len=-1)


def _shape(**kw):
    base = dict(batch=32, n_q_heads=8, n_kv_heads=2, head_dim=128, q_tokens=512, page_size=16, num_pages=64,
                max_pages_per_seq=1000, kv_dtype=da.KV_INT4, sm_scale=0.0)
    base.update(kw)
    return da.ShapeT(*[base[f] for f, _ in da.ShapeT._fields_])


def test_packed_workspace_goes_by_the_rows_there_are(lib):
    def base(s):
        return lib.dec_attn_prefill_int4_workspace_bytes(C.byref(s))

    def packed(s, rows):
        return lib.dec_attn_prefill_int4_packed_workspace_bytes(C.byref(s), rows)
    s = _shape()                                              # 512 CTAs: one part
    full, part = base(s), 8 * 129 * 4
    assert packed(s, 32 * 512) == packed(s, 10 ** 6) == full and packed(s, 0) == full
    assert packed(s, 543) == full + -(-4 * 543 * part // 256) * 256   # 36 steps of 4 pairs of heads: four parts
    short = _shape(max_pages_per_seq=16)                      # 256 keys at most
    assert packed(short, 543) == base(short)
    assert packed(s, -1) == da.EINVAL and packed(_shape(batch=-1), 5) == da.EINVAL
    assert lib.dec_attn_prefill_int4_packed_workspace_bytes(None, 5) == da.EINVAL


def test_the_binding_asks_for_the_packed_size(lib):
    k, tab = torch.empty((64, 2, 16, 64), dtype=torch.uint8), torch.empty((32, 1000), dtype=torch.int32)
    s = _shape()
    assert da.prefill_int4_workspace_bytes((543, 8, 128), k, tab, 512) == lib.dec_attn_prefill_int4_packed_workspace_bytes(
        C.byref(s), 543)
    assert da.prefill_int4_workspace_bytes((32, 512, 8, 128), k, tab) == lib.dec_attn_prefill_int4_workspace_bytes(C.byref(s))
