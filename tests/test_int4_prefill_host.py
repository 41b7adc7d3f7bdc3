"""Sizes of the INT4 prefill's workspace, on the host."""
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
