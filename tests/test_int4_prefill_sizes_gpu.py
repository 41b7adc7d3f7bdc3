"""Prefill over an INT4 cache where the table, the batch or the padding is much larger than the work."""
import numpy as np
import pytest
import torch

import paged_kv_decode_29_b200 as da
from tests import _int4 as I4
from tests.test_int4_gpu import _bf16_dev, _check_prefill, _int32, _prefill

pytestmark = pytest.mark.gpu


def _widen(cache, width):
    """The table of a server that allows for longer contexts: what lies behind a request's pages is never read."""
    table = np.full((len(cache.lens), width), 1 << 30, dtype=np.int32)
    for b, n in enumerate(cache.lens):
        table[b, :-(-n // cache.P)] = cache.table[b, :-(-n // cache.P)]
    cache.table = table


@pytest.mark.parametrize("width", [40, 41, 3000])
def test_prefill_with_a_table_wider_than_any_request(width):
    """Also more pages than the expansion has CTAs (40 requests of 16 KV heads: 15 each)."""
    rng = np.random.default_rng(131)
    lens = [640] + [int(x) for x in rng.integers(0, 600, 39)]
    cache = I4.Cache(lens, Hkv=16, d=128, P=16, seed=132)
    _widen(cache, width)
    rows = [min(n, int(x)) for n, x in zip(lens, rng.integers(0, 3, 40))]
    q = I4.bf16(rng.standard_normal((sum(rows), 16, 128)))
    out, lse = _prefill(cache, q, rows, uniform=False, max_rows=3)
    _check_prefill(cache, q, rows, out, lse)


def test_prefill_with_a_bound_on_the_lengths():
    lens, rows = [500, 20, 200], [70, 20, 1]
    cache = I4.Cache(lens, Hkv=2, d=128, P=16, seed=133)
    ref_q = I4.bf16(np.random.default_rng(134).standard_normal((91, 4, 128)))
    ref = _prefill(cache, ref_q, rows, uniform=False)
    _widen(cache, 5000)
    dev, q, cu = cache.to_device(), _bf16_dev(ref_q), _int32([0, 70, 90, 91])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for bound, want in ((500, da.OK), (512, da.OK), (80000, da.OK), (10 ** 9, da.OK), (496, da.EDEVICE), (0, da.EDEVICE)):
        for stream in (None, s):
            st = torch.zeros((), dtype=torch.int32, device="cuda")
            ws = torch.full((da.prefill_int4_workspace_bytes(q.shape, dev["k"], dev["tab"], 70, bound),), 0, dtype=torch.uint8,
                            device="cuda")
            torch.cuda.synchronize()
            out, lse = da.prefill_int4(q, dev["k"], dev["v"], dev["words"], dev["tab"], dev["lens"], cu_q_lens=cu, max_q_rows=70,
                                       max_kv_len=bound, workspace=ws, status=st, stream=stream)
            torch.cuda.synchronize()
            assert int(st) == want
            got = out.to(torch.float64).cpu().numpy(), lse.to(torch.float64).cpu().numpy()
            if want == da.OK:
                _check_prefill(cache, ref_q, rows, *got)
            if bound == 496:                                 # the others are right
                assert np.abs(got[0][70:] - ref[0][70:]).max() < 2.0 ** -6 and np.abs(got[1][70:] - ref[1][70:]).max() < 1e-4
