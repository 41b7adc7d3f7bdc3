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


def _mixed(B, seed, chunk, longest, none=0.0):
    """Lengths and rows of a batch: one chunk, single rows, and requests without a row."""
    rng = np.random.default_rng(seed)
    lens = [int(x) for x in rng.integers(1, longest, B)]
    rows = [0 if x < none else 1 for x in rng.random(B)]
    at = int(rng.integers(0, B))
    lens[at], rows[at] = max(lens[at], chunk), chunk
    return lens, rows


@pytest.mark.parametrize("hq,hkv", [(2, 1), (3, 1)])
@pytest.mark.parametrize("B,chunk,longest,none,pad", [
    (2, 400, 500, 0.0, 0),
    (31, 300, 900, 0.2, 5),
    (32, 513, 700, 0.0, 0),
    (33, 300, 900, 0.3, 0),        # more requests than lanes
    (100, 260, 300, 0.5, 40),
    (300, 129, 60, 0.9, 0),
])
def test_prefill_of_a_chunk_among_single_rows(B, chunk, longest, none, pad, hq, hkv):
    lens, rows = _mixed(B, 141 + B, chunk, longest, none)
    cache = I4.Cache(lens, Hkv=hkv, d=128, P=16, seed=142)
    q = I4.bf16(np.random.default_rng(143).standard_normal((sum(rows), hq, 128)))
    out, lse = _prefill(cache, q, rows, uniform=False, pad=pad)
    _check_prefill(cache, q, rows, out, lse)


def test_prefill_takes_the_parts_that_its_workspace_has_room_for():
    """The least workspace, the one for the batch's rows, and sizes between them. 10 requests of 4 steps each would be
    40 x 16 CTAs: one part. 409 rows come to 13 steps at most: three parts."""
    lens, rows = [2500, 3000, 100, 900, 16, 1, 700, 64, 200, 5], [400] + [1] * 9
    cache = I4.Cache(lens, Hkv=4, d=128, P=16, seed=151)
    ref_q = I4.bf16(np.random.default_rng(152).standard_normal((409, 32, 128)))
    dev, q, cu = cache.to_device(), _bf16_dev(ref_q), _int32(np.concatenate(([0], np.cumsum(rows))))
    least = da.prefill_int4_workspace_bytes((10, 400, 32, 128), dev["k"], dev["tab"])
    most = da.prefill_int4_workspace_bytes(q.shape, dev["k"], dev["tab"], 400)
    assert most > least
    refs, at = [], 0
    for b, t in enumerate(rows):
        refs.append((at, t, I4.attend(cache, b, ref_q[at:at + t], lens[b] - t + np.arange(t))))
        at += t
    for n in (least, (least + most) // 2, most, most + (1 << 20)):
        ws = torch.full((n + 256,), 0x5A, dtype=torch.uint8, device="cuda")
        st = torch.zeros((), dtype=torch.int32, device="cuda")
        out, lse = da.prefill_int4(q, dev["k"], dev["v"], dev["words"], dev["tab"], dev["lens"], cu_q_lens=cu, max_q_rows=400,
                                   workspace=ws[:n], status=st)
        torch.cuda.synchronize()
        assert int(st) == da.OK and bool((ws[n:] == 0x5A).all())
        out, lse = out.to(torch.float64).cpu().numpy(), lse.to(torch.float64).cpu().numpy()
        for at, t, ref in refs:
            I4.check(out[at:at + t], lse[at:at + t], ref, 2.0 ** -8, what=f"{n} bytes")


@pytest.mark.parametrize("B", [511, 700])
def test_prefill_of_a_chunk_among_hundreds_of_single_rows(B):
    """Batches on both sides of the point from which every request has the same number of CTAs."""
    lens, rows = _mixed(B, 155, 300, 40, 0.1)
    cache = I4.Cache(lens, Hkv=1, d=128, P=16, seed=156)
    q = I4.bf16(np.random.default_rng(157).standard_normal((sum(rows), 2, 128)))
    out, lse = _prefill(cache, q, rows, uniform=False, pad=3)
    _check_prefill(cache, q, rows, out, lse)
