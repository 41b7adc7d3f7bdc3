"""Packed calls over an INT4 cache with offsets that are wrong: which rows are skipped, that the others are right, and that
nothing else is written."""
import numpy as np
import pytest
import torch

import paged_kv_decode_29_b200 as da
from tests import _int4 as I4
from tests.test_int4_gpu import _bf16_dev, _f64, _int32, _new_rows, _prefill

pytestmark = pytest.mark.gpu


# offsets of three requests of 40 tokens over three rows -> per row its request and position (None: not covered), and
# the status. A row belongs to the last request that starts at or before it, if that request ends behind it and within the
# rows.
@pytest.mark.parametrize("cu,rows,status", [
    ([0, 1, 2, 3], [(0, 39), (1, 39), (2, 39)], da.OK),
    ([0, 1, 2, 9], [(0, 39), (1, 39), None], da.EDEVICE),
    ([0, 2, 1, 3], [(0, 38), (0, 39), (2, 39)], da.OK),       # decreasing, but every row is covered
    ([1, 2, 2, 3], [None, (0, 39), (2, 39)], da.EDEVICE),
    ([-5, 1, 2, 3], [None, (1, 39), (2, 39)], da.EDEVICE),
    ([0, 1, 1, 2], [(0, 39), (2, 39), "behind"], da.OK),      # a padded batch
    ([0, 0, 0, 0], ["behind"] * 3, da.OK),
    ([0, 1, 2, -1], ["behind"] * 3, da.OK),                   # no row at all
    ([3, 3, 3, 3], [None] * 3, da.EDEVICE),
    ([0, 1 << 30, 1 << 30, 1 << 30], [None] * 3, da.EDEVICE),
])
@pytest.mark.parametrize("d", [64, 128])
def test_append_skips_the_rows_that_no_request_covers(cu, rows, status, d):
    rng = np.random.default_rng(161)
    cache = I4.Cache([40, 40, 40], Hkv=2, d=d, P=16, seed=162)
    q, k, v = _new_rows(rng, 3, 4, 2, d)
    pools, words = [p.copy() for p in cache.pools], cache.words.copy()
    q_out, vals = np.full(q.shape, 3.0), [np.full(k.shape, 3.0) for _ in range(2)]
    for i, at in enumerate(rows):
        if not isinstance(at, tuple):
            continue
        b, pos = at
        q_out[i] = I4.rotate(q[i:i + 1], [pos])[0]
        pid, slot = cache.table[b, pos // 16], pos % 16
        for which, x in enumerate((I4.rotate(k[i:i + 1], [pos]), v[i:i + 1])):
            codes, wd, val = I4.quantise(x)
            pools[which][pid, :, slot], words[which, pid, :, slot], vals[which][i] = codes[0], wd[0], val[0]
    dev = cache.to_device()
    st = torch.zeros((), dtype=torch.int32, device="cuda")
    bufs = [torch.full(x.shape, 3.0, dtype=torch.bfloat16, device="cuda") for x in (q, k, k)]
    da.append_rope_int4(*[_bf16_dev(x) for x in (q, k, v)], dev["tab"], dev["lens"], dev["k"], dev["v"], dev["words"],
                        cu_q_lens=_int32(cu), q_out=bufs[0], k_values=bufs[1], v_values=bufs[2], status=st)
    torch.cuda.synchronize()
    assert int(st) == status
    assert np.array_equal(_f64(bufs[0]), q_out) and all(np.array_equal(_f64(b), x) for b, x in zip(bufs[1:], vals))
    assert np.array_equal(dev["k"].cpu().numpy(), pools[0]) and np.array_equal(dev["v"].cpu().numpy(), pools[1])
    assert np.array_equal(dev["words"].cpu().numpy().view(np.uint16), words)


# good offsets are [0, 100, 250]; requests listed are right, rows outside them are left as they were
@pytest.mark.parametrize("cu,max_rows,right", [
    ([0, 100, 400], 300, [0]),            # past the rows
    ([0, 100, 250], 149, [0]),            # more rows than the bound
    ([0, 240, 390], 150, []),
    ([-1, 100, 250], 150, [1]),
    ([100, 100, 250], 150, [1]),          # the first request has no row
    ([0, 100, 90], 150, [0]),             # decreasing
    ([0, 100, -7], 150, [0]),
])
def test_prefill_skips_requests_whose_offsets_lie_outside(cu, max_rows, right):
    lens, rows, at = [200, 150], [100, 150], [0, 100, 250]
    cache = I4.Cache(lens, Hkv=2, d=128, P=16, seed=163)
    q = I4.bf16(np.random.default_rng(164).standard_normal((250, 4, 128)))
    ref = _prefill(cache, q, rows, uniform=False)
    bad = cu != [100, 100, 250]
    got = _prefill(cache, q, rows, uniform=False, cu=cu, max_rows=max_rows, expect=da.EDEVICE if bad else da.OK)
    written = np.zeros(250, dtype=bool)
    for b in right:
        written[at[b]:at[b + 1]] = True
        # the parts may be cut elsewhere, as the bound and the offsets count: two roundings of the weights to bf16, and of out
        assert np.abs(got[0][at[b]:at[b + 1]] - ref[0][at[b]:at[b + 1]]).max() <= 2.0 ** -6 * np.abs(cache.dense(1, b)).max()
        assert np.abs(got[1][at[b]:at[b + 1]] - ref[1][at[b]:at[b + 1]]).max() <= 1e-4
    assert np.all(got[0][~written] == 5.0) and np.all(got[1][~written] == 5.0)


@pytest.mark.parametrize("B", [20, 70])
def test_prefill_of_many_requests_with_one_bad_offset(B):
    """Grids that go by the rows: the requests are found by their offsets, and a bad one takes no other's place."""
    rng = np.random.default_rng(165)
    lens = [int(x) for x in rng.integers(1, 200, B)]
    lens[7], rows = 300, [1] * B
    rows[7] = 270
    cache = I4.Cache(lens, Hkv=1, d=128, P=16, seed=166)
    q = I4.bf16(rng.standard_normal((sum(rows), 2, 128)))
    cu = np.concatenate(([0], np.cumsum(rows)))
    ref = _prefill(cache, q, rows, uniform=False)
    for i, to in ((3, cu[-1] + 5), (12, -3), (B, cu[-1] + 1), (0, -1)):
        x = cu.copy()
        x[i] = to
        got = _prefill(cache, q, rows, uniform=False, cu=x, max_rows=270, expect=da.EDEVICE)
        for b in range(B):
            at = slice(cu[b], cu[b + 1])
            if i not in (b, b + 1):                          # neither of its offsets was touched
                assert np.abs(got[0][at] - ref[0][at]).max() <= 2.0 ** -6 * np.abs(cache.dense(1, b)).max()
                assert np.abs(got[1][at] - ref[1][at]).max() <= 1e-4
