"""The INT4 cache at the ends of its numbers: V rows whose scales lie far apart, channels of zeros, NaN rows, queries of
any magnitude, and the quantiser's scale where the range of a row is no fp32 number."""
from fractions import Fraction

import numpy as np
import pytest
import torch

import paged_kv_decode_29_b200 as da
from tests import _int4 as I4
from tests.test_int4_gpu import _append_case, _check_decode, _decode, _prefill

pytestmark = pytest.mark.gpu


def _set_row(cache, which, b, h, pos, word, codes=None):
    """Word (and packed codes) of one row of request b."""
    pid, slot = cache.table[b, pos // cache.P], pos % cache.P
    cache.words[which, pid, h, slot] = word
    if codes is not None:
        cache.pools[which][pid, h, slot] = codes


def _add_exponent(cache, which, b, h, pos, k):
    """That row's scale times 2^k."""
    pid, slot = cache.table[b, pos // cache.P], pos % cache.P
    cache.words[which, pid, h, slot] = int(cache.words[which, pid, h, slot]) + (k << 7)


# ---------------------------------------------------------------------------- V scales that lie far apart
@pytest.mark.parametrize("k", [4, 11, 20, 24, 28, 34, 40, 60, 100])
@pytest.mark.parametrize("d,pos", [(128, 5), (128, 150), (64, 150), (128, 199)])
def test_a_large_v_row_of_no_weight_takes_nothing_from_the_others(d, pos, k):
    cache = I4.Cache([200], Hkv=1, d=d, P=16, seed=101)
    q = I4.bf16(np.abs(np.random.default_rng(102).standard_normal((1, 1, 4, d))) + 0.1)
    _set_row(cache, 0, 0, 0, pos, 0x40FF, 0)                 # K: -15 times 7.5 in every channel: a weight below 2^-200
    _add_exponent(cache, 1, 0, 0, pos, k)
    for tile in (64, 256):
        out, lse = _decode(cache, q, 1, tile=tile)
        _check_decode(cache, q, 1, out, lse, what=f"tile {tile}")


@pytest.mark.parametrize("k", [11, 24, 28, 34, 60, 100, -40, -100])
@pytest.mark.parametrize("hq,d", [(4, 128), (4, 64), (2, 128)])
def test_rows_do_not_depend_on_the_v_rows_of_later_tokens(hq, d, k):
    T, L = 4, 130
    cache = I4.Cache([L, 3], Hkv=1, d=d, P=16, seed=103)
    q = I4.bf16(np.random.default_rng(104).standard_normal((2, T, hq, d)))
    for b, n in enumerate(cache.lens):
        _add_exponent(cache, 1, b, 0, n - 1, k)              # the last token: seen by the last row alone
    for tile in (64, 256):
        out, lse = _decode(cache, q, T, tile=tile)
        _check_decode(cache, q, T, out, lse, what=f"tile {tile}")


@pytest.mark.parametrize("span", [5, 12, 25, 60, 110])
@pytest.mark.parametrize("hq,T,d", [(4, 1, 128), (4, 4, 64), (8, 5, 128)])
def test_v_scales_of_any_spread(hq, T, d, span):
    """Every row's scale times a power of two of its own; equal weights, and queries that pick out single keys, each
    with the scale of its own key."""
    lens = [300, 65, 1000]
    cache = I4.Cache(lens, Hkv=2, d=d, P=16, seed=105 + span)
    rng = np.random.default_rng(106)
    w = cache.words[1].astype(np.int64)
    w += rng.integers(-span, span + 1, w.shape) << 7
    for b, n in enumerate(lens):
        for i, pid in enumerate(cache.table[b, :-(-n // 16)]):
            used = min(16, n - 16 * i)
            cache.words[1, pid, :, :used] = w[pid, :, :used]
    q = rng.standard_normal((3, T, hq, d))
    for b, n in enumerate(lens):
        k = cache.dense(0, b)
        for t in range(T):
            for h in range(0, hq, 2):
                q[b, t, h] = 100 * np.sign(k[h // (hq // 2), rng.integers(0, n - T + 1)])
    q = I4.bf16(q)
    for tile in (64, 1024):
        out, lse = _decode(cache, q, T, tile=tile)
        _check_decode(cache, q, T, out, lse, what=f"tile {tile}")


@pytest.mark.parametrize("low,high", [(1, 4), (3, 12), (8, 20), (1, 60), (240, 250)])
@pytest.mark.parametrize("d", [64, 128])
def test_v_scales_at_the_ends_of_their_range(low, high, d):
    """Biased exponents low .. high."""
    cache = I4.Cache([130, 700], Hkv=2, d=d, P=16, seed=127)
    rng = np.random.default_rng(128)
    cache.words[1] = (rng.integers(low, high + 1, cache.words[1].shape) << 7) | rng.integers(0, 8, cache.words[1].shape) << 4 | 7
    q = I4.bf16(rng.standard_normal((2, 2, 6, d)))
    for tile in (64, 1024):
        out, lse = _decode(cache, q, 2, tile=tile)
        if low > 1:                                          # else out may be no normal number
            _check_decode(cache, q, 2, out, lse, what=f"tile {tile}")
        else:
            for b, n in enumerate(cache.lens):
                ref, ref_l, mass, _ = I4.attend(cache, b, q[b], n - 2 + np.arange(2))
                assert np.all(np.abs(out[b] - ref) <= 2.0 ** -8 * np.abs(ref) + 2.0 ** -10 * mass[..., None] + 2.0 ** -134)
                assert np.abs(lse[b] - ref_l).max() <= 1e-4


def test_zero_v_rows_among_others():
    """An all-zero row is stored with the least scale there is."""
    cache = I4.Cache([400], Hkv=1, d=128, P=16, seed=107)
    for pos in (0, 1, 2, 63, 64, 200, 399):
        _set_row(cache, 1, 0, 0, pos, 0x0080, 0)
    q = I4.bf16(np.random.default_rng(108).standard_normal((1, 1, 8, 128)))
    for tile in (64, 512):
        out, lse = _decode(cache, q, 1, tile=tile)
        _check_decode(cache, q, 1, out, lse, what=f"tile {tile}")
    cache.words[1] = 0x0080                                  # and nothing else
    cache.pools[1][:] = 0
    out, _ = _decode(cache, q, 1, tile=512)
    assert np.all(out == 0)


# ---------------------------------------------------------------------------- weights and zero points
@pytest.mark.parametrize("d", [64, 128])
def test_a_channel_of_zeros_comes_out_near_zero(d):
    """V elements with c = z = 15 under weights that f16 rounds by 2^-13 of their value, all to the same side: a product
    with rounded weights less zero points under others would leave 15 times that. What may be left: the 16 products of an
    MMA and its accumulator are added with an error of 17 units of 2^-23 of the sum, 16 MMAs in a row; the zero points'
    share, added in fp32, 2^-19; both of sums that come to 15 times the weights."""
    L = 256
    cache = I4.Cache([L], Hkv=1, d=d, P=16, seed=109)
    cache.words[0] = 0x3F88
    cache.pools[0][:] = 0x88                                 # K is zero
    _set_row(cache, 0, 0, 0, 3, 0x3F88, np.array([0x89] + [0x88] * (d // 2 - 1)))   # but for one element
    cache.words[1] = 0x3F8F                                  # V: scale 1, zero point 15
    cache.pools[1][..., ::2] |= 0x0F                         # channels 0, 4, 8 ..: zero
    p = np.exp(-0.3)
    assert abs(float(np.float16(p)) / p - 1) > 2.0 ** -13
    q = np.zeros((1, 1, 1, d))
    q[..., 0] = 1.0
    out, lse = _decode(cache, q, 1, tile=256, sm_scale=0.3)
    _check_decode(cache, q, 1, out, lse, sm_scale=0.3)
    assert np.abs(out[..., ::4]).max() <= 15 * (17 * 16 * 2.0 ** -23 + 2.0 ** -19)


# ---------------------------------------------------------------------------- NaN rows
@pytest.mark.parametrize("tile", [64, 512])
@pytest.mark.parametrize("which", [0, 1])
@pytest.mark.parametrize("word", [0x7FC0, 0xFFC0])
def test_a_nan_row_reaches_out_and_lse_wherever_it_lies(word, which, tile):
    T, L = 2, 300
    cache = I4.Cache([L, 40], Hkv=2, d=128, P=16, seed=110)
    q = I4.bf16(np.random.default_rng(111).standard_normal((2, T, 4, 128)))
    ref, ref_l = _decode(cache, q, T, tile=tile)
    for pos in (0, 70, 192, 255, 297, 299):                  # first and later blocks, the masked last one
        pid, slot = cache.table[0, pos // 16], pos % 16
        saved = cache.words[which, pid, 1, slot]
        cache.words[which, pid, 1, slot] = word
        out, lse = _decode(cache, q, T, tile=tile)
        cache.words[which, pid, 1, slot] = saved
        sees = np.zeros(out.shape[:3], dtype=bool)
        sees[0, :, 2:] = (L - T + np.arange(T) >= pos)[:, None]
        assert np.isnan(out[sees]).all() and np.isnan(lse[sees]).all(), pos
        assert np.array_equal(out[~sees], ref[~sees]) and np.array_equal(lse[~sees], ref_l[~sees]), pos


def test_an_infinite_v_scale_is_a_nan_row():
    cache = I4.Cache([200], Hkv=1, d=128, P=16, seed=112)
    q = I4.bf16(np.random.default_rng(113).standard_normal((1, 3, 4, 128)))
    ref, ref_l = _decode(cache, q, 3, tile=256)
    pref, pref_l = _prefill(cache, q[0], [3], uniform=True)
    for word in (0x7F80, 0x7F83, 0xFF80):
        _set_row(cache, 1, 0, 0, 198, word)
        out, lse = _decode(cache, q, 3, tile=256)
        assert np.isnan(out[0, 1:]).all() and np.isnan(lse[0, 1:]).all()
        assert np.array_equal(out[0, 0], ref[0, 0]) and np.array_equal(lse[0, 0], ref_l[0, 0])
        out, lse = _prefill(cache, q[0], [3], uniform=True)
        assert np.isnan(out[1:]).all() and np.isnan(lse[1:]).all()
        assert np.array_equal(out[0], pref[0]) and np.array_equal(lse[0], pref_l[0])


# ---------------------------------------------------------------------------- queries
@pytest.mark.parametrize("bad", [np.nan, np.inf, -np.inf])
def test_a_query_row_that_is_not_finite_stays_alone(bad):
    """... and has out = 0 and lse = -inf like any other where it sees no key. Where it sees some, decode gives NaN; so does
    prefill, but for a row all of whose scores are -inf (an infinite element times keys of one sign), which has no weight
    anywhere and comes out like a row without a key, as over the other caches."""
    T, lens = 4, [2, 130, 1]
    cache = I4.Cache(lens, Hkv=2, d=128, P=16, seed=114)
    q = I4.bf16(np.random.default_rng(115).standard_normal((3, T, 4, 128)))
    x = q.copy()
    x[0, 1, 0, 5] = x[0, 0, 3] = x[0, 2, 2, 127] = x[1, 0, 1, 64] = x[1, 3] = x[2, :3, 0, 0] = bad
    hit = ~np.isfinite(x).all(-1)
    empty = np.array([[n - T + t < 0 for t in range(T)] for n in lens])[:, :, None] & np.ones((1, 1, 4), dtype=bool)
    pre = [[y.reshape(q.shape[:y.ndim + 1]) for y in _prefill(cache, z.reshape(12, 4, 128), [T] * 3, uniform=True)] for z in (q, x)]
    for ref, got in ((_decode(cache, q, T, tile=64), _decode(cache, x, T, tile=64)), pre):
        assert np.all(got[0][empty] == 0) and np.all(np.isneginf(got[1][empty]))
        assert np.array_equal(got[0][~hit], ref[0][~hit]) and np.array_equal(got[1][~hit], ref[1][~hit])
        nan = hit & ~empty
        if got is pre[1]:
            with np.errstate(invalid="ignore"):
                for b, n in enumerate(lens):
                    for t in range(T):
                        for h in range(4):
                            s = cache.dense(0, b)[h // 2, :max(n - T + t + 1, 0)] * x[b, t, h]
                            if nan[b, t, h] and np.all(np.isneginf(s.sum(-1))):
                                nan[b, t, h] = False
                                assert np.all(got[0][b, t, h] == 0) and np.isneginf(got[1][b, t, h])
        assert np.isnan(got[0][nan]).all() and np.isnan(got[1][nan]).all()


@pytest.mark.parametrize("tile", [64, 512])
@pytest.mark.parametrize("d", [64, 128])
def test_queries_of_any_magnitude(d, tile):
    """Keys small enough that the scores of the largest rows are ordinary numbers; rows of every magnitude side by
    side."""
    cache = I4.Cache([300, 70], Hkv=2, d=d, P=16, seed=116)
    w = cache.words[0].astype(np.int64)
    small = w - (120 << 7)                                   # K scales about 2^-122
    cache.words[0] = np.where((w >> 7 & 255) > 120, small, w).astype(np.uint16)
    q = np.random.default_rng(117).standard_normal((2, 2, 16, d))
    q *= 2.0 ** np.array([123, 119, 116, 115, 110, 0, -40, -130, 122, 120, 117, 116, 100, 60, -80, -125])[:, None]
    q = I4.bf16(q)
    assert np.isfinite(q).all() and np.abs(q).max() > 2.0 ** 123
    out, lse = _decode(cache, q, 2, tile=tile)
    _check_decode(cache, q, 2, out, lse)


def test_large_queries_over_ordinary_keys():
    """Scores of 2^100 and more: the weights are those of the largest score, and finite."""
    cache = I4.Cache([200], Hkv=1, d=128, P=16, seed=118)
    q = np.random.default_rng(119).standard_normal((1, 1, 4, 128)) * 2.0 ** np.array([100, 113, 116, 118])[:, None]
    q = I4.bf16(q)
    out, lse = _decode(cache, q, 1, tile=256)
    assert np.isfinite(out).all() and np.isfinite(lse).all()
    _check_decode(cache, q, 1, out, lse)


@pytest.mark.parametrize("qs,ks", [(2.0 ** -125, 2.0 ** 121), (2.0 ** -110, 2.0 ** 110), (2.0 ** -90, 2.0 ** 88)])
def test_small_queries_over_large_keys(qs, ks):
    cache = I4.Cache([300], Hkv=1, d=128, P=16, seed=120)
    k = int(np.log2(ks))
    for i, pid in enumerate(cache.table[0]):
        used = min(16, 300 - 16 * i)
        cache.words[0, pid, :, :used] += k << 7
    q = I4.bf16(np.random.default_rng(121).standard_normal((1, 1, 4, 128)) * qs)
    out, lse = _decode(cache, q, 1, tile=64)
    _check_decode(cache, q, 1, out, lse)


# ---------------------------------------------------------------------------- the quantiser's scale
def _quantise_row_exactly(x):
    """I4.quantise_row in rational numbers (a float64 difference rounds where the ends lie 2^53 apart)."""
    F = [Fraction(float(v)) for v in x]
    lo, hi = min(Fraction(0), *F), max(Fraction(0), *F)
    m, e = 8, -129                                           # m 2^e: from 2^-126 on
    while 15 * m * Fraction(2) ** e < hi - lo:
        m, e = (m + 1, e) if m < 15 else (8, e + 1)
    s = m * Fraction(2) ** e
    z = round(-lo / s)                                       # ties to even
    return np.array([min(15, max(0, round(v / s) + z)) for v in F]), float(s), z


def test_the_scale_covers_the_range_exactly(monkeypatch):
    """Rows whose hi - lo is no fp32 number: 15 s = hi and a lo below hi's last place make the next larger scale the
    smallest one that covers the range."""
    rng = np.random.default_rng(123)
    for _ in range(50):                                      # the two oracles agree where both are exact
        x = I4.bf16(rng.standard_normal(64) * 2.0 ** rng.integers(-20, 20))
        for a, b in zip(I4.quantise_row(x), _quantise_row_exactly(x)):
            assert np.array_equal(a, b)
    monkeypatch.setattr(I4, "quantise_row", _quantise_row_exactly)

    def edit(q, k, v):
        for i, (hi, lo) in enumerate([(15.0, -2.0 ** -21), (15.0, -2.0 ** -40), (2.0 ** -21, -15.0), (2.0 ** -100, -15.0),
                                      (15.0, -2.0 ** -133), (15.0 * 2.0 ** 100, -1.0), (120.0, -2.0 ** -16), (8.0, -2.0 ** -30),
                                      (15.0 * 2.0 ** -126, -2.0 ** -133)]):
            v[i] = 0.0
            v[i, 0, 0], v[i, 0, 9], v[i, 1, 64], v[i, 1, 65] = hi, lo, lo, hi
    _append_case([60, 61], [5, 5], hq=4, hkv=2, d=128, P=16, packed=True, seed=122, edit=edit)
    _, s, z = I4.quantise_row([15.0, -2.0 ** -21])
    assert s == 1.125 and z == 0


# ---------------------------------------------------------------------------- second passes
def _spread(cache, seed, span):
    """V scales times powers of two of their own."""
    rng = np.random.default_rng(seed)
    for b, n in enumerate(cache.lens):
        for i, pid in enumerate(cache.table[b, :-(-n // cache.P)]):
            used = min(cache.P, n - cache.P * i)
            w = cache.words[1, pid, :, :used].astype(np.int64)
            cache.words[1, pid, :, :used] = w + (rng.integers(-span, span + 1, w.shape) << 7)


@pytest.mark.parametrize("n_bins", [1, 2, 5])
@pytest.mark.parametrize("hq,T", [(8, 1), (16, 2), (24, 2)])
def test_far_scales_in_many_short_tiles_of_few_bins(hq, T, n_bins):
    """A CTA walks more tiles than it fetches descriptors for at a time, twice over."""
    cache = I4.Cache([16 * 70, 0, 5, 16 * 33 + 1], Hkv=2, d=128, P=16, seed=171)
    _spread(cache, 172, 40)
    q = I4.bf16(np.random.default_rng(173).standard_normal((4, T, hq, 128)))
    out, lse = _decode(cache, q, T, tile=16, n_bins=n_bins)
    _check_decode(cache, q, T, out, lse)


def test_far_scales_in_one_tile_of_a_ctas_many():
    """The tiles that need no second pass come out as in the first."""
    cache = I4.Cache([640, 300], Hkv=2, d=128, P=16, seed=174)
    q = I4.bf16(np.random.default_rng(175).standard_normal((2, 2, 8, 128)))
    ref = _decode(cache, q, 2, tile=64, n_bins=3)
    _add_exponent(cache, 1, 0, 1, 300, 60)
    out, lse = _decode(cache, q, 2, tile=64, n_bins=3)
    _check_decode(cache, q, 2, out, lse)
    assert np.array_equal(out[1], ref[0][1]) and np.array_equal(lse[1], ref[1][1])
    assert np.array_equal(out[0, :, :4], ref[0][0, :, :4]) and np.array_equal(lse[0, :, :4], ref[1][0, :, :4])


def test_far_scales_under_a_block_sparse_plan():
    lens, tile = [900, 64, 0, 2000], 64
    cache = I4.Cache(lens, Hkv=2, d=128, P=16, seed=176)
    _spread(cache, 177, 30)
    q = I4.bf16(np.random.default_rng(178).standard_normal((4, 2, 8, 128)))
    bits = np.random.default_rng(179).random((4, 2, 32)) < 0.4
    bits[0, 1] = False
    mask = (bits.astype(np.uint64) << np.arange(32, dtype=np.uint64)).sum(-1).astype(np.uint32)
    keep = np.repeat(bits, tile, axis=-1)
    out, lse = _decode(cache, q, 2, tile=tile, mask=torch.from_numpy(mask.view(np.int32)[..., None].copy()).cuda())
    _check_decode(cache, q, 2, out, lse, keep=[keep[b][:, :n] for b, n in enumerate(lens)])


def test_far_scales_bad_pages_and_nan_rows_together():
    cache = I4.Cache([500, 300], Hkv=1, d=64, P=16, seed=180)
    _spread(cache, 181, 50)
    q = I4.bf16(np.random.default_rng(182).standard_normal((2, 3, 4, 64)))
    ref = _decode(cache, q, 3, tile=128)
    _check_decode(cache, q, 3, *ref)
    _set_row(cache, 1, 1, 0, 299, 0x7FC0)                    # seen by the last row alone
    dev = cache.to_device()
    dev["tab"][0, 5] = -1
    out, lse = _decode(cache, q, 3, tile=128, dev=dev, expect=da.EDEVICE)
    assert np.isnan(out[1, 2]).all() and np.isnan(lse[1, 2]).all()
    cache.words[1, cache.table[1, 18], 0, 299 % 16] = 0x3F80
    want = _decode(cache, q, 3, tile=128)
    assert np.array_equal(out[1, :2], want[0][1, :2]) and np.array_equal(lse[1, :2], want[1][1, :2])


@pytest.mark.parametrize("span", [0, 40])
@pytest.mark.parametrize("tile", [64, 512])
def test_out_over_q(tile, span):
    """out may be q, also where a second pass reads q again."""
    cache = I4.Cache([64, 40, 500, 0, 3], Hkv=2, d=128, P=16, seed=183)
    if span:
        _spread(cache, 184, span)
    ref_q = I4.bf16(np.random.default_rng(185).standard_normal((5, 2, 24, 128)))
    ref = _decode(cache, ref_q, 2, tile=tile)
    _check_decode(cache, ref_q, 2, *ref)
    dev, q = cache.to_device(), torch.from_numpy(ref_q).to(torch.bfloat16).cuda()
    pl = da.plan(dev["lens"], 2, tile, max_total_kv_tokens=sum(cache.lens))
    out, lse = da.run_int4(q, dev["k"], dev["v"], dev["words"], dev["tab"], dev["lens"], pl, out=q)
    torch.cuda.synchronize()
    assert out is q and np.array_equal(out.to(torch.float64).cpu().numpy(), ref[0])
    assert np.array_equal(lse.to(torch.float64).cpu().numpy(), ref[1])
