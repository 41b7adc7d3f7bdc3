"""The INT4 cache on the GPU against plain 64-bit arithmetic (tests/_int4.py), through the binding: the
quantising append bit for bit, decode and prefill within derived tolerances, and the three as a serving
program runs them."""
import numpy as np
import pytest
import torch

import oracle
import paged_kv_decode_29_b200 as da
from tests import _int4 as I4

pytestmark = pytest.mark.gpu

CANARY = 0x5A


def _bf16_dev(x):
    """float64 bf16 numbers -> a bf16 CUDA tensor."""
    return torch.from_numpy(np.ascontiguousarray(x)).to(torch.float32).to(torch.bfloat16).cuda()


def _f64(t):
    return t.to(torch.float64).cpu().numpy()


def _int32(x):
    return torch.tensor(np.asarray(x, dtype=np.int32), device="cuda")


# ---------------------------------------------------------------------------- append
def _new_rows(rng, n, hq, hkv, d):
    q = I4.bf16(rng.standard_normal((n, hq, d)))
    k = I4.bf16(rng.standard_normal((n, hkv, d)) * np.exp(rng.standard_normal((n, hkv, 1))))
    v = I4.bf16(rng.standard_normal((n, hkv, d)) * np.exp(3 * rng.standard_normal((n, hkv, 1))))
    return q, k, v


def _expected(cache, lens, rows, q, k, v, base=10000.0):
    """Pools, words, rotated q and values after the append of packed rows, by the definition."""
    pos = np.concatenate([np.arange(L - T, L) for L, T in zip(lens, rows)]) if len(lens) else np.zeros(0, int)
    req = np.repeat(np.arange(len(rows)), rows)
    qr, kr = I4.rotate(q, pos, base), I4.rotate(k, pos, base)
    pools, words = [p.copy() for p in cache.pools], cache.words.copy()
    vals = []
    for which, x in enumerate((kr, v)):
        codes, wd, val = I4.quantise(x)
        vals.append(val)
        for i in range(len(pos)):
            if pos[i] >= 0:
                pid, slot = cache.table[req[i], pos[i] // cache.P], pos[i] % cache.P
                pools[which][pid, :, slot] = codes[i]
                words[which, pid, :, slot] = wd[i]
    return pools, words, qr, vals


def _append_case(lens, rows, *, hq, hkv, d, P, packed, seed, base=10000.0, pad=0, edit=None, values=True):
    """Runs the append and compares every byte. lens count the new rows; pad: rows behind the last one."""
    rng = np.random.default_rng(seed)
    cache = I4.Cache([max(x, 0) for x in lens], Hkv=hkv, d=d, P=P, seed=seed + 1)
    n = int(sum(rows))
    q, k, v = _new_rows(rng, n, hq, hkv, d)
    if edit:
        edit(q, k, v)
    pools, words, qr, vals = _expected(cache, lens, rows, q, k, v, base)
    dev = cache.to_device()
    lens_dev = _int32(lens)

    def rows_dev(x):
        t = torch.full((n + pad,) + x.shape[1:], 7.0, dtype=torch.bfloat16, device="cuda")
        t[:n] = _bf16_dev(x)
        return t if packed else t.view((len(lens), rows[0]) + x.shape[1:])

    cu = _int32(np.concatenate(([0], np.cumsum(rows)))) if packed else None
    qd, kd, vd = rows_dev(q), rows_dev(k), rows_dev(v)
    q_out = torch.full_like(qd, 3.0)
    kv_vals = [torch.full_like(kd, 3.0) for _ in range(2)] if values else [None, None]
    st = torch.zeros((), dtype=torch.int32, device="cuda")
    got = da.append_rope_int4(qd, kd, vd, dev["tab"], lens_dev, dev["k"], dev["v"], dev["words"], cu_q_lens=cu,
                              rope_base=base, q_out=q_out, k_values=kv_vals[0], v_values=kv_vals[1], status=st)
    torch.cuda.synchronize()
    assert got is q_out and int(st) == da.OK
    flat = _f64(q_out).reshape(n + pad, hq, d)
    assert np.array_equal(flat[:n], qr, equal_nan=True), "rotated q"
    assert np.all(flat[n:] == 3.0), "rows behind the last one"
    assert np.array_equal(dev["k"].cpu().numpy(), pools[0]), "K codes"
    assert np.array_equal(dev["v"].cpu().numpy(), pools[1]), "V codes"
    assert np.array_equal(dev["words"].cpu().numpy().view(np.uint16), words), "words"
    for got_v, want in zip(kv_vals, vals):
        if got_v is not None:
            f = _f64(got_v).reshape(n + pad, hkv, d)
            assert np.array_equal(f[:n], want, equal_nan=True), "values"
            assert np.all(f[n:] == 3.0)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lens,T,hq,hkv,P", [
    ([1], 1, 1, 1, 16),
    ([1, 16, 17, 33, 100], 1, 8, 2, 16),
    ([3, 40, 64, 65], 4, 15, 3, 16),         # pages crossed; an odd group of heads
    ([0, 2, 5, 31], 4, 6, 6, 32),            # an empty request; fewer tokens than new rows
    ([5000, 131072 - 1], 2, 4, 1, 64),       # far positions
    ([200], 130, 5, 5, 48),                  # rows over several pages; a page of 48 slots
])
def test_append_uniform_rows_bit_for_bit(lens, T, hq, hkv, P, d):
    _append_case(lens, [T] * len(lens), hq=hq, hkv=hkv, d=d, P=P, packed=False, seed=len(lens) + T + d)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lens,rows,pad", [
    ([1], [1], 0),
    ([70, 5, 300], [33, 5, 1], 0),
    ([70, 9, 0, 300, 20], [0, 9, 0, 17, 25], 6),   # requests without rows, more rows than length, a padded batch
    ([9], [0], 3),
])
def test_append_packed_rows_bit_for_bit(lens, rows, pad, d):
    _append_case(lens, rows, hq=6, hkv=2, d=d, P=16, packed=True, seed=sum(rows) + pad + d, pad=pad)


def test_append_of_special_rows():
    def edit(q, k, v):
        v[0] = 0.0
        v[1] = 2.5                                          # one sign: zero stays a code
        v[2] = -1.0
        v[3, 0], v[3, 0, 7] = 0.0, 2.0 ** -133              # the smallest bf16
        v[4, 0] = I4.bf16(v[4, 0] * 2.0 ** 120)
        v[4, 1, 0] = 2.0 ** 126
        v[5, 0, 3] = np.nan                                 # NaN rows
        v[5, 1, 3] = np.inf
        v[6, 0, 63] = -(2.0 ** 127)
        v[7, 0] = 0.0
        v[7, 0, 0], v[7, 0, 1] = 15.0, 2.5                  # scale 1, a tie of the rounding
        v[8, 0] = np.where(np.arange(128) % 2, 3.389531389251535e38, -3.389531389251535e38)
        k[9] = 0.0
    _append_case([60, 61], [5, 5], hq=4, hkv=2, d=128, P=16, packed=True, seed=3, edit=edit)


def test_append_without_values_in_place_and_other_base():
    _append_case([77, 12], [3, 3], hq=4, hkv=2, d=128, P=16, packed=False, seed=4, base=500000.0, values=False)
    rng = np.random.default_rng(5)
    cache = I4.Cache([40], Hkv=2, d=64, P=16, seed=6)
    q, k, v = _new_rows(rng, 2, 4, 2, 64)
    dev = cache.to_device()
    qd = _bf16_dev(q).view(1, 2, 4, 64)
    out = da.append_rope_int4(qd, _bf16_dev(k).view(1, 2, 2, 64), _bf16_dev(v).view(1, 2, 2, 64), dev["tab"], dev["lens"],
                              dev["k"], dev["v"], dev["words"], q_out=qd)
    torch.cuda.synchronize()
    assert out is qd and np.array_equal(_f64(qd)[0], I4.rotate(q, [38, 39]))


def test_append_reports_bad_pages_and_offsets_and_leaves_the_rest():
    rng = np.random.default_rng(7)
    cache = I4.Cache([40, 40, 40], Hkv=2, d=128, P=16, seed=8)
    q, k, v = _new_rows(rng, 3, 4, 2, 128)
    good = _expected(cache, [40, 40, 40], [1, 1, 1], q, k, v)
    for bad in (-1, cache.num_pages, 1 << 30):
        dev = cache.to_device()
        dev["tab"][1, 2] = bad
        st = torch.zeros((), dtype=torch.int32, device="cuda")
        da.append_rope_int4(*[_bf16_dev(x).view(3, 1, -1, 128) for x in (q, k, v)], dev["tab"], dev["lens"], dev["k"], dev["v"],
                            dev["words"], status=st)
        torch.cuda.synchronize()
        assert int(st) == da.EDEVICE
        keep = np.ones(cache.num_pages, dtype=bool)
        keep[cache.table[1, 2]] = False                     # that request's page is as it was
        assert np.array_equal(dev["k"].cpu().numpy()[keep], good[0][0][keep])
        assert np.array_equal(dev["k"].cpu().numpy()[~keep], cache.pools[0][~keep])
        assert np.array_equal(dev["words"].cpu().numpy().view(np.uint16)[:, ~keep], cache.words[:, ~keep])
    # a table too short for the position, and offsets outside the rows
    dev = cache.to_device()
    st = torch.zeros((), dtype=torch.int32, device="cuda")
    da.append_rope_int4(*[_bf16_dev(x).view(3, 1, -1, 128) for x in (q, k, v)], dev["tab"], _int32([40, 49, 40]), dev["k"],
                        dev["v"], dev["words"], status=st)
    torch.cuda.synchronize()
    assert int(st) == da.EDEVICE
    for cu in ([0, 1, 2, 9], [0, 2, 1, 3], [1, 2, 2, 3], [-5, 1, 2, 3]):
        dev = cache.to_device()
        st.zero_()
        da.append_rope_int4(*[_bf16_dev(x) for x in (q, k, v)], dev["tab"], dev["lens"], dev["k"], dev["v"], dev["words"],
                            cu_q_lens=_int32(cu), status=st)
        torch.cuda.synchronize()
        assert int(st) == da.EDEVICE or cu == [0, 2, 1, 3]


# ---------------------------------------------------------------------------- decode
def _decode(cache, q, T, *, tile=64, sm_scale=0.0, lens=None, mask=None, n_bins=0, dev=None, expect=da.OK):
    """q float64 [B][T][Hq][d]; plan + run with guard bytes behind every buffer. Returns (out, lse) float64."""
    dev = dev or cache.to_device()
    B, _, hq, d = q.shape
    lens_dev = dev["lens"] if lens is None else _int32(lens)
    total = int(sum(cache.lens))
    pl = (da.plan(lens_dev, cache.Hkv, tile, max_total_kv_tokens=total, n_bins=n_bins) if mask is None else
          da.plan_sparse(lens_dev, mask, cache.Hkv, tile, max_total_kv_tokens=total, n_bins=n_bins))
    shape = da.ShapeT(B, hq, cache.Hkv, d, T, cache.P, cache.num_pages, dev["tab"].shape[1], da.KV_INT4, sm_scale)
    ws = torch.full((da.workspace_bytes(shape, pl) + 256,), CANARY, dtype=torch.uint8, device="cuda")
    ob = torch.full((q.size + 128,), 5.0, dtype=torch.bfloat16, device="cuda")
    lb = torch.full((q.size // d + 64,), 5.0, dtype=torch.float32, device="cuda")
    out, lse = da.run_int4(_bf16_dev(q), dev["k"], dev["v"], dev["words"], dev["tab"], lens_dev, pl, sm_scale=sm_scale,
                           workspace=ws[:-256], out=ob[:-128].view(q.shape), lse=lb[:-64].view(q.shape[:-1]))
    assert da.read_status(pl) == expect
    assert bool((ws[-256:] == CANARY).all()) and bool((ob[-128:] == 5.0).all()) and bool((lb[-64:] == 5.0).all())
    return _f64(out), _f64(lse)


def _check_decode(cache, q, T, out, lse, *, sm_scale=0.0, keep=None, what=""):
    worst = [0.0, 0.0]
    for b, L in enumerate(cache.lens):
        last = L - T + np.arange(T)
        ref = I4.attend(cache, b, q[b], last, None if keep is None else keep[b], sm_scale)
        got = I4.check(out[b], lse[b], ref, what=f"{what} request {b} of {L} keys")
        worst = [max(x, y) for x, y in zip(worst, got)]
    return worst


@pytest.mark.parametrize("hq,hkv,d,T,P,lens,tile", [
    (1, 1, 64, 1, 16, [1], 16),
    (1, 1, 128, 1, 16, [1], 16),
    (4, 1, 64, 1, 16, [17, 300], 64),
    (8, 2, 128, 1, 16, [0, 1, 15, 16, 17, 63, 64, 65, 127, 129, 1000], 64),
    (8, 2, 128, 2, 16, [1, 2, 3, 200, 64], 128),            # rows without a key
    (15, 3, 128, 1, 32, [500, 31, 2000], 256),              # an odd group
    (16, 2, 128, 1, 64, [3000, 64], 512),                   # 8 query rows
    (9, 1, 128, 1, 48, [100, 1500], 96),                    # 9 rows; a page of 48 slots
    (8, 2, 128, 4, 16, [3, 700, 1025], 64),                 # 16 rows
    (8, 2, 64, 4, 16, [3, 700, 1025], 64),
    (20, 4, 64, 5, 32, [3, 4, 2500], 256),                  # 25 rows
    (20, 4, 128, 5, 32, [3, 4, 2500], 256),
    (8, 1, 128, 5, 16, [900], 64),                          # 40 rows
    (64, 1, 128, 1, 16, [1100, 70], 64),                    # 64 rows
    (16, 2, 64, 8, 256, [1100, 70], 256),                   # 64 rows, the largest page
    (10, 5, 128, 3, 16, [4096, 5, 4097], 4096),             # one tile a request
    (3, 3, 64, 1, 16, [3000], 2048),
])
def test_decode_matches_64_bit_attention(hq, hkv, d, T, P, lens, tile):
    cache = I4.Cache(lens, Hkv=hkv, d=d, P=P, seed=hq + T + P)
    q = I4.bf16(np.random.default_rng(hq + d).standard_normal((len(lens), T, hq, d)))
    out, lse = _decode(cache, q, T, tile=tile)
    _check_decode(cache, q, T, out, lse)


@pytest.mark.parametrize("n_bins", [1, 3, 592, 1500])
def test_decode_with_other_bins_and_scale(n_bins):
    cache = I4.Cache([700, 33, 1200], Hkv=2, d=128, P=16, seed=11)
    q = I4.bf16(np.random.default_rng(12).standard_normal((3, 1, 8, 128)))
    out, lse = _decode(cache, q, 1, tile=64, sm_scale=0.02, n_bins=n_bins)
    _check_decode(cache, q, 1, out, lse, sm_scale=0.02)


def test_decode_of_a_long_context_and_peaked_weights():
    """Values whose scales differ by far, and queries that pick out single keys."""
    cache = I4.Cache([20000, 513], Hkv=1, d=128, P=64, seed=13, spread=2.5)
    q = I4.bf16(np.random.default_rng(14).standard_normal((2, 2, 4, 128)) * np.array([0.01, 1.0, 3.0, 30.0])[:, None])
    for tile in (256, 8192):
        out, lse = _decode(cache, q, 2, tile=tile)
        _check_decode(cache, q, 2, out, lse, what=f"tile {tile}")


@pytest.mark.parametrize("qs,ks,vs", [(2.0 ** -60, 2.0 ** 60, 1.0), (2.0 ** 40, 2.0 ** -40, 2.0 ** 100), (1.0, 1.0, 2.0 ** -100)])
def test_decode_of_extreme_magnitudes(qs, ks, vs):
    cache = I4.Cache([300, 40], Hkv=2, d=128, P=16, seed=15)
    for which, factor in ((0, ks), (1, vs)):
        w = cache.words[which].astype(np.int64)             # scales times a power of two: the exponent field
        cache.words[which] = np.where((w >> 7 & 255) + int(np.log2(factor)) > 0, (w + (int(np.log2(factor)) << 7)), w) & 0xFFFF
    q = I4.bf16(np.random.default_rng(16).standard_normal((2, 1, 4, 128)) * qs)
    out, lse = _decode(cache, q, 1, tile=64)
    _check_decode(cache, q, 1, out, lse)


def test_decode_with_a_zero_query_and_constant_rows():
    cache = I4.Cache([100], Hkv=1, d=128, P=16, seed=17)
    cache.words[0] = (cache.words[0] & 0xFFF0) | 8
    cache.pools[0][:] = 0x88                                # every K element zero: equal weights
    q = I4.bf16(np.random.default_rng(18).standard_normal((1, 2, 4, 128)))
    q[0, 0] = 0.0
    out, lse = _decode(cache, q, 2, tile=64)
    _check_decode(cache, q, 2, out, lse)


def test_decode_block_sparse():
    lens, hkv, tile = [900, 64, 0, 2000], 2, 64
    cache = I4.Cache(lens, Hkv=hkv, d=128, P=16, seed=19)
    q = I4.bf16(np.random.default_rng(20).standard_normal((4, 2, 8, 128)))
    rng = np.random.default_rng(21)
    bits = rng.random((4, hkv, 32)) < 0.4
    bits[0, 1] = False                                      # a head without a tile
    mask = (bits.astype(np.uint64) << np.arange(32, dtype=np.uint64)).sum(-1).astype(np.uint32)
    keep = np.repeat(bits, tile, axis=-1)
    out, lse = _decode(cache, q, 2, tile=tile, mask=torch.from_numpy(mask.view(np.int32)[..., None].copy()).cuda())
    _check_decode(cache, q, 2, out, lse, keep=[keep[b][:, :L] for b, L in enumerate(lens)])


def test_a_nan_row_reaches_the_rows_that_see_it_and_no_others():
    lens, T = [70, 200, 300], 4
    cache = I4.Cache(lens, Hkv=2, d=128, P=16, seed=22)
    q = I4.bf16(np.random.default_rng(23).standard_normal((3, T, 4, 128)))
    clean = {tile: _decode(cache, q, T, tile=tile) for tile in (64, 512)}
    for which, b, pos in ((0, 0, 67), (1, 0, 67), (0, 1, 10), (1, 1, 10), (1, 2, 299)):
        pid, slot = cache.table[b, pos // 16], pos % 16
        saved = cache.words[which, pid, 1, slot]
        cache.words[which, pid, 1, slot] = 0x7FC0
        for tile in (64, 512):
            out, lse = _decode(cache, q, T, tile=tile)
            ref, ref_l = clean[tile]
            sees = np.zeros(out.shape[:3], dtype=bool)
            sees[b, :, 2:] = (lens[b] - T + np.arange(T) >= pos)[:, None]
            assert np.isnan(out[sees]).all(), (which, b, pos, tile)
            if which == 0:
                assert np.isnan(lse[sees]).all()
            assert np.array_equal(out[~sees], ref[~sees]) and np.array_equal(lse[~sees], ref_l[~sees])
        cache.words[which, pid, 1, slot] = saved


def test_decode_does_not_depend_on_what_lies_behind_a_request():
    lens = [5, 70, 200]
    cache = I4.Cache(lens, Hkv=2, d=128, P=64, seed=24)
    q = I4.bf16(np.random.default_rng(25).standard_normal((3, 1, 8, 128)))
    a = _decode(cache, q, 1, tile=64)
    rng = np.random.default_rng(26)
    for b, L in enumerate(lens):
        pid, used = cache.table[b, (L - 1) // 64], (L - 1) % 64 + 1
        cache.words[:, pid, :, used:] = rng.choice([0x7FC0, 0xFFFF, 0x7F80, 0, 0x7F7F], cache.words[:, pid, :, used:].shape)
        for p in cache.pools:
            p[pid, :, used:] = 0xFF
    b = _decode(cache, q, 1, tile=64)
    assert np.array_equal(a[0], b[0]) and np.array_equal(a[1], b[1])


def test_decode_reports_bad_pages():
    cache = I4.Cache([100, 300], Hkv=2, d=128, P=16, seed=27)
    q = I4.bf16(np.random.default_rng(28).standard_normal((2, 1, 4, 128)))
    ref = _decode(cache, q, 1, tile=64)
    for bad in (-1, cache.num_pages, 1 << 30):
        dev = cache.to_device()
        dev["tab"][1, 7] = bad
        out, lse = _decode(cache, q, 1, tile=64, dev=dev, expect=da.EDEVICE)
        assert np.array_equal(out[0], ref[0][0])            # the other request is right
    dev = cache.to_device()
    dev["tab"] = dev["tab"][:, :10].contiguous()            # a table too short for request 1
    _decode(cache, q, 1, tile=64, dev=dev, expect=da.EDEVICE)


def test_decode_is_the_same_twice_on_a_stream_and_in_a_graph():
    cache = I4.Cache([700, 1300, 64], Hkv=2, d=128, P=16, seed=29)
    q = I4.bf16(np.random.default_rng(30).standard_normal((3, 2, 8, 128)))
    ref = _decode(cache, q, 2, tile=64)
    _check_decode(cache, q, 2, *ref)
    dev = cache.to_device()
    total = sum(cache.lens)
    bufs = []
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):                              # warm: functions loaded before the capture
        qd = _bf16_dev(q)
        pl = da.plan(dev["lens"], 2, 64, max_total_kv_tokens=total)
        out, lse = da.run_int4(qd, dev["k"], dev["v"], dev["words"], dev["tab"], dev["lens"], pl)
    s.synchronize()
    assert np.array_equal(_f64(out), ref[0]) and np.array_equal(_f64(lse), ref[1])
    # two graphs over one workspace, replayed in turn
    shape = da.ShapeT(3, 8, 2, 128, 2, 16, cache.num_pages, dev["tab"].shape[1], da.KV_INT4, 0.0)
    ws = torch.empty(da.workspace_bytes(shape, pl), dtype=torch.uint8, device="cuda")
    q2 = torch.flip(qd, (0, 1)).contiguous()
    for x in (qd, q2):
        o, m = torch.zeros_like(out), torch.zeros_like(lse)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            pg = da.plan(dev["lens"], 2, 64, max_total_kv_tokens=total)
            da.run_int4(x, dev["k"], dev["v"], dev["words"], dev["tab"], dev["lens"], pg, workspace=ws, out=o, lse=m)
        bufs.append((g, o, m, pg))
    for _ in range(3):
        for g, *_r in bufs:
            g.replay()
    torch.cuda.synchronize()
    assert np.array_equal(_f64(bufs[0][1]), ref[0]) and np.array_equal(_f64(bufs[0][2]), ref[1])
    ref2 = _decode(cache, _f64(q2), 2, tile=64)
    assert np.array_equal(_f64(bufs[1][1]), ref2[0]) and np.array_equal(_f64(bufs[1][2]), ref2[1])


@pytest.mark.parametrize("n_bins", [1, 2, 5])
@pytest.mark.parametrize("hq,T", [(8, 1), (16, 2), (24, 2), (48, 2)])
def test_decode_of_many_short_tiles_in_few_bins(hq, T, n_bins):
    """A CTA walks hundreds of tiles of one block, more than it fetches descriptors for at a time."""
    cache = I4.Cache([16 * 70, 0, 5, 16 * 33 + 1], Hkv=2, d=128, P=16, seed=33)
    q = I4.bf16(np.random.default_rng(34).standard_normal((4, T, hq, 128)))
    out, lse = _decode(cache, q, T, tile=16, n_bins=n_bins)
    _check_decode(cache, q, T, out, lse)


# ---------------------------------------------------------------------------- prefill
def _prefill(cache, q, rows, *, uniform, max_rows=None, pad=0, sm_scale=0.0, expect=da.OK, dev=None, cu=None):
    """q float64 [sum rows][Hq][128]."""
    dev = dev or cache.to_device()
    n, hq = q.shape[:2]
    qd = torch.full((n + pad, hq, 128), 9.0, dtype=torch.bfloat16, device="cuda")
    qd[:n] = _bf16_dev(q)
    lead = (len(rows), rows[0]) if uniform else (n + pad,)
    ob = torch.full(((n + pad) * hq * 128 + 128,), 5.0, dtype=torch.bfloat16, device="cuda")
    lb = torch.full(((n + pad) * hq + 64,), 5.0, dtype=torch.float32, device="cuda")
    need = da.prefill_int4_workspace_bytes(lead + (hq, 128), dev["k"], dev["tab"], max_rows or max(rows))
    ws = torch.full((need + 256,), CANARY, dtype=torch.uint8, device="cuda")
    st = torch.zeros((), dtype=torch.int32, device="cuda")
    if cu is None and not uniform:
        cu = np.concatenate(([0], np.cumsum(rows)))
    out, lse = da.prefill_int4(qd.view(lead + (hq, 128)), dev["k"], dev["v"], dev["words"], dev["tab"], dev["lens"],
                               cu_q_lens=None if uniform else _int32(cu), max_q_rows=max_rows or max(rows),
                               sm_scale=sm_scale, workspace=ws[:-256], out=ob[:-128].view(lead + (hq, 128)),
                               lse=lb[:-64].view(lead + (hq,)), status=st)
    torch.cuda.synchronize()
    assert int(st) == expect
    assert bool((ws[-256:] == CANARY).all()) and bool((ob[n * hq * 128:] == 5.0).all()) and bool((lb[n * hq:] == 5.0).all())
    return _f64(out).reshape(n + pad, hq, 128)[:n], _f64(lse).reshape(n + pad, hq)[:n]


def _check_prefill(cache, q, rows, out, lse, sm_scale=0.0):
    at = 0
    for b, (L, T) in enumerate(zip(cache.lens, rows)):
        ref = I4.attend(cache, b, q[at:at + T], L - T + np.arange(T), sm_scale=sm_scale)
        # the weights are rounded to bf16
        I4.check(out[at:at + T], lse[at:at + T], ref, 2.0 ** -8, what=f"request {b}: {T} rows, {L} keys")
        at += T


@pytest.mark.parametrize("hq,hkv,P,lens,T", [
    (1, 1, 16, [1], 1),
    (4, 2, 16, [130, 128, 257], 130),        # more rows than keys in one request
    (6, 2, 32, [300, 0, 40], 40),            # an odd group; an empty request
    (4, 1, 64, [513], 257),
    (2, 2, 48, [700, 33], 33),
])
def test_prefill_uniform_matches_64_bit_attention(hq, hkv, P, lens, T):
    cache = I4.Cache(lens, Hkv=hkv, d=128, P=P, seed=hq + T)
    q = I4.bf16(np.random.default_rng(T).standard_normal((len(lens) * T, hq, 128)))
    out, lse = _prefill(cache, q, [T] * len(lens), uniform=True)
    _check_prefill(cache, q, [T] * len(lens), out, lse)


@pytest.mark.parametrize("lens,rows,pad", [
    ([300, 40, 129], [1, 40, 129], 0),
    ([500, 20, 0, 64], [160, 0, 3, 64], 37),  # no rows; rows without a key; a padded batch
    ([5000, 700, 130], [257, 130, 1], 3),     # keys split over CTAs: many parts, few, one
    ([2000], [5], 300),                       # far more padding than rows
])
def test_prefill_packed_matches_64_bit_attention(lens, rows, pad):
    cache = I4.Cache(lens, Hkv=2, d=128, P=16, seed=41 + pad)
    q = I4.bf16(np.random.default_rng(42).standard_normal((sum(rows), 6, 128)))
    out, lse = _prefill(cache, q, rows, uniform=False, pad=pad, sm_scale=0.05)
    _check_prefill(cache, q, rows, out, lse, sm_scale=0.05)


def test_prefill_of_more_requests_than_lanes_with_split_keys():
    rng = np.random.default_rng(69)
    lens = [1000, 300] + [int(x) for x in rng.integers(0, 700, 38)]
    rows = [min(n, int(x)) for n, x in zip(lens, rng.integers(0, 9, 40))]
    cache = I4.Cache(lens, Hkv=1, d=128, P=32, seed=70)
    q = I4.bf16(rng.standard_normal((sum(rows), 2, 128)))
    out, lse = _prefill(cache, q, rows, uniform=False, max_rows=8, pad=2)
    _check_prefill(cache, q, rows, out, lse)


def test_prefill_of_single_keys_returns_the_caches_values():
    # one key a request: its weight is 1, and out is the row of V itself
    B, Hkv = 40, 4
    cache = I4.Cache([1] * B, Hkv=Hkv, d=128, P=16, seed=67)
    rng = np.random.default_rng(68)
    for b in range(B):
        pid = cache.table[b, 0]
        for h in range(Hkv):
            i = b * Hkv + h                                   # every zero point; scales 2^-40 .. 15 * 2^37
            s = np.array((8 + i % 8) * 2.0 ** (i % 79 - 42), dtype=np.float32)
            cache.words[1, pid, h, 0] = I4.word_of(s, i // 8 % 16)
            cache.pools[1][pid, h, 0] = (np.arange(64) * 37 + 64 * i) % 256 if i % 2 else rng.integers(0, 256, 64)
    q = I4.bf16(rng.standard_normal((B, Hkv, 128)))
    out, _ = _prefill(cache, q, [1] * B, uniform=True)
    want = np.stack([cache.dense(1, b)[:, 0] for b in range(B)])
    assert np.array_equal(out, want)


def test_prefill_nan_rows_bad_pages_and_offsets():
    lens, rows = [200, 150], [100, 150]
    cache = I4.Cache(lens, Hkv=2, d=128, P=16, seed=43)
    q = I4.bf16(np.random.default_rng(44).standard_normal((250, 4, 128)))
    ref, ref_l = _prefill(cache, q, rows, uniform=False)
    for which in (0, 1):
        pid, slot = cache.table[0, 150 // 16], 150 % 16
        saved = cache.words[which, pid, 1, slot]
        cache.words[which, pid, 1, slot] = 0x7FC0
        out, lse = _prefill(cache, q, rows, uniform=False)
        cache.words[which, pid, 1, slot] = saved
        sees = np.zeros((250, 4), dtype=bool)
        sees[50:100, 2:] = True                              # rows 50 .. 99 sit at positions 150 .. 199
        assert np.isnan(out[sees]).all() and np.isnan(lse[sees]).all()
        assert np.array_equal(out[~sees], ref[~sees]) and np.array_equal(lse[~sees], ref_l[~sees])
    for bad in (-1, cache.num_pages, 1 << 30):
        dev = cache.to_device()
        dev["tab"][0, 3] = bad
        out, _ = _prefill(cache, q, rows, uniform=False, dev=dev, expect=da.EDEVICE)
        assert np.array_equal(out[100:], ref[100:])
    for cu, max_rows in (([0, 100, 400], 300), ([0, 100, 250], 149), ([0, 240, 390], 150), ([-1, 100, 250], 150)):
        out, _ = _prefill(cache, q, rows, uniform=False, cu=cu, max_rows=max_rows, expect=da.EDEVICE)
        if cu[1] == 100 and cu[0] == 0:                      # offsets outside the rows: only that request is not written
            assert np.array_equal(out[:100], ref[:100]) and np.all(out[100:] == 5.0)


def test_prefill_nan_rows_in_split_keys():
    cache = I4.Cache([3000], Hkv=2, d=128, P=16, seed=62)
    q = I4.bf16(np.random.default_rng(63).standard_normal((100, 4, 128)))
    ref, ref_l = _prefill(cache, q, [100], uniform=True)
    for which, pos in ((0, 100), (1, 100), (0, 2950), (1, 2950)):
        pid, slot = cache.table[0, pos // 16], pos % 16
        saved = cache.words[which, pid, 0, slot]
        cache.words[which, pid, 0, slot] = 0x7FC0
        out, lse = _prefill(cache, q, [100], uniform=True)
        cache.words[which, pid, 0, slot] = saved
        sees = np.zeros((100, 4), dtype=bool)
        sees[max(pos - 2900, 0):, :2] = True
        assert np.isnan(out[sees]).all() and np.isnan(lse[sees]).all(), (which, pos)
        assert np.array_equal(out[~sees], ref[~sees]) and np.array_equal(lse[~sees], ref_l[~sees])


def test_prefill_is_the_bf16_prefill_over_the_caches_values():
    """Where the keys are not split: the same kernel over the same numbers, so equal to dec_attn_prefill over the
    values, rounded to bf16."""
    lens, T, hq = [400, 333], 200, 592
    cache = I4.Cache(lens, Hkv=2, d=128, P=16, seed=45)
    q = I4.bf16(np.random.default_rng(46).standard_normal((2 * T, hq, 128)))
    out, lse = _prefill(cache, q, [T, T], uniform=True)
    dev = cache.to_device()
    for b, L in enumerate(lens):                             # the bf16 pools need numbers behind the last key
        pid, used = cache.table[b, (L - 1) // 16], (L - 1) % 16 + 1
        cache.words[:, pid, :, used:] = 0x3F80
    pools = [_bf16_dev(np.nan_to_num(I4.values(cache.pools[w], cache.words[w]), posinf=0, neginf=0)) for w in (0, 1)]
    o2, l2 = da.prefill(_bf16_dev(q).view(2, T, hq, 128), pools[0], pools[1], dev["tab"], dev["lens"])
    assert np.array_equal(_f64(l2).reshape(-1, hq), lse)
    assert np.array_equal(_f64(o2.to(torch.bfloat16)).reshape(-1, hq, 128), out)


def test_prefill_wait_runs_out_then_the_context_is_usable():
    cache = I4.Cache([1000, 700], Hkv=2, d=128, P=16, seed=47)
    q = I4.bf16(np.random.default_rng(48).standard_normal((600, 4, 128)))
    dev = cache.to_device()
    st = torch.zeros((), dtype=torch.int32, device="cuda")
    try:
        da.test_set_waits(1_000_000, 1)
        da.prefill_int4(_bf16_dev(q).view(2, 300, 4, 128), dev["k"], dev["v"], dev["words"], dev["tab"], dev["lens"], status=st)
        torch.cuda.synchronize()
    finally:
        da.test_set_waits(0, -1)
    assert int(st) == da.ETIMEOUT
    out, lse = _prefill(cache, q, [300, 300], uniform=True)
    _check_prefill(cache, q, [300, 300], out, lse)


# ---------------------------------------------------------------------------- as they are used
def test_prompt_then_decode_steps_over_one_cache():
    """A prompt enters the cache packed and attends to itself, then steps of one and of three tokens follow;
    the tokens' keys and values are kept in 64 bits beside the cache, as the append gives them back."""
    rng = np.random.default_rng(51)
    B, hq, hkv, d, P = 3, 8, 2, 128, 16
    prompt, steps = [37, 1, 90], [1, 3, 1]
    total = [n + sum(steps) for n in prompt]
    cache = I4.Cache(total, Hkv=hkv, d=d, P=P, seed=52)
    dev = cache.to_device()
    st = torch.zeros((), dtype=torch.int32, device="cuda")
    have = [0] * B
    for rows in [prompt] + [[t] * B for t in steps]:
        n = sum(rows)
        q, k, v = _new_rows(rng, n, hq, hkv, d)
        have = [h + r for h, r in zip(have, rows)]
        lens, cu = _int32(have), _int32(np.concatenate(([0], np.cumsum(rows))))
        kv = torch.empty((n, hkv, d), dtype=torch.bfloat16, device="cuda")
        vv = torch.empty_like(kv)
        qr = da.append_rope_int4(_bf16_dev(q), _bf16_dev(k), _bf16_dev(v), dev["tab"], lens, dev["k"], dev["v"], dev["words"],
                                 cu_q_lens=cu, k_values=kv, v_values=vv, status=st)
        if rows is prompt:
            out, lse = da.prefill_int4(qr, dev["k"], dev["v"], dev["words"], dev["tab"], lens, cu_q_lens=cu,
                                       max_q_rows=max(rows), status=st)
        else:
            pl = da.plan(lens, hkv, 64, max_total_kv_tokens=sum(have))
            out, lse = da.run_int4(qr.view(B, rows[0], hq, d), dev["k"], dev["v"], dev["words"], dev["tab"], lens, pl)
            assert da.read_status(pl) == da.OK
        torch.cuda.synchronize()
        assert int(st) == da.OK
        now = I4.Cache(have, Hkv=hkv, d=d, P=P, seed=0)
        now.table, now.pools = cache.table, [dev["k"].cpu().numpy(), dev["v"].cpu().numpy()]
        now.words = dev["words"].cpu().numpy().view(np.uint16)
        at = 0
        for b, r in enumerate(rows):
            for which, vals in ((0, kv), (1, vv)):          # the values returned are the cache's
                assert np.array_equal(now.dense(which, b)[:, have[b] - r:].transpose(1, 0, 2), _f64(vals)[at:at + r])
            want = I4.rotate(q[at:at + r], np.arange(have[b] - r, have[b]))
            assert np.array_equal(_f64(qr)[at:at + r], want)
            ref = I4.attend(now, b, want, have[b] - r + np.arange(r))
            rounding = 2.0 ** -8 if rows is prompt else 2.0 ** -11
            I4.check(_f64(out).reshape(-1, hq, d)[at:at + r], _f64(lse).reshape(-1, hq)[at:at + r], ref, rounding)
            at += r


def test_one_plan_serves_every_layer_behind_its_append():
    """plan, then append and attention layer by layer: the attention follows the planner in the first layer and the
    append, whose rows it has to see, in the others. Many requests: the append is the longer kernel."""
    rng = np.random.default_rng(55)
    B, hq, hkv, d, P, layers = 96, 8, 2, 128, 16, 3
    have = [int(x) for x in rng.integers(1, 700, B)]
    lens = _int32(have)
    caches = [I4.Cache(have, Hkv=hkv, d=d, P=P, seed=56 + i) for i in range(layers)]
    devs = [c.to_device() for c in caches]
    rows = [_new_rows(rng, B, hq, hkv, d) for _ in range(layers)]
    dev_rows = [[_bf16_dev(x).view(B, 1, -1, d) for x in r] for r in rows]
    torch.cuda.synchronize()
    for order in ("plan first", "append first"):
        outs = []
        for i in range(layers):
            dev = devs[i]
            if i == 0 and order == "plan first":
                pl = da.plan(lens, hkv, 128, max_total_kv_tokens=sum(have))
            qr = da.append_rope_int4(*dev_rows[i], dev["tab"], lens, dev["k"], dev["v"], dev["words"])
            if i == 0 and order == "append first":
                pl = da.plan(lens, hkv, 128, max_total_kv_tokens=sum(have))
            outs.append((qr,) + da.run_int4(qr, dev["k"], dev["v"], dev["words"], dev["tab"], lens, pl))
        assert da.read_status(pl) == da.OK
        for i in range(layers):
            now = I4.Cache(have, Hkv=hkv, d=d, P=P, seed=56 + i)
            now.pools = [devs[i]["k"].cpu().numpy(), devs[i]["v"].cpu().numpy()]
            now.words = devs[i]["words"].cpu().numpy().view(np.uint16)
            q, out, lse = (_f64(x) for x in outs[i])
            for b in range(B):
                ref = I4.attend(now, b, q[b], np.array([have[b] - 1]))
                I4.check(out[b], lse[b], ref, what=f"{order}, layer {i}, request {b}")
            for d_, orig in zip(("k", "v"), caches[i].pools):    # as before the append, for the next order
                devs[i][d_].copy_(torch.from_numpy(orig))
            devs[i]["words"].copy_(torch.from_numpy(caches[i].words.view(np.int16)))


def test_pools_beyond_32_bit_offsets():
    """The same cache with its pages at the end of pools of 5 GB: appended to, decoded and prefilled alike."""
    cache = I4.Cache([700, 300], Hkv=8, d=128, P=64, seed=57)
    small = cache.to_device()
    shift = 160_000                                          # rows from 82 million, bytes from 5.2 billion on
    n = shift + cache.num_pages
    large = dict(k=torch.zeros((n, 8, 64, 64), dtype=torch.uint8, device="cuda"),
                 v=torch.zeros((n, 8, 64, 64), dtype=torch.uint8, device="cuda"),
                 words=torch.zeros((2, n, 8, 64), dtype=torch.uint16, device="cuda").view(torch.int16),
                 tab=torch.where(small["tab"] >= 0, small["tab"] + shift, small["tab"]), lens=small["lens"])
    large["k"][shift:], large["v"][shift:], large["words"][:, shift:] = small["k"], small["v"], small["words"]
    rng = np.random.default_rng(58)
    rows = [_bf16_dev(x).view(2, 3, -1, 128) for x in _new_rows(rng, 6, 16, 8, 128)]
    res = []
    for dev in (small, large):
        st = torch.zeros((), dtype=torch.int32, device="cuda")
        q = da.append_rope_int4(*rows, dev["tab"], dev["lens"], dev["k"], dev["v"], dev["words"], status=st)
        pl = da.plan(dev["lens"], 8, 256, max_total_kv_tokens=1000)
        res.append((q,) + da.run_int4(q, dev["k"], dev["v"], dev["words"].view(torch.uint16), dev["tab"], dev["lens"], pl)
                   + da.prefill_int4(q, dev["k"], dev["v"], dev["words"], dev["tab"], dev["lens"], status=st))
        assert da.read_status(pl) == da.OK and int(st) == da.OK
    for x, y in zip(*res):
        assert torch.equal(x, y)
    assert torch.equal(small["k"], large["k"][shift:]) and torch.equal(small["v"], large["v"][shift:])
    assert torch.equal(small["words"], large["words"][:, shift:])
    assert not large["k"][:shift].any() and not large["v"][:shift].any()


def test_two_streams_at_once():
    caches = [I4.Cache([4000, 900, 64], Hkv=4, d=128, P=16, seed=64 + i) for i in range(2)]
    qs = [I4.bf16(np.random.default_rng(66 + i).standard_normal((3, 2, 16, 128))) for i in range(2)]
    ref = [_decode(c, q, 2, tile=128) for c, q in zip(caches, qs)]
    devs, dq, streams = [c.to_device() for c in caches], [_bf16_dev(q) for q in qs], [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(10):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                d = devs[i]
                pl = da.plan(d["lens"], 4, 128, max_total_kv_tokens=4964)
                got[i].append((pl,) + da.run_int4(dq[i], d["k"], d["v"], d["words"], d["tab"], d["lens"], pl))
    torch.cuda.synchronize()
    for i in range(2):
        for _, out, lse in got[i]:
            assert np.array_equal(_f64(out), ref[i][0]) and np.array_equal(_f64(lse), ref[i][1])


def test_the_binding_refuses_what_it_can_see():
    cache = I4.Cache([40, 50], Hkv=2, d=128, P=16, seed=61)
    dev = cache.to_device()
    q = torch.zeros((2, 1, 4, 128), dtype=torch.bfloat16, device="cuda")
    kv = torch.zeros((2, 1, 2, 128), dtype=torch.bfloat16, device="cuda")
    pl = da.plan(dev["lens"], 2, 64, max_total_kv_tokens=90)
    pools = (dev["k"], dev["v"], dev["words"])

    def run(q=q, k=dev["k"], v=dev["v"], w=dev["words"], tab=dev["tab"], lens=dev["lens"], **kw):
        return da.run_int4(q, k, v, w, tab, lens, pl, **kw)
    for kw in (dict(q=q.float()), dict(k=dev["k"].to(torch.int8)), dict(w=dev["words"].to(torch.int32)),
               dict(tab=dev["tab"].long()), dict(lens=dev["lens"].long())):
        with pytest.raises(TypeError):
            run(**kw)
    for kw in (dict(q=q[:1]), dict(q=q[0]), dict(k=dev["k"][..., :32]), dict(w=dev["words"][:1]), dict(tab=dev["tab"][:1]),
               dict(q=q.cpu()), dict(q=torch.zeros((2, 1, 128, 4), dtype=torch.bfloat16, device="cuda").transpose(2, 3)),
               dict(out=torch.empty((2, 1, 4, 128), device="cuda")), dict(lse=torch.empty((2, 4, 1), device="cuda")),
               dict(tab=torch.zeros((4, 2), dtype=torch.int32, device="cuda").t())):
        with pytest.raises(ValueError):
            run(**kw)
    with pytest.raises(da.DecAttnError):
        run(workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        da.append_rope_int4(q, kv[:, :, :1], kv, dev["tab"], dev["lens"], *pools)
    with pytest.raises(ValueError):
        da.append_rope_int4(q, kv, kv.float(), dev["tab"], dev["lens"], *pools)
    with pytest.raises(da.DecAttnError):
        da.append_rope_int4(q, kv, kv, dev["tab"], dev["lens"], *pools, k_values=torch.empty_like(kv))
    with pytest.raises(ValueError):
        da.prefill_int4(q[0], *pools, dev["tab"], dev["lens"])
    with pytest.raises(da.DecAttnError):                     # packed rows need their largest count
        da.prefill_int4(q[:, 0].contiguous(), *pools, dev["tab"], dev["lens"], cu_q_lens=_int32([0, 1, 2]))
    out, lse = run()
    torch.cuda.synchronize()
    assert out.dtype == torch.bfloat16 and lse.dtype == torch.float32
