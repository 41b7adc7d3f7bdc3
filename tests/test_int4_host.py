"""The INT4 cache on the host: the tests' own quantiser against the definition, and every argument check of
the INT4 entry points (each case fails before a launch: no pointer is dereferenced)."""
import ctypes as C

import numpy as np
import pytest

import paged_kv_decode_29_b200 as da
from tests import _int4 as I4

FAKE = 0x7f0000000000


@pytest.fixture(scope="module")
def lib():
    from paged_kv_decode_29_b200 import build
    build.build()
    return da.load_library()


# ---------------------------------------------------------------------------- the format
def _rows():
    rng = np.random.default_rng(1)
    rows = [I4.bf16(rng.standard_normal(64) * s) for s in (1e-38, 1e-3, 1.0, 3e4, 1e37)]
    rows += [np.zeros(64), np.full(64, 1.5), np.full(64, -2.0), I4.bf16(np.abs(rng.standard_normal(64)) + 3)]
    rows.append(np.concatenate((np.zeros(63), [2.0 ** -133])))       # the smallest denormal bf16
    rows.append(np.concatenate((np.full(63, -(2.0 ** 126)), [2.0 ** 126])))
    return rows


def test_quantised_rows_follow_the_definition():
    for x in _rows():
        c, s, z = I4.quantise_row(x)
        assert c.min() >= 0 and c.max() <= 15 and 0 <= z <= 15
        m, _ = np.frexp(s)
        assert m * 16 == int(m * 16) and s >= 2.0 ** -126            # four significant bits
        lo, hi = min(0.0, x.min()), max(0.0, x.max())
        assert 15 * s >= hi - lo
        if s > 2.0 ** -126:                                          # the next smaller scale does not cover the range
            m16, e = int(m * 16), np.frexp(s)[1]
            smaller = (m16 - 1) * 2.0 ** (e - 4) if m16 > 8 else 15 * 2.0 ** (e - 5)
            assert 15 * smaller < hi - lo
        vals = s * (c - z)
        assert np.all(np.abs(vals - x) <= s / 2 * (1 + 2.0 ** -40))
        assert np.array_equal(I4.bf16(vals), vals)                   # every value is a bf16 number
        assert np.all(vals[x == 0] == 0)


def test_a_row_that_is_not_finite_is_a_nan_row():
    for bad in (np.nan, np.inf, -np.inf, 2.0 ** 127, -(2.0 ** 127)):
        x = np.ones(64)
        x[5] = bad
        c, s, z = I4.quantise_row(x)
        assert not c.any() and np.isnan(s) and z == 0 and I4.word_of(s, z) == 0x7FC0


def test_pack_and_values_are_inverse():
    rng = np.random.default_rng(2)
    x = I4.bf16(rng.standard_normal((3, 4, 64)))
    pool, words, vals = I4.quantise(x)
    assert pool.shape == (3, 4, 32) and words.shape == (3, 4)
    assert np.array_equal(I4.values(pool, words), vals)
    assert np.abs(vals - x).max() < 0.3


# ---------------------------------------------------------------------------- argument checks
def _shape(**kw):
    base = dict(batch=2, n_q_heads=8, n_kv_heads=2, head_dim=128, q_tokens=1, page_size=16, num_pages=64,
                max_pages_per_seq=8, kv_dtype=da.KV_INT4, sm_scale=0.0)
    base.update(kw)
    return da.ShapeT(*[base[f] for f, _ in da.ShapeT._fields_])


def _plan(**kw):
    base = dict(buf=0x10000, buf_bytes=1 << 20, batch=2, n_kv_heads=2, tile_len=64, n_bins=8, max_units=64,
                sparse=0, reserved_=0)
    base.update(kw)
    return da.PlanT(*[base[f] for f, _ in da.PlanT._fields_])


def _append(lib, s, total=None, base=10000.0, **ptrs):
    a = dict(qn=FAKE, kn=FAKE, vn=FAKE, tab=FAKE, lens=FAKE, cu=None, qo=FAKE, kp=FAKE, vp=FAKE, w=FAKE, kv=None, vv=None,
             st=None)
    a.update(ptrs)
    total = s.batch * s.q_tokens if total is None else total
    return lib.dec_attn_append_rope_int4(C.byref(s), a["qn"], a["kn"], a["vn"], a["tab"], a["lens"], a["cu"], total, base,
                                         a["qo"], a["kp"], a["vp"], a["w"], a["kv"], a["vv"], a["st"], None)


def test_append_rejects_bad_args(lib):
    s = _shape()
    assert lib.dec_attn_append_rope_int4(None, *[FAKE] * 6, 2, 10000.0, *[FAKE] * 7, None) == da.EINVAL
    for kw, code in ((dict(kv_dtype=da.KV_BF16), da.ENOTSUP), (dict(kv_dtype=da.KV_FP8E4M3), da.ENOTSUP),
                     (dict(head_dim=96), da.ENOTSUP), (dict(head_dim=256), da.ENOTSUP), (dict(batch=-1), da.EINVAL),
                     (dict(q_tokens=0), da.EINVAL), (dict(n_q_heads=6, n_kv_heads=4), da.EINVAL),
                     (dict(page_size=0), da.EINVAL)):
        assert _append(lib, _shape(**kw), total=2) == code
    for base in (0.0, -1.0, float("inf"), float("nan")):
        assert _append(lib, s, base=base) == da.EINVAL
    assert _append(lib, s, total=3) == da.EINVAL                     # no offsets: batch * q_tokens rows
    assert _append(lib, s, total=-1, cu=FAKE) == da.EINVAL
    for name in ("qn", "kn", "vn", "tab", "lens", "qo", "kp", "vp", "w"):
        assert _append(lib, s, **{name: None}) == da.EINVAL
    assert _append(lib, s, kv=FAKE) == da.EINVAL                     # both values or neither
    assert _append(lib, s, vv=FAKE) == da.EINVAL
    for name in ("qn", "kn", "vn", "qo", "kp", "vp"):
        assert _append(lib, s, **{name: FAKE + 8}) == da.EALIGN
        assert _append(lib, _shape(head_dim=64), **{name: FAKE + 4}) == da.EALIGN
    assert _append(lib, s, kv=FAKE + 8, vv=FAKE) == da.EALIGN
    assert _append(lib, s, w=FAKE + 1) == da.EALIGN
    for name in ("tab", "lens", "cu", "st"):
        assert _append(lib, s, **{name: FAKE + 2}) == da.EALIGN
    none = {n: None for n in ("qn", "kn", "vn", "tab", "lens", "qo", "kp", "vp", "w")}
    assert _append(lib, _shape(batch=0), **none) == da.OK
    assert _append(lib, s, total=0, cu=FAKE, **none) == da.OK


def _run(lib, s, p, ws_bytes=1 << 30, **ptrs):
    a = dict(q=FAKE, k=FAKE, v=FAKE, w=FAKE, tab=FAKE, lens=FAKE, ws=FAKE, out=FAKE, lse=FAKE)
    a.update(ptrs)
    return lib.dec_attn_run_int4(C.byref(s), a["q"], a["k"], a["v"], a["w"], a["tab"], a["lens"], C.byref(p), a["ws"],
                                 ws_bytes, a["out"], a["lse"], None)


@pytest.mark.parametrize("kw,plan_kw,code", [
    (dict(kv_dtype=da.KV_BF16), {}, da.ENOTSUP),
    (dict(kv_dtype=da.KV_FP8E4M3), {}, da.ENOTSUP),
    (dict(head_dim=96), {}, da.ENOTSUP),
    (dict(page_size=8), {}, da.ENOTSUP),
    (dict(page_size=48), dict(tile_len=64), da.ENOTSUP),
    (dict(n_q_heads=130), {}, da.ENOTSUP),                    # 65 query rows per KV head
    (dict(q_tokens=9, n_q_heads=2), {}, da.ENOTSUP),
    (dict(batch=3), {}, da.EINVAL),
    (dict(q_tokens=0), {}, da.EINVAL),
    (dict(num_pages=0), {}, da.EINVAL),
    (dict(num_pages=1 << 27), {}, da.ENOTSUP),                # 2^32 rows: row numbers are 32-bit
])
def test_run_rejects_bad_shapes(lib, kw, plan_kw, code):
    assert _run(lib, _shape(**kw), _plan(**plan_kw)) == code


def test_run_rejects_null_misaligned_and_small(lib):
    s, p = _shape(), _plan()
    for name in ("q", "k", "v", "w", "tab", "lens", "ws", "out", "lse"):
        assert _run(lib, s, p, **{name: None}) == da.EINVAL
    for name in ("q", "k", "v", "w", "ws", "out"):
        assert _run(lib, s, p, **{name: FAKE + 8}) == da.EALIGN
    for name in ("tab", "lens", "lse"):
        assert _run(lib, s, p, **{name: FAKE + 2}) == da.EALIGN
    need = lib.dec_attn_workspace_bytes(C.byref(s), C.byref(p))
    assert need > 0 and _run(lib, s, p, ws_bytes=need - 1) == da.ESMALL


def test_entry_points_with_fp32_scales_refuse_the_int4_cache(lib):
    s, p = _shape(), _plan()
    args = (C.byref(s), FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, C.byref(p), FAKE, 1 << 30, FAKE, FAKE, None)
    assert lib.dec_attn_run(*args) == da.ENOTSUP
    assert lib.dec_attn_split(*args) == da.ENOTSUP
    assert lib.dec_attn_combine(*args) == da.ENOTSUP
    assert lib.dec_attn_run_noalloc(C.byref(s), FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, C.byref(p), FAKE, FAKE,
                                    None) == da.ENOTSUP
    assert lib.dec_attn_append_rope(C.byref(s), *[FAKE] * 5, 10000.0, *[FAKE] * 4, None) == da.ENOTSUP
    assert lib.dec_attn_prefill(C.byref(s), *[FAKE] * 8, None) == da.ENOTSUP


def test_prefill_host_checks(lib):
    s = _shape(q_tokens=300)
    B, mpps, Hkv, P = s.batch, s.max_pages_per_seq, s.n_kv_heads, s.page_size
    kv = -(-(B * mpps * Hkv * P * 128 * 2) // 256) * 256
    pools = 2 * kv + -(-(B * mpps * 4) // 256) * 256
    need = lib.dec_attn_prefill_int4_workspace_bytes(C.byref(s))
    assert need == pools                                             # 128 keys at most: one part
    long = _shape(q_tokens=300, max_pages_per_seq=1000)
    wide = 2 * (B * 1000 * Hkv * P * 128 * 2) + -(-(B * 1000 * 4) // 256) * 256
    assert lib.dec_attn_prefill_int4_workspace_bytes(C.byref(long)) == wide + 6 * (B * 300 * 8 * 129 * 4)  # 24 CTAs: 6 parts
    many = _shape(q_tokens=300, n_q_heads=592)                       # a grid that fills the GPU: no parts
    assert lib.dec_attn_prefill_int4_workspace_bytes(C.byref(many)) == pools
    assert lib.dec_attn_prefill_int4_workspace_bytes(C.byref(_shape(q_tokens=0))) == da.EINVAL
    assert lib.dec_attn_prefill_int4_workspace_bytes(None) == da.EINVAL
    assert lib.dec_attn_prefill_int4_workspace_bytes(C.byref(_shape(batch=-1))) == da.EINVAL

    def call(shape, ws_bytes=need, total=None, **kw):
        a = dict(q=FAKE, k=FAKE, v=FAKE, w=FAKE, tab=FAKE, lens=FAKE, cu=None, ws=FAKE, out=FAKE, lse=FAKE, st=None)
        a.update(kw)
        total = shape.batch * shape.q_tokens if total is None else total
        return lib.dec_attn_prefill_int4(C.byref(shape), a["q"], a["k"], a["v"], a["w"], a["tab"], a["lens"], a["cu"],
                                         total, a["ws"], ws_bytes, a["out"], a["lse"], a["st"], None)
    assert lib.dec_attn_prefill_int4(None, *[FAKE] * 7, 1, FAKE, need, FAKE, FAKE, None, None) == da.EINVAL
    for kw, code in ((dict(kv_dtype=da.KV_BF16), da.ENOTSUP), (dict(kv_dtype=da.KV_FP8E4M3), da.ENOTSUP),
                     (dict(head_dim=64), da.ENOTSUP), (dict(page_size=8), da.ENOTSUP), (dict(q_tokens=0), da.EINVAL),
                     (dict(n_q_heads=6, n_kv_heads=4), da.EINVAL), (dict(num_pages=0), da.EINVAL),
                     (dict(batch=70000), da.ENOTSUP)):
        assert call(_shape(**{**dict(q_tokens=300), **kw}), ws_bytes=1 << 60) == code
    assert call(s, total=5) == da.EINVAL
    for name in ("q", "k", "v", "w", "tab", "lens", "ws", "out", "lse"):
        assert call(s, **{name: None}) == da.EINVAL
    for name in ("q", "k", "v", "w", "ws", "out"):
        assert call(s, **{name: FAKE + 8}) == da.EALIGN
    for name in ("tab", "lens", "lse", "st"):
        assert call(s, **{name: FAKE + 2}) == da.EALIGN
    assert call(s, ws_bytes=need - 1) == da.ESMALL
    assert call(_shape(batch=0, q_tokens=300), **{n: None for n in ("q", "k", "v", "w", "tab", "lens", "ws", "out",
                                                                    "lse")}) == da.OK


def test_default_tile_len_of_int4(lib):
    f = lib.dec_attn_default_tile_len
    for P in (16, 32, 48, 256):
        tl = f(8, 8, 100000, P, 128, 4, da.KV_INT4, 592)
        assert tl > 0 and tl % P == 0
    assert f(2, 2, 822, 16, 128, 4, da.KV_INT4, 592) == 64           # tiny: one block of the kernel
    # fewer bytes per key than E4M3: a tile is never shorter
    for total in (2000, 40000, 500000):
        assert f(8, 8, total, 16, 128, 4, da.KV_INT4, 592) >= f(8, 8, total, 16, 128, 4, da.KV_FP8E4M3, 592)
