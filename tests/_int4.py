"""The INT4 cache in plain 64-bit arithmetic, for the tests: the quantisation of a row, the values of a
cache, and dense attention over them, each written from its definition."""
from __future__ import annotations

import math

import numpy as np
import torch

import oracle


def bf16(x) -> np.ndarray:
    """float64 values -> the nearest bf16 (by way of fp32, as the library rounds), as float64."""
    t = torch.from_numpy(np.ascontiguousarray(x, dtype=np.float64)).to(torch.float32).to(torch.bfloat16)
    return t.to(torch.float64).numpy()


def quantise_row(x):
    """One row of bf16 numbers (float64 [d]) -> (codes int [d], scale, zero point), element by element."""
    if any(not abs(v) < 2.0 ** 127 for v in x):
        return np.zeros(len(x), dtype=np.int64), math.nan, 0
    lo, hi = min(0.0, min(x)), max(0.0, max(x))
    if hi == lo:
        s = 2.0 ** -126
    else:
        need = (hi - lo) / 15.0
        e = math.floor(math.log2(need)) - 5
        m = 8
        while 15.0 * (m * 2.0 ** e) < hi - lo:      # the smallest m 2^e, 8 <= m <= 15, that covers the range
            m += 1
            if m == 16:
                m, e = 8, e + 1
        s = max(m * 2.0 ** e, 2.0 ** -126)
    z = int(np.rint(-lo / s))
    return np.array([min(15, max(0, int(np.rint(v / s)) + z)) for v in x]), s, z


def word_of(s, z) -> int:
    if math.isnan(s):
        return 0x7FC0
    bits = int(np.array(s, dtype=np.float32).view(np.uint32))
    assert bits & 0xFFFFF == 0
    return (bits >> 16) | z


def pack(codes) -> np.ndarray:
    c = np.asarray(codes, dtype=np.uint8)
    return c[..., 0::2] | (c[..., 1::2] << 4)


def quantise(rows):
    """float64 [..., d] (bf16 numbers) -> (packed uint8 [..., d / 2], words uint16 [...], values float64)."""
    flat = np.asarray(rows, dtype=np.float64).reshape(-1, rows.shape[-1])
    codes = np.empty(flat.shape, dtype=np.int64)
    words = np.empty(len(flat), dtype=np.uint16)
    vals = np.empty_like(flat)
    for i, x in enumerate(flat):
        codes[i], s, z = quantise_row(x)
        words[i] = word_of(s, z)
        vals[i] = s * (codes[i] - z)
    lead = rows.shape[:-1]
    return pack(codes).reshape(lead + (rows.shape[-1] // 2,)), words.reshape(lead), vals.reshape(rows.shape)


def values(pool, words) -> np.ndarray:
    """Packed codes uint8 [..., d / 2], words uint16 [...] -> float64 [..., d]."""
    w = np.asarray(words).view(np.uint16).astype(np.uint32)
    s = ((w & 0xFFF0) << 16).view(np.float32).astype(np.float64)
    c = np.stack((pool & 15, pool >> 4), -1).reshape(pool.shape[:-1] + (2 * pool.shape[-1],)).astype(np.float64)
    with np.errstate(invalid="ignore"):
        return (c - (w & 15)[..., None]) * s[..., None]


class Cache:
    """A random INT4 cache of some requests: codes and words anywhere in the format, pages shuffled, and in
    the slots behind each request codes and words at random."""

    def __init__(self, lens, *, Hkv, d, P, seed, spread=1.0, extra_pages=3):
        rng = np.random.default_rng(seed)
        self.lens, self.Hkv, self.d, self.P = [int(x) for x in lens], Hkv, d, P
        per = [-(-n // P) for n in self.lens]
        n = sum(per) + extra_pages
        self.num_pages = n
        perm = rng.permutation(n)
        self.table = np.full((len(per), max(max(per, default=0), 1)), -1, dtype=np.int32)
        at = 0
        for b, m in enumerate(per):
            self.table[b, :m] = perm[at:at + m]
            at += m
        self.pools = [rng.integers(0, 256, (n, Hkv, P, d // 2), dtype=np.uint8) for _ in range(2)]
        self.words = rng.integers(0, 1 << 16, (2, n, Hkv, P), dtype=np.uint16)
        for b, m in enumerate(per):
            for i in range(m):
                used = min(P, self.lens[b] - i * P)
                s = 0.25 * np.exp(spread * rng.standard_normal((2, Hkv, used)))
                bits = (s.astype(np.float32).view(np.uint32) >> 16).astype(np.uint16) & 0xFFF0
                z = rng.integers(5, 11, bits.shape).astype(np.uint16)
                self.words[:, self.table[b, i], :, :used] = bits | z

    def dense(self, which, b):
        """Values of request b as float64 [Hkv][L][d]."""
        L = self.lens[b]
        ids = self.table[b, : -(-L // self.P)]
        v = values(self.pools[which][ids], self.words[which][ids])     # [pages][Hkv][P][d]
        return v.transpose(1, 0, 2, 3).reshape(self.Hkv, len(ids) * self.P, self.d)[:, :L]

    def scales(self, which, b):
        """Row scales of request b as float64 [Hkv][L]."""
        L = self.lens[b]
        ids = self.table[b, : -(-L // self.P)]
        w = self.words[which][ids].astype(np.uint32)                   # [pages][Hkv][P]
        return ((w & 0xFFF0) << 16).view(np.float32).astype(np.float64).transpose(1, 0, 2).reshape(
            self.Hkv, len(ids) * self.P)[:, :L]

    def to_device(self, device="cuda"):
        pools = [torch.from_numpy(p).to(device) for p in self.pools]
        return dict(k=pools[0], v=pools[1], words=torch.from_numpy(self.words.view(np.int16)).to(device),
                    tab=torch.from_numpy(self.table).to(device),
                    lens=torch.tensor(self.lens, dtype=torch.int32, device=device))


def attend(cache, b, q, last, keep=None, sm_scale=0.0):
    """Request b's rows q float64 [T][Hq][d] over the cache; last [T]: the last key that row t sees; keep:
    optional bool [Hkv][L]. Returns (out, lse, mass, reach), mass = sum_j p_j 15 s_j (the codes' range under
    the weights) per row and reach = max_j 15 s_j sum_d |q_d| times the scale: the quantities that the
    tolerances are made of."""
    k, v = cache.dense(0, b), cache.dense(1, b)
    ks, vs = 15 * cache.scales(0, b), 15 * cache.scales(1, b)
    T, Hq, d = q.shape
    Hkv, L, _ = k.shape
    g = Hq // Hkv
    sc = sm_scale if sm_scale > 0 else d ** -0.5
    out, mass = np.zeros((T, Hq, d)), np.zeros((T, Hq))
    lse, reach = np.full((T, Hq), -np.inf), np.zeros((T, Hq))
    for t in range(T):
        n = min(L, int(last[t]) + 1)
        for h in range(Hq if n > 0 else 0):
            sel = np.arange(n) if keep is None else np.flatnonzero(keep[h // g, :n])
            if not len(sel):
                continue
            s = k[h // g, sel] @ q[t, h] * sc
            m = s.max()
            w = np.exp(s - m)
            lse[t, h] = m + np.log(w.sum())
            w /= w.sum()
            out[t, h] = w @ v[h // g, sel]
            mass[t, h] = w @ vs[h // g, sel]
            reach[t, h] = ks[h // g, sel].max() * np.abs(q[t, h]).sum() * sc
    return out, lse, mass, reach


def check(out, lse, ref, weight_rounding=2.0 ** -11, what=""):
    """out / lse against attend()'s result. The tolerances:
      * a score: its products are exact in fp32; they are added in at most 8 steps and the zero point's share
        in one more, each off by at most 2 units of 2^-23 of a running sum that stays below reach: with the
        final products e = 2^-18 reach, which moves lse by e and a weight by a factor of at most e^(2 e);
      * 2^x and log2 in fp32: 2^-20 (1 + |lse|) on lse, 2^-18 on a weight's factor;
      * a weight (times its V scale) is rounded once, relative error weight_rounding; a weight far below the
        largest one may be lost: 2^-24 of mass covers it;
      * out is rounded to bf16: 2^-8 of the value."""
    ref_o, ref_l, mass, reach = ref
    out, lse = np.asarray(out, dtype=np.float64), np.asarray(lse, dtype=np.float64)
    empty = np.isneginf(ref_l)
    assert np.array_equal(np.isneginf(lse), empty), f"{what}: rows without a key differ"
    assert np.all(out[empty] == 0), f"{what}: rows without a key must be 0"
    e = 2.0 ** -18 * reach
    tol_l = e + 2.0 ** -20 * (1 + np.abs(np.where(empty, 0, ref_l)))
    tol_o = 2.0 ** -8 * np.abs(ref_o) + (mass * (weight_rounding + 2.0 ** -18 + 2.0 ** -24 + np.expm1(2 * e)))[..., None]
    d_l = np.abs(np.where(empty, 0, lse) - np.where(empty, 0, ref_l))
    assert np.all(d_l <= tol_l), f"{what}: lse {float((d_l / tol_l).max()):.2f} times its tolerance"
    d_o = np.abs(out - ref_o)
    bad = ~(d_o <= tol_o + 1e-300)
    assert not bad.any(), f"{what}: out {float(np.nanmax(d_o / (tol_o + 1e-300))):.2f} times its tolerance, {int(bad.sum())} elements"
    return float((d_l / tol_l).max(initial=0)), float((d_o / (tol_o + 1e-300)).max(initial=0))


def rotate(x, positions, base=10000.0):
    """Rows float64 [n][heads][d] at positions [n]: the oracle's rotary embedding, rounded to bf16."""
    y = np.empty(x.shape)
    for i, p in enumerate(positions):
        y[i] = oracle.rope_rows(x[i], np.full(x.shape[1], max(int(p), 0)), base)
    return bf16(y)
