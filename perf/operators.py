"""The INT4 KV-cache operators as they are measured: the append of a step's keys and values into a
paged cache held in 4 bits (with the rotary embedding), the decode attention over such a cache,
and the causal prefill over it.

The cache: codes uint8 [num_pages][Hkv][P][d / 2], two to a byte (element 2 i in the low four
bits, 2 i + 1 in the high four), and one 16-bit word per row (page, KV head, slot) in params
[2][num_pages][Hkv][P] (K, then V): the word without its four low bits is the row's scale s as a bf16
bit pattern, its four low bits the zero point z, and element i of the row is s (c_i - z). A scale has
at most four significant bits, so every such value is a bf16 number.
"""
import math
import random

import numpy as np
import torch

own = False

KINDS = ("append", "decode", "prefill", "step")


# ---------------------------------------------------------------------------- the cases
def listed():
    return [
        # one decode step's new tokens of eight sequences: the call whose latency every layer pays
        dict(name="append_b8", kind="append", batch=8, hq=32, hkv=8, d=128, page=16, rows=1, max_rows=1, min_len=512,
             max_len=4096, packed=False, lens=1),
        # speculative tokens of an odd batch over head_dim 64, an odd group of query heads
        dict(name="append_spec_d64", kind="append", batch=37, hq=15, hkv=3, d=64, page=32, rows=4, max_rows=4,
             min_len=2, max_len=3000, packed=False, lens=2),
        # prompts entering the cache: packed rows of several requests
        dict(name="append_prompts", kind="append", batch=12, hq=32, hkv=8, d=128, page=16, rows=300, max_rows=2048,
             min_len=300, max_len=2048, packed=True, lens=3),
        # a short context and one token: latency only
        dict(name="decode_short", kind="decode", batch=2, hq=8, hkv=2, d=128, page=16, rows=1, min_len=100,
             max_len=700, lens=4),
        # a serving batch of equal contexts, four query heads to a KV head
        dict(name="decode_uniform", kind="decode", batch=32, hq=32, hkv=8, d=128, page=16, rows=1, min_len=4096,
             max_len=4096, lens=5),
        # a ragged serving batch, lengths spread over their logarithm
        dict(name="decode_mixed", kind="decode", batch=64, hq=32, hkv=8, d=128, page=16, rows=1, min_len=128,
             max_len=16384, lens=6),
        # one long context, eight query heads to a KV head
        dict(name="decode_long", kind="decode", batch=1, hq=64, hkv=8, d=128, page=64, rows=1, min_len=131072,
             max_len=131072, lens=7),
        # speculative decode: four tokens times four heads, 16 query rows to a KV head
        dict(name="decode_spec", kind="decode", batch=16, hq=32, hkv=8, d=128, page=16, rows=4, min_len=16384,
             max_len=16384, lens=8),
        # head_dim 64, an odd group, five tokens: 25 query rows to a KV head over ragged contexts
        dict(name="decode_d64_wide", kind="decode", batch=9, hq=20, hkv=4, d=64, page=32, rows=5, min_len=3,
             max_len=20000, lens=9),
        # a prompt's own attention, whole prompts of equal length
        dict(name="prefill_prompt", kind="prefill", batch=4, hq=32, hkv=8, d=128, page=16, rows=2048, max_rows=2048,
             min_len=2048, max_len=2048, packed=False, lens=10),
        # ragged chunks of prompts behind cached histories, an odd group of heads
        dict(name="prefill_chunks", kind="prefill", batch=5, hq=15, hkv=5, d=128, page=32, rows=60, max_rows=700,
             min_len=500, max_len=7000, packed=True, lens=11),
        # a decode step as it is used: append, plan, attention
        dict(name="step_b32", kind="step", batch=32, hq=32, hkv=8, d=128, page=16, rows=1, max_rows=1, min_len=600,
             max_len=6000, packed=False, lens=12),
    ]


def _between(rng, lo, hi):
    """A whole number spread over the logarithm of lo .. hi."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)) - 0.3 / hi)))))


def draw(rng):
    kind = rng.choice(KINDS + ("decode",))
    hkv = rng.choice((1, 2, 3, 4, 5, 8))
    d = rng.choice((64, 128, 128))
    page = rng.choice((16, 32, 64))
    lens = rng.randrange(1 << 20)
    if kind == "append":
        packed = rng.random() < 0.5
        rows = 1 if packed else rng.randint(1, 8)
        max_rows = _between(rng, 16, 1500) if packed else rows
        hi = _between(rng, max(max_rows, 64), 4096)
        return dict(kind=kind, batch=_between(rng, 1, 12 if packed else 64), hq=hkv * rng.randint(1, 5), hkv=hkv, d=d,
                    page=page, rows=rows, max_rows=max_rows, min_len=_between(rng, 1, hi), max_len=hi, packed=packed,
                    lens=lens)
    if kind == "decode":
        rows = rng.choice((1, 1, 1, 2, 3, 4, 7, 8))
        group = rng.randint(1, 64 // rows) if rng.random() < 0.2 else rng.randint(1, 8)
        hi = _between(rng, 64, 65536)
        batch = _between(rng, 1, max(1, min(64, (1 << 18) // hi)))
        return dict(kind=kind, batch=batch, hq=hkv * group, hkv=hkv, d=d, page=page, rows=rows,
                    min_len=_between(rng, 1, hi), max_len=hi, lens=lens)
    if kind == "prefill":
        hi = _between(rng, 64, 6000)
        max_rows = _between(rng, 16, min(hi, 1024))
        packed = rng.random() < 0.6
        return dict(kind=kind, batch=_between(rng, 1, 5), hq=hkv * rng.randint(1, 4), hkv=hkv, d=128, page=page,
                    rows=1 if packed else max_rows, max_rows=max_rows, min_len=_between(rng, 16, hi), max_len=hi,
                    packed=packed, lens=lens)
    rows = rng.randint(1, 4)
    hi = _between(rng, 64, 6000)
    return dict(kind=kind, batch=_between(rng, 1, 32), hq=hkv * rng.randint(1, 4), hkv=hkv, d=d, page=page, rows=rows,
                max_rows=rows, min_len=_between(rng, 8, hi), max_len=hi, packed=False, lens=lens)


def _sizes(case):
    """Lengths and query rows of the requests, from the case alone: the lengths count the new rows."""
    r = random.Random(case["lens"])
    n = case["batch"]
    lens = [_between(r, case["min_len"], case["max_len"]) for _ in range(n)]
    lens[0] = case["max_len"]
    if not case.get("packed"):
        return lens, [case["rows"]] * n
    rows = [min(lens[i], _between(r, case["rows"], case["max_rows"])) for i in range(n)]
    return lens, rows


# ---------------------------------------------------------------------------- plain forms
def _quantise(x):
    """Rows x fp32 [..., d] (bf16 numbers) -> (codes uint8 [..., d], scale fp32 [...], zero fp32 [...])."""
    lo = x.amin(-1).clamp(max=0.0)
    hi = x.amax(-1).clamp(min=0.0)
    h = 0.5 * hi - 0.5 * lo
    bits = (h / 7.5).view(torch.int32) & -(1 << 20)         # four significant bits, rounded down
    s = bits.view(torch.float32)
    s = torch.where(7.5 * s < h, (bits + (1 << 20)).view(torch.float32), s).clamp(min=2.0 ** -126)
    z = torch.round(-lo / s)
    codes = (torch.round(x / s[..., None]) + z[..., None]).clamp(0, 15)
    return codes.to(torch.uint8), s, z


def _pack(codes):
    return codes[..., 0::2] | (codes[..., 1::2] << 4)


def _words(s, z):
    return ((s.view(torch.int32) >> 16) | z.to(torch.int32)).to(torch.int16)


def _unpack(pool, params):
    """(codes uint8 [..., d / 2], words int16 [...]) -> fp32 values [..., d]."""
    w = params.to(torch.int32)
    s = ((w & 0xFFF0) << 16).view(torch.float32)
    z = (w & 15).to(torch.float32)
    c = torch.stack((pool & 15, pool >> 4), -1).flatten(-2).to(torch.float32)
    return (c - z[..., None]) * s[..., None]


def _rotate(x, pos, base):
    """Rows x [n][heads][d] at positions pos [n] (not below 0): rotate-half rotary embedding, in 64 bits."""
    half = x.shape[-1] // 2
    theta = torch.pow(torch.tensor(base, dtype=torch.float64, device=x.device),
                      -2.0 * torch.arange(half, dtype=torch.float64, device=x.device) / x.shape[-1])
    ang = pos.clamp(min=0).double()[:, None] * theta
    c, s = torch.cos(ang)[:, None], torch.sin(ang)[:, None]
    a, b = x[..., :half].double(), x[..., half:].double()
    return torch.cat((a * c - b * s, b * c + a * s), -1).float().to(torch.bfloat16)


def _append(st):
    """The plain append: rotated q, the rows' values as the cache gives them back; pools updated in place."""
    pos, page = st["pos"], st["case"]["page"]
    q = _rotate(st["q_new"].flatten(0, -3), pos, st["base"]).view(st["q_new"].shape)
    k = _rotate(st["k_new"].flatten(0, -3), pos, st["base"]).float()
    v = st["v_new"].flatten(0, -3).float()
    has = pos >= 0
    at = pos.clamp(min=0)
    pid = st["table"][st["req"], at // page].long()[has]
    slot = (at % page)[has]
    values = []
    for which, x, pool in ((0, k, st["k_pages"]), (1, v, st["v_pages"])):
        codes, s, z = _quantise(x)
        pool[pid, :, slot] = _pack(codes)[has]
        st["params"][which, pid, :, slot] = _words(s, z)[has]
        values.append(((codes.float() - z[..., None]) * s[..., None]).to(torch.bfloat16).view(st["k_new"].shape))
    return q, values[0], values[1]


def _gather(st, which):
    """K or V of every request, padded: fp32 [B][Hkv][pages * P][d]."""
    pool = (st["k_pages"], st["v_pages"])[which]
    t = st["table"].clamp(min=0).long()
    x = _unpack(pool[t], st["params"][which][t])            # [B][pages][Hkv][P][d]
    return x.permute(0, 2, 1, 3, 4).flatten(2, 3)


def _attend(q, st, last):
    """q bf16 [B][T][Hq][d], last [B][T]: the last key that a row sees (below 0: none).
    Returns (out bf16 [B][T][Hq][d], lse fp32 [B][T][Hq])."""
    B, T, hq, d = q.shape
    hkv = st["case"]["hkv"]
    g = hq // hkv
    k, v = _gather(st, 0), _gather(st, 1)
    key = torch.arange(k.shape[2], device=q.device)
    inside = key < st["lens"][:, None]                       # what lies behind a request is anything at all
    k = torch.where(inside[:, None, :, None], k, 0.0)
    v = torch.where(inside[:, None, :, None], v, 0.0)
    rows = q.float().view(B, T, hkv, g, d).permute(0, 2, 1, 3, 4).flatten(2, 3)       # [B][Hkv][T g][d]
    s = torch.matmul(rows, k.transpose(-1, -2)) / math.sqrt(d)
    sees = (key <= last[..., None])[:, None, :, None].expand(B, 1, T, g, -1).flatten(2, 3)
    s = torch.where(sees, s, -math.inf)
    m = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(m == -math.inf, 0.0, m))
    del s
    l = p.sum(-1, keepdim=True)
    out = torch.matmul(p, v) / torch.where(l > 0, l, 1.0)
    lse = torch.where(l > 0, m + torch.log(l), -math.inf)[..., 0]
    out = out.view(B, hkv, T, g, d).permute(0, 2, 1, 3, 4).reshape(B, T, hq, d)
    return out.to(torch.bfloat16), lse.view(B, hkv, T, g).permute(0, 2, 1, 3).reshape(B, T, hq)


def _decode(st, q):
    T = st["case"]["rows"]
    last = st["lens"][:, None] - T + torch.arange(T, device=q.device)
    return _attend(q, st, last)


def _prefill(st):
    if not st["case"]["packed"]:
        return _decode(st, st["q"])
    B, T = len(st["host_rows"]), max(st["host_rows"])        # packed rows to one padded block and back
    q = torch.zeros((B, T) + st["q"].shape[1:], dtype=torch.bfloat16, device=st["q"].device)
    q[st["req"], st["row"]] = st["q"]
    t = torch.arange(T, device=q.device)
    last = torch.where(t < st["rows"][:, None], st["lens"][:, None] - st["rows"][:, None] + t, -1)
    out, lse = _attend(q, st, last)
    return out[st["req"], st["row"]], lse[st["req"], st["row"]]


# ---------------------------------------------------------------------------- inputs
def _cache(case, lens, gen, device):
    """A filled cache: rows of keys with a few strong channels, as the rotary embedding leaves them, and
    of values; pages in a shuffled order, one page in eight unused, and in the slots behind a request
    whatever the memory held."""
    page, hkv, d = case["page"], case["hkv"], case["d"]
    per = [-(-n // page) for n in lens]
    total = sum(per) + max(1, sum(per) // 8)
    perm = torch.randperm(total, generator=gen, device=device).to(torch.int32)
    width = max(max(per), 1)
    table = torch.full((len(lens), width), -1, dtype=torch.int32, device=device)
    at = 0
    for b, n in enumerate(per):
        table[b, :n] = perm[at:at + n]
        at += n
    pools = []
    params = torch.empty((2, total, hkv, page), dtype=torch.int16, device=device)
    strong = torch.ones((hkv, 1, d), device=device)
    strong[:, :, torch.randperm(d, generator=gen, device=device)[:4]] = 4.0
    step = max(1, (1 << 28) // (hkv * page * d * 4))
    for which in (0, 1):
        pool = torch.empty((total, hkv, page, d // 2), dtype=torch.uint8, device=device)
        for a in range(0, total, step):
            n = min(step, total - a)
            x = torch.randn((n, hkv, page, d), generator=gen, device=device)
            x *= torch.exp(0.3 * torch.randn((n, hkv, page, 1), generator=gen, device=device))
            if which == 0:
                x *= strong
            codes, s, z = _quantise(x.to(torch.bfloat16).float())
            pool[a:a + n] = _pack(codes)
            params[which, a:a + n] = _words(s, z)
        pools.append(pool)
    behind = torch.ones((total, page), dtype=torch.bool, device=device)
    slot = torch.arange(width * page, device=device).view(width, page)
    used = slot[None] < torch.tensor(lens, device=device)[:, None, None]
    ok = table >= 0
    behind[table[ok].long()] = ~used[ok]
    junk = torch.randint(-(1 << 15), 1 << 15, params.shape, generator=gen, device=device, dtype=torch.int32)
    params = torch.where(behind[None, :, None, :], junk.to(torch.int16), params)
    return pools[0], pools[1], params, table


def prepare(case, seed):
    device = torch.device("cuda")
    gen = torch.Generator(device=device)
    gen.manual_seed(int(seed))
    lens, rows = _sizes(case)
    kind, hq, hkv, d = case["kind"], case["hq"], case["hkv"], case["d"]
    st = dict(case=case, base=10000.0, host_lens=lens, host_rows=rows)
    st["k_pages"], st["v_pages"], st["params"], st["table"] = _cache(case, lens, gen, device)
    st["lens"] = torch.tensor(lens, dtype=torch.int32, device=device)
    st["rows"] = torch.tensor(rows, dtype=torch.int32, device=device)
    packed = bool(case.get("packed"))
    n = sum(rows)
    lead = (n,) if packed else (len(lens), case["rows"])
    normal = lambda heads: torch.randn(lead + (heads, d), generator=gen, device=device).to(torch.bfloat16)  # noqa: E731
    if kind in ("append", "step"):
        st["q_new"], st["k_new"], st["v_new"] = normal(hq), normal(hkv), normal(hkv)
    else:
        st["q"] = normal(hq)
    cu = np.concatenate(([0], np.cumsum(rows))).astype(np.int32)
    st["cu"] = torch.from_numpy(cu).to(device) if packed else None
    st["req"] = torch.repeat_interleave(torch.arange(len(lens), device=device), st["rows"].long(), output_size=n)
    st["row"] = torch.arange(n, device=device) - torch.from_numpy(cu[:-1]).to(device).long()[st["req"]]
    st["pos"] = (st["lens"] - st["rows"]).long()[st["req"]] + st["row"]
    if own:
        import paged_kv_decode_29_b200 as da
        # what a serving program keeps from step to step: output buffers, the plan buffer, the workspace,
        # and for the decode alone the step's plan, which all layers share
        empty = lambda shape, dtype: torch.empty(shape, dtype=dtype, device=device)  # noqa: E731
        if kind in ("append", "step"):
            st["q_out"] = torch.empty_like(st["q_new"])
            st["k_values"], st["v_values"] = torch.empty_like(st["k_new"]), torch.empty_like(st["v_new"])
        if kind in ("decode", "step"):
            st["total"] = sum(lens)
            st["tile"] = da.default_tile_len(len(lens), hkv, st["total"], case["page"], d, hq // hkv * case["rows"],
                                             da.KV_INT4)
            st["plan"] = da.plan(st["lens"], hkv, st["tile"], max_total_kv_tokens=st["total"])
            shape = da.ShapeT(len(lens), hq, hkv, d, case["rows"], case["page"], st["k_pages"].shape[0],
                              st["table"].shape[1], da.KV_INT4, 0.0)
            st["workspace"] = empty(da.workspace_bytes(shape, st["plan"]), torch.uint8)
        if kind != "append":
            st["out"] = empty(lead + (hq, d), torch.bfloat16)
            st["lse"] = empty(lead + (hq,), torch.float32)
    return st


# ---------------------------------------------------------------------------- one pass
def run(st):
    kind = st["case"]["kind"]
    if own:
        import paged_kv_decode_29_b200 as da
        if kind in ("append", "step"):
            q = da.append_rope_int4(st["q_new"], st["k_new"], st["v_new"], st["table"], st["lens"], st["k_pages"],
                                    st["v_pages"], st["params"], cu_q_lens=st["cu"], rope_base=st["base"],
                                    q_out=st["q_out"], k_values=st["k_values"], v_values=st["v_values"])
            done = (q, st["k_values"], st["v_values"], st["k_pages"], st["v_pages"], st["params"])
            if kind == "append":
                return done
            pl = da.plan(st["lens"], st["case"]["hkv"], st["tile"], max_total_kv_tokens=st["total"],
                         buf=st["plan"].buf)
            return done + da.run_int4(q, st["k_pages"], st["v_pages"], st["params"], st["table"], st["lens"], pl,
                                      workspace=st["workspace"], out=st["out"], lse=st["lse"])
        if kind == "decode":
            return da.run_int4(st["q"], st["k_pages"], st["v_pages"], st["params"], st["table"], st["lens"],
                               st["plan"], workspace=st["workspace"], out=st["out"], lse=st["lse"])
        return da.prefill_int4(st["q"], st["k_pages"], st["v_pages"], st["params"], st["table"], st["lens"],
                               cu_q_lens=st["cu"], max_q_rows=max(st["host_rows"]), out=st["out"], lse=st["lse"])
    if kind in ("append", "step"):
        q, kv, vv = _append(st)
        done = (q, kv, vv, st["k_pages"], st["v_pages"], st["params"])
        return done if kind == "append" else done + _decode(st, q)
    return _decode(st, st["q"]) if kind == "decode" else _prefill(st)


def work(case):
    lens, rows = _sizes(case)
    kind, hq, hkv, d, page = case["kind"], case["hq"], case["hkv"], case["d"], case["page"]
    n = sum(rows)
    size = flops = 0.0
    row = hkv * (d // 2 + 2) * 2                             # codes and word of K and V of a token
    if kind in ("append", "step"):
        stored = sum(min(r, m) for r, m in zip(rows, lens))
        size += 2 * n * (2 * hq + 4 * hkv) * d               # q in and out; k, v in and their values out
        size += stored * row + 4 * stored                    # the cache, and page ids
        flops += 3.0 * n * (hq + hkv) * d + 6.0 * n * 2 * hkv * d
    if kind != "append":
        size += sum(lens) * row + 4 * sum(-(-m // page) for m in lens)
        size += n * hq * (4 * d + 4)                         # q, out, lse
        seen = sum(max(0, m - r + t + 1) for m, r in zip(lens, rows) for t in range(r))
        flops += 4.0 * d * hq * seen
    return {"bytes": size + 4 * len(lens), "flops": flops}


# ---------------------------------------------------------------------------- in 64 bits
def _exact_row(x):
    """Quantises rows x [n][d] of 64-bit numbers: (codes, scale, zero), straight from the definition:
    s is the smallest number of four significant bits with 15 s >= max(0, x) - min(0, x)."""
    lo, hi = torch.clamp(x.min(-1).values, max=0.0), torch.clamp(x.max(-1).values, min=0.0)
    need = (hi - lo) / 15.0
    mant, ex = torch.frexp(need)                             # need = mant 2^ex, mant in [0.5, 1)
    s = torch.ldexp(torch.ceil(mant * 16.0 - 1e-13), ex - 4)
    s = torch.clamp(s, min=2.0 ** -126)
    z = torch.round(-lo / s)
    return torch.clamp(torch.round(x / s[:, None]) + z[:, None], 0, 15), s, z


def _exact_kv(st, which, b, h):
    """K or V of request b, KV head h, as 64-bit values [L][d]."""
    page, L = st["case"]["page"], st["host_lens"][b]
    ids = st["table"][b, : -(-L // page)].long()
    raw = (st["k_pages"], st["v_pages"])[which][ids, h].reshape(-1, st["case"]["d"] // 2)[:L].to(torch.int64)
    w = st["params"][which][ids, h].reshape(-1)[:L].to(torch.int64) & 0xFFFF
    e, man = (w >> 7) & 255, (w >> 4) & 7                    # exponent and three fraction bits of the scale
    s = torch.ldexp(1.0 + man.double() / 8.0, e - 127)
    c = torch.empty((L, st["case"]["d"]), dtype=torch.float64, device=raw.device)
    c[:, 0::2] = raw.remainder(16).double()
    c[:, 1::2] = raw.div(16, rounding_mode="floor").double()
    return (c - w.remainder(16).double()[:, None]) * s[:, None]


def _exact_attention(st, q):
    """Rows q [n][Hq][d] of all requests, packed."""
    case = st["case"]
    n, hq, d = q.shape
    g = hq // case["hkv"]
    out = torch.zeros((n, hq, d), dtype=torch.float64, device=q.device)
    lse = torch.full((n, hq), -math.inf, dtype=torch.float64, device=q.device)
    at = 0
    for b, (L, T) in enumerate(zip(st["host_lens"], st["host_rows"])):
        last = L - T + torch.arange(T, device=q.device)
        dark = torch.arange(L, device=q.device)[None, :] > last[:, None]
        for h in range(case["hkv"]):
            k, v = _exact_kv(st, 0, b, h), _exact_kv(st, 1, b, h)
            for j in range(h * g, (h + 1) * g):
                s = q[at:at + T, j].double() @ k.t() * d ** -0.5
                s.masked_fill_(dark, -math.inf)
                lse[at:at + T, j] = torch.logsumexp(s, -1)
                w = torch.softmax(s, -1)
                w[last < 0] = 0.0
                out[at:at + T, j] = w @ v
        at += T
    return out, lse


def exact(case, seed):
    st = prepare(case, seed)
    kind = case["kind"]
    if kind in ("append", "step"):
        d = case["d"]
        n = st["pos"].shape[0]
        i = torch.arange(d // 2, dtype=torch.float64, device=st["pos"].device)
        turn = torch.exp(1j * (st["pos"].clamp(min=0).double()[:, None] * _theta(st["base"], i, d)))

        def spin(x):
            x = x.reshape(n, -1, d).double()
            y = torch.complex(x[..., : d // 2], x[..., d // 2:]) * turn[:, None]
            return torch.cat((y.real, y.imag), -1)

        q = spin(st["q_new"])
        rows = (spin(st["k_new"]).float().bfloat16().double(), st["v_new"].reshape(n, case["hkv"], d).double())
        back = []
        page = case["page"]
        for which, x in enumerate(rows):
            codes, s, z = _exact_row(x.reshape(-1, d))
            back.append(((codes - z[:, None]) * s[:, None]).reshape(st["k_new"].shape))
            codes = codes.reshape(n, case["hkv"], d).to(torch.int64)
            s, z = s.reshape(n, -1), z.reshape(n, -1).to(torch.int64)
            mant, ex = torch.frexp(s)
            word = (ex.to(torch.int64) + 126) * 128 + ((mant * 16 - 8).to(torch.int64) << 4) + z
            keep = st["pos"] >= 0
            pid = st["table"][st["req"][keep], st["pos"][keep] // page].long()
            slot = st["pos"][keep] % page
            pool = (st["k_pages"], st["v_pages"])[which]
            pool[pid, :, slot] = (codes[..., 0::2] + 16 * codes[..., 1::2])[keep].to(torch.uint8)
            st["params"][which, pid, :, slot] = word[keep].to(torch.int16)
        head = [q.reshape(st["q_new"].shape), back[0], back[1], st["k_pages"], st["v_pages"], st["params"]]
        if kind == "append":
            return head
        q = q.float().bfloat16()                             # the attention takes the rotated q as it is stored
    else:
        head, q = [], st["q"]
    lead = tuple((st["q"] if "q" in st else st["q_new"]).shape[:-2])
    out, lse = _exact_attention(st, q.reshape(-1, case["hq"], case["d"]))
    return head + [out.reshape(lead + out.shape[1:]), lse.reshape(lead + lse.shape[1:])]


def _theta(base, i, d):
    """The rotary embedding's angles per position, base^(-2 i / d)."""
    return torch.exp(-2.0 * i / d * math.log(base))
