"""Calls with stream= from another current stream, the buffers left to the binding: the current stream allocates and
writes at once, so memory that still belonged to the kernels would show in the results."""
import numpy as np
import pytest
import torch

import paged_kv_decode_29_b200 as da
from tests import _int4 as I4

pytestmark = pytest.mark.gpu


def _bf16_dev(x):
    return torch.from_numpy(np.ascontiguousarray(x)).to(torch.float32).to(torch.bfloat16).cuda()


def _int4_calls():
    cache = I4.Cache([3000, 1700, 64], Hkv=4, d=128, P=16, seed=81)
    dev = cache.to_device()
    q = _bf16_dev(I4.bf16(np.random.default_rng(82).standard_normal((3, 4, 16, 128))))
    args = (dev["k"], dev["v"], dev["words"], dev["tab"], dev["lens"])

    def decode(**kw):
        pl = da.plan(dev["lens"], 4, 64, max_total_kv_tokens=4764, **kw)
        return (pl,) + da.run_int4(q, *args, pl, **kw)
    return decode, lambda **kw: (None,) + da.prefill_int4(q, *args, **kw)


def _bf16_calls():
    torch.manual_seed(83)
    n, B = 300, 3
    k, v = (torch.randn((n, 4, 16, 128), device="cuda").to(torch.bfloat16) for _ in range(2))
    tab = torch.randperm(n, device="cuda")[:B * 90].to(torch.int32).view(B, 90).contiguous()
    lens = torch.tensor([1440, 900, 77], dtype=torch.int32, device="cuda")
    q = torch.randn((B, 2, 16, 128), device="cuda").to(torch.bfloat16)
    codes = [(x * 16).to(torch.float8_e4m3fn).view(torch.uint8) for x in (k.float(), v.float())]
    scales = torch.full((2, n, 4), 1 / 16, device="cuda")

    def decode(**kw):
        pl = da.plan(lens, 4, 64, max_total_kv_tokens=2417, **kw)
        return (pl,) + da.run(q, k, v, tab, lens, pl, **kw)
    return decode, lambda **kw: (None,) + da.prefill_fp8(q, *codes, scales, tab, lens, **kw)


@pytest.mark.parametrize("calls", [_int4_calls, _bf16_calls])
@pytest.mark.parametrize("by_handle", [False, True])
def test_a_call_on_another_stream_keeps_its_buffers(calls, by_handle):
    s = torch.cuda.Stream()
    for call in calls():
        _, out, lse = call()
        torch.cuda.synchronize()
        for _ in range(8):
            _, o, m = call(stream=s.cuda_stream if by_handle else s)
            for n in (1 << 16, 1 << 18, 1 << 20, 1 << 22, 1 << 24):  # whatever was just given up, overwritten
                torch.empty(n, dtype=torch.uint8, device="cuda").fill_(0xFF)
            s.synchronize()
            assert torch.equal(o, out) and torch.equal(m, lse)
