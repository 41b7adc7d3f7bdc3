"""Buffers that the binding makes itself for a call with stream=: their memory has to belong to the stream that the
kernels run on, and results have to be kept from it while the caller's stream uses them. Checked on the host, with
stand-ins for the library and for torch's streams."""
import contextlib

import pytest
import torch

import paged_kv_decode_29_b200 as da

HERE, THERE = 0x1000, 0x2000


class Stream:
    def __init__(self, handle):
        self.cuda_stream = handle

    def __eq__(self, other):
        return self.cuda_stream == other.cuda_stream


class Library:
    """Every call succeeds; sizes are 256 bytes."""

    def __init__(self):
        self.streams = []

    def __getattr__(self, name):
        def call(*args):
            if name.endswith("_bytes"):
                return 256
            self.streams.append(args[-1])
            return da.OK
        return call


@pytest.fixture
def world(monkeypatch):
    """Records (stream current at the allocation, result kept for) of each tensor made; lib.streams: of the launches."""
    lib, made, current = Library(), [], [Stream(HERE)]
    monkeypatch.setattr(da, "_lib", lib)
    monkeypatch.setattr(da, "load_library", lambda *a: lib)
    monkeypatch.setattr(da, "_raw_stream", lambda device: current[-1].cuda_stream)

    @contextlib.contextmanager
    def use(s):
        current.append(s or current[-1])
        yield
        current.pop()
    monkeypatch.setattr(torch.cuda, "stream", use)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: current[-1])
    monkeypatch.setattr(torch.cuda, "default_stream", lambda device=None: Stream(0))
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle, device=None: Stream(handle))
    monkeypatch.setattr(torch.cuda, "current_device", lambda: -1)      # where a CPU tensor says it is
    empty, empty_like = torch.empty, torch.empty_like

    def note(t):
        made.append([current[-1].cuda_stream, None, t])
        return t
    monkeypatch.setattr(torch, "empty", lambda *a, **kw: note(empty(*a, **kw)))
    monkeypatch.setattr(torch, "empty_like", lambda *a, **kw: note(empty_like(*a, **kw)))

    def record(t, s):
        next(m for m in made if m[2] is t)[1] = s.cuda_stream
    monkeypatch.setattr(torch.Tensor, "record_stream", record)
    return lib, made


def _calls():
    bf = torch.bfloat16
    q, kv = torch.zeros((2, 1, 4, 128), dtype=bf), torch.zeros((2, 1, 2, 128), dtype=bf)
    tab, lens = torch.zeros((2, 1), dtype=torch.int32), torch.ones(2, dtype=torch.int32)
    wide = [torch.zeros((2, 2, 16, 128), dtype=bf) for _ in range(2)]
    codes = [torch.zeros((2, 2, 16, 128), dtype=torch.uint8) for _ in range(2)]
    nib = [torch.zeros((2, 2, 16, 64), dtype=torch.uint8) for _ in range(2)]
    words, scales = torch.zeros((2, 2, 2, 16), dtype=torch.int16), torch.zeros((2, 2, 2))
    cu = torch.tensor([0, 1, 2], dtype=torch.int32)
    pl = da.Plan(buf=torch.zeros(16, dtype=torch.uint8), handle=da.PlanT())
    # name -> (call, tensors returned, tensors made and dropped)
    return {
        "run": (lambda **kw: da.run(q, *wide, tab, lens, pl, **kw), 2, 1),
        "run_int4": (lambda **kw: da.run_int4(q, *nib, words, tab, lens, pl, **kw), 2, 1),
        "append_rope": (lambda **kw: da.append_rope(q, kv, kv, tab, lens, *wide, **kw), 1, 0),
        "append_rope_fp8": (lambda **kw: da.append_rope_fp8(q, kv, kv, tab, lens, *codes, scales, **kw), 1, 0),
        "append_rope_int4": (lambda **kw: da.append_rope_int4(q, kv, kv, tab, lens, *nib, words, **kw), 1, 0),
        "prefill": (lambda **kw: da.prefill(q, *wide, tab, lens, **kw), 2, 0),
        "prefill_varlen": (lambda **kw: da.prefill_varlen(q[:, 0], *wide, tab, lens, cu, 1, **kw), 2, 0),
        "prefill_fp8": (lambda **kw: da.prefill_fp8(q, *codes, scales, tab, lens, **kw), 2, 1),
        "prefill_int4": (lambda **kw: da.prefill_int4(q, *nib, words, tab, lens, **kw), 2, 1),
        "plan": (lambda **kw: da.plan(lens, 2, 16, 2, **kw).buf, 1, 0),
        "plan_sparse": (lambda **kw: da.plan_sparse(lens, torch.zeros((2, 2, 1), dtype=torch.int32), 2, 16, 2, **kw).buf, 1, 0),
    }


@pytest.fixture(autouse=True)
def on_the_device(monkeypatch):
    monkeypatch.setattr(torch.Tensor, "is_cuda", True, raising=False)


@pytest.mark.parametrize("name", list(_calls()))
@pytest.mark.parametrize("stream,handle", [(Stream(THERE), THERE), (THERE, THERE), (0, None)])
def test_buffers_belong_to_the_stream_of_the_call(world, name, stream, handle):
    lib, made = world
    call, results, dropped = _calls()[name]
    made.clear()
    call(stream=stream)
    assert lib.streams == [handle]
    assert [m[0] for m in made] == [handle or 0] * (results + dropped)
    assert sorted((m[1] for m in made), key=str) == sorted([HERE] * results + [None] * dropped, key=str)


@pytest.mark.parametrize("name", list(_calls()))
@pytest.mark.parametrize("stream", [None, Stream(HERE), HERE])
def test_buffers_of_a_call_on_the_current_stream(world, name, stream):
    lib, made = world
    call, results, dropped = _calls()[name]
    made.clear()
    call(stream=stream)
    assert lib.streams == [HERE]
    assert [m[:2] for m in made] == [[HERE, None]] * (results + dropped)


@pytest.mark.parametrize("stream,where", [(Stream(THERE), THERE), (THERE, THERE), (HERE, HERE), (None, HERE)])
def test_a_plans_contents_are_read_behind_their_export(world, monkeypatch, stream, where):
    lib, made = world
    pl = da.Plan(buf=torch.zeros(128, dtype=torch.uint8), handle=da.PlanT(n_bins=3, max_units=2))
    lens, read, cpu, item = torch.ones(2, dtype=torch.int32), [], torch.Tensor.cpu, torch.Tensor.item

    def at(f):
        def g(t):
            read.append(torch.cuda.current_stream().cuda_stream)
            t.zero_() if t.dtype == torch.int32 else None
            return f(t)
        return g
    monkeypatch.setattr(torch.Tensor, "cpu", at(cpu))
    monkeypatch.setattr(torch.Tensor, "item", at(item))
    made.clear()
    assert da.plan_contents(pl, lens, stream=stream)["n_units"] == 0
    assert lib.streams == [where] and [m[0] for m in made] == [where] * 3 and read == [where] * 4
