"""A library call recorded into a step without a workspace of the caller's: the
one it allocates lives as long as the step, which writes to it at every launch.
CPU: the binding's bookkeeping over a stand-in library.  GPU: memory allocated
after the recording is left alone by the step's launches."""
import contextlib
import ctypes
import gc
import types
import weakref

import pytest
import torch

from biased_gqa_attention_gb300 import extkv as ek

HANDLE = 0xABC0


class FakeLibrary:
    """Entry points that succeed without doing anything."""

    def extkv_step_begin(self, out):
        out._obj.value = HANDLE
        return 0

    def extkv_step_end(self, stream, out):
        out._obj.value = 0x77
        return 0

    def extkv_step_launch(self, step, stream):
        return 0

    def extkv_step_free(self, step):
        return None

    def extkv_last_error(self):
        return b""

    def __getattr__(self, name):
        return (lambda *a: 4096) if name.endswith(("_size", "_size_dv")) else (lambda *a: 0)


class External:
    def __init__(self, handle, *a):
        self.cuda_stream = handle


noted = []  # streams that workspaces were recorded on


@pytest.fixture
def fake(monkeypatch):
    lib, made = FakeLibrary(), []
    empty = torch.empty

    def noted_empty(*a, **kw):
        t = empty(*a, **kw)
        if t.dtype == torch.uint8:
            made.append(weakref.ref(t))
        return t

    monkeypatch.setattr(ek, "load", lambda *a: lib)
    monkeypatch.setattr(ek, "_lib", lib)
    monkeypatch.setattr(ek, "_on_current_device", lambda **t: None)
    monkeypatch.setattr(torch, "empty", noted_empty)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: types.SimpleNamespace(cuda_stream=5))
    monkeypatch.setattr(torch.cuda, "ExternalStream", External)
    monkeypatch.setattr(torch.cuda, "stream", lambda s: contextlib.nullcontext())
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda self, s: noted.append(s.cuda_stream))
    noted.clear()
    return made


def calls():
    f = torch.bfloat16
    x, c = torch.zeros((2, 4, 1, 64), dtype=f), torch.zeros((2, 2, 32, 64), dtype=f)
    new, at = torch.zeros((2, 2, 1, 64), dtype=f), torch.zeros(2, dtype=torch.int64)
    q, k = torch.zeros((2, 4, 64), dtype=f), torch.zeros((2, 2, 64), dtype=f)
    pages, table = torch.zeros((8, 2, 16, 64), dtype=f), torch.zeros((2, 4), dtype=torch.int64)
    cu = torch.tensor([0, 2])
    return {
        "attention_ext_kv": lambda s: ek.attention_ext_kv(x, x, c, c, at, 1.0, stream=s),
        "attention_ext_kv_scatter": lambda s: ek.attention_ext_kv_scatter(x, x, c, c, new, new, at, at, 1.0, stream=s),
        "attention_paged_decode": lambda s: ek.attention_paged_decode(q, q, pages, pages, table, at, 1.0, stream=s),
        "attention_packed_prefill": lambda s: ek.attention_packed_prefill(q, q, k, k, cu, 1.0, stream=s),
    }


@pytest.mark.parametrize("name", sorted(calls()))
def test_a_step_keeps_the_workspace_that_a_recorded_call_allocated(fake, name):
    call = calls()[name]
    call(None)
    gc.collect()
    assert len(fake) == 1 and fake[0]() is None  # an ordinary call gives its own back
    with ek.StepRecorder() as rec:
        call(rec.stream)
        call(7)  # another stream's call is not the step's
    step = rec.step
    del rec
    gc.collect()
    assert [w() is not None for w in fake] == [False, True, False]
    for stream in (None, None, types.SimpleNamespace(cuda_stream=9), 5, 11, External(12)):
        step(stream)
    assert noted == [5, 9]  # once a stream; a raw handle may be gone when the workspace is freed
    del step
    gc.collect()
    assert all(w() is None for w in fake)
    assert not ek._recording


def test_an_aborted_recording_keeps_nothing(fake):
    with pytest.raises(KeyError):
        with ek.StepRecorder() as rec:
            calls()["attention_paged_decode"](rec.stream)
            raise KeyError
    gc.collect()
    assert fake[0]() is None and not ek._recording
    assert ctypes.c_void_p(HANDLE).value == HANDLE


@pytest.mark.gpu
@pytest.mark.parametrize("op", ["decode", "prefill"])
def test_launches_leave_later_allocations_alone(op):
    import test_gpu_packed_prefill as packed
    import test_gpu_paged_decode as paged
    if op == "decode":
        q, k, v, table, nonpad = paged.make((9000, 700, 33), 8, 4, 128, 16, torch.bfloat16)
        y = torch.empty_like(q)

        def call(stream=None):
            with ek.use_algo(ek.ALGO_DECODE_STREAMK):
                ek.attention_paged_decode(y, q, k, v, table, nonpad, 0.1, stream=stream)
        need = ek.attention_paged_decode_workspace_size(3, 8, 4, 128, torch.bfloat16)
    else:
        q, k, v, cu = packed.make((900, 33, 128), 8, 4, 128, torch.bfloat16)
        y = torch.empty_like(q)

        def call(stream=None):
            ek.attention_packed_prefill(y, q, k, v, cu, 0.1, stream=stream)
        need = ek.attention_packed_prefill_workspace_size(q.shape[0], 3, 8, 4, 128, torch.bfloat16)
    call()
    good = y.clone()
    torch.cuda.synchronize()
    with ek.StepRecorder() as rec:
        call(rec.stream)
        call(rec.stream)
    side = torch.cuda.Stream()
    # blocks of the workspace's size from both pools, as a program that goes on allocates them
    mine = [torch.full((need,), 0x5A, dtype=torch.uint8, device="cuda") for _ in range(4)]
    for stream in (None, side, side.cuda_stream):
        y.zero_()
        torch.cuda.synchronize()
        rec.step(stream)
        torch.cuda.synchronize()
        assert torch.equal(y, good)
        for t in mine:
            assert bool((t == 0x5A).all())
