"""Host threads that share a stream, without a GPU: a call that takes a cached workspace and
several launches is not interrupted by another's.  The library is a fake that records when it
is entered and left; tensors are stand-ins that are asked for their shapes and addresses only."""

import threading
import time

import pytest
import torch

from quantized_weight_dequantization_gb300 import _attention, _binding

STREAM = 0x70


class Tensor:
    """What the binding asks of a contiguous CUDA tensor."""

    is_cuda = True
    device = torch.device("cuda", 0)

    def __init__(self, shape, dtype):
        self.shape, self.dtype = torch.Size(shape), dtype
        self._stride = torch.empty(shape, device="meta").stride()

    def get_device(self):
        return 0

    def dim(self):
        return len(self.shape)

    def numel(self):
        return self.shape.numel()

    def stride(self, i=None):
        return self._stride if i is None else self._stride[i]

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return 1 << 12


class Library:
    """Entry points that take a while, as two launches do, and the order of their events."""

    def __init__(self):
        self.events = []

    def __getattr__(self, name):
        if name.endswith("_bytes"):
            return lambda *a: 256

        def call(*args):
            self.events.append("in")
            time.sleep(0.02)
            self.events.append("out")
            return 0

        return call


@pytest.fixture
def library(monkeypatch):
    lib = Library()
    monkeypatch.setattr(_attention, "_lib", lambda: lib)
    monkeypatch.setattr(_binding, "_LIB", lib)
    monkeypatch.setattr(_binding, "get_lib", lambda: lib)
    _attention._attention_need.cache_clear()
    _attention._norm_need.cache_clear()
    yield lib
    _attention._attention_need.cache_clear()
    _attention._norm_need.cache_clear()


def attention(stream):
    i32, f8 = torch.int32, torch.float8_e4m3fn
    page = Tensor((4, 2, 16, 64), f8)
    cache = _attention.KV8Cache(page, page, Tensor((4, 2), torch.float32),
                                Tensor((4, 2), torch.float32))
    q = Tensor((6, 4, 64), torch.float16)
    _attention.kv8_attention(cache, q, Tensor((2, 3), i32), Tensor((2,), i32), Tensor((3,), i32),
                             out=Tensor((6, 4, 64), torch.float16), stream=stream,
                             workspace=Tensor((256,), torch.uint8))


def out_prod(stream):
    u8, f32 = torch.uint8, torch.float32
    _binding.out_prod(Tensor((2048,), u8), Tensor((64,), u8), Tensor((1,), f32),
                      Tensor((256,), f32), Tensor((16,), f32), 0.0, 64, 64, Tensor((64, 8), f32),
                      dst=Tensor((64, 8), f32), workspace=Tensor((64,), f32), stream=stream)


def run(calls):
    start = threading.Barrier(len(calls))

    def one(call, stream):
        start.wait()
        call(stream)

    threads = [threading.Thread(target=one, args=c) for c in calls]
    for t in threads:
        t.start()
    for t in threads:
        t.join()


@pytest.mark.parametrize("call", [attention, out_prod])
def test_calls_on_one_stream_do_not_interrupt_each_other(library, call):
    run([(call, STREAM)] * 4)
    assert library.events == ["in", "out"] * 4


def test_calls_on_different_streams_do_not_wait_for_each_other(library):
    run([(attention, STREAM + i) for i in range(4)])
    assert library.events.count("in") == 4 and library.events != ["in", "out"] * 4


def test_one_lock_for_a_device_and_stream():
    locks = []
    run([(lambda s: locks.append(_binding._call_lock(3, s)), 5)] * 8)
    assert len(set(map(id, locks))) == 1
    assert _binding._call_lock(3, 6) is not locks[0]
