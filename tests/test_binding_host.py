"""The binding without a GPU: the device that is current when it calls the
library, and the stream it hands over, from tensors that only say where they
are."""

from contextlib import contextmanager

import pytest
import torch

import masked_varlen_prefill_gb300 as mvp
from masked_varlen_prefill_gb300 import _cache, _lib

DEV = torch.device("cuda", 1)
I32, F32, BF16 = torch.int32, torch.float32, torch.bfloat16


class FakeTensor:
    """What the binding asks a tensor on the second GPU."""

    is_cuda = True
    device = DEV

    def __init__(self, shape, dtype=I32):
        self.shape, self.dtype = torch.Size(shape), dtype

    def dim(self):
        return len(self.shape)

    def is_contiguous(self):
        return True

    def stride(self):
        return torch.empty(self.shape, device="meta").stride()

    def numel(self):
        return self.shape.numel()

    def element_size(self):
        return self.dtype.itemsize

    def data_ptr(self):
        return 1 << 20


class FakeLibrary:
    """Notes the device that is current in each call."""

    def __init__(self, calls, current):
        self._calls, self._current = calls, current

    def __getattr__(self, name):
        def call(*args):
            self._calls.append((name, self._current[0], args))
            return mvp.MVP_OK

        return call


@pytest.fixture
def calls(monkeypatch):
    """The calls that reach the library while GPU 0 is current."""
    made, current = [], [0]

    @contextmanager
    def device(dev):
        before, current[0] = current[0], torch.device(dev).index
        yield
        current[0] = before

    lib = FakeLibrary(made, current)
    for module in (_lib, _cache):
        monkeypatch.setattr(module, "load_library", lambda: lib)
    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: current[0])
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda index: 100 + index, raising=False)
    return made


def _packed():
    q, k = FakeTensor((6, 4, 64), BF16), FakeTensor((9, 2, 64), BF16)
    return q, k, FakeTensor((9, 2, 64), BF16), FakeTensor((6, 4, 64), BF16), FakeTensor((3,)), FakeTensor((3,)), 5, 7


def _paged():
    q, k, v, out, cu, _, a, b = _packed()
    k, v = FakeTensor((32, 2, 64), BF16), FakeTensor((32, 2, 64), BF16)
    return q, k, v, out, cu, FakeTensor((2,)), FakeTensor((2, 4)), 16, a, b


def _rope():
    q, k, v, out, cu, sl, bt, _, _, _ = _paged()
    new = FakeTensor((6, 2, 64), BF16)
    return q, new, new, out, k, v, FakeTensor((1, 6)), mvp.RopeTable(FakeTensor((16, 4)), 1), cu, sl, bt, 16


def _weights():
    q, k, _, _, cu, sl, bt, block, a, b = _paged()
    return q, k, FakeTensor((4, 6), F32), FakeTensor((2, 2, 7), F32), cu, sl, bt, block, a, b


def _evict():
    _, k, v, _, _, sl, bt, block, _, b = _paged()
    return (k, v, FakeTensor((2, 2, 7), F32), sl, bt, block, 4, FakeTensor((2,)), FakeTensor((2, 2, 4)),
            FakeTensor((512,), torch.uint8), b)


def _key_weights_packed():
    q, k, _, _, cu, cu_k, a, b = _packed()
    return q, k, FakeTensor((4, 6), F32), FakeTensor((2, 2, 7), F32), cu, cu_k, a, b


CALLS = [
    ("mvp_fill_query_ranges", lambda **kw: mvp.fill_query_ranges(FakeTensor((2, 3, 2)), FakeTensor((3,)),
                                                                 FakeTensor((2,)), FakeTensor((6, 2)), 6, **kw)),
    ("mvp_attn_fwd_varlen", lambda **kw: mvp.attn_fwd_varlen(*_packed(), **kw)),
    ("mvp_attn_fwd_varlen_first", lambda **kw: mvp.attn_fwd_varlen(*_packed(), window_left=3, first_tokens=2, **kw)),
    ("mvp_attn_fwd_varlen_ext", lambda **kw: mvp.attn_fwd_varlen(*_packed(), mixed_prefill_sms=-1, **kw)),
    ("mvp_attn_fwd_varlen_scan", lambda **kw: mvp.attn_fwd_varlen_scan(*_packed(), FakeTensor((2, 3, 2)), **kw)),
    ("mvp_attn_fwd_varlen_static_ws", lambda **kw: mvp.attn_fwd_varlen_static_ws(*_packed(), **kw)),
    ("mvp_attn_fwd_paged", lambda **kw: mvp.attn_fwd_paged(*_paged(), **kw)),
    ("mvp_attn_fwd_paged_first", lambda **kw: mvp.attn_fwd_paged(*_paged(), window_left=3, first_tokens=2, **kw)),
    ("mvp_rope_append_paged", lambda **kw: mvp.rope_append_paged(*_rope(), **kw)),
    ("mvp_attn_key_weights_varlen", lambda **kw: mvp.attn_key_weights_varlen(*_key_weights_packed(), **kw)),
    ("mvp_attn_key_weights_paged", lambda **kw: mvp.attn_key_weights_paged(*_weights(), **kw)),
    ("mvp_kv_evict_paged", lambda **kw: mvp.kv_evict_paged(*_evict(), **kw)),
]


@pytest.mark.parametrize("name,call", CALLS, ids=[n for n, _ in CALLS])
def test_the_tensors_device_is_current_in_the_call(calls, name, call):
    """Tensors on another GPU than the current one: the library launches where
    they are, on that GPU's current stream or the one given."""
    call()
    assert [c[:2] for c in calls] == [(name, 1)]
    assert 101 in calls[0][2], "not the stream of the tensors' device"

    class Stream:
        device = DEV
        cuda_stream = 777

    call(stream=Stream())
    assert calls[1][:2] == (name, 1) and 777 in calls[1][2]
    assert torch.cuda.current_device() == 0


def test_the_error_word_is_that_of_the_streams_device(calls):
    class Stream:
        device = DEV
        cuda_stream = 777

    mvp.get_last_device_error()
    mvp.get_last_device_error(Stream())
    assert calls == [("mvp_get_last_device_error", 0, (100,)), ("mvp_get_last_device_error", 1, (777,))]


def test_the_current_stream_by_the_public_interface(calls, monkeypatch):
    monkeypatch.delattr(torch._C, "_cuda_getCurrentRawStream", raising=False)

    class Stream:
        cuda_stream = 555

    monkeypatch.setattr(torch.cuda, "current_stream", lambda dev: Stream() if dev == DEV else None)
    mvp.attn_fwd_varlen(*_packed())
    assert calls[0][:2] == ("mvp_attn_fwd_varlen", 1) and 555 in calls[0][2]
