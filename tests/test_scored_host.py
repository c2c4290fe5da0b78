"""Functions of the score and documents without a GPU: refusals before any
launch, and what the binding hands over."""

import ctypes

import pytest
import torch

import masked_varlen_prefill_gb300 as mvp
from masked_varlen_prefill_gb300 import _lib

from .test_binding_host import BF16, F32, FakeTensor, _packed, _paged, calls  # noqa: F401

P = 1 << 20


@pytest.fixture(scope="module")
def lib():
    return mvp.load_library()


def _scored(lib, softcap=0.0, slopes=None, docs=None, **over):
    a = dict(q=P, k=P, v=P, out=P, lse=None, cu_q=P, cu_k=P, ctx=None, num_reqs=1, total_q=4, total_k=4, max_q=4,
             max_k=4, ndec=-1, hq=4, hkv=2, d=128, table=None, covered=None, causal=1, wl=-1, wr=-1, first=0, sinks=None,
             sink_mode=0, scale=0.1, ws=None, ws_bytes=0, stream=None)
    a.update(over)
    return lib.mvp_attn_fwd_varlen_scored(*a.values(), ctypes.byref(_lib.ScoreOptions(softcap, slopes, docs)))


def test_scored_argument_errors(lib):
    for cap in (-1.0, float("nan"), float("inf"), -float("inf"), 1e31, 1e-31):
        assert _scored(lib, cap) == mvp.MVP_ERR_ARG
    assert _scored(lib, 30.0, docs=P + 4) == mvp.MVP_ERR_UNSUPPORTED  # not 8-byte aligned
    assert _scored(lib, 30.0, d=96) == mvp.MVP_ERR_UNSUPPORTED
    assert _scored(lib, 30.0, first=-1) == mvp.MVP_ERR_ARG
    assert _scored(lib, 30.0, hq=3) == mvp.MVP_ERR_ARG
    assert _scored(lib, 30.0, total_q=0) == mvp.MVP_OK
    assert _scored(lib, -1.0, total_q=0) == mvp.MVP_ERR_ARG


def test_paged_scored_argument_errors(lib):
    a = dict(q=P, kc=P, vc=P, out=P, lse=None, cu_q=P, seq_k=P, bt=P, bs=16, max_blocks=4, num_blocks=8, ctx=None,
             num_reqs=1, total_q=4, max_q=4, max_k=64, ndec=-1, hq=4, hkv=2, d=128, table=None, covered=None, causal=1,
             wl=-1, wr=-1, first=0, sinks=None, sink_mode=0, scale=0.1, ws=None, ws_bytes=0, stream=None)
    call = lambda cap=30.0, **over: lib.mvp_attn_fwd_paged_scored(  # noqa: E731
        *{**a, **over}.values(), ctypes.byref(_lib.ScoreOptions(cap, None, None)))
    assert call(-2.0) == mvp.MVP_ERR_ARG
    assert call(bs=48) == mvp.MVP_ERR_ARG
    assert call(max_blocks=3) == mvp.MVP_ERR_ARG
    assert call(total_q=0) == mvp.MVP_OK


def test_document_fill_argument_errors(lib):
    f = lib.mvp_fill_query_documents
    assert f(None, 1, 2, P, P, 4, P, 4, None) == mvp.MVP_ERR_ARG  # starts missing
    assert f(P, 1, 2, None, P, 4, P, 4, None) == mvp.MVP_ERR_ARG
    assert f(P, 1, 2, P, None, 4, P, 4, None) == mvp.MVP_ERR_ARG
    assert f(P, 1, 2, P, P, 4, None, 4, None) == mvp.MVP_ERR_ARG
    assert f(P, 1, -1, P, P, 4, P, 4, None) == mvp.MVP_ERR_ARG
    assert f(P, 0, 2, P, P, 4, P, 4, None) == mvp.MVP_ERR_ARG
    assert f(P, 1, 2, P, P, 4, P, 3, None) == mvp.MVP_ERR_CAPACITY
    assert f(P, 1, 2, P, P, 4, P + 4, 4, None) == mvp.MVP_ERR_UNSUPPORTED
    assert f(None, 0, 0, None, None, 0, None, 0, None) == mvp.MVP_OK


def _options(call):
    return ctypes.cast(call[2][-1], ctypes.POINTER(_lib.ScoreOptions)).contents


def test_the_binding_hands_over_what_is_given(calls):  # noqa: F811
    mvp.attn_fwd_varlen(*_packed(), softcap=30, first_tokens=2, window_left=5)
    mvp.attn_fwd_paged(*_paged(), distance_slopes=FakeTensor((4,), F32))
    mvp.attn_fwd_paged(*_paged(), doc_table=FakeTensor((6, 2)), first_tokens=3, window_left=5)
    mvp.attn_fwd_varlen(*_packed())
    assert [c[:2] for c in calls] == [("mvp_attn_fwd_varlen_scored", 1), ("mvp_attn_fwd_paged_scored", 1),
                                      ("mvp_attn_fwd_paged_scored", 1), ("mvp_attn_fwd_varlen", 1)]
    assert calls[0][2][22] == 2 and calls[1][2][25] == 0 and calls[2][2][25] == 3  # first_tokens


def test_the_bindings_refusals(calls):  # noqa: F811
    bad = [dict(distance_slopes=FakeTensor((3,), F32)), dict(distance_slopes=FakeTensor((4,), BF16)),
           dict(doc_table=FakeTensor((5, 2))), dict(doc_table=FakeTensor((6, 2), torch.int64)),
           dict(softcap=5.0, mixed_prefill_sms=-1)]
    for kw in bad:
        with pytest.raises(ValueError):
            mvp.attn_fwd_varlen(*_packed(), **kw)
    for kw in bad[:4]:
        with pytest.raises(ValueError):
            mvp.attn_fwd_paged(*_paged(), **kw)
    with pytest.raises(ValueError):
        mvp.fill_query_documents(FakeTensor((3, 2)), FakeTensor((3,)), FakeTensor((2,)), FakeTensor((6, 2)), 6)
    with pytest.raises(ValueError):
        mvp.fill_query_documents(FakeTensor((2, 2)), FakeTensor((4,)), FakeTensor((2,)), FakeTensor((6, 2)), 6)
    assert calls == []


def test_the_document_fill_runs_on_its_tensors_device(calls):  # noqa: F811
    mvp.fill_query_documents(FakeTensor((2, 3)), FakeTensor((3,)), FakeTensor((2,)), FakeTensor((6, 2)), 6)
    assert calls[0][:2] == ("mvp_fill_query_documents", 1) and 101 in calls[0][2]
