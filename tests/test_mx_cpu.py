"""Refusals of the 4-bit cache's calls and of the page tables', which need no GPU; the tests'
definitions against one another."""
import ctypes

import pytest
import torch

import __graft_entry__
import paged_kv_decode_19_gb300 as pd
from paged_kv_decode_19_gb300 import _lib
from tests import _mx


@pytest.fixture(scope="module")
def L():
    __graft_entry__.build()
    return _lib.lib()


def _cache(B=2, H=2, P=32, D=64, sc="e4m3"):
    i32 = lambda *n: torch.zeros(*n, dtype=torch.int32)  # noqa: E731
    return dict(pages=torch.zeros(4, 2, H, P, D // 2, dtype=torch.uint8),
                scales=torch.zeros(4, 2, H, P, D // _mx.BLOCK[sc], dtype=torch.uint8).view(_mx.SC[sc]),
                page_table_indptr=i32(B + 1), page_table_values=i32(3), length_info=i32(B))


def _decode(**kw):
    Q = torch.zeros(2, 4, 64, dtype=torch.bfloat16)
    a = dict(_cache(), Q=Q, output=Q.clone(), lse=torch.zeros(2, 4))
    return pd.batch_decode_paged_kv_mx(**{**a, **kw})


def _append(**kw):
    k = torch.zeros(5, 2, 64, dtype=torch.bfloat16)
    c = _cache()
    a = dict(pages=c["pages"], scales=c["scales"], k_new=k, v_new=k, slot_mapping=torch.zeros(5, dtype=torch.int64))
    return pd.append_paged_kv_mx(**{**a, **kw})


def _tables(**kw):
    i32 = lambda *n: torch.zeros(*n, dtype=torch.int32)  # noqa: E731
    a = dict(page_table=i32(3, 4), lengths=i32(3), new_tokens=i32(3), state=torch.zeros(4, dtype=torch.int64), page_size=16,
             page_table_indptr=i32(4), page_table_values=i32(9), length_info=i32(3), append_indptr=i32(4),
             slot_mapping=torch.zeros(7, dtype=torch.int64), positions=i32(7), free_pages=i32(12))
    return pd.build_page_tables(**{**a, **kw})


def _bytes(*n, t=torch.uint8):
    return torch.zeros(*n, dtype=torch.uint8).view(t)


E4, E8 = torch.float8_e4m3fn, torch.float8_e8m0fnu


@pytest.mark.parametrize("call", [_decode, _append])
@pytest.mark.parametrize("bad,name", [
    (dict(pages=torch.zeros(4, 2, 2, 32, 32, dtype=torch.int8)), "pages"),
    (dict(pages=_bytes(4, 2, 2, 32)), "pages"),
    (dict(pages=_bytes(4, 3, 2, 32, 32)), "pages"),
    (dict(scales=_bytes(4, 2, 2, 32, 4)), "scales"),                # bytes do not say which scales
    (dict(scales=torch.zeros(4, 2, 2, 32, 4)), "scales"),
    (dict(scales=_bytes(4, 2, 2, 32, 2, t=E4)), "scales"),
    (dict(scales=_bytes(4, 2, 2, 32, 4, t=E8)), "scales"),
    (dict(scales=_bytes(4, 2, 2, 31, 4, t=E4)), "scales"),
    (dict(scales=_bytes(3, 2, 2, 32, 4, t=E4)), "scales"),
    (dict(scales=_bytes(4, 2, 2, 4, t=E4)), "scales"),
])
def test_caches_are_refused(call, bad, name):
    with pytest.raises(ValueError, match=name):
        call(**bad)


@pytest.mark.parametrize("bad,name", [
    (dict(Q=torch.zeros(2, 4, 64).double()), "Q"), (dict(Q=torch.zeros(2, 4, 128)), "Q"),
    (dict(Q=torch.zeros(8, 64)), "Q"), (dict(output=torch.zeros(2, 4, 64).double()), "output"),
    (dict(output=torch.zeros(2, 4, 32)), "output"), (dict(lse=torch.zeros(2, 5)), "lse"),
    (dict(lse=torch.zeros(2, 4).double()), "lse"),
    (dict(length_info=torch.zeros(1, 2, dtype=torch.int32)), "length_info"),
    (dict(length_info=torch.zeros(6, dtype=torch.int32)), "length_info"),
    (dict(length_info=torch.zeros(2, dtype=torch.int64)), "length_info"),
    (dict(page_table_indptr=torch.zeros(4, dtype=torch.int32)), "page_table_indptr"),
    (dict(page_table_values=torch.zeros(4, dtype=torch.int64)), "page_table_values"),
])
def test_decode_arguments_are_refused(bad, name):
    with pytest.raises(ValueError, match=name):
        _decode(**bad)


def test_what_is_left_is_the_device():
    for call in (_decode, _append, _tables):
        with pytest.raises(ValueError, match="current GPU"):
            call()
    with pytest.raises(ValueError, match="current GPU"):
        _decode(scales=_bytes(4, 2, 2, 32, 2, t=E8))
    if hasattr(torch, "float4_e2m1fn_x2"):
        with pytest.raises(ValueError, match="current GPU"):
            _append(pages=_bytes(4, 2, 2, 32, 32, t=torch.float4_e2m1fn_x2))


@pytest.mark.parametrize("bad,name", [
    (dict(k_new=torch.zeros(5, 2, 64).double(), v_new=torch.zeros(5, 2, 64).double()), "k_new"),
    (dict(k_new=torch.zeros(5, 2, 64)), "k_new"), (dict(k_new=torch.zeros(5, 3, 64, dtype=torch.bfloat16)), "k_new"),
    (dict(slot_mapping=torch.zeros(5, dtype=torch.int32)), "slot_mapping"),
    (dict(slot_mapping=torch.zeros(4, dtype=torch.int64)), "slot_mapping"),
    (dict(k_new=torch.zeros(5, 64, 2, dtype=torch.bfloat16).transpose(1, 2)), "heads"),
])
def test_append_arguments_are_refused(bad, name):
    with pytest.raises(ValueError, match=name):
        _append(**bad)


I32 = torch.int32


@pytest.mark.parametrize("bad,name", [
    (dict(page_table=torch.zeros(12, dtype=I32)), "page_table"), (dict(page_table=torch.zeros(3, 4).long()), "page_table"),
    (dict(lengths=torch.zeros(4, dtype=I32)), "lengths"), (dict(new_tokens=torch.zeros(3).long()), "new_tokens"),
    (dict(state=torch.zeros(2, dtype=torch.int64)), "state"), (dict(state=torch.zeros(4, dtype=I32)), "state"),
    (dict(page_table_indptr=torch.zeros(3, dtype=I32)), "page_table_indptr"),
    (dict(page_table_values=torch.zeros(3, 3, dtype=I32)), "page_table_values"),
    (dict(length_info=torch.zeros(3, 3, dtype=I32)), "length_info"), (dict(window=8), "length_info"),
    (dict(append_indptr=torch.zeros(3, dtype=I32)), "append_indptr"),
    (dict(slot_mapping=torch.zeros(7, dtype=I32)), "slot_mapping"), (dict(positions=torch.zeros(6, dtype=I32)), "positions"),
    (dict(positions=torch.zeros(7).long()), "positions"), (dict(free_pages=torch.zeros(0, dtype=I32)), "free_pages"),
    (dict(free_pages=torch.zeros(9).long()), "free_pages"),
])
def test_tables_arguments_are_refused(bad, name):
    with pytest.raises(ValueError, match=name):
        _tables(**bad)


def _desc(**kw):
    d = dict(B=4, H_qo=8, H_kv=2, D=128, page_size=16, q_dtype=2, kv_dtype=5, out_dtype=2,
             sliding_window=0, num_splits=0, max_pages=100, nnz_pages=40, max_kv_len_hint=0,
             k_scale=1.0, v_scale=1.0, workspace=None, workspace_bytes=0, sink=None)
    d.update(kw)
    return _lib.DecodeDesc(**d)


@pytest.mark.parametrize("bad,status", [
    (dict(H_qo=7), "PD_ERR_INVALID_ARG"), (dict(D=96), "PD_ERR_UNSUPPORTED"), (dict(D=32), "PD_ERR_UNSUPPORTED"),
    (dict(page_size=0), "PD_ERR_INVALID_ARG"), (dict(page_size=257), "PD_ERR_INVALID_ARG"),
    (dict(kv_dtype=3), "PD_ERR_INVALID_ARG"), (dict(kv_dtype=4), "PD_ERR_INVALID_ARG"),
    (dict(kv_dtype=7), "PD_ERR_INVALID_ARG"), (dict(q_dtype=5), "PD_ERR_INVALID_ARG"),
    (dict(k_scale=0.0), "PD_ERR_INVALID_ARG"), (dict(k_scale=-1.0), "PD_ERR_INVALID_ARG"),
    (dict(v_scale=float("nan")), "PD_ERR_INVALID_ARG"), (dict(v_scale=float("inf")), "PD_ERR_INVALID_ARG"),
    (dict(max_pages=1 << 30), "PD_ERR_UNSUPPORTED"), (dict(flags=4), "PD_ERR_INVALID_ARG"),
    (dict(), "PD_ERR_INVALID_ARG"),  # NULL pointers
])
def test_decode_desc_is_validated(L, bad, status):
    d = _desc(**bad)
    st = L.pd_batch_decode_paged_kv_mx(*[None] * 8, 1, 0.1, ctypes.byref(d), None)
    assert _lib.STATUS[st] == status, L.pd_get_last_error_string()


def test_decode_calls_are_validated(L):
    d, p = _desc(), ctypes.c_void_p
    f = L.pd_batch_decode_paged_kv_mx
    ptr = lambda q=16, pages=32, scales=48: (p(q), p(pages), p(scales), p(64), p(64), p(64), p(64), p(64))  # noqa: E731
    for args, word in ((ptr(q=18), b"16-byte"), (ptr(pages=40), b"16-byte"), (ptr(scales=56), b"16-byte"),
                       (ptr(scales=0), b"scales")):
        assert _lib.STATUS[f(*args, 1, 0.1, ctypes.byref(d), None)] == "PD_ERR_INVALID_ARG"
        assert word in L.pd_get_last_error_string()
    assert _lib.STATUS[f(*ptr(), 0, 0.1, ctypes.byref(d), None)] == "PD_ERR_INVALID_ARG"
    assert _lib.STATUS[f(*ptr(), 1, float("nan"), ctypes.byref(d), None)] == "PD_ERR_INVALID_ARG"
    w = _desc(sliding_window=1)
    assert _lib.STATUS[f(*ptr(), 2, 0.1, ctypes.byref(w), None)] == "PD_ERR_UNSUPPORTED"
    assert f(*[None] * 8, 1, 0.1, ctypes.byref(_desc(B=0)), None) == 0
    # the other decodes do not take the 4-bit types
    assert _lib.STATUS[L.pd_batch_decode_paged_kv(*[None] * 9, 0, 1.0, 1e4, 0.1, ctypes.byref(d), None)] == "PD_ERR_INVALID_ARG"
    assert _lib.STATUS[L.pd_batch_decode_paged_kv_bs(*[None] * 8, 1, 16, 0.1, ctypes.byref(d), None)] == "PD_ERR_INVALID_ARG"


def test_append_desc_is_validated(L):
    def status(pages=16, scales=32, k=48, **kw):
        d = dict(T=3, H_kv=2, D=128, page_size=16, in_dtype=2, kv_dtype=5, max_pages=10, k_stride=256, v_stride=256,
                 k_scale=1.0, v_scale=1.0, flags=0, reserved=0)
        d = _lib.AppendMxDesc(**{**d, **kw})
        p = ctypes.c_void_p
        return _lib.STATUS[L.pd_append_paged_kv_mx(p(pages), p(scales), p(k), p(k), None, ctypes.byref(d), None)]
    for bad in (dict(T=-1), dict(H_kv=0), dict(page_size=300), dict(in_dtype=3), dict(kv_dtype=3), dict(k_scale=0.0),
                dict(v_scale=float("inf")), dict(flags=1), dict(reserved=1), dict(k_stride=255), dict(max_pages=0), dict()):
        assert status(**bad) == "PD_ERR_INVALID_ARG", bad
    for bad in (dict(D=80), dict(max_pages=1 << 30), dict(T=(1 << 30) + 1), dict(T=1 << 30, H_kv=8, k_stride=1024, v_stride=1024)):
        assert status(**bad) == "PD_ERR_UNSUPPORTED", bad
    assert status(T=0) == "PD_OK"


def test_tables_desc_is_validated(L):
    def status(state=16, free=32, ptr=64, **kw):
        d = dict(B=3, page_size=16, max_pages_per_seq=4, T=7, window=0, sinks=0, flags=0, reserved=0, table_stride=4,
                 values_capacity=9, free_capacity=12)
        d = _lib.TablesDesc(**{**d, **kw})
        p = ctypes.c_void_p
        # (no indptr: sizes that are accepted are refused for that)
        st = L.pd_build_page_tables(p(ptr), p(ptr), p(ptr), p(state), p(free), None, p(ptr), p(ptr), None, p(ptr), p(ptr),
                                    ctypes.byref(d), None)
        return _lib.STATUS[st], L.pd_get_last_error_string()
    for bad in (dict(B=-1), dict(page_size=0), dict(page_size=257), dict(max_pages_per_seq=0), dict(T=-1), dict(window=-1),
                dict(sinks=2), dict(window=5, sinks=-1), dict(flags=1), dict(reserved=1), dict(table_stride=3),
                dict(values_capacity=-1), dict(free_capacity=-1)):
        st, text = status(**bad)
        assert st == "PD_ERR_INVALID_ARG" and b"pointer" not in text, (bad, text)
    for bad in (dict(B=8193), dict(B=8000, max_pages_per_seq=1 << 20, table_stride=1 << 20), dict(T=1 << 30)):
        assert status(**bad)[0] == "PD_ERR_UNSUPPORTED", bad
    assert b"pointer" in status()[1] and b"pointer" in status(B=8192)[1]


def test_quantisation_of_the_tests():
    """The definition by trial on values whose codes are known."""
    x = torch.zeros(3, 32, dtype=torch.float64)
    x[0, :8] = torch.tensor([6.0, 5.0, 3.5, 2.5, 1.75, 1.25, 0.75, 0.25])   # ties: to the even code
    x[1, :8] = -x[0, :8]
    x[2, 0] = float("inf")
    for sc, one, nan in (("e4m3", 0x38, 0x7f), ("e8m0", 127, 255)):
        codes, s = _mx.quantise_ref(x, 1.0, sc)
        assert s[0, 0] == one and s[1, 0] == one and s[2, 0] == nan and (codes[2] == 0).all()
        assert codes[0, :4].tolist() == [0x67, 0x46, 0x24, 0x02]
        assert codes[1, :4].tolist() == [0xef, 0xce, 0xac, 0x8a]
        v = _mx.row_values(codes[:2], s[:2], sc)
        assert v[0, :8].tolist() == [6.0, 4.0, 4.0, 2.0, 2.0, 1.0, 1.0, 0.0]
    assert _mx.quantise_ref(x[:1] * 0, 1.0, "e4m3")[1][0, 0] == 1 and _mx.quantise_ref(x[:1] * 0, 1.0, "e8m0")[1][0, 0] == 113
