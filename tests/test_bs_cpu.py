"""Checks of the block-scaled cache and qk_norm_rope that need no GPU: struct layout, host
validation, the binding's own refusals, and the frequency tables against their formulas."""
import ctypes
import math

import numpy as np
import pytest
import torch

import __graft_entry__
from paged_kv_decode_19_gb300 import _lib
import paged_kv_decode_19_gb300 as pd


@pytest.fixture(scope="module")
def L():
    __graft_entry__.build()
    return _lib.lib()


def _name(st):
    return _lib.STATUS[st]


def _desc(**kw):
    d = dict(B=4, H_qo=8, H_kv=2, D=128, page_size=32, q_dtype=2, kv_dtype=4, out_dtype=2, sliding_window=0,
             num_splits=0, max_pages=100, nnz_pages=40, max_kv_len_hint=0, k_scale=0.0, v_scale=0.0)
    d.update(kw)
    return _lib.DecodeDesc(**d)


def _decode(L, d, q_len=1, scale_rows=16, Q=4096, pages=8192, scales=64, scale=0.1):
    p = ctypes.c_void_p
    return L.pd_batch_decode_paged_kv_bs(p(Q), p(pages), p(scales), p(64), p(128), p(192), p(256), p(320), q_len,
                                         scale_rows, scale, ctypes.byref(d), None)


@pytest.mark.parametrize("kw,call,status", [
    (dict(kv_dtype=2), {}, "PD_ERR_INVALID_ARG"), (dict(kv_dtype=5), {}, "PD_ERR_INVALID_ARG"),
    (dict(D=96), {}, "PD_ERR_UNSUPPORTED"), (dict(H_qo=7), {}, "PD_ERR_INVALID_ARG"),
    (dict(q_dtype=3), {}, "PD_ERR_INVALID_ARG"), (dict(out_dtype=4), {}, "PD_ERR_INVALID_ARG"),
    (dict(), dict(scale_rows=0), "PD_ERR_INVALID_ARG"), (dict(), dict(scale_rows=12), "PD_ERR_INVALID_ARG"),
    (dict(), dict(scale_rows=64), "PD_ERR_INVALID_ARG"), (dict(), dict(q_len=0), "PD_ERR_INVALID_ARG"),
    (dict(sliding_window=1), dict(q_len=2), "PD_ERR_UNSUPPORTED"),
    (dict(D=256), dict(q_len=2), "PD_ERR_UNSUPPORTED"), (dict(q_dtype=0), dict(q_len=2), "PD_ERR_UNSUPPORTED"),
    (dict(), dict(Q=4104), "PD_ERR_INVALID_ARG"), (dict(), dict(pages=8200), "PD_ERR_INVALID_ARG"),
    (dict(), dict(scales=66), "PD_ERR_INVALID_ARG"), (dict(), dict(scales=None), "PD_ERR_INVALID_ARG"),
    (dict(), dict(Q=None), "PD_ERR_INVALID_ARG"), (dict(flags=4), {}, "PD_ERR_INVALID_ARG"),
    (dict(), dict(scale=float("nan")), "PD_ERR_INVALID_ARG"),
    (dict(max_pages=1 << 30), {}, "PD_ERR_UNSUPPORTED"), (dict(page_size=257), {}, "PD_ERR_INVALID_ARG"),
])
def test_decode_refusals(L, kw, call, status):
    assert _name(_decode(L, _desc(**kw), **call)) == status, L.pd_get_last_error_string()


def test_decode_of_nothing_and_codes_elsewhere(L):
    assert _decode(L, _desc(B=0)) == 0
    assert L.pd_batch_decode_paged_kv_bs(None, None, None, None, None, None, None, None, 1, 16, 0.1, None, None) == 1
    # int8 codes exist only with block scales
    p = ctypes.c_void_p
    st = L.pd_batch_decode_paged_kv(p(4096), p(8192), p(64), p(128), p(192), None, None, p(256), p(320), 0, 1.0, 1e4,
                                    0.1, ctypes.byref(_desc(k_scale=1.0, v_scale=1.0)), None)
    assert _name(st) == "PD_ERR_INVALID_ARG"
    assert L.pd_workspace_size_bs(ctypes.byref(_desc(kv_dtype=2)), 1, 16) == 0
    assert L.pd_workspace_size_bs(ctypes.byref(_desc()), 0, 16) == 0


def _append(L, **kw):
    a = dict(pages=8192, scales=64, k=4096, v=4096, at=64, ip=64, vals=64, li=64, T=5, B=2, H_kv=2, D=128,
             page_size=32, scale_rows=16, max_pages=10, nnz_pages=4, k_stride=256, v_stride=256, in_dtype=2, kv_dtype=4,
             flags=0, reserved=0)
    a.update(kw)
    d = _lib.AppendBsDesc(**{n: a[n] for n, _ in _lib.AppendBsDesc._fields_})
    return _name(L.pd_append_paged_kv_bs(*(a[n] for n in ("pages", "scales", "k", "v", "at", "ip", "vals", "li")),
                                         ctypes.byref(d), None))


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), "PD_ERR_INVALID_ARG"), (dict(B=-1), "PD_ERR_INVALID_ARG"), (dict(H_kv=0), "PD_ERR_INVALID_ARG"),
    (dict(D=96), "PD_ERR_UNSUPPORTED"), (dict(page_size=0), "PD_ERR_INVALID_ARG"), (dict(page_size=512), "PD_ERR_INVALID_ARG"),
    (dict(scale_rows=0), "PD_ERR_INVALID_ARG"), (dict(scale_rows=12), "PD_ERR_INVALID_ARG"), (dict(in_dtype=3), "PD_ERR_INVALID_ARG"),
    (dict(kv_dtype=2), "PD_ERR_INVALID_ARG"), (dict(k_stride=255), "PD_ERR_INVALID_ARG"), (dict(v_stride=0), "PD_ERR_INVALID_ARG"),
    (dict(max_pages=0), "PD_ERR_INVALID_ARG"), (dict(max_pages=1 << 30), "PD_ERR_UNSUPPORTED"),
    (dict(nnz_pages=-1), "PD_ERR_INVALID_ARG"), (dict(B=(1 << 31) - 1), "PD_ERR_UNSUPPORTED"),
    (dict(pages=None), "PD_ERR_INVALID_ARG"), (dict(pages=8200), "PD_ERR_INVALID_ARG"),
    (dict(scales=62), "PD_ERR_INVALID_ARG"), (dict(at=None), "PD_ERR_INVALID_ARG"),
    (dict(vals=None), "PD_ERR_INVALID_ARG"), (dict(T=0), "PD_OK"), (dict(B=0), "PD_OK"),
    (dict(flags=1), "PD_ERR_INVALID_ARG"), (dict(reserved=1), "PD_ERR_INVALID_ARG"), (dict(k=4097), "PD_ERR_INVALID_ARG"),
    (dict(max_pages=1 << 62), "PD_ERR_UNSUPPORTED"),
])
def test_append_refusals(L, kw, status):
    assert _append(L, **kw) == status, L.pd_get_last_error_string()


def _qk(L, q=4096, k=4096, qo=8192, ko=8192, wq=None, wk=None, pos=64, freq=64, **kw):
    d = dict(T=3, H_q=4, H_k=2, D=64, dtype=2, weight_dtype=2, rotary_mode=1, rotary_dim=64, eps=1e-6,
             weight_offset=0.0, attention_factor=1.0, q_stride=256, k_stride=128, q_head_stride=64, k_head_stride=64,
             q_out_stride=256, k_out_stride=128, q_out_head_stride=64, k_out_head_stride=64)
    d.update(kw)
    return _name(L.pd_qk_norm_rope(q, k, wq, wk, pos, freq, qo, ko, ctypes.byref(_lib.QkDesc(**d)), None))


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), "PD_ERR_INVALID_ARG"), (dict(H_q=-1), "PD_ERR_INVALID_ARG"), (dict(H_k=70000), "PD_ERR_INVALID_ARG"),
    (dict(D=0), "PD_ERR_UNSUPPORTED"), (dict(D=513), "PD_ERR_UNSUPPORTED"), (dict(dtype=3), "PD_ERR_INVALID_ARG"),
    (dict(wq=64, weight_dtype=4), "PD_ERR_INVALID_ARG"), (dict(rotary_mode=3), "PD_ERR_INVALID_ARG"),
    (dict(rotary_dim=63), "PD_ERR_INVALID_ARG"), (dict(rotary_dim=66), "PD_ERR_INVALID_ARG"),
    (dict(rotary_dim=-2), "PD_ERR_INVALID_ARG"), (dict(eps=-1.0), "PD_ERR_INVALID_ARG"),
    (dict(eps=float("nan")), "PD_ERR_INVALID_ARG"), (dict(attention_factor=float("inf")), "PD_ERR_INVALID_ARG"),
    (dict(q=None), "PD_ERR_INVALID_ARG"), (dict(ko=None), "PD_ERR_INVALID_ARG"), (dict(pos=None), "PD_ERR_INVALID_ARG"),
    (dict(freq=None), "PD_ERR_INVALID_ARG"), (dict(q=4097), "PD_ERR_INVALID_ARG"), (dict(T=0), "PD_OK"),
    (dict(H_q=0, H_k=0), "PD_OK"),
])
def test_qk_refusals(L, kw, status):
    assert _qk(L, **kw) == status, L.pd_get_last_error_string()
    assert _name(L.pd_qk_norm_rope(None, None, None, None, None, None, None, None, None, None)) == "PD_ERR_INVALID_ARG"


def test_layouts():
    import struct
    assert struct.calcsize("@10i2qi2fi5Q") == ctypes.sizeof(_lib.DecodeDesc)
    assert struct.calcsize("@8i3f8q") == ctypes.sizeof(_lib.QkDesc)
    for a in (np.arange(4, dtype=np.int32), np.arange(4, dtype=np.int32)[:0], np.arange(8, dtype=np.int32)[2:5]):
        assert _lib._host_i32(a, a.size) == a.__array_interface__["data"][0]
    a = np.arange(4, dtype=np.int32)
    a.flags.writeable = False
    assert _lib._host_i32(a, 4) == a.__array_interface__["data"][0]
    for bad in (np.arange(4), np.arange(8, dtype=np.int32)[::2], np.arange(5, dtype=np.int32), [0, 1, 2, 3], None,
                np.arange(4, dtype=np.uint32), np.arange(4, dtype=np.float32)):
        with pytest.raises(ValueError):
            _lib._host_i32(bad, 4)
    v = _lib._PACK_DECODE(*range(1, 11), 11, 12, 13, 14.0, 15.0, 16, 17, 18, 19, 20, 21)
    d = _lib.DecodeDesc.from_buffer_copy(v)
    assert [getattr(d, n) for n, _ in d._fields_] == list(range(1, 22))
    v = _lib._PACK_APPEND(*range(1, 15))
    assert len(v) == ctypes.sizeof(_lib.AppendBsDesc)
    d = _lib.AppendBsDesc.from_buffer_copy(v)
    assert [getattr(d, n) for n, _ in d._fields_] == list(range(1, 15))
    v = _lib._PACK_QK(*range(1, 9), 9.0, 10.0, 11.0, *range(12, 20))
    d = _lib.QkDesc.from_buffer_copy(v)
    assert [getattr(d, n) for n, _ in d._fields_] == list(range(1, 20))
    assert ctypes.sizeof(_lib.QkDesc) == 112
    assert _lib.QkDesc.q_stride.offset == 48 and _lib.QkDesc.k_out_head_stride.offset == 104


def test_binding_refusals():
    """The Python front refuses shapes, types and strides before it touches an address."""
    B, H, P, D = 2, 2, 32, 64
    pages = torch.zeros(4, 2, H, P, D, dtype=torch.int8)
    scales = torch.ones(4, 2, H, 2)
    Q = torch.zeros(B, 4, D, dtype=torch.bfloat16)
    ip, vals, li = (torch.zeros(n, dtype=torch.int32) for n in (B + 1, 3, B))
    lse = torch.zeros(B, 4)
    ok = dict(Q=Q, pages=pages, scales=scales, page_table_indptr=ip, page_table_values=vals, length_info=li,
              output=Q.clone(), lse=lse)
    for bad in (dict(pages=pages.float()), dict(pages=pages[0]), dict(scales=scales.double()),
                dict(scales=torch.ones(4, 2, H, 3)), dict(scales=torch.ones(3, 2, H, 2)), dict(Q=Q[..., :32]),
                dict(Q=Q[0]), dict(output=Q[:1]), dict(lse=lse.double()), dict(lse=lse[:1]),
                dict(page_table_indptr=ip.long()), dict(page_table_indptr=ip[:2]), dict(length_info=li[:1]),
                dict(sink=torch.zeros(3)), dict()):  # (the last: CPU tensors)
        with pytest.raises(ValueError):
            pd.batch_decode_paged_kv_bs(**{**ok, **bad})
    k = torch.zeros(5, H, D, dtype=torch.bfloat16)
    at = torch.zeros(B + 1, dtype=torch.int32)
    ok = dict(pages=pages, scales=scales, k_new=k, v_new=k, append_indptr=at, page_table_indptr=ip,
              page_table_values=vals, length_info=li)
    for bad in (dict(k_new=k[:, :1]), dict(v_new=k.float()), dict(v_new=k[:4]), dict(append_indptr=at.long()),
                dict(append_indptr=at[:2]), dict(k_new=torch.zeros(5, H, 2 * D, dtype=torch.bfloat16)[..., ::2]),
                dict(k_new=torch.zeros(H, 5, D, dtype=torch.bfloat16).transpose(0, 1)), dict()):
        with pytest.raises(ValueError):
            pd.append_paged_kv_bs(**{**ok, **bad})
    q = torch.zeros(5, 4, D)
    w, pos, freq = torch.ones(D), torch.zeros(5, dtype=torch.int32), torch.ones(D // 2, dtype=torch.float64)
    ok = dict(q=q, k=q, q_weight=w, k_weight=w, positions=pos, inv_freq=freq)
    for bad in (dict(k=q.half()), dict(k=q[:4]), dict(q_weight=w[:3]), dict(k_weight=w.half()),
                dict(positions=pos.long()), dict(positions=pos[:4]), dict(inv_freq=freq.float()),
                dict(q_out=q[:, :1].expand(5, 4, D)), dict(q_out=q[:, :2]), dict(q=torch.zeros(5, 4, 2 * D)[..., ::2]),
                dict(k_out=q.half()), dict()):
        with pytest.raises(ValueError):
            pd.qk_norm_rope(**{**ok, **bad})


def test_rope_frequencies(L):
    """Each entry is a handful of correctly rounded fp64 steps and two pow: 1e-14 relative."""
    for rd in (2, 64, 128, 20):
        n = rd // 2
        plain = [5e5 ** (-i / n) for i in range(n)]
        want = {None: plain, "linear": [f / 8 for f in plain]}
        th = 5e5 * 8 ** (n / (n - 1)) if n > 1 else 5e5
        want["theta"] = [th ** (-i / n) for i in range(n)]
        parts = []
        for f in plain:
            wavelength = 2 * math.pi / f
            if wavelength < 8192 / 4:
                parts.append(f)
            elif wavelength > 8192 / 1:
                parts.append(f / 8)
            else:
                g = (8192 / wavelength - 1) / (4 - 1)
                parts.append((1 - g) * f / 8 + g * f)
        want["parts"] = parts
        for name, w in want.items():
            got = pd.rope_frequencies(rd, 5e5, name, 8.0, 8192, 1.0, 4.0, device="cpu")
            assert got.dtype == torch.float64 and got.shape == (n,)
            for a, b in zip(got.tolist(), w):
                assert abs(a - b) <= 1e-14 * b
    if n > 1:  # theta scaling keeps the highest frequency and divides the lowest by the factor
        got = pd.rope_frequencies(128, 1e4, "theta", 4.0, device="cpu")
        plain = pd.rope_frequencies(128, 1e4, device="cpu")
        assert got[0] == plain[0] and abs(got[-1] * 4 / plain[-1] - 1) < 1e-13


@pytest.mark.parametrize("kw", [dict(rotary_dim=3), dict(rotary_dim=0), dict(rope_theta=0.0),
                                dict(rope_theta=float("nan")), dict(scaling="linear", factor=0.0),
                                dict(scaling="parts", factor=8.0), dict(scaling="theta", factor=float("inf")),
                                dict(scaling="parts", factor=8.0, original_context=100.0, low_turns=4.0, high_turns=4.0)])
def test_rope_frequencies_refusals(L, kw):
    a = dict(rotary_dim=64, device="cpu")
    a.update(kw)
    with pytest.raises(pd.PDError):
        pd.rope_frequencies(**a)
    with pytest.raises(ValueError):
        pd.rope_frequencies(64, scaling="other", device="cpu")
