"""Refusals of the block-scaled cache's calls, and of what they share with the other decodes, that
need no GPU."""
import ctypes
import os
import subprocess

import numpy as np
import pytest
import torch

import __graft_entry__
import paged_kv_decode_19_gb300 as pd
from paged_kv_decode_19_gb300 import _lib


def _cache(B=2, H=2, P=32, D=64):
    i32 = lambda *n: torch.zeros(*n, dtype=torch.int32)  # noqa: E731
    return dict(pages=torch.zeros(4, 2, H, P, D, dtype=torch.int8), scales=torch.ones(4, 2, H, 2),
                page_table_indptr=i32(B + 1), page_table_values=i32(3), length_info=i32(B))


def _decode_args(B=2):
    Q = torch.zeros(B, 4, 64, dtype=torch.bfloat16)
    return dict(_cache(B), Q=Q, output=Q.clone(), lse=torch.zeros(B, 4))


def _append_args(B=2):
    k = torch.zeros(5, 2, 64, dtype=torch.bfloat16)
    return dict(_cache(B), k_new=k, v_new=k, append_indptr=torch.zeros(B + 1, dtype=torch.int32))


CALLS = [(pd.batch_decode_paged_kv_bs, _decode_args), (pd.append_paged_kv_bs, _append_args)]


@pytest.mark.parametrize("call,args", CALLS)
@pytest.mark.parametrize("B", [1, 2, 3])
def test_length_info_is_taken_by_its_shape(call, args, B):
    """[B], or [3, B] of a windowed cache: a [1, B] or [B, 1] read as a window would be read past
    its end, a flat [3 B] or a [B, 3] is not what its reader means."""
    a = args(B)
    for shape in ((1, B), (B, 1), (3 * B,), (B, 3), (2, B), (1, 3, B), (3, B, 1), (B + 1,), (3, B + 1), ()):
        if shape in ((B,), (3, B)):  # (B = 1, 3: one of the two forms)
            continue
        with pytest.raises(ValueError, match="length_info"):
            call(**{**a, "length_info": torch.zeros(shape, dtype=torch.int32)})
    for shape in ((B,), (3, B)):  # taken: what is wrong then is the device
        with pytest.raises(ValueError, match="current GPU"):
            call(**{**a, "length_info": torch.zeros(shape, dtype=torch.int32)})


@pytest.mark.parametrize("B", [1, 2, 3])
def test_length_info_of_the_other_decodes(B):
    """The desc of the other entry points: windowed by a [3, B], else the first B of a list (a
    longer buffer is taken as before, but no flat window)."""
    Q = torch.zeros(B, 4, 64)
    pages, ip = torch.zeros(4, 2, 2, 16, 64), torch.zeros(B + 1, dtype=torch.int32)

    def desc(*shape):
        return pd.make_desc(Q, pages, ip, ip, torch.zeros(shape, dtype=torch.int32), Q)
    for shape in ((1, B), (B, 1), (B, 3), (2, B), (3, B + 1), (3 * B,), (B - 1,), (3, 1, B), ()):
        if shape not in ((3, B), (B,)):
            with pytest.raises(ValueError, match="length_info"):
                desc(*shape)
    assert desc(B).sliding_window == 0 and desc(3, B).sliding_window == 1 and desc(3 * B + 1).sliding_window == 0
    none = torch.zeros(0, dtype=torch.int32)
    assert pd.make_desc(Q[:0], pages, ip[:1], ip, none, Q[:0]).B == 0


def test_host_copies_in_another_byte_order_are_refused():
    for writable in (True, False):
        for dt in (">i4", ">u4", ">f4"):
            a = np.arange(4).astype(dt)
            a.flags.writeable = writable
            with pytest.raises(ValueError):
                _lib._host_i32(a, 4)
        for a in (np.arange(4, dtype="<i4"), np.arange(4, dtype="=i4"), np.arange(4).astype(">i4").astype(np.int32)):
            a.flags.writeable = writable
            assert _lib._host_i32(a, 4) == a.__array_interface__["data"][0]


def test_append_takes_the_heads_that_its_grid_holds():
    """Grid y, at most 65535, is (2 H_kv + 3) / 4 blocks of four (K | V, head) pairs: H_kv <= 131070."""
    __graft_entry__.build()

    def status(H):
        # sizes alone are looked at before the pointers: with those NULL, accepted sizes say so
        d = _lib.AppendBsDesc(T=1, B=1, H_kv=H, D=64, page_size=1, scale_rows=1, in_dtype=2, kv_dtype=4, max_pages=1,
                              nnz_pages=1, k_stride=H * 64, v_stride=H * 64)
        return _lib.STATUS[_lib.lib().pd_append_paged_kv_bs(*[None] * 8, ctypes.byref(d), None)]
    for H in (1, 65535, 131070):
        assert status(H) == "PD_ERR_INVALID_ARG"
    for H in (131071, 150000, 200000, 200001, (1 << 30) - 1):
        assert status(H) == "PD_ERR_UNSUPPORTED"


def _qk_args():
    q = torch.zeros(5, 4, 64)
    return dict(q=q, k=q, q_weight=torch.ones(64), k_weight=torch.ones(64),
                positions=torch.zeros(5, dtype=torch.int32), inv_freq=torch.ones(32, dtype=torch.float64))


@pytest.mark.parametrize("call,args,bad", [
    (pd.batch_decode_paged_kv_bs, _decode_args, dict(Q=torch.zeros(2, 4, 64, dtype=torch.float64))),
    (pd.batch_decode_paged_kv_bs, _decode_args, dict(Q=torch.zeros(2, 4, 64, dtype=torch.int32))),
    (pd.batch_decode_paged_kv_bs, _decode_args, dict(output=torch.zeros(2, 4, 64, dtype=torch.float64))),
    (pd.append_paged_kv_bs, _append_args, dict(k_new=torch.zeros(5, 2, 64).double(), v_new=torch.zeros(5, 2, 64).double())),
    (pd.append_paged_kv_bs, _append_args, dict(page_table_values=None)),
    (pd.qk_norm_rope, _qk_args, dict(q=torch.zeros(5, 4, 64).double(), k=None)),
    (pd.qk_norm_rope, _qk_args, dict(q_weight=torch.ones(64).double(), k_weight=None)),
    (pd.qk_norm_rope, _qk_args, dict(q_weight=None, k_weight=torch.ones(64).int())),
    (pd.qk_norm_rope, _qk_args, dict(positions=None)),
    (pd.qk_norm_rope, _qk_args, dict(k=torch.zeros(64))),
    (pd.qk_norm_rope, _qk_args, dict(q=torch.zeros(4, 64))),
])
def test_types_and_missing_arguments_are_refused_as_such(call, args, bad):
    """A ValueError that names the argument, before the device is looked at."""
    with pytest.raises(ValueError) as e:
        call(**{**args(), **bad})
    assert any(name in str(e.value) for name in bad) or "weights" in str(e.value)
    assert "current GPU" not in str(e.value)


def test_device_planned_grid(tmp_path):
    """Blocks of a short batch planned on the device, for any number of column slices."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    exe = tmp_path / "bs_plan_check"
    subprocess.check_call(["g++", "-std=c++17", "-Wall", "-Werror", "-I",
                           os.path.join(root, "paged_kv_decode_19_gb300", "csrc"),
                           os.path.join(root, "tests", "c", "bs_plan_check.cpp"), "-o", str(exe)])
    out = subprocess.run([str(exe)], capture_output=True, text=True)
    assert out.returncode == 0, out.stdout
    assert out.stdout.strip() == "block-scaled plan ok"
