"""4-bit decode, scores of any size: what counts is their differences.

Rows of K hold one or two values that are not zero, and Q likewise, powers of two or short whole numbers:
every score is exact in the kernel's arithmetic but for one factor of the whole column, which is off
by 3 roundings of fp32 at most."""
import math

import pytest
import torch

import paged_kv_decode_19_gb300 as pd
from tests import _mx
from tests.test_mx_gpu import _decode_case, _run

pytestmark = pytest.mark.gpu
dev = "cuda"
LOG2E = 1 / math.log(2)


def _rows(c, b):
    """Pages and slots of a sequence's rows."""
    r = torch.arange(c["lengths"][b], device=dev)
    return c["vals"][c["indptr"].tolist()[b] + r // c["P"]].long(), r % c["P"]


def _case(lengths, D, P, dt, q_len, k_of_row, scale=0x38, q=(0.0, 0.0), seed=0):
    """Q: its first two dims q, the others zero; K of row r of n: k_of_row(r, n) in its first byte (two
    codes), the others zero, under the e4m3 scale `scale`; V random."""
    c = _decode_case(lengths, 6, 2, D, P, dt, "e4m3", q_len=q_len, seed=seed)
    c["codes"][:, 0], c["scales"][:, 0] = 0, scale
    c["Q"].zero_()
    c["Q"][..., 0], c["Q"][..., 1] = q
    for b, n in enumerate(lengths):
        page, slot = _rows(c, b)
        for h in range(2):
            c["codes"][page, 0, h, slot, 0] = k_of_row(torch.arange(n, device=dev), n).to(torch.uint8)
    return c


def _ref(c, sm, sink):
    """The definition in 64 bits by differences to the largest score (a log-sum-exp of 2^60 holds no ln n)."""
    B, n, Hq, D = c["Q"].shape
    G, f64 = Hq // 2, torch.float64
    out, A = (torch.zeros(B, n, Hq, D, dtype=f64, device=dev) for _ in range(2))
    lse, vmax = torch.full((B, n, Hq), -5e4, dtype=f64, device=dev), torch.zeros(B, n, Hq, dtype=f64, device=dev)
    for b, L in enumerate(c["lengths"]):
        page, slot = _rows(c, b)
        for h in range(Hq):
            k, v = (_mx.row_values(c["codes"][page, w, h // G, slot], c["scales"][page, w, h // G, slot], "e4m3") for w in (0, 1))
            for t in range(n):
                e = max(L - n + 1 + t, 0)
                s = k[:e] @ c["Q"][b, t, h].double() * sm
                if sink is not None:
                    s = torch.cat([s, sink[h:h + 1].double()])
                if not len(s) or s.max() == -math.inf:
                    continue
                p = torch.exp(s - s.max())
                lse[b, t, h] = (s.max() + torch.log(p.sum())) * LOG2E
                p = p[:e] / p.sum()
                if e:
                    out[b, t, h], A[b, t, h], vmax[b, t, h] = p @ v[:e], p @ v[:e].abs(), v[:e].abs().max()
    return out, lse, A, vmax


def _check(c, sm=1.0, sink=None, out_dt=None, **kw):
    """A weight is exact but for f16 (half a step, 2^-11 of it; F32 Q: 22 bits), ex2 and its argument (2^-20 and
    18 2^-24 in log2 units); the sums of few rows as in _mx.check_decode.  lse: the column's factor, its product
    with the maximum and the last sum, half a step of fp32 each.  A sink times log2 e and the log-sum-exp that it
    joins are fp32 numbers: the weight of the one against the other is off by ln 2 times their roundings, half a
    step of the sink's and three of the lse's, all within 4 2^-24 of the larger."""
    out, lse = _run(c, out_dt, sm_scale=sm, sink=sink, **kw)
    assert pd.check_device_errors() == "PD_OK"
    o, l, A, vmax = _ref(c, sm, sink)
    o, A, l, vmax = o.view(out.shape), A.view(out.shape), l.view(lse.shape), vmax.view(lse.shape)
    assert torch.isfinite(out.float()).all() and torch.isfinite(lse).all()
    split = c["Q"].dtype == torch.float32
    rows = max(c["lengths"])
    rel = 2.0 ** -17 + (2.0 ** -22 if split else 2.0 ** -11) + 2 * (17 * rows / 16 + 40) * 2.0 ** -24
    if sink is not None:
        low = torch.where(sink.isinf(), 0.0, sink.double()).abs() * LOG2E
        rel = rel + math.log(2) * 4 * 2.0 ** -24 * torch.maximum(low, l.abs())[..., None]
    tol = A * rel + o.abs() * torch.finfo(out.dtype).eps / 2 + rows * 2.0 ** -32 * vmax[..., None]
    if out.dtype == torch.float16:
        tol = tol + 2.0 ** -25
    err = (out.double() - o).abs()
    assert (err <= tol + 1e-30).all(), f"{(err / (tol + 1e-30)).max().item():.2f} of the bound"
    assert ((lse.double() - l).abs() <= l.abs() * 2.0 ** -22 + 2.0 ** -12).all()


@pytest.mark.parametrize("e", [10, 20, 27, 30, 60, 100])
@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("dt,D,P,q_len", [("bf16", 128, 16, 1), ("f32", 64, 20, 1), ("bf16", 64, 32, 3), ("f32", 256, 16, 2)])
def test_the_largest_scores_alone_count(dt, D, P, q_len, sign, e):
    """Scores of up to 6 2^e, far apart: the running maximum moves several times, and the output is the
    mean of the rows that have the largest."""
    def k(r, n):
        step = torch.clamp(1 + r * 6 // max(n - 40, 1), max=6)   # codes 1 to 6, rising over the rows
        top = torch.where((r * 7 // 5) % 29 == 3, 7, step)       # and 7 (6.0) here and there
        return torch.where(r > n // 3, top, step) if sign > 0 else 8 - top  # (negative: the smallest is largest)
    c = _case([700, 33, 1, 2100], D, P, dt, q_len, k, q=(sign * 2.0 ** e, 0.0), seed=e)
    for n in (0, 1, 9):
        _check(c, num_splits=n)
    _check(c, num_splits=1, out_dt=torch.float32)


@pytest.mark.parametrize("dt,e", [("bf16", 8), ("bf16", 16), ("bf16", 20), ("f16", 15), ("f32", 14), ("f32", 20), ("f32", 22)])
@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("q_len", [1, 2])
def test_small_differences_of_large_scores(q_len, sign, dt, e):
    """Scores sign * 2^e + {0, 6, 12}: 1500 rows, then 150 rows 6 above them and 12 rows 12 above, so that the
    running maximum moves while the rows before it still hold most of the sum."""
    def k(r, n):  # (under a scale of 2, codes 0.5 and 0, 3, 6)
        return 1 + 16 * torch.where(r >= n - 12, 7, torch.where(r >= n - 162, 5, 0))
    c = _case([1662, 1700, 3000], 128, 16, dt, q_len, k, scale=0x40, q=(sign * 2.0 ** e, 1.0), seed=e)
    for n in (1, 0, 9):
        _check(c, num_splits=n, out_dt=torch.float32)


@pytest.mark.parametrize("dt,q0,D,P", [("bf16", -2.0 ** 17, 128, 16), ("f32", -2.0 ** 17, 64, 20), ("f32", -34660.0, 128, 16),
                                       ("f16", -40000.0, 256, 16), ("f32", -34660.0, 128, 7)])
@pytest.mark.parametrize("q_len", [1, 2])
def test_scores_below_the_empty_mark(q_len, dt, q0, D, P):
    """Every score, or some shares' all, below -5e4 in log2 units, the log-sum-exp of a sequence without
    rows: the rows count, however they are split."""
    def k(r, n):
        return 1 + 16 * (r * 13 // 7 % 8)
    c = _case([700, 33, 0, 1, 3000, 5000], D, P, dt, q_len, k, scale=0x40, q=(q0, 1.0), seed=1)
    sink = torch.tensor([q0, q0 + 9, q0 - 3, 1.5 * q0, -math.inf, q0 + 12], device=dev)
    for s in (None, sink):
        for n in (1, 0, 5, 64):
            _check(c, num_splits=n, sink=s)
        _check(c, sink=s, host_meta=pd.host_meta_of(c["indptr"], c["li"]))
