"""batch_decode_paged_kv_bs against its definition in 64 bits within the error that its f16 weights
can make, each output by its own rows and weights."""
import math

import pytest
import torch

from tests._bs import attended, values
from tests.test_bs_gpu import _case, _run, pd

pytestmark = pytest.mark.gpu


def _reference(c):
    """Per output: its value, sum p |v| / sum p, and the sum of |code| min(p vs, 2^-25 of the largest
    p vs) / sum p; per query and head: lse (log2), the largest sum |q k| of a score, the rows."""
    Q, codes, scales, P = c["Q"], c["codes"], c["scales"], c["P"]
    B, n, Hq, D = Q.shape
    H, S = codes.shape[2], P // scales.shape[3]
    G, ip, f64 = Hq // codes.shape[2], c["indptr"].tolist(), dict(dtype=torch.float64, device=Q.device)
    o, A, W = (torch.zeros(B, n, Hq, D, **f64) for _ in range(3))
    lse, smag, rows_of = torch.full((B, n, Hq), -5e4, **f64), *(torch.zeros(B, n, Hq, **f64) for _ in range(2))
    for b, L in enumerate(c["lengths"]):
        rows = attended(L, n, c["wins"][b] if c["wins"] else None).to(Q.device)
        if not len(rows):
            continue
        page, slot = c["vals"][ip[b] + rows // P].long(), rows % P
        # query token t sees the rows up to itself
        last = len(rows) - n + torch.arange(n, device=Q.device)
        seen = torch.arange(len(rows), device=Q.device) <= last[:, None]  # [n, rows]
        for h in range(H):
            ck, cv = (values(codes[page, w, h, slot], c["kv"]) for w in (0, 1))
            ck, cv = ck.nan_to_num(0.0), cv.nan_to_num(0.0)
            ks, vs = (scales[page, w, h, slot // S].double() for w in (0, 1))
            q = Q[b, :, h * G:(h + 1) * G].double()
            s = torch.einsum("tgd,rd->tgr", q, ck * ks[:, None]) * D ** -0.5
            m = torch.einsum("tgd,rd->tgr", q.abs(), (ck * ks[:, None]).abs()) * D ** -0.5
            s = s.masked_fill(~seen[:, None], -math.inf)
            z = torch.logsumexp(s, -1)
            p = torch.exp(s - torch.where(z > -math.inf, z, 0.0)[..., None])
            hs = slice(h * G, (h + 1) * G)
            o[b, :, hs] = p @ (cv * vs[:, None])
            A[b, :, hs] = p @ (cv * vs[:, None]).abs()
            w = p * vs
            W[b, :, hs] = torch.minimum(w, 2.0 ** -25 * w.amax(-1, keepdim=True)) @ cv.abs()
            lse[b, :, hs] = torch.where(z > -math.inf, z / math.log(2), -5e4)
            smag[b, :, hs] = m.masked_fill(~seen[:, None], 0.0).amax(-1) / math.log(2)
            rows_of[b, :, hs] = seen.sum(-1)[:, None]
    return o, A, W, lse, smag, rows_of


def _check(c, out_dt=None, **kw):
    """A score is off by at most 24 roundings of 2^-24 of its sum of magnitudes, ex2 and the scale
    products by 2^-20, sums over the rows by (rows / 16 + 40) 2^-24: r relative in a weight, 2 r A in
    the mean.  Rounding the weights 2^(s - n) vs to f16 is 2^-11 A, and below the normal range at most
    2^-25 or the weight itself, times its code: n is at most the largest s + log2 vs, so 2^-25 is, in
    units of the mean, at most 2^-25 of the largest normalised p vs.  The output: half its own step.
    Returns the largest bound over the largest sum p |v|."""
    out, lse = _run(c, out_dt, **kw)
    assert pd.check_device_errors() == "PD_OK" and pd.last_decode_variant() == "mma"
    o, A, W, l, S, rows = (x.view(out.shape) if x.dim() == 4 and x.shape[-1] == out.shape[-1] else x.view(lse.shape)
                           for x in _reference(c))
    r = 0.694 * 24 * 2.0 ** -24 * S + 2.0 ** -20 + (rows / 16 + 40) * 2.0 ** -24
    tol = A * (2 * r[..., None] + 2.0 ** -11) + W + torch.finfo(out.dtype).eps / 2 * o.abs()
    if out.dtype == torch.float16:
        tol = tol + 2.0 ** -25  # subnormal outputs
    err = (out.double() - o).abs()
    assert (err <= tol + 1e-30).all(), f"out error {(err / (tol + 1e-30)).max().item():.2f} of its bound"
    lerr, lt = (lse.double() - l).abs(), 1.4427 * r + l.abs() * 2.0 ** -23 + 1e-6
    assert (lerr <= lt).all(), f"lse error {(lerr / lt).max().item():.2f} of its bound"
    return (tol.max() / A.max()).item()


@pytest.mark.parametrize("gain", [0.05, 1.0])
def test_one_long_sequence(gain):
    c = _case([70001], 8, 1, 128, 64, 16, "int8", "bf16", seed=8, q_gain=gain)
    # (2^-9 of a bf16 output, 2^-11 of the weights, the scores' roundings; no term grows with the rows)
    assert max(_check(c, dt) for dt in (torch.bfloat16, torch.float32)) < 5e-3


@pytest.mark.parametrize("kv", ["e4m3", "int8"])
@pytest.mark.parametrize("D,P,S", [(128, 16, 16), (64, 32, 16), (128, 8, 4), (64, 20, 5)])
@pytest.mark.parametrize("splits", [0, 1, 5])
def test_lengths_side_by_side(kv, D, P, S, splits):
    """Short sequences keep their own bound beside long ones."""
    _check(_case([9000, 0, 1, 17, 300, 4096], 8, 2, D, P, S, kv, "bf16", seed=9), torch.float32, num_splits=splits)


@pytest.mark.parametrize("gain", [0.1, 1.0, 5.0])
@pytest.mark.parametrize("n,P,S", [(1, 16, 16), (1, 8, 8), (3, 16, 16), (4, 8, 8)])
def test_flat_and_peaked(gain, n, P, S):
    c = _case([2500, 40, 700], 8, 2, 128, P, S, "int8", "bf16", n=n, seed=10, q_gain=gain)
    _check(c, torch.float32)


def test_scales_of_values_far_apart():
    c = _case([1500, 200], 8, 2, 128, 16, 16, "int8", "bf16", seed=11, spread=0.5)
    g = torch.Generator().manual_seed(12)
    c["scales"][:, 1] *= torch.exp2(torch.randint(-12, 13, c["scales"][:, 1].shape, generator=g).float()).to(c["scales"].device)
    _check(c, torch.float32)
    _check(c, torch.float32, num_splits=9)


@pytest.mark.parametrize("P", [16, 8])
def test_windows(P):
    wins = [(0, 0), (50, 4), (301, 1), (999, 20), (17, 17)]
    _check(_case([5, 100, 333, 2000, 64], 8, 2, 128, P, P, "e4m3", "f16", wins=wins, seed=13))
