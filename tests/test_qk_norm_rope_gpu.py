"""GPU parity of qk_norm_rope against its formula in 64 bits."""
import math

import pytest
import torch

from tests._bs import DT

pd = pytest.importorskip("paged_kv_decode_19_gb300")
pytestmark = pytest.mark.gpu
DEV = "cuda"


def norm_rope_ref(x, w, pos, freq, mode, eps, offset, factor):
    """(result, the sum of magnitudes that enters each output) in fp64."""
    y = x.double()
    if w is not None:
        y = y / torch.sqrt((y * y).mean(-1, keepdim=True) + eps) * (w.double() + offset)
    n = 0 if freq is None else freq.numel()
    z, m = y.clone(), y.abs()
    if n:
        ang = pos.double()[:, None] * freq.double()
        co, si = ang.cos()[:, None] * factor, ang.sin()[:, None] * factor
        first = slice(0, n) if mode == 1 else slice(0, 2 * n, 2)
        second = slice(n, 2 * n) if mode == 1 else slice(1, 2 * n, 2)
        a, b = y[..., first], y[..., second]
        z[..., first], z[..., second] = a * co - b * si, b * co + a * si
        m[..., first] = m[..., second] = (a.abs() + b.abs()) * abs(factor)
    return z, m


def check_norm_rope(x, w, pos, freq, got, mode=1, eps=1e-6, offset=0.0, factor=1.0):
    """fp32 steps: the sum of squares (21 roundings on a path, halved by the root), the mean, eps,
    the reciprocal root (2 ulp), weight and offset (4), cosine and sine with the factor (4 ulp), the
    rotation (3): under 32 roundings of 2^-24 of the magnitudes that enter; then half a step."""
    z, m = norm_rope_ref(x, w, pos, freq, mode, eps, offset, factor)
    tol = 32 * 2.0 ** -24 * m + torch.finfo(got.dtype).eps / 2 * z.abs() * 1.001 + 1e-37
    if got.dtype == torch.float16:
        tol = tol + 2.0 ** -25
    err = (got.double() - z).abs()
    assert torch.isfinite(got.float()).all()
    assert (err <= tol).all(), f"error {(err / tol).max().item():.2f} of its bound"


def _inputs(T, Hq, Hk, D, dt, seed=0, wdt=None, far=0):
    g = torch.Generator().manual_seed(seed)
    q, k = (torch.randn(T, H, D, generator=g).to(DT[dt]).to(DEV) for H in (Hq, Hk))
    wq, wk = ((1 + 0.3 * torch.randn(D, generator=g)).to(DT[wdt or dt]).to(DEV) for _ in range(2))
    pos = (torch.randint(0, 5000, (T,), generator=g) + far).to(torch.int32).to(DEV)
    return q, k, wq, wk, pos


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("mode", [1, 2])
@pytest.mark.parametrize("T,Hq,Hk,D,rd", [(1, 32, 8, 128, 128), (5, 7, 1, 64, 32), (300, 4, 4, 256, 64), (3, 2, 3, 80, 80),
                                          (2, 1, 1, 96, 20), (9, 3, 2, 200, 48), (2, 5, 1, 512, 512), (4, 2, 1, 6, 4),
                                          (3, 1, 1, 33, 32), (1500, 40, 10, 128, 128), (2, 70, 9, 128, 64),
                                          (2, 200, 1, 64, 64), (1, 9, 1, 8, 0)])
def test_shapes(dt, mode, T, Hq, Hk, D, rd):
    q, k, wq, wk, pos = _inputs(T, Hq, Hk, D, dt, seed=T + D)
    freq = pd.rope_frequencies(rd, 1e4, device=DEV) if rd else None
    qo, ko = pd.qk_norm_rope(q, k, wq, wk, pos, freq, rotary_mode=mode)
    check_norm_rope(q, wq, pos, freq, qo, mode)
    check_norm_rope(k, wk, pos, freq, ko, mode)


@pytest.mark.parametrize("D", [128, 72, 50])
def test_either_norm_and_no_keys(D):
    """A norm on one side only, and queries alone."""
    q, k, wq, wk, pos = _inputs(33, 5, 2, D, "bf16", seed=1)
    freq = pd.rope_frequencies(48, 1e4, device=DEV)
    for a, b in ((wq, None), (None, wk), (None, None)):
        qo, ko = pd.qk_norm_rope(q, k, a, b, pos, freq)
        check_norm_rope(q, a, pos, freq, qo)
        check_norm_rope(k, b, pos, freq, ko)
    qo, ko = pd.qk_norm_rope(q, None, wq, None, pos, freq)
    assert ko is None
    check_norm_rope(q, wq, pos, freq, qo)
    e = torch.empty(33, 0, D, dtype=torch.bfloat16, device=DEV)
    _, ko = pd.qk_norm_rope(e, k, None, wk, pos, freq)
    check_norm_rope(k, wk, pos, freq, ko)


@pytest.mark.parametrize("D", [64, 42])
def test_norm_alone(D):
    q, k, wq, wk, pos = _inputs(20, 3, 2, D, "f16", seed=2)
    qo, ko = pd.qk_norm_rope(q, k, wq, wk, None, None, eps=1e-5, weight_offset=1.0)
    check_norm_rope(q, wq, pos, None, qo, eps=1e-5, offset=1.0)
    check_norm_rope(k, wk, pos, None, ko, eps=1e-5, offset=1.0)


@pytest.mark.parametrize("wdt", ["f32", "f16", "bf16"])
def test_weight_types(wdt):
    q, k, wq, wk, pos = _inputs(6, 3, 2, 128, "bf16", seed=3, wdt=wdt)
    freq = pd.rope_frequencies(128, 1e4, device=DEV)
    qo, ko = pd.qk_norm_rope(q, k, wq, wk, pos, freq, attention_factor=1.2079)
    check_norm_rope(q, wq, pos, freq, qo, factor=1.2079)
    check_norm_rope(k, wk, pos, freq, ko, factor=1.2079)


@pytest.mark.parametrize("far", [1 << 20, (1 << 31) - 6000, -4000])
@pytest.mark.parametrize("D", [128, 30])
def test_far_and_negative_positions(far, D):
    q, k, wq, wk, pos = _inputs(40, 2, 1, D, "f32", seed=4, far=far)
    # frequencies with few bits, so that the 64-bit reference's own angle is exact
    freq = torch.exp2(-torch.arange(D // 2, device=DEV, dtype=torch.float64) % 23)
    qo, ko = pd.qk_norm_rope(q, k, wq, wk, pos, freq)
    check_norm_rope(q, wq, pos, freq, qo)
    check_norm_rope(k, wk, pos, freq, ko)


@pytest.mark.parametrize("odd", [0, 4, 1])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_slices_in_place_and_transposed(dt, odd):
    """q and k as slices of one projection, written back in place; and heads-first storage."""
    g = torch.Generator().manual_seed(5)
    T, Hq, Hk, D = 50, 6, 2, 64
    x = torch.randn(T, (Hq + 2 * Hk) * D + odd, generator=g).to(DT[dt]).to(DEV)
    q, k = x[:, odd:odd + Hq * D].unflatten(1, (Hq, D)), x[:, odd + Hq * D:odd + (Hq + Hk) * D].unflatten(1, (Hk, D))
    w = torch.ones(D, dtype=DT[dt], device=DEV)
    pos = torch.arange(T, dtype=torch.int32, device=DEV)
    freq = pd.rope_frequencies(D, 1e4, device=DEV)
    was = x.clone()
    wq, wk = was[:, odd:odd + Hq * D].unflatten(1, (Hq, D)), was[:, odd + Hq * D:odd + (Hq + Hk) * D].unflatten(1, (Hk, D))
    pd.qk_norm_rope(q, k, w, w, pos, freq, q, k)
    check_norm_rope(wq, w, pos, freq, q)
    check_norm_rope(wk, w, pos, freq, k)
    assert torch.equal(x[:, odd + (Hq + Hk) * D:], was[:, odd + (Hq + Hk) * D:])
    assert torch.equal(x[:, :odd], was[:, :odd])
    t = wq.transpose(0, 1).contiguous().transpose(0, 1)  # [T, H, D] stored heads first
    out = torch.empty(Hq, T, D, dtype=DT[dt], device=DEV).transpose(0, 1)
    pd.qk_norm_rope(t, None, w, None, pos, freq, out)
    check_norm_rope(wq, w, pos, freq, out)


def test_no_tokens_and_large_values():
    q, k, wq, wk, pos = _inputs(0, 2, 1, 64, "bf16")
    freq = pd.rope_frequencies(64, 1e4, device=DEV)
    qo, ko = pd.qk_norm_rope(q, k, wq, wk, pos, freq)
    assert qo.shape == q.shape and ko.shape == k.shape
    q, k, wq, wk, pos = _inputs(8, 2, 1, 64, "bf16", seed=6)
    q[0] *= 1e15   # squares near 1e30
    q[1] *= 1e-15  # below eps
    q[2] = 0
    q[3, 0, 5] = float("nan")
    qo, _ = pd.qk_norm_rope(q, k, wq, wk, pos, freq)
    rows = [0, 1, 2, 4, 5, 6, 7]
    check_norm_rope(q[rows], wq, pos[rows], freq, qo[rows])
    assert torch.isnan(qo[3, 0]).all() and torch.isfinite(qo[3, 1].float()).all()


def test_rope_agrees_with_the_append_that_rotates():
    """The same rotation as append_paged_kv_rope's, through a cache of the rows' own type."""
    T, H, D, P = 30, 2, 128, 16
    _, k, _, _, pos = _inputs(T, 1, H, D, "f32", seed=7)
    freq = pd.rope_frequencies(D, 5e5, device=DEV)
    for mode in (1, 2):
        pages = torch.zeros(2, 2, H, P, D, device=DEV)
        pd.append_paged_kv_rope(pages, k, k, torch.arange(T, dtype=torch.int64, device=DEV), pos, mode, 1.0, 5e5)
        stored = pages[:, 0].transpose(1, 2).reshape(-1, H, D)[:T]
        _, ko = pd.qk_norm_rope(k[:, :0], k, None, None, pos, freq, rotary_mode=mode)
        assert (stored - ko).abs().max() <= 8 * 2.0 ** -24 * 2 * k.abs().max()


def test_captured_and_replayed():
    q, k, wq, wk, pos = _inputs(64, 8, 2, 128, "bf16", seed=8)
    freq = pd.rope_frequencies(128, 1e4, device=DEV)
    qo, ko = torch.empty_like(q), torch.empty_like(k)
    pd.qk_norm_rope(q, k, wq, wk, pos, freq, qo, ko)
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        pd.qk_norm_rope(q, k, wq, wk, pos, freq, qo, ko)
    a = _inputs(64, 8, 2, 128, "bf16", seed=9)
    for x, y in zip((q, k, wq, wk, pos), a):
        x.copy_(y)
    gr.replay()
    torch.cuda.synchronize()
    check_norm_rope(q, wq, pos, freq, qo)
    check_norm_rope(k, wk, pos, freq, ko)
    assert math.isfinite(float(qo.float().sum()))
