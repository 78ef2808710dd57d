"""append_paged_kv_mx and batch_decode_paged_kv_mx against their definitions in 64 bits."""
import math

import pytest
import torch

import paged_kv_decode_19_gb300 as pd
from tests import _mx
from tests._mx import BLOCK, DT, SC

pytestmark = pytest.mark.gpu
dev = "cuda"


# ------------------------------------------------------------------------------- append
def _append_case(T, H, D, P, dt, sc, seed=0, spread=1.5, ks=1.0, vs=1.0, fused=False, hole=0.2):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(T, 3 if fused else 2, H, D, generator=g) * torch.exp(spread * torch.randn(T, 3 if fused else 2, H, D // 16, 1, generator=g)).expand(-1, -1, -1, -1, 16).flatten(-2)
    x = x.to(DT[dt]).to(dev)
    k, v = (x[:, 1], x[:, 2]) if fused else (x[:, 0].contiguous(), x[:, 1].contiguous())
    total = -(-T // P) + 2
    slots = torch.randperm(total * P, generator=g)[:T]
    slots[torch.rand(T, generator=g) < hole] = -1
    codes, scales = _mx.cache(total, H, P, D, sc, dev, g)
    return dict(k=k, v=v, slots=slots.to(dev), codes=codes, scales=scales, ks=ks, vs=vs, P=P, sc=sc)


def _append_ref(c):
    codes, scales = c["codes"].clone(), c["scales"].clone()
    keep = c["slots"] >= 0
    page, slot = c["slots"][keep] // c["P"], c["slots"][keep] % c["P"]
    for w, (x, g) in enumerate(((c["k"], c["ks"]), (c["v"], c["vs"]))):
        cc, ss = _mx.quantise_ref(x[keep].double(), g, c["sc"])
        codes[page, w, :, slot] = cc
        scales[page, w, :, slot] = ss
    return codes, scales


def _append(c, **kw):
    pd.append_paged_kv_mx(c["codes"], c["scales"].view(SC[c["sc"]]), c["k"], c["v"], c["slots"], c["ks"], c["vs"], **kw)


def _same(c, ref):
    assert torch.equal(c["scales"], ref[1])
    assert torch.equal(c["codes"], ref[0])


@pytest.mark.parametrize("sc", ["e4m3", "e8m0"])
@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("T,H,D,P,fused", [(1, 8, 128, 16, False), (37, 3, 64, 20, True), (300, 8, 128, 32, True),
                                          (129, 2, 256, 7, False), (5, 1, 64, 1, False), (700, 5, 128, 256, False)])
def test_append(sc, dt, T, H, D, P, fused):
    c = _append_case(T, H, D, P, dt, sc, seed=T, fused=fused, hole=0.0 if T == 1 else 0.2)
    ref = _append_ref(c)
    _append(c)
    assert pd.check_device_errors() == "PD_OK"
    _same(c, ref)


@pytest.mark.parametrize("sc", ["e4m3", "e8m0"])
@pytest.mark.parametrize("ks,vs", [(0.125, 8.0), (0.37, 1.9)])
def test_append_with_cache_scales(sc, ks, vs):
    """Also ones that are no power of two: the quotient is the fp32 one."""
    c = _append_case(200, 4, 128, 16, "f32", sc, seed=3, ks=ks, vs=vs)
    ref = _append_ref(c)
    _append(c)
    _same(c, ref)


@pytest.mark.parametrize("sc", ["e4m3", "e8m0"])
def test_append_on_the_borders(sc):
    """Values on and one step beside every border between codes, under every e4m3 significand and at
    the ends of the scales' ranges."""
    g = torch.Generator().manual_seed(1)
    edges = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], dtype=torch.float64)
    rows = []
    for e in range(-24, 19):
        for m in range(8):
            s = (1 + m / 8) * 2.0 ** e
            x = torch.cat([torch.tensor([6.0], dtype=torch.float64), edges, edges]) * s
            x = torch.cat([x, torch.zeros(1, dtype=torch.float64)]).float()
            x[8:15] = torch.nextafter(x[8:15], torch.tensor(math.inf if m % 2 else -math.inf))
            rows.append(x * torch.where(torch.rand(16, generator=g) < 0.5, -1.0, 1.0))
    x = torch.stack(rows + [-rows[0] * 0, torch.full((16,), 65504.0), torch.full((16,), 3e38), torch.full((16,), 1e-40)])
    x = x[: len(x) // 8 * 8].view(-1, 1, 128)
    T = len(x)
    codes, scales = _mx.cache(-(-T // 16), 1, 16, 128, sc, dev, g)
    c = dict(k=x.to(dev), v=-x.to(dev), slots=torch.arange(T, device=dev), codes=codes, scales=scales, ks=1.0, vs=1.0, P=16, sc=sc)
    ref = _append_ref(c)
    _append(c)
    _same(c, ref)


@pytest.mark.parametrize("sc", ["e4m3", "e8m0"])
@pytest.mark.parametrize("ks,vs", [(0.1, 3.0), (1 + 2.0 ** -23, 1 - 2.0 ** -24), (2.0 ** -60, 2.0 ** 60), (7e-19, 1.6e18),
                                   (1e-30, 1e30), (1.2e-38, 3e38), (1e-44, 0.7)])
def test_append_on_the_borders_of_a_cache_scale(sc, ks, vs):
    """x / g on a border or a step or two beside it, for large and small x and g: the fp32 quotient, and
    a zero's sign."""
    g = torch.Generator().manual_seed(2)
    edges = torch.tensor([6.0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], dtype=torch.float64)
    ks, vs = torch.tensor([ks, vs], dtype=torch.float32).tolist()
    sides = []
    for scale in (ks, vs):
        rows = []
        for e in range(-10, 10):
            x = (edges.repeat(2) * (1 + torch.randint(8, (1,), generator=g) / 8) * 2.0 ** e * scale).float()
            up = torch.nextafter(x, torch.tensor(math.inf))
            x = torch.where(torch.rand(16, generator=g) < 0.5, x, torch.where(torch.rand(16, generator=g) < 0.5, up, torch.nextafter(x, torch.tensor(0.0))))
            x[15] = 0
            rows += [x.clamp(max=3.4e38), (torch.randn(16, generator=g).double() * scale).clamp(-3e38, 3e38).float()]
        rows += [torch.randn(16, generator=g) * 1e-38, torch.full((16,), 1e-44), torch.full((16,), 3.4e38), torch.rand(16, generator=g) * 3.4e38]
        x = torch.stack(rows[: len(rows) // 4 * 4])
        sides.append((x * torch.where(torch.rand(x.shape, generator=g) < 0.5, -1.0, 1.0)).view(-1, 1, 64))
    k, v = sides
    T = len(k)
    codes, scales = _mx.cache(-(-T // 4), 1, 4, 64, sc, dev, g)
    c = dict(k=k.to(dev), v=v.to(dev), slots=torch.arange(T, device=dev), codes=codes, scales=scales, ks=ks, vs=vs, P=4, sc=sc)
    ref = _append_ref(c)
    _append(c)
    assert pd.check_device_errors() == "PD_OK"
    _same(c, ref)


@pytest.mark.parametrize("sc", ["e4m3", "e8m0"])
@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
def test_append_non_finite(sc, dt):
    """A non-finite value takes its block alone."""
    c = _append_case(40, 2, 128, 16, dt, sc, seed=4, spread=0.3, hole=0.0)
    c["k"][3, 1, 17], c["v"][7, 0, 100], c["k"][9, 0, 0] = math.nan, math.inf, -math.inf
    ref = _append_ref(c)
    _append(c)
    _same(c, ref)
    assert (c["scales"] == (0x7f if sc == "e4m3" else 0xff)).sum() == 3


def test_append_bad_slots_and_alignment():
    c = _append_case(64, 2, 64, 16, "bf16", "e4m3", seed=5, hole=0.0)
    wide = torch.zeros(64, 2 * 64 + 1, dtype=torch.bfloat16, device=dev)
    wide[:, 1:] = c["k"].flatten(1)  # rows two bytes off any 16-byte border
    c["k"] = wide[:, 1:].unflatten(1, (2, 64))
    n = c["codes"].shape[0] * 16
    bad = torch.tensor([3, 40], device=dev)
    c["slots"][bad] = torch.tensor([n, 1 << 40], device=dev)
    good = c["slots"].clone()
    good[bad] = -1
    ref = _append_ref({**c, "slots": good})
    _append(c)
    assert pd.check_device_errors() == "PD_ERR_BAD_SLOT"
    _same(c, ref)
    assert pd.check_device_errors() == "PD_OK"


# ------------------------------------------------------------------------------- decode
def _decode_case(lengths, Hq, H, D, P, dt, sc, q_len=1, seed=0, wins=None, ks=1.0, vs=1.0, total=None, qs=1.0):
    g = torch.Generator().manual_seed(seed)
    indptr, vals, last, total = _mx.table(lengths, P, dev, g, total=total)
    codes, scales = _mx.cache(total, H, P, D, sc, dev, g)
    Q = (torch.randn(len(lengths), q_len, Hq, D, generator=g) * qs).to(DT[dt]).to(dev)
    li = last
    if wins:
        li = torch.stack([last, torch.tensor([w[0] for w in wins], dtype=torch.int32, device=dev),
                          torch.tensor([w[1] for w in wins], dtype=torch.int32, device=dev)])
    return dict(Q=Q, codes=codes, scales=scales, sc=sc, indptr=indptr, vals=vals, li=li, lengths=lengths, P=P, wins=wins,
                ks=ks, vs=vs)


def _ref(c, sink=None, sm=None):
    return _mx.decode_ref(c["Q"], c["codes"], c["scales"], c["sc"], c["indptr"], c["vals"], c["lengths"], c["P"],
                          c["Q"].shape[-1] ** -0.5 if sm is None else sm, c["ks"], c["vs"], c["wins"], sink)


def _run(c, out_dt=None, **kw):
    Q = c["Q"] if c["Q"].shape[1] > 1 else c["Q"][:, 0].contiguous()
    out = torch.full(Q.shape, 7.0, dtype=out_dt or Q.dtype, device=dev)
    lse = torch.full(Q.shape[:-1], 7.0, device=dev)
    pd.batch_decode_paged_kv_mx(Q, c["codes"], c["scales"].view(SC[c["sc"]]), c["indptr"], c["vals"], c["li"], out, lse,
                                k_scale=c["ks"], v_scale=c["vs"], **kw)
    return out, lse


def _check(c, out_dt=None, ref=None, sink=None, **kw):
    out, lse = _run(c, out_dt, sink=sink, **kw)
    assert pd.check_device_errors() == "PD_OK"
    sm = kw.get("sm_scale")
    _mx.check_decode(out, lse, ref or _ref(c, sink, sm), max(c["lengths"], default=0), c["Q"].dtype == torch.float32,
                     c["Q"].shape[-1])
    return out, lse


LENS = [0, 1, 15, 16, 17, 31, 33, 200, 640, 1111]


@pytest.mark.parametrize("sc", ["e4m3", "e8m0"])
@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("Hq,H,D", [(8, 2, 128), (16, 2, 64), (6, 2, 256), (10, 1, 128)])
@pytest.mark.parametrize("P", [16, 20])
def test_decode(sc, dt, Hq, H, D, P):
    c = _decode_case(LENS, Hq, H, D, P, dt, sc, seed=P + D)
    ref = _ref(c)
    out, lse = _check(c, ref=ref)
    assert (out[0] == 0).all() and (lse[0] == -5e4).all()
    _check(c, ref=ref, host_meta=pd.host_meta_of(c["indptr"], c["li"]))


@pytest.mark.parametrize("P", [1, 7, 8, 32, 48, 64, 256])
@pytest.mark.parametrize("sc,dt,D", [("e4m3", "bf16", 128), ("e8m0", "f16", 64), ("e8m0", "bf16", 256), ("e4m3", "f32", 64)])
def test_decode_page_sizes(P, sc, dt, D):
    c = _decode_case(LENS, 4, 2, D, P, dt, sc, seed=P)
    _check(c)


@pytest.mark.parametrize("sc", ["e4m3", "e8m0"])
@pytest.mark.parametrize("dt,D,P", [("bf16", 128, 16), ("f16", 64, 32), ("f32", 128, 16), ("bf16", 64, 20), ("f16", 256, 16),
                                    ("f32", 256, 10)])
@pytest.mark.parametrize("q_len", [2, 5])
def test_decode_several_queries(sc, dt, D, P, q_len):
    c = _decode_case([0, 1, 2, 4, 5, 6, 16, 17, 48, 333], 6, 2, D, P, dt, sc, q_len=q_len, seed=q_len)
    ref = _ref(c)
    _check(c, ref=ref)
    _check(c, ref=ref, host_meta=pd.host_meta_of(c["indptr"], c["li"]))


@pytest.mark.parametrize("sc,dt,D,P", [("e4m3", "bf16", 128, 16), ("e8m0", "f16", 64, 32), ("e4m3", "f16", 128, 20),
                                       ("e8m0", "f32", 256, 16)])
def test_decode_windows(sc, dt, D, P):
    """Windows that start inside a page and a tile, with and without sinks; garbage rows outside."""
    lengths = [40, 100, 100, 333, 640, 17, 0, 500]
    wins = [(0, 0), (37, 4), (99, 0), (101, 17), (333, 1), (0, 0), (0, 0), (16, 16)]
    c = _decode_case(lengths, 8, 2, D, P, dt, sc, wins=wins, seed=D)
    ip = c["indptr"].tolist()
    nan = 0x7f if sc == "e4m3" else 0xff
    for b, (n, w) in enumerate(zip(lengths, wins)):
        gone = torch.arange(w[1], w[0])  # rows between the sinks and the window, and behind the end
        gone = torch.cat([gone, torch.arange(n, (ip[b + 1] - ip[b]) * P)]).to(dev)
        c["scales"][c["vals"][ip[b] + gone // P].long(), :, :, gone % P] = nan
    ref = _ref(c)
    out, _ = _check(c, ref=ref)
    assert torch.isfinite(out.float()).all()
    _check(c, ref=ref, host_meta=pd.host_meta_of(c["indptr"], c["li"]))


@pytest.mark.parametrize("q_len", [1, 3])
@pytest.mark.parametrize("dt,D,P", [("bf16", 128, 16), ("f32", 64, 20)])
def test_decode_sinks_splits_and_types(q_len, dt, D, P):
    c = _decode_case([700, 0, 33, 1500], 8, 2, D, P, dt, "e4m3", q_len=q_len, seed=9, ks=0.5, vs=3.0)
    sink = torch.tensor([0.5, -1.0, 8.0, -math.inf, 2.0, 0.0, 30.0, -30.0], device=dev)
    ref = _ref(c, sink)
    for n in (0, 1, 5, 64):
        _check(c, ref=ref, sink=sink, num_splits=n)
    for t in DT.values():
        _check(c, t, ref=ref, sink=sink)
    for sm in (0.0, -0.07, 1e-30, 0.5):
        _check(c, sm_scale=sm)


def test_decode_extreme_values():
    """Q over the range of its type, scores in the thousands, scales at the ends of their ranges."""
    for dt, qs in (("bf16", 1e30), ("bf16", 1e-30), ("f16", 500.0), ("f32", 1e25), ("f32", 1e-25)):
        c = _decode_case([50, 300], 4, 2, 128, 16, dt, "e4m3", seed=2, qs=qs)
        _check(c, sm_scale=1.0 / qs if dt != "f16" else 0.1)
    for sc, lo, hi in (("e4m3", 0x01, 0x7e), ("e8m0", 113, 140)):
        for dt in ("f16", "f32"):
            c = _decode_case([50, 300], 4, 2, 128, 16, dt, sc, seed=3)
            c["scales"].copy_(torch.where(torch.rand(c["scales"].shape, device=dev) < 0.5, lo, hi))
            _check(c, torch.float32, sm_scale=1e-5)


@pytest.mark.parametrize("sc", ["e4m3", "e8m0"])
@pytest.mark.parametrize("q_len", [1, 3])
@pytest.mark.parametrize("dt,D,P", [("bf16", 128, 16), ("f16", 64, 16), ("bf16", 256, 16), ("f32", 128, 9)])
def test_decode_nan_scales(sc, q_len, dt, D, P):
    """A NaN scale reaches the tokens that attend its row, of V its own dims, and nothing else."""
    c = _decode_case([20, 64, 130, 7], 8, 2, D, P, dt, sc, q_len=q_len, seed=6)
    nan, ip, n = (0x7f if sc == "e4m3" else 0xff), c["indptr"].tolist(), D // BLOCK[sc]
    for b, r, side, h, blk in ((0, 19, 1, 0, n - 1), (1, 63, 0, 1, 0), (1, 5, 1, 0, 1), (2, 128, 1, 1, 0), (2, 0, 1, 0, 1)):
        c["scales"][c["vals"][ip[b] + r // P].long(), side, h, r % P, blk] = nan
    out, lse = _check(c)
    assert out.isnan().any() and not out.isnan().all()
    assert torch.isfinite(out.view(4, -1)[3].float()).all()


def test_decode_bad_pages_are_skipped():
    """A page id out of range: its rows count for nothing."""
    for P, dt in ((16, "bf16"), (20, "bf16"), (16, "f32")):
        c = _decode_case([100, 64], 4, 2, 128, P, dt, "e4m3", seed=7)
        c["vals"][1] = c["codes"].shape[0]
        c["vals"][c["indptr"].tolist()[1]] = -5
        out, lse = _run(c)
        assert pd.check_device_errors() == "PD_ERR_BAD_PAGE"
        for b, bad in ((0, 1), (1, 0)):
            rows = [r for r in range(c["lengths"][b]) if r // P != bad]
            page = c["vals"][c["indptr"].tolist()[b] + torch.tensor(rows, device=dev) // P].long()
            slot = torch.tensor(rows, device=dev) % P
            for h in range(2):
                k, v = (_mx.row_values(c["codes"][page, w, h, slot], c["scales"][page, w, h, slot], "e4m3") for w in (0, 1))
                p = torch.softmax(c["Q"][b, 0, 2 * h:2 * h + 2].double() @ k.T * 128 ** -0.5, -1)
                err = (out[b, 2 * h:2 * h + 2].double() - p @ v).abs().max()
                assert err <= 2.0 ** -7 * (p @ v.abs()).max()


def test_decode_offsets_past_32_bits():
    """Pages whose bytes lie beyond 2^32 of the cache."""
    H, P, D = 8, 64, 128
    n = (5 << 30) // (2 * H * P * D // 2)
    pages = torch.empty(n, 2, H, P, D // 2, dtype=torch.uint8, device=dev)
    scales = torch.empty(n, 2, H, P, D // 16, dtype=torch.uint8, device=dev)
    ids = torch.tensor([n - 1, 0, n - 7, n // 2, n * 9 // 10], dtype=torch.int32, device=dev)
    g = torch.Generator().manual_seed(0)
    codes, sc = _mx.cache(5, H, P, D, "e4m3", dev, g)
    pages[ids.long()], scales[ids.long()] = codes, sc
    c = dict(codes=pages, scales=scales, sc="e4m3", P=P, wins=None, ks=1.0, vs=1.0, lengths=[3 * P, 2 * P - 5], vals=ids,
             indptr=torch.tensor([0, 3, 5], dtype=torch.int32, device=dev), li=torch.tensor([P, P - 5], dtype=torch.int32, device=dev),
             Q=torch.randn(2, 1, 16, D, generator=g).bfloat16().to(dev))
    _check(c)
    c["Q"] = c["Q"].float()
    _check(c)
    # and the append there
    k = torch.randn(4, H, D, generator=g).to(dev)
    slots = torch.tensor([(n - 1) * P + 3, (n - 7) * P + 63, -1, n * P - 1], device=dev)
    a = dict(k=k, v=-k, slots=slots, ks=1.0, vs=1.0, P=P, sc="e4m3", codes=pages, scales=scales)
    cc, ss = _mx.quantise_ref(k.double(), 1.0, "e4m3")
    _append(a)
    for t, s in enumerate(slots.tolist()):
        if s >= 0:
            assert torch.equal(pages[s // P, 0, :, s % P], cc[t]) and torch.equal(scales[s // P, 0, :, s % P], ss[t])


def test_decode_many_sequences_and_long_ones():
    g = torch.Generator().manual_seed(8)
    lengths = torch.randint(0, 400, (300,), generator=g).tolist()
    c = _decode_case(lengths, 8, 1, 128, 16, "bf16", "e4m3", seed=1)
    ref = _ref(c)
    _check(c, ref=ref)
    _check(c, ref=ref, host_meta=pd.host_meta_of(c["indptr"], c["li"]))
    c = _decode_case([40000, 9, 7000], 40, 2, 128, 64, "f16", "e8m0", seed=2)  # three slices of columns
    ref = _ref(c)
    _check(c, ref=ref)
    _check(c, ref=ref, host_meta=pd.host_meta_of(c["indptr"], c["li"]))


def test_decode_streams_workspaces_and_unaligned_outputs():
    c = _decode_case([900, 50, 3000], 8, 2, 128, 16, "bf16", "e4m3", seed=5)
    ref = _ref(c)
    d = pd.make_desc(c["Q"][:, 0].contiguous(), torch.empty(c["codes"].shape[0], 2, 2, 16, 128, dtype=torch.float8_e4m3fn),
                     c["indptr"], c["vals"], c["li"], c["Q"])
    d.kv_dtype = 5
    n = pd.workspace_size_mx(d, 1)
    assert n > 0
    ws = torch.zeros(n, dtype=torch.uint8, device=dev)
    _check(c, ref=ref, workspace=ws)
    _check(c, ref=ref, workspace=ws)
    with pytest.raises(pd.PDError, match="WORKSPACE"):
        _run(c, workspace=ws[:256])
    outs, streams = [], [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    for i in range(9):
        with torch.cuda.stream(streams[i % 3]):
            outs.append(_run(c))
    torch.cuda.synchronize()
    for out, lse in outs:
        _mx.check_decode(out, lse, ref, 3000, False, 128)
    big = torch.zeros(3 * 8 * 128 + 1, dtype=torch.bfloat16, device=dev)
    out, lse = big[1:].view(3, 8, 128), torch.empty(3, 8, device=dev)
    pd.batch_decode_paged_kv_mx(c["Q"][:, 0].contiguous(), c["codes"], c["scales"].view(SC["e4m3"]), c["indptr"], c["vals"],
                                c["li"], out, lse)
    _mx.check_decode(out, lse, ref, 3000, False, 128)
    assert big[0] == 0


@pytest.mark.parametrize("q_len", [1, 3])
@pytest.mark.parametrize("B,P,dt", [(1500, 16, "bf16"), (700, 20, "f32")])
def test_decode_more_sequences_than_threads(B, P, dt, q_len):
    """The places of the sequences are summed on the device, several to a thread."""
    g = torch.Generator().manual_seed(B)
    lengths = torch.where(torch.rand(B, generator=g) < 0.3, 0, torch.randint(0, 60, (B,), generator=g)).tolist()
    lengths[-1] = 900
    c = _decode_case(lengths, 2, 1, 64, P, dt, "e4m3", seed=3, q_len=q_len)
    _check(c)


@pytest.mark.parametrize("Hq,H,q_len", [(16, 1, 1), (32, 1, 1), (20, 1, 1), (8, 2, 8), (64, 2, 1), (3, 1, 7)])
@pytest.mark.parametrize("dt,D", [("bf16", 128), ("f32", 64), ("f16", 256)])
def test_decode_slices_of_columns(Hq, H, q_len, dt, D):
    """Two to five slices of eight query columns, on warps that walk the pages side by side or not."""
    c = _decode_case([0, 17, 3000, 640, 5], Hq, H, D, 16, dt, "e8m0", q_len=q_len, seed=Hq)
    ref = _ref(c)
    _check(c, ref=ref)
    _check(c, ref=ref, host_meta=pd.host_meta_of(c["indptr"], c["li"]))
    _check(c, ref=ref, num_splits=7)


@pytest.mark.parametrize("D,P", [(64, 16), (128, 32), (128, 20), (256, 16), (256, 12)])
def test_decode_f32_sums_over_many_tiles(D, P):
    """Equal values of V come out as they are, whatever the weights: what is off is the sums.  n tiles of
    16 rows go into a sum one after the other, each rounded to nearest: an error that is even over +-2^-24
    of the sum, and independent, so that six deviations of all are 6 2^-24 sqrt(n / 3).  (Each rounded
    down instead: n 2^-24, seven times the bound.)  A weight's split into two f16 parts, of 22 bits, and the
    denominator's own sums add the same again at most."""
    n = 2500
    c = _decode_case([16 * n, 16 * n - 5], 8, 1, D, P, "f32", "e4m3", seed=D, qs=0.3)
    c["codes"][:, 1] = 0x22   # 1.0
    c["scales"][:, 1] = 0x38  # 1.0
    out, _ = _run(c, num_splits=1)
    assert pd.check_device_errors() == "PD_OK"
    assert (out.double() - 1).abs().max().item() <= 2 * 6 * 2.0 ** -24 * math.sqrt(n / 3)


@pytest.mark.parametrize("n", [1, 2, 3, 7, 40, 200])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_decode_shares_of_every_size(n, dt):
    """Few rows on many warps, one sequence over all blocks, sequences of one length: the merges."""
    for lengths in ([n], [16 * n], [16 * n + 1] * 5, [50 * n] * 3, [1, 400 * n, 1]):
        c = _decode_case(lengths, 8, 2, 128, 16, dt, "e4m3", seed=n)
        ref = _ref(c)
        _check(c, ref=ref)
        _check(c, ref=ref, host_meta=pd.host_meta_of(c["indptr"], c["li"]))


def test_decode_right_behind_the_append():
    """early_inputs: the decode starts under the append that writes the rows it reads."""
    c = _decode_case([600, 33, 5, 1024] * 8, 8, 2, 128, 16, "bf16", "e4m3", seed=4)
    ip, B = c["indptr"].tolist(), 32
    last = torch.tensor([n - 1 for n in c["lengths"]], device=dev)
    page = c["vals"][torch.tensor([ip[b] + (n - 1) // 16 for b, n in enumerate(c["lengths"])], device=dev)].long()
    slots = page * 16 + last % 16
    g = torch.Generator().manual_seed(0)
    hm = pd.host_meta_of(c["indptr"], c["li"])
    for i in range(6):
        k, v = torch.randn(2, B, 2, 128, generator=g).bfloat16().to(dev) * (i + 1)
        torch.cuda.synchronize()
        pd.append_paged_kv_mx(c["codes"], c["scales"].view(SC["e4m3"]), k, v, slots)
        out, lse = _run(c, early_inputs=True, host_meta=hm if i % 2 else None)
        assert pd.check_device_errors() == "PD_OK"
        _mx.check_decode(out, lse, _ref(c), 1024, False, 128)
