"""GPU parity of the block-scaled 8-bit cache: batch_decode_paged_kv_bs and
append_paged_kv_bs against their definitions in 64 bits."""
import math

import pytest
import torch

from tests._bs import DT, KV, TOP, cache, check_decode, decode_ref, encode, pow2_need, table, values

pd = pytest.importorskip("paged_kv_decode_19_gb300")
pytestmark = pytest.mark.gpu
DEV = "cuda"


def _case(lengths, Hq, H, D, P, S, kv, dt, n=1, seed=0, wins=None, spread=1.0, q_gain=1.0, pow2=False):
    g = torch.Generator().manual_seed(seed)
    indptr, vals, last, total = table(lengths, P, DEV, g)
    codes, scales = cache(total, H, P, S, D, kv, DEV, g, spread, pow2)
    # what no sequence attends holds whatever: NaN codes (-128 for int8) and, where a whole
    # block is unattended, NaN scales
    junk = 0x7F if kv == "e4m3" else -128
    ip, used = indptr.tolist(), torch.zeros(total, P, dtype=torch.bool)
    for b, L in enumerate(lengths):
        from tests._bs import attended
        rows = attended(L, n, wins[b] if wins else None)
        used[vals[ip[b] + rows // P].long().cpu(), rows % P] = True
    used = used.to(DEV)
    codes[~used[:, None, None, :, None].expand_as(codes)] = junk
    blk = used.view(total, 1, 1, P // S, S).any(-1).expand_as(scales)
    scales[~blk] = float("nan")
    Q = (torch.randn(len(lengths), n, Hq, D, generator=g) * q_gain).to(DT[dt]).to(DEV)
    li = last
    if wins:
        li = torch.stack([last, torch.tensor([w[0] for w in wins], dtype=torch.int32, device=DEV),
                          torch.tensor([w[1] for w in wins], dtype=torch.int32, device=DEV)])
    return dict(Q=Q, codes=codes, scales=scales, indptr=indptr, vals=vals, li=li, lengths=lengths,
                P=P, kv=kv, wins=wins, n=n, D=D)


def _run(c, out_dt=None, ws=None, **kw):
    Q = c["Q"] if c["n"] > 1 else c["Q"][:, 0].contiguous()
    out = torch.full(Q.shape, float("nan"), dtype=out_dt or Q.dtype, device=DEV)
    lse = torch.full(Q.shape[:-1], float("nan"), device=DEV)
    pd.batch_decode_paged_kv_bs(Q, c["codes"].view(KV[c["kv"]]), c["scales"], c["indptr"], c["vals"],
                                c["li"], out, lse, workspace=ws, **kw)
    return out, lse


def _ref(c, **kw):
    return decode_ref(c["Q"], c["codes"], c["scales"], c["kv"], c["indptr"], c["vals"], c["lengths"],
                      c["P"], c["D"] ** -0.5, c["wins"], **kw)


def _check(c, variant=None, out_dt=None, sink=None, **kw):
    out, lse = _run(c, out_dt, sink=sink, **kw)
    assert pd.check_device_errors() == "PD_OK"
    if variant:
        assert pd.last_decode_variant() == variant
    check_decode(out, lse, _ref(c, sink=sink), max(c["lengths"]), f16_weights=pd.last_decode_variant() == "mma")
    return out, lse


SHORT = [0, 1, 15, 16, 17, 31, 33, 64, 65, 130, 300]


@pytest.mark.parametrize("kv", ["e4m3", "int8"])
@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("D,P,S,Hq,H", [(128, 16, 16, 8, 2), (64, 32, 16, 8, 2), (128, 64, 64, 16, 2),
                                        (64, 48, 48, 7, 7), (128, 256, 32, 10, 1), (128, 16, 16, 32, 2)])
def test_decode_tensor_core(kv, dt, D, P, S, Hq, H):
    _check(_case(SHORT, Hq, H, D, P, S, kv, dt, seed=D + P), "mma")


@pytest.mark.parametrize("kv", ["e4m3", "int8"])
@pytest.mark.parametrize("dt,D,P,S,Hq,H", [("bf16", 256, 16, 16, 4, 2), ("f16", 128, 8, 8, 8, 2),
                                           ("bf16", 64, 20, 5, 6, 2), ("f32", 128, 16, 16, 9, 1),
                                           ("bf16", 128, 1, 1, 4, 4), ("f16", 128, 32, 8, 4, 1),
                                           ("f32", 64, 7, 7, 3, 3), ("f32", 256, 3, 1, 2, 1),
                                           ("f16", 64, 255, 85, 8, 2), ("bf16", 128, 11, 11, 32, 2),
                                           ("f16", 64, 32, 2, 7, 7), ("bf16", 128, 256, 8, 16, 1)])
def test_decode_other_shapes(kv, dt, D, P, S, Hq, H):
    _check(_case(SHORT, Hq, H, D, P, S, kv, dt, seed=D + P), "simt" if D == 256 or dt == "f32" else "mma")


@pytest.mark.parametrize("splits", [0, 1, 2, 7])
@pytest.mark.parametrize("kv,D,P,S", [("e4m3", 128, 32, 32), ("int8", 64, 32, 32), ("int8", 128, 8, 8), ("e4m3", 64, 20, 4)])
def test_decode_splits_and_lengths(splits, kv, D, P, S):
    c = _case([3000, 0, 1, 4096, 517, 16], 8, 2, D, P, S, kv, "bf16", seed=7)
    _check(c, "mma", num_splits=splits)
    _check(c, "mma", num_splits=splits, out_dt=torch.float32)


@pytest.mark.parametrize("lengths,Hq,H,n", [([300], 32, 8, 1), ([64, 1, 0, 70, 3], 8, 8, 1), ([5000, 30, 200], 8, 2, 1),
                                            ([40] * 37, 4, 4, 1), ([900, 3, 77], 8, 2, 2), ([700, 20], 32, 2, 1),
                                            ([100, 16, 4000, 0], 16, 4, 4)])
@pytest.mark.parametrize("kv,D,P,S", [("int8", 128, 16, 16), ("e4m3", 64, 64, 32), ("e4m3", 128, 8, 4)])
def test_decode_planned_on_the_host(lengths, Hq, H, n, kv, D, P, S):
    """Host copies of the table: a block per segment for short or even sequences, else equal
    shares, at every warp count a segment can have."""
    c = _case(lengths, Hq, H, D, P, S, kv, "bf16", n=n, seed=len(lengths))
    host = pd.host_meta_of(c["indptr"], c["li"])
    for early in (False, True):
        _check(c, "mma", host_meta=host, early_inputs=early)
    _check(c, "mma", host_meta=host, num_splits=3)
    if n == 1:
        w = _case(lengths, Hq, H, D, P, S, kv, "bf16", n=n, seed=len(lengths),
                  wins=[(L // 2, min(4, L // 2)) for L in lengths])
        _check(w, "mma", host_meta=pd.host_meta_of(w["indptr"], w["li"]), sink=torch.randn(Hq, device=DEV))


def test_decode_one_long_sequence():
    _check(_case([70001], 8, 1, 128, 64, 16, "int8", "bf16", seed=8), "mma")


@pytest.mark.parametrize("P,D", [(16, 128), (64, 64), (8, 128), (20, 64)])
def test_decode_window_and_sinks(P, D):
    lengths = [5, 100, 333, 1000, 64]
    wins = [(0, 0), (50, 4), (301, 1), (999, 20), (17, 17)]
    _check(_case(lengths, 8, 2, D, P, P, "e4m3", "bf16", wins=wins, seed=9))
    _check(_case(lengths, 8, 2, D, P, P, "int8", "f16", wins=wins, seed=9), num_splits=5)


@pytest.mark.parametrize("n,Hq,H,D,P,S", [(2, 8, 2, 128, 16, 16), (3, 8, 8, 64, 32, 16), (5, 12, 2, 128, 32, 32),
                                          (4, 16, 2, 64, 16, 16), (9, 4, 4, 128, 64, 16),
                                             (2, 8, 2, 128, 8, 8), (3, 8, 8, 64, 20, 5), (5, 12, 2, 128, 1, 1)])
@pytest.mark.parametrize("kv", ["e4m3", "int8"])
def test_decode_several_queries(n, Hq, H, D, P, S, kv):
    # lengths below q_len leave the first tokens without a row
    _check(_case([0, 1, 2, n, 40, 333, 1025], Hq, H, D, P, S, kv, "bf16", n=n, seed=n), "mma")


@pytest.mark.parametrize("pow2", [False, True])
@pytest.mark.parametrize("kv,dt,S", [("e4m3", "bf16", 16), ("int8", "f16", 16), ("int8", "bf16", 4)])
def test_decode_scales_far_apart(kv, dt, S, pow2):
    """V scales over 2^+-24 (K's tame, or every softmax would have one row), with zero and
    smallest scales among them: blocks of small weight and large scale count as much as others."""
    c = _case([200, 1500, 40], 8, 2, 128, 16, S, kv, dt, seed=11, spread=0.5, pow2=pow2)
    g = torch.Generator().manual_seed(12)
    ok = ~torch.isnan(c["scales"][:, 1])
    f = torch.exp2(torch.randint(-24, 25, ok.shape, generator=g).float()).to(DEV)
    f[torch.rand(ok.shape, generator=g).to(DEV) < 0.1] = 0.0
    f[torch.rand(ok.shape, generator=g).to(DEV) < 0.1] = 2.0 ** -110
    c["scales"][:, 1] *= f
    _check(c, "mma", out_dt=torch.float32)
    _check(c, "mma", out_dt=torch.float32, num_splits=9)


def test_decode_rising_scores():
    """Scores that grow along the sequence, and a peaked softmax: the running maxima move."""
    c = _case([2000, 700], 8, 2, 128, 16, 16, "int8", "bf16", seed=13, q_gain=6.0)
    ip = c["indptr"].tolist()
    for b in range(2):
        pages = c["vals"][ip[b]:ip[b + 1]].long()
        c["scales"][pages, 0] *= torch.linspace(0.1, 2.0, len(pages), device=DEV)[:, None, None]
    _check(c, "mma")
    _check(c, "mma", num_splits=6)


@pytest.mark.parametrize("gain", [1e-6, 3e4])
def test_decode_query_magnitudes(gain):
    """Q far from 1, undone by the scale of K: the column scaling keeps every bit."""
    c = _case([100, 900], 8, 2, 128, 16, 16, "e4m3", "bf16", seed=14, q_gain=gain)
    c["scales"][:, 0] /= gain
    _check(c, "mma")


def test_decode_learned_sink_and_host_plan():
    c = _case([0, 1, 700, 2100], 8, 2, 128, 32, 32, "e4m3", "bf16", seed=15)
    sink = torch.randn(8, device=DEV)
    dev = _check(c, "mma", sink=sink)
    host = pd.host_meta_of(c["indptr"], c["li"])
    got = _check(c, "mma", sink=sink, host_meta=host)
    assert torch.equal(dev[0], got[0]) and torch.equal(dev[1], got[1])
    _check(c, "mma", sink=sink, num_splits=1)


@pytest.mark.parametrize("P", [16, 8])
def test_decode_more_sequences_than_the_scan_caches(P):
    g = torch.Generator().manual_seed(22)
    lengths = torch.randint(0, 60, (1300,), generator=g).tolist()
    _check(_case(lengths, 2, 1, 64, P, P, "int8", "f16", seed=23))


@pytest.mark.parametrize("lengths,splits", [([40, 1000, 7], 0), ([40, 1000, 7], 1), ([5000], 0)])
def test_decode_into_unaligned_outputs(lengths, splits):
    c = _case(lengths, 8, 2, 128, 16, 16, "e4m3", "bf16", seed=24)
    ref = _ref(c)
    for dt in (torch.bfloat16, torch.float32):
        buf = torch.zeros(len(lengths) * 8 * 128 + 9, dtype=dt, device=DEV)
        out = buf[3:3 + len(lengths) * 8 * 128].view(len(lengths), 8, 128)
        lse = torch.empty(len(lengths), 8, device=DEV)
        pd.batch_decode_paged_kv_bs(c["Q"][:, 0].contiguous(), c["codes"].view(KV["e4m3"]), c["scales"], c["indptr"],
                                    c["vals"], c["li"], out, lse, num_splits=splits)
        assert pd.check_device_errors() == "PD_OK"
        check_decode(out, lse, ref, max(lengths))
        assert (buf[:3] == 0).all() and (buf[-6:] == 0).all()


def test_decode_two_streams_at_once():
    """Split decodes in flight together, each with its stream's own workspace."""
    cs = [_case([3000, 900, 40], 8, 2, 128, 16, 16, "int8", "bf16", seed=25 + i) for i in range(2)]
    refs = [_ref(c) for c in cs]
    st = [torch.cuda.Stream() for _ in cs]
    Q = [c["Q"][:, 0].contiguous() for c in cs]
    outs = [torch.empty_like(q) for q in Q]
    lses = [torch.empty(q.shape[:-1], device=DEV) for q in Q]
    torch.cuda.synchronize()
    for _ in range(20):
        for c, s, q, o, l in zip(cs, st, Q, outs, lses):
            pd.batch_decode_paged_kv_bs(q, c["codes"], c["scales"], c["indptr"], c["vals"], c["li"], o, l, stream=s)
    torch.cuda.synchronize()
    assert pd.check_device_errors() == "PD_OK"
    for o, l, r in zip(outs, lses, refs):
        check_decode(o, l, r, 3000)


def test_decode_is_the_same_every_time():
    c = _case([5000, 3, 900], 16, 2, 128, 16, 16, "int8", "bf16", seed=16)
    a = _run(c)
    for _ in range(5):
        b = _run(c)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("S", [16, 8])
def test_decode_nonfinite_scale_stays_in_its_block(S):
    for n, dt in ((1, "bf16"), (2, "f16")):
        c = _case([100, 100, 40], 8, 2, 128, 16, S, "e4m3", dt, n=n, seed=17)
        ref = _ref(c)
        ip = c["indptr"].tolist()
        # the last page of sequence 1, V of head 0: only heads 0-3 of sequence 1 are touched,
        # and of several queries only those that attend a row of the block
        c["scales"][int(c["vals"][ip[2] - 1]), 1, 0, 0] = float("nan")  # (rows 96-99 of 100)
        out, lse = _run(c)
        out, lse = out.view(3, n, 8, 128), lse.view(3, n, 8)
        assert torch.isnan(out[1, :, :4]).all() and torch.isfinite(out[1, :, 4:]).all()
        keep = [0, 2]
        check_decode(out[keep], lse[keep], (ref[0][keep], ref[1][keep], tuple(x[keep] for x in ref[2])), 100)
    # a block that an earlier query token does not attend: 17 rows, 2 tokens, token 0 sees 16
    c = _case([17], 4, 1, 128, 16, S, "e4m3", "bf16", n=2, seed=18)
    ref = _ref(c)
    for side in (0, 1):
        d = dict(c, scales=c["scales"].clone())
        d["scales"][int(c["vals"][1]), side, 0, 0] = float("nan")
        out, lse = _run(d)
        assert torch.isnan(out[0, 1]).all()
        check_decode(out[:, :1], lse[:, :1], (ref[0][:, :1], ref[1][:, :1], tuple(x[:, :1] for x in ref[2])), 17)


def test_decode_bad_page_ids_are_skipped_and_reported():
    for P in (16, 8):
        c = _case([200, 100], 8, 2, 128, P, P, "int8", "bf16", seed=19)
        good = _ref(c)
        c["vals"][2] = c["codes"].shape[0]
        c["vals"][3] = -1
        out, lse = _run(c)
        assert pd.check_device_errors() == "PD_ERR_BAD_PAGE"
        assert torch.isfinite(out.float()).all()
        check_decode(out[1:], lse[1:], (good[0][1:], good[1][1:], tuple(x[1:] for x in good[2])), 100,
                     f16_weights=True)
        assert pd.check_device_errors() == "PD_OK"


def test_decode_far_into_a_large_pool():
    """Page ids whose codes lie beyond 2^32 bytes."""
    H, P, D = 8, 64, 128
    n = (5 << 30) // (2 * H * P * D)
    g = torch.Generator().manual_seed(20)
    codes = torch.zeros(n, 2, H, P, D, dtype=torch.int8, device=DEV)
    scales = torch.ones(n, 2, H, 1, device=DEV)
    ids = torch.tensor([n - 1, n - 2, 0, n // 2, n - 7], device=DEV)
    small, s = cache(5, H, P, P, D, "int8", DEV, g)
    codes[ids], scales[ids] = small, s
    c = dict(Q=torch.randn(1, 1, 16, D, generator=g).bfloat16().to(DEV), codes=codes, scales=scales,
             indptr=torch.tensor([0, 5], dtype=torch.int32, device=DEV), vals=ids.int(),
             li=torch.tensor([9], dtype=torch.int32, device=DEV), lengths=[4 * P + 9], P=P, kv="int8",
             wins=None, n=1, D=D)
    _check(c, "mma")


def test_decode_workspaces():
    c = _case([3000, 900, 40], 8, 2, 128, 16, 16, "int8", "bf16", seed=21)
    Q = c["Q"][:, 0].contiguous()
    from paged_kv_decode_19_gb300 import _lib
    d = _lib.DecodeDesc(3, 8, 2, 128, 16, 2, 4, 2, 0, 0, c["codes"].shape[0], c["vals"].numel(), 0, 1.0, 1.0, 0)
    need = pd.workspace_size_bs(d, 1, 16)
    assert need > 0
    ws = torch.zeros(need, dtype=torch.uint8, device=DEV)
    a, b = _run(c), _run(c, ws=ws)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    with pytest.raises(pd.PDError) as e:
        _run(c, ws=ws[: need - 256])
    assert e.value.status_name == "PD_ERR_WORKSPACE"
    assert Q.shape == a[0].shape


# ------------------------------------------------------------------------------- append
def _append_ref(codes, scales, kv, k, v, at, indptr, vals, last, P):
    """The definition, block by block, in 64 bits: (codes, scales) after the append."""
    codes, scales = codes.clone(), scales.clone()
    S = P // scales.shape[3]
    for b in range(len(at) - 1):
        n = at[b + 1] - at[b]
        L = (indptr[b + 1] - indptr[b] - 1) * P + last[b] if indptr[b + 1] > indptr[b] else 0
        lo = L - n
        while lo < L:
            hi = min(L, (lo // S + 1) * S)
            page, sb = vals[indptr[b] + lo // P], lo % P // S
            base = sb * S
            r0, r1 = lo % P, lo % P + hi - lo
            for w, x in ((0, k), (1, v)):
                rows = x[at[b + 1] - (L - lo):at[b + 1] - (L - hi)].double().transpose(0, 1)  # [H, rows, D]
                finite = torch.isfinite(rows).all(-1).all(-1)
                amax = torch.where(torch.isfinite(rows), rows.abs(), 0.0).amax((-1, -2))
                need = torch.where(finite, pow2_need(amax, kv), float("nan"))
                was = scales[page, w, :, sb].double()
                new = need
                if r0 > base:
                    new = torch.where(torch.isnan(was), was, torch.where(torch.isnan(need), need, torch.maximum(was, need)))
                    ratio = (was.float() / new.float()).double()
                    move = (new != was) & ~torch.isnan(new)
                    old = values(codes[page, w, :, base:r0], kv)
                    moved = encode((old * ratio[:, None, None]).float().double(), kv)
                    codes[page, w, :, base:r0] = torch.where(move[:, None, None], moved, codes[page, w, :, base:r0])
                q = (rows.float() / new.float()[:, None, None]).double()
                ok = ~torch.isnan(new)
                codes[page, w, :, r0:r1] = torch.where(ok[:, None, None], encode(torch.where(ok[:, None, None], q, 0.0), kv), 0)
                scales[page, w, :, sb] = new.float()
            lo = hi
    return codes, scales


def _append_case(new, old, H, D, P, S, kv, dt, seed=0, fused=False, gain=1.0, odd=0):
    g = torch.Generator().manual_seed(seed)
    indptr, vals, last, total = table([a + b for a, b in zip(new, old)], P, DEV, g)
    codes, scales = cache(total, H, P, S, D, kv, DEV, g, spread=1.5, pow2=True)
    at = [0]
    for n in new:
        at.append(at[-1] + n)
    T = at[-1]
    if fused:  # k and v as slices of a projection's output, possibly not 16-byte aligned
        x = torch.randn(T, 3 * H * D + odd, generator=g).to(DT[dt]).to(DEV) * gain
        k, v = (x[:, odd + i * H * D: odd + (i + 1) * H * D].unflatten(1, (H, D)) for i in (1, 2))
    else:
        k, v = ((torch.randn(T, H, D, generator=g) * gain).to(DT[dt]).to(DEV) for _ in range(2))
    return codes, scales, k, v, at, indptr, vals, last


def _append_check(new, old, H, D, P, S, kv, dt, mutate=None, **kw):
    codes, scales, k, v, at, indptr, vals, last = _append_case(new, old, H, D, P, S, kv, dt, **kw)
    if mutate:
        mutate(codes, scales, k, v)
    want = _append_ref(codes, scales, kv, k, v, at, indptr.tolist(), vals.tolist(), last.tolist(), P)
    pd.append_paged_kv_bs(codes.view(KV[kv]), scales, k, v, torch.tensor(at, dtype=torch.int32, device=DEV),
                          indptr, vals, last)
    assert pd.check_device_errors() == "PD_OK"
    assert torch.equal(scales.nan_to_num(-1.0), want[1].nan_to_num(-1.0))
    # e4m3 has two zeros; both stand for 0
    same = codes == want[0]
    if kv == "e4m3":
        same |= ((codes & 0x7F) == 0) & ((want[0] & 0x7F) == 0)
    assert same.all()
    return codes, scales, k, v


@pytest.mark.parametrize("kv", ["e4m3", "int8"])
@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("H,D,P,S", [(2, 128, 16, 16), (3, 64, 32, 8), (1, 256, 20, 20), (8, 128, 256, 256),
                                     (2, 64, 1, 1), (5, 128, 48, 16)])
def test_append(kv, dt, H, D, P, S):
    _append_check([1, 0, 5, 300, 1, 17, 2, 33], [0, 9, 3, 40, 15, 0, 100, 31], H, D, P, S, kv, dt, seed=D + P)


@pytest.mark.parametrize("kv", ["e4m3", "int8"])
def test_append_one_token_each(kv):
    n = 100
    _append_check([1] * n, [i % 37 for i in range(n)], 8, 128, 16, 16, kv, "bf16", seed=2)
    # large new rows: every part-filled block grows and is recoded
    _append_check([1] * n, [i % 37 for i in range(n)], 8, 128, 16, 16, kv, "bf16", seed=3, gain=100.0)
    # tiny ones: no scale moves, the new codes are small
    _append_check([1] * n, [i % 37 for i in range(n)], 8, 128, 16, 16, kv, "f16", seed=4, gain=1e-4)


@pytest.mark.parametrize("odd", [0, 8, 1])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_append_slices_of_a_projection(dt, odd):
    _append_check([3, 40, 1], [5, 0, 31], 4, 64, 32, 16, "int8", dt, fused=True, odd=odd, seed=5)


def test_append_many_sequences():
    """More sequences than one round of the search, empty ones among them."""
    for B, seed in ((33, 1), (1025, 2), (3000, 3)):
        g = torch.Generator().manual_seed(seed)
        new = torch.randint(0, 3, (B,), generator=g).tolist()
        old = torch.randint(0, 20, (B,), generator=g).tolist()
        _append_check(new, old, 1, 64, 16, 16, "int8", "bf16", seed=seed)


def test_append_scales_of_the_caller():
    """Scales that are no powers of two stay until they must grow."""
    def mutate(codes, scales, k, v):
        scales *= 1.37
    for kv in ("e4m3", "int8"):
        _append_check([1, 2, 7], [3, 14, 9], 2, 64, 16, 16, kv, "f32", mutate=mutate, seed=6)
        _append_check([1, 2, 7], [3, 14, 9], 2, 64, 16, 16, kv, "f32", mutate=mutate, seed=6, gain=50.0)


def test_append_extremes():
    def zeros(codes, scales, k, v):
        k.zero_()
        v[1:] = 0

    def largest(codes, scales, k, v):
        k.fill_(3.3e38)
        v.fill_(-3.4028234663852886e38)

    def smallest(codes, scales, k, v):
        k.fill_(1e-45)
        v.fill_(1.2e-38)

    def broken(codes, scales, k, v):
        k[0, 0, 5] = float("nan")
        v[3, 1, 0] = float("-inf")
        scales[:, 1, 0] = float("nan")
    for kv in ("e4m3", "int8"):
        for f in (zeros, largest, smallest, broken):
            _append_check([1, 4, 20, 3], [5, 0, 16, 2], 2, 64, 16, 16, kv, "f32", mutate=f, seed=7)
    # the borders of the rule: amax exactly the largest code times a power of two, and one step above
    for kv, top in (("e4m3", 448.0), ("int8", 127.0)):
        for x in (top, math.nextafter(top, 1e9), top / 8, top * 4):
            def fill(codes, scales, k, v, x=x):
                k.fill_(x)
                v.copy_(torch.nextafter(k, torch.full_like(k, 1e9)))
            _append_check([16, 3], [0, 0], 1, 64, 16, 16, kv, "f32", mutate=fill, seed=8)


def test_append_token_by_token_is_a_chunk_for_normal_codes():
    """e4m3 with powers of two: values whose codes stay normal come out the same however the
    sequence was cut into appends."""
    H, D, P = 2, 64, 16
    g = torch.Generator().manual_seed(9)
    x = (1.0 + torch.rand(40, 2, H, D, generator=g)).to(torch.bfloat16).to(DEV)
    x *= torch.exp2(torch.randint(-2, 3, (40, 1, 1, 1), generator=g).float()).to(DEV).bfloat16()
    res = []
    for step in (40, 1, 7):
        pages = torch.zeros(3, 2, H, P, D, dtype=torch.int8, device=DEV)
        scales = torch.zeros(3, 2, H, 1, device=DEV)
        for i in range(0, 40, step):
            j = min(40, i + step)
            t = lambda a: torch.tensor(a, dtype=torch.int32, device=DEV)
            npg = -(-j // P)
            pd.append_paged_kv_bs(pages.view(KV["e4m3"]), scales, x[i:j, 0].contiguous(), x[i:j, 1].contiguous(),
                                  t([0, j - i]), t([0, npg]), t(list(range(npg))), t([j - (npg - 1) * P]))
        assert pd.check_device_errors() == "PD_OK"
        res.append((pages, scales))
    for r in res[1:]:
        assert torch.equal(r[0], res[0][0]) and torch.equal(r[1], res[0][1])


def test_append_leaves_bad_tables_alone():
    codes, scales, k, v, at, indptr, vals, last = _append_case([4, 3, 20, 2], [5, 0, 16, 2], 2, 64, 16, 16, "int8", "bf16")
    t = lambda a: torch.tensor(a, dtype=torch.int32, device=DEV)

    def run(at=at, indptr=indptr, vals=vals, last=last):
        c, s = codes.clone(), scales.clone()
        pd.append_paged_kv_bs(c.view(torch.int8), s, k, v, t(at), indptr, vals, last)
        return c, s, pd.check_device_errors()
    good = run()
    assert good[2] == "PD_OK"
    # a sequence longer than its table: its pages stay, the others are written
    bad = last.clone()
    bad[1] = 2
    c, s, st = run(last=bad)
    assert st == "PD_ERR_BAD_LENGTH"
    mine = vals[int(indptr[1]):int(indptr[2])].long()
    others = torch.ones(codes.shape[0], dtype=torch.bool, device=DEV)
    others[mine] = False
    assert torch.equal(c[mine], codes[mine]) and torch.equal(c[others], good[0][others])
    for wrong in ([0, 4, 7, 200, 29], [0, -4, 7, 27, 29], [0, 9, 7, 27, 29]):
        assert run(at=wrong)[2] == "PD_ERR_BAD_LENGTH"
    over = last.clone()
    over[0] = 17
    assert run(last=over)[2] == "PD_ERR_BAD_LENGTH"
    for page in (-1, codes.shape[0]):
        bad = vals.clone()
        bad[0] = page
        assert run(vals=bad)[2] == "PD_ERR_BAD_PAGE"
    assert run()[2] == "PD_OK"


# ------------------------------------------------------------------------------- together
def _step_buffers(lengths, Hq, H, D, P, kv, dt, seed):
    g = torch.Generator().manual_seed(seed)
    indptr, vals, last, total = table(lengths, P, DEV, g)
    codes, scales = cache(total, H, P, P, D, kv, DEV, g, pow2=True)
    B = len(lengths)
    qkv = torch.randn(B, Hq + 2 * H, D, generator=g).to(DT[dt]).to(DEV)
    w = [(1 + 0.1 * torch.randn(D, generator=g)).to(DT[dt]).to(DEV) for _ in range(2)]
    pos = torch.tensor([max(0, n - 1) for n in lengths], dtype=torch.int32, device=DEV)
    at = torch.arange(B + 1, dtype=torch.int32, device=DEV)
    return dict(qkv=qkv, w=w, pos=pos, at=at, indptr=indptr, vals=vals, last=last, codes=codes, scales=scales,
                q=torch.empty(B, Hq, D, dtype=DT[dt], device=DEV), k=torch.empty(B, H, D, dtype=DT[dt], device=DEV),
                out=torch.empty(B, Hq, D, dtype=DT[dt], device=DEV), lse=torch.empty(B, Hq, device=DEV))


def _step(s, freq, Hq, H, kv, early=True):
    pd.qk_norm_rope(s["qkv"][:, :Hq], s["qkv"][:, Hq:Hq + H], *s["w"], s["pos"], freq, s["q"], s["k"])
    pd.append_paged_kv_bs(s["codes"].view(KV[kv]), s["scales"], s["k"], s["qkv"][:, Hq + H:], s["at"], s["indptr"],
                          s["vals"], s["last"])
    pd.batch_decode_paged_kv_bs(s["q"], s["codes"].view(KV[kv]), s["scales"], s["indptr"], s["vals"], s["last"],
                                s["out"], s["lse"], early_inputs=early)


def _step_check(s, was, lengths, Hq, H, D, P, kv, freq):
    """The step's cache from its own q and k, and its output from that cache."""
    from tests.test_qk_norm_rope_gpu import check_norm_rope
    check_norm_rope(s["qkv"][:, :Hq], s["w"][0], s["pos"], freq, s["q"])
    check_norm_rope(s["qkv"][:, Hq:Hq + H], s["w"][1], s["pos"], freq, s["k"])
    want = _append_ref(*was, kv, s["k"], s["qkv"][:, Hq + H:], s["at"].tolist(), s["indptr"].tolist(),
                       s["vals"].tolist(), s["last"].tolist(), P)
    assert torch.equal(s["scales"], want[1]) and torch.equal(values(s["codes"], kv), values(want[0], kv))
    ref = decode_ref(s["q"][:, None], s["codes"], s["scales"], kv, s["indptr"], s["vals"], lengths, P, D ** -0.5)
    check_decode(s["out"], s["lse"], ref, max(lengths))


@pytest.mark.parametrize("kv", ["e4m3", "int8"])
def test_a_decode_step(kv):
    Hq, H, D, P = 8, 2, 128, 16
    lengths = [1, 17, 32, 900, 2049]
    freq = pd.rope_frequencies(D, 5e5, "parts", 8.0, 8192, device=DEV)
    s = _step_buffers(lengths, Hq, H, D, P, kv, "bf16", 31)
    was = s["codes"].clone(), s["scales"].clone()
    for early in (False, True):
        s["codes"].copy_(was[0])
        s["scales"].copy_(was[1])
        _step(s, freq, Hq, H, kv, early)
        assert pd.check_device_errors() == "PD_OK"
        _step_check(s, was, lengths, Hq, H, D, P, kv, freq)


def test_a_decode_step_captured_and_on_two_streams():
    Hq, H, D, P, kv = 8, 2, 128, 16, "int8"
    freq = pd.rope_frequencies(D, 1e4, device=DEV)
    sets = [([1000, 5, 300, 4000], 41), ([900, 2, 310, 3999], 42)]
    graphs, kept = [], []
    for lengths, seed in sets:
        s = _step_buffers(lengths, Hq, H, D, P, kv, "bf16", seed)
        was = s["codes"].clone(), s["scales"].clone()
        st = torch.cuda.Stream()
        st.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(st):
            _step(s, freq, Hq, H, kv)
        st.synchronize()
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr, stream=st):
            _step(s, freq, Hq, H, kv)
        graphs.append((gr, st))
        kept.append((s, was, lengths))
    for _ in range(3):
        for (s, was, _), (gr, st) in zip(kept, graphs):  # both in flight at once, each on its stream
            with torch.cuda.stream(st):
                s["codes"].copy_(was[0])
                s["scales"].copy_(was[1])
                s["out"].fill_(float("nan"))
                gr.replay()
        torch.cuda.synchronize()
        assert pd.check_device_errors() == "PD_OK"
        for s, was, lengths in kept:
            _step_check(s, was, lengths, Hq, H, D, P, kv, freq)


def test_a_decode_step_on_a_replayed_table():
    """One captured step, replayed with another table and other lengths in its buffers."""
    Hq, H, D, P, kv = 8, 2, 64, 32, "e4m3"
    freq = pd.rope_frequencies(D, 1e4, device=DEV)
    a = _step_buffers([1000, 40, 300], Hq, H, D, P, kv, "f16", 51)
    lengths = [993, 64, 289]  # the same page counts
    b = _step_buffers(lengths, Hq, H, D, P, kv, "f16", 52)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        _step(a, freq, Hq, H, kv)
    st.synchronize()
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr, stream=st):
        _step(a, freq, Hq, H, kv)
    for n in ("qkv", "pos", "at", "indptr", "vals", "last", "codes", "scales"):
        a[n].copy_(b[n])
    for x, y in zip(a["w"], b["w"]):
        x.copy_(y)
    was = a["codes"].clone(), a["scales"].clone()
    gr.replay()
    torch.cuda.synchronize()
    assert pd.check_device_errors() == "PD_OK"
    _step_check(a, was, lengths, Hq, H, D, P, kv, freq)


def test_context_split_over_ranks():
    """A rank's slice of the context decoded to fp32 partials, merged: the unsplit decode."""
    Hq, H, D, P, kv = 8, 2, 128, 16, "int8"
    c = _case([1000, 37, 0, 2048], Hq, H, D, P, P, kv, "bf16", seed=61)
    V, S = [], []
    for r in range(3):
        ip, vals, li, _ = pd.cp_shard_plan(c["indptr"].cpu().numpy(), c["vals"].cpu().numpy(), c["li"].cpu().numpy(),
                                           None, P, 3, r)
        t = lambda a: torch.from_numpy(a).to(DEV)
        part = dict(c, indptr=t(ip), vals=t(vals), li=t(li))
        o, l = _run(part, torch.float32)
        V.append(o)
        S.append(l)
    out = torch.empty(4, Hq, D, dtype=torch.bfloat16, device=DEV)
    lse = torch.empty(4, Hq, device=DEV)
    pd.merge_states(out, lse, torch.stack(V), torch.stack(S))
    assert pd.check_device_errors() == "PD_OK"
    check_decode(out, lse, _ref(c), 2048)
    assert TOP[kv] == 127.0
