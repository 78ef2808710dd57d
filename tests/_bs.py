"""Block-scaled 8-bit caches for the tests: seeded inputs, and the operators' definitions in
64 bits (plain torch, one sequence and head at a time)."""
import math

import torch

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
KV = {"e4m3": torch.float8_e4m3fn, "int8": torch.int8}
TOP = {"e4m3": 448.0, "int8": 127.0}


def values(codes, kv):
    """fp64 values of 8-bit codes stored as int8 bytes."""
    return codes.view(KV[kv]).float().double()


def encode(x, kv):
    """Nearest code (ties to even) of fp64 values within the range, as bytes."""
    if kv == "int8":
        return x.round().clamp(-127, 127).to(torch.int8)
    # every e4m3 value is exact in fp32; quantise in fp64 first, so the cast is exact
    quantum = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6))) - 3)
    y = (x / quantum).round() * quantum
    y = y.clamp(-448, 448).float().to(torch.float8_e4m3fn).view(torch.int8)
    return y


def pow2_need(amax, kv):
    """Smallest 2^k, k >= -126, with amax <= top * 2^k, in fp64, by trial."""
    k = torch.full_like(amax, -126.0)
    for step in (128.0, 64.0, 32.0, 16.0, 8.0, 4.0, 2.0, 1.0):  # largest k that is too small
        try_k = k + step
        k = torch.where(amax > TOP[kv] * torch.exp2(try_k - 1), try_k, k)
    return torch.exp2(k)


def table(lengths, P, dev, gen, extra=3):
    """indptr, values, last page lengths (device int32) of a shuffled table, and the pool's pages."""
    counts = [-(-n // P) for n in lengths]
    indptr = [0]
    for n in counts:
        indptr.append(indptr[-1] + n)
    total = indptr[-1] + extra
    vals = torch.randperm(total, generator=gen)[: indptr[-1]].to(torch.int32)
    last = [n - (c - 1) * P if c else 0 for n, c in zip(lengths, counts)]
    t = lambda a: torch.tensor(a, dtype=torch.int32, device=dev)
    return t(indptr), vals.to(dev), t(last), total


def cache(total, H, P, S, D, kv, dev, gen, spread=1.0, pow2=False):
    """Random codes (bytes) and scales 2^(spread * N(0,1)) / top."""
    pages = torch.randn(total, 2, H, P, D, generator=gen)
    codes = encode((pages * (TOP[kv] / 3.0)).double().clamp(-TOP[kv], TOP[kv]), kv)
    e = spread * torch.randn(total, 2, H, P // S, generator=gen)
    scales = torch.exp2(e.round() if pow2 else e) * (2.0 ** -7 if pow2 else 3.0 / TOP[kv])
    return codes.to(dev), scales.float().to(dev)


def attended(length, q_len=1, win=None):
    """Sequence offsets of the attended rows; win = (window start, sink rows)."""
    rows = torch.arange(length)
    if win is not None:
        start, sink = win
        rows = rows[(rows < sink) | (rows >= start)]
    return rows


def decode_ref(Q, codes, scales, kv, indptr, vals, lengths, P, sm_scale, wins=None, sink=None):
    """out, lse and, for error bounds, (A, vmax, S): per output sum p |v| / sum p, the largest
    |v|, and the largest sum |q k| of a score (log2 units); all fp64, Q [B, n, H_qo, D]."""
    B, n, Hq, D = Q.shape
    H, n_sb = codes.shape[2], scales.shape[3]
    S, G, dev = P // n_sb, Hq // H, Q.device
    out = torch.zeros(B, n, Hq, D, dtype=torch.float64, device=dev)
    A, vmax = out.clone(), torch.zeros(B, n, Hq, dtype=torch.float64, device=dev)
    lse = torch.full((B, n, Hq), -5e4, dtype=torch.float64, device=dev)
    sabs = torch.zeros(B, n, Hq, dtype=torch.float64, device=dev)
    ip = indptr.tolist()
    log2e = 1 / math.log(2)
    for b in range(B):
        rows = attended(lengths[b], n, wins[b] if wins else None).to(dev)
        if len(rows):
            page, slot = vals[ip[b] + rows // P].long(), rows % P
        for h in range(H):
            if len(rows):
                k, v = (values(codes[page, w, h, slot], kv) * scales[page, w, h, slot // S].double()[:, None]
                        for w in (0, 1))
            for t in range(n):
                end = len(rows) - n + 1 + t
                for g in range(G):
                    hq = h * G + g
                    q = Q[b, t, hq].double()
                    s = (k[:end] @ q) * sm_scale if end > 0 else torch.zeros(0, dtype=torch.float64, device=dev)
                    if sink is not None:
                        s = torch.cat([s, sink[hq].double().view(1)])
                    if not len(s):
                        continue
                    z = torch.logsumexp(s, 0)
                    lse[b, t, hq] = z * log2e
                    if end > 0:
                        p = torch.exp(s[:end] - z)
                        out[b, t, hq] = p @ v[:end]
                        A[b, t, hq] = p @ v[:end].abs()
                        vmax[b, t, hq] = v[:end].abs().max()
                        sabs[b, t, hq] = ((k[:end].abs() @ q.abs()).max()) * sm_scale * log2e
    return out, lse, (A, vmax, sabs)


def check_decode(out, lse, ref, max_len, f16_weights=True):
    """Bounds from the arithmetic.  A score is a sum of D exact products held in fp32 (at most
    24 roundings on a path of the tree, each of 2^-24 of the sum of magnitudes S) and ex2 and the
    scale products add 2^-21, so a weight is off by r = ln2 (24 2^-24 S) + 2^-20 relative, the
    weighted mean and its denominator by 2 r A; rounding the weights to f16 adds 2^-11 A, and
    2^-25 of the largest weight for each row below its normal range; the sums over the rows
    (max_len / 16 + 40) 2^-24; the output its own half step."""
    o, l, (A, vmax, S) = ref
    o, A = o.view(out.shape), A.view(out.shape)
    l, vmax, S = l.view(lse.shape), vmax.view(lse.shape), S.view(lse.shape)
    r = 0.694 * 24 * 2.0 ** -24 * S + 2.0 ** -20 + (max_len / 16 + 40) * 2.0 ** -24
    half = torch.finfo(out.dtype).eps / 2
    tol = A * (2 * r[..., None] + (2.0 ** -11 if f16_weights else 0.0)) + half * o.abs()
    if f16_weights:
        tol = tol + (max_len * 2.0 ** -25) * vmax[..., None]
    if out.dtype == torch.float16:
        tol = tol + 2.0 ** -25  # subnormal outputs
    err = (out.double() - o).abs()
    assert torch.isfinite(out.float()).all()
    worst = (err / (tol + 1e-30)).max().item() if err.numel() else 0.0
    assert (err <= tol + 1e-30).all(), f"out error {worst:.2f} of its bound"
    lt = 1.4427 * r + l.abs() * 2.0 ** -23 + 1e-6
    lerr = (lse.double() - l).abs()
    assert (lerr <= lt).all(), f"lse error {(lerr / lt).max().item():.2f} of its bound"
    return worst
