"""4-bit caches and page tables for the tests: seeded inputs, and the operators' definitions in 64
bits or on lists, one row, block or request at a time."""
import math

import torch

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SC = {"e4m3": torch.float8_e4m3fn, "e8m0": torch.float8_e8m0fnu}
BLOCK = {"e4m3": 16, "e8m0": 32}
MAG = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def scale_values(b, sc):
    """fp64 values of scale bytes."""
    if sc == "e4m3":
        return b.view(torch.float8_e4m3fn).float().double()
    v = torch.exp2(b.double() - 127)
    return torch.where(b == 255, math.nan, v)


def code_values(codes):
    """fp64 values of packed codes [..., D / 2] -> [..., D]."""
    v = torch.tensor(MAG + [-x for x in MAG], dtype=torch.float64, device=codes.device)
    return torch.stack([v[(codes & 15).long()], v[(codes >> 4).long()]], -1).flatten(-2)


def row_values(codes, scales, sc):
    return (code_values(codes).unflatten(-1, (-1, BLOCK[sc])) * scale_values(scales, sc)[..., None]).flatten(-2)


def quantise_ref(x, g, sc):
    """Rows [..., D] (fp64 of the inputs) -> packed codes and scale bytes, from the definition: the
    scale by trial over all stored values, the code as the nearest of the eight magnitudes."""
    n = BLOCK[sc]
    # the quotient by g is rounded to fp32 by definition
    y = (x / g).float().double().unflatten(-1, (-1, n))
    finite = torch.isfinite(y).all(-1)
    y0 = torch.where(finite[..., None], y, 0.0)
    a = y0.abs().amax(-1)
    if sc == "e4m3":
        grid = torch.arange(1, 127, dtype=torch.uint8, device=x.device)  # 2^-9 .. 448
        v = scale_values(grid, sc)
        t = (a / 6).clamp(v[0].item(), v[-1].item())
        hi = torch.searchsorted(v, t).clamp(1, len(v) - 1)
        up, down = v[hi] - t, t - v[hi - 1]
        # ties to the even code (grid[i] = i + 1)
        byte = torch.where((up < down) | ((up == down) & (grid[hi] % 2 == 0)), grid[hi], grid[hi - 1])
        byte = torch.where(finite, byte, torch.tensor(0x7f, dtype=torch.uint8, device=x.device))
    else:
        k = torch.full_like(a, 13)
        for e in range(12, -15, -1):
            k = torch.where(a <= 6 * 2.0 ** e, float(e), k)
        byte = (k + 127).to(torch.uint8)
        byte = torch.where(finite, byte, torch.tensor(0xff, dtype=torch.uint8, device=x.device))
    s = torch.where(finite, scale_values(byte, sc), 1.0)
    m = (y0.abs() / s[..., None]).clamp(max=6.0)
    mag = torch.tensor(MAG, dtype=torch.float64, device=x.device)
    d = (m[..., None] - mag).abs()
    best = d.amin(-1, keepdim=True)
    near = d == best
    even = near & (torch.arange(8, device=x.device) % 2 == 0)
    code = torch.where(even.any(-1), even.double().argmax(-1), near.double().argmax(-1))
    code = code + 8 * torch.signbit(y0)
    code = torch.where(finite[..., None], code, 0).flatten(-2).to(torch.uint8)
    return code[..., 0::2] | (code[..., 1::2] << 4), byte


def table(lengths, P, dev, gen, extra=3, total=None):
    """indptr, values, last page lengths (device int32) of a shuffled table, and the pool's pages."""
    counts = [-(-n // P) for n in lengths]
    indptr = [0]
    for n in counts:
        indptr.append(indptr[-1] + n)
    total = total or indptr[-1] + extra
    vals = torch.randperm(total, generator=gen)[: indptr[-1]].to(torch.int32)
    last = [n - (c - 1) * P if c else 0 for n, c in zip(lengths, counts)]
    t = lambda a: torch.tensor(a, dtype=torch.int32, device=dev)  # noqa: E731
    return t(indptr), vals.to(dev), t(last), total


def cache(total, H, P, D, sc, dev, gen):
    """Random codes and scales (bytes); a few blocks are all zero."""
    codes = torch.randint(0, 256, (total, 2, H, P, D // 2), generator=gen, dtype=torch.uint8)
    n = D // BLOCK[sc]
    if sc == "e4m3":
        scales = torch.randint(0x20, 0x48, (total, 2, H, P, n), generator=gen, dtype=torch.uint8)
    else:
        scales = torch.randint(127 - 4, 127 + 2, (total, 2, H, P, n), generator=gen, dtype=torch.uint8)
    return codes.to(dev), scales.to(dev)


def attended(length, win=None):
    rows = torch.arange(length)
    if win is not None:
        start, sink = win
        rows = rows[(rows < sink) | (rows >= start)]
    return rows


def decode_ref(Q, codes, scales, sc, indptr, vals, lengths, P, sm, ks=1.0, vs=1.0, wins=None, sink=None):
    """out, lse (fp64) and, per output, A = sum p |v| / sum p; per query and head the largest |v|, the
    largest sum |q k| of a score (log2 units), both of the rows that are numbers.  Q [B, n, H_qo, D]."""
    B, n, Hq, D = Q.shape
    H = codes.shape[2]
    G, dev, f64 = Hq // H, Q.device, torch.float64
    out, A = (torch.zeros(B, n, Hq, D, dtype=f64, device=dev) for _ in range(2))
    lse = torch.full((B, n, Hq), -5e4, dtype=f64, device=dev)
    vmax, S = (torch.zeros(B, n, Hq, dtype=f64, device=dev) for _ in range(2))
    ip = indptr.tolist()
    for b in range(B):
        rows = attended(lengths[b], wins[b] if wins else None).to(dev)
        page, slot = vals[ip[b] + rows // P].long(), rows % P
        seen = torch.arange(len(rows), device=dev) <= (len(rows) - n + torch.arange(n, device=dev))[:, None]
        for h in range(H):
            k, v = (row_values(codes[page, w, h, slot], scales[page, w, h, slot], sc) * g for w, g in ((0, ks), (1, vs)))
            q = Q[b, :, h * G:(h + 1) * G].double()  # [n, G, D]
            s = torch.einsum("tgd,rd->tgr", q, k) * sm
            s = s.masked_fill(~seen[:, None], -math.inf)
            if sink is not None:
                extra = sink[h * G:(h + 1) * G].double().view(1, G, 1).expand(n, G, 1)
                s = torch.cat([s, extra], -1)
            if not s.shape[-1]:
                continue
            z = torch.logsumexp(s, -1)
            some = z > -math.inf
            p = torch.exp(s - torch.where(some, z, 0.0)[..., None])[..., :len(rows)]
            hs = slice(h * G, (h + 1) * G)
            lse[b, :, hs] = torch.where(some | z.isnan(), z / math.log(2), -5e4)
            if len(rows):
                # (a row that a token does not attend counts for nothing, whatever its scale)
                for t in range(n):
                    e = int(seen[t].sum())
                    out[b, t, hs] = p[t, :, :e] @ v[:e]
                    A[b, t, hs] = p[t, :, :e] @ v[:e].abs()
                    vmax[b, t, hs] = v[:e].abs().nan_to_num(0.0).amax() if e else 0.0
                mag = torch.einsum("tgd,rd->tgr", q.abs(), k.abs()) * abs(sm) / math.log(2)
                S[b, :, hs] = mag.nan_to_num(0.0).masked_fill(~seen[:, None], 0.0).amax(-1)
    return out, lse, (A, vmax, S)


def check_decode(out, lse, ref, rows, split, D):
    """Bounds from the arithmetic.  A tensor-core product aligns its 16 terms and the sum so far to the
    largest and may drop a unit of 2^-24 of it for each: a score of D / 16 of them (with F32 Q twice as
    many) is off by (D + D / 16) 2^-24 of its sum of magnitudes S; F32 Q as two f16 parts adds 2^-22 S.
    ex2 and the fma before it: 2^-20.  A weight is off by r = that, relative, the weighted mean by 2 r A,
    its sums over the rows by (17 rows / 16 + 40) 2^-24 A (twice as many products with F32 Q).  Weights
    are held between 2^7 and 2^15 for the largest; rounding them: 2^-11 A in f16, 2^-22 A in two parts,
    and half the least f16 step, 2^-25 of 2^7, for each row.  The output: half its own step."""
    o, l, (A, vmax, S) = ref
    o, A = o.view(out.shape), A.view(out.shape)
    l, vmax, S = l.view(lse.shape), vmax.view(lse.shape), S.view(lse.shape)
    two = 2 if split else 1
    r = math.log(2) * S * (two * (D + D / 16) * 2.0 ** -24 + (2.0 ** -22 if split else 0.0)) + 2.0 ** -20
    sums = two * (17 * rows / 16 + 40) * 2.0 ** -24
    half = torch.finfo(out.dtype).eps / 2
    tol = A * (2 * r[..., None] + sums + (2.0 ** -22 if split else 2.0 ** -11)) + half * o.abs()
    tol = tol + rows * 2.0 ** -32 * vmax[..., None]
    if out.dtype == torch.float16:
        tol = tol + 2.0 ** -25  # subnormal outputs
    err = (out.double() - o).abs()
    assert torch.equal(out.isnan(), o.isnan())
    fine = ~o.isnan()
    assert (err[fine] <= tol[fine] + 1e-30).all(), f"out error {(err / (tol + 1e-30))[fine].max().item():.2f} of its bound"
    lt = 1.4427 * (r + sums) + l.abs() * 2.0 ** -23 + 1e-6
    assert torch.equal(lse.isnan(), l.isnan())
    lerr, fl = (lse.double() - l).abs(), ~l.isnan()
    assert (lerr[fl] <= lt[fl]).all(), f"lse error {(lerr / lt)[fl].max().item():.2f} of its bound"


def tables_ref(page_table, lengths, new, state, ring, P, caps, window=0, sinks=0):
    """The step on lists: changes page_table, lengths, state and ring in place and returns (indptr,
    values written, append_indptr, length_info rows, slots, positions)."""
    indptr, values, at, info, slots, pos = [0], [], [0], [[], [], []], [], []
    need = lambda n: -(-n // P)  # noqa: E731
    width = len(page_table[0]) if page_table else 0
    good = [0 <= a <= width * P and 0 <= a + n <= width * P for a, n in zip(lengths, new)]
    grown = sum(max(0, need(a + n) - need(a)) for a, n, g in zip(lengths, new, good) if g)
    freed = sum(max(0, need(a) - need(a + n)) for a, n, g in zip(lengths, new, good) if g)
    pages = sum(need(a + n) for a, n, g in zip(lengths, new, good) if g)
    tokens = sum(max(n, 0) for n, g in zip(new, good) if g)
    spare = state[1] - state[0]
    fits = pages <= caps[0] and (caps[1] is None or tokens <= caps[1])
    fits = fits and (ring is None or (grown <= spare and spare + freed <= len(ring)))
    for b, (a, n) in enumerate(zip(lengths, new)):
        rows = a + n if fits and good[b] else 0
        if fits and good[b]:
            if ring is not None:
                for k in range(need(a), need(rows)):
                    page_table[b][k] = ring[state[0] % len(ring)]
                    state[0] += 1
                for k in range(need(rows), need(a)):
                    ring[state[1] % len(ring)] = page_table[b][k]
                    state[1] += 1
            for o in range(a, rows):
                page = page_table[b][o // P]
                slots.append(page * P + o % P if page >= 0 else -1)
                pos.append(o)
            lengths[b] = rows
        values += page_table[b][:need(rows)]
        indptr.append(len(values))
        at.append(len(slots))
        info[0].append(rows - (need(rows) - 1) * P if rows else 0)
        cut = window and rows > window + sinks
        info[1].append(rows - window if cut else 0)
        info[2].append(sinks if cut else 0)
    return indptr, values, at, info if window else info[:1], slots, pos
