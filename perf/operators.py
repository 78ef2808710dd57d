"""What the 8-bit, block-scaled cache path costs: the head norms with the rotation, the append that
quantises, and the decode that reads the codes, at sizes of the serving loads this library runs.

Each operator has its plain form here (elementary torch operations in 32 bits, rounded once at the
end) and, where `own` is set, the library's call.  `exact` is the definition in 64 bits."""
import math
import random

import torch

own = False

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
LOG2E = 1.4426950408889634
EMPTY = -5e4  # log-sum-exp of a sequence that attends nothing


# ------------------------------------------------------------------------------- cases
def listed():
    return [
        # one new token of one sequence: launch latency
        dict(name="norm_rope one token", op="norm_rope", T=1, H_qo=32, H_kv=8, D=128, rd=128,
             mode=1, dt="bf16", norm=True, fused=True, scaling="none", far=0),
        # a decode step of 256 sequences, q and k as slices of the fused projection's output
        dict(name="norm_rope step of 256", op="norm_rope", T=256, H_qo=64, H_kv=8, D=128, rd=128,
             mode=1, dt="bf16", norm=True, fused=True, scaling="parts", far=0),
        # a long prefill chunk
        dict(name="norm_rope prefill 8192", op="norm_rope", T=8192, H_qo=32, H_kv=8, D=128, rd=128,
             mode=1, dt="bf16", norm=True, fused=True, scaling="linear", far=0),
        # half of each head rotated in the interleaved layout, no norm, positions far out
        dict(name="rope part interleaved", op="norm_rope", T=1777, H_qo=32, H_kv=4, D=64, rd=32,
             mode=2, dt="f32", norm=False, fused=False, scaling="parts", far=1000000),
        # one token for each of 256 sequences into part-filled blocks
        dict(name="append step of 256", op="append", H_kv=8, D=128, P=32, S=32, dt="bf16", kv="e4m3",
             seqs=256, n_lo=1, n_hi=1, old_hi=200, lens=3),
        # the tokens of a prefill chunk of few sequences
        dict(name="append prefill chunk", op="append", H_kv=8, D=128, P=16, S=16, dt="bf16", kv="int8",
             seqs=5, n_lo=700, n_hi=2900, old_hi=40, lens=4),
        # a mixed step: some sequences bring nothing, some one token, some a chunk; two blocks a page
        dict(name="append mixed", op="append", H_kv=4, D=64, P=64, S=32, dt="f16", kv="int8",
             seqs=37, n_lo=0, n_hi=90, old_hi=150, lens=5),
        # one short sequence: latency
        dict(name="decode one short", op="decode", B=1, H_qo=32, H_kv=8, D=128, P=16, S=16, dt="bf16",
             kv="int8", lo=200, hi=400, q_len=1, window=0, lens=6),
        # a batch of middling contexts
        dict(name="decode batch of 32", op="decode", B=32, H_qo=32, H_kv=8, D=128, P=16, S=16, dt="bf16",
             kv="int8", lo=512, hi=4096, q_len=1, window=0, lens=7),
        # many sequences, 64 query heads
        dict(name="decode batch of 256", op="decode", B=256, H_qo=64, H_kv=8, D=128, P=32, S=32, dt="bf16",
             kv="e4m3", lo=300, hi=4200, q_len=1, window=0, lens=8),
        # long contexts, four scales to a page
        dict(name="decode long contexts", op="decode", B=8, H_qo=32, H_kv=8, D=128, P=64, S=16, dt="bf16",
             kv="int8", lo=32768, hi=131072, q_len=1, window=0, lens=9),
        # verification of three drafted tokens, heads of 64
        dict(name="decode four queries", op="decode", B=24, H_qo=16, H_kv=8, D=64, P=32, S=16, dt="f16",
             kv="e4m3", lo=700, hi=6000, q_len=4, window=0, lens=10),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm_rope", "append", "decode", "decode"])
    H_qo, H_kv = rng.choice([(8, 2), (32, 8), (32, 4), (64, 8), (12, 4), (7, 7), (16, 1)])
    D = rng.choice([64, 128, 128])
    if op == "norm_rope":
        D = rng.choice([64, 128, 128, 256, 80])
        rd = rng.choice([D, D, D // 2, D // 4])
        return dict(op=op, T=_log(rng, 1, 9000), H_qo=H_qo, H_kv=H_kv, D=D, rd=rd, mode=rng.choice([1, 2]),
                    dt=rng.choice(["bf16", "bf16", "f16", "f32"]), norm=rng.random() < 0.75,
                    fused=rng.random() < 0.5, scaling=rng.choice(["none", "linear", "theta", "parts"]),
                    far=rng.choice([0, 0, 30000, 1000000]))
    P = rng.choice([16, 16, 32, 64, 128, 48, 8, 20])
    S = rng.choice([s for s in (4, 8, 16, 32, P) if P % s == 0 and (s >= 16 or s == P or rng.random() < 0.2)] or [P])
    kv = rng.choice(["e4m3", "int8"])
    dt = rng.choice(["bf16", "bf16", "f16"])
    if op == "append":
        if rng.random() < 0.5:
            seqs, n_lo, n_hi = _log(rng, 1, 600), 1, 1
        else:
            seqs = _log(rng, 1, 60)
            n_lo, n_hi = rng.choice([0, 1]), _log(rng, 2, 20000 // seqs)
        return dict(op=op, H_kv=H_kv, D=D, P=P, S=S, dt=dt, kv=kv, seqs=seqs, n_lo=n_lo, n_hi=n_hi,
                    old_hi=rng.choice([0, 30, 200]), lens=rng.randrange(1 << 30))
    B = _log(rng, 1, 256)
    hi = _log(rng, 2, min(131072, 800000 // B * 8 // max(8, H_kv)))
    lo = rng.choice([0, 1, max(1, hi // 8), max(1, hi // 2)])
    q_len = rng.choice([1, 1, 1, 2, 3, 5]) if P % 16 == 0 and S % 16 == 0 else 1
    window = rng.choice([0, 0, 0, 100, 1024]) if q_len == 1 else 0
    return dict(op=op, B=B, H_qo=H_qo, H_kv=H_kv, D=D, P=P, S=S, dt=dt, kv=kv, lo=lo, hi=hi, q_len=q_len,
                window=window, lens=rng.randrange(1 << 30))


def _lengths(c):
    """Rows of each sequence (decode), or (new, old) rows of each (append): the case's own."""
    r = random.Random(c["lens"])
    if c["op"] == "decode":
        return [r.randint(c["lo"], c["hi"]) for _ in range(c["B"])]
    new = [r.randint(c["n_lo"], c["n_hi"]) for _ in range(c["seqs"])]
    new[0] = max(new[0], 1)
    return new, [r.randint(0, c["old_hi"]) for _ in range(c["seqs"])]


SINKS = 4  # attention-sink rows of a windowed case


def _attended(c, length):
    """(rows attended, window's start) of a sequence of `length` rows."""
    w = c["window"]
    if not w or length <= w + SINKS:
        return length, 0
    return SINKS + w, length - w


def work(c):
    if c["op"] == "norm_rope":
        n = c["T"] * (c["H_qo"] + c["H_kv"]) * c["D"]
        b = 2 * n * DT[c["dt"]].itemsize + c["T"] * 4 + c["rd"] * 4 + 4 * c["D"]
        return {"bytes": b, "flops": n * (4 if c["norm"] else 0) + c["T"] * (c["H_qo"] + c["H_kv"]) * c["rd"] * 3}
    if c["op"] == "append":
        new, _ = _lengths(c)
        t = sum(new)
        n = 2 * t * c["H_kv"] * c["D"]
        blocks = sum(-(-x // c["S"]) for x in new)
        return {"bytes": n * (DT[c["dt"]].itemsize + 1) + blocks * 2 * c["H_kv"] * 4, "flops": 2 * n}
    rows = sum(_attended(c, x)[0] for x in _lengths(c))
    q = c["B"] * c["q_len"] * c["H_qo"]
    return {"bytes": rows * 2 * c["H_kv"] * (c["D"] + 4 / c["S"]) + 4 * q * c["D"] + 4 * q,
            "flops": 4 * rows * c["q_len"] * c["H_qo"] * c["D"]}


# ------------------------------------------------------------------------------- inputs
def _frequencies(c, dev):
    """Radians per position of each rotated pair, in 64 bits, as the context-extension recipes give them."""
    n, theta, factor = c["rd"] // 2, 500000.0, 8.0
    i = torch.arange(n, dtype=torch.float64)
    if c["scaling"] == "theta" and n > 1:
        theta *= factor ** (n / (n - 1))
    f = theta ** (-i / n)
    if c["scaling"] == "linear":
        f = f / factor
    if c["scaling"] == "parts":
        turns = 8192 * f / (2 * math.pi)
        keep = ((turns - 1.0) / (4.0 - 1.0)).clamp(0, 1)
        f = (1 - keep) * f / factor + keep * f
    return f.to(dev)


def _pow2(amax, kv):
    """The smallest power of two 2^k, k >= -126, with amax <= largest code * 2^k (in float32)."""
    m, e = torch.frexp(amax)
    frac, bits = (0.875, 9) if kv == "e4m3" else (0.9921875, 7)  # 448 = 0.875 2^9, 127 = 0.9921875 2^7
    k = torch.where(m <= frac, e - bits, e - bits + 1).clamp(min=-126)
    k = torch.where(amax > 0, k, torch.full_like(k, -126))
    return ((k + 127) << 23).to(torch.int32).view(torch.float32)


def _encode(x, kv):
    """Values already divided by their scale -> codes, as bytes."""
    if kv == "e4m3":
        return x.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.int8)
    return x.round().clamp(-127, 127).to(torch.int8)


def _values(codes, kv, to=torch.float32):
    """Bytes -> the values of the codes."""
    return codes.view(torch.float8_e4m3fn).to(to) if kv == "e4m3" else codes.to(to)


def _pool(c, n_pages, g, dev):
    """A cache of `n_pages` pages in use: codes (as bytes) and scales."""
    H, P, S, D = c["H_kv"], c["P"], c["S"], c["D"]
    pages = torch.empty(n_pages, 2, H, P, D, dtype=torch.int8, device=dev)
    scales = torch.empty(n_pages, 2, H, P // S, dtype=torch.float32, device=dev)
    step = max(1, (1 << 27) // (2 * H * P * D))
    for i in range(0, n_pages, step):
        n = min(step, n_pages - i)
        x = torch.randn(n, 2, H, P // S, S, D, generator=g, device=dev)
        x *= torch.exp(0.7 * torch.randn(n, 2, H, P // S, 1, 1, generator=g, device=dev))
        s = _pow2(x.abs().amax((-1, -2)), c["kv"])
        scales[i:i + n] = s
        pages[i:i + n] = _encode(x / s[..., None, None], c["kv"]).view(n, 2, H, P, D)
    return pages, scales


def _table(c, lengths, g, dev):
    """A shuffled page table of sequences of these lengths: indptr, values, last page lengths, pages."""
    P = c["P"]
    counts = [-(-x // P) for x in lengths]
    indptr = [0]
    for n in counts:
        indptr.append(indptr[-1] + n)
    values = torch.randperm(max(1, indptr[-1]), generator=g, device=dev).to(torch.int32)[: indptr[-1]]
    last = [x - (n - 1) * P if n else 0 for x, n in zip(lengths, counts)]
    t = lambda a: torch.tensor(a, dtype=torch.int32, device=dev)  # noqa: E731
    return t(indptr), values, t(last), indptr, last, max(1, indptr[-1])


def prepare(c, seed):
    dev = "cuda"
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    s = {"c": c}
    dt = DT[c["dt"]]
    if c["op"] == "norm_rope":
        T, Hq, Hk, D = c["T"], c["H_qo"], c["H_kv"], c["D"]
        if c["fused"]:  # q, k and v side by side in the projection's output
            x = torch.randn(T, Hq + 2 * Hk, D, generator=g, device=dev).to(dt)
            s["q"], s["k"] = x[:, :Hq], x[:, Hq:Hq + Hk]
        else:
            s["q"] = torch.randn(T, Hq, D, generator=g, device=dev).to(dt)
            s["k"] = torch.randn(T, Hk, D, generator=g, device=dev).to(dt)
        for n in ("qw", "kw"):
            s[n] = (1 + 0.2 * torch.randn(D, generator=g, device=dev)).to(dt) if c["norm"] else None
        s["pos"] = (torch.randint(0, 4096, (T,), generator=g, device=dev) + c["far"]).to(torch.int32)
        s["freq"] = _frequencies(c, dev)
        s["factor"] = 1.0 if c["scaling"] == "none" else 0.1 * math.log(8.0) + 1.0
        s["q_out"] = torch.empty(T, Hq, D, dtype=dt, device=dev)
        s["k_out"] = torch.empty(T, Hk, D, dtype=dt, device=dev)
        return s
    if c["op"] == "append":
        new, old = _lengths(c)
        s["indptr"], s["values"], s["last"], _, _, n_pages = _table(c, [a + b for a, b in zip(new, old)], g, dev)
        s["pages"], s["scales"] = _pool(c, n_pages, g, dev)
        at = [0]
        for n in new:
            at.append(at[-1] + n)
        s["at"] = torch.tensor(at, dtype=torch.int32, device=dev)
        x = torch.randn(at[-1], 2, c["H_kv"], c["D"], generator=g, device=dev)
        x *= torch.exp(0.7 * torch.randn(at[-1], 2, c["H_kv"], 1, generator=g, device=dev))
        s["k"], s["v"] = x[:, 0].to(dt), x[:, 1].to(dt)
        return s
    lengths = _lengths(c)
    s["indptr"], s["values"], last, indptr, last_h, n_pages = _table(c, lengths, g, dev)
    s["pages"], s["scales"] = _pool(c, n_pages, g, dev)
    s["length_info"], host = last, last_h
    if c["window"]:
        att = [_attended(c, x) for x in lengths]
        sink = [SINKS if w else 0 for _, w in att]
        host = last_h + [w for _, w in att] + sink
        s["length_info"] = torch.tensor(host, dtype=torch.int32, device=dev).view(3, -1)
    B, n, Hq, D = c["B"], c["q_len"], c["H_qo"], c["D"]
    s["Q"] = torch.randn(B, n, Hq, D, generator=g, device=dev).to(dt)
    if n == 1:
        s["Q"] = s["Q"][:, 0].contiguous()
    s["out"] = torch.empty_like(s["Q"])
    s["lse"] = torch.empty(s["Q"].shape[:-1], dtype=torch.float32, device=dev)
    s["max_pages_of_one"] = max(1, max(b - a for a, b in zip(indptr, indptr[1:])))
    import numpy
    s["host"] = (numpy.array(indptr, numpy.int32), numpy.array(host, numpy.int32))  # what a scheduler holds
    return s


# ------------------------------------------------------------------------------- plain forms
def _plain_rotated(x, w, s):
    c = s["c"]
    y = x.float()
    if w is not None:
        y = y / torch.sqrt((y * y).mean(-1, keepdim=True) + 1e-6) * w.float()
    n = c["rd"] // 2
    turns = s["pos"].double()[:, None] * s["freq"] / (2 * math.pi)  # far positions: 64 bits
    a = ((turns - turns.floor()) * (2 * math.pi)).float()[:, None, :]
    co, si = torch.cos(a) * s["factor"], torch.sin(a) * s["factor"]
    r, rest = y[..., : 2 * n], y[..., 2 * n:]
    if c["mode"] == 1:
        p, q = r[..., :n], r[..., n:]
        r = torch.cat([p * co - q * si, q * co + p * si], -1)
    else:
        p, q = r[..., 0::2], r[..., 1::2]
        r = torch.stack([p * co - q * si, q * co + p * si], -1).flatten(-2)
    return torch.cat([r, rest], -1).to(x.dtype)


def _plain_append(s):
    c = s["c"]
    P, S, kv, H = c["P"], c["S"], c["kv"], c["H_kv"]
    at, indptr, pages, scales = s["at"].long(), s["indptr"].long(), s["pages"], s["scales"]
    T = s["k"].shape[0]
    t = torch.arange(T, device=pages.device)
    b = torch.searchsorted(at, t, right=True) - 1
    npages = indptr[1:] - indptr[:-1]
    first = (npages - 1) * P + s["last"] - (at[1:] - at[:-1])  # offset of the sequence's first new row
    off = first[b] + t - at[b]
    page, slot = s["values"].long()[indptr[b] + off // P], off % P
    blk = page * (P // S) + slot // S
    x = torch.stack([s["k"], s["v"]], 1).float()
    n_blk = pages.shape[0] * (P // S)
    amax = torch.zeros(n_blk, 2, H, device=pages.device).scatter_reduce(
        0, blk[:, None, None].expand(-1, 2, H), x.abs().amax(-1), "amax")
    fresh_from = torch.full((n_blk,), S, device=pages.device).scatter_reduce(0, blk, slot % S, "amin")
    need = _pow2(amax, kv).view(-1, P // S, 2, H).permute(0, 2, 3, 1)
    fresh_from = fresh_from.view(-1, 1, 1, P // S)
    grown = torch.where(fresh_from == 0, need, torch.where(fresh_from < S, torch.maximum(scales, need), scales))
    ratio = (scales / grown)[..., None, None]
    rows = pages.view(-1, 2, H, P // S, S, c["D"])
    is_old = torch.arange(S, device=pages.device)[:, None] < fresh_from[..., None, None]
    moved = is_old & (ratio != 1)
    rows.copy_(torch.where(moved, _encode(_values(rows, kv) * ratio, kv), rows))
    scales.copy_(grown)
    i, h = torch.arange(2, device=pages.device)[None, :, None], torch.arange(H, device=pages.device)
    page, slot = page[:, None, None], slot[:, None, None]
    pages[page, i, h, slot] = _encode(x / scales[page, i, h, slot // S][..., None], kv)


def _plain_decode(s):
    c = s["c"]
    B, n, Hq, Hk, D, P, S = c["B"], c["q_len"], c["H_qo"], c["H_kv"], c["D"], c["P"], c["S"]
    G, dev = Hq // Hk, s["Q"].device
    indptr, last = s["indptr"].long(), s["length_info"].view(-1, B).long()
    npages = indptr[1:] - indptr[:-1]
    length = torch.where(npages > 0, (npages - 1) * P + last[0], 0)
    slot = torch.arange(s["max_pages_of_one"], device=dev)
    if s["values"].numel() == 0:
        s["out"].zero_()
        s["lse"].fill_(EMPTY)
        return
    idx = s["values"].long()[(indptr[:-1, None] + slot).clamp(max=s["values"].numel() - 1)]

    def side(which):
        x = _values(s["pages"][:, which][idx], c["kv"])  # [B, pages, Hk, P, D]
        x = x.view(*x.shape[:3], P // S, S, D) * s["scales"][:, which][idx][..., None, None]
        return x.permute(0, 2, 1, 3, 4, 5).reshape(B, Hk, -1, D)

    q = s["Q"].float().view(B, n, Hk, G, D).permute(0, 2, 1, 3, 4).reshape(B, Hk, n * G, D)
    score = torch.matmul(q, side(0).transpose(-1, -2)) * D ** -0.5  # [B, Hk, n G, rows]
    row = torch.arange(score.shape[-1], device=dev)
    seen = row < length[:, None]
    if c["window"]:
        seen = seen & ((row < last[2][:, None]) | (row >= last[1][:, None]))
    seen = seen[:, None, None, :]
    if n > 1:  # token t sees the rows up to itself
        limit = length[:, None] - n + 1 + torch.arange(n, device=dev)
        seen = seen & (row < limit[:, :, None]).repeat_interleave(G, 1)[:, None]
    score = torch.where(seen, score, -math.inf)
    m = score.amax(-1, keepdim=True)
    m = torch.where(m > -math.inf, m, 0.0)
    p = torch.exp(score - m)
    d = p.sum(-1, keepdim=True)
    o = torch.matmul(p, side(1)) / torch.where(d > 0, d, 1.0)
    lse = torch.where(d > 0, (m + torch.log(d)) * LOG2E, EMPTY)[..., 0]
    order = lambda x: x.view(B, Hk, n, G, -1).permute(0, 2, 1, 3, 4)  # noqa: E731
    s["out"].copy_(order(o).reshape(s["out"].shape))
    s["lse"].copy_(order(lse[..., None]).reshape(s["lse"].shape))


def run(s):
    c = s["c"]
    if own:
        import paged_kv_decode_19_gb300 as pd
    if c["op"] == "norm_rope":
        if own:
            pd.qk_norm_rope(s["q"], s["k"], s["qw"], s["kw"], s["pos"], s["freq"], s["q_out"], s["k_out"],
                            rotary_mode=c["mode"], attention_factor=s["factor"])
        else:
            s["q_out"].copy_(_plain_rotated(s["q"], s["qw"], s))
            s["k_out"].copy_(_plain_rotated(s["k"], s["kw"], s))
        return s["q_out"], s["k_out"]
    kvt = torch.float8_e4m3fn if c["kv"] == "e4m3" else torch.int8
    if c["op"] == "append":
        if own:
            pd.append_paged_kv_bs(s["pages"].view(kvt), s["scales"], s["k"], s["v"], s["at"], s["indptr"],
                                  s["values"], s["last"])
        else:
            _plain_append(s)
        return s["pages"].view(kvt), s["scales"]
    if own:
        pd.batch_decode_paged_kv_bs(s["Q"], s["pages"].view(kvt), s["scales"], s["indptr"], s["values"],
                                    s["length_info"], s["out"], s["lse"], host_meta=s["host"])
    else:
        _plain_decode(s)
    return s["out"], s["lse"]


# ------------------------------------------------------------------------------- the definition, in 64 bits
def _exact_norm_rope(s, x, w):
    c, n = s["c"], s["c"]["rd"] // 2
    y = x.double()
    if w is not None:
        y = y * torch.rsqrt(y.pow(2).sum(-1, keepdim=True) / c["D"] + 1e-6) * w.double()
    z = y.clone()
    ang = s["pos"].double()[:, None] * s["freq"]
    for i in range(n):
        a, b = (i, i + n) if c["mode"] == 1 else (2 * i, 2 * i + 1)
        co, si = ang[:, i].cos()[:, None] * s["factor"], ang[:, i].sin()[:, None] * s["factor"]
        z[..., a] = y[..., a] * co - y[..., b] * si
        z[..., b] = y[..., b] * co + y[..., a] * si
    return z


def _exact_code(x, kv):
    """The code nearest to x (ties to even), as a value."""
    if kv == "int8":
        return torch.round(x).clamp(-127, 127)
    quantum = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6))) - 3)
    return (torch.round(x / quantum) * quantum).clamp(-448, 448)


def _exact_append(s):
    c = s["c"]
    P, S, kv = c["P"], c["S"], c["kv"]
    top = 448.0 if kv == "e4m3" else 127.0
    val = _values(s["pages"], kv, torch.float64)
    sc = s["scales"].double()
    at, indptr, values, last = s["at"].tolist(), s["indptr"].tolist(), s["values"].tolist(), s["last"].tolist()
    x = torch.stack([s["k"], s["v"]], 1).double()
    for b in range(len(last)):
        new, total = at[b + 1] - at[b], (indptr[b + 1] - indptr[b] - 1) * P + last[b]
        lo = total - new
        while lo < total:  # one block of S rows at a time
            hi = min(total, lo // S * S + S)
            page, blk = values[indptr[b] + lo // P], lo % P // S
            r0, r1 = lo % P, lo % P + hi - lo
            rows = x[at[b + 1] - (total - lo): at[b + 1] - (total - hi)].permute(1, 2, 0, 3)  # [2, H, rows, D]
            amax = rows.abs().amax((-1, -2)).clamp(min=top * 2.0 ** -126)
            k = torch.ceil(torch.log2(amax / top))
            k = torch.where(amax > top * torch.exp2(k), k + 1, k)
            k = torch.where(amax <= top * torch.exp2(k - 1), k - 1, k)
            need, was = torch.exp2(k), sc[page, :, :, blk]
            if lo % S:
                need = torch.maximum(need, was)
                old = val[page, :, :, blk * S:r0]
                val[page, :, :, blk * S:r0] = _exact_code(old * (was / need)[..., None, None], kv)
            sc[page, :, :, blk] = need
            val[page, :, :, r0:r1] = _exact_code(rows / need[..., None, None], kv)
            lo = hi
    return val if kv == "e4m3" else val.to(torch.int8), sc


def _exact_decode(s):
    c = s["c"]
    B, n, Hq, Hk, D, P, S = c["B"], c["q_len"], c["H_qo"], c["H_kv"], c["D"], c["P"], c["S"]
    Q = s["Q"].double().view(B, n, Hk, Hq // Hk, D)
    out = torch.zeros(B, n, Hk, Hq // Hk, D, dtype=torch.float64, device=Q.device)
    lse = torch.full((B, n, Hk, Hq // Hk), EMPTY, dtype=torch.float64, device=Q.device)
    indptr = s["indptr"].tolist()
    for b, length in enumerate(_lengths(c)):
        if not length:
            continue
        ids = s["values"][indptr[b]:indptr[b + 1]].long()
        att, start = _attended(c, length)
        rows = torch.arange(length, device=Q.device)
        rows = rows[(rows < SINKS) | (rows >= start)] if start else rows
        for h in range(Hk):
            k, v = (_values(s["pages"][ids, w, h], c["kv"], torch.float64).reshape(-1, D)[rows]
                    * s["scales"][ids, w, h].double().reshape(-1)[rows // S][:, None] for w in (0, 1))
            for t in range(n):
                end = len(rows) - n + 1 + t
                if end <= 0:
                    continue
                z = Q[b, t, h] @ k[:end].T / math.sqrt(D)
                total = torch.logsumexp(z, -1)
                out[b, t, h] = torch.exp(z - total[:, None]) @ v[:end]
                lse[b, t, h] = total / math.log(2)
    return out.reshape(s["out"].shape), lse.reshape(s["lse"].shape)


def exact(c, seed):
    s = prepare(c, seed)
    if c["op"] == "norm_rope":
        return _exact_norm_rope(s, s["q"], s["qw"]), _exact_norm_rope(s, s["k"], s["kw"])
    return _exact_append(s) if c["op"] == "append" else _exact_decode(s)
