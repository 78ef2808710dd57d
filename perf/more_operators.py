"""What a serving step on a 4-bit cache costs: the page tables and slot maps built from the requests'
lengths, the append that quantises, and the decode that reads the codes, at sizes of the serving
loads this library runs.

Each operator has its plain form here (elementary torch operations in 32 bits, rounded once at the
end) and, where `own` is set, the library's call.  `exact` is the definition in 64 bits."""
import math
import random

import torch

own = False

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
LOG2E = 1.4426950408889634
EMPTY = -5e4  # log-sum-exp of a sequence that attends nothing
BLOCK = {"e4m3": 16, "e8m0": 32}  # dims that share a scale of this type
MAGNITUDE = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)  # of the eight magnitude codes


# ------------------------------------------------------------------------------- cases
def listed():
    return [
        # the next token of one request: launch latency
        dict(name="tables one request", op="tables", B=1, P=16, lo=100, hi=400, n_lo=1, n_hi=1, pool=True,
             window=0, lens=1),
        # a decode step of 256 requests that draft three tokens, some of which open a page
        dict(name="tables step of 256", op="tables", B=256, P=32, lo=300, hi=4200, n_lo=1, n_hi=4, pool=True,
             window=0, lens=2),
        # requests with long contexts in small pages beside ones that bring a prefill chunk
        dict(name="tables long and prefill", op="tables", B=61, P=16, lo=2000, hi=120000, n_lo=0, n_hi=2500,
             pool=True, window=4096, lens=3),
        # one token for each of 256 sequences
        dict(name="append step of 256", op="append", H_kv=8, D=128, P=32, dt="bf16", sc="e4m3", T=256, skip=0.0,
             ks=1.0, fused=True),
        # a long prefill chunk
        dict(name="append prefill 8192", op="append", H_kv=8, D=128, P=16, dt="bf16", sc="e4m3", T=8192, skip=0.0,
             ks=1.0, fused=True),
        # a padded batch (slots of -1) into a cache with power-of-two scales and a scale of its own
        dict(name="append padded", op="append", H_kv=4, D=64, P=20, dt="f16", sc="e8m0", T=1777, skip=0.3,
             ks=0.25, fused=False),
        # one short sequence: latency
        dict(name="decode one short", op="decode", B=1, H_qo=32, H_kv=8, D=128, P=16, dt="bf16", sc="e4m3",
             lo=200, hi=400, q_len=1, window=0, ks=1.0, lens=6),
        # a batch of middling contexts
        dict(name="decode batch of 32", op="decode", B=32, H_qo=32, H_kv=8, D=128, P=16, dt="bf16", sc="e4m3",
             lo=512, hi=4096, q_len=1, window=0, ks=1.0, lens=7),
        # many sequences, 64 query heads
        dict(name="decode batch of 256", op="decode", B=256, H_qo=64, H_kv=8, D=128, P=32, dt="bf16", sc="e4m3",
             lo=300, hi=4200, q_len=1, window=0, ks=1.0, lens=8),
        # long contexts, power-of-two scales
        dict(name="decode long contexts", op="decode", B=8, H_qo=32, H_kv=8, D=128, P=64, dt="bf16", sc="e8m0",
             lo=32768, hi=131072, q_len=1, window=0, ks=0.5, lens=9),
        # verification of three drafted tokens, heads of 64
        dict(name="decode four queries", op="decode", B=24, H_qo=16, H_kv=8, D=64, P=32, dt="f16", sc="e4m3",
             lo=700, hi=6000, q_len=4, window=0, ks=1.0, lens=10),
        # queries in 32 bits, wide heads, pages that no tile divides
        dict(name="decode wide f32", op="decode", B=7, H_qo=12, H_kv=4, D=256, P=20, dt="f32", sc="e4m3",
             lo=1, hi=3000, q_len=1, window=0, ks=1.0, lens=11),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["tables", "append", "decode", "decode"])
    P = rng.choice([16, 16, 32, 64, 128, 48, 8, 20])
    lens = rng.randrange(1 << 30)
    if op == "tables":
        B = _log(rng, 1, 2000)
        hi = _log(rng, 2, min(131072, 6000000 // B))
        n_lo, n_hi = rng.choice([(1, 1), (1, 5), (0, _log(rng, 2, max(3, 60000 // B)))])
        return dict(op=op, B=B, P=P, lo=rng.choice([0, 1, max(1, hi // 8)]), hi=hi, n_lo=n_lo, n_hi=n_hi,
                    pool=rng.random() < 0.8, window=rng.choice([0, 0, 100, 4096]), lens=lens)
    H_qo, H_kv = rng.choice([(8, 2), (32, 8), (32, 4), (64, 8), (12, 4), (7, 7), (16, 1)])
    D, sc = rng.choice([64, 128, 128, 256]), rng.choice(["e4m3", "e4m3", "e8m0"])
    dt, ks = rng.choice(["bf16", "bf16", "f16", "f32"]), rng.choice([1.0, 1.0, 0.25, 8.0])
    if op == "append":
        return dict(op=op, H_kv=H_kv, D=D, P=P, dt=dt, sc=sc, T=_log(rng, 1, 8000 * 1024 // (H_kv * D)),
                    skip=rng.choice([0.0, 0.0, 0.2]), ks=ks, fused=rng.random() < 0.5)
    B = _log(rng, 1, 256)
    hi = _log(rng, 2, min(131072, 800000 // B * 1024 // max(1024, H_kv * D)))
    lo = rng.choice([0, 1, max(1, hi // 8), max(1, hi // 2)])
    q_len = rng.choice([1, 1, 1, 2, 3, 5])
    window = rng.choice([0, 0, 0, 100, 1024]) if q_len == 1 else 0
    return dict(op=op, B=B, H_qo=H_qo, H_kv=H_kv, D=D, P=P, dt=dt, sc=sc, lo=lo, hi=hi, q_len=q_len,
                window=window, ks=ks, lens=lens)


def _lengths(c):
    """Rows of each sequence (decode), or (rows, new tokens) of each request (tables): the case's own."""
    r = random.Random(c["lens"])
    if c["op"] == "decode":
        return [r.randint(c["lo"], c["hi"]) for _ in range(c["B"])]
    old = [r.randint(c["lo"], c["hi"]) for _ in range(c["B"])]
    new = [r.randint(c["n_lo"], c["n_hi"]) for _ in range(c["B"])]
    new[0] = max(new[0], 1)
    return old, new


SINKS = 4  # attention-sink rows of a windowed case


def _attended(c, length):
    """(rows attended, window's start) of a sequence of `length` rows."""
    w = c["window"]
    if not w or length <= w + SINKS:
        return length, 0
    return SINKS + w, length - w


def work(c):
    if c["op"] == "tables":
        old, new = _lengths(c)
        pages = lambda n: -(-n // c["P"])  # noqa: E731
        before, after = sum(map(pages, old)), sum(pages(a + b) for a, b in zip(old, new))
        per = 8 * c["B"] + 4 * c["B"] * (3 if c["window"] else 1) + 8 * (c["B"] + 1) + 4 * c["B"]
        moved = 8 * (after - before) if c["pool"] else 0
        return {"bytes": 2 * per + 8 * after + 8 * before + 12 * sum(new) + 2 * moved,
                "flops": 2 * (after + before) + 4 * sum(new)}
    if c["op"] == "append":
        n = round(c["T"] * (1 - c["skip"])) * 2 * c["H_kv"] * c["D"]
        return {"bytes": n * (DT[c["dt"]].itemsize + 0.5 + 1 / BLOCK[c["sc"]]) + 8 * c["T"], "flops": 3 * n}
    rows = sum(_attended(c, x)[0] for x in _lengths(c))
    q = c["B"] * c["q_len"] * c["H_qo"]
    return {"bytes": rows * 2 * c["H_kv"] * c["D"] * (0.5 + 1 / BLOCK[c["sc"]])
            + 2 * DT[c["dt"]].itemsize * q * c["D"] + 4 * q,
            "flops": 4 * rows * c["q_len"] * c["H_qo"] * c["D"]}


# ------------------------------------------------------------------------------- inputs
def _scale_bytes(amax, sc):
    """The scale (as stored, one byte) of blocks with these largest magnitudes."""
    if sc == "e4m3":
        return (amax / 6.0).clamp(2.0 ** -9, 448.0).to(torch.float8_e4m3fn).view(torch.uint8)
    m, e = torch.frexp(amax)  # amax = m 2^e; 6 = 0.75 2^3
    k = torch.where(m <= 0.75, e - 3, e - 2)
    k = torch.where(amax > 0, k, -14).clamp(-14, 13)
    return (k + 127).to(torch.uint8)


def _scale_values(b, sc, to=torch.float32):
    """Stored scales -> their values."""
    if sc == "e4m3":
        return b.view(torch.float8_e4m3fn).to(to)
    return torch.exp2((b.to(torch.int32) - 127).to(to))


def _encode(q, negative):
    """Magnitudes already divided by their scale, and signs -> packed codes (two dims a byte, the
    even one in the low half).  Nearest, ties to the even code."""
    code = (q > 0.25).to(torch.uint8)
    for edge, up in ((0.75, True), (1.25, False), (1.75, True), (2.5, False), (3.5, True), (5.0, False)):
        code += (q >= edge) if up else (q > edge)
    code += negative.to(torch.uint8) * 8
    return code[..., 0::2] | (code[..., 1::2] << 4)


def _quantise(y, sc):
    """float32 rows [..., D] -> packed codes [..., D / 2] and scales [..., D / block] as bytes."""
    n = BLOCK[sc]
    blocks = y.unflatten(-1, (-1, n))
    s = _scale_bytes(blocks.abs().amax(-1), sc)
    q = blocks.abs() / _scale_values(s, sc)[..., None]
    return _encode(q.flatten(-2), torch.signbit(y)), s


def _pairs(dev, to=torch.float32):
    """The two values of each of the 256 bytes."""
    v = torch.tensor(MAGNITUDE + tuple(-x for x in MAGNITUDE), dtype=to, device=dev)
    b = torch.arange(256, device=dev)
    return torch.stack([v[b & 15], v[b >> 4]], -1)


def _rows(codes, scales, sc, to=torch.float32):
    """Packed codes [..., D / 2] and their scales -> values [..., D]."""
    x = _pairs(codes.device, to)[codes.int()].flatten(-2)
    return (x.unflatten(-1, (-1, BLOCK[sc])) * _scale_values(scales, sc, to)[..., None]).flatten(-2)


def _pool(c, n_pages, g, dev):
    """A cache of `n_pages` pages in use: packed codes and scales (both as bytes)."""
    H, P, D = c["H_kv"], c["P"], c["D"]
    pages = torch.empty(n_pages, 2, H, P, D // 2, dtype=torch.uint8, device=dev)
    scales = torch.empty(n_pages, 2, H, P, D // BLOCK[c["sc"]], dtype=torch.uint8, device=dev)
    channel = torch.exp(0.5 * torch.randn(2, H, 1, D, generator=g, device=dev))  # some dims run large
    step = max(1, (1 << 27) // (2 * H * P * D))
    for i in range(0, n_pages, step):
        n = min(step, n_pages - i)
        x = torch.randn(n, 2, H, P, D, generator=g, device=dev) * channel
        pages[i:i + n], scales[i:i + n] = _quantise(x, c["sc"])
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


def _prepare_tables(c, seed, g, dev, s):
    # the seed shifts the lengths by a little, so that other seeds are other requests of the same load
    P, B = c["P"], c["B"]
    old, new = _lengths(c)
    r = random.Random(seed)
    old = [min(max(c["lo"], x + r.randint(-P, P)), c["hi"]) for x in old]
    t = lambda a, dt=torch.int32: torch.tensor(a, dtype=dt, device=dev)  # noqa: E731
    s["lengths"], s["new"] = t(old), t(new)
    s["back"] = -s["new"]  # every draft is rejected, so that the next pass finds the same lengths
    held = [-(-x // P) for x in old]
    most = [-(-(x + n) // P) for x, n in zip(old, new)]
    room = sum(-(-(x + P + n) // P) for x, n in zip(*_lengths(c)))  # the largest step of any seed
    n_pages = room + 50
    ids = torch.randperm(n_pages, generator=g, device=dev).to(torch.int32)
    width = max(max(most), -(-(c["hi"] + c["n_hi"]) // P))
    s["page_table"] = torch.full((B, width), -1, dtype=torch.int32, device=dev)
    col = torch.arange(width, device=dev)
    own_pages = t(held if c["pool"] else most)
    seen = col < own_pages[:, None]
    s["page_table"][seen] = ids[: int(own_pages.sum())]
    s["free"] = ids.roll(-sum(held)).contiguous() if c["pool"] else None  # the ring holds room for every page
    s["state"] = t([0, n_pages - sum(held) if c["pool"] else 0, 0, 0], torch.int64)
    s["steps"] = []
    for _ in range(2):  # of the step, and of its rejection
        z = lambda *n, dt=torch.int32: torch.zeros(*n, dtype=dt, device=dev)  # noqa: E731
        # capacities: what the program allocated for its largest step
        s["steps"].append(dict(indptr=z(B + 1), values=z(room), length_info=z(3, B) if c["window"] else z(B),
                               append_indptr=z(B + 1), slots=z(sum(new) + 17, dt=torch.int64), positions=z(sum(new) + 17)))


def prepare(c, seed):
    dev = "cuda"
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    s = {"c": c}
    if c["op"] == "tables":
        _prepare_tables(c, seed, g, dev, s)
        return s
    dt = DT[c["dt"]]
    if c["op"] == "append":
        T, H, D, P = c["T"], c["H_kv"], c["D"], c["P"]
        n_pages = -(-T // P) + 3
        s["pages"], s["scales"] = _pool(c, n_pages, g, dev)
        x = torch.randn(T, 4 if c["fused"] else 2, H, D, generator=g, device=dev)
        x *= torch.exp(0.7 * torch.randn(T, x.shape[1], H, 1, generator=g, device=dev)) * c["ks"]
        x = x.to(dt)
        if c["fused"]:  # k and v behind q in the projection's output
            s["k"], s["v"] = x[:, 2], x[:, 3]
        else:
            s["k"], s["v"] = x[:, 0].contiguous(), x[:, 1].contiguous()
        s["slots"] = torch.randperm(n_pages * P, generator=g, device=dev)[:T]
        skip = torch.rand(T, generator=g, device=dev) < c["skip"]
        s["slots"] = torch.where(skip, -1, s["slots"])
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
    s["Q"] = (torch.randn(B, n, Hq, D, generator=g, device=dev) / c["ks"] * 0.7).to(dt)
    if n == 1:
        s["Q"] = s["Q"][:, 0].contiguous()
    s["out"] = torch.empty_like(s["Q"])
    s["lse"] = torch.empty(s["Q"].shape[:-1], dtype=torch.float32, device=dev)
    s["max_pages_of_one"] = max(1, max(b - a for a, b in zip(indptr, indptr[1:])))
    import numpy
    s["host"] = (numpy.array(indptr, numpy.int32), numpy.array(host, numpy.int32))  # what a scheduler holds
    return s


# ------------------------------------------------------------------------------- plain forms
def _plain_tables(s, new, to):
    c, P, ring, table = s["c"], s["c"]["P"], s["free"], s["page_table"]
    B, dev = c["B"], table.device
    old = s["lengths"].long()
    now = old + new
    held, need = (old + P - 1) // P, (now + P - 1) // P
    zero = torch.zeros(1, dtype=torch.int64, device=dev)
    start = lambda n: torch.cat([zero, n.cumsum(0)])  # noqa: E731
    indptr, grown, freed = start(need), start((need - held).clamp(min=0)), start((held - need).clamp(min=0))
    at = start(new.long().clamp(min=0))
    col = torch.arange(table.shape[1], device=dev)
    if ring is not None:
        C, head, tail = ring.numel(), s["state"][0], s["state"][1]
        fresh = (col >= held[:, None]) & (col < need[:, None])
        place = (head + grown[:-1, None] + col - held[:, None]) % C
        table.copy_(torch.where(fresh, ring[place], table))
        gone = (col < held[:, None]) & (col >= need[:, None])
        place = torch.where(gone, (tail + freed[:-1, None] + col - need[:, None]) % C, C)
        ring.copy_(torch.cat([ring, ring[:1]]).scatter(0, place.flatten(), table.flatten())[:C])
        s["state"][0] += grown[-1]
        s["state"][1] += freed[-1]
    seen = col < need[:, None]
    cap = to["values"].numel()
    place = torch.where(seen, indptr[:-1, None] + col, cap)
    to["values"].copy_(torch.cat([to["values"], to["values"][:1]]).scatter(0, place.flatten(), table.flatten())[:cap])
    to["indptr"].copy_(indptr)
    to["append_indptr"].copy_(at)
    info = to["length_info"].view(-1, B)
    info[0] = now - (need - 1).clamp(min=0) * P
    if c["window"]:
        cut = now > c["window"] + SINKS
        info[1] = torch.where(cut, now - c["window"], 0)
        info[2] = torch.where(cut, SINKS, 0)
    t = torch.arange(to["slots"].numel(), device=dev)
    b = (torch.searchsorted(at, t, right=True) - 1).clamp(max=B - 1)
    off = old[b] + t - at[b]
    ours = t < at[-1]
    page = table[b, torch.where(ours, off // P, 0)].long()
    to["slots"].copy_(torch.where(ours, page * P + off % P, -1))
    to["positions"].copy_(torch.where(ours, off, 0))
    s["lengths"].copy_(now)


def _plain_append(s):
    c = s["c"]
    P, slot = c["P"], s["slots"]
    y = torch.stack([s["k"], s["v"]], 1).float() / c["ks"]
    codes, scales = _quantise(y, c["sc"])
    keep = slot >= 0  # a skipped token goes to a row that is cut off again
    n = s["pages"].shape[0] * P
    place = torch.where(keep, slot, n)

    def put(cache, rows):
        flat = cache.permute(0, 3, 1, 2, 4).reshape(n, -1)
        flat = torch.cat([flat, flat[:1]])
        flat[place] = rows.flatten(1)
        cache.copy_(flat[:n].view(-1, P, 2, c["H_kv"], cache.shape[-1]).permute(0, 2, 3, 1, 4))

    put(s["pages"], codes)
    put(s["scales"], scales)


def _plain_decode(s):
    c = s["c"]
    B, n, Hq, Hk, D, P = c["B"], c["q_len"], c["H_qo"], c["H_kv"], c["D"], c["P"]
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
        x = _rows(s["pages"][:, which][idx], s["scales"][:, which][idx], c["sc"])  # [B, pages, Hk, P, D]
        return x.permute(0, 2, 1, 3, 4).reshape(B, Hk, -1, D) * c["ks"]

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
    if c["op"] == "tables":  # a step, and the return of its tokens: two calls
        for new, to in zip((s["new"], s["back"]), s["steps"]):
            if own:
                pd.build_page_tables(s["page_table"], s["lengths"], new, s["state"], c["P"], to["indptr"], to["values"],
                                     to["length_info"], to["append_indptr"], to["slots"], to["positions"],
                                     free_pages=s["free"], window=c["window"], sinks=SINKS if c["window"] else 0)
            else:
                _plain_tables(s, new, to)
        return s["steps"], s["page_table"], s["lengths"], s["state"], s["free"]
    sct = torch.float8_e4m3fn if c["sc"] == "e4m3" else torch.float8_e8m0fnu
    if c["op"] == "append":
        if own:
            pd.append_paged_kv_mx(s["pages"], s["scales"].view(sct), s["k"], s["v"], s["slots"], k_scale=c["ks"],
                                  v_scale=c["ks"])
        else:
            _plain_append(s)
        # (two codes a byte, and scales, as stored: every rounding is determined, so the bytes are equal)
        return s["pages"], s["scales"]
    if own:
        pd.batch_decode_paged_kv_mx(s["Q"], s["pages"], s["scales"].view(sct), s["indptr"], s["values"],
                                    s["length_info"], s["out"], s["lse"], k_scale=c["ks"], v_scale=c["ks"],
                                    host_meta=s["host"])
    else:
        _plain_decode(s)
    return s["out"], s["lse"]


# ------------------------------------------------------------------------------- the definition, in 64 bits
def _exact_tables(s):
    """One request, page and token after the other, on lists."""
    c, P = s["c"], s["c"]["P"]
    lengths, table, state = s["lengths"].tolist(), s["page_table"].tolist(), s["state"].tolist()
    ring = s["free"].tolist() if s["free"] is not None else None
    steps = []
    for new, to in ((s["new"].tolist(), s["steps"][0]), (s["back"].tolist(), s["steps"][1])):
        r = {k: v.tolist() for k, v in to.items()}
        info = [[0] * c["B"] for _ in range(3)]
        r["slots"], r["positions"] = [-1] * len(r["slots"]), [0] * len(r["positions"])
        at = tokens = 0
        for b, n in enumerate(new):
            held, need = -(-lengths[b] // P), -(-(lengths[b] + n) // P)
            if ring is not None:
                for k in range(held, need):
                    table[b][k] = ring[state[0] % len(ring)]
                    state[0] += 1
                for k in range(need, held):
                    ring[state[1] % len(ring)] = table[b][k]
                    state[1] += 1
            r["values"][at:at + need] = table[b][:need]
            for o in range(lengths[b], lengths[b] + n):
                r["slots"][tokens], r["positions"][tokens] = table[b][o // P] * P + o % P, o
                tokens += 1
            lengths[b] += n
            at += need
            r["indptr"][b + 1], r["append_indptr"][b + 1] = at, tokens
            info[0][b] = lengths[b] - (need - 1) * P if need else 0
            info[1][b] = _attended(c, lengths[b])[1]
            info[2][b] = SINKS if info[1][b] else 0
        r["length_info"] = info if c["window"] else info[0]
        steps.append({k: torch.tensor(v, dtype=to[k].dtype) for k, v in r.items()})
    t = lambda v, like: torch.tensor(v, dtype=like.dtype) if v is not None else None  # noqa: E731
    return steps, t(table, s["page_table"]), t(lengths, s["lengths"]), t(state, s["state"]), t(ring, s["free"])


def _exact_append(s):
    """Each code as the nearest of the sixteen values, by distance."""
    c, n = s["c"], BLOCK[s["c"]["sc"]]
    pages, scales = s["pages"].clone(), s["scales"].clone()
    keep = torch.nonzero(s["slots"] >= 0)[:, 0]
    page, slot = s["slots"][keep] // c["P"], s["slots"][keep] % c["P"]
    value = torch.tensor(MAGNITUDE, dtype=torch.float64, device=pages.device)
    for side, rows in enumerate((s["k"], s["v"])):
        y = (rows[keep].double() / c["ks"]).unflatten(-1, (-1, n))
        a = y.abs().amax(-1)
        if c["sc"] == "e4m3":
            q = torch.exp2(torch.floor(torch.log2((a / 6).clamp(min=2.0 ** -6))) - 3)
            sv = (torch.round(a / 6 / q) * q).clamp(2.0 ** -9, 448)
            byte = sv.float().to(torch.float8_e4m3fn).view(torch.uint8)
        else:
            k = torch.ceil(torch.log2(a.clamp(min=1e-30) / 6))
            k = torch.where(a > 6 * torch.exp2(k), k + 1, torch.where(a <= 6 * torch.exp2(k - 1), k - 1, k)).clamp(-14, 13)
            sv, byte = torch.exp2(k), (k + 127).to(torch.uint8)
        m = (y.abs() / sv[..., None]).clamp(max=6.0).flatten(-2)
        hi = torch.searchsorted(value, m).clamp(min=1, max=7)  # value[hi - 1] <= m <= value[hi]
        up, down = value[hi] - m, m - value[hi - 1]
        code = torch.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, hi - 1)
        code = (code + 8 * torch.signbit(rows[keep].double())).to(torch.uint8)
        pages[page, side, :, slot] = code[..., 0::2] + 16 * code[..., 1::2]
        scales[page, side, :, slot] = byte
    return pages, scales


def _exact_decode(s):
    c = s["c"]
    B, n, Hq, Hk, D, P = c["B"], c["q_len"], c["H_qo"], c["H_kv"], c["D"], c["P"]
    Q = s["Q"].double().view(B, n, Hk, Hq // Hk, D)
    out = torch.zeros(B, n, Hk, Hq // Hk, D, dtype=torch.float64, device=Q.device)
    lse = torch.full((B, n, Hk, Hq // Hk), EMPTY, dtype=torch.float64, device=Q.device)
    indptr, f64 = s["indptr"].tolist(), torch.float64
    for b, length in enumerate(_lengths(c)):
        if not length:
            continue
        ids = s["values"][indptr[b]:indptr[b + 1]].long()
        att, start = _attended(c, length)
        rows = torch.arange(length, device=Q.device)
        rows = rows[(rows < SINKS) | (rows >= start)] if start else rows
        for h in range(Hk):
            k, v = (_rows(s["pages"][ids, w, h].flatten(0, 1)[rows], s["scales"][ids, w, h].flatten(0, 1)[rows],
                          c["sc"], f64) * c["ks"] for w in (0, 1))
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
    return {"tables": _exact_tables, "append": _exact_append, "decode": _exact_decode}[c["op"]](s)
