"""build_page_tables against its definition on lists, and a serving loop of all calls together."""
import random

import pytest
import torch

import paged_kv_decode_19_gb300 as pd
from tests import _mx

pytestmark = pytest.mark.gpu
dev = "cuda"


def _t(a, dt=torch.int32):
    return torch.tensor(a, dtype=dt, device=dev)


class Pool:
    """A batch of requests on the device, and the same on lists."""

    def __init__(self, lengths, P, width, spare, T, caps=None, ring=True, window=0, sinks=0, head=0, seed=0):
        r = random.Random(seed)
        B, need = len(lengths), [-(-n // P) for n in lengths]
        n_pages = sum(need) + spare
        ids = list(range(n_pages))
        r.shuffle(ids)
        self.P, self.B, self.T, self.window, self.sinks = P, B, T, window, sinks
        self.cap = sum(need) + spare + 5 if caps is None else caps
        self.table = [[-7] * width for _ in range(B)]
        for b, n in enumerate(need):
            self.table[b][:n] = [ids.pop() for _ in range(n)]
        self.lengths = list(lengths)
        # free pages at head .. head + spare - 1 of the ring
        self.ring = [-1] * n_pages if ring else None
        self.state = [head, head + spare, 0, 0] if ring else [0, 0, 0, 0]
        if ring:
            for i, page in enumerate(ids):
                self.ring[(head + i) % n_pages] = page
        self.d_table, self.d_lengths = _t(self.table).view(B, width), _t(self.lengths)
        self.d_ring, self.d_state = _t(self.ring) if ring else None, _t(self.state, torch.int64)
        self.fresh()

    def fresh(self):
        B, f = self.B, lambda *n, dt=torch.int32: torch.full(n, 99, dtype=dt, device=dev)
        self.indptr, self.values, self.at = f(B + 1), f(self.cap), f(B + 1)
        self.info = f(3, B) if self.window else f(B)
        self.slots, self.pos = f(self.T, dt=torch.int64), f(self.T)

    def call(self, new, **kw):
        a = dict(append_indptr=self.at, slot_mapping=self.slots, positions=self.pos, free_pages=self.d_ring,
                 window=self.window, sinks=self.sinks)
        pd.build_page_tables(self.d_table, self.d_lengths, new, self.d_state, self.P, self.indptr, self.values, self.info,
                             **{**a, **kw})

    def step(self, new, error="PD_OK"):
        self.fresh()
        self.call(_t(new))
        self.check(new, error)

    def check(self, new, error="PD_OK"):
        indptr, values, at, info, slots, pos = _mx.tables_ref(self.table, self.lengths, new, self.state, self.ring, self.P,
                                                              (self.cap, self.T), self.window, self.sinks)
        assert pd.check_device_errors() == error
        assert self.indptr.tolist() == indptr and self.at.tolist() == at
        assert self.values.tolist() == values + [99] * (self.cap - len(values))
        assert self.info.view(-1, self.B).tolist() == info
        assert self.slots.tolist() == slots + [-1] * (self.T - len(slots))
        assert self.pos.tolist() == pos + [0] * (self.T - len(pos))
        assert self.d_lengths.tolist() == self.lengths and self.d_table.tolist() == self.table
        assert self.d_state.tolist() == self.state
        if self.ring is not None:
            assert self.d_ring.tolist() == self.ring


@pytest.mark.parametrize("B,P,hi", [(1, 16, 100), (3, 1, 9), (7, 20, 300), (256, 32, 900), (511, 16, 60), (513, 8, 60),
                                   (3000, 16, 50), (8192, 256, 600)])
@pytest.mark.parametrize("ring", [True, False])
def test_steps(B, P, hi, ring):
    """Growth, drafts taken back, requests that end and others in their place."""
    r = random.Random(B)
    lengths = [r.choice([0, 1, P, r.randint(0, hi)]) for _ in range(B)]
    width = -(-hi // P) + 4
    p = Pool(lengths, P, width, spare=B * 4 + 9, T=B * 4 + 33, ring=ring, window=0 if P < 20 else 50, sinks=0 if P < 20 else 3)
    if not ring:  # a table that holds its pages
        p.table = [[b * width + k for k in range(width)] for b in range(B)]
        p.d_table.copy_(_t(p.table))
        p.cap = B * width
    for step in range(5):
        new = []
        for n in p.lengths:
            x = r.choice([0, 1, 1, 3, -1, -2, -n, r.randint(0, 5)])
            new.append(max(x, -n) if n + x <= width * P else 0)
        p.step(new)


def test_the_ring_wraps_and_state_counts_on():
    p = Pool([5, 40, 0, 17], 16, 20, spare=7, T=200, head=(1 << 40) + 3)
    r = random.Random(0)
    for _ in range(40):
        new = [r.randint(-n, 30) for n in p.lengths]
        p.step(new, "PD_OK" if _fits(p, new) else "PD_ERR_NO_PAGES")


def _fits(p, new):
    need = lambda n: -(-n // p.P)  # noqa: E731
    return sum(max(0, need(a + n) - need(a)) for a, n in zip(p.lengths, new)) <= p.state[1] - p.state[0]


def test_a_step_that_does_not_fit_changes_nothing():
    p = Pool([30, 5, 0], 16, 8, spare=2, T=40)
    p.step([16, 16, 16], "PD_ERR_BAD_LENGTH")   # three pages, two free; and 48 tokens for 40 slots, named first
    p.step([16, 16, 7], "PD_ERR_NO_PAGES")      # three pages, two free
    p.step([30, 11, 0], "PD_ERR_BAD_LENGTH")    # 41 tokens for 40 slots
    p.step([2, 11, 16])                         # one page
    p.step([16, -16, 0])                        # the one that is free (a page is given back, for the next step)
    p.step([16, 0, 0])
    p.step([0, 1, 0], "PD_ERR_NO_PAGES")
    q = Pool([30, 5, 0], 16, 8, spare=9, T=40, caps=4)
    q.step([2, 11, 1])
    q.step([1, 0, 0], "PD_ERR_BAD_LENGTH")      # five pages for a list of four
    q.step([-1, 0, -1])
    # a pool whose counts cannot be: nothing is taken from it
    p = Pool([30, 5, 0], 16, 8, spare=2, T=40)
    p.state[1] = p.state[0] - 1
    p.d_state.copy_(_t(p.state, torch.int64))
    p.step([16, 0, 0], "PD_ERR_NO_PAGES")


def test_requests_out_of_range_are_left_alone():
    p = Pool([30, 5, 0, 64, 17], 16, 4, spare=9, T=40)
    p.step([2, -6, 1, 1, 1], "PD_ERR_BAD_LENGTH")  # below zero; a fifth page
    p.lengths[1], p.lengths[4] = -3, 1 << 30
    p.d_lengths.copy_(_t(p.lengths))
    p.step([1, 5, 1, -64, 1 << 30], "PD_ERR_BAD_LENGTH")
    p.step([2147483647, -2147483648, 1, 0, 0], "PD_ERR_BAD_LENGTH")


def test_a_table_without_its_pages():
    p = Pool([30, 5], 16, 4, spare=0, T=40, ring=False)
    p.cap = 8
    p.step([3, 12], "PD_ERR_BAD_PAGE")


def test_without_the_optional_outputs_and_none_at_all():
    p = Pool([30, 5, 0], 16, 8, spare=9, T=10)
    p.call(_t([9, 0, 9]), append_indptr=None, slot_mapping=None, positions=None)  # (no slots: any number of tokens)
    assert pd.check_device_errors() == "PD_OK" and p.indptr.tolist() == [0, 3, 4, 5] and p.d_lengths.tolist() == [39, 5, 9]
    assert p.slots.tolist() == [99] * 10
    p.call(_t([1, 1, 1]), append_indptr=None, slot_mapping=None)
    assert p.pos.tolist() == [39, 5, 9] + [0] * 7
    z = torch.zeros(0, dtype=torch.int32, device=dev)
    ip, at, slots = _t([7]), _t([7]), _t([5, 5], torch.int64)
    pd.build_page_tables(z.view(0, 3), z, z, _t([0, 0, 0, 0], torch.int64), 16, ip, z, z, at, slots)
    assert ip.tolist() == [0] and at.tolist() == [0] and slots.tolist() == [-1, -1]


def test_strided_table_and_streams():
    """Rows of a wider buffer; several pools on several streams at once."""
    pools, streams = [Pool([100 * i + 5, 17, 0, 900], 16, 64, spare=200, T=300, seed=i) for i in range(4)], []
    for p in pools:
        wide = torch.full((4, 70), 55, dtype=torch.int32, device=dev)
        wide[:, 3:67] = p.d_table
        p.d_table, p.wide = wide[:, 3:67], wide
        streams.append(torch.cuda.Stream())
    steps = [[3, 5, 100, -1], [16, -22, 5, 30]]
    news = [_t(n) for n in steps]
    torch.cuda.synchronize()
    for new in news:
        for p, s in zip(pools, streams):
            p.call(new, stream=s)
    torch.cuda.synchronize()
    for p in pools:
        _mx.tables_ref(p.table, p.lengths, steps[0], p.state, p.ring, 16, (p.cap, p.T))
        # (the lists of the second step)
        indptr, values, at, info, slots, pos = _mx.tables_ref(p.table, p.lengths, steps[1], p.state, p.ring, 16, (p.cap, p.T))
        assert p.indptr.tolist() == indptr and p.values.tolist()[: len(values)] == values and p.slots.tolist()[: len(slots)] == slots
        assert p.d_lengths.tolist() == p.lengths and p.d_state.tolist() == p.state and p.d_ring.tolist() == p.ring
        assert p.d_table.tolist() == p.table and (p.wide[:, :3] == 55).all() and (p.wide[:, 67:] == 55).all()


@pytest.mark.parametrize("sc,window", [("e4m3", 0), ("e8m0", 0), ("e4m3", 24)])
def test_a_captured_serving_loop(sc, window):
    """Tables, norm and rotation, quantising append and decode captured once and replayed: prompts
    come, drafts are taken back, a request ends and another takes its place.  Against the definition
    on what the loop was given, kept apart."""
    P, Hq, H, D, B, T, sinks = 16, 8, 2, 128, 4, 48, 4 if window else 0
    g = torch.Generator().manual_seed(0)
    n_pages = 40
    free, state = pd.page_pool(n_pages)
    table = torch.full((B, 16), -1, dtype=torch.int32, device=dev)
    lengths, new = _t([0] * B), _t([0] * B)
    i32 = lambda *n: torch.zeros(*n, dtype=torch.int32, device=dev)  # noqa: E731
    indptr, values, at, pos = i32(B + 1), i32(n_pages), i32(B + 1), i32(T)
    info = i32(3, B) if window else i32(B)
    slots = torch.zeros(T, dtype=torch.int64, device=dev)
    qkv = torch.zeros(T, Hq + 2 * H, D, dtype=torch.bfloat16, device=dev)
    w = torch.ones(D, dtype=torch.bfloat16, device=dev)
    freq = pd.rope_frequencies(D, 1e4)
    pages = torch.zeros(n_pages, 2, H, P, D // 2, dtype=torch.uint8, device=dev)
    scales = torch.zeros(n_pages, 2, H, P, D // _mx.BLOCK[sc], dtype=torch.uint8, device=dev).view(_mx.SC[sc])
    k_out = torch.zeros(T, H, D, dtype=torch.bfloat16, device=dev)
    q_out = torch.zeros(T, Hq, D, dtype=torch.bfloat16, device=dev)
    last = torch.zeros(B, dtype=torch.int64, device=dev)  # the token of each request that decodes
    q = torch.zeros(B, Hq, D, dtype=torch.bfloat16, device=dev)
    out, lse = torch.zeros_like(q), torch.zeros(B, Hq, device=dev)

    def step():
        pd.build_page_tables(table, lengths, new, state, P, indptr, values, info, at, slots, pos, free_pages=free,
                             window=window, sinks=sinks)
        pd.qk_norm_rope(qkv[:, :Hq], qkv[:, Hq:Hq + H], w, w, pos, freq, q_out, k_out)
        torch.index_select(q_out, 0, last, out=q)
        pd.append_paged_kv_mx(pages, scales, k_out, qkv[:, Hq + H:], slots)
        pd.batch_decode_paged_kv_mx(q, pages, scales, indptr, values, info, out, lse)

    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        step()
    kept = [([], []) for _ in range(B)]  # rows of K and V of each request
    plan = [[30, 1, 0, 17], [1, 1, 3, 1], [4, 4, 4, 4], [-3, -1, 0, -4], [1, 1, 1, 1], [-33, 9, 1, 1], [16, 1, 1, 1], [1, 0, 1, 1]]
    for n in plan:
        new.copy_(_t(n))
        qkv.copy_(torch.randn(qkv.shape, generator=g))
        ends = torch.tensor([sum(max(x, 0) for x in n[: b + 1]) - 1 for b in range(B)]).clamp(min=0)
        last.copy_(ends)
        graph.replay()
        assert pd.check_device_errors() == "PD_OK"
        t = 0
        for b, x in enumerate(n):
            K, V = kept[b]
            for i in range(max(x, 0)):
                K.append(k_out[t].double())
                V.append(qkv[t, Hq + H:].double())
                t += 1
            if x < 0:
                del K[len(K) + x:], V[len(V) + x:]
            rows = len(K)
            assert lengths[b] == rows
            if not rows:
                assert (out[b] == 0).all() and (lse[b] == -5e4).all()
                continue
            seen = _mx.attended(rows, (rows - window, sinks) if window and rows > window + sinks else None)
            k, v = (_mx.row_values(*_mx.quantise_ref(torch.stack(x_)[seen], 1.0, sc), sc) for x_ in (K, V))
            kq, vq = k.transpose(0, 1).repeat_interleave(Hq // H, 0), v.transpose(0, 1).repeat_interleave(Hq // H, 0)
            z = torch.einsum("hd,hrd->hr", q[b].double(), kq) * D ** -0.5
            p = torch.softmax(z, -1)[:, None]
            ref, A = (p @ vq)[:, 0], (p @ vq.abs())[:, 0]
            # f16 weights and the output's own half step, and the scores' error (as in _mx.check_decode)
            S = torch.einsum("hd,hrd->hr", q[b].double().abs(), kq.abs()).amax(-1) * D ** -0.5
            tol = A * (2.0 ** -11 + 2.0 ** -16 + 2 * S[:, None] * (D + D / 16) * 2.0 ** -24) + ref.abs() * 2.0 ** -8
            tol = tol + rows * 2.0 ** -32 * v.abs().max()
            assert ((out[b].double() - ref).abs() <= tol).all()
    assert state[1] - state[0] == n_pages - sum(-(-len(K) // P) for K, _ in kept)
