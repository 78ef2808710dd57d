"""What non-finite scales, and weights far below the largest, do to batch_decode_paged_kv_bs."""
import pytest
import torch

from tests._bs import DT, KV, check_decode, decode_ref

pd = pytest.importorskip("paged_kv_decode_19_gb300")
pytestmark = pytest.mark.gpu
DEV = "cuda"
NAN, INF = float("nan"), float("inf")
# (D, type of Q, P, S, query tokens): SIMT by head dim and by Q, boxes, gathered rows
SIMT = [(256, "bf16", 16, 16, 1), (128, "f32", 16, 8, 1), (64, "f32", 20, 5, 1), (256, "f32", 32, 32, 1)]
MMA = [(128, "bf16", 16, 16, 1), (64, "f16", 32, 16, 1), (128, "f16", 8, 8, 1), (64, "bf16", 20, 5, 1),
       (128, "bf16", 16, 16, 3), (64, "f16", 16, 8, 2)]


def _case(D, dt, P, S, n, lengths, kv="int8", seed=0, Hq=4, H=2):
    """Random codes in (0, 100], scales 0.02 and a positive Q: every score is positive."""
    g = torch.Generator().manual_seed(seed)
    counts = [-(-L // P) for L in lengths]
    indptr = [0]
    for c in counts:
        indptr.append(indptr[-1] + c)
    vals = torch.randperm(indptr[-1] + 2, generator=g)[: indptr[-1]]
    codes = torch.randint(1, 101, (indptr[-1] + 2, 2, H, P, D), generator=g).to(torch.int8)
    if kv == "e4m3":
        codes = codes.float().to(torch.float8_e4m3fn).view(torch.int8)
    Q = (0.5 + torch.rand(len(lengths), n, Hq, D, generator=g)).to(DT[dt])
    t = lambda a: torch.tensor(a, dtype=torch.int32, device=DEV)  # noqa: E731
    return dict(Q=Q.to(DEV), codes=codes.to(DEV), scales=torch.full((indptr[-1] + 2, 2, H, P // S), 0.02, device=DEV),
                indptr=t(indptr), vals=vals.to(torch.int32).to(DEV), lengths=lengths, P=P, S=S, kv=kv, n=n, D=D,
                li=t([L - (c - 1) * P if c else 0 for L, c in zip(lengths, counts)]))


def _at(c, b, row):
    """(page, block) of a sequence's row."""
    return int(c["vals"][int(c["indptr"][b]) + row // c["P"]]), row % c["P"] // c["S"]


def _run(c, **kw):
    Q = c["Q"] if c["n"] > 1 else c["Q"][:, 0].contiguous()
    out = torch.full(Q.shape, 7.0, dtype=torch.float32, device=DEV)
    lse = torch.full(Q.shape[:-1], 7.0, device=DEV)
    pd.batch_decode_paged_kv_bs(Q, c["codes"].view(KV[c["kv"]]), c["scales"], c["indptr"], c["vals"], c["li"], out,
                                lse, **kw)
    assert pd.check_device_errors() == "PD_OK"
    return out.view(c["Q"].shape), lse.view(c["Q"].shape[:-1])


def _ref(c, **kw):
    return decode_ref(c["Q"], c["codes"], c["scales"], c["kv"], c["indptr"], c["vals"], c["lengths"], c["P"],
                      c["D"] ** -0.5, **kw)


def _others_stand(c, out, lse, touched, f16_weights, sink=None):
    """Heads outside `touched` ([B, n, Hq] bool) are what they are without the bad scale."""
    d = dict(c, scales=torch.nan_to_num(c["scales"], 0.02, 0.02, 0.02))
    o, l, (A, vmax, S) = _ref(d, sink=sink)
    keep = ~touched
    check_decode(out[keep], lse[keep], (o[keep], l[keep], (A[keep], vmax[keep], S[keep])), max(c["lengths"]),
                 f16_weights=f16_weights)


@pytest.mark.parametrize("shape", SIMT + MMA)
@pytest.mark.parametrize("splits", [0, 1, 4])
@pytest.mark.parametrize("side", [0, 1])
def test_a_nan_scale_reaches_what_attends_it(shape, splits, side):
    """And nothing else, on either kernel, whole or split."""
    c = _case(*shape, [40, 700, 3], seed=1)
    page, blk = _at(c, 1, 300)
    c["scales"][page, side, 0, blk] = NAN
    out, lse = _run(c, num_splits=splits)
    touched = torch.zeros(3, c["n"], 4, dtype=torch.bool, device=DEV)
    touched[1, :, :2] = True  # KV head 0 serves query heads 0 and 1
    assert torch.isnan(out[touched]).all()
    if side == 0:
        assert torch.isnan(lse[touched]).all()
    _others_stand(c, out, lse, touched, pd.last_decode_variant() == "mma")


@pytest.mark.parametrize("shape", SIMT)
@pytest.mark.parametrize("splits", [1, 7])
def test_nothing_but_nan_is_not_nothing(shape, splits):
    """Every K scale of a sequence NaN: its states are NaN, not empty."""
    c = _case(*shape, [500, 20], seed=5)
    page = c["vals"][int(c["indptr"][0]):int(c["indptr"][1])].long()
    c["scales"][page, 0, 1] = NAN
    out, lse = _run(c, num_splits=splits)
    touched = torch.zeros(2, 1, 4, dtype=torch.bool, device=DEV)
    touched[0, :, 2:] = True
    assert torch.isnan(out[touched]).all() and torch.isnan(lse[touched]).all()
    _others_stand(c, out, lse, touched, False)


@pytest.mark.parametrize("shape", SIMT + MMA)
@pytest.mark.parametrize("splits", [0, 1, 4])
@pytest.mark.parametrize("side", [0, 1])
def test_an_infinite_scale_reaches_what_attends_it(shape, splits, side):
    c = _case(*shape, [40, 700, 3], seed=1)
    page, blk = _at(c, 1, 300)
    c["scales"][page, side, 0, blk] = INF
    out, lse = _run(c, num_splits=splits)
    touched = torch.zeros(3, c["n"], 4, dtype=torch.bool, device=DEV)
    touched[1, :, :2] = True
    assert torch.isnan(out[touched]).all()
    if side == 0:
        assert torch.isnan(lse[touched]).all()
    _others_stand(c, out, lse, touched, pd.last_decode_variant() == "mma")


@pytest.mark.parametrize("shape", SIMT + MMA)
@pytest.mark.parametrize("length,splits", [(16, 0), (400, 0), (400, 1), (400, 5)])
def test_an_infinite_key_scale_with_scores_of_one_sign(shape, length, splits):
    """Scores of -inf alone would look like rows that do not count."""
    c = _case(*shape, [length, 50], seed=2)
    c["Q"] = -c["Q"]
    for row in range(0, length, c["S"]):
        page, blk = _at(c, 0, row)
        c["scales"][page, 0, 1, blk] = INF
    out, lse = _run(c, num_splits=splits)
    touched = torch.zeros(2, c["n"], 4, dtype=torch.bool, device=DEV)
    touched[0, :, 2:] = True
    assert not torch.isfinite(out[touched]).any() and not torch.isfinite(lse[touched]).any()
    _others_stand(c, out, lse, touched, pd.last_decode_variant() == "mma")


@pytest.mark.parametrize("shape", SIMT + MMA)
@pytest.mark.parametrize("top", [0.0, 2.0 ** -126, 2.0 ** -100])
@pytest.mark.parametrize("rest", [1.0, 4.0, 1e4, 1e30])
def test_finite_scales_give_finite_outputs(shape, top, rest):
    """The rows of by far the largest weight hold zeros under a tiny scale, the others, whose
    weights underflow, large values: 0 * anything finite is 0."""
    c = _case(*shape, [80], seed=4)
    page, blk = _at(c, 0, 0)
    c["scales"][:, 1] = rest
    c["scales"][page, 0, :, blk] = 4.0
    c["scales"][page, 1, :, blk] = top
    c["codes"][page, 1, :, blk * c["S"]:(blk + 1) * c["S"]] = 0
    out, lse = _run(c, num_splits=1)
    ref = _ref(c)
    # the first block's scores lead by thousands in log2 units: 1e30 * 100 * 2^-1000 counts as 0
    assert torch.isfinite(out).all() and (out.double() - ref[0]).abs().max() <= 1e-30
    # a score is off by at most 24 roundings of 2^-24 of its sum of magnitudes, here itself
    assert ((lse.double() - ref[1]).abs() <= 2.0 ** -19 * ref[1].abs() + 1e-6).all()


@pytest.mark.parametrize("shape", SIMT + MMA)
@pytest.mark.parametrize("splits", [1, 3])
@pytest.mark.parametrize("bad", [NAN, INF])
def test_a_bad_value_scale_under_a_weight_of_zero(shape, splits, bad):
    """A peaked softmax: the block's weights underflow, its values are still attended."""
    c = _case(*shape, [200, 60], seed=3)
    page, blk = _at(c, 0, 0)
    c["scales"][page, 0, 0, blk] = 4.0  # scores of the first block hundreds above the others'
    page, blk = _at(c, 0, 100)
    c["scales"][page, 1, 0, blk] = bad
    out, lse = _run(c, num_splits=splits)
    touched = torch.zeros(2, c["n"], 4, dtype=torch.bool, device=DEV)
    touched[0, :, :2] = True
    assert not torch.isfinite(out[touched]).any() and torch.isfinite(lse).all()
    _others_stand(c, out, lse, touched, pd.last_decode_variant() == "mma")


@pytest.mark.parametrize("shape", [x for x in MMA if x[-1] > 1])
@pytest.mark.parametrize("bad", [NAN, INF])
def test_a_bad_value_scale_stays_from_earlier_tokens(shape, bad):
    """Of several queries those whose limit lies before the block are untouched, whatever the others
    weigh it with."""
    n, S = shape[-1], shape[3]
    L = 4 * S + 1  # the last row opens a block that the last token alone attends
    for lead in (0.02, 4.0):
        c = _case(*shape, [L], seed=6)
        page, blk = _at(c, 0, 0)
        c["scales"][page, 0, 0, blk] = lead
        page, blk = _at(c, 0, L - 1)
        c["scales"][page, 1, 0, blk] = bad
        out, lse = _run(c)
        touched = torch.zeros(1, n, 4, dtype=torch.bool, device=DEV)
        touched[0, -1, :2] = True
        assert not torch.isfinite(out[touched]).any()
        _others_stand(c, out, lse, touched, True)


@pytest.mark.parametrize("shape", SIMT + MMA)
@pytest.mark.parametrize("splits", [0, 1, 4])
@pytest.mark.parametrize("side", [0, 1])
@pytest.mark.parametrize("bad", [NAN, INF])
def test_a_bad_scale_with_a_learned_sink(shape, splits, side, bad):
    """The sink's weight joins a NaN denominator: lse is NaN beside the output."""
    c = _case(*shape, [40, 700, 3], seed=1)
    page, blk = _at(c, 1, 300)
    c["scales"][page, side, 0, blk] = bad
    sink = torch.tensor([0.0, 3.0, 60.0, -2.0], device=DEV)
    out, lse = _run(c, num_splits=splits, sink=sink)
    touched = torch.zeros(3, c["n"], 4, dtype=torch.bool, device=DEV)
    touched[1, :, :2] = True
    assert torch.isnan(out[touched]).all()
    assert torch.isnan(lse[touched]).all() if side == 0 else torch.isfinite(lse[touched]).all()
    _others_stand(c, out, lse, touched, pd.last_decode_variant() == "mma", sink)


def test_merge_states_keeps_a_nan():
    """Partials of a decode split over ranks: one that is NaN shows, also beside empty ones only."""
    D = 64
    for R in (2, 5, 40):
        V, S = torch.zeros(R, 3, 2, D, device=DEV), torch.full((R, 3, 2), -5e4, device=DEV)
        S[R - 1, 0, 0], V[R - 1, 0, 0] = NAN, NAN      # among empty partners
        S[R - 1, 1, 0], V[R - 1, 1, 0] = NAN, NAN      # beside one with rows
        S[0, 1, 0], V[0, 1, 0] = 2.0, 1.0
        S[0, 2, 1], V[0, 2, 1] = 3.0, 0.5
        out, lse = torch.empty(3, 2, D, device=DEV), torch.empty(3, 2, device=DEV)
        pd.merge_states(out, lse, V, S)
        assert torch.isnan(out[:2, 0]).all() and torch.isnan(lse[:2, 0]).all()
        assert (out[2, 1] == 0.5).all() and lse[2, 1] == 3.0
        assert (out[:, 1][:2] == 0).all() and (lse[:, 1][:2] == -5e4).all() and (out[2, 0] == 0).all()
