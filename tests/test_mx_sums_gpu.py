"""4-bit decode, 16-bit Q: the sums over a long share."""
import math

import pytest
import torch

import paged_kv_decode_19_gb300 as pd
from tests import _mx
from tests.test_mx_gpu import _check as _checked, _decode_case, _run
from tests.test_mx_large_scores_gpu import _case, _check

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("sc", ["e4m3", "e8m0"])
@pytest.mark.parametrize("dt,D,P,q_len", [("bf16", 128, 16, 1), ("f16", 64, 32, 1), ("bf16", 128, 20, 1), ("f16", 256, 16, 1),
                                          ("bf16", 64, 64, 2)])
def test_sums_of_a_long_share(dt, D, P, q_len, sc):
    """Equal values of V over 8192 tiles of 16 rows in one share come out as they are, but for the weights'
    rounding to f16, at most 2^-11 of each, either way and independent: six deviations of their sum are 6
    (2^-11 / sqrt 3) sqrt(sum p^2) with p the normalised weights.  The sums: 256 tiles at a time are added in the
    products' own accumulation, which cuts off up to two units of 2^-23 of the sum so far a tile; as the sum
    grows evenly that is 256 2^-23 of the whole.  Such sums are added rounded to nearest.  (All 8192 tiles in
    one sum: 4e-4.)"""
    n = 8192
    c = _decode_case([16 * n], 2, 1, D, P, dt, sc, seed=D, qs=0.2, q_len=q_len)
    c["codes"][:, 1] = 0x22   # 1.0
    c["scales"][:, 1] = 0x38 if sc == "e4m3" else 127
    out, lse = _run(c, torch.float32, num_splits=1)
    assert pd.check_device_errors() == "PD_OK"
    r = torch.arange(16 * n, device="cuda")
    page = c["vals"][r // P].long()
    k = _mx.row_values(c["codes"][page, 0, 0, r % P], c["scales"][page, 0, 0, r % P], sc)
    s = torch.einsum("thd,rd->thr", c["Q"][0].double(), k) * D ** -0.5
    for t in range(q_len):
        p = torch.softmax(s[t, :, :16 * n - (q_len - 1 - t)], -1)
        bound = 6 * 2.0 ** -11 / math.sqrt(3) * p.square().sum(-1).sqrt() + 256 * 2.0 ** -23
        assert bound.max() < 6e-5  # (many rows count)
        err = (out.view(q_len, 2, D)[t].double() - 1).abs().amax(-1)
        assert (err <= bound).all(), (err / bound).max().item()


@pytest.mark.parametrize("dt,D,P,q_len", [("bf16", 128, 16, 1), ("f16", 64, 20, 1), ("bf16", 256, 32, 2), ("f16", 128, 9, 3),
                                          ("bf16", 256, 12, 1), ("f32", 128, 16, 1)])
def test_the_maximum_moves_from_sum_to_sum(dt, D, P, q_len):
    """Scores in steps of 6 and 12 over shares of up to 1100 tiles, the largest ones late: sums that were taken
    against a smaller maximum join under the last one."""
    def k(r, n):  # (under a scale of 2, codes 0.5 and 0, 3, 6)
        return 1 + 16 * torch.where(r >= n - 3, 7, torch.where(r >= n - n // 2, 5, 0))
    c = _case([17600, 4096, 4097, 8200, 4500], D, P, dt, q_len, k, scale=0x40, q=(-2.0, 1.0), seed=D)
    for n in (1, 2):
        _check(c, num_splits=n)


@pytest.mark.parametrize("sc", ["e4m3", "e8m0"])
@pytest.mark.parametrize("dt,D,P,q_len", [("bf16", 128, 16, 1), ("f16", 64, 20, 2), ("bf16", 256, 16, 1)])
def test_nan_scales_of_a_long_share(dt, D, P, q_len, sc):
    """A NaN scale in any of a share's sums: of V its own dims, of K everything, and nothing else."""
    c = _decode_case([9000, 4100, 9000, 9000], 8, 2, D, P, dt, sc, q_len=q_len, seed=6)
    nan, ip = (0x7f if sc == "e4m3" else 0xff), c["indptr"].tolist()
    for b, r, side, h, blk in ((0, 4, 1, 0, 1), (0, 8990, 1, 1, 0), (1, 4099, 1, 0, 0), (2, 5000, 1, 1, 1), (2, 4000, 0, 0, 0)):
        c["scales"][c["vals"][ip[b] + r // P].long(), side, h, r % P, blk] = nan
    out, _ = _checked(c, num_splits=1)
    assert out.isnan().any() and torch.isfinite(out.view(4, -1)[3].float()).all()
