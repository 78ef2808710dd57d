"""4-bit decode, several query tokens: tokens that attend no row of a share beside tokens that do, under
column factors (2^(e - 14) |sm_scale| log2(e) k_scale, 2^e the column's largest |Q|) above 1."""
import pytest
import torch

import paged_kv_decode_19_gb300 as pd
from tests.test_mx_gpu import _check, _decode_case, _ref

pytestmark = pytest.mark.gpu

# a last page or tile of fewer rows than tokens, and sequences of fewer rows than tokens
LENS = [1, 2, 4, 17, 33, 49, 161, 16, 0, 340]


@pytest.mark.parametrize("q_len", [2, 3, 5])
@pytest.mark.parametrize("dt,D,P,ks", [("bf16", 64, 16, 2.0 ** 16), ("f16", 128, 32, 2.0 ** 17), ("bf16", 128, 20, 2.0 ** 17),
                                       ("f16", 256, 16, 2.0 ** 17), ("f32", 64, 7, 2.0 ** 16), ("f32", 128, 16, 2.0 ** 17)])
def test_least_scales_under_a_large_cache_scale(dt, D, P, ks, q_len):
    """Power-of-two scales of 2^-14: ordinary K and scores, factors above 1."""
    c = _decode_case(LENS, 6, 2, D, P, dt, "e8m0", q_len=q_len, seed=q_len, ks=ks, vs=2.0 ** 14)
    c["scales"].fill_(113)
    ref = _ref(c)
    for n in (0, 1, 3, 64):
        out, lse = _check(c, ref=ref, num_splits=n)
        assert torch.isfinite(out.float()).all() and torch.isfinite(lse).all()
    _check(c, ref=ref, host_meta=pd.host_meta_of(c["indptr"], c["li"]))


@pytest.mark.parametrize("q_len", [2, 5])
@pytest.mark.parametrize("dt,D,P,qs,ks", [("f16", 128, 16, 5000.0, 8.0), ("bf16", 128, 16, 1000.0, 128.0), ("f32", 64, 20, 1e6, 1.0)])
def test_large_queries(dt, D, P, qs, ks, q_len):
    c = _decode_case(LENS, 6, 2, D, P, dt, "e4m3", q_len=q_len, seed=q_len, ks=ks, qs=qs)
    sink = torch.tensor([0.5, -1.0, 8.0, 2.0, 0.0, 30.0], device="cuda")
    for n in (0, 1, 3):
        out, lse = _check(c, sink=sink if n else None, num_splits=n)
        assert torch.isfinite(out.float()).all() and torch.isfinite(lse).all()
