"""A learned sink of -inf is a head without one, of empty sequences too."""
import math

import pytest
import torch

import paged_kv_decode_19_gb300 as pd
from tests import _bs

pytestmark = pytest.mark.gpu
dev = "cuda"


@pytest.mark.parametrize("kind,dt,D", [("plain", "bf16", 128), ("plain", "f32", 64), ("bs", "bf16", 128), ("bs", "f32", 128)])
@pytest.mark.parametrize("splits", [0, 1])
def test_minus_infinity(kind, dt, D, splits):
    g = torch.Generator().manual_seed(0)
    lengths, H, Hq, P = [0, 1, 700], 2, 4, 16
    indptr, vals, li, total = _bs.table(lengths, P, dev, g)
    Q = torch.randn(3, Hq, D, generator=g).to(_bs.DT[dt]).to(dev)
    if kind == "bs":
        codes, scales = _bs.cache(total, H, P, 16, D, "int8", dev, g)
    else:
        pages = torch.randn(total, 2, H, P, D, generator=g).to(_bs.DT[dt]).to(dev)

    def run(sink):
        out, lse = torch.full_like(Q, 7.0), torch.full((3, Hq), 7.0, device=dev)
        if kind == "bs":
            pd.batch_decode_paged_kv_bs(Q, codes, scales, indptr, vals, li, out, lse, sink=sink, num_splits=splits)
        else:
            pd.batch_decode_paged_kv(Q, pages, indptr, vals, li, None, None, out, lse, sink=sink, num_splits=splits)
        return out, lse

    out, lse = run(torch.tensor([-math.inf, 1.0, -math.inf, -2.0], device=dev))
    ref, ref_lse = run(None)
    for h in (0, 2):
        assert torch.equal(out[:, h], ref[:, h]) and torch.equal(lse[:, h], ref_lse[:, h])
    assert (out[0] == 0).all() and (lse[0, ::2] == -5e4).all()
    want = torch.tensor([1.0, -2.0], device=dev) / math.log(2)
    assert (lse[0, 1::2] - want).abs().max() < 1e-5
