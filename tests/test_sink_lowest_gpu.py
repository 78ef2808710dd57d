"""A learned sink far below every score: a sequence without rows gives zeros and the sink's own
log-sum-exp, others what they give without it."""
import math

import pytest
import torch

import paged_kv_decode_19_gb300 as pd
from tests import _bs, _mx

pytestmark = pytest.mark.gpu
dev = "cuda"
LOW = [-1e9, -65504.0, -4e4, -3e4, -1e30, float(torch.finfo(torch.float32).min), float(torch.finfo(torch.bfloat16).min), -2e38]


@pytest.mark.parametrize("kind,dt,D", [("plain", "bf16", 128), ("plain", "f32", 64), ("noalloc", "f16", 128), ("bs", "bf16", 128),
                                       ("bs", "f32", 128), ("mx", "bf16", 128), ("mx", "f32", 64)])
@pytest.mark.parametrize("q_len", [1, 2])
@pytest.mark.parametrize("splits", [0, 1])
def test_lowest(kind, dt, D, q_len, splits):
    if q_len > 1 and (kind == "noalloc" or (kind != "mx" and dt == "f32")):
        pytest.skip("one query token only")
    g = torch.Generator().manual_seed(0)
    lengths, H, Hq, P = [0, 2, 700], 2, 8, 16
    indptr, vals, li, total = _bs.table(lengths, P, dev, g)
    Q = torch.randn(3, *([q_len] if q_len > 1 else []), Hq, D, generator=g).to(_bs.DT[dt]).to(dev)
    if kind == "bs":
        codes, scales = _bs.cache(total, H, P, 16, D, "int8", dev, g)
    elif kind == "mx":
        codes, scales = _mx.cache(total, H, P, D, "e4m3", dev, g)
    else:
        pages = torch.randn(total, 2, H, P, D, generator=g).to(_bs.DT[dt]).to(dev)

    def run(sink):
        out, lse = torch.full_like(Q, 7.0), torch.full(Q.shape[:-1], 7.0, device=dev)
        a = dict(sink=sink, num_splits=splits)
        if kind == "bs":
            pd.batch_decode_paged_kv_bs(Q, codes, scales, indptr, vals, li, out, lse, **a)
        elif kind == "mx":
            pd.batch_decode_paged_kv_mx(Q, codes, scales.view(torch.float8_e4m3fn), indptr, vals, li, out, lse, **a)
        elif kind == "noalloc":
            pd.batch_decode_paged_kv_noalloc(Q, pages, indptr, vals, li, None, None, out, lse, sink=sink)
        elif q_len > 1:
            pd.batch_decode_paged_kv_mq(Q, pages, indptr, vals, li, None, None, out, lse, **a)
        else:
            pd.batch_decode_paged_kv(Q, pages, indptr, vals, li, None, None, out, lse, **a)
        assert pd.check_device_errors() == "PD_OK"
        return out, lse

    sink = torch.tensor(LOW, device=dev)
    out, lse = run(sink)
    ref, ref_lse = run(None)
    assert torch.equal(out, ref) and torch.equal(lse[1:], ref_lse[1:])
    assert (out[0] == 0).all()
    want = sink.double() / math.log(2)
    # (a product beyond fp32 is the -inf of a head without a sink)
    want = torch.where(want < torch.finfo(torch.float32).min, -5e4, want)
    assert ((lse[0].double() - want).abs() <= want.abs() * 2.0 ** -23).all()
