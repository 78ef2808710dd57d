"""Short batches with any number of query columns a KV head, planned on the device and on the host."""
import pytest
import torch

from tests.test_bs_gpu import _case, _check, pd

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("lengths,Hq,H,n,D,P,S,kv", [
    ([640], 64, 8, 5, 128, 16, 16, "int8"),            # a block for each of 40 segments
    ([300, 2, 0, 517], 24, 1, 1, 64, 8, 8, "e4m3"),    # three slices
    ([100, 100, 100], 16, 1, 16, 128, 16, 16, "e4m3"), # sixteen
    ([70] * 9, 12, 3, 12, 64, 32, 16, "int8"),         # six
    ([40] * 40, 24, 8, 5, 64, 16, 16, "int8"),         # 640 segments: both slices in a block
    ([16, 700] * 8, 18, 2, 8, 128, 16, 16, "int8"),    # nine, uneven
    ([90, 30], 32, 2, 4, 128, 8, 4, "int8"),           # eight, gathered rows
    ([500, 1], 48, 2, 2, 128, 16, 16, "e4m3"),
])
def test_decode_short_batches_of_many_columns(lengths, Hq, H, n, D, P, S, kv):
    c = _case(lengths, Hq, H, D, P, S, kv, "bf16", n=n, seed=len(lengths) + n)
    a = _check(c, "mma")
    assert torch.equal(_check(c, "mma")[0], a[0])
    _check(c, "mma", host_meta=pd.host_meta_of(c["indptr"], c["li"]))
