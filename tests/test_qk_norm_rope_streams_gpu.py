"""qk_norm_rope on another stream than the current one."""
import pytest
import torch

from tests.test_qk_norm_rope_gpu import DEV, _inputs, check_norm_rope, pd

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("raw", [False, True])
def test_new_outputs_are_allocated_on_the_call_s_stream(raw):
    """Memory freed on the current stream may still be read there: outputs that the call makes for
    work on another stream do not come from it."""
    q, k, wq, wk, pos = _inputs(64, 8, 8, 128, "bf16", seed=1)
    freq = pd.rope_frequencies(128, 1e4, device=DEV)
    st = torch.cuda.Stream()
    old = [torch.ones_like(q), torch.ones_like(k)]
    kept = [torch.empty_like(q), torch.empty_like(k)]
    torch.cuda.synchronize()
    torch.cuda._sleep(100_000_000)  # about 50 ms of the current stream
    for a, b in zip(kept, old):
        a.copy_(b)                  # reads `old` after that
    del old, a, b
    qo, ko = pd.qk_norm_rope(q, k, wq, wk, pos, freq, stream=st.cuda_stream if raw else st)
    st.synchronize()
    torch.cuda.synchronize()
    assert all((x == 1).all() for x in kept)
    check_norm_rope(q, wq, pos, freq, qo)
    check_norm_rope(k, wk, pos, freq, ko)


def test_new_outputs_on_the_default_stream():
    q, k, wq, wk, pos = _inputs(5, 2, 1, 64, "f16", seed=2)
    freq = pd.rope_frequencies(64, 1e4, device=DEV)
    torch.cuda.synchronize()
    for stream in (0, torch.cuda.default_stream()):
        qo, ko = pd.qk_norm_rope(q, k, wq, wk, pos, freq, stream=stream)
        torch.cuda.synchronize()
        check_norm_rope(q, wq, pos, freq, qo)
        check_norm_rope(k, wk, pos, freq, ko)


def test_new_outputs_on_a_stream_of_another_kind():
    """Anything that turns into a handle, as the calls take it."""
    class Handle:
        def __init__(self, st):
            self.st = st

        def __int__(self):
            return self.st.cuda_stream
    q, k, wq, wk, pos = _inputs(5, 2, 1, 64, "f16", seed=3)
    freq = pd.rope_frequencies(64, 1e4, device=DEV)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    qo, ko = pd.qk_norm_rope(q, k, wq, wk, pos, freq, stream=Handle(st))
    torch.cuda.synchronize()
    check_norm_rope(q, wq, pos, freq, qo)
    check_norm_rope(k, wk, pos, freq, ko)
