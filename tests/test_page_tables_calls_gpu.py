"""build_page_tables: calls of several host threads, a first call under capture, and slot maps without room."""
import os
import subprocess
import sys
import threading

import pytest
import torch

import paged_kv_decode_19_gb300 as pd

pytestmark = pytest.mark.gpu
dev = "cuda"
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _args(B, T):
    i32 = lambda *n: torch.zeros(*n, dtype=torch.int32, device=dev)  # noqa: E731
    return dict(page_table=torch.arange(2 * B, dtype=torch.int32, device=dev).view(B, 2), lengths=i32(B) + 5,
                new_tokens=i32(B) + 1, state=torch.zeros(4, dtype=torch.int64, device=dev), page_size=16,
                page_table_indptr=i32(B + 1), page_table_values=i32(2 * B), length_info=i32(B),
                slot_mapping=torch.zeros(T, dtype=torch.int64, device=dev), positions=i32(T))


def test_host_threads_with_batches_of_different_size():
    """Batches whose sums need different amounts of shared memory, from two threads at once."""
    calls, failed = 3000, []

    def work(B):
        try:
            a, s = _args(B, B), torch.cuda.Stream()
            s.wait_stream(torch.cuda.current_stream())
            a["new_tokens"].zero_()
            torch.cuda.synchronize()
            for _ in range(calls):
                pd.build_page_tables(**a, stream=s)
            a["new_tokens"].fill_(1)
            torch.cuda.synchronize()
            pd.build_page_tables(**a, stream=s)
            torch.cuda.synchronize()
            assert (a["lengths"] == 6).all() and (a["length_info"] == 6).all()
            assert torch.equal(a["slot_mapping"], 32 * torch.arange(B, device=dev) + 5)
        except Exception as e:  # noqa: BLE001 (shown by the assertion below)
            failed.append((B, e))

    threads = [threading.Thread(target=work, args=(B,)) for B in (3000, 8192, 2500, 5000)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed, failed
    assert pd.check_device_errors() == "PD_OK"


@pytest.mark.parametrize("given", [("slot_mapping",), ("positions",), ("slot_mapping", "positions")])
def test_slot_maps_without_room(given):
    """A slot map (or positions) of no entries holds no new token: a step that brings some changes nothing."""
    a = _args(3, 0)
    for name in {"slot_mapping", "positions"} - set(given):
        a[name] = None
    pd.build_page_tables(**a)
    assert pd.check_device_errors() == "PD_ERR_BAD_LENGTH"
    assert a["lengths"].tolist() == [5, 5, 5] and a["page_table_indptr"].tolist() == [0, 0, 0, 0]
    a["new_tokens"].copy_(torch.tensor([0, -5, -1]))
    pd.build_page_tables(**a)
    assert pd.check_device_errors() == "PD_OK"
    assert a["lengths"].tolist() == [5, 0, 4] and a["page_table_indptr"].tolist() == [0, 1, 1, 2]


FIRST = """
import sys
import torch
sys.path.insert(0, %r)
import paged_kv_decode_19_gb300 as pd
from tests.test_page_tables_calls_gpu import _args
a = _args(%d, %d)
s, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
torch.cuda.synchronize()
with torch.cuda.graph(graph, stream=s):
    pd.build_page_tables(**a)
assert (a["lengths"] == 5).all()
for n in (6, 7):
    graph.replay()
    torch.cuda.synchronize()
    assert pd.check_device_errors() == "PD_OK" and (a["lengths"] == n).all() and (a["length_info"] == n).all()
"""


@pytest.mark.parametrize("B", [3, 8192])
def test_the_first_call_of_a_process_is_captured(B):
    r = subprocess.run([sys.executable, "-c", FIRST % (ROOT, B, B)], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr
