"""The package imports with a torch that lacks the types which only the 4-bit cache takes."""
import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CODE = """
import torch
for name in ("float8_e8m0fnu", "float4_e2m1fn_x2"):
    if hasattr(torch, name):
        delattr(torch, name)
import paged_kv_decode_19_gb300 as pd
z = lambda *n: torch.zeros(*n, dtype=torch.uint8)
k = torch.zeros(5, 2, 64, dtype=torch.bfloat16)
try:
    pd.append_paged_kv_mx(z(4, 2, 2, 32, 32), z(4, 2, 2, 32, 4).view(torch.float8_e4m3fn), k, k, torch.zeros(5, dtype=torch.int64))
except ValueError as e:
    assert "current GPU" in str(e), e  # (the only thing wrong)
else:
    raise SystemExit("not refused")
"""


def test_without_the_newest_types():
    r = subprocess.run([sys.executable, "-c", CODE], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr
