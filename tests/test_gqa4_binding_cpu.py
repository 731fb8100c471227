"""The binding of the 4-bit cache on CPU: torch without a 4-bit type."""
import os
import subprocess
import sys

_IMPORT = """
import torch
if hasattr(torch, "float4_e2m1fn_x2"):
    del torch.float4_e2m1fn_x2
from hybrid_sparse_mqa_gb300 import attn as A
table = torch.zeros(1, 2, dtype=torch.int32)
wide = torch.zeros(2, 2, 16, 64, dtype=torch.bfloat16)
assert A.make_gqa_cache(wide, wide, table).format == A.DSV4_GQA_BF16
codes, blocks = torch.zeros(2, 2, 16, 32, dtype=torch.uint8), torch.zeros(2, 2, 16, 4).to(torch.float8_e4m3fn)
assert A.make_gqa_cache(codes, codes, table, k_blocks=blocks, v_blocks=blocks).format == A.DSV4_GQA_E2M1
print("imported")
"""


def test_torch_without_a_4_bit_type():
    # caches of the other types, and 4-bit ones of bytes, need no more than they did
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    run = subprocess.run([sys.executable, "-c", _IMPORT], cwd=root, capture_output=True, text=True, timeout=300)
    assert run.returncode == 0 and "imported" in run.stdout, run.stderr[-2000:]
