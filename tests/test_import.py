"""CPU test: the binding imports with a torch that was built without CUDA."""
import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CODE = """
import torch
for name in [n for n in dir(torch._C) if n.startswith("_cuda_")]:
    delattr(torch._C, name)
from tiled_online_softmax_fwd_gb300 import fattn
x = torch.zeros(1, 2, 3, 64, dtype=torch.bfloat16)
lists = [torch.zeros(n, dtype=torch.int32) for n in (1, 2, 1)]
for call in (lambda: fattn.qk_norm_rope(x, x), lambda: fattn.qk_norm_rope_bwd(x, x, x, x),
             lambda: fattn.kv_append(x[0], x[0], x, x, *lists),
             lambda: fattn.attn_fwd_paged(x[0], x, x, *lists, 1)):
    try:
        call()
    except ValueError:
        continue
    raise SystemExit("a call with CPU tensors was not refused")
print(fattn.rope_table(4, 16, device="cpu").shape[0])
"""


def test_import_without_cuda_in_torch():
    r = subprocess.run([sys.executable, "-c", CODE], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "4", r.stderr[-2000:]
