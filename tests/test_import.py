"""The package imports where torch was built without CUDA; its calls then say
what they need."""
import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROGRAM = """
import torch
for name in [n for n in dir(torch._C) if n.startswith(("_cuda_", "_CudaStream", "_CudaEvent", "_CUDAGraph"))]:
    delattr(torch._C, name)
torch.cuda.is_available = lambda: False
import gated_softmax_attention_fp32_b200 as pkg
q = torch.zeros(1, 2, 2, 64, dtype=torch.bfloat16)
f = torch.zeros(32)
calls = (lambda: pkg.fix_rotary(q, q, f), lambda: pkg.fix_attn_rotary(q, q, f),
         lambda: pkg.fix_attn_append_paged(q, q, q.float(), q, q, q.float(), None, None),
         lambda: pkg.fix_attn_decode_paged(q[0], q, q, q.float(), None, None))
for call in calls:
    try:
        call()
    except ValueError as e:
        assert "must be a CUDA tensor" in str(e), e
    else:
        raise SystemExit("a call on CPU tensors went through")
"""


def test_import_and_refusals_without_cuda_in_torch():
    r = subprocess.run([sys.executable, "-c", PROGRAM], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
