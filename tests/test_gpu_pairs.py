"""The per-tensor GEMM's CTA-pair kernels, launched some millions of pairs long
beside casts on another stream: every pair gets its tensor memory and the
results stay the same."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

CODE = """
import torch
from fp8_mixed_precision_tensor_b200 import fp8, synth
M, N, K = {M}, {N}, 128
u8 = dict(dtype=torch.uint8, device="cuda")
xq, wq = (torch.randint(0, 120, s, **u8) for s in ((M, K), (N, K)))
inv = torch.ones(1, device="cuda")
y, amax = torch.empty((M, N), dtype=torch.bfloat16, device="cuda"), torch.zeros(1, device="cuda")
h, hq, one = synth.device_normal((1 << 20,), 1.0, 3, torch.bfloat16, "cuda"), torch.empty(1 << 20, **u8), torch.ones(1, device="cuda")
fp8.fp8_linear_fwd(xq, inv, wq, inv, y, amax)
first = y.clone()
side = torch.cuda.Stream()
torch.cuda.synchronize()
for _ in range(20):
    for i in range(1000):
        fp8.fp8_linear_fwd(xq, inv, wq, inv, y, amax)
        if i % 4 == 0:
            fp8.fp8_cast(h, fp8.FP8_E4M3, one, hq, stream=side)
    torch.cuda.synchronize()
assert torch.equal(y, first) and fp8.fp8_get_status() == 0
print("ok")
"""


@pytest.mark.parametrize("M,N", [(2560, 2048), (2560, 4096)])  # 256 x 256 and 256 x 512 tiles
def test_pairs_take_and_give_back_tensor_memory_many_times(M, N):
    # in a process of its own, so that it could be ended
    r = subprocess.run([sys.executable, "-c", CODE.format(M=M, N=N)], capture_output=True, text=True, timeout=120,
                       cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
    assert r.returncode == 0 and r.stdout.strip().endswith("ok"), r.stderr[-2000:]
