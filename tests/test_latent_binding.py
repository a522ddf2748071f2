"""The latent-cache operators' binding without a GPU."""
import subprocess
import sys

import exact_bf16_top_gb300 as tk

ROOT = tk._build.ROOT


def test_a_torch_without_cuda_gets_the_refusal():
    # Builds of torch without CUDA lack the private functions that ask for the current device and stream.
    code = """
import torch
for name in ("_cuda_getCurrentRawStream", "_cuda_getDevice"):
    if hasattr(torch._C, name):
        delattr(torch._C, name)
import exact_bf16_top_gb300 as tk
a = torch.zeros(2, 16, 576, dtype=torch.bfloat16)
c = torch.zeros(64, 576, dtype=torch.bfloat16)
i = torch.zeros(2, 4, dtype=torch.int32)
for call in (lambda: tk.latent_attend_selected(a, c, i, 0.1), lambda: tk.latent_attend_paged(a, c, i[:, 0], i, 0.1),
             lambda: tk.latent_append(c, a[:, 0, :512], a[:, 0, 512:], i[:, 0], c.float(), i[:, 0])):
    try:
        call()
    except TypeError as e:
        assert "CUDA tensor" in str(e), e
    else:
        raise AssertionError("not refused")
"""
    subprocess.run([sys.executable, "-c", code], cwd=ROOT, check=True)
