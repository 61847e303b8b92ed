"""The binding of the 8-bit rows loads on a torch built without a GPU, and refuses its tensors by name."""
import subprocess
import sys

CODE = """
import torch
for name in ("_cuda_getDevice", "_cuda_getCurrentRawStream"):
    delattr(torch._C, name)
from moe_layer_03_amd import binding as B, quantized as Q
x = torch.zeros(4, 64)
a, p = x.to(torch.int8), torch.zeros(1 << 16, dtype=torch.uint8)
for call in (lambda: Q.moe_add_rmsnorm(x, q_dtype=Q.MOE_I8), lambda: Q.moe_quantize_int8(x),
             lambda: Q.moe_pack_dense_int8(B.DenseShape(4, 64, 4), x),
             lambda: Q.moe_dense_gemm_int8(B.DenseShape(4, 64, 64), a, x[:, 0], p)):
    try:
        call()
    except ValueError as e:
        print("GPU tensor" in str(e))
"""


def test_a_torch_without_a_gpu():
    r = subprocess.run([sys.executable, "-c", CODE], capture_output=True, text=True, timeout=110)
    assert r.returncode == 0, r.stderr
    assert r.stdout.split() == ["True"] * 4
