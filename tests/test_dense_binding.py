"""Host side of the dense layers' binding, without a GPU."""
import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_package_imports_on_a_torch_without_gpu_support():
    """Only a torch built for GPUs has the private raw-stream call."""
    code = ("import torch\n"
            "if hasattr(torch._C, '_cuda_getCurrentRawStream'): del torch._C._cuda_getCurrentRawStream\n"
            "import submanifold_sparse_convolution_hash_amd as sc\n"
            "assert callable(sc.linear)\n")
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
