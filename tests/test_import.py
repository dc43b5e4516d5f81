"""The package imports where torch lacks the newest dtypes."""
import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_import_without_the_scale_dtype():
    code = ("import torch\n"
            "if hasattr(torch, 'float8_e8m0fnu'): del torch.float8_e8m0fnu\n"
            "import sparse_attention_07_b200 as sa\n"
            "assert sa._SCALE_TYPES == (torch.uint8,)\n")
    got = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True)
    assert got.returncode == 0, got.stderr
