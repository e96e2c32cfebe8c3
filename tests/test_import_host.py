"""What importing the package brings with it."""
import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def run(code):
    return subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=300)


def test_import_leaves_torch_to_the_tensor_functions():
    """The C-named functions and the sizes they report need no torch, nor the second it takes to import."""
    r = run("import sys, latency_skinny_bf16_gb300 as sk\n"
            "assert sk.skinny_lora_workspace(5, 48, 8, sk.SKINNY_F32) == 5 * 32 * 6\n"
            "assert 'torch' not in sys.modules, 'torch came along'")
    assert r.returncode == 0, r.stderr


def test_tensor_functions_import_torch_themselves():
    r = run("import latency_skinny_bf16_gb300 as sk\n"
            "class F:\n"
            "    dtype = 'float32'\n"
            "assert sk.lora_workspace(5, 48, 8, F.dtype) == 5 * 32 * 6\n"
            "import torch\n"
            "assert sk.lora_workspace(5, 48, 8, torch.bfloat16) == 5 * 32 * 6 + 5 * 48 * 4")
    assert r.returncode == 0, r.stderr
