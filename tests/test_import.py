"""The package imports, and its host-side parts work, with a torch that was built without CUDA."""
import os
import subprocess
import sys

from conftest import ROOT


def test_import_without_cudas_private_names():
    code = ("import torch\n"
            "for name in [n for n in dir(torch._C) if n.startswith('_cuda_')]: delattr(torch._C, name)\n"
            "import hashed_gram_conditional_gb300 as eg\n"
            "assert eg.build_layout(1000, 4099, [1]).n_cols == 24\n")
    if not os.path.exists(os.path.join(ROOT, "hashed_gram_conditional_gb300", "libengram.so")):
        from hashed_gram_conditional_gb300 import build
        build.build()
    done = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert done.returncode == 0, done.stderr[-2000:]
