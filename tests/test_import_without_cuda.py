"""The package, its build step and its generators import with a torch that was built without CUDA."""
import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CODE = """
import torch
for name in [n for n in dir(torch._C) if n.startswith("_cuda_")]:
    delattr(torch._C, name)
import model_free_suffix_gb300 as m
from model_free_suffix_gb300 import build, workload
assert m.SuffixDrafter and m.KVCache and m.Verdict and build.SOURCES and workload
"""


def test_import():
    subprocess.run([sys.executable, "-c", CODE], cwd=ROOT, check=True, timeout=300)
