"""The paged grouped-query operators from plain C99: tests/c/kvq_paged_client.c
compiles and links against include/kvq.h and libkvq.so on the host, and runs
its exact-by-construction case on the GPU."""
import os
import shutil
import subprocess

import pytest

import kv_quant_cache_gb300 as kvq

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SRC = os.path.join(ROOT, "tests", "c", "kvq_paged_client.c")
CUDA_HOME = os.environ.get("CUDA_HOME", "/usr/local/cuda")


def _compile(out_dir):
    gcc = shutil.which("gcc")
    if gcc is None or not os.path.exists(os.path.join(CUDA_HOME, "include", "cuda_runtime.h")):
        pytest.skip("gcc or the CUDA runtime headers are not available")
    kvq.lib()  # the library is built
    pkg = os.path.dirname(kvq.LIB_PATH)
    exe = os.path.join(out_dir, "kvq_paged_client")
    cmd = [gcc, "-std=c99", "-O2", "-Wall", "-Wextra", "-Werror",
           "-I", os.path.join(ROOT, "include"), "-I", os.path.join(CUDA_HOME, "include"),
           SRC, "-o", exe, "-L", pkg, "-lkvq", "-L", os.path.join(CUDA_HOME, "lib64"), "-lcudart",
           f"-Wl,-rpath,{pkg}", f"-Wl,-rpath,{os.path.join(CUDA_HOME, 'lib64')}"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stdout + r.stderr
    return exe


def test_paged_client_compiles_and_links(tmp_path):
    assert os.path.exists(_compile(str(tmp_path)))


@pytest.mark.gpu
def test_paged_client_runs(tmp_path, cuda_device):
    r = subprocess.run([_compile(str(tmp_path))], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stdout + r.stderr
    assert "paged c client ok" in r.stdout
