"""A plain C program as a user of include/ag_moe.h (tests/c_client/ag_moe_client.c): it
compiles and links with gcc here, and checks a small layer on a GB300."""
import os
import shutil
import subprocess

import pytest

from all_gather_gemm_chunked_gb300 import build as _build

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CUDA = os.environ.get("CUDA_HOME", "/usr/local/cuda")


@pytest.fixture(scope="module")
def client(tmp_path_factory):
    if shutil.which("gcc") is None:
        pytest.skip("gcc not found")
    libdir = os.path.dirname(_build.build())
    exe = str(tmp_path_factory.mktemp("c_moe_client") / "ag_moe_client")
    cmd = ["gcc", "-O2", "-std=c99", "-Wall", "-Werror", "-I", os.path.join(ROOT, "include"), "-I", os.path.join(CUDA, "include"),
           os.path.join(HERE, "c_client", "ag_moe_client.c"), "-o", exe, "-L", libdir, "-laggemm",
           "-L", os.path.join(CUDA, "lib64"), "-lcudart", f"-Wl,-rpath,{libdir}:{os.path.join(CUDA, 'lib64')}"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    return exe


def test_compiles_and_links(client):
    assert os.access(client, os.X_OK)


@pytest.mark.gpu
def test_small_layer(client):
    r = subprocess.run([client], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stderr
