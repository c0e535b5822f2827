"""How prompt-side attention cuts its work over the CTAs: the kernel's own
arithmetic, compiled for the host (tests/c_abi/prefill_cuts.cpp)."""
import os
import shutil
import subprocess

import pytest

from paged_kv_cache_268_gb300 import build
from test_c_abi import cuda_home

SRC = os.path.join(os.path.dirname(os.path.abspath(__file__)), "c_abi", "prefill_cuts.cpp")


def test_cuts_cover_the_work(tmp_path):
    if shutil.which("g++") is None:
        pytest.skip("no g++")
    exe = str(tmp_path / "cuts")
    # (signed overflow, which the 32-bit scheduler must not reach, aborts)
    r = subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Wextra", "-Werror", "-fsanitize=signed-integer-overflow",
                        "-fsanitize-undefined-trap-on-error", "-I", build.INCLUDE, "-I", build.CSRC,
                        "-isystem", os.path.join(cuda_home(), "include"), SRC, "-o", exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([exe], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr
    assert r.stdout.endswith("ok\n")
    print(r.stdout)
