"""The walk of the linear layers over their output tiles, built for the host
with the undefined-behaviour sanitizer (tests/native/linear_tiles_check.cpp):
every tile once, no product past 32 bits.  No GPU."""
import os
import shutil
import subprocess

import pytest

from conftest import ROOT

CSRC = os.path.join(ROOT, "quantized_mixture_experts_router_amd", "csrc")


@pytest.mark.timeout(300)
def test_every_tile_once(tmp_path):
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("no host C++ compiler")
    exe = tmp_path / "linear_tiles_check"
    cmd = [cxx, "-std=c++17", "-O1", "-fsanitize=undefined", "-fno-sanitize-recover=all", "-I", CSRC,
           os.path.join(ROOT, "tests", "native", "linear_tiles_check.cpp"), "-o", str(exe)]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    env = dict(os.environ)
    env.pop("LD_PRELOAD", None)
    r = subprocess.run([str(exe)], capture_output=True, text=True, env=env, timeout=200)
    print(r.stdout)
    assert r.returncode == 0 and " 0 failures" in r.stdout, r.stdout + r.stderr[-2000:]
    assert "runtime error" not in r.stderr
