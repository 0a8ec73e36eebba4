"""The attention's workgroups and their shares, walked on the host."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_every_share_has_one_workgroup(tmp_path):
    gxx = shutil.which("g++")
    if not gxx:
        pytest.skip("g++ is missing")
    exe = str(tmp_path / "kv_grid")
    r = subprocess.run([gxx, "-std=c++17", "-O1", f"-I{os.path.join(ROOT, 'rank_adapter_gemm_build_amd', 'csrc')}",
                        os.path.join(ROOT, "tests", "sanitize", "kv_grid.cpp"), "-o", exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-4000:]
    r = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and r.stdout.strip().endswith("0 failures"), r.stdout[-3000:]
