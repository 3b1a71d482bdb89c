"""Which parts of its workspace a call of gdn_attn_extend writes and joins, replayed on the host with the kernels' own
plan and order of parts (tests/extend_parts_driver.cpp): no workgroup writes past the workspace, also where the
sequences' offsets go back and ask for more than the plan counts on, and the join reads only what was written."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PKG = os.path.join(ROOT, "gated_deltanet_linear_prefill_amd")
CLANG = "/opt/rocm/lib/llvm/bin/clang++"


@pytest.mark.skipif(shutil.which("hipcc") is None or shutil.which("nm") is None or not os.path.exists(CLANG), reason="needs the ROCm toolchain")
def test_parts_stay_in_the_workspace(tmp_path):
    tiles = os.path.join(PKG, "_build", "gdn_attn_extend_tile.hip.o")
    if not os.path.exists(tiles):
        pytest.skip("build the library first")
    obj, exe = tmp_path / "parts.o", tmp_path / "parts"
    subprocess.run(["hipcc", "-x", "hip", "--offload-arch=gfx950", "--offload-host-only", "-O1", "-std=c++17", "-I", os.path.join(ROOT, "include"),
                    "-I", os.path.join(PKG, "csrc"), "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
                    "-c", os.path.join(ROOT, "tests", "extend_parts_driver.cpp"), "-o", str(obj)], check=True, capture_output=True, text=True)
    # the kernels are not compiled: their code is an empty symbol
    names = subprocess.run(["nm", "-u", str(obj)], check=True, capture_output=True, text=True).stdout.split()
    empty = sorted({f"-Wl,--defsym={x}=0" for x in names if x.startswith("__hip_fatbin")})
    subprocess.run([CLANG, str(obj), tiles, *empty, "-lstdc++", "-lm", "-L/opt/rocm/lib", "-lamdhip64", "-Wl,-rpath,/opt/rocm/lib", "-o", str(exe)],
                   check=True, capture_output=True, text=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr
    assert "extend parts ok" in r.stdout
