"""The host code of the entry points around the attention layers built with AddressSanitizer and
UndefinedBehaviorSanitizer, checks and size computations, and driven through refusals and sizes by a
standalone program, as tests/test_sanitize_attn_cpu.py does for the attention layers'. No HIP call is
made."""
import os
import shutil
import subprocess

import pytest

from test_sanitize_abi_cpu import CLANG, PKG, ROOT, SAN_HOST


@pytest.mark.skipif(shutil.which("hipcc") is None or shutil.which("nm") is None or not os.path.exists(CLANG), reason="needs the ROCm toolchain")
def test_extend_validation_under_asan_ubsan(tmp_path):
    rope = os.path.join(PKG, "_build", "gdn_rope.hip.o")
    if not os.path.exists(rope):
        pytest.skip("build the library first")
    objs, exe, builds = [rope], tmp_path / "extend_san", []
    for name in ("gdn_extend_api", "gdn_attn_extend", "gdn_attn_extend_tile"):
        obj = tmp_path / f"{name}.o"
        objs.append(str(obj))
        builds.append(subprocess.Popen(
            ["hipcc", "--offload-arch=gfx950", "--offload-host-only", "-O1", "-g", "-std=c++17", "-fPIC", "-I", os.path.join(ROOT, "include"),
             "-I", os.path.join(PKG, "csrc"), "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops", *SAN_HOST,
             "-c", os.path.join(PKG, "csrc", f"{name}.hip"), "-o", str(obj)], stdout=subprocess.PIPE, stderr=subprocess.PIPE, text=True))
    for b in builds:
        err = b.communicate()[1]
        assert b.returncode == 0, err
    # the kernels are not compiled: their code is an empty symbol
    names = subprocess.run(["nm", "-u", *objs[1:]], check=True, capture_output=True, text=True).stdout.split()
    empty = sorted({f"-Wl,--defsym={x}=0" for x in names if x.startswith("__hip_fatbin")})
    subprocess.run([CLANG, "-O1", "-g", "-std=c++17", "-fsanitize=address,undefined", "-fno-sanitize-recover=all",
                    "-fno-omit-frame-pointer", "-I", os.path.join(ROOT, "include"),
                    os.path.join(ROOT, "tests", "sanitize", "extend_driver.cpp"), *objs, *empty, "-L/opt/rocm/lib",
                    "-lamdhip64", "-Wl,-rpath,/opt/rocm/lib", "-o", str(exe)], check=True, capture_output=True, text=True)
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=1:verify_asan_link_order=0", UBSAN_OPTIONS="print_stacktrace=1")
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=300, env=env)
    assert r.returncode == 0, r.stdout + r.stderr
    assert "extend driver ok" in r.stdout
    assert "Sanitizer" not in r.stderr and "runtime error" not in r.stderr, r.stderr
