"""The host code of the attention entry points built with AddressSanitizer and
UndefinedBehaviorSanitizer and driven through their refusals by a standalone program, as
tests/test_sanitize_abi_cpu.py does for the recurrence. No HIP call is made."""
import os
import shutil
import subprocess

import pytest

from test_sanitize_abi_cpu import CLANG, PKG, ROOT, SAN_HOST


@pytest.mark.skipif(shutil.which("hipcc") is None or not os.path.exists(CLANG), reason="needs the ROCm toolchain")
def test_attention_validation_under_asan_ubsan(tmp_path):
    objs = [os.path.join(PKG, "_build", f"{name}.hip.o") for name in ("gdn_kv_cache", "gdn_attn_prefill", "gdn_attn_decode")]
    if not all(os.path.exists(o) for o in objs):
        pytest.skip("build the library first")
    api, exe = tmp_path / "api_san.o", tmp_path / "attn_san"
    subprocess.run(["hipcc", "--offload-arch=gfx950", "-O1", "-g", "-std=c++17", "-fPIC", "-I", os.path.join(ROOT, "include"),
                    "-I", os.path.join(PKG, "csrc"), "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops", *SAN_HOST,
                    "-c", os.path.join(PKG, "csrc", "gdn_attn_api.hip"), "-o", str(api)],
                   check=True, capture_output=True, text=True)
    subprocess.run([CLANG, "-O1", "-g", "-std=c++17", "-fsanitize=address,undefined", "-fno-sanitize-recover=all",
                    "-fno-omit-frame-pointer", "-I", os.path.join(ROOT, "include"),
                    os.path.join(ROOT, "tests", "sanitize", "attn_driver.cpp"), str(api), *objs, "-L/opt/rocm/lib",
                    "-lamdhip64", "-Wl,-rpath,/opt/rocm/lib", "-o", str(exe)], check=True, capture_output=True, text=True)
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=1:verify_asan_link_order=0", UBSAN_OPTIONS="print_stacktrace=1")
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=300, env=env)
    assert r.returncode == 0, r.stdout + r.stderr
    assert "attention driver ok" in r.stdout
    assert "Sanitizer" not in r.stderr and "runtime error" not in r.stderr, r.stderr
