"""The size computations of the attention entry points (how a call is divided, its workspace) built with
AddressSanitizer and UndefinedBehaviorSanitizer and asked for sizes up to the ends of their
types. No HIP call is made."""
import os
import shutil
import subprocess

import pytest

from test_sanitize_abi_cpu import CLANG, PKG, ROOT, SAN_HOST


@pytest.mark.skipif(shutil.which("hipcc") is None or not os.path.exists(CLANG), reason="needs the ROCm toolchain")
def test_attention_sizes_under_asan_ubsan(tmp_path):
    objs, builds = [os.path.join(PKG, "_build", "gdn_kv_cache.hip.o")], []
    if not os.path.exists(objs[0]):
        pytest.skip("build the library first")
    for name in ("gdn_attn_api", "gdn_attn_prefill", "gdn_attn_decode"):
        out = tmp_path / f"{name}.o"
        objs.append(str(out))
        builds.append(subprocess.Popen(
            ["hipcc", "--offload-arch=gfx950", "-O1", "-g", "-std=c++17", "-fPIC", "-I", os.path.join(ROOT, "include"),
             "-I", os.path.join(PKG, "csrc"), "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops", *SAN_HOST,
             "-c", os.path.join(PKG, "csrc", f"{name}.hip"), "-o", str(out)], stdout=subprocess.PIPE, stderr=subprocess.PIPE, text=True))
    for b in builds:
        err = b.communicate()[1]
        assert b.returncode == 0, err
    exe = tmp_path / "sizes_san"
    subprocess.run([CLANG, "-O1", "-g", "-std=c++17", "-fsanitize=address,undefined", "-fno-sanitize-recover=all",
                    "-fno-omit-frame-pointer", "-I", os.path.join(ROOT, "include"),
                    os.path.join(ROOT, "tests", "sanitize", "attn_sizes_driver.cpp"), *objs, "-L/opt/rocm/lib",
                    "-lamdhip64", "-Wl,-rpath,/opt/rocm/lib", "-o", str(exe)], check=True, capture_output=True, text=True)
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=1:verify_asan_link_order=0", UBSAN_OPTIONS="print_stacktrace=1")
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=300, env=env)
    assert r.returncode == 0, r.stdout + r.stderr
    assert "sizes ok" in r.stdout
    assert "Sanitizer" not in r.stderr and "runtime error" not in r.stderr, r.stderr
