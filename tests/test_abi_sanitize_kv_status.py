"""The exact statuses of the key/value cache's entry points under AddressSanitizer and
UndefinedBehaviorSanitizer: as test_abi_sanitize_kv.py, with a workspace given, by
tests/abi_sanitize_kv_status_driver.c.  Nothing is launched."""
import concurrent.futures
import os
import shutil
import subprocess

import pytest

from test_abi_sanitize import B, HERE, SAN_HOST

INSTRUMENTED = ["nvfp4_api.hip", "kv_cache.hip", "kv_attention.hip"]


def test_kv_statuses_under_address_and_ub_sanitizers(tmp_path):
    try:
        hipcc = B.hipcc()
    except RuntimeError:
        pytest.skip("hipcc not found")
    clang = os.path.join(os.path.dirname(os.path.realpath(hipcc)), "..", "lib", "llvm", "bin", "clang")
    if not os.path.exists(clang):
        clang = shutil.which("clang") or "/opt/rocm/lib/llvm/bin/clang"
    objects = [os.path.join(B.BUILD, s.replace(".hip", ".o")) for s in B.SOURCES if s not in INSTRUMENTED]
    if not all(os.path.exists(o) for o in objects):
        pytest.skip("the library's kernel objects are not built (run __graft_entry__.build())")

    def run(cmd):
        r = subprocess.run(cmd, capture_output=True, text=True)
        assert r.returncode == 0, r.stderr[-3000:]

    def compile_one(s):
        obj = str(tmp_path / s.replace(".hip", "_san.o"))
        run([hipcc] + B.flags() + SAN_HOST + ["-c", os.path.join(B.CSRC, s), "-o", obj])
        return obj

    with concurrent.futures.ThreadPoolExecutor(max_workers=4) as ex:
        objects += ex.map(compile_one, INSTRUMENTED)
    run([hipcc, f"--offload-arch={B.ARCH}", "-shared", "-fPIC", "-o", str(tmp_path / "libnvfp4_san.so")] + objects)
    exe = str(tmp_path / "abi_sanitize_kv_status")
    run([clang, "-std=c11", "-O1", "-g", "-fsanitize=address,undefined", "-fno-sanitize-recover=all",
         "-fno-omit-frame-pointer", "-Wall", "-Wextra", "-Werror", "-I", B.INCLUDE, "-o", exe,
         os.path.join(HERE, "abi_sanitize_kv_status_driver.c"), "-L", str(tmp_path), "-lnvfp4_san",
         "-Wl,-rpath," + str(tmp_path)])
    # (leak checking off: the HIP runtime keeps allocations until exit)
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=0", UBSAN_OPTIONS="print_stacktrace=1:halt_on_error=1")
    r = subprocess.run([exe], capture_output=True, text=True, env=env, timeout=300)
    assert r.returncode == 0, (r.stdout[-2000:], r.stderr[-4000:])
    assert "ok" in r.stdout.split()
    assert "runtime error" not in r.stderr and "AddressSanitizer" not in r.stderr, r.stderr[-4000:]
