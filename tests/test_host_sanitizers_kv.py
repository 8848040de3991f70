"""The key/value cache's and the epilogue's host code (argument validation, the
attention's plan) under AddressSanitizer and UndefinedBehaviorSanitizer, on the
CPU: their sources are compiled with the sanitizers on the host side only, the
rest comes from the built library, and tests/host_kv_abi_check.cpp drives them
without a GPU."""

import os
import shutil
import subprocess
import tempfile

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
SOURCES = ("api.cpp", "api_kv.cpp", "kv_cache.hip", "kv_attention.hip")


@pytest.mark.slow
@pytest.mark.skipif(shutil.which("hipcc") is None and not os.path.exists("/opt/rocm/bin/hipcc"),
                    reason="needs hipcc")
def test_cache_host_code_under_asan_and_ubsan():
    from bit_weight_only_quantize_amd import build as B
    if not os.path.exists(B.LIB_PATH):
        pytest.skip("libawq355.so not built")
    san = ["-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fsanitize=undefined",
           "-Xarch_host", "-fno-sanitize-recover=all", "-Xarch_host", "-fno-omit-frame-pointer"]
    with tempfile.TemporaryDirectory(prefix="awq355_san_kv_") as tmp:
        procs, objs = [], []
        for src in SOURCES:
            obj = os.path.join(tmp, os.path.splitext(src)[0] + ".o")
            cmd = [B.hipcc(), *B.common_flags(), *san, "-x", "hip", "-c", os.path.join(B.CSRC, src), "-o", obj]
            procs.append((src, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)))
            objs.append(obj)
        drv = os.path.join(tmp, "host_kv_abi_check.o")
        subprocess.run([B.hipcc(), "-std=c++17", *san, "-I", os.path.join(ROOT, "include"), "-c",
                        os.path.join(HERE, "host_kv_abi_check.cpp"), "-o", drv],
                       check=True, capture_output=True, text=True)
        for src, p in procs:
            out, _ = p.communicate(timeout=900)
            assert p.returncode == 0, f"{src}:\n{out}"
        exe = os.path.join(tmp, "host_kv_abi_check")
        link_flags = ["-fno-gpu-sanitize", "-fsanitize=address", "-fsanitize=undefined"]
        link = subprocess.run([B.hipcc(), *link_flags, drv, *objs, B.LIB_PATH, "-o", exe,
                               f"-Wl,-rpath,{os.path.dirname(B.LIB_PATH)}"], capture_output=True, text=True)
        assert link.returncode == 0, link.stdout + link.stderr
        env = dict(os.environ, ASAN_OPTIONS="detect_leaks=0:abort_on_error=1",
                   UBSAN_OPTIONS="print_stacktrace=1:halt_on_error=1")
        res = subprocess.run([exe], capture_output=True, text=True, timeout=300, env=env)
    out = res.stdout + res.stderr
    assert res.returncode == 0, out
    assert "host cache ABI check ok" in out
    assert "runtime error" not in out and "AddressSanitizer" not in out, out
