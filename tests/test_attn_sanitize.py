"""The attention operators' host code, and the index arithmetic of their kernels
(where tokens lie, which a row sees, how work is divided), under the address and
undefined-behaviour sanitizers, on the CPU."""
import concurrent.futures
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "tensor_sharded_linear_plan_amd", "csrc")
HERE = os.path.join(ROOT, "tests", "sanitize")
HIPCC = "/opt/rocm/bin/hipcc"
CLANG = "/opt/rocm/lib/llvm/bin/clang++"


@pytest.mark.skipif(not (os.path.exists(HIPCC) and os.path.exists(CLANG) and
                         os.path.exists(os.path.join(HERE, "attn_driver.cpp"))), reason="no ROCm")
def test_host_code_and_index_arithmetic_under_sanitizers(tmp_path):
    from tensor_sharded_linear_plan_amd import build
    srcs = [(os.path.join(CSRC, s), s) for s in build.ATTN_SOURCES]
    srcs.append((os.path.join(HERE, "attn_driver.cpp"), "attn_driver.cpp"))
    flags = ["-x", "hip", "--offload-arch=gfx950", "-std=c++17", "-O1", "-g",
             "-fno-omit-frame-pointer", "-Xclang", "-target-feature", "-Xclang",
             "-packed-fp32-ops", "-Wno-inline-asm",
             "-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fsanitize=undefined",
             "-Xarch_host", "-fno-sanitize-recover=all",
             "-I" + os.path.join(ROOT, "include"), "-I" + CSRC]

    def run(cmd, **kw):
        r = subprocess.run(cmd, capture_output=True, text=True, **kw)
        assert r.returncode == 0, "%s\n%s%s" % (" ".join(cmd), r.stdout, r.stderr)
        return r

    def compile_one(src):
        obj = str(tmp_path / (os.path.splitext(src[1])[0] + ".o"))
        run([HIPCC] + flags + ["-c", src[0], "-o", obj])
        return obj

    with concurrent.futures.ThreadPoolExecutor(8) as ex:
        objs = list(ex.map(compile_one, srcs))
    exe = str(tmp_path / "attn_driver")
    run([CLANG, "--hip-link", "--offload-arch=gfx950", "-fsanitize=address,undefined", "-o", exe] +
        objs + ["-L/opt/rocm/lib", "-lamdhip64", "-Wl,-rpath,/opt/rocm/lib"])
    r = run([exe], env=dict(os.environ, ASAN_OPTIONS="detect_leaks=0:abort_on_error=0",
                            UBSAN_OPTIONS="halt_on_error=1:print_stacktrace=1"))
    assert "all checks passed" in r.stdout and "runtime error" not in r.stderr
