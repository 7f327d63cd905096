"""The host-side checks and launch plans of a serving loop's other operators under
AddressSanitizer and UBSan, as tests/test_abi_sanitized.py does it for the other entry points:
the host half of the same build, and tests/abi_serve_sanitized_run.py in a child process.  No
GPU is needed."""
import os
import subprocess
import sys

import pytest

from test_abi_sanitized import CSRC, HIPCC, ROOT, _runtime

RUN = os.path.join(ROOT, "tests", "abi_serve_sanitized_run.py")


def _run(lib, env):
    r = subprocess.run([sys.executable, RUN, lib], env=env, capture_output=True, text=True,
                       timeout=600)
    return r.returncode, r.stdout.strip().splitlines(), r.stderr


def test_serving_checks_run_clean_under_sanitizers(tmp_path):
    rt = _runtime()
    if not os.path.exists(HIPCC) or rt is None:
        pytest.skip("hipcc or clang's sanitizer runtime is not installed")
    lib = str(tmp_path / "libsvd_hostsan.so")
    san = []
    for flag in ("-fsanitize=address", "-fsanitize=undefined", "-fno-sanitize-recover=all",
                 "-fno-omit-frame-pointer"):
        san += ["-Xarch_host", flag]
    subprocess.run([HIPCC, "--offload-arch=gfx950", "-O1", "-g", "-std=c++17", "-fPIC", "-shared",
                    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops", "-fno-fast-math",
                    "-I", os.path.join(ROOT, "include"), "-I", CSRC] + san +
                   ["-shared-libsan", "-o", lib, os.path.join(CSRC, "svd_api.hip"),
                    os.path.join(CSRC, "svd_noalloc.hip")], check=True, capture_output=True)
    env = dict(os.environ, LD_PRELOAD=rt, ASAN_OPTIONS="detect_leaks=0:abort_on_error=1",
               UBSAN_OPTIONS="print_stacktrace=1:halt_on_error=1")
    rc, out, err = _run(lib, env)
    assert rc == 0, err[-4000:]
    product = os.path.join(ROOT, "lossless_draft_verification_verifier_amd", "libsvd.so")
    rc0, out0, err0 = _run(product, dict(os.environ))
    assert rc0 == 0, err0[-4000:]
    assert out[-1] == out0[-1]
