"""The host-side checks and launch plans of a serving loop's other operators under
AddressSanitizer and UBSan, as tests/test_abi_sanitized.py does it for the other entry points,
and tests/abi_serve_sanitized_run.py in a child process.  Only the host's half is built: no
kernel is launched, and an empty object stands in for the device's code.  No GPU is needed."""
import os
import re
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
    objects = []
    for name in ("svd_api", "svd_noalloc"):
        objects.append(str(tmp_path / (name + ".o")))
        subprocess.run([HIPCC, "--offload-arch=gfx950", "--offload-host-only", "-cuid=" + name,
                        "-O1", "-g", "-std=c++17", "-fPIC", "-c", "-fno-fast-math",
                        "-I", os.path.join(ROOT, "include"), "-I", CSRC] + san +
                       ["-o", objects[-1], os.path.join(CSRC, name + ".hip")],
                       check=True, capture_output=True)
    names = subprocess.run(["nm", "-u"] + objects, check=True, capture_output=True, text=True).stdout
    nodev = tmp_path / "nodev.c"
    nodev.write_text("".join("const char %s[4096] __attribute__((aligned(4096)));\n" % n
                             for n in re.findall(r"\b__hip_fatbin_\w+", names)))
    objects.append(str(tmp_path / "nodev.o"))
    subprocess.run(["gcc", "-c", "-fPIC", "-o", objects[-1], str(nodev)], check=True)
    rocm = os.path.dirname(os.path.dirname(HIPCC))
    subprocess.run([os.path.join(rocm, "lib", "llvm", "bin", "clang++"), "-shared",
                    "-fsanitize=address", "-fsanitize=undefined", "-shared-libsan", "-o", lib] +
                   objects + ["-L", os.path.join(rocm, "lib"), "-lamdhip64"],
                   check=True, capture_output=True)
    env = dict(os.environ, LD_PRELOAD=rt, ASAN_OPTIONS="detect_leaks=0:abort_on_error=1",
               UBSAN_OPTIONS="print_stacktrace=1:halt_on_error=1")
    rc, out, err = _run(lib, env)
    assert rc == 0, err[-4000:]
    product = os.path.join(ROOT, "lossless_draft_verification_verifier_amd", "libsvd.so")
    rc0, out0, err0 = _run(product, dict(os.environ))
    assert rc0 == 0, err0[-4000:]
    assert out[-1] == out0[-1]
