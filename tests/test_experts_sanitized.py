"""tests/test_experts_boundary.py against a copy of the library whose host-side validation layer
is built with AddressSanitizer and UndefinedBehaviorSanitizer (host
pass only), as tests/test_sanitized_boundary.py does for the other entry points."""
import os
import subprocess
import sys

import pytest

from ternary_weight_linear_token_amd import build as bw_build

import test_sanitized_boundary as base


def test_experts_boundary_under_host_sanitizers(tmp_path):
    rt = base.asan_runtime()
    if not os.path.exists(bw_build.HIPCC) or rt is None:
        pytest.skip("hipcc or the sanitizer runtime is not installed")
    if not bw_build.is_current():
        bw_build.build()
    san = ["-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fsanitize=undefined",
           "-Xarch_host", "-fno-omit-frame-pointer"]
    flags = [f for f in bw_build.FLAGS if f != "-O3"] + ["-O1", "-g"]
    objs = []
    for src in bw_build.sources():
        if not src.endswith(".hip"):
            continue
        name = os.path.basename(src)
        if name == "api.hip":
            obj = str(tmp_path / (name + ".o"))
            subprocess.run([bw_build.HIPCC] + flags + san + ["-c", src, "-o", obj], check=True,
                           capture_output=True)
        else:
            obj = os.path.join(bw_build.BUILD_DIR, name + ".o")
        objs.append(obj)
    lib = str(tmp_path / "libbitnet_w2a8_san.so")
    subprocess.run([bw_build.HIPCC, f"--offload-arch={bw_build.ARCH}", "-shared", "-fPIC"] + san +
                   ["-o", lib] + objs, check=True, capture_output=True)
    env = dict(os.environ, BITNET_LIBRARY=lib, LD_PRELOAD=rt,
               ASAN_OPTIONS="detect_leaks=0:halt_on_error=1:abort_on_error=1",
               UBSAN_OPTIONS="halt_on_error=1:print_stacktrace=1")
    res = subprocess.run([sys.executable, "-m", "pytest", "-q", "-p", "no:cacheprovider",
                          os.path.join(base.ROOT, "tests", "test_experts_boundary.py")],
                         cwd=base.ROOT, env=env, capture_output=True, text=True, timeout=600)
    assert res.returncode == 0, res.stdout[-3000:] + res.stderr[-3000:]
    assert "passed" in res.stdout
