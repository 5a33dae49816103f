"""The host code of the attention-side C entry points built with the address and
undefined-behaviour sanitizers and run without a GPU: tests/host/attention_checks.cpp
calls them with sizes at the ends of their ranges and with launches that fail (the
launchers are faked, tests/host/fake_attention.cpp)."""
import os
import subprocess

import pytest

from tests.test_host_hardening import CLANG, HIPCC, ROOT, SAN


def test_sizes_plans_and_hip_errors_under_sanitizers(tmp_path):
    if not (os.path.exists(HIPCC) and os.path.exists(CLANG)):
        pytest.skip("hipcc / clang++ not available")
    csrc = os.path.join(ROOT, "activation_sparse_ffn_amd", "csrc")
    host = os.path.join(ROOT, "tests", "host")
    objs = []
    for src in (os.path.join(csrc, "attn_capi.cpp"), os.path.join(host, "fake_attention.cpp"),
                os.path.join(host, "attention_checks.cpp")):
        obj = str(tmp_path / (os.path.basename(src) + ".o"))
        r = subprocess.run([HIPCC, "-x", "hip", "--cuda-host-only", "-std=c++17", "-O1", "-g", "-w", *SAN,
                            "-I", os.path.join(ROOT, "include"), "-I", csrc, "-c", src, "-o", obj],
                           capture_output=True, text=True)
        assert r.returncode == 0, r.stderr[-3000:]
        objs.append(obj)
    exe = str(tmp_path / "attention_checks")
    r = subprocess.run([CLANG, "-fsanitize=address,undefined", "-g", *objs, "-o", exe, "-lpthread"],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-3000:]
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=1", UBSAN_OPTIONS="print_stacktrace=1:halt_on_error=1")
    r = subprocess.run([exe], capture_output=True, text=True, env=env, timeout=120)
    assert r.returncode == 0, r.stdout[-4000:] + r.stderr[-4000:]
    assert "host checks passed" in r.stdout
