"""The launchers of the attention-side operators on the host alone, against a faked
HIP runtime that records every launch (tests/host/launch_limits.cpp): no grid of
2^32 threads or more, no workgroups for tokens that cannot exist."""
import os
import re
import subprocess
from concurrent.futures import ThreadPoolExecutor

import pytest

from tests.test_host_hardening import CLANG, HIPCC, ROOT, SAN


def test_launches_keep_to_the_limits(tmp_path):
    if not (os.path.exists(HIPCC) and os.path.exists(CLANG)):
        pytest.skip("hipcc / clang++ not available")
    csrc = os.path.join(ROOT, "activation_sparse_ffn_amd", "csrc")
    srcs = [os.path.join(csrc, f) for f in ("attn_capi.cpp", "rope.hip", "kvcache.hip", "cache_attention.hip")]
    srcs.append(os.path.join(ROOT, "tests", "host", "launch_limits.cpp"))

    def compiled(src):
        obj = str(tmp_path / (os.path.basename(src) + ".o"))
        r = subprocess.run([HIPCC, "-x", "hip", "--cuda-host-only", "-std=c++17", "-O1", "-g", "-w", *SAN,
                            "-I", os.path.join(ROOT, "include"), "-I", csrc, "-c", src, "-o", obj],
                           capture_output=True, text=True)
        assert r.returncode == 0, r.stderr[-3000:]
        return obj

    with ThreadPoolExecutor(4) as ex:
        objs = list(ex.map(compiled, srcs))
    # the host objects name device code objects that are not built here
    undef = subprocess.run(["nm", "-u", *objs], capture_output=True, text=True, check=True).stdout
    fatbins = sorted(set(re.findall(r"\b(__hip_fatbin\w*)", undef)))
    exe = str(tmp_path / "launch_limits")
    r = subprocess.run([CLANG, "-fsanitize=address,undefined", "-g", *objs, "-o", exe, "-lpthread",
                        *[f"-Wl,--defsym,{f}=fake_fatbin" for f in fatbins]], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-3000:]
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=1", UBSAN_OPTIONS="print_stacktrace=1:halt_on_error=1")
    r = subprocess.run([exe], capture_output=True, text=True, env=env, timeout=120)
    assert r.returncode == 0, r.stdout[-4000:] + r.stderr[-4000:]
    assert "launch checks passed" in r.stdout
