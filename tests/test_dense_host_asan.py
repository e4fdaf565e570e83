"""The dense operators' host code under AddressSanitizer (CPU only): the library's sources with
the host half instrumented (the device code is untouched), linked with a C driver of their host
paths, as tests/test_host_asan.py does for the layer's."""
import os
import subprocess
from concurrent.futures import ThreadPoolExecutor

import pytest

from routing_dispatch_expert_logits_amd import build as libbuild

DRIVER = os.path.join(os.path.dirname(os.path.abspath(__file__)), "asan", "dense_host_driver.c")
# host-only instrumentation: -Xarch_host in front of each sanitizer flag
ASAN = ["-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fno-omit-frame-pointer"]


@pytest.mark.skipif(not os.path.exists(libbuild.HIPCC), reason="hipcc not available")
def test_dense_host_code_under_asan(tmp_path):
    flags = [f for f in libbuild.DEVICE_FLAGS if f != "-O3"] + ["-O1", "-g"]
    objs, cmds = [], []
    for src in libbuild.sources() + [DRIVER]:
        objs.append(str(tmp_path / (os.path.basename(src) + ".o")))
        base = ([libbuild.HIPCC, "-x", "c", "-I", os.path.join(libbuild.ROOT, "include")] if src.endswith(".c")
                else [libbuild.HIPCC, *flags])
        cmds.append(base + ASAN + ["-c", src, "-o", objs[-1]])
    with ThreadPoolExecutor(8) as pool:
        for r in pool.map(lambda c: subprocess.run(c, capture_output=True, text=True), cmds):
            assert r.returncode == 0, r.stderr[-3000:]
    exe = str(tmp_path / "dense_host_driver")
    r = subprocess.run([libbuild.HIPCC, f"--offload-arch={libbuild.ARCH}", *ASAN, *objs, "-o", exe],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-3000:]
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=0:abort_on_error=0:halt_on_error=1")
    r = subprocess.run([exe], capture_output=True, text=True, env=env, timeout=300)
    assert r.returncode == 0 and "all checks passed" in r.stdout, (r.stdout[-2000:], r.stderr[-4000:])
