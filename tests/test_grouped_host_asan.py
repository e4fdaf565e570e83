"""The grouped and integer calls' host code under AddressSanitizer (CPU only): their sources compiled for
the host alone, linked with a C driver of their host paths and stand-ins for the runtime."""
import os
import subprocess
from concurrent.futures import ThreadPoolExecutor

import pytest

from routing_dispatch_expert_logits_amd import build as libbuild

HERE = os.path.dirname(os.path.abspath(__file__))
SOURCES = ("grouped_api", "grouped_mm", "grouped_decode", "int8", "dense_grad")
# host-only instrumentation: -Xarch_host in front of each sanitizer flag
ASAN = ["-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fno-omit-frame-pointer"]


@pytest.mark.skipif(not os.path.exists(libbuild.HIPCC), reason="hipcc not available")
def test_grouped_host_code_under_asan(tmp_path):
    include = ["-I", os.path.join(libbuild.ROOT, "include"), "-I", libbuild.CSRC]
    objs, cmds = [], []
    for name in SOURCES:
        objs.append(str(tmp_path / (name + ".o")))
        cmds.append([libbuild.HIPCC, "--offload-host-only", "-x", "hip", "-O1", "-g", "-std=c++17", *include, *ASAN, "-c",
                     os.path.join(libbuild.CSRC, name + ".hip"), "-o", objs[-1]])
    for path in (os.path.join(HERE, "asan", "grouped_host_driver.c"), os.path.join(HERE, "host", "no_hip.c")):
        objs.append(str(tmp_path / (os.path.basename(path) + ".o")))
        cmds.append([libbuild.HIPCC, "-x", "c", *include, *ASAN, "-c", path, "-o", objs[-1]])
    with ThreadPoolExecutor(8) as pool:
        for r in pool.map(lambda c: subprocess.run(c, capture_output=True, text=True), cmds):
            assert r.returncode == 0, r.stderr[-3000:]
    exe = str(tmp_path / "grouped_host_driver")
    # no device code is linked: its symbols stay unresolved, and nothing reads them
    r = subprocess.run([libbuild.HIPCC, *ASAN, "-no-pie", "-Wl,--unresolved-symbols=ignore-all", *objs, "-o", exe],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-3000:]
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=0:abort_on_error=0:halt_on_error=1")
    r = subprocess.run([exe], capture_output=True, text=True, env=env, timeout=300)
    assert r.returncode == 0 and "all checks passed" in r.stdout, (r.stdout[-2000:], r.stderr[-4000:])
