"""What the dense products may read, on the host: tests/host/dense_bounds.hip replays the loads of
every launch against their operands (CPU only; the kernels are not compiled)."""
import os
import random
import shutil
import subprocess

import pytest

from routing_dispatch_expert_logits_amd import build as libbuild
from tests.dense_sizes import CUT_BACKWARD, CUT_FORWARD

HOST = os.path.join(os.path.dirname(os.path.abspath(__file__)), "host")

# whole tiles, ragged ones, single rows; column operands that end at a page's end after a cut
SIZES = [(1, 64, 64), (17, 72, 56), (33, 333, 77), (130, 515, 260), (256, 256, 256), (300, 64, 1000), (1000, 1032, 72),
         (1021, 1416, 2120), (3800, 4072, 4000), (515, 1001, 1777), (4096, 2048, 8192), (4096, 4096, 4096),
         (8192, 2048, 7168), (8192, 7208, 2048), (131072, 520, 32768), (100, 7168, 1000), (300000, 8, 16),
         # the largest row count and widths
         (1 << 28, 1, 8), (1 << 28, 8, 32), (40, 1 << 21, 24), (40, 24, 1 << 21), (4096, 1 << 21, 40), (1 << 12, 1 << 20, 1 << 13)]


def spread_sizes(n):
    r = random.Random(4)
    size = lambda hi: max(1, int(2 ** r.uniform(0, hi)) // r.choice((1, 8, 64)) * r.choice((1, 8, 64)))  # noqa: E731
    return [(size(14), size(13), size(13)) for _ in range(n)]


@pytest.fixture(scope="module")
def bounds(tmp_path_factory):
    if not os.path.exists(libbuild.HIPCC) or not shutil.which("g++"):
        pytest.skip("no compilers")
    d = tmp_path_factory.mktemp("bounds")
    objs = [str(d / "bounds.o"), str(d / "no_hip.o")]
    for cmd in ([libbuild.HIPCC, "--offload-host-only", "-x", "hip", "-O1", "-std=c++17", "-I",
                 os.path.join(libbuild.ROOT, "include"), "-I", libbuild.CSRC, "-c",
                 os.path.join(HOST, "dense_bounds.hip"), "-o", objs[0]],
                ["gcc", "-c", os.path.join(HOST, "no_hip.c"), "-o", objs[1]],
                # no device code is linked: its symbol stays unresolved, and nothing reads it
                ["g++", "-no-pie", "-Wl,--unresolved-symbols=ignore-all", *objs, "-o", str(d / "bounds")]):
        r = subprocess.run(cmd, capture_output=True, text=True)
        assert r.returncode == 0, r.stderr[-3000:]

    def run(dtype, terms, sizes):
        r = subprocess.run([str(d / "bounds"), dtype, str(terms), *(str(v) for s in sizes for v in s)],
                           capture_output=True, text=True, timeout=300)
        assert r.returncode == 0, r.stderr[-4000:]
        cuts = [tuple(map(int, line.split())) for line in r.stdout.splitlines()]
        assert len(cuts) == len(sizes)
        return cuts

    return run


@pytest.mark.parametrize("dtype,terms", (("bf16", 1), ("bf16", 2), ("bf16", 3), ("f32", 1)))
def test_loads_stay_in_their_operands(bounds, dtype, terms):
    bounds(dtype, terms, SIZES + CUT_BACKWARD + CUT_FORWARD + spread_sizes(300))


@pytest.mark.parametrize("terms", (1, 2, 3))
def test_cut_sizes_are_cut(bounds, terms):
    """Both backward products, gated and linear, and the linear forward product take a second launch."""
    for c, (T, K, N) in zip(bounds("bf16", terms, CUT_BACKWARD), CUT_BACKWARD):
        assert all(0 < v < K for v in c[2:]), (T, K, N, c)
    for c, (T, K, N) in zip(bounds("bf16", terms, CUT_FORWARD), CUT_FORWARD):
        assert 0 < c[1] < N, (T, K, N, c)
