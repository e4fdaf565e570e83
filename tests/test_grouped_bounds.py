"""What the grouped products may read, on the host: tests/host/grouped_bounds.hip replays the loads of
their launches against their operands (CPU only; the kernels are not compiled)."""
import os
import random
import shutil
import subprocess

import pytest

from routing_dispatch_expert_logits_amd import build as libbuild

HOST = os.path.join(os.path.dirname(os.path.abspath(__file__)), "host")

# R, K, N and the offsets
CASES = [(1, 64, 64, [0, 1]), (3, 257, 131, [0, 0, 0, 3]), (14, 8, 8, [2, 7, 7, 10]), (258, 128, 96, [0, 64, 65, 65, 195, 258]),
         (264, 72, 264, [0, 257]), (40, 72, 136, [-7, 11, 30, 999]), (30, 40, 24, [20, 5, 40]), (1 << 28, 8, 16, [0, 1 << 28]),
         (1 << 28, 1, 8, [5, 1 << 27, (1 << 28) - 1]), (40, 1 << 17, 24, [0, 17, 40]), (40, 24, 1 << 21, [0, 17, 40]),
         (4096, 2048, 768, list(range(0, 4097, 32))), (32768, 2048, 768, list(range(0, 32769, 256))),
         (62580, 7168, 2048, list(range(0, 62581, 1956))[:32] + [62580]), (2048, 1024, 4096, list(range(0, 2049, 2)))]


def spread_cases(n):
    r = random.Random(6)
    size = lambda hi: max(1, int(2 ** r.uniform(0, hi)) // r.choice((1, 8, 64)) * r.choice((1, 8, 64)))  # noqa: E731
    cases = []
    for _ in range(n):
        R, E = size(15), min(1024, size(10))
        cases.append((R, size(13), size(13), sorted(r.randint(0, R) for _ in range(E + 1))))
    return cases


@pytest.fixture(scope="module")
def bounds(tmp_path_factory):
    if not os.path.exists(libbuild.HIPCC) or not shutil.which("g++"):
        pytest.skip("no compilers")
    d = tmp_path_factory.mktemp("bounds")
    objs = [str(d / "bounds.o"), str(d / "no_hip.o")]
    for cmd in ([libbuild.HIPCC, "--offload-host-only", "-x", "hip", "-O1", "-std=c++17", "-I",
                 os.path.join(libbuild.ROOT, "include"), "-I", libbuild.CSRC, "-c",
                 os.path.join(HOST, "grouped_bounds.hip"), "-o", objs[0]],
                ["gcc", "-c", os.path.join(HOST, "no_hip.c"), "-o", objs[1]],
                # no device code is linked: its symbol stays unresolved, and nothing reads it
                ["g++", "-no-pie", "-Wl,--unresolved-symbols=ignore-all", *objs, "-o", str(d / "bounds")]):
        r = subprocess.run(cmd, capture_output=True, text=True)
        assert r.returncode == 0, r.stderr[-3000:]

    def run(dtype, case):
        R, K, N, off = case
        r = subprocess.run([str(d / "bounds"), dtype, *map(str, (R, K, N, len(off) - 1, *off))], capture_output=True, text=True,
                           timeout=300)
        assert r.returncode == 0, (case, r.stderr[-4000:])
        return tuple(map(int, r.stdout.split()))

    return run


@pytest.mark.parametrize("dtype", ("bf16", "f32", "int8"))
def test_loads_stay_in_their_operands(bounds, dtype):
    for case in CASES + spread_cases(200):
        bounds(dtype, case)


def test_every_tile_height_is_reached(bounds):
    """What the replay covers: forward products and dx on 64, 128 and 320 rows, dw on 64, 128 and 256."""
    seen = [set() for _ in range(4)]
    for case in CASES + spread_cases(200):
        for s, h in zip(seen, bounds("bf16", case)):
            s.add(h)
    assert all(s == {64, 128, 320} for s in seen[:3]) and seen[3] == {64, 128, 256}, seen
