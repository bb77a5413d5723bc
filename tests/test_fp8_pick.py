"""The FP8 product's choice of a tile (rotated_bit_amd/csrc/fp8_pick.hpp),
compiled for the host: the limit of a launch, and that the GPU's cases reach
every tile."""
import itertools
import os
import shutil
import subprocess

import pytest

import test_gpu_fp8_tiles as G

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def pick(tmp_path_factory):
    if shutil.which("g++") is None:
        pytest.skip("g++ not available")
    exe = tmp_path_factory.mktemp("pick") / "fp8_pick"
    build = subprocess.run(["g++", "-std=c++17", "-O2", "-Wall", "-Werror",
                            os.path.join(ROOT, "tests", "native", "fp8_pick.cpp"), "-o", str(exe)],
                           capture_output=True, text=True)
    assert build.returncode == 0, build.stderr[-4000:]

    def run(*args, text=""):
        r = subprocess.run([str(exe), *args], input=text, capture_output=True, text=True,
                           timeout=120)
        assert r.returncode == 0, r.stderr
        return r.stdout.splitlines()

    return run


def test_no_launch_has_more_threads_than_the_hardware_takes(pick):
    # a launch counts its threads in 32 bits: with the tables' costs, and with
    # costs by which only that limit keeps the smallest tiles from being picked
    for line in pick("launches"):
        dt, now, free = line.split()
        assert 0 < int(now) < 2 ** 32, dt
        assert 2 ** 31 < int(free) < 2 ** 32, dt


def test_gpu_cases_run_the_tiles_they_name(pick):
    lines = []
    for case in G.CASES:
        M, N, K, E, grouped = G.call_of(case)
        lines.append(f"{case[0]} {M} {N} {K} {E} {int(grouped)}")
    got = pick(text="\n".join(lines) + "\n")
    assert len(got) == len(G.CASES)
    for case, line in zip(G.CASES, got):
        index, bn, bm = (int(v) for v in line.split()[:3])
        assert (index, f"{bn}x{bm}") == case[1:3], (case, line)
        assert (case[6] * (2 if case[0] == "bf16" else 4) % 16 == 0) == (case[4] == "direct"), case
        # ragged in outputs, more than one of them; the largest tile asks for
        # lines three runs ahead
        assert case[6] % bn and case[6] > bn
        assert case[7] > (640 if bn + bm > 384 else 256)


def test_gpu_cases_leave_no_tile_out(pick):
    every = set()
    for line in pick("tables"):
        dt, n = line.split()
        every |= {(dt, i, f, s) for i, f, s in itertools.product(
            range(int(n)), ("dense", "gather", "sorted"), ("direct", "staged"))}
    assert every == {(c[0], c[1], c[3], c[4]) for c in G.CASES}
