"""The FP8 product's choice of a tile (rotated_bit_amd/csrc/fp8_pick.hpp),
compiled for the host: the limit of a launch."""
import os
import shutil
import subprocess

import pytest

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
