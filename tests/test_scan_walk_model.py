"""Which rows, saved states and span totals the selective scan's kernels touch, run on the CPU
(tests/protocol_model/scan_walk_model.cpp, compiled with the kernels' own integer code): for random
sizes and offsets, those that descend or lie outside the rows included, no index leaves its array
and every walk ends; for ascending offsets nothing is read before it is written and every row is
walked once."""
import os
import shutil
import subprocess

import pytest

SRC = os.path.join(os.path.dirname(os.path.abspath(__file__)), "protocol_model", "scan_walk_model.cpp")


@pytest.fixture(scope="module")
def model(tmp_path_factory):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("g++ not available")
    exe = str(tmp_path_factory.mktemp("scan_walk") / "model")
    subprocess.run([gxx, "-O1", "-std=c++17", "-Wall", "-Werror", "-fsanitize=address,undefined", SRC, "-o", exe], check=True)
    return exe


@pytest.mark.parametrize("seed", [1, 2, 3])
def test_walks_stay_inside_the_arrays(model, seed):
    env = dict(os.environ, ASAN_OPTIONS="verify_asan_link_order=0:detect_leaks=0")
    r = subprocess.run([model, "seed=%d" % seed, "cases=20000"], capture_output=True, text=True, timeout=120, env=env)
    assert r.returncode == 0 and "result ok=1 cases=20000" in r.stdout, r.stdout + r.stderr[-2000:]
    assert int(r.stdout.split("joins=")[1]) > 10000
