"""The embedding and dropout entry points at the limits of their sizes
(tests/layers_limits.cpp): which calls are taken, that no launch holds more than 2^31
work-items, and that blocks which go over more than their own part do it right, the
kernels run on the CPU under AddressSanitizer."""
import concurrent.futures
import os
import subprocess

import pytest

from tests.test_layers_host import CLANG, ROOT


@pytest.fixture(scope="module")
def prog(tmp_path_factory):
    if not os.path.exists(CLANG):
        pytest.skip("clang++ not found")
    exe = str(tmp_path_factory.mktemp("layers") / "layers_limits")
    subprocess.run([CLANG, "-x", "c++", "-std=c++17", "-O2", "-g", "-ffp-contract=off", "-w",
                    "-fsanitize=address", "-I", os.path.join(ROOT, "tests", "host_gpu"),
                    "-I", os.path.join(ROOT, "include"),
                    "-I", os.path.join(ROOT, "gradient_sync_zero_amd", "layers"),
                    os.path.join(ROOT, "tests", "layers_limits.cpp"), "-o", exe],
                   check=True, capture_output=True)
    return exe


def test_calls_at_the_documented_limits(prog):
    r = subprocess.run([prog, "sizes"], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stdout[-3000:] + r.stderr[-2000:]


@pytest.mark.parametrize("op", ["dropout", "lookup", "grad"])
def test_random_cases_in_the_fewest_blocks(prog, op):
    def run(seed):
        r = subprocess.run([prog, op, str(seed)], capture_output=True, text=True, timeout=300)
        return (seed, r.returncode, r.stdout[-2000:], r.stderr[-2000:])

    with concurrent.futures.ThreadPoolExecutor(4) as pool:
        bad = [x for x in pool.map(run, range(1, 11)) if x[1] != 0]
    assert not bad, bad[:2]
