"""The embedding and dropout entry points and their kernels run on the CPU, one
fiber per work-item, in buffers of exactly the documented sizes under
AddressSanitizer (tests/layers_host.cpp): every index a kernel forms is checked
before a GPU sees it, and the results are checked against a plain reference."""
import concurrent.futures
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CLANG = "/opt/rocm/lib/llvm/bin/clang++"


@pytest.fixture(scope="module")
def prog(tmp_path_factory):
    if not os.path.exists(CLANG):
        pytest.skip("clang++ not found")
    exe = str(tmp_path_factory.mktemp("layers") / "layers_host")
    subprocess.run([CLANG, "-x", "c++", "-std=c++17", "-O2", "-g", "-ffp-contract=off", "-w",
                    "-fsanitize=address", "-I", os.path.join(ROOT, "tests", "host_gpu"),
                    "-I", os.path.join(ROOT, "include"),
                    "-I", os.path.join(ROOT, "gradient_sync_zero_amd", "layers"),
                    os.path.join(ROOT, "tests", "layers_host.cpp"), "-o", exe],
                   check=True, capture_output=True)
    return exe


@pytest.mark.parametrize("op", ["dropout", "lookup", "grad"])
def test_random_cases(prog, op):
    def run(seed):
        r = subprocess.run([prog, op, str(seed)], capture_output=True, text=True, timeout=300)
        return (seed, r.returncode, r.stdout[-2000:], r.stderr[-2000:])

    with concurrent.futures.ThreadPoolExecutor(4) as pool:
        bad = [x for x in pool.map(run, range(1, 29)) if x[1] != 0]
    assert not bad, bad[:2]
