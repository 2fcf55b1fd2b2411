"""Sizes that the random cases of test_layers_host do not reach (tests/layers_shapes.cpp):
lookups with several vectors per lane, and the compare-all sort on tables of about 2^19
rows, run on the CPU under AddressSanitizer."""
import os
import subprocess

import pytest

from tests.test_layers_host import CLANG, ROOT

BF16, F32 = 0, 1


@pytest.fixture(scope="module")
def prog(tmp_path_factory):
    if not os.path.exists(CLANG):
        pytest.skip("clang++ not found")
    exe = str(tmp_path_factory.mktemp("layers") / "layers_shapes")
    subprocess.run([CLANG, "-x", "c++", "-std=c++17", "-O2", "-g", "-ffp-contract=off", "-w",
                    "-fsanitize=address", "-I", os.path.join(ROOT, "tests", "host_gpu"),
                    "-I", os.path.join(ROOT, "include"),
                    "-I", os.path.join(ROOT, "gradient_sync_zero_amd", "layers"),
                    os.path.join(ROOT, "tests", "layers_shapes.cpp"), "-o", exe],
                   check=True, capture_output=True)
    return exe


def run(prog, *args):
    r = subprocess.run([prog, *map(str, args)], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, (args, r.stdout[-2000:], r.stderr[-2000:])


# two vectors a lane from 2^21 in the call on, four from 2^22 on; rows of up to 128
# vectors side by side, longer ones in pieces
@pytest.mark.parametrize("n,dim", [(2_200_003, 1), (4_200_003, 1), (1_100_003, 9), (33_001, 1016), (16_401, 1030),
                                   (16_503, 2060), (5601, 6150), (2111, 8200)])
def test_lookup_of_several_vectors_a_lane(prog, n, dim):
    vectors = -(-dim // 8)
    assert n * vectors >= 1 << 21
    run(prog, "lookup", n, 97, dim, BF16 if n % 2 else F32, F32 if dim % 2 else BF16, 0, n)


@pytest.mark.parametrize("rows", [(1 << 19) - 1, 1 << 19, 600_001])
@pytest.mark.parametrize("n", [129, 700, 8192])
def test_grad_of_some_tokens_on_tall_tables(prog, rows, n):
    for ids in range(3):
        run(prog, "grad", n, rows, 2, ids % 2, ids, n == 700, rows + n)
