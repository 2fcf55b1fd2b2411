"""The orthogonalising update's and the relative position bias's entry points and kernels run on
the CPU, one fiber per work-item, in buffers of exactly the documented sizes under AddressSanitizer
(tests/muon_host.cpp, tests/relpos_host.cpp), against a plain reference."""
import concurrent.futures
import os
import subprocess

import pytest

from oracle import relpos
from tests.test_layers_host import CLANG, ROOT


def build(tmp_path_factory, name, *include):
    if not os.path.exists(CLANG):
        pytest.skip("clang++ not found")
    exe = str(tmp_path_factory.mktemp(name) / name)
    subprocess.run([CLANG, "-x", "c++", "-std=c++17", "-O2", "-g", "-mf16c", "-ffp-contract=off", "-w", "-fsanitize=address",
                    *[a for d in include for a in ("-I", os.path.join(ROOT, d))],
                    os.path.join(ROOT, "tests", name + ".cpp"), "-o", exe], check=True, capture_output=True)
    return exe


@pytest.fixture(scope="module")
def muon(tmp_path_factory):
    return build(tmp_path_factory, "muon_host", "tests/host_matrix", "tests/host_gpu", "include", "gradient_sync_zero_amd/optim",
                 "gradient_sync_zero_amd/csrc")


@pytest.fixture(scope="module")
def product(tmp_path_factory):
    return build(tmp_path_factory, "product_host", "tests/host_matrix", "tests/host_gpu", "include", "gradient_sync_zero_amd/optim",
                 "gradient_sync_zero_amd/csrc")


@pytest.fixture(scope="module")
def relpos_host(tmp_path_factory):
    return build(tmp_path_factory, "relpos_host", "tests/host_matrix", "tests/host_gpu", "include", "gradient_sync_zero_amd/layers",
                 "gradient_sync_zero_amd/csrc")


def all_pass(exe, cases):
    def run(args):
        r = subprocess.run([exe, *map(str, args)], capture_output=True, text=True, timeout=600)
        return (args, r.returncode, r.stdout[-2000:], r.stderr[-2000:])

    with concurrent.futures.ThreadPoolExecutor(4) as pool:
        bad = [x for x in pool.map(run, cases) if x[1] != 0]
    assert not bad, bad[:2]


@pytest.mark.parametrize("form", [0, 1, 2])
def test_products(product, form):
    """Every tile size, plain and turned operands, symmetric results, tiles that reach past the result,
    and tiles cut along k."""
    # parts, split, turned left, turned right, symmetric, M, N, K
    all_pass(product, [(form, *c) for c in (
        (1, 0, 0, 0, 0, 192, 320, 128), (1, 0, 0, 1, 0, 320, 192, 192), (1, 0, 1, 1, 0, 64, 256, 64), (1, 0, 1, 1, 1, 320, 320, 64),
        (1, 0, 0, 0, 1, 320, 320, 128), (3, 2, 0, 1, 0, 192, 320, 448), (2, 99, 1, 1, 1, 192, 192, 320), (5, 1, 0, 0, 1, 320, 320, 320))])


# count, rows, cols, type (0 bf16, 1 fp32), steps, seed: in one block (both orientations, and its
# limits), in panels, as products
@pytest.mark.parametrize("case", [(1, 1, 1, 1, 5, 1), (2, 5, 9, 0, 5, 2), (1, 9, 5, 1, 3, 3), (2, 130, 40, 1, 2, 4), (1, 33, 300, 0, 2, 5),
                                  (1, 129, 200, 1, 2, 6), (1, 200, 129, 0, 2, 7), (3, 1, 64, 1, 5, 8), (1, 64, 1, 0, 5, 9),
                                  (1, 128, 128, 1, 2, 10), (1, 128, 256, 0, 2, 11), (1, 256, 128, 1, 2, 12), (2, 97, 33, 1, 2, 13),
                                  (1, 128, 257, 1, 2, 14), (2, 700, 100, 0, 2, 15), (3, 20, 1500, 1, 3, 16), (1, 1, 3000, 0, 5, 17), (1, 300, 1, 1, 5, 18), (1, 130, 1100, 1, 3, 19), (1, 1100, 130, 1, 2, 20)])
def test_orthogonalize(muon, case):
    all_pass(muon, [case])


@pytest.mark.parametrize("case", [(1, 7, 5, "step", 1, 1), (3, 20, 33, "step", 0, 2), (2, 140, 30, "step", 1, 3), (2, 300, 128, "step", 1, 4), (1, 130, 200, "step", 0, 5)])
def test_update(muon, case):
    all_pass(muon, [case])


@pytest.mark.parametrize("op", ["bias", "grad"])
def test_relpos(relpos_host, op):
    shapes = [(2, 3, 17, 33, 8, 20, 1), (3, 2, 1, 131, 32, 128, 0), (1, 2, 70, 90, 10, 7, 1), (1, 1, 300, 9, 32, 128, 1),
              (1, 1, 40, 2100, 54, 333, 0), (2, 2, 1, 1, 2, 2, 0), (1, 2, 65, 64, 256, 300, 0), (1, 1, 513, 515, 32, 128, 0), (1, 1, 1100, 3, 32, 128, 1)]
    all_pass(relpos_host, [(op, *s, seed) for s in shapes for seed in (1, 2, 3)])


@pytest.mark.parametrize("buckets,far,both", [(32, 128, 1), (32, 128, 0), (8, 20, 1), (54, 333, 1), (2, 2, 0), (4, 2, 1), (5, 3, 0), (256, 300, 1),
                                              (256, 1 << 30, 0), (64, 1 << 20, 1), (16, 4096, 0), (34, 17 * 17, 0)])
def test_borders_are_the_whole_numbers(relpos_host, buckets, far, both):
    r = subprocess.run([relpos_host, "map", str(buckets), str(far), str(both)], capture_output=True, text=True, check=True)
    assert [int(v) for v in r.stdout.split()] == relpos.borders(buckets, far, bool(both))
