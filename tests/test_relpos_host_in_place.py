"""The relative position bias added to scores in place, on the CPU (tests/relpos_in_place_host.cpp):
the lanes at a row's end load the next row's scores, which another lane writes."""
import pytest

from tests.test_optim_host import all_pass, build


@pytest.fixture(scope="module")
def host(tmp_path_factory):
    return build(tmp_path_factory, "relpos_in_place_host", "tests/host_matrix", "tests/host_gpu", "include", "gradient_sync_zero_amd/layers",
                 "gradient_sync_zero_amd/csrc")


@pytest.mark.parametrize("type", [0, 1])
def test_in_place(host, type):
    shapes = [(2, 3, 17, 33, 8, 20, 1), (3, 2, 1, 131, 32, 128, 0), (1, 2, 70, 90, 10, 7, 1), (1, 1, 300, 9, 32, 128, 1), (1, 1, 40, 2100, 54, 333, 0),
              (2, 2, 1, 1, 2, 2, 0), (1, 2, 65, 64, 256, 300, 0), (1, 1, 40, 515, 32, 128, 0), (1, 1, 1100, 3, 32, 128, 1)]
    all_pass(host, [(*s, type, shift, seed) for s in shapes for seed, shift in enumerate((0, 1, 8, 3))])
