"""layer_decode's gate / up claims, on a CPU model that runs the kernel's own arithmetic
(csrc/decode_chunks.h): whatever number of the grid's blocks is resident, and in whatever order
their waves move, every pair is done once and no wave is left waiting."""
import ctypes
import os
import shutil
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
pytestmark = pytest.mark.skipif(shutil.which("g++") is None, reason="needs g++")


@pytest.fixture(scope="module")
def model(tmp_path_factory):
    so = str(tmp_path_factory.mktemp("claims") / "claims.so")
    subprocess.run(["g++", "-O2", "-std=c++17", "-Wall", "-shared", "-fPIC", os.path.join(HERE, "claims_model.cpp"),
                    "-o", so], check=True)
    lib = ctypes.CDLL(so)
    lib.claims_run.argtypes = [ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.c_uint64, ctypes.c_int]
    return lib


RESIDENT = (1, 2, 3, 4, 8, 16, 20, 24, 64)


def test_every_number_of_pairs_on_a_full_grid(model):
    """Distinct experts times F / 32, F a multiple of 128: all multiples of 4 up to where chunks
    have grown to their four pairs for good."""
    for pairs in range(4, 2600, 4):
        for i, resident in enumerate(RESIDENT):
            assert model.claims_run(pairs, 256, resident, pairs + i, 0) == 0, (pairs, resident)


def test_other_grids_and_the_largest(model):
    for grid in (1, 2, 7, 8, 16, 31, 32, 33, 100, 255, 304):
        for pairs in (4, 12, 20, 28, 52, 100, 224, 560, 656, 1312, 4100):
            for resident in (1, 2, 5, 16, 33, grid):
                if resident <= grid:
                    assert model.claims_run(pairs, grid, resident, 3, 0) == 0, (pairs, grid, resident)
    for pairs in (64 * 224, 63 * 224, 61 * 220):
        for resident in (1, 3, 32):
            assert model.claims_run(pairs, 256, resident, 1, 0) == 0, (pairs, resident)


def test_the_model_shows_a_tile_that_nobody_hands_on(model):
    """Numbers for pairs that a short last chunk does not have leave a block waiting, once few
    blocks are resident: the model must find that, or the tests above say nothing."""
    for pairs in (560, 656, 1280, 1312, 1088):
        assert model.claims_chunk(pairs, 256) == 3 and pairs % 3
        assert model.claims_run(pairs, 256, 1, 1, 1) == 1, pairs
        assert model.claims_run(pairs, 256, 4, 1, 1) == 1, pairs
    assert model.claims_run(1536, 256, 1, 1, 1) == 0  # no place over
