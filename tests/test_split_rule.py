"""How many slices of K a small block-FP8 product is cut into: the clusters of all its
tiles have to run at once, which a second wave would double the time of."""

import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
# clusters of so many CTAs, one an SM, that a B200 runs at once (as the device reports)
AT_ONCE = {8: 15, 4: 33, 2: 74, 1: 148}


@pytest.fixture(scope="module")
def slices(tmp_path_factory):
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(nvcc):
        pytest.skip("nvcc not available")
    exe = str(tmp_path_factory.mktemp("split") / "check")
    subprocess.run([nvcc, "-std=c++17", "-O1", "-gencode", "arch=compute_100a,code=sm_100a", "-I",
                    os.path.join(ROOT, "include"), os.path.join(ROOT, "tests", "split_check.cu"),
                    "-o", exe], check=True, capture_output=True)

    def run(rows):
        text = "".join("%d %d %d\n" % r for r in rows)
        out = subprocess.run([exe], input=text, check=True, capture_output=True, text=True)
        return [int(v) for v in out.stdout.split()]

    return run


def test_every_cluster_runs_at_once_and_no_fewer_slices_than_fit(slices):
    rows = [(tiles, blocks, 148) for tiles in range(1, 149)
            for blocks in (1, 2, 3, 4, 7, 8, 16, 32, 1024)]
    for (tiles, blocks, _), S in zip(rows, slices(rows)):
        fit = max(n for n, most in AT_ONCE.items() if tiles <= most and n <= blocks)
        assert S == fit, (tiles, blocks, S)


def test_more_tiles_than_sms_are_not_cut_here(slices):
    assert slices([(149, 32, 148), (1 << 33, 32, 148), (100, 32, 96)]) == [0, 0, 0]


def test_fewer_sms(slices):
    assert slices([(12, 32, 64), (13, 32, 64), (33, 32, 64), (16, 32, 64)]) == [4, 4, 1, 4]
