"""The condition under which a kernel may hand registers from one warpgroup to others
(setmaxnreg): the shares add up to at most what its launch allocates, which a compiler
decides. A warpgroup that asks for more would wait for good, so the library looks at the
compiled kernel before it launches it."""

import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def fits(tmp_path_factory):
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(nvcc):
        pytest.skip("nvcc not available")
    exe = str(tmp_path_factory.mktemp("split") / "check")
    subprocess.run([nvcc, "-std=c++17", "-O1", "-gencode", "arch=compute_100a,code=sm_100a",
                    os.path.join(ROOT, "tests", "register_split_check.cu"), "-o", exe],
                   check=True, capture_output=True)

    def run(rows):
        text = "".join("%d %d %d %d\n" % r for r in rows)
        out = subprocess.run([exe], input=text, check=True, capture_output=True, text=True)
        return [v == "1" for v in out.stdout.split()]

    return run


def test_shares_are_within_the_launch(fits):
    rows = [(few, many, groups, regs) for few in (24, 72, 80) for many in (168, 216, 224)
            for groups in (1, 2) for regs in range(96, 256)]
    for row, ok in zip(rows, fits(rows)):
        few, many, groups, regs = row
        allocated = -(-regs // 8) * 8          # a warp's registers come in steps of 8 a thread
        assert ok == (few * 128 + many * groups * 128 <= allocated * 128 * (1 + groups)), row


def test_the_splits_in_use_refuse_fewer_registers(fits):
    # 72 for one warpgroup, 216 for two: a launch with 161 to 168 a thread
    assert fits([(72, 216, 2, r) for r in (168, 161, 160, 156, 128)]) == [True, True, False,
                                                                         False, False]
    assert fits([(0, 0, 0, 32)]) == [True]     # no hand-over


def test_every_kernel_that_hands_registers_over_is_looked_at():
    """Each source with a hand-over passes its split to the check before the launch."""
    csrc = os.path.join(ROOT, "sparse_moe_transformer_gemm_b200", "csrc")
    users = 0
    for name in sorted(os.listdir(csrc)):
        text = open(os.path.join(csrc, name)).read()
        if name.endswith(".cu") and "regs_inc<" in text:
            users += 1
            assert "RegSplit REGS = {REGS_FEW, REGS_MANY," in text, name
            assert "allow_smem(" in text and "REGS" in text.split("allow_smem(")[1][:160], name
    assert users == 2
