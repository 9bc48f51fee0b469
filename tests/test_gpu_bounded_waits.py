"""The self-test runs every form of bounded wait that the kernels use: the plain one and
the pipelines' one each run out their limit, and the latter returns at once where
another role has given up. Nothing faults, traps or hangs."""

import pytest
import torch

from sparse_moe_transformer_gemm_b200 import build as moe_build
from sparse_moe_transformer_gemm_b200 import moe
from synthetic import CONFIGS

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("limit_ms", [5, 40])
def test_both_waits_run_out_and_a_raised_flag_ends_one_at_once(limit_ms):
    moe_build.build()
    ws = moe.workspace(moe.config_of(CONFIGS["tiny"]))
    moe.moe_selftest_bounded_wait(ws, 1_000_000)
    torch.cuda.synchronize()
    moe.moe_read_status(ws)
    a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    a.record()
    moe.moe_selftest_bounded_wait(ws, limit_ms * 1_000_000)
    b.record()
    torch.cuda.synchronize()
    took = a.elapsed_time(b)
    assert moe.moe_read_status(ws) == moe.MOE_ERR_TIMEOUT
    # two limits; a third wait with the kernels' limit of 2 s ends on the flag
    assert 2 * limit_ms <= took < 2 * limit_ms + 500, took
