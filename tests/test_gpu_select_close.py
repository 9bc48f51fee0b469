"""moe_select where fp32 evaluations mislead: choice values and group scores in which
large terms cancel. Indices against the 64-bit definition, token by token."""

import numpy as np
import pytest
import torch

from sparse_moe_transformer_gemm_b200 import build as moe_build
from test_gpu_select import check, logits

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    moe_build.build()


@pytest.mark.parametrize("fn", ["sigmoid", "sqrtsoftplus", "softmax"])
@pytest.mark.parametrize("E", [32, 64, 256])
@pytest.mark.parametrize("big", [100.0, 1e4])
@pytest.mark.parametrize("k,renorm", [(4, True), (3, False)])
def test_group_sums_of_large_biases_that_cancel(fn, E, big, k, renorm):
    """8 groups, one expert of each with the bias +big, the others with -big: a group's
    two best sum to about the sum of their scores, whose differences are below the fp32
    step of the biases."""
    n = E // 8
    z = logits(1, E, E).repeat(200, 1)
    z[:, n:] = z[:, :n].repeat(1, 7)      # all groups alike ...
    step = float(np.spacing(np.float32(big)))
    # ... but for differences of some steps of the sum (a softmax score's slope is about 1 / E)
    z += logits(200, E, 7, 8 * step * (E if fn == "softmax" else 1))
    b = torch.full((E,), -big, device="cuda")
    b[::n] = big
    check(z, k, fn=fn, bias=b, groups=8, keep=4, by="top2", renorm=renorm)


def test_group_sums_that_overflow_fp32():
    """Biases of the type's lowest value: sums of two of them are ranked, not lost."""
    low = float(torch.finfo(torch.float32).min)
    z = logits(40, 16, 9)
    b = torch.full((16,), low, device="cuda")
    b[::4] = low / 4 * torch.arange(1, 5, device="cuda")
    check(z, 3, bias=b, groups=4, keep=2, by="top2")
    z[::2, 2:4] = float("-inf")
    z[::3, 5:8] = float("-inf")
    check(z, 3, bias=b, groups=4, keep=2, by="top2")
