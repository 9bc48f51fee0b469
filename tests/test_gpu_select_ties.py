"""moe_select on logits of bf16 precision, where many tokens have equal values within
their choice or at its border: the lower index first."""

import pytest
import torch

from sparse_moe_transformer_gemm_b200 import build as moe_build
from test_gpu_select import bias_of, check, logits

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    moe_build.build()


@pytest.mark.parametrize("fn", ["sigmoid", "sqrtsoftplus", "softmax"])
@pytest.mark.parametrize("T,E,k,groups,keep,by", [
    (400, 256, 8, 1, 1, "max"), (400, 160, 6, 8, 3, "max"), (200, 256, 8, 8, 4, "top2"),
    (200, 64, 32, 1, 1, "max"), (200, 12, 12, 1, 1, "max"), (300, 60, 1, 3, 1, "max")])
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("renorm", [True, False])
def test_logits_of_bf16_precision(fn, T, E, k, groups, keep, by, bias, renorm):
    z = logits(T, E, T + E).to(torch.bfloat16).float()
    b = bias_of(E, std=0.1).to(torch.bfloat16).float() if bias else None
    check(z, k, fn=fn, bias=b, groups=groups, keep=keep, by=by, renorm=renorm)
