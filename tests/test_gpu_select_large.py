"""moe_select with sqrt(softplus) scores so large that fp32 resolves them coarsely, and
biases that cancel them. Indices against the 64-bit definition, token by token."""

import numpy as np
import pytest
import torch

import block_reference as ref
from sparse_moe_transformer_gemm_b200 import build as moe_build
from test_gpu_select import check, logits

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    moe_build.build()


@pytest.mark.parametrize("m", [6, 7, 13, 20])
@pytest.mark.parametrize("k", [1, 6])
@pytest.mark.parametrize("groups,keep,by", [(1, 1, "max"), (8, 3, "max"), (8, 3, "top2")])
def test_large_scores_that_biases_cancel(m, k, groups, keep, by):
    """Scores just above 2^m, biases just above -2^m, whose fp32 step is half of the
    scores': the choice values lie half a step of the score apart."""
    E = 64
    gen = torch.Generator("cuda")
    gen.manual_seed(m)
    z = 4.0 ** m * (1.0002 + 0.0148 * torch.rand(1, E, device="cuda", generator=gen))
    s = ref.score64(z.cpu().numpy()[0], "sqrtsoftplus")
    half = 2.0 ** (m - 24)
    value = 0.008 * 2.0 ** m + 0.5 + half * np.random.default_rng(m).permutation(E)
    b = torch.tensor((value - s).astype(np.float32), device="cuda")
    z = z * (1 + logits(150, E, 4, 2e-7))
    check(z, k, fn="sqrtsoftplus", bias=b, groups=groups, keep=keep, by=by)


@pytest.mark.parametrize("groups,keep,by", [(1, 1, "max"), (8, 3, "max"), (8, 3, "top2")])
def test_one_infinite_logit_among_ordinary_ones(groups, keep, by):
    """+infinity counts as the largest finite float, whose score is 1.8e19: the others
    keep their order."""
    z = logits(60, 64, 5)
    z[::2, 17] = float("inf")
    check(z, 6, fn="sqrtsoftplus", bias=logits(1, 64, 6, 0.05)[0].contiguous(), groups=groups,
          keep=keep, by=by)
