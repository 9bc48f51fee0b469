"""moe_select on logits whose scores are close to or below fp32's smallest numbers: the
weights keep their ratios, and biased values of 0 bias the order of fp64's scores."""

import pytest
import torch

from sparse_moe_transformer_gemm_b200 import build as moe_build
from test_gpu_select import check, logits

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    moe_build.build()


@pytest.mark.parametrize("fn", ["sigmoid", "sqrtsoftplus"])
@pytest.mark.parametrize("centre", [-15.0, -20.0, -40.0, -72.0, -79.5, -85.0, -100.0])
@pytest.mark.parametrize("bias", [False, True])
def test_renormalised_weights_keep_their_ratios(fn, centre, bias):
    """The largest score may be an ordinary number and the next one below fp32's range."""
    z = centre + logits(100, 48, 2, 10.0)
    b = logits(1, 48, 3, 0.05)[0].contiguous() if bias else None
    check(z, 8, fn=fn, bias=b)


@pytest.mark.parametrize("centre", [-14.0, -17.0, -60.0, -100.0, -150.0])
@pytest.mark.parametrize("groups,keep,by", [(1, 1, "max"), (8, 3, "top2")])
def test_small_sqrt_softplus_weights(centre, groups, keep, by):
    """sqrt(softplus(z)) is e^(z/2) there, a number of fp32 where e^z is none."""
    check(centre + logits(100, 48, 4, 4.0), 8, fn="sqrtsoftplus", renorm=False, groups=groups,
          keep=keep, by=by)


def test_scores_below_the_normal_numbers_of_fp64_keep_their_order():
    z = -717.0 + logits(60, 64, 5, 2.0)
    check(z, 8, bias=torch.zeros(64, device="cuda"))
    z = -690.0 + logits(60, 64, 6, 10.0)
    check(z, 8, fn="sqrtsoftplus", bias=torch.zeros(64, device="cuda"))
