"""A row of a grouped block-FP8 product has the same bits in each of the four kernels
(tiles of 32, 64 and 128 tokens, and of 256), which the call chooses by the rows per
group on average: M <= G, <= 32 G, <= 112 G, more."""

import pytest
import torch

import block_reference as ref
from sparse_moe_transformer_gemm_b200 import build as moe_build
from sparse_moe_transformer_gemm_b200 import moe
from test_gpu_block_fp8 import activations, check_h, gen, product, quantised

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    moe_build.build()


def groups_of(M):
    """G for which M rows take the 256-, 128-, 64- and 32-token kernels."""
    gs = [1, -(-M // 112), -(-M // 32), M]
    assert M > 112 and gs[-1] <= 256 and 32 * gs[1] < M and gs[2] < M
    return gs


def one_in(G, e, t, fill):
    """[G, ...] with t at e, `fill` elsewhere."""
    out = torch.full((G,) + t.shape, fill, dtype=t.dtype, device=t.device)
    out[e] = t
    return out


@pytest.mark.parametrize("M", [113, 200, 256])
@pytest.mark.parametrize("N,K", [(512, 1536), (384, 4096), (400, 912), (130, 7168), (64, 16)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_product_rows(M, N, K, dtype):
    g = gen(M + K)
    q, s = quantised(activations(g, M, K))
    w, v = ref.random_weight(g, N, K)
    outs = []
    for G in groups_of(M):
        e = G // 2  # the group that holds all rows; the others are empty
        offsets = torch.zeros(G + 1, dtype=torch.int32, device="cuda")
        offsets[e + 1:] = M
        outs.append(product(q, s, one_in(G, e, w, 0), one_in(G, e, v, 1.0), N, dtype, offsets))
    ref.check_product(outs[0], ref.values(q, s), ref.weight_values(w, v))
    for o in outs[1:]:
        assert torch.equal(o, outs[0])


@pytest.mark.parametrize("M", [113, 256])
@pytest.mark.parametrize("d,F", [(4096, 1536), (512, 384), (7168, 256)])
def test_gate_up_and_down_rows(M, d, F):
    """The same for the layer's steps: codes and scales of h, and y."""
    g = gen(M + d)
    x = activations(g, M, d)
    q, s = quantised(x)
    wgu, sgu = ref.random_weight(g, 2 * F, d)
    wd, sd = ref.random_weight(g, d, F)
    outs = []
    for E in groups_of(M):
        e = E // 2
        cfg = moe.config(M, d, E, 1, F, fp8_block=True)
        ws = moe.workspace(cfg)
        offsets = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
        offsets[e + 1:] = M
        hq = torch.zeros(M, F, dtype=torch.uint8, device="cuda")
        sh = torch.zeros(M, F // 128, device="cuda")
        y = torch.zeros(M, d, dtype=torch.bfloat16, device="cuda")
        moe.moe_block_gate_up(cfg, q, s, offsets, one_in(E, e, wgu, 0), one_in(E, e, sgu, 1.0), hq,
                              sh, ws)
        moe.moe_block_down(cfg, hq, sh, offsets, one_in(E, e, wd, 0), one_in(E, e, sd, 1.0), y, ws)
        assert moe.moe_read_status(ws) == moe.MOE_OK
        outs.append((hq, sh, y))
    hq, sh, y = outs[0]
    check_h(hq, sh, ref.values(q, s), ref.weight_values(wgu, sgu), F)
    ref.check_product(y, ref.values(hq, sh), ref.weight_values(wd, sd))
    for other in outs[1:]:
        assert all(torch.equal(a, b) for a, b in zip(outs[0], other))
