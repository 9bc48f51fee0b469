"""Expert parallelism with block-FP8 weights whose experts have few scales: a rank's
slice of the scales may begin anywhere, the library takes 16-byte aligned ones."""

import pytest
import torch

import block_reference as ref
from sparse_moe_transformer_gemm_b200 import build as moe_build
from sparse_moe_transformer_gemm_b200 import ep, moe


@pytest.mark.parametrize("E,P", [(4, 4), (6, 3), (6, 2), (8, 1)])
@pytest.mark.parametrize("d,F", [(128, 128), (640, 384), (256, 256)])
def test_a_ranks_scales_are_aligned(E, P, d, F):
    part = ep.Partition(E, P)
    sgu = torch.rand(E, 2 * F // 128, d // 128)
    sd = torch.rand(E, d // 128, F // 128)
    w = torch.zeros(E, 16, dtype=torch.uint8)
    for r in range(P):
        gu, sgu_r, dn, sd_r = ep.local_expert_weights(part, r, w, w, sgu, sd)
        own = slice(r * part.E_local, (r + 1) * part.E_local)
        for got, whole in ((sgu_r, sgu), (sd_r, sd)):
            assert torch.equal(got, whole[own]) and got.data_ptr() % 16 == 0
            assert got.is_contiguous()
        # the weights stay views of the layer's
        assert gu.data_ptr() == w[own].data_ptr() and dn.data_ptr() == w[own].data_ptr()
    assert ep.local_expert_weights(part, 0, w, w)[1] is None


@pytest.mark.gpu
@pytest.mark.parametrize("d,F", [(128, 128), (640, 384)])
@pytest.mark.parametrize("T,E,k,P", [(24, 4, 2, 4), (60, 6, 3, 2)])
def test_ranks_equal_the_layer_on_one_gpu(d, F, T, E, k, P):
    moe_build.build()
    g = torch.Generator(device="cuda")
    g.manual_seed(d + T)
    gu = [ref.random_weight(g, 2 * F, d) for _ in range(E)]
    dn = [ref.random_weight(g, d, F) for _ in range(E)]
    weights = [torch.stack([p[i] for p in ws]) for ws in (gu, dn) for i in (0, 1)]
    x = torch.randn(T, d, generator=g, device="cuda").to(torch.bfloat16)
    wg = (torch.randn(E, d, generator=g, device="cuda") * 0.05).to(torch.bfloat16)
    cfg = moe.config(T, d, E, k, F, fp8_block=True)
    part = ep.Partition(E, P)
    ops = [ep.ep_layer_ops(cfg, part, r, wg, None, *weights) for r in range(P)]
    xs = [c.contiguous() for c in torch.chunk(x, P)]
    for c, out in zip(xs, ep.ep_forward_lockstep(ops, part, xs)):
        one = moe.config(c.shape[0], d, E, k, F, fp8_block=True)
        ws, want = moe.workspace(one), torch.empty_like(c)
        moe.moe_forward(one, c, wg, None, *weights, want, ws)
        assert torch.equal(out, want) and moe.moe_read_status(ws) == moe.MOE_OK


@pytest.mark.gpu
def test_the_copied_scales_are_ready_on_any_stream():
    """The rank is made behind long work on one stream and runs on another."""
    moe_build.build()
    T, E, k, d, F, P = 24, 4, 2, 128, 128, 4
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    gu = [ref.random_weight(g, 2 * F, d) for _ in range(E)]
    dn = [ref.random_weight(g, d, F) for _ in range(E)]
    weights = [torch.stack([p[i] for p in ws]) for ws in (gu, dn) for i in (0, 1)]
    x = torch.randn(T, d, generator=g, device="cuda").to(torch.bfloat16)
    wg = (torch.randn(E, d, generator=g, device="cuda") * 0.05).to(torch.bfloat16)
    cfg = moe.config(T, d, E, k, F, fp8_block=True)
    part = ep.Partition(E, P)
    xs = [c.contiguous() for c in torch.chunk(x, P)]

    def outputs():
        ops = [ep.ep_layer_ops(cfg, part, r, wg, None, *weights) for r in range(P)]
        other = torch.cuda.Stream()
        with torch.cuda.stream(other):
            outs = ep.ep_forward_lockstep(ops, part, xs)
        torch.cuda.synchronize()
        return outs

    first = outputs()
    torch.cuda.synchronize()
    a = torch.randn(8192, 8192, device="cuda")
    for _ in range(3):
        junk = [torch.full((64,), float("nan"), device="cuda") for _ in range(64)]
        del junk
        torch.cuda.synchronize()
        for _ in range(20):
            a @ a  # some tens of milliseconds
        for got, want in zip(outputs(), first):
            assert torch.equal(got, want)
