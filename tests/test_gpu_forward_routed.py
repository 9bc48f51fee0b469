"""moe_forward_routed in every weight format: with the router's own choice the layer's
bits, with slots that hold no expert or the same expert twice the weighted sum of the
slots taken one at a time."""

import pytest
import torch

from sparse_moe_transformer_gemm_b200 import build as moe_build
from sparse_moe_transformer_gemm_b200 import moe
from synthetic import LayerShape, make_layer

pytestmark = pytest.mark.gpu
FORMATS = ["bf16", "packed", "fp8", "fp4", "shared", "stream", "fp8 stream"]


@pytest.fixture(scope="module", autouse=True)
def _built():
    moe_build.build()


def layer_of(fmt, T, E, k, d=512, F=256):
    """(config arguments, x, w_gate, the four weight arguments)."""
    L = make_layer(LayerShape(T=T, d=d, E=E, k=k, F=F, fp8="fp8" in fmt, fp4=fmt == "fp4",
                              shared=fmt == "shared"), seed=T, device="cuda")
    kw = dict(fp8="fp8" in fmt, fp4=fmt == "fp4", packed=fmt == "packed", shared=fmt == "shared",
              path="stream" if "stream" in fmt else None)
    weights = list(moe.layer_args(L))
    if fmt == "packed":
        cfg = moe.config(T, d, E, k, F, packed=True)
        for which, i in ((moe.MOE_WEIGHTS_GATE_UP, 0), (moe.MOE_WEIGHTS_DOWN, 2)):
            out = torch.empty_like(weights[i])
            moe.moe_pack_weights(cfg, which, weights[i], out)
            weights[i] = out
    return kw, L["x"], L["w_gate"], weights


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("T,E,k", [(3, 8, 2), (70, 32, 4), (1200, 16, 4)])
def test_the_routers_choice_gives_the_layers_bits(fmt, T, E, k):
    kw, x, wg, weights = layer_of(fmt, T, E, k)
    cfg = moe.config(T, 512, E, k, 256, **kw)
    ws = moe.workspace(cfg)
    idx = torch.empty(T, k, dtype=torch.int32, device="cuda")
    w = torch.empty(T, k, device="cuda")
    a, b = torch.empty_like(x), torch.empty_like(x)
    moe.moe_forward(cfg, x, wg, None, *weights, a, ws)
    moe.moe_route(cfg, x, wg, None, idx, w, ws)
    moe.moe_forward_routed(cfg, x, idx, w, *weights, b, ws)
    assert torch.equal(a, b) and bool(torch.isfinite(a).all())
    assert moe.moe_read_status(ws) == moe.MOE_OK


@pytest.mark.parametrize("fmt", [f for f in FORMATS if f != "shared"])
@pytest.mark.parametrize("T,E,k", [(5, 8, 3), (70, 32, 3), (1500, 16, 3)])
def test_slots_without_an_expert_and_the_same_expert_twice(fmt, T, E, k):
    kw, x, _, weights = layer_of(fmt, T, E, k)
    g = torch.Generator(device="cuda")
    g.manual_seed(E)
    idx = torch.rand(T, E, generator=g, device="cuda").topk(k)[1].to(torch.int32)
    w = torch.rand(T, k, generator=g, device="cuda") + 0.1
    idx[::2, 1] = -1
    idx[1::4, 2] = E + 7
    idx[3, :] = 5
    idx[4, :] = -1
    cfg = moe.config(T, 512, E, k, 256, **kw)
    ws, out = moe.workspace(cfg), torch.full_like(x, 7.0)
    ws[256:] = 0xA5  # what the grouping leaves alone is not read as an index
    moe.moe_workspace_init(cfg, ws)
    moe.moe_forward_routed(cfg, x, idx, w, *weights, out, ws)
    assert (out[4] == 0).all()
    assert moe.moe_read_status(ws) == moe.MOE_OK
    # one slot at a time, weight 1, in the same kernels: the slots' bf16 outputs
    want = torch.zeros(T, 512, dtype=torch.float64, device="cuda")
    size = torch.zeros(T, 512, dtype=torch.float64, device="cuda")
    for j in range(k):
        alone, o = torch.full_like(idx, -1), torch.empty_like(x)
        alone[:, j] = idx[:, j]
        moe.moe_forward_routed(cfg, x, alone, torch.ones_like(w), *weights, o, ws)
        want += o.double() * w[:, j].double()[:, None]
        size += o.double().abs() * w[:, j].double()[:, None]
    # three fp32 multiply-adds, one rounding to bf16
    tol = 2.0 ** -8 * want.abs() + 3 * 2.0 ** -24 * size * (1 + 2.0 ** -8)
    assert ((out.double() - want).abs() <= tol).all()
