"""The routers with w_gate and x at the very end of a memory segment: K slices whose last
chunk has 128 columns read nothing past the last row. Logits are exact (integers), so
the choice is the definition's."""

import numpy as np
import pytest
import torch

from sparse_moe_transformer_gemm_b200 import build as moe_build
from sparse_moe_transformer_gemm_b200 import moe

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    moe_build.build()


def at_the_end(t):
    """t's values in the last bytes of an allocation of whole 2 MB pages."""
    n = t.numel() * t.element_size()
    whole = torch.zeros(-(-max(n, 20 << 20) // (2 << 20)) * (2 << 20), dtype=torch.uint8,
                        device="cuda")
    tail = whole[whole.numel() - n:].view(t.dtype).view(t.shape)
    tail.copy_(t)
    return whole, tail


@pytest.mark.parametrize("d", [128, 256, 384, 512, 640, 1152, 4224])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (5, 8, 2), (24, 4, 2), (64, 33, 8), (140, 20, 4)])
def test_nothing_is_read_past_the_last_row(d, T, E, k):
    g = torch.Generator(device="cuda")
    g.manual_seed(d + T)
    x = torch.randint(-2, 3, (T, d), generator=g, device="cuda").to(torch.bfloat16)
    wg = (torch.randint(-3, 4, (E, d), generator=g, device="cuda") / 64).to(torch.bfloat16)
    z = x.double() @ wg.double().T
    keep, wg = at_the_end(wg)
    keep2, x = at_the_end(x)
    cfg = moe.config(T, d, E, k, 128)
    ws = moe.workspace(cfg)
    idx = torch.empty(T, k, dtype=torch.int32, device="cuda")
    w = torch.empty(T, k, device="cuda")
    want = (-z).sort(dim=1, stable=True)[1][:, :k].int()
    s = torch.sigmoid(z).gather(1, want.long())
    s = cfg.scale * s / s.sum(1, keepdim=True)
    for call in (lambda: moe.moe_route(cfg, x, wg, None, idx, w, ws),
                 lambda: moe.moe_route4(cfg, x, wg, None, None, None, idx, w, ws),
                 lambda: moe.moe_route_noalloc(cfg, x, wg, None, idx, w)):
        idx.fill_(-7)
        call()
        assert torch.equal(idx, want)
        assert np.allclose(w.cpu().numpy(), s.cpu().numpy(), rtol=4e-6, atol=0)
    assert moe.moe_read_status(ws) == moe.MOE_OK
