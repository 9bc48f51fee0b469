"""The expert choice and block FP8 with every input and output in the last bytes of an
allocation of whole pages: nothing past their ends is read or written (values as with
the tensors elsewhere)."""

import pytest
import torch

import block_reference as ref
from sparse_moe_transformer_gemm_b200 import build as moe_build
from sparse_moe_transformer_gemm_b200 import moe
from test_gpu_block_fp8 import activations, gen, make, quantised
from test_gpu_router_edges import at_the_end
from test_gpu_select import bias_of, logits

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    moe_build.build()


class Ends:
    """Tensors at the ends of their allocations, which live as long as this."""

    def __init__(self):
        self.whole = []

    def __call__(self, t):
        whole, tail = at_the_end(t.contiguous())
        self.whole.append(whole)
        return tail


@pytest.mark.parametrize("T,E,k,groups,keep,by", [(1, 1, 1, 1, 1, "max"), (7, 33, 5, 3, 2, "top2"),
                                                  (40, 256, 8, 8, 4, "top2"),
                                                  (5, 254, 7, 127, 40, "max")])
@pytest.mark.parametrize("fn", ["sigmoid", "softmax"])
def test_select(T, E, k, groups, keep, by, fn):
    at = Ends()
    z, b = logits(T, E, T), bias_of(E)
    cfg, grp = moe.config(T, 128, E, k, 128), moe.group_options(groups, keep, by)
    out = [(torch.zeros(T, k, dtype=torch.int32, device="cuda"), torch.zeros(T, k, device="cuda"))
           for _ in range(2)]
    moe.moe_select(cfg, z, moe.route_options(b, score_fn=fn), grp, *out[0])
    ends = [at(t) for t in out[1]]
    moe.moe_select(cfg, at(z), moe.route_options(at(b), score_fn=fn), grp, *ends)
    assert all(torch.equal(a, b) for a, b in zip(out[0], ends))


@pytest.mark.parametrize("M,K", [(1, 16), (3, 144), (33, 1552), (130, 512)])
def test_quant(M, K):
    at = Ends()
    x = activations(gen(M), M, K)
    q, s = quantised(x)
    q2, s2 = at(torch.zeros_like(q)), at(torch.zeros_like(s))
    moe.moe_block_quant(at(x), q2, s2)
    assert torch.equal(q, q2) and torch.equal(s, s2)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("G,M,N,K", [
    (0, 1, 1, 16), (0, 5, 130, 144), (0, 129, 260, 2064),             # K split
    (0, 20, 19001, 144), (0, 100, 19004, 272), (0, 1300, 1301, 144),  # pair kernels
    (7, 5, 130, 144), (3, 50, 257, 400), (2, 130, 257, 272), (2, 300, 500, 144)])
def test_product(G, M, N, K, dtype):
    at = Ends()
    g = gen(M + N)
    q, s = quantised(activations(g, M, K))
    ws = [ref.random_weight(g, N, K) for _ in range(max(G, 1))]
    wq, sw = (torch.stack([w[i] for w in ws]) if G else ws[0][i] for i in (0, 1))
    offsets = torch.linspace(0, M, G + 1, device="cuda").to(torch.int32) if G else None
    work = moe.block_workspace(M, N, K, max(G, 1))
    a = torch.zeros(M, N, dtype=dtype, device="cuda")
    moe.moe_block_gemm(q, s, wq, sw, a, work, offsets)
    if a.numel() * a.element_size() % 16 == 0:  # the output's address has to be a multiple of 16
        b = at(torch.zeros_like(a))
    else:
        b = torch.zeros_like(a)
    moe.moe_block_gemm(at(q), at(s), at(wq), at(sw), b, work, None if G == 0 else at(offsets))
    assert torch.equal(a, b) and moe.moe_read_status(work) == moe.MOE_OK


@pytest.mark.parametrize("T,d,E,k,F", [(1, 128, 1, 1, 128), (9, 256, 4, 2, 384), (70, 512, 3, 3, 128),
                                       (400, 384, 2, 1, 256)])
def test_layer(T, d, E, k, F):
    at = Ends()
    p = make(T, d, E, k, F, T)
    wg = (torch.randn(E, d, device="cuda", generator=gen(T)) * 0.05).to(torch.bfloat16)
    a, b = (torch.zeros(T, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    names = ("wgu", "sgu", "wd", "sd")
    moe.moe_forward4(p["cfg"], p["x"], wg, None, None, None, *(p[n] for n in names), a, p["ws"])
    aligned = lambda t: at(t) if t.numel() * t.element_size() % 16 == 0 else t  # noqa: E731
    b = at(b)
    ws = at(torch.zeros_like(p["ws"][:p["ws"].numel() // 256 * 256]))
    moe.moe_workspace_init(p["cfg"], ws)
    moe.moe_forward4(p["cfg"], at(p["x"]), at(wg), None, None, None,
                     *(aligned(p[n]) for n in names), b, ws)
    assert torch.equal(a, b) and moe.moe_read_status(ws) == moe.MOE_OK
