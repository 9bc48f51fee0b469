"""Block-scaled FP8 (moe_block_quant, moe_block_gemm, the block-FP8 experts and
layer) against 64-bit definitions; tolerances in block_reference.py."""

import pytest
import torch

import block_reference as ref
from sparse_moe_transformer_gemm_b200 import build as moe_build
from sparse_moe_transformer_gemm_b200 import ep, moe

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    moe_build.build()


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def activations(g, M, K):
    x = torch.randn(M, K, generator=g, device="cuda")
    x[:, ::37] *= 20.0
    return x.to(torch.bfloat16)


def quantised(x):
    M, K = x.shape
    q = torch.empty(M, K, dtype=torch.uint8, device="cuda")
    s = torch.empty(M, ref.nblocks(K), device="cuda")
    moe.moe_block_quant(x, q, s)
    return q, s


# ------------------------------------------------------------------ quantisation

def check_quant(x):
    q, s = quantised(x)
    want, a = ref.quant64(x)
    # a / 448 in 64 bits and rounded once: torch divides fp32 tensors by a number
    # with a rounded reciprocal, an ulp off. A quotient of an 8-bit integer by 7
    # is 2^-28 or more away from a midpoint of two fp32 values, far beyond fp64's error.
    assert torch.equal(s, torch.where(a == 0, 1.0, a / 448.0).float())
    assert torch.equal(q.view(ref.FP8).double(), want)


@pytest.mark.parametrize("M,K", [(1, 16), (1, 128), (3, 144), (5, 240), (64, 4096), (33, 1536),
                                 (7, 8208), (130, 256), (2, 1040)])
def test_quant_is_the_exact_rounding(M, K):
    check_quant(activations(gen(M + K), M, K))


def test_quant_of_every_bf16_significand_against_every_amax():
    """Quotients of all pairs of 8-bit significands, midpoints among them."""
    a = torch.arange(128, 256, device="cuda").float()
    x = torch.zeros(128, 256, device="cuda")
    x[:, 0:128] = a[None, :] / 256          # significands below ...
    x[:, 0] = a                             # ... each amax
    x[:, 128:256] = a[None, :] / 4096
    x[:, 128] = a
    check_quant(x.to(torch.bfloat16))
    check_quant((-x).to(torch.bfloat16))


def test_quant_extremes():
    """Zero blocks, the smallest and largest magnitudes, a block of one value."""
    x = torch.zeros(8, 384, device="cuda")
    x[1, 5] = 1.0
    # (in 64 bits: the fp32 linspace overflows to NaN between these ends)
    x[2] = torch.linspace(-3e38, 3e38, 384, device="cuda", dtype=torch.float64).float()
    x[3] = torch.linspace(-1e-30, 1e-30, 384, device="cuda")
    x[4, 128:256] = torch.linspace(0, 1e-37, 128, device="cuda")
    x[5] = -7.0
    x[6, 300] = -448.0
    x[7, 0:128] = 2.0 ** torch.arange(-64, 64, device="cuda").float()
    check_quant(x.to(torch.bfloat16))


def test_quant_of_subnormals():
    """Blocks whose largest magnitude is a subnormal bf16 (m 2^-133, m < 128): the scale is
    m 1024 / 7 steps of 2^-149, never halfway between two."""
    m = torch.arange(0, 128, device="cuda").double()
    x = torch.zeros(128, 128, device="cuda", dtype=torch.float64)
    for r in range(128):
        x[r] = torch.minimum(m, m[r]) * 2.0 ** -133
    check_quant(x.to(torch.bfloat16))


def test_quant_past_two_to_the_31_elements():
    M, K = 131075, 16400
    x = torch.zeros(M, K, dtype=torch.bfloat16, device="cuda")
    rows = torch.cat([torch.arange(0, 3), torch.randint(0, M, (60,)),
                      torch.arange(M - 3, M)]).unique().to("cuda")
    x[rows] = activations(gen(32), rows.numel(), K)
    q, s = quantised(x)
    q2, s2 = quantised(x[rows].contiguous())
    assert torch.equal(q[rows], q2) and torch.equal(s[rows], s2)
    assert int((s != 1).any(1).sum()) == rows.numel()


def test_quant_in_a_graph_on_another_stream():
    x = activations(gen(33), 70, 1536)
    q, s = quantised(x)
    q2, s2 = torch.zeros_like(q), torch.zeros_like(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.moe_block_quant(x, q2, s2)
    x.neg_()
    graph.replay()
    assert torch.equal(s, s2) and torch.equal(q.view(ref.FP8).float(), -q2.view(ref.FP8).float())


def test_quant_of_infinities_and_nan_is_not_finite_in_that_block_only():
    x = activations(gen(1), 3, 384)
    x[0, 5], x[1, 200], x[2, 383] = float("inf"), float("nan"), float("-inf")
    q, s = quantised(x)
    v = ref.values(q, s)
    for r, b in ((0, 0), (1, 1), (2, 2)):
        bad = torch.isnan(v[r]).view(3, 128)
        assert bad[b].all() and not bad[[i for i in range(3) if i != b]].any()


def test_quant_of_strided_rows():
    wide = activations(gen(2), 20, 1024)
    view = wide[:, 256:784]
    q, s = quantised(view)
    q2, s2 = quantised(view.contiguous())
    assert torch.equal(q, q2) and torch.equal(s, s2)


# ------------------------------------------------------------------ product

def product(q, s, wq, sw, N, dtype=torch.bfloat16, offsets=None, fill=-99.0):
    out = torch.full((q.shape[0], N), fill, dtype=dtype, device="cuda")
    G = 1 if offsets is None else wq.shape[0]
    ws = moe.block_workspace(q.shape[0], N, q.shape[1], G)
    moe.moe_block_gemm(q, s, wq, sw, out, ws, offsets)
    assert moe.moe_read_status(ws) == moe.MOE_OK
    return out


SIZES = [(1, 1, 16), (1, 128, 128), (1, 4096, 4096), (2, 130, 144), (7, 500, 2064),
         (16, 256, 256), (17, 520, 640), (31, 129, 1040), (33, 257, 384), (64, 1024, 4096),
         (65, 512, 512), (100, 1, 256), (128, 640, 1536), (129, 384, 128), (200, 1000, 912),
         (300, 513, 272), (1000, 768, 2048),
         # enough tiles for the pair kernels: tokens in the MMA's rows, ...
         (1300, 1301, 144), (1300, 1400, 272), (1537, 1284, 528),
         # ... or weights, in tiles of up to 32, 64 and 128 tokens
         (20, 19000, 128), (40, 19001, 144), (100, 19004, 272), (128, 19200, 400)]


@pytest.mark.parametrize("M,N,K", SIZES)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_product(M, N, K, dtype):
    g = gen(M * 7 + N + K)
    q, s = quantised(activations(g, M, K))
    wq, sw = ref.random_weight(g, N, K)
    out = product(q, s, wq, sw, N, dtype)
    ref.check_product(out, ref.values(q, s), ref.weight_values(wq, sw), (M, N, K))


@pytest.mark.parametrize("counts", [[3, 0, 5, 1], [0, 0, 0, 0], [200, 1, 0, 33],
                                    [0, 129, 128, 127], [16, 17, 31, 32, 64, 65, 0, 1],
                                    [300, 0, 129, 513], [257, 256, 255, 1], [40, 64, 33, 65]])
@pytest.mark.parametrize("N,K", [(256, 384), (200, 144), (640, 1024), (333, 272)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_grouped_product_leaves_other_rows(counts, N, K, dtype):
    g = gen(sum(counts) + N)
    G, pad = len(counts), 5
    offsets = torch.tensor([0] + counts, device="cuda").cumsum(0).to(torch.int32) + 2
    M = sum(counts) + 2 + pad
    q, s = quantised(activations(g, M, K))
    ws = [ref.random_weight(g, N, K) for _ in range(G)]
    wq, sw = torch.stack([w for w, _ in ws]), torch.stack([v for _, v in ws])
    out = product(q, s, wq, sw, N, dtype, offsets)
    xv = ref.values(q, s)
    at = 2
    for e, n in enumerate(counts):
        if n:
            ref.check_product(out[at:at + n], xv[at:at + n], ref.weight_values(wq[e], sw[e]), e)
        at += n
    assert (out[:2] == -99).all() and (out[at:] == -99).all()


def test_outputs_past_two_to_the_31_elements_and_more_tiles_than_a_list_holds():
    """131075 x 20008 (2.6e9 outputs, 40527 tiles), rows from all over checked."""
    g = gen(30)
    M, N, K = 131075, 20008, 16
    q, s = quantised(activations(g, M, K))
    wq, sw = ref.random_weight(g, N, K)
    out = product(q, s, wq, sw, N)
    rows = torch.cat([torch.arange(0, 5), torch.randint(0, M, (200,)),
                      torch.arange(M - 5, M)]).to("cuda")
    ref.check_product(out[rows], ref.values(q[rows], s[rows]), ref.weight_values(wq, sw))


def test_more_weight_tiles_than_a_list_holds():
    """256 groups of one row times 131072 weight rows: 65536 tiles of the few-rows kernel."""
    g = gen(31)
    G, N, K = 256, 131072, 16
    q, s = quantised(activations(g, G, K))
    wq = torch.randint(0, 256, (G, N, K), generator=g, device="cuda", dtype=torch.uint8)
    wq = torch.where(wq & 0x7F == 0x7F, 0, wq).to(torch.uint8)
    sw = torch.rand(G, N // 128, 1, generator=g, device="cuda") + 0.5
    offsets = torch.arange(G + 1, dtype=torch.int32, device="cuda")
    out = product(q, s, wq, sw, N, offsets=offsets)
    xv = ref.values(q, s)
    for e in (0, 1, 100, 254, 255):
        ref.check_product(out[e:e + 1], xv[e:e + 1], ref.weight_values(wq[e], sw[e]), e)


def test_grouped_product_clamps_offsets():
    g = gen(4)
    q, s = quantised(activations(g, 12, 256))
    ws = [ref.random_weight(g, 128, 256) for _ in range(2)]
    wq, sw = torch.stack([w for w, _ in ws]), torch.stack([v for _, v in ws])
    offsets = torch.tensor([-3, 8, 99], dtype=torch.int32, device="cuda")
    out = product(q, s, wq, sw, 128, offsets=offsets)
    xv = ref.values(q, s)
    ref.check_product(out[:8], xv[:8], ref.weight_values(wq[0], sw[0]))
    ref.check_product(out[8:], xv[8:], ref.weight_values(wq[1], sw[1]))


def test_product_scales_differ_per_block():
    """All codes 1, scales powers of two that differ in every block: exact sums."""
    M, N, K = 40, 300, 528
    q = torch.full((M, K), 0x38, dtype=torch.uint8, device="cuda")   # 1.0
    wq = torch.full((N, K), 0x38, dtype=torch.uint8, device="cuda")
    s = 2.0 ** (torch.arange(M * 5, device="cuda").view(M, 5) % 7 - 3).float()
    sw = 2.0 ** (torch.arange(15, device="cuda").view(3, 5) % 5 - 2).float()
    out = product(q, s, wq, sw, N, torch.float32)
    want = ref.values(q, s) @ ref.weight_values(wq, sw).T
    assert torch.equal(out.double(), want)


def test_every_code_pair_survives():
    """Each finite e4m3 code against a one-hot weight: exact values back."""
    codes = torch.tensor([c for c in range(256) if c & 0x7F != 0x7F], dtype=torch.uint8,
                         device="cuda")
    q = torch.zeros(254, 128, dtype=torch.uint8, device="cuda")
    q[:, 77] = codes
    wq = torch.zeros(16, 128, dtype=torch.uint8, device="cuda")
    wq[:, 77] = 0x38
    out = product(q, torch.ones(254, 1, device="cuda"), wq, torch.ones(1, 1, device="cuda"), 16,
                  torch.float32)
    assert torch.equal(out, codes.view(ref.FP8).float()[:, None].expand(254, 16))


def test_nan_in_one_row_stays_in_that_row():
    g = gen(9)
    x = activations(g, 50, 512)
    x[20, 300] = float("nan")
    q, s = quantised(x)
    wq, sw = ref.random_weight(g, 256, 512)
    out = product(q, s, wq, sw, 256)
    bad = torch.isnan(out)
    assert bad[20].all() and int(bad.sum()) == 256


def test_product_is_the_same_every_time_and_in_a_graph():
    g = gen(10)
    for M, N, K in ((1, 1024, 4096), (300, 520, 1024)):
        q, s = quantised(activations(g, M, K))
        wq, sw = ref.random_weight(g, N, K)
        ws = moe.block_workspace(M, N, K)
        out = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
        moe.moe_block_gemm(q, s, wq, sw, out, ws)
        first = out.clone()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            moe.moe_block_gemm(q, s, wq, sw, out, ws)
        for _ in range(3):
            out.zero_()
            graph.replay()
            assert torch.equal(out, first)
        assert moe.moe_read_status(ws) == moe.MOE_OK


def test_two_products_at_once_on_two_streams():
    g = gen(11)
    jobs = []
    for i, (M, N, K) in enumerate(((64, 2048, 4096), (3, 4096, 2048))):
        q, s = quantised(activations(g, M, K))
        wq, sw = ref.random_weight(g, N, K)
        jobs.append((q, s, wq, sw, torch.empty(M, N, dtype=torch.bfloat16, device="cuda"),
                     moe.block_workspace(M, N, K), torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(10):
        for q, s, wq, sw, out, ws, st in jobs:
            moe.moe_block_gemm(q, s, wq, sw, out, ws, stream=st)
    torch.cuda.synchronize()
    for q, s, wq, sw, out, ws, _ in jobs:
        ref.check_product(out, ref.values(q, s), ref.weight_values(wq, sw))
        assert moe.moe_read_status(ws) == moe.MOE_OK


# ------------------------------------------------------------------ experts and layer

def make(T, d, E, k, F, seed=0, shared=False):
    g = gen(seed)
    n = E + int(shared)
    gu = [ref.random_weight(g, 2 * F, d) for _ in range(n)]
    dn = [ref.random_weight(g, d, F) for _ in range(n)]
    p = dict(cfg=moe.config(T, d, E, k, F, fp8_block=True, shared=shared),
             x=activations(g, T, d),
             idx=torch.rand(T, E, generator=g, device="cuda").topk(k)[1].to(torch.int32),
             w=torch.rand(T, k, generator=g, device="cuda") + 0.1,
             wgu=torch.stack([a for a, _ in gu]), sgu=torch.stack([a for _, a in gu]),
             wd=torch.stack([a for a, _ in dn]), sd=torch.stack([a for _, a in dn]))
    p["ws"] = moe.workspace(p["cfg"])
    return p


def stages(p):
    """The layer's steps one call at a time: (row_of, offsets, xq, sx, hq, sh, y, out)."""
    cfg, n = p["cfg"], p["wgu"].shape[0]
    kk = cfg.k + n - cfg.E
    R = cfg.T * kk
    i32 = lambda m: torch.zeros(m, dtype=torch.int32, device="cuda")  # noqa: E731
    counts, offsets, row_of, tok = i32(n), i32(n + 1), i32(R), i32(R)
    moe.moe_permute_index(cfg, p["idx"], counts, offsets, row_of, tok, p["ws"])
    xq = torch.zeros(R, cfg.d, dtype=torch.uint8, device="cuda")
    sx = torch.zeros(R, cfg.d // 128, device="cuda")
    moe.moe_block_permute(cfg, p["x"], row_of, xq, sx)
    hq = torch.zeros(R, cfg.d_ff, dtype=torch.uint8, device="cuda")
    sh = torch.zeros(R, cfg.d_ff // 128, device="cuda")
    moe.moe_block_gate_up(cfg, xq, sx, offsets, p["wgu"], p["sgu"], hq, sh, p["ws"])
    y = torch.zeros(R, cfg.d, dtype=torch.bfloat16, device="cuda")
    moe.moe_block_down(cfg, hq, sh, offsets, p["wd"], p["sd"], y, p["ws"])
    out = torch.zeros(cfg.T, cfg.d, dtype=torch.bfloat16, device="cuda")
    moe.moe_combine(cfg, y, row_of, p["w"], out, p["ws"])
    assert moe.moe_read_status(p["ws"]) == moe.MOE_OK
    return row_of, offsets, tok, xq, sx, hq, sh, y, out


def check_h(hq, sh, xv, wv, F):
    """hq * sh against h = SiLU(g) u: the products' tolerances through SiLU (its
    slope is below 1.1), 1e-5 for its fast exponential and division, and half a
    step of e4m3: 2^-4 of the value, or 2^-10 of the block's scale below the
    smallest normal."""
    g, u = xv @ wv[:F].T, xv @ wv[F:].T
    tol = ref.product_tol(xv.shape[1])
    dg, du = tol * (xv.abs() @ wv[:F].abs().T), tol * (xv.abs() @ wv[F:].abs().T)
    silu = torch.nn.functional.silu(g)
    h = silu * u
    dh = 1.1 * dg * (u.abs() + du) + silu.abs() * du + 1e-5 * h.abs()
    cols = torch.arange(F, device=hq.device) // 128
    a = h.abs().view(h.shape[0], -1, 128).amax(2)
    da = dh.view(h.shape[0], -1, 128).amax(2)
    assert ((sh.double() - a / 448).abs() <= (da + 1e-6 * a) / 448 + 1e-30).all()
    step = torch.maximum(2.0 ** -4 * (h.abs() + dh), 2.0 ** -10 * sh.double()[:, cols])
    err = (ref.values(hq, sh) - h).abs()
    assert (err <= step * 1.0001 + dh + 1e-30).all(), float((err / (step + dh + 1e-30)).max())


LAYERS = [(1, 128, 1, 1, 128), (1, 512, 8, 4, 256), (5, 256, 4, 4, 384), (64, 512, 16, 4, 128),
          (77, 384, 6, 2, 640), (300, 256, 3, 2, 256), (513, 640, 2, 1, 384),
          (40, 1024, 64, 8, 256), (100, 256, 8, 3, 384), (200, 384, 4, 2, 256),
          (1100, 256, 8, 2, 640), (3, 8192, 4, 2, 128), (260, 128, 255, 1, 128)]


@pytest.mark.parametrize("T,d,E,k,F", LAYERS)
@pytest.mark.parametrize("shared", [False, True])
def test_layer_steps(T, d, E, k, F, shared):
    p = make(T, d, E, k, F, T + d, shared)
    row_of, offsets, tok, xq, sx, hq, sh, y, out = stages(p)
    q, s = quantised(p["x"])
    assert torch.equal(xq, q[tok.long()]) and torch.equal(sx, s[tok.long()])
    off = offsets.tolist()
    for e in range(p["wgu"].shape[0]):
        a, b = off[e], off[e + 1]
        if a == b:
            continue
        check_h(hq[a:b], sh[a:b], ref.values(xq[a:b], sx[a:b]),
                ref.weight_values(p["wgu"][e], p["sgu"][e]), F)
        ref.check_product(y[a:b], ref.values(hq[a:b], sh[a:b]),
                          ref.weight_values(p["wd"][e], p["sd"][e]), e)
    # one call for all of it: the same bits
    whole = torch.empty_like(out)
    moe.moe_forward_routed(p["cfg"], p["x"], p["idx"], p["w"], p["wgu"], p["sgu"], p["wd"],
                           p["sd"], whole, p["ws"])
    assert torch.equal(whole, out)
    # moe_experts quantises the rows it is given
    xp, y2 = p["x"][tok.long()].contiguous(), torch.empty_like(y)
    moe.moe_experts(p["cfg"], xp, offsets, p["wgu"], p["sgu"], p["wd"], p["sd"], y2, p["ws"])
    assert torch.equal(y2, y)
    assert moe.moe_read_status(p["ws"]) == moe.MOE_OK


def test_layer_with_router_and_groups_is_its_two_halves():
    p = make(70, 512, 32, 4, 256, 3)
    wg = (torch.randn(32, 512, device="cuda", generator=gen(5)) * 0.05).to(torch.bfloat16)
    opt = moe.route_options(torch.randn(32, device="cuda", generator=gen(6)) * 0.1,
                            score_fn="softmax")
    grp = moe.group_options(4, 2, "top2", True)
    a, b = (torch.empty(70, 512, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    weights = (p["wgu"], p["sgu"], p["wd"], p["sd"])
    moe.moe_forward4(p["cfg"], p["x"], wg, None, opt, grp, *weights, a, p["ws"])
    moe.moe_route4(p["cfg"], p["x"], wg, None, opt, grp, p["idx"], p["w"], p["ws"])
    moe.moe_forward_routed(p["cfg"], p["x"], p["idx"], p["w"], *weights, b, p["ws"])
    assert torch.equal(a, b) and bool(torch.isfinite(a).all())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.moe_forward4(p["cfg"], p["x"], wg, None, opt, grp, *weights, a, p["ws"])
    a.zero_()
    graph.replay()
    graph.replay()
    assert torch.equal(a, b)
    # the earlier entry points take the format too (their own sigmoid choice)
    c, d = torch.empty_like(a), torch.empty_like(a)
    moe.moe_forward(p["cfg"], p["x"], wg, None, *weights, c, p["ws"])
    moe.moe_route(p["cfg"], p["x"], wg, None, p["idx"], p["w"], p["ws"])
    moe.moe_forward_routed(p["cfg"], p["x"], p["idx"], p["w"], *weights, d, p["ws"])
    assert torch.equal(c, d)
    assert moe.moe_read_status(p["ws"]) == moe.MOE_OK


def test_slots_without_an_expert_and_the_same_expert_twice():
    p = make(33, 256, 8, 3, 128, 7)
    p["idx"][::2, 1] = -1
    p["idx"][1::4, 2] = 99
    p["idx"][3, :] = 5
    p["idx"][4, :] = -1
    out = torch.full((33, 256), 7.0, dtype=torch.bfloat16, device="cuda")
    moe.moe_forward_routed(p["cfg"], p["x"], p["idx"], p["w"], p["wgu"], p["sgu"], p["wd"],
                           p["sd"], out, p["ws"])
    assert (out[4] == 0).all()
    want = torch.zeros(33, 256, dtype=torch.float64, device="cuda")
    for j in range(3):  # one slot at a time
        one = moe.config(33, 256, 8, 1, 128, fp8_block=True)
        o = torch.empty_like(out)
        moe.moe_forward_routed(one, p["x"], p["idx"][:, j].contiguous(),
                               torch.ones(33, 1, device="cuda"), p["wgu"], p["sgu"], p["wd"],
                               p["sd"], o, moe.workspace(one))
        want += o.double() * p["w"][:, j].double()[:, None]
    # the slots' y are the same bf16 values; fp32 sum of 3 terms, one bf16 rounding
    assert ((out.double() - want).abs() <= 2.0 ** -8 * want.abs() + 1e-5).all()


def test_layer_on_another_stream_with_its_own_workspace():
    p = make(64, 512, 16, 4, 256, 8)
    weights = (p["wgu"], p["sgu"], p["wd"], p["sd"])
    a, b = (torch.empty(64, 512, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    moe.moe_forward_routed(p["cfg"], p["x"], p["idx"], p["w"], *weights, a, p["ws"])
    ws2, st = moe.workspace(p["cfg"]), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(5):
        moe.moe_forward_routed(p["cfg"], p["x"], p["idx"], p["w"], *weights, b, ws2, stream=st)
        moe.moe_forward_routed(p["cfg"], p["x"], p["idx"], p["w"], *weights, a, p["ws"])
    torch.cuda.synchronize()
    assert torch.equal(a, b)


# The kernels that take many, up to 128, 64 and 32 rows a group on average, by the
# number of (empty) groups beside the one with rows.
@pytest.mark.parametrize("M", [1, 77, 300])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_a_row_has_the_same_bits_in_every_grouped_kernel(M, dtype):
    """Every kernel adds a row's blocks in order with one fused multiply-add each."""
    g = gen(M)
    N, K = 400, 912
    q, s = quantised(activations(g, M, K))
    w, v = ref.random_weight(g, N, K)
    outs = []
    for per_group in (200, 100, 20, 1):
        G = max(1, -(-M // per_group))
        if G > 256:
            G = 256
        if per_group == 1 and G < M:
            continue
        wq = torch.stack([w] + [torch.zeros_like(w)] * (G - 1))
        sw = torch.stack([v] + [torch.ones_like(v)] * (G - 1))
        offsets = torch.full((G + 1,), M, dtype=torch.int32, device="cuda")
        offsets[0] = 0
        outs.append(product(q, s, wq, sw, N, dtype, offsets))
    for o in outs[1:]:
        assert torch.equal(o, outs[0])


@pytest.mark.parametrize("counts", [[3, 5, 1, 7], [40, 33, 64, 2], [90, 100, 70, 128],
                                    [257, 200, 130, 300]])
def test_nan_rows_and_nan_weights_stay_in_their_group(counts):
    """A NaN row changes no other row, NaN weights of one group no other group."""
    g = gen(sum(counts))
    G, N, K = len(counts), 264, 400
    offsets = torch.tensor([0] + counts, device="cuda").cumsum(0).to(torch.int32)
    M = sum(counts)
    x = activations(g, M, K)
    ws = [ref.random_weight(g, N, K) for _ in range(G)]
    wq, sw = torch.stack([w for w, _ in ws]), torch.stack([v for _, v in ws])
    q, s = quantised(x)
    clean = product(q, s, wq, sw, N, offsets=offsets)
    bad = offsets[1:-1].tolist() + [M - 1]  # the first row of each later group, the last row
    x[bad] = float("nan")
    q, s = quantised(x)
    wq[2] = 0x7F
    out = product(q, s, wq, sw, N, offsets=offsets)
    keep = torch.ones(M, dtype=torch.bool, device="cuda")
    keep[bad] = False
    keep[offsets[2]:offsets[3]] = False
    assert torch.equal(out[keep], clean[keep])
    assert bool(torch.isnan(out[~keep]).all())


def test_a_nan_token_leaves_the_other_tokens_alone():
    p = make(200, 512, 16, 4, 256, 12)
    weights = (p["wgu"], p["sgu"], p["wd"], p["sd"])
    a, b = (torch.empty(200, 512, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    moe.moe_forward_routed(p["cfg"], p["x"], p["idx"], p["w"], *weights, a, p["ws"])
    p["x"][[0, 57, 199], 5] = float("nan")
    moe.moe_forward_routed(p["cfg"], p["x"], p["idx"], p["w"], *weights, b, p["ws"])
    keep = torch.ones(200, dtype=torch.bool, device="cuda")
    keep[[0, 57, 199]] = False
    assert torch.equal(a[keep], b[keep]) and bool(torch.isnan(b[~keep]).all())


@pytest.mark.parametrize("T,P", [(64, 2), (400, 4)])
def test_expert_parallel_ranks_equal_the_layer_on_one_gpu(T, P):
    """Ranks in lockstep on one GPU: bitwise moe_forward on each rank's tokens."""
    p = make(T, 512, 32, 4, 256, 13)
    wg = (torch.randn(32, 512, device="cuda", generator=gen(14)) * 0.05).to(torch.bfloat16)
    weights = (p["wgu"], p["sgu"], p["wd"], p["sd"])
    part = ep.Partition(32, P)
    ops = [ep.ep_layer_ops(p["cfg"], part, r, wg, None, *weights) for r in range(P)]
    xs = [x.contiguous() for x in torch.chunk(p["x"], P)]
    outs = ep.ep_forward_lockstep(ops, part, xs)
    for x, out in zip(xs, outs):
        cfg = moe.config(x.shape[0], 512, 32, 4, 256, fp8_block=True)
        ws, want = moe.workspace(cfg), torch.empty_like(x)
        moe.moe_forward(cfg, x, wg, None, *weights, want, ws)
        assert torch.equal(out, want) and moe.moe_read_status(ws) == moe.MOE_OK
