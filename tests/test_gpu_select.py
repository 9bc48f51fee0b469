"""The choice of experts (moe_select, moe_route4, moe_forward4) against its
64-bit definition, token by token.

Indices are equal. Weights: fp32 exponentials within 2 ulp, one division, a sum
of at most 32 terms: 4e-6 relative; a softmax's argument z - max is rounded
once, which adds its magnitude times 2^-24.
"""

import math

import numpy as np
import pytest
import torch

import block_reference as ref
from sparse_moe_transformer_gemm_b200 import build as moe_build
from sparse_moe_transformer_gemm_b200 import moe

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    moe_build.build()


def run(z, k, scale=2.826, fn="sigmoid", bias=None, groups=1, keep=1, by="max", renorm=True):
    T, E = z.shape
    cfg = moe.config(T, 128, E, k, 128, scale)
    idx = torch.full((T, k), -7, dtype=torch.int32, device="cuda")
    w = torch.full((T, k), math.nan, device="cuda")
    moe.moe_select(cfg, z, moe.route_options(bias, score_fn=fn),
                   moe.group_options(groups, keep, by, renorm), idx, w)
    return idx.cpu().numpy(), w.cpu().numpy()


def check(z, k, **kw):
    idx, w = run(z, k, **kw)
    bias = kw.pop("bias", None)
    zh = z.cpu().numpy()
    bh = None if bias is None else bias.cpu().numpy()
    kw.setdefault("scale", 2.826)
    for t in range(z.shape[0]):
        ei, ew = ref.select_row(zh[t], k, bias=bh, **kw)
        assert idx[t].tolist() == ei.tolist(), (t, idx[t], ei)
        tol = 4e-6
        if kw.get("fn") == "softmax":
            fin = zh[t][np.isfinite(zh[t])]
            tol += (float(fin.max() - fin.min()) if fin.size else 0.0) * 2.0 ** -24
        assert np.all(np.abs(w[t] - ew) <= tol * np.abs(ew) + 1e-37), (t, w[t], ew)


def logits(T, E, seed=0, std=1.28):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.randn(T, E, generator=g, device="cuda") * std


def bias_of(E, seed=1, std=0.05):
    return logits(1, E, seed, std)[0].contiguous()


@pytest.mark.parametrize("fn", ["sigmoid", "sqrtsoftplus", "softmax"])
@pytest.mark.parametrize("T,E,k,groups,keep,by", [
    (1, 1, 1, 1, 1, "max"),
    (64, 192, 8, 1, 1, "max"),
    (33, 256, 32, 1, 1, "max"),
    (257, 256, 8, 8, 4, "top2"),
    (97, 160, 6, 8, 3, "max"),
    (50, 60, 4, 3, 2, "top2"),      # 20 experts a group: not a power of two
    (50, 256, 5, 256, 6, "max"),    # groups of one expert
    (50, 254, 7, 127, 40, "top2"),  # groups of two, more than 32 of them
    (20, 48, 1, 16, 1, "max"),
    (5, 18, 18, 2, 2, "max"),
])
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("renorm", [True, False])
def test_choice(fn, T, E, k, groups, keep, by, bias, renorm):
    check(logits(T, E, E + k), k, fn=fn, bias=bias_of(E) if bias else None, groups=groups,
          keep=keep, by=by, renorm=renorm, scale=1.5)


@pytest.mark.parametrize("fn", ["sigmoid", "sqrtsoftplus", "softmax"])
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("groups,keep,by", [(1, 1, "max"), (4, 2, "max"), (4, 2, "top2")])
def test_equal_values_take_the_lower_index(fn, bias, groups, keep, by):
    z = torch.zeros(6, 64, device="cuda")
    z[1] = 3.0
    z[2, 40:] = 1.0
    z[3, ::2] = -2.0
    z[4] = torch.arange(64, device="cuda").float() // 16
    z[5] = 100.0  # saturated scores
    b = torch.full((64,), 0.25, device="cuda") if bias else None
    check(z, 8, fn=fn, bias=b, groups=groups, keep=keep, by=by)


@pytest.mark.parametrize("fn", ["sigmoid", "sqrtsoftplus", "softmax"])
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("groups,keep,by", [(1, 1, "max"), (4, 2, "max"), (4, 2, "top2")])
@pytest.mark.parametrize("renorm", [True, False])
def test_experts_that_are_out(fn, bias, groups, keep, by, renorm):
    """Rows with -inf, NaN and +inf, down to rows without any expert left."""
    z = logits(9, 32, 3)
    z[0, 5:] = -math.inf           # fewer left than k
    z[1, :] = -math.inf            # none left
    z[2, :] = math.nan
    z[3, 8:16] = -math.inf         # a whole group out
    z[4, 3] = math.nan
    z[5, :] = -math.inf
    z[5, 31] = -3.0
    z[6, 0::2] = -math.inf
    z[7, 9] = math.inf
    z[8, :] = float(torch.finfo(torch.float32).min)  # the type's lowest value is no mask
    check(z, 8, fn=fn, bias=bias_of(32, std=0.5) if bias else None, groups=groups, keep=keep,
          by=by, renorm=renorm)


def test_values_closer_than_fp32_resolves_keep_the_exact_order():
    """Biases that cancel the score differences to within 1e-9: the order is the
    64-bit one, in the choice, at its border and between groups."""
    E = 128
    z = logits(300, E, 11)
    s = ref.score64(z.cpu().numpy()[0], "sigmoid")
    b = torch.tensor((0.7 - s).astype(np.float32), device="cuda")  # row 0: all about 0.7
    z[1:] = z[0] + logits(299, E, 12, 1e-6)
    check(z, 8, bias=b)
    check(z, 8, bias=b, groups=8, keep=3, by="top2")
    check(z, 8, bias=b, groups=8, keep=3, by="max")
    check(z, 8, bias=b * 0.5, fn="softmax", groups=8, keep=3, by="max")


@pytest.mark.parametrize("fn", ["sigmoid", "sqrtsoftplus", "softmax"])
@pytest.mark.parametrize("k", [1, 2, 7, 8, 31, 32])
def test_pairs_closer_than_fp32_resolves_keep_the_exact_order(fn, k):
    """Pairs of experts whose choice values are within 1e-7 of each other and 0.02 from
    the next pair's: within the choice (k even) and across its border (k odd); rows
    0 to 9 have equal logits in a pair with equal biases."""
    E = 80
    z = logits(1, E, 13).repeat(200, 1)
    z[:, 1:20:2] = z[:, 0:20:2]
    s = (ref.score64(z.cpu().numpy()[0], fn) if fn != "softmax"
         else torch.softmax(z[0].double(), 0).cpu().numpy())
    pair = np.random.default_rng(3).permutation(E // 2).repeat(2)
    b = torch.tensor((0.02 * pair - s).astype(np.float32), device="cuda")
    z[10:] += logits(190, E, 14, 1e-7)
    check(z, k, fn=fn, bias=b)
    if k <= 10:
        check(z, k, fn=fn, bias=b, groups=8, keep=3, by="top2")
        check(z, k, fn=fn, bias=b, groups=8, keep=5, by="max", renorm=False)


@pytest.mark.parametrize("fn", ["sigmoid", "sqrtsoftplus", "softmax"])
def test_very_small_scores_renormalise(fn):
    z = logits(20, 40, 5) - 300.0
    check(z, 6, fn=fn)
    check(z * 0.3, 6, fn=fn)


def test_extreme_biases():
    z = logits(10, 64, 6)
    b = bias_of(64)
    b[3], b[10], b[20] = math.inf, -math.inf, 1e30
    idx, w = run(z, 8, bias=b)
    assert np.all(idx[:, 0] == 3) and np.all(idx[:, 1] == 20)
    assert not np.any(idx == 10) and np.all(np.isfinite(w))
    b[5] = math.nan
    assert not np.any(run(z, 8, bias=b)[0] == 5)


def test_strided_rows_and_untouched_neighbours():
    wide = torch.full((41, 200), 50.0, device="cuda")
    wide[:, 3:99] = logits(41, 96, 8)
    view = wide[:, 3:99]
    idx, w = run(view, 8)
    idx2, w2 = run(view.contiguous(), 8)
    assert np.array_equal(idx, idx2) and np.array_equal(w, w2)


def test_rows_past_two_to_the_31_elements():
    """Row 5 begins 2.7e9 logits behind row 0."""
    ld = 1 << 29
    z = torch.empty(5 * ld + 64, device="cuda")
    rows = torch.as_strided(z, (6, 64), (ld, 1))
    rows.copy_(logits(6, 64, 40))
    check(rows, 6, fn="softmax")
    check(rows, 6, bias=bias_of(64), groups=4, keep=2, by="top2")


def test_whole_batch_of_a_long_prefill_agrees_with_sorted_logits():
    z = logits(16384, 192, 9)
    idx, w = run(z, 8)
    want = (-z).sort(dim=1, stable=True)[1][:, :8].cpu().numpy()
    assert np.array_equal(idx, want)
    assert np.allclose(w.sum(1), 2.826, rtol=1e-5)


def test_captured_call_replays_on_new_logits():
    z = logits(64, 192, 20)
    cfg = moe.config(64, 128, 192, 8, 128)
    idx = torch.empty(64, 8, dtype=torch.int32, device="cuda")
    w = torch.empty(64, 8, device="cuda")
    moe.moe_select(cfg, z, None, None, idx, w)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.moe_select(cfg, z, None, None, idx, w)
    z.copy_(logits(64, 192, 21))
    graph.replay()
    torch.cuda.synchronize()
    want, ww = run(z, 8)
    assert np.array_equal(idx.cpu().numpy(), want) and np.array_equal(w.cpu().numpy(), ww)


# ------------------------------------------------------------------ behind the router

@pytest.mark.parametrize("T,E,k,d", [(7, 48, 4, 256), (64, 192, 8, 512), (300, 64, 8, 512),
                                     (200, 40, 12, 256)])
@pytest.mark.parametrize("norm", [False, True])
def test_route4_is_the_choice_from_the_routers_logits(T, E, k, d, norm):
    """Integer-valued x and w (route_norm: a power-of-two rms): the logits are
    exact in fp32 whatever the order of the sums, so the choice is the
    definition's on logits computed apart."""
    g = torch.Generator(device="cuda")
    g.manual_seed(T + E)
    x = torch.randint(-2, 3, (T, d), generator=g, device="cuda").to(torch.bfloat16)
    if norm:
        x = torch.where(torch.rand(T, d, generator=g, device="cuda") < 0.5, 1.0, -1.0).to(torch.bfloat16)
    wg = (torch.randint(-3, 4, (E, d), generator=g, device="cuda") / 64).to(torch.bfloat16)
    gb = (torch.randint(-8, 9, (E,), generator=g, device="cuda") / 4).float()
    sb = bias_of(E)
    nw = torch.ones(d, device="cuda") if norm else None
    z = (x.float() @ wg.float().T) + gb
    cfg = moe.config(T, d, E, k, 128)
    ws = moe.workspace(cfg)
    idx = torch.empty(T, k, dtype=torch.int32, device="cuda")
    w = torch.empty(T, k, device="cuda")
    for fn, grp in (("softmax", moe.group_options(4, 3, "max", False)),
                    ("sigmoid", moe.group_options(4, 2 if E // 2 >= k else 4, "top2", True))):
        # mean(x^2) + eps = 1 for the +-1 rows: eps is below fp32's resolution of 1
        opt = moe.route_options(sb, nw, 1e-9, fn)
        moe.moe_route4(cfg, x, wg, gb, opt, grp, idx, w, ws)
        idx2, w2 = run(z, k, fn=fn, bias=sb, groups=4, keep=grp.topk_group,
                       by="max" if fn == "softmax" else "top2", renorm=fn == "sigmoid")
        assert np.array_equal(idx.cpu().numpy(), idx2)
        assert np.allclose(w.cpu().numpy(), w2, rtol=4e-6, atol=0)
        assert moe.moe_read_status(ws) == moe.MOE_OK


@pytest.mark.parametrize("T", [5, 300])
def test_forward4_without_options_is_forward3_and_forward_routed(T):
    """No groups, sigmoid, renormalised: the layer's own choice, so the same layer."""
    from synthetic import LayerShape, make_layer

    layer = make_layer(LayerShape(T=T, d=512, E=32, k=4, F=256), seed=2, device="cuda")
    cfg = moe.config_of(layer["cfg"])
    ws = moe.workspace(cfg)
    args = moe.layer_args(layer)
    outs = [torch.empty(T, 512, dtype=torch.bfloat16, device="cuda") for _ in range(3)]
    moe.moe_forward(cfg, layer["x"], layer["w_gate"], None, *args, outs[0], ws)
    moe.moe_forward4(cfg, layer["x"], layer["w_gate"], None, None, None, *args, outs[1], ws)
    idx = torch.empty(T, 4, dtype=torch.int32, device="cuda")
    w = torch.empty(T, 4, device="cuda")
    moe.moe_route(cfg, layer["x"], layer["w_gate"], None, idx, w, ws)
    moe.moe_forward_routed(cfg, layer["x"], idx, w, *args, outs[2], ws)
    torch.cuda.synchronize()
    assert torch.equal(outs[0], outs[2])
    # the weights' last bits may differ (another sum order): bf16 neighbours
    a, b = outs[0].double(), outs[1].double()
    assert ((a - b).abs() <= 2.0 ** -7 * a.abs() + 1e-6).all()
    assert moe.moe_read_status(ws) == moe.MOE_OK
