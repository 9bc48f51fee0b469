"""Cases and plain forms of the block-scaled FP8 and expert-choice operators.

Four operators: the choice of experts from router logits (``select``), the
quantisation of activation rows to e4m3 with a scale per 128 columns
(``quant``), the FP8 matrix product with a scale per block of 128 (``gemm``)
and the SwiGLU experts of a routed-MoE layer on it (``experts``: group,
quantise, gate_up, SwiGLU, quantise, down, weighted sum). ``run`` computes them
with elementary torch operations, or calls the library where ``own`` is true.
"""

import math

import torch

own = False

B = 128            # columns (and weight rows) per scale
FP8 = torch.float8_e4m3fn
FP8_MAX = 448.0


def listed():
    hy3 = dict(d=4096, E=192, k=8, F=1536)
    return [
        # the choice for one decode batch of the Hy3 router (latency)
        dict(name="select decode", op="select", T=64, E=192, k=8, fn="sigmoid", bias=True,
             groups=1, keep=1, by="max", renorm=True, scale=2.826, masked=0),
        # a long prefill over 256 experts in 8 groups, 4 kept by their two best
        dict(name="select grouped prefill", op="select", T=16384, E=256, k=8, fn="sigmoid",
             bias=True, groups=8, keep=4, by="top2", renorm=True, scale=2.5, masked=0),
        # softmax scores without renormalisation, groups by their best expert, 3 experts
        # taken out of service, a ragged batch
        dict(name="select softmax", op="select", T=4099, E=160, k=6, fn="softmax", bias=False,
             groups=8, keep=3, by="max", renorm=False, scale=1.0, masked=3),
        # activations of a decode batch, and of the longest prefill batch
        dict(name="quant decode", op="quant", M=64, K=4096),
        dict(name="quant prefill", op="quant", M=16384, K=4096),
        # a projection for one token, for a ragged decode batch, for a long prefill
        dict(name="gemm one token", op="gemm", M=1, N=4096, K=4096),
        dict(name="gemm ragged", op="gemm", M=77, N=7000, K=2064),
        dict(name="gemm prefill", op="gemm", M=8192, N=8192, K=4096),
        # the Hy3 layer's experts: one token, decode, prefill, a large skewed prefill
        dict(name="experts one token", op="experts", T=1, skew=0.0, **hy3),
        dict(name="experts decode", op="experts", T=64, skew=0.0, **hy3),
        dict(name="experts prefill", op="experts", T=4096, skew=0.0, **hy3),
        dict(name="experts skewed", op="experts", T=8192, skew=0.5, **hy3),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["select", "quant", "gemm", "experts"])
    if op == "select":
        groups = rng.choice([1, 1, 2, 4, 8])
        per = rng.randint(2, 256 // groups)
        keep = rng.randint(1, groups)
        by = rng.choice(["max", "top2"]) if groups > 1 else "max"
        return dict(op=op, T=_log_int(rng, 1, 16384), E=groups * per,
                    k=rng.randint(1, min(16, keep * per)),
                    fn=rng.choice(["sigmoid", "sqrtsoftplus", "softmax"]),
                    bias=rng.random() < 0.6, groups=groups, keep=keep, by=by,
                    renorm=rng.random() < 0.7, scale=rng.choice([1.0, 1.5, 2.5, 2.826]),
                    masked=rng.choice([0, 0, 1, per]))
    if op == "quant":
        return dict(op=op, M=_log_int(rng, 1, 16384), K=16 * rng.randint(1, 256))
    if op == "gemm":
        return dict(op=op, M=_log_int(rng, 1, 8192), N=_log_int(rng, 64, 8192),
                    K=16 * rng.randint(8, 256))
    return dict(op=op, T=_log_int(rng, 1, 8192), skew=round(rng.uniform(0.0, 0.5), 2),
                d=128 * rng.randint(2, 32), E=_log_int(rng, 8, 192), k=rng.randint(1, 8),
                F=128 * rng.randint(1, 12))


# ------------------------------------------------------------------ inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _activations(g, M, K):
    """Rows of unit variance with a few columns that are much larger, as hidden states have."""
    x = torch.randn(M, K, generator=g, device="cuda")
    x[:, :: 97] *= 8.0
    return x.to(torch.bfloat16)


def _blocks(n):
    return (n + B - 1) // B


def _weight(g, N, K):
    """[N, K] N(0, 0.02^2) as e4m3 codes (uint8) with an fp32 scale per 128 x 128 block."""
    w = torch.randn(_blocks(N) * B, _blocks(K) * B, generator=g, device="cuda").mul_(0.02)
    w = w.view(_blocks(N), B, _blocks(K), B)
    s = w.abs().amax(dim=(1, 3)) / FP8_MAX
    q = (w / s[:, None, :, None]).to(FP8).view(torch.uint8)
    return q.view(_blocks(N) * B, -1)[:N, :K].contiguous(), s


def _choices(g, T, E, k, skew):
    """A routing as a router gives it: per token k distinct experts, best first, and weights."""
    z = torch.randn(T, E, generator=g, device="cuda") * 1.28
    z -= skew * torch.log(torch.arange(1, E + 1, device="cuda", dtype=torch.float32))
    s, idx = torch.sigmoid(z).topk(k, dim=1)
    return idx.to(torch.int32), (2.826 * s / s.sum(1, keepdim=True)).contiguous()


def prepare(case, seed):
    g = _gen(seed)
    st = dict(case)
    op = case["op"]
    if op == "select":
        T, E = case["T"], case["E"]
        st["logits"] = torch.randn(T, E, generator=g, device="cuda") * 1.28
        if case["masked"]:
            out = torch.randperm(E, generator=g, device="cuda")[: min(case["masked"], E - 1)]
            st["logits"][:, out] = -math.inf
        st["sbias"] = torch.randn(E, generator=g, device="cuda") * 0.05 if case["bias"] else None
        st["idx"] = torch.empty(T, case["k"], dtype=torch.int32, device="cuda")
        st["w"] = torch.empty(T, case["k"], device="cuda")
    elif op == "quant":
        M, K = case["M"], case["K"]
        st["x"] = _activations(g, M, K)
        st["q"] = torch.empty(M, K, dtype=torch.uint8, device="cuda")
        st["s"] = torch.empty(M, _blocks(K), device="cuda")
    elif op == "gemm":
        M, N, K = case["M"], case["N"], case["K"]
        st["xq"], st["sx"] = _quantised(_activations(g, M, K))
        st["wq"], st["sw"] = _weight(g, N, K)
        st["out"] = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
    else:
        T, d, E, F, k = (case[n] for n in ("T", "d", "E", "F", "k"))
        st["x"] = _activations(g, T, d)
        k = st["k"] = min(k, E)
        st["idx"], st["w"] = _choices(g, T, E, k, case["skew"])
        st["wgu"] = torch.empty(E, 2 * F, d, dtype=torch.uint8, device="cuda")
        st["sgu"] = torch.empty(E, 2 * F // B, d // B, device="cuda")
        st["wd"] = torch.empty(E, d, F, dtype=torch.uint8, device="cuda")
        st["sd"] = torch.empty(E, d // B, F // B, device="cuda")
        for e in range(E):
            st["wgu"][e], st["sgu"][e] = _weight(g, 2 * F, d)
            st["wd"][e], st["sd"][e] = _weight(g, d, F)
        # the experts in use, and the rows of the busiest one
        st["used"], rows = st["idx"].long().unique(return_counts=True)
        st["rows"] = int(rows.max())
        st["out"] = torch.empty(T, d, dtype=torch.bfloat16, device="cuda")
    _handles(st)
    return st


def _quantised(x):
    """e4m3 codes (uint8) and scales of an activation that the gemm cases start from."""
    q, s = _quant_plain(x)
    return q.view(torch.uint8), s


# ------------------------------------------------------------------ the library's calls

def _handles(st):
    """What a program keeps for its calls: configurations, options and the workspace."""
    if not own:
        return
    from sparse_moe_transformer_gemm_b200 import moe

    if st["op"] == "select":
        st["cfg"] = moe.config(st["T"], 128, st["E"], st["k"], 128, st["scale"])
        st["opt"] = moe.route_options(st["sbias"], score_fn=st["fn"])
        st["grp"] = moe.group_options(st["groups"], st["keep"], st["by"], st["renorm"])
    elif st["op"] == "gemm":
        st["ws"] = moe.block_workspace(st["M"], st["N"], st["K"])
    elif st["op"] == "experts":
        st["cfg"] = moe.config(st["T"], st["d"], st["E"], st["k"], st["F"], fp8_block=True)
        st["ws"] = moe.workspace(st["cfg"])


def _run_own(st):
    from sparse_moe_transformer_gemm_b200 import moe

    if st["op"] == "select":
        moe.moe_select(st["cfg"], st["logits"], st["opt"], st["grp"], st["idx"], st["w"])
        return st["idx"], st["w"]
    if st["op"] == "quant":
        moe.moe_block_quant(st["x"], st["q"], st["s"])
        return st["q"].view(FP8), st["s"]
    if st["op"] == "gemm":
        moe.moe_block_gemm(st["xq"], st["sx"], st["wq"], st["sw"], st["out"], st["ws"])
        return st["out"]
    moe.moe_forward_routed(st["cfg"], st["x"], st["idx"], st["w"], st["wgu"], st["sgu"],
                           st["wd"], st["sd"], st["out"], st["ws"])
    return st["out"]


# ------------------------------------------------------------------ plain forms

def _quant_plain(x):
    """e4m3(448 x / a) and a / 448 with a the largest magnitude of a row's 128 columns."""
    M, K = x.shape
    v = torch.nn.functional.pad(x.float(), (0, _blocks(K) * B - K)).view(M, -1, B)
    a = v.abs().amax(2, keepdim=True)
    s = torch.where(a == 0, 1.0, a / FP8_MAX)
    q = torch.where(a == 0, 0.0, v * FP8_MAX / a).to(FP8)
    return q.view(M, -1)[:, :K].contiguous(), s[..., 0]


def _dequant_rows(q, s):
    return q.view(FP8).float() * s.repeat_interleave(B, -1)[..., : q.shape[-1]]


def _dequant_weight(q, s):
    N, K = q.shape[-2:]
    if N % B or K % B:
        return q.view(FP8).float() * s.repeat_interleave(B, -2).repeat_interleave(B, -1)[..., :N, :K]
    w = q.view(FP8).float().view(*q.shape[:-2], N // B, B, K // B, B)
    return w.mul_(s.unsqueeze(-1).unsqueeze(-3)).view(*q.shape)


def _select_plain(st):
    # in 64 bits: values next to the border of the choice
    z, T, E, k = st["logits"].double(), st["T"], st["E"], st["k"]
    if st["fn"] == "sigmoid":
        s = 1.0 / (1.0 + torch.exp(-z))
    elif st["fn"] == "softmax":
        p = torch.exp(z - z.amax(1, keepdim=True))
        s = p / p.sum(1, keepdim=True)
    else:
        s = torch.sqrt(torch.clamp(z, min=0.0) + torch.log1p(torch.exp(-z.abs())))
    c = s + st["sbias"].double() if st["sbias"] is not None else s
    c = torch.where(z == -math.inf, -math.inf, c)
    G = st["groups"]
    best = c.view(T, G, E // G).sort(dim=2, descending=True)[0]
    of_group = best[..., 0] if st["by"] == "max" else best[..., 0] + best[..., 1]
    kept = (-of_group).sort(dim=1, stable=True)[1][:, : st["keep"]]
    allowed = torch.zeros(T, G, dtype=torch.bool, device=z.device).scatter_(1, kept, True)
    allowed = allowed.repeat_interleave(E // G, 1)
    # experts outside the kept groups come after every kept one, masked ones included
    order = (-c).sort(dim=1, stable=True)[1]
    order = order.gather(1, (~allowed.gather(1, order)).int().sort(dim=1, stable=True)[1])
    idx = order[:, :k]
    w = s.gather(1, idx)
    if st["renorm"]:
        total = w.sum(1, keepdim=True)
        w = torch.where(total == 0, 0.0, w / total)
    return idx.to(torch.int32), (st["scale"] * w).float()


def _experts_plain(st):
    T, d, k, F, R, used = st["T"], st["d"], st["k"], st["F"], st["rows"], st["used"]
    E = used.numel()
    x = _dequant_rows(*_quant_plain(st["x"]))
    e = torch.searchsorted(used, st["idx"].flatten().long())
    order = e.sort(stable=True)[1]
    first = torch.cumsum(torch.bincount(e, minlength=E), 0) - torch.bincount(e, minlength=E)
    place = torch.empty_like(e)
    place[order] = torch.arange(T * k, device=e.device) - first[e[order]]
    at = e * R + place                       # a row of its own in [E, R] for every token-slot
    xs = torch.zeros(E * R, d, device=x.device)
    xs[at] = x.repeat_interleave(k, 0)
    gu = torch.bmm(xs.view(E, R, d), _dequant_weight(st["wgu"][used], st["sgu"][used]).transpose(1, 2))
    gate, up = gu[..., :F], gu[..., F:]
    h = (gate / (1.0 + torch.exp(-gate)) * up).view(E * R, F)
    hq = _dequant_rows(*_quant_plain(h)).view(E, R, F)
    y = torch.bmm(hq, _dequant_weight(st["wd"][used], st["sd"][used]).transpose(1, 2)).view(E * R, d)
    return (y[at].view(T, k, d) * st["w"].unsqueeze(2)).sum(1).to(torch.bfloat16)


def run(state):
    if own:
        return _run_own(state)
    op = state["op"]
    if op == "select":
        return _select_plain(state)
    if op == "quant":
        return _quant_plain(state["x"])
    if op == "gemm":
        x = _dequant_rows(state["xq"], state["sx"])
        return (x @ _dequant_weight(state["wq"], state["sw"]).T).to(torch.bfloat16)
    return _experts_plain(state)


# ------------------------------------------------------------------ work and the definition

def work(case):
    op = case["op"]
    if op == "select":
        T, E, k = case["T"], case["E"], case["k"]
        return {"bytes": 4 * T * E + 8 * T * k, "flops": 12 * T * E}
    if op == "quant":
        M, K = case["M"], case["K"]
        return {"bytes": 3 * M * K + 4 * M * _blocks(K), "flops": 3 * M * K}
    if op == "gemm":
        M, N, K = case["M"], case["N"], case["K"]
        kb = _blocks(K)
        return {"bytes": M * K + N * K + 4 * kb * (M + _blocks(N)) + 2 * M * N,
                "flops": 2 * M * N * K}
    T, d, E, F, k = (case[n] for n in ("T", "d", "E", "F", "k"))
    k = min(k, E)
    touched = E * (1.0 - (1.0 - k / E) ** T)
    return {"bytes": touched * 3 * d * F * (1 + 4 / B ** 2) + 4 * T * d + 8 * T * k,
            "flops": 6 * T * k * d * F}


def _e4m3_64(v):
    """The nearest e4m3 value (ties to even), in 64 bits."""
    m = v.abs().clamp(max=FP8_MAX)
    _, e = torch.frexp(m)                                   # m in [2^(e-1), 2^e)
    step = torch.exp2((e.double() - 1).clamp(min=-6.0) - 3)
    return torch.sign(v) * torch.round(m / step) * step


def _block_amax_64(v):
    """Per column: the largest magnitude of its row's block."""
    M, K = v.shape
    cols = torch.arange(K, device=v.device) // B
    a = torch.zeros(M, _blocks(K), dtype=torch.float64, device=v.device)
    a.scatter_reduce_(1, cols.expand(M, K), v.abs(), "amax")
    return a, a[:, cols]


def _requantised_64(v):
    a, per = _block_amax_64(v)
    safe = torch.where(per == 0, 1.0, per)
    return _e4m3_64(v * FP8_MAX / safe) * safe / FP8_MAX


def _weight_64(q, s):
    r = torch.arange(q.shape[0], device=q.device) // B
    c = torch.arange(q.shape[1], device=q.device) // B
    return q.view(FP8).double() * s.double()[r][:, c]


def _select_64(st):
    z = st["logits"].double()
    if st["fn"] == "softmax":
        s = torch.softmax(z, 1)
    elif st["fn"] == "sigmoid":
        s = torch.special.expit(z)
    else:
        s = torch.logaddexp(z, torch.zeros_like(z)).sqrt()
    c = s.clone() if st["sbias"] is None else s + st["sbias"].double()
    c[z == -math.inf] = -math.inf
    T, E = z.shape
    G, n = st["groups"], E // st["groups"]
    value = torch.stack([c[:, g * n:(g + 1) * n].topk(2 if st["by"] == "top2" else 1, 1)[0].sum(1)
                         for g in range(G)], 1)
    # rank of a group: the number of groups that are better, or equal and before it
    g = torch.arange(G, device=z.device)
    ahead = (value[:, None, :] > value[:, :, None]) | (
        (value[:, None, :] == value[:, :, None]) & (g[None, None, :] < g[None, :, None]))
    in_kept = (ahead.sum(2) < st["keep"]).repeat_interleave(n, 1)
    idx, left = [], in_kept.clone()
    for _ in range(st["k"]):
        top = torch.where(left, c, -math.inf).amax(1, keepdim=True)
        hit = left & (c == top)
        j = hit.int().argmax(1, keepdim=True)               # the first expert that holds it
        idx.append(j)
        left.scatter_(1, j, False)
    idx = torch.cat(idx, 1)
    w = s.gather(1, idx)
    if st["renorm"]:
        w = (w / w.sum(1, keepdim=True)).nan_to_num(0.0)
    return idx.to(torch.int32), st["scale"] * w


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "select":
        return _select_64(st)
    if op == "quant":
        x = st["x"].double()
        a, per = _block_amax_64(x)
        q = _e4m3_64(x * FP8_MAX / torch.where(per == 0, 1.0, per))
        return q, torch.where(a == 0, 1.0, a / FP8_MAX)
    if op == "gemm":
        cols = torch.arange(case["K"], device="cuda") // B
        x = st["xq"].view(FP8).double() * st["sx"].double()[:, cols]
        return x @ _weight_64(st["wq"], st["sw"]).T
    T, d, E, F = (case[n] for n in ("T", "d", "E", "F"))
    x = _requantised_64(st["x"].double())
    out = torch.zeros(T, d, dtype=torch.float64, device="cuda")
    for e in range(E):
        t, j = (st["idx"] == e).nonzero(as_tuple=True)
        if t.numel() == 0:
            continue
        gu = x[t] @ _weight_64(st["wgu"][e], st["sgu"][e]).T
        h = _requantised_64(torch.nn.functional.silu(gu[:, :F]) * gu[:, F:])
        y = h @ _weight_64(st["wd"][e], st["sd"][e]).T
        out.index_add_(0, t, y * st["w"][t, j].double()[:, None])
    return out
