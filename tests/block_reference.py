"""64-bit definitions of the expert choice and of block-scaled FP8, written from
the formulas in include/moe.h (numpy for the choice, torch doubles for the rest)."""

import math

import numpy as np
import torch

FP8 = torch.float8_e4m3fn


def nblocks(n):
    return -(-n // 128)


# ------------------------------------------------------------------ choice

def score64(z, fn):
    z = np.asarray(z, np.float64)
    with np.errstate(over="ignore", invalid="ignore"):
        if fn == "sigmoid":
            return np.where(z >= 0, 1 / (1 + np.exp(-z)), np.exp(z) / (1 + np.exp(z)))
        if fn == "sqrtsoftplus":
            return np.sqrt(np.maximum(z, 0) + np.log1p(np.exp(-np.abs(z))))
    m = z.max()
    p = np.exp(z - m) if m > -math.inf else np.zeros_like(z)
    return p / p.sum() if p.sum() else p


def select_row(z, k, scale, fn="sigmoid", bias=None, groups=1, keep=1, by="max", renorm=True):
    """(experts, weights) of one token, one comparison at a time."""
    z = np.array(z, np.float64)
    z[np.isnan(z)] = -math.inf
    z = np.minimum(z, float(np.finfo(np.float32).max))
    s = score64(z, fn)
    s[z == -math.inf] = 0.0
    # increasing scores rank like their logits, also where fp64 scores saturate
    c = z.copy() if bias is None else s + np.asarray(bias, np.float64)
    c[z == -math.inf] = -math.inf
    v = s.copy() if bias is None else c.copy()
    v[z == -math.inf] = -math.inf
    n = len(z) // groups
    worth = []
    for g in range(groups):
        part = sorted((c if by == "max" else v)[g * n:(g + 1) * n], reverse=True)
        worth.append(part[0] if by == "max" else part[0] + part[1])
    best = sorted(range(groups), key=lambda g: (-worth[g], g))[:keep]
    allowed = [e for e in range(len(z)) if e // n in best]
    idx = sorted(allowed, key=lambda e: (-c[e], e))[:k]
    w = s[idx]
    if renorm:
        if fn != "softmax" and w.max() < 1e-30 and z[idx].max() > -math.inf:
            w = np.exp((z[idx] - z[idx].max()) * (1.0 if fn == "sigmoid" else 0.5))
        if fn == "softmax" and z[idx].max() > -math.inf:
            w = np.exp(z[idx] - z[idx].max())
        w = w / w.sum() if w.sum() > 0 else np.zeros_like(w)
    return np.array(idx, np.int32), scale * w


# ------------------------------------------------------------------ block FP8

def e4m3_64(v):
    m = v.abs().clamp(max=448.0)
    _, e = torch.frexp(m)
    step = torch.exp2((e.double() - 1).clamp(min=-6.0) - 3)
    return torch.sign(v) * torch.round(m / step) * step


def quant64(x):
    """(code values, amax) in doubles of x [M, K], amax [M, ceil(K/128)]."""
    M, K = x.shape
    pad = torch.zeros(M, nblocks(K) * 128, dtype=torch.float64, device=x.device)
    pad[:, :K] = x.double()
    v = pad.view(M, -1, 128)
    a = v.abs().amax(2)
    safe = torch.where(a == 0, 1.0, a)
    q = e4m3_64(v * 448.0 / safe.unsqueeze(2)).view(M, -1)[:, :K]
    return q, a


def values(q, s):
    """Doubles of row codes [M, K] with scales [M, ceil(K/128)]."""
    cols = torch.arange(q.shape[1], device=q.device) // 128
    return q.view(FP8).double() * s.double()[:, cols]


def weight_values(q, s):
    r = torch.arange(q.shape[0], device=q.device) // 128
    c = torch.arange(q.shape[1], device=q.device) // 128
    return q.view(FP8).double() * s.double()[r][:, c]


def random_weight(g, N, K, std=0.02):
    """[N, K] e4m3 codes (uint8) and [ceil(N/128), ceil(K/128)] scales."""
    w = torch.randn(nblocks(N) * 128, nblocks(K) * 128, generator=g, device="cuda") * std
    w = w.view(nblocks(N), 128, nblocks(K), 128)
    s = w.abs().amax(dim=(1, 3)) / 448.0
    q = (w / s[:, None, :, None]).to(FP8).view(torch.uint8)
    return q.view(nblocks(N) * 128, -1)[:N, :K].contiguous(), s


# The product's tolerance, relative to S = sum |x w| of the output's terms. The
# products of two e4m3 values are exact in fp32. Within a block of 128 columns
# 128 additions each lose at most 2^-23 of the running sum (a truncating fp32
# adder), the two scale multiplications and the addition over the blocks at
# most 2^-24 each.
def product_tol(K):
    return 128 * 2.0 ** -23 + (nblocks(K) + 3) * 2.0 ** -24


def check_product(out, xv, wv, what=""):
    """out against xv @ wv.T, element by element."""
    ref = xv @ wv.T
    s = xv.abs() @ wv.abs().T
    half = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}[out.dtype]
    tol = half * ref.abs() + product_tol(xv.shape[1]) * s * (1 + half) + 1e-38
    bad = (out.double() - ref).abs() > tol
    assert not bad.any(), (what, int(bad.sum()), bad.nonzero()[:4].tolist(),
                           float(((out.double() - ref).abs() / tol).max()))
