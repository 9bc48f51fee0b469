"""Refusals of the expert-choice and block-FP8 entry points, before any launch
(no GPU), and their structures against the header."""

import ctypes
import os
import re

import pytest
import torch

from sparse_moe_transformer_gemm_b200 import build as moe_build
from sparse_moe_transformer_gemm_b200 import moe

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = ctypes.c_void_p
FAKE = 0x10000000  # never dereferenced: the checks come first
HY3 = dict(T=64, d=4096, E=192, k=8, d_ff=1536)


@pytest.fixture(scope="module", autouse=True)
def lib():
    moe_build.build()
    return moe.lib()


def call(name, *args):
    return getattr(moe.lib(), name)(*args)


def select(cfg, opt=None, grp=None, logits=FAKE, ld=None, idx=FAKE):
    return call("moe_select", ctypes.byref(cfg), P(logits) if logits else None,
                cfg.E if ld is None else ld, moe._opt(opt), moe._opt(grp),
                P(idx) if idx else None, P(FAKE), None)


def test_constants_and_structs_match_the_header():
    text = open(os.path.join(ROOT, "include", "moe.h")).read()
    for name, value in (("MOE_FLAG_FP8_BLOCK", r"(0x[0-9a-f]+)u"), ("MOE_SCORE_SOFTMAX", r"(\d+)"),
                        ("MOE_GROUP_MAX", r"(\d+)"), ("MOE_GROUP_TOP2", r"(\d+)"),
                        ("MOE_OUT_BF16", r"(\d+)"), ("MOE_OUT_F32", r"(\d+)")):
        m = re.search(r"#define %s %s" % (name, value), text)
        assert m and int(m.group(1), 0) == getattr(moe, name), name
    body = re.search(r"typedef struct moe_group_options \{(.*?)\} moe_group_options;", text,
                     re.S).group(1)
    assert re.findall(r"(\w+);", body) == [f for f, _ in moe.MoeGroupOptions._fields_]
    assert ctypes.sizeof(moe.MoeGroupOptions) == 16


def test_select_refusals():
    cfg = moe.config(**HY3)
    bad_arg, bad_shape = moe.MOE_ERR_INVALID_ARG, moe.MOE_ERR_UNSUPPORTED_SHAPE
    assert select(cfg, logits=0) == bad_arg
    assert select(cfg, idx=0) == bad_arg
    assert select(cfg, ld=191) == bad_arg
    assert select(cfg, moe.MoeRouteOptions(None, FAKE, 1e-6, 0)) == bad_arg  # route_norm
    assert select(cfg, moe.MoeRouteOptions(None, None, 0.0, 3)) == bad_arg
    assert select(cfg, moe.MoeRouteOptions(None, None, 0.0, -1)) == bad_arg
    G = moe.MoeGroupOptions
    assert select(cfg, grp=G(8, 4, 2, 1)) == bad_arg
    assert select(cfg, grp=G(8, 4, 0, 2)) == bad_arg
    for n, keep in ((0, 1), (5, 1), (193, 1), (8, 0), (8, 9), (-8, 1)):
        assert select(cfg, grp=G(n, keep, 0, 1)) == bad_shape, (n, keep)
    assert select(cfg, grp=G(32, 1, 0, 1)) == bad_shape       # 6 experts for k = 8
    assert select(cfg, grp=G(192, 8, 1, 1)) == bad_shape      # two best of one expert
    cfg.T = 0
    assert select(cfg) == bad_shape


def test_routing_entry_points_check_their_options():
    cfg = moe.config(**HY3)
    n = moe.moe_workspace_size(cfg)
    soft = moe.route_options(score_fn="softmax")
    bad = moe.MoeGroupOptions(7, 1, 0, 1)
    a = (P(FAKE), P(FAKE), None)
    rc = call("moe_route4", ctypes.byref(cfg), *a, ctypes.byref(soft), ctypes.byref(bad), P(FAKE),
              P(FAKE), P(FAKE), n, None)
    assert rc == moe.MOE_ERR_UNSUPPORTED_SHAPE
    rc = call("moe_forward4", ctypes.byref(cfg), *a, ctypes.byref(soft), ctypes.byref(bad),
              P(FAKE), None, P(FAKE), None, P(FAKE), P(FAKE), n, None)
    assert rc == moe.MOE_ERR_UNSUPPORTED_SHAPE
    # softmax stays refused where the choice is fused into the router
    rc = call("moe_route3", ctypes.byref(cfg), *a, ctypes.byref(soft), P(FAKE), P(FAKE), P(FAKE),
              n, None)
    assert rc == moe.MOE_ERR_INVALID_ARG
    rc = call("moe_route4", ctypes.byref(cfg), *a, None, None, P(FAKE), P(FAKE), P(FAKE), n - 256,
              None)
    assert rc == moe.MOE_ERR_WORKSPACE
    rc = call("moe_forward_routed", ctypes.byref(cfg), P(FAKE), None, P(FAKE), P(FAKE), None,
              P(FAKE), None, P(FAKE), P(FAKE), n, None)
    assert rc == moe.MOE_ERR_INVALID_ARG


def test_block_flag_rules():
    assert moe.moe_workspace_size(moe.config(**HY3, fp8_block=True)) > 0
    assert moe.moe_workspace_size(moe.config(**HY3, fp8_block=True, path="gemm")) > 0
    assert moe.moe_workspace_size(moe.config(**HY3, fp8_block=True, shared=True)) > 0
    for bad in (dict(fp8=True), dict(fp4=True), dict(packed=True), dict(path="stream")):
        assert moe.moe_workspace_size(moe.config(**HY3, fp8_block=True, **bad)) == 0, bad
    cfg = moe.config(**HY3, fp8_block=True)
    n = moe.moe_workspace_size(cfg)
    c = ctypes.byref(cfg)
    for rc in (
            call("moe_expert_gate_up", c, P(FAKE), P(FAKE), P(FAKE), P(FAKE), P(FAKE), P(FAKE), n,
                 None),
            call("moe_expert_gate_up_gather", c, P(FAKE), P(FAKE), P(FAKE), P(FAKE), P(FAKE),
                 P(FAKE), P(FAKE), n, None),
            call("moe_expert_down", c, P(FAKE), P(FAKE), P(FAKE), P(FAKE), P(FAKE), P(FAKE), n,
                 None),
            call("moe_pack_weights", c, 0, P(FAKE), P(FAKE << 8), None),
            # scales missing, and misaligned
            call("moe_block_down", c, P(FAKE), P(FAKE), P(FAKE), P(FAKE), None, P(FAKE), P(FAKE),
                 n, None),
            call("moe_block_down", c, P(FAKE), P(FAKE), P(FAKE), P(FAKE), P(FAKE + 4), P(FAKE),
                 P(FAKE), n, None),
            call("moe_block_gate_up", c, None, P(FAKE), P(FAKE), P(FAKE), P(FAKE), P(FAKE),
                 P(FAKE), P(FAKE), n, None),
            call("moe_block_permute", c, P(FAKE), None, P(FAKE), P(FAKE), None)):
        assert rc == moe.MOE_ERR_INVALID_ARG
    plain = moe.config(**HY3)
    assert call("moe_block_permute", ctypes.byref(plain), P(FAKE), P(FAKE), P(FAKE), P(FAKE),
                None) == moe.MOE_ERR_INVALID_ARG
    rc = call("moe_block_down", c, P(FAKE), P(FAKE), P(FAKE), P(FAKE), P(FAKE), P(FAKE), P(FAKE),
              n - 256, None)
    assert rc == moe.MOE_ERR_WORKSPACE


def gemm(G=1, M=8, N=256, K=256, offsets=0, xq=FAKE, out=FAKE, out_type=0, ws=FAKE, n=None):
    n = moe.lib().moe_block_workspace_size(G, M, N, K) if n is None else n
    return call("moe_block_gemm", P(xq) if xq else None, P(FAKE), P(FAKE), P(FAKE),
                P(offsets) if offsets else None, G, M, N, K, P(out) if out else None, out_type,
                P(ws) if ws else None, n, None)


def test_block_gemm_refusals():
    for bad in (dict(G=0), dict(G=257), dict(M=-1), dict(M=(1 << 24) + 1), dict(N=0),
                dict(N=(1 << 17) + 1), dict(K=0), dict(K=8), dict(K=264), dict(K=1 << 18),
                dict(G=256, N=1 << 23)):
        assert gemm(**bad, n=1 << 20, offsets=FAKE) == moe.MOE_ERR_UNSUPPORTED_SHAPE, bad
    for bad in (dict(xq=0), dict(xq=FAKE + 8), dict(out=0), dict(out=FAKE + 2), dict(ws=0),
                dict(ws=FAKE + 128), dict(out_type=2), dict(G=2)):
        assert gemm(**bad) == moe.MOE_ERR_INVALID_ARG, bad
    assert gemm(n=0) == moe.MOE_ERR_WORKSPACE
    assert moe.lib().moe_block_workspace_size(1, 8, 256, 264) == 0
    # nothing to do: accepted without looking at the pointers
    assert gemm(M=0, xq=0, out=0, ws=0) == moe.MOE_OK


def test_block_quant_refusals():
    def quant(M=4, K=256, ldx=256, x=FAKE, codes=FAKE, scales=FAKE):
        return call("moe_block_quant", P(x) if x else None, ldx, M, K, P(codes) if codes else None,
                    P(scales) if scales else None, None)

    for bad in (dict(K=8), dict(K=264, ldx=272), dict(M=-1), dict(K=1 << 18, ldx=1 << 18)):
        assert quant(**bad) == moe.MOE_ERR_UNSUPPORTED_SHAPE, bad
    for bad in (dict(ldx=240), dict(ldx=264), dict(x=0), dict(x=FAKE + 8), dict(codes=0),
                dict(codes=FAKE + 4), dict(scales=0)):
        assert quant(**bad) == moe.MOE_ERR_INVALID_ARG, bad
    assert quant(M=0, x=0, codes=0, scales=0) == moe.MOE_OK


def test_binding_checks_shapes_and_types():
    f8 = lambda *s: torch.zeros(*s, dtype=torch.uint8)  # noqa: E731
    ws = torch.zeros(256, dtype=torch.uint8)
    ok = dict(xq=f8(4, 256), sx=torch.zeros(4, 2), wq=f8(128, 256), sw=torch.zeros(1, 2),
              out=torch.zeros(4, 128, dtype=torch.bfloat16), ws=ws)
    for bad in (dict(sx=torch.zeros(4, 1)), dict(sw=torch.zeros(2, 2)), dict(wq=f8(128, 128)),
                dict(out=torch.zeros(4, 128, dtype=torch.float16)),
                dict(out=torch.zeros(4, 127, dtype=torch.bfloat16)),
                dict(xq=f8(4, 512)[:, ::2]), dict(offsets=torch.zeros(3, dtype=torch.int64))):
        with pytest.raises(moe.MoeError):
            moe.moe_block_gemm(**{**ok, **bad}, stream=0)
    x = torch.zeros(4, 256, dtype=torch.bfloat16)
    for bad in ((x.float(), f8(4, 256), torch.zeros(4, 2)), (x, f8(4, 128), torch.zeros(4, 1)),
                (x, f8(4, 256), torch.zeros(4, 3)), (x.t(), f8(256, 4), torch.zeros(256, 1))):
        with pytest.raises(moe.MoeError):
            moe.moe_block_quant(*bad, stream=0)
    cfg = moe.config(T=4, d=128, E=16, k=2, d_ff=128)
    idx, w = torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 2)
    for bad in (torch.zeros(4, 15), torch.zeros(3, 16), torch.zeros(4, 16).double(),
                torch.zeros(4, 32)[:, ::2]):
        with pytest.raises(moe.MoeError):
            moe.moe_select(cfg, bad, None, None, idx, w, stream=0)
