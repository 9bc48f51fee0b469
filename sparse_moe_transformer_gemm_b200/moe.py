"""ctypes binding of libmoe_b200.so (the C ABI of include/moe.h).

Argument marshalling only: every function here turns torch tensors into device
pointers, calls the C entry point of the same name on the current (or given)
CUDA stream and raises ``MoeError`` on a non-zero status. All arithmetic runs
in the library's CUDA kernels; there is no fallback. Loading fails loudly if
the library has not been built (``python -m sparse_moe_transformer_gemm_b200.build``).
"""

from __future__ import annotations

import ctypes
import os
from typing import Optional

import torch

# MOE_B200_LIB selects another build of the same library (e.g. for A/B timing).
LIB_PATH = os.environ.get("MOE_B200_LIB") or os.path.join(
    os.path.dirname(os.path.abspath(__file__)), "libmoe_b200.so")

MOE_OK = 0
MOE_ERR_INVALID_ARG = -1
MOE_ERR_UNSUPPORTED_SHAPE = -2
MOE_ERR_WORKSPACE = -3
MOE_ERR_CUDA = -4
MOE_ERR_TIMEOUT = -5

MOE_FLAG_FP8_WEIGHTS = 0x1
MOE_FLAG_STREAM_PATH = 0x2
MOE_FLAG_GEMM_PATH = 0x4
MOE_FLAG_PACKED_WEIGHTS = 0x8
MOE_FLAG_SHARED_EXPERT = 0x10
MOE_FLAG_FP4_WEIGHTS = 0x20
MOE_FLAG_FP8_BLOCK = 0x40
MOE_WEIGHTS_GATE_UP = 0
MOE_WEIGHTS_DOWN = 1
MOE_SCORE_SIGMOID = 0
MOE_SCORE_SQRT_SOFTPLUS = 1
MOE_SCORE_SOFTMAX = 2  # moe_select, moe_route4 and moe_forward4 only
SCORE_FNS = {"sigmoid": MOE_SCORE_SIGMOID, "sqrtsoftplus": MOE_SCORE_SQRT_SOFTPLUS,
             "softmax": MOE_SCORE_SOFTMAX}
MOE_GROUP_MAX = 0
MOE_GROUP_TOP2 = 1
GROUP_SCORES = {"max": MOE_GROUP_MAX, "top2": MOE_GROUP_TOP2}
MOE_OUT_BF16 = 0
MOE_OUT_F32 = 1

EXPORTED = ("moe_workspace_size", "moe_workspace_init", "moe_route", "moe_permute",
            "moe_permute_index", "moe_expert_gate_up", "moe_expert_gate_up_gather",
            "moe_expert_down", "moe_experts", "moe_combine", "moe_forward", "moe_read_status",
            "moe_status_string", "moe_route_noalloc", "moe_pack_weights", "moe_route2",
            "moe_forward2", "moe_route3", "moe_forward3", "moe_selftest_bounded_wait",
            "moe_ep_row_experts", "moe_select", "moe_route4", "moe_forward4",
            "moe_forward_routed", "moe_block_quant", "moe_block_gemm",
            "moe_block_workspace_size", "moe_block_permute", "moe_block_gate_up",
            "moe_block_down")

MOE_NOALLOC_SCRATCH_BYTES = 2 << 20
MOE_EP_MAX_SEGMENTS = 8192
# batches of at most this many token-slots (T*k) gather their token rows inside
# the gate_up GEMM; larger ones write the permuted copy (moe_forward's rule)
MOE_GATHER_MAX_SLOTS = 4096


class MoeConfig(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int32), ("d", ctypes.c_int32), ("E", ctypes.c_int32),
                ("k", ctypes.c_int32), ("d_ff", ctypes.c_int32), ("scale", ctypes.c_float),
                ("flags", ctypes.c_uint32)]

    def __repr__(self):
        return (f"MoeConfig(T={self.T}, d={self.d}, E={self.E}, k={self.k}, d_ff={self.d_ff}, "
                f"scale={self.scale}, flags={self.flags:#x})")


class MoeRouteOptions(ctypes.Structure):
    """moe_route_options: score_bias [E], norm_weight [d] (device pointers), norm_eps,
    score_fn (MOE_SCORE_*)."""
    _fields_ = [("score_bias", ctypes.c_void_p), ("norm_weight", ctypes.c_void_p),
                ("norm_eps", ctypes.c_float), ("score_fn", ctypes.c_int32)]


def route_options(score_bias=None, norm_weight=None, norm_eps: float = 1e-6,
                  score_fn: str = "sigmoid"):
    """Router options; score_fn is "sigmoid", "sqrtsoftplus" or, for moe_select, moe_route4
    and moe_forward4, "softmax" (or a MOE_SCORE_* value). The tensors, contiguous fp32, live
    as long as the options."""
    fn = SCORE_FNS[score_fn] if isinstance(score_fn, str) else int(score_fn)
    for t in (score_bias, norm_weight):
        if t is not None and (t.dtype != torch.float32 or not t.is_contiguous()):
            raise MoeError("route_options", MOE_ERR_INVALID_ARG)
    opt = MoeRouteOptions(None if score_bias is None else score_bias.data_ptr(),
                          None if norm_weight is None else norm_weight.data_ptr(),
                          float(norm_eps), fn)
    opt.tensors = (score_bias, norm_weight)
    return opt


class MoeGroupOptions(ctypes.Structure):
    """moe_group_options: n_group, topk_group, group_score (MOE_GROUP_*), renormalize."""
    _fields_ = [("n_group", ctypes.c_int32), ("topk_group", ctypes.c_int32),
                ("group_score", ctypes.c_int32), ("renormalize", ctypes.c_int32)]


def group_options(n_group: int = 1, topk_group: int = 1, group_score: str = "max",
                  renormalize: bool = True):
    """The choice in groups; group_score is "max" or "top2" (or a MOE_GROUP_* value)."""
    gs = GROUP_SCORES[group_score] if isinstance(group_score, str) else int(group_score)
    return MoeGroupOptions(int(n_group), int(topk_group), gs, int(renormalize))


class MoeError(RuntimeError):
    def __init__(self, fn: str, code: int):
        super().__init__(f"{fn} failed: {code} ({moe_status_string(code)})")
        self.code = code


_lib = None


def lib() -> ctypes.CDLL:
    """Load libmoe_b200.so once, declaring the C signatures."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is missing: build it with "
                          "`python -m sparse_moe_transformer_gemm_b200.build`")
    L = ctypes.CDLL(LIB_PATH)
    P, I, S = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
    I32, L64 = ctypes.c_int32, ctypes.c_int64
    C = ctypes.POINTER(MoeConfig)
    sig = {
        "moe_workspace_size": (S, [C]),
        "moe_workspace_init": (I, [C, P, S, P]),
        "moe_route": (I, [C, P, P, P, P, P, P, S, P]),
        "moe_permute": (I, [C, P, P, P, P, P, P, P, S, P]),
        "moe_permute_index": (I, [C, P, P, P, P, P, P, S, P]),
        "moe_expert_gate_up": (I, [C, P, P, P, P, P, P, S, P]),
        "moe_expert_gate_up_gather": (I, [C, P, P, P, P, P, P, P, S, P]),
        "moe_expert_down": (I, [C, P, P, P, P, P, P, S, P]),
        "moe_experts": (I, [C, P, P, P, P, P, P, P, P, S, P]),
        "moe_combine": (I, [C, P, P, P, P, P, S, P]),
        "moe_forward": (I, [C, P, P, P, P, P, P, P, P, P, S, P]),
        "moe_read_status": (I, [P, P]),
        "moe_status_string": (ctypes.c_char_p, [I]),
        "moe_route_noalloc": (I, [C, P, P, P, P, P, P]),
        "moe_pack_weights": (I, [C, I, P, P, P]),
        "moe_route2": (I, [C, P, P, P, P, P, P, P, S, P]),
        "moe_forward2": (I, [C, P, P, P, P, P, P, P, P, P, P, S, P]),
        "moe_route3": (I, [C, P, P, P, P, P, P, P, S, P]),
        "moe_forward3": (I, [C, P, P, P, P, P, P, P, P, P, P, S, P]),
        "moe_selftest_bounded_wait": (I, [P, ctypes.c_ulonglong, P]),
        "moe_ep_row_experts": (I, [P, ctypes.c_int32, ctypes.c_int32, P, ctypes.c_int32, P]),
        "moe_select": (I, [C, P, L64, P, P, P, P, P]),
        "moe_route4": (I, [C, P, P, P, P, P, P, P, P, S, P]),
        "moe_forward4": (I, [C, P, P, P, P, P, P, P, P, P, P, P, S, P]),
        "moe_forward_routed": (I, [C, P, P, P, P, P, P, P, P, P, S, P]),
        "moe_block_quant": (I, [P, L64, I32, I32, P, P, P]),
        "moe_block_gemm": (I, [P, P, P, P, P, I32, I32, I32, I32, P, I32, P, S, P]),
        "moe_block_workspace_size": (S, [I32, I32, I32, I32]),
        "moe_block_permute": (I, [C, P, P, P, P, P]),
        "moe_block_gate_up": (I, [C, P, P, P, P, P, P, P, P, S, P]),
        "moe_block_down": (I, [C, P, P, P, P, P, P, P, S, P]),
    }
    for name, (res, args) in sig.items():
        fn = getattr(L, name)
        fn.restype = res
        fn.argtypes = args
    _lib = L
    return L


def config(T: int, d: int, E: int, k: int, d_ff: int, scale: float = 2.826, fp8: bool = False,
           path: Optional[str] = None, packed: bool = False, shared: bool = False,
           fp4: bool = False, fp8_block: bool = False) -> MoeConfig:
    """Build a moe_config. path: None (automatic), "stream" or "gemm"; packed: the
    bf16 expert weights are in moe_pack_weights' layout; shared: expert E of the
    weight arrays is a shared expert; fp4: E2M1 expert weights with E8M0 block
    scales; fp8_block: e4m3 expert weights and activations with a scale per block of
    128."""
    flags = MOE_FLAG_FP8_WEIGHTS if fp8 else 0
    if fp4:
        flags |= MOE_FLAG_FP4_WEIGHTS
    if fp8_block:
        flags |= MOE_FLAG_FP8_BLOCK
    if packed:
        flags |= MOE_FLAG_PACKED_WEIGHTS
    if shared:
        flags |= MOE_FLAG_SHARED_EXPERT
    if path == "stream":
        flags |= MOE_FLAG_STREAM_PATH
    elif path == "gemm":
        flags |= MOE_FLAG_GEMM_PATH
    elif path is not None:
        raise ValueError(f"unknown path {path!r}")
    return MoeConfig(T, d, E, k, d_ff, scale, flags)


def _p(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _s(stream) -> int:
    """The stream's handle (None: the current stream of the current device)."""
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _check(fn: str, rc: int) -> None:
    if rc != MOE_OK:
        raise MoeError(fn, rc)


def moe_status_string(code: int) -> str:
    return lib().moe_status_string(int(code)).decode()


def moe_workspace_size(cfg: MoeConfig) -> int:
    return int(lib().moe_workspace_size(ctypes.byref(cfg)))


def moe_workspace_init(cfg: MoeConfig, ws: torch.Tensor, stream=None) -> None:
    _check("moe_workspace_init",
           lib().moe_workspace_init(ctypes.byref(cfg), _p(ws), ws.numel(), _s(stream)))


def workspace(cfg: MoeConfig, device="cuda", stream=None) -> torch.Tensor:
    """Allocate (through torch) and initialise a workspace for cfg."""
    n = moe_workspace_size(cfg)
    if n == 0:
        raise MoeError("moe_workspace_size", MOE_ERR_UNSUPPORTED_SHAPE)
    ws = torch.empty(n, dtype=torch.uint8, device=device)
    moe_workspace_init(cfg, ws, stream)
    return ws


def moe_route(cfg, x, w_gate, gate_bias, topk_idx, topk_w, ws, stream=None) -> None:
    _check("moe_route", lib().moe_route(ctypes.byref(cfg), _p(x), _p(w_gate), _p(gate_bias),
                                        _p(topk_idx), _p(topk_w), _p(ws), ws.numel(), _s(stream)))


def moe_permute(cfg, topk_idx, x, counts, offsets, row_of, x_perm, ws, stream=None) -> None:
    _check("moe_permute", lib().moe_permute(ctypes.byref(cfg), _p(topk_idx), _p(x), _p(counts),
                                            _p(offsets), _p(row_of), _p(x_perm), _p(ws),
                                            ws.numel(), _s(stream)))


def moe_permute_index(cfg, topk_idx, counts, offsets, row_of, token_of_row, ws,
                      stream=None) -> None:
    _check("moe_permute_index",
           lib().moe_permute_index(ctypes.byref(cfg), _p(topk_idx), _p(counts), _p(offsets),
                                   _p(row_of), _p(token_of_row), _p(ws), ws.numel(), _s(stream)))


def moe_expert_gate_up_gather(cfg, x, token_of_row, offsets, w_gate_up, s_gate_up, h, ws,
                              stream=None) -> None:
    _check("moe_expert_gate_up_gather",
           lib().moe_expert_gate_up_gather(ctypes.byref(cfg), _p(x), _p(token_of_row),
                                           _p(offsets), _p(w_gate_up), _p(s_gate_up), _p(h),
                                           _p(ws), ws.numel(), _s(stream)))


def moe_expert_gate_up(cfg, x_perm, offsets, w_gate_up, s_gate_up, h, ws, stream=None) -> None:
    _check("moe_expert_gate_up",
           lib().moe_expert_gate_up(ctypes.byref(cfg), _p(x_perm), _p(offsets), _p(w_gate_up),
                                    _p(s_gate_up), _p(h), _p(ws), ws.numel(), _s(stream)))


def moe_expert_down(cfg, h, offsets, w_down, s_down, y, ws, stream=None) -> None:
    _check("moe_expert_down",
           lib().moe_expert_down(ctypes.byref(cfg), _p(h), _p(offsets), _p(w_down), _p(s_down),
                                 _p(y), _p(ws), ws.numel(), _s(stream)))


def moe_experts(cfg, x_perm, offsets, w_gate_up, s_gate_up, w_down, s_down, y, ws,
                stream=None) -> None:
    _check("moe_experts",
           lib().moe_experts(ctypes.byref(cfg), _p(x_perm), _p(offsets), _p(w_gate_up),
                             _p(s_gate_up), _p(w_down), _p(s_down), _p(y), _p(ws), ws.numel(),
                             _s(stream)))


def moe_combine(cfg, y, row_of, topk_w, out, ws, stream=None) -> None:
    _check("moe_combine", lib().moe_combine(ctypes.byref(cfg), _p(y), _p(row_of), _p(topk_w),
                                            _p(out), _p(ws), ws.numel(), _s(stream)))


def moe_forward(cfg, x, w_gate, gate_bias, w_gate_up, s_gate_up, w_down, s_down, out, ws,
                stream=None) -> None:
    _check("moe_forward",
           lib().moe_forward(ctypes.byref(cfg), _p(x), _p(w_gate), _p(gate_bias), _p(w_gate_up),
                             _p(s_gate_up), _p(w_down), _p(s_down), _p(out), _p(ws), ws.numel(),
                             _s(stream)))


def moe_route2(cfg, x, w_gate, gate_bias, score_bias, topk_idx, topk_w, ws, stream=None) -> None:
    _check("moe_route2", lib().moe_route2(ctypes.byref(cfg), _p(x), _p(w_gate), _p(gate_bias),
                                          _p(score_bias), _p(topk_idx), _p(topk_w), _p(ws),
                                          ws.numel(), _s(stream)))


def moe_forward2(cfg, x, w_gate, gate_bias, score_bias, w_gate_up, s_gate_up, w_down, s_down,
                 out, ws, stream=None) -> None:
    _check("moe_forward2",
           lib().moe_forward2(ctypes.byref(cfg), _p(x), _p(w_gate), _p(gate_bias),
                              _p(score_bias), _p(w_gate_up), _p(s_gate_up), _p(w_down),
                              _p(s_down), _p(out), _p(ws), ws.numel(), _s(stream)))


def moe_route3(cfg, x, w_gate, gate_bias, opt, topk_idx, topk_w, ws, stream=None) -> None:
    _check("moe_route3", lib().moe_route3(ctypes.byref(cfg), _p(x), _p(w_gate), _p(gate_bias),
                                          None if opt is None else ctypes.byref(opt),
                                          _p(topk_idx), _p(topk_w), _p(ws), ws.numel(),
                                          _s(stream)))


def moe_forward3(cfg, x, w_gate, gate_bias, opt, w_gate_up, s_gate_up, w_down, s_down, out, ws,
                 stream=None) -> None:
    _check("moe_forward3",
           lib().moe_forward3(ctypes.byref(cfg), _p(x), _p(w_gate), _p(gate_bias),
                              None if opt is None else ctypes.byref(opt), _p(w_gate_up),
                              _p(s_gate_up), _p(w_down), _p(s_down), _p(out), _p(ws), ws.numel(),
                              _s(stream)))


def moe_route_noalloc(cfg, x, w_gate, gate_bias, topk_idx, topk_w, stream=None) -> None:
    """moe_route without a workspace, for callers that cannot allocate device
    memory; the scratch is a fixed 2 MiB device array inside the library."""
    _check("moe_route_noalloc",
           lib().moe_route_noalloc(ctypes.byref(cfg), _p(x), _p(w_gate), _p(gate_bias),
                                   _p(topk_idx), _p(topk_w), _s(stream)))


def moe_pack_weights(cfg, which, w, w_packed, stream=None) -> None:
    """Rearrange one bf16 expert weight into the packed 128 x 64 block layout."""
    _check("moe_pack_weights", lib().moe_pack_weights(ctypes.byref(cfg), int(which), _p(w),
                                                      _p(w_packed), _s(stream)))


def moe_selftest_bounded_wait(ws, limit_ns: int, stream=None) -> None:
    """Run the bounded-wait self-test; its MOE_ERR_TIMEOUT lands in ws's status word."""
    _check("moe_selftest_bounded_wait",
           lib().moe_selftest_bounded_wait(_p(ws), int(limit_ns), _s(stream)))


def moe_ep_row_experts(counts, n_src: int, e_local: int, expert_of_row, stream=None) -> None:
    """Local expert of every received row (expert parallelism): counts [n_src, e_local]
    int32, expert_of_row [n_rows] int32, both on the device."""
    _check("moe_ep_row_experts",
           lib().moe_ep_row_experts(_p(counts), int(n_src), int(e_local), _p(expert_of_row),
                                    int(expert_of_row.numel()), _s(stream)))


def _opt(o):
    return o if o is None else ctypes.byref(o)


def _rows(fn: str, t: torch.Tensor, rows: int, cols: int) -> int:
    """Row stride, in elements, of a [rows, cols] tensor whose rows are contiguous."""
    if t.shape != (rows, cols):
        raise MoeError(fn, MOE_ERR_INVALID_ARG)
    if t.is_contiguous():
        return cols
    if cols > 1 and t.stride(1) != 1:
        raise MoeError(fn, MOE_ERR_INVALID_ARG)
    return t.stride(0) if rows > 1 else max(cols, t.stride(0))


def _on(fn: str, stream, first, *others):
    """The stream's handle; refuses tensors that are not on the current device, on which
    the call launches."""
    device = first.get_device()  # -1: host memory
    for t in others:
        if t is not None and t.get_device() != device:
            raise MoeError(fn, MOE_ERR_INVALID_ARG)
    if device < 0 or device != torch.cuda.current_device():
        raise MoeError(fn, MOE_ERR_INVALID_ARG)
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(device)
    return _s(stream)


def _take(fn: str, t: Optional[torch.Tensor], dtype: torch.dtype, n: int) -> None:
    """Refuse a tensor that is not n (or more) contiguous elements of dtype."""
    if t is None or t.dtype is not dtype or t.numel() < n or not t.is_contiguous():
        raise MoeError(fn, MOE_ERR_INVALID_ARG)


def _take_routing(fn: str, cfg, topk_idx, topk_w) -> None:
    n = cfg.T * cfg.k
    _take(fn, topk_idx, torch.int32, n)
    _take(fn, topk_w, torch.float32, n)


def _options(fn: str, cfg, opt):
    """(score_bias, norm_weight) of opt, as route_options made it."""
    bias, norm = getattr(opt, "tensors", (None, None))
    if (bias is not None and bias.numel() < cfg.E) or (norm is not None and norm.numel() < cfg.d):
        raise MoeError(fn, MOE_ERR_INVALID_ARG)
    return bias, norm


def _take_router(fn: str, cfg, x, w_gate, gate_bias) -> None:
    _take(fn, x, torch.bfloat16, cfg.T * cfg.d)
    _take(fn, w_gate, torch.bfloat16, cfg.E * cfg.d)
    if gate_bias is not None:
        _take(fn, gate_bias, torch.float32, cfg.E)


def _take_bytes(fn: str, t: Optional[torch.Tensor], n: int) -> None:
    """Refuse a tensor that is not n (or more) contiguous one-byte elements."""
    if t is None or t.element_size() != 1 or t.numel() < n or not t.is_contiguous():
        raise MoeError(fn, MOE_ERR_INVALID_ARG)


def _grouped(cfg):
    """(experts, rows, d, d_ff) of the grouped products, the shared expert's among them."""
    shared = 1 if cfg.flags & MOE_FLAG_SHARED_EXPERT else 0
    return cfg.E + shared, cfg.T * (cfg.k + shared), cfg.d, cfg.d_ff


def _take_block(fn: str, codes, scales, rows: int, cols: int) -> None:
    """Rows quantised in blocks of 128 columns."""
    _take_bytes(fn, codes, rows * cols)
    _take(fn, scales, torch.float32, rows * (cols // 128))


def _take_weight(fn: str, flags: int, w, s, rows: int, cols: int) -> None:
    """One expert weight, rows in all, in the format of flags, with its scales."""
    if flags & MOE_FLAG_FP8_BLOCK:
        _take_bytes(fn, w, rows * cols)
        _take(fn, s, torch.float32, (rows // 128) * (cols // 128))
    elif flags & MOE_FLAG_FP8_WEIGHTS:
        _take_bytes(fn, w, rows * cols)
        _take(fn, s, torch.float32, rows)
    elif flags & MOE_FLAG_FP4_WEIGHTS:
        _take_bytes(fn, w, rows * (cols // 2))
        _take_bytes(fn, s, rows * (cols // 32))
    else:
        _take(fn, w, torch.bfloat16, rows * cols)
        if s is not None:
            raise MoeError(fn, MOE_ERR_INVALID_ARG)


def _take_experts(fn: str, cfg, w_gate_up, s_gate_up, w_down, s_down, out) -> None:
    (E, _, d, F), flags = _grouped(cfg), cfg.flags
    _take_weight(fn, flags, w_gate_up, s_gate_up, E * 2 * F, d)
    _take_weight(fn, flags, w_down, s_down, E * d, F)
    _take(fn, out, torch.bfloat16, cfg.T * d)


def moe_select(cfg, logits, opt, grp, topk_idx, topk_w, stream=None) -> None:
    """The choice of experts from logits [T, E] fp32 (rows may be strided)."""
    fn, T, E = "moe_select", cfg.T, cfg.E
    if logits.dtype is not torch.float32:
        raise MoeError(fn, MOE_ERR_INVALID_ARG)
    ld = _rows(fn, logits, T, E)
    _take_routing(fn, cfg, topk_idx, topk_w)
    if opt is None:
        st = _on(fn, stream, logits, topk_idx, topk_w)
    else:
        st = _on(fn, stream, logits, topk_idx, topk_w, *_options(fn, cfg, opt))
    rc = lib().moe_select(ctypes.byref(cfg), logits.data_ptr(), ld, _opt(opt), _opt(grp),
                          topk_idx.data_ptr(), topk_w.data_ptr(), st)
    if rc != MOE_OK:
        raise MoeError(fn, rc)


def moe_route4(cfg, x, w_gate, gate_bias, opt, grp, topk_idx, topk_w, ws, stream=None) -> None:
    _take_router("moe_route4", cfg, x, w_gate, gate_bias)
    _take_routing("moe_route4", cfg, topk_idx, topk_w)
    st = _on("moe_route4", stream, x, w_gate, gate_bias, topk_idx, topk_w, ws,
             *_options("moe_route4", cfg, opt))
    _check("moe_route4", lib().moe_route4(ctypes.byref(cfg), _p(x), _p(w_gate), _p(gate_bias),
                                          _opt(opt), _opt(grp), _p(topk_idx), _p(topk_w), _p(ws),
                                          ws.numel(), st))


def moe_forward4(cfg, x, w_gate, gate_bias, opt, grp, w_gate_up, s_gate_up, w_down, s_down, out,
                 ws, stream=None) -> None:
    _take_router("moe_forward4", cfg, x, w_gate, gate_bias)
    _take_experts("moe_forward4", cfg, w_gate_up, s_gate_up, w_down, s_down, out)
    st = _on("moe_forward4", stream, x, w_gate, gate_bias, w_gate_up, s_gate_up, w_down, s_down,
             out, ws, *_options("moe_forward4", cfg, opt))
    _check("moe_forward4",
           lib().moe_forward4(ctypes.byref(cfg), _p(x), _p(w_gate), _p(gate_bias), _opt(opt),
                              _opt(grp), _p(w_gate_up), _p(s_gate_up), _p(w_down), _p(s_down),
                              _p(out), _p(ws), ws.numel(), st))


def moe_forward_routed(cfg, x, topk_idx, topk_w, w_gate_up, s_gate_up, w_down, s_down, out, ws,
                       stream=None) -> None:
    """The layer after its router, for a given routing."""
    _take("moe_forward_routed", x, torch.bfloat16, cfg.T * cfg.d)
    _take_routing("moe_forward_routed", cfg, topk_idx, topk_w)
    _take_experts("moe_forward_routed", cfg, w_gate_up, s_gate_up, w_down, s_down, out)
    st = _on("moe_forward_routed", stream, x, topk_idx, topk_w, w_gate_up, s_gate_up, w_down,
             s_down, out, ws)
    _check("moe_forward_routed",
           lib().moe_forward_routed(ctypes.byref(cfg), _p(x), _p(topk_idx), _p(topk_w),
                                    _p(w_gate_up), _p(s_gate_up), _p(w_down), _p(s_down),
                                    _p(out), _p(ws), ws.numel(), st))


def moe_block_quant(x, codes, scales, stream=None) -> None:
    """Quantise rows: x [M, K] bf16 (rows may be strided), codes [M, K] e4m3 (or uint8),
    scales [M, ceil(K/128)] fp32."""
    M, K = codes.shape
    if x.dtype != torch.bfloat16 or scales.shape != (M, -(-K // 128)) or \
            scales.dtype != torch.float32 or codes.element_size() != 1 or \
            not codes.is_contiguous() or not scales.is_contiguous():
        raise MoeError("moe_block_quant", MOE_ERR_INVALID_ARG)
    st = _on("moe_block_quant", stream, x, codes, scales)
    _check("moe_block_quant",
           lib().moe_block_quant(_p(x), _rows("moe_block_quant", x, M, K), M, K, _p(codes),
                                 _p(scales), st))


def block_workspace(M: int, N: int, K: int, G: int = 1, device="cuda") -> torch.Tensor:
    """A zeroed workspace for moe_block_gemm calls of these sizes."""
    n = int(lib().moe_block_workspace_size(G, M, N, K))
    if n == 0:
        raise MoeError("moe_block_workspace_size", MOE_ERR_UNSUPPORTED_SHAPE)
    return torch.zeros(n, dtype=torch.uint8, device=device)


def moe_block_gemm(xq, sx, wq, sw, out, ws, offsets=None, stream=None) -> None:
    """out [M, N] (bf16 or fp32) = xq [M, K] times wq [N, K] transposed, e4m3 codes with a
    scale per block of 128 (sx [M, ceil(K/128)], sw [ceil(N/128), ceil(K/128)]). With offsets
    [G+1] int32, wq [G, N, K] and sw [G, ...]: rows [offsets[g], offsets[g+1]) take weight g."""
    G = 1 if offsets is None else wq.shape[0]
    N, K = wq.shape[-2:]
    M = xq.shape[0]
    kb, nb = -(-K // 128), -(-N // 128)
    lead = () if offsets is None else (G,)
    if xq.shape != (M, K) or sx.shape != (M, kb) or wq.shape != lead + (N, K) or \
            sw.shape != lead + (nb, kb) or out.shape != (M, N) or \
            out.dtype not in (torch.bfloat16, torch.float32) or \
            (offsets is not None and (offsets.numel() != G + 1 or offsets.dtype != torch.int32 or
                                      not offsets.is_contiguous())) or \
            xq.element_size() != 1 or wq.element_size() != 1 or sx.dtype != torch.float32 or \
            sw.dtype != torch.float32 or not all(t.is_contiguous() for t in (xq, sx, wq, sw, out)):
        raise MoeError("moe_block_gemm", MOE_ERR_INVALID_ARG)
    st = _on("moe_block_gemm", stream, xq, sx, wq, sw, out, ws, offsets)
    _check("moe_block_gemm",
           lib().moe_block_gemm(_p(xq), _p(sx), _p(wq), _p(sw), _p(offsets), G, M, N, K, _p(out),
                                MOE_OUT_F32 if out.dtype == torch.float32 else MOE_OUT_BF16,
                                _p(ws), ws.numel(), st))


def moe_block_permute(cfg, x, row_of, xq, sx, stream=None) -> None:
    fn, (_, R, d, _) = "moe_block_permute", _grouped(cfg)
    _take(fn, x, torch.bfloat16, cfg.T * d)
    _take(fn, row_of, torch.int32, R)
    _take_block(fn, xq, sx, R, d)
    st = _on(fn, stream, x, row_of, xq, sx)
    _check(fn, lib().moe_block_permute(ctypes.byref(cfg), _p(x), _p(row_of), _p(xq), _p(sx), st))


def moe_block_gate_up(cfg, xq, sx, offsets, w_gate_up, s_gate_up, hq, sh, ws, stream=None) -> None:
    fn, (E, R, d, F) = "moe_block_gate_up", _grouped(cfg)
    _take_block(fn, xq, sx, R, d)
    _take(fn, offsets, torch.int32, E + 1)
    _take_weight(fn, MOE_FLAG_FP8_BLOCK, w_gate_up, s_gate_up, E * 2 * F, d)
    _take_block(fn, hq, sh, R, F)
    st = _on(fn, stream, xq, sx, offsets, w_gate_up, s_gate_up, hq, sh, ws)
    _check(fn, lib().moe_block_gate_up(ctypes.byref(cfg), _p(xq), _p(sx), _p(offsets),
                                       _p(w_gate_up), _p(s_gate_up), _p(hq), _p(sh), _p(ws),
                                       ws.numel(), st))


def moe_block_down(cfg, hq, sh, offsets, w_down, s_down, y, ws, stream=None) -> None:
    fn, (E, R, d, F) = "moe_block_down", _grouped(cfg)
    _take_block(fn, hq, sh, R, F)
    _take(fn, offsets, torch.int32, E + 1)
    _take_weight(fn, MOE_FLAG_FP8_BLOCK, w_down, s_down, E * d, F)
    _take(fn, y, torch.bfloat16, R * d)
    st = _on(fn, stream, hq, sh, offsets, w_down, s_down, y, ws)
    _check(fn, lib().moe_block_down(ctypes.byref(cfg), _p(hq), _p(sh), _p(offsets), _p(w_down),
                                    _p(s_down), _p(y), _p(ws), ws.numel(), st))


def moe_read_status(ws, stream=None) -> int:
    return int(lib().moe_read_status(_p(ws), _s(stream)))


def layer_args(layer: dict):
    """(w_gate_up, s_gate_up, w_down, s_down) of a synthetic layer dict, FP4, FP8 or
    bf16; with a shared expert, its weights follow the routed ones as expert E."""
    cfg = layer["cfg"]
    if getattr(cfg, "fp4", False):
        return (layer["q4_gate_up"], layer["s4_gate_up"], layer["q4_down"], layer["s4_down"])
    if cfg.fp8:
        args = [layer["q_gate_up"], layer["s_gate_up"], layer["q_down"], layer["s_down"]]
        sh = ("q_shared_gate_up", "s_shared_gate_up", "q_shared_down", "s_shared_down")
    else:
        args = [layer["w_gate_up"], None, layer["w_down"], None]
        sh = ("w_shared_gate_up", None, "w_shared_down", None)
    if getattr(cfg, "shared", False):
        args = [a if n is None else torch.cat([a, layer[n][None]]) for a, n in zip(args, sh)]
    return tuple(args)


def config_of(shape, path: Optional[str] = None, packed: bool = False) -> MoeConfig:
    """moe_config for a synthetic LayerShape."""
    return config(shape.T, shape.d, shape.E, shape.k, shape.F, shape.scale, shape.fp8, path,
                  packed, getattr(shape, "shared", False), getattr(shape, "fp4", False))


def pack_layer_weights(cfg: MoeConfig, w_gate_up: torch.Tensor, w_down: torch.Tensor,
                       stream=None):
    """(packed w_gate_up, packed w_down): new tensors in moe_pack_weights' layout."""
    gu = torch.empty_like(w_gate_up)
    dn = torch.empty_like(w_down)
    moe_pack_weights(cfg, MOE_WEIGHTS_GATE_UP, w_gate_up, gu, stream)
    moe_pack_weights(cfg, MOE_WEIGHTS_DOWN, w_down, dn, stream)
    return gu, dn
