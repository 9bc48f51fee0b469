"""What the bindings of the expert choice refuse before any launch (no GPU): outputs and
inputs that the library would read or write past."""

import pytest
import torch

from sparse_moe_transformer_gemm_b200 import build as moe_build
from sparse_moe_transformer_gemm_b200 import moe


@pytest.fixture(scope="module", autouse=True)
def lib():
    moe_build.build()
    return moe.lib()


def refused(fn, *args, **kw):
    with pytest.raises(moe.MoeError) as e:
        fn(*args, stream=0, **kw)
    assert e.value.code == moe.MOE_ERR_INVALID_ARG, e.value


T, E, K, D, F = 4, 16, 2, 128, 128
BAD_IDX = [torch.zeros(T, K, dtype=torch.int64), torch.zeros(T, 1, dtype=torch.int32),
           torch.zeros(T, 2 * K, dtype=torch.int32)[:, ::2],
           torch.zeros(K, T, dtype=torch.int32).t(), None]
BAD_W = [torch.zeros(T, K, dtype=torch.bfloat16), torch.zeros(T - 1, K),
         torch.zeros(T, K, dtype=torch.float64), torch.zeros(T, 2 * K)[:, ::2], None]


def test_select_refuses_outputs_of_another_type_or_size():
    cfg = moe.config(T, D, E, K, F)
    z, idx, w = torch.zeros(T, E), torch.zeros(T, K, dtype=torch.int32), torch.zeros(T, K)
    for bad in BAD_IDX:
        refused(moe.moe_select, cfg, z, None, None, bad, w)
    for bad in BAD_W:
        refused(moe.moe_select, cfg, z, None, None, idx, bad)


def test_route4_refuses_outputs_of_another_type_or_size():
    cfg = moe.config(T, D, E, K, F)
    x, wg = torch.zeros(T, D, dtype=torch.bfloat16), torch.zeros(E, D, dtype=torch.bfloat16)
    idx, w = torch.zeros(T, K, dtype=torch.int32), torch.zeros(T, K)
    ws = torch.zeros(moe.moe_workspace_size(cfg) + 256, dtype=torch.uint8)
    ws = ws[-ws.data_ptr() % 256:]
    for bad in BAD_IDX:
        refused(moe.moe_route4, cfg, x, wg, None, None, None, bad, w, ws)
    for bad in BAD_W:
        refused(moe.moe_route4, cfg, x, wg, None, None, None, idx, bad, ws)
    for bad in (x.float(), x[:3], torch.zeros(T, 2 * D, dtype=torch.bfloat16)[:, ::2]):
        refused(moe.moe_route4, cfg, bad, wg, None, None, None, idx, w, ws)
    for bad in (wg.float(), wg[:15]):
        refused(moe.moe_route4, cfg, x, bad, None, None, None, idx, w, ws)
    for bad in (torch.zeros(E - 1), torch.zeros(E, dtype=torch.bfloat16)):
        refused(moe.moe_route4, cfg, x, wg, bad, None, None, idx, w, ws)


def worse(t):
    """Tensors in t's place that must be refused: of a wider type, too few, strided, none."""
    other = {torch.uint8: torch.int16, torch.int32: torch.int64, torch.float32: torch.float64,
             torch.bfloat16: torch.float32}[t.dtype]
    flat = torch.zeros(2 * t.numel(), dtype=t.dtype)
    return [torch.zeros(t.shape, dtype=other), flat[:t.numel() - 1], flat[::2], None]


def each_refused(fn, args, at):
    """Every argument of `at` replaced by tensors that do not fit."""
    for i in at:
        for bad in worse(args[i]):
            refused(fn, *args[:i], bad, *args[i + 1:])


def step_args(shared):
    """Arguments of moe_block_permute, moe_block_gate_up and moe_block_down."""
    cfg = moe.config(T, D, E, K, F, fp8_block=True, shared=shared)
    n, R = E + shared, T * (K + shared)
    u8 = lambda *s: torch.zeros(*s, dtype=torch.uint8)  # noqa: E731
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)  # noqa: E731
    f32 = torch.zeros
    ws = u8(moe.moe_workspace_size(cfg) + 256)
    ws = ws[-ws.data_ptr() % 256:]
    xq, sx, hq, sh, off = u8(R, D), f32(R, D // 128), u8(R, F), f32(R, F // 128), i32(n + 1)
    return (cfg, ws, [cfg, bf(T, D), i32(R), xq, sx],
            [cfg, xq, sx, off, u8(n, 2 * F, D), f32(n, 2 * F // 128, D // 128), hq, sh, ws],
            [cfg, hq, sh, off, u8(n, D, F), f32(n, D // 128, F // 128), bf(R, D), ws])


@pytest.mark.parametrize("shared", [False, True])
def test_block_steps_refuse_tensors_that_do_not_fit(shared):
    cfg, ws, permute, gate_up, down = step_args(shared)
    each_refused(moe.moe_block_permute, permute, range(1, 5))
    each_refused(moe.moe_block_gate_up, gate_up, range(1, 8))
    each_refused(moe.moe_block_down, down, range(1, 7))


# Expert weights a format takes: (config arguments, elements of an expert's weight rows of
# n columns, their type, elements and type of the scales of r rows)
FORMATS = {
    "bf16": ({}, lambda n: n, torch.bfloat16, None),
    "packed": (dict(packed=True), lambda n: n, torch.bfloat16, None),
    "fp8": (dict(fp8=True), lambda n: n, torch.uint8, (lambda r, n: (r,), torch.float32)),
    "fp4": (dict(fp4=True), lambda n: n // 2, torch.uint8,
            (lambda r, n: (r, n // 32), torch.uint8)),
    "fp8_block": (dict(fp8_block=True), lambda n: n, torch.uint8,
                  (lambda r, n: (r // 128, n // 128), torch.float32)),
    "bf16 shared": (dict(shared=True), lambda n: n, torch.bfloat16, None),
    "fp8_block shared": (dict(shared=True, fp8_block=True), lambda n: n, torch.uint8,
                         (lambda r, n: (r // 128, n // 128), torch.float32)),
}


@pytest.mark.parametrize("fmt", list(FORMATS))
def test_layers_refuse_tensors_that_do_not_fit(fmt):
    kw, cols, wtype, scales = FORMATS[fmt]
    d, f = 256, 512
    cfg = moe.config(T, d, E, K, f, **kw)
    n = E + int("shared" in fmt)
    ws = torch.zeros(moe.moe_workspace_size(cfg) + 256, dtype=torch.uint8)
    ws = ws[-ws.data_ptr() % 256:]
    weights = []
    for rows, width in ((2 * f, d), (d, f)):
        weights.append(torch.zeros(n, rows, cols(width), dtype=wtype))
        weights.append(None if scales is None
                       else torch.zeros(n, *scales[0](rows, width), dtype=scales[1]))
    x = torch.zeros(T, d, dtype=torch.bfloat16)
    out = torch.zeros(T, d, dtype=torch.bfloat16)
    idx, w = torch.zeros(T, K, dtype=torch.int32), torch.zeros(T, K)
    given = [i for i in range(4) if weights[i] is not None]
    routed = [cfg, x, idx, w, *weights, out, ws]
    each_refused(moe.moe_forward_routed, routed, [1, 2, 3, *(4 + i for i in given), 8])
    wg = torch.zeros(E, d, dtype=torch.bfloat16)
    whole = [cfg, x, wg, None, None, None, *weights, out, ws]
    each_refused(moe.moe_forward4, whole, [1, 2, *(6 + i for i in given), 10])
    if not scales:
        refused(moe.moe_forward_routed, *routed[:5], torch.zeros(n, f), *routed[6:])


class Elsewhere:
    """A tensor's attributes, on a device of its own."""

    def __init__(self, t, index):
        self.t, self.index = t, index

    def get_device(self):
        return self.index

    def data_ptr(self):
        raise AssertionError("the call went on")

    def __getattr__(self, name):
        return getattr(self.t, name)


@pytest.mark.parametrize("index", [-1, 1])
def test_tensors_of_another_device_are_refused(monkeypatch, index):
    """One tensor in host memory (-1), or on another device than the current one, which
    would launch on it."""
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    cfg, ws, permute, gate_up, down = step_args(False)
    plain = moe.config(T, D, E, K, F)
    ws1 = torch.zeros(moe.moe_workspace_size(plain), dtype=torch.uint8)
    x, out = torch.zeros(T, D, dtype=torch.bfloat16), torch.zeros(T, D, dtype=torch.bfloat16)
    idx, w = torch.zeros(T, K, dtype=torch.int32), torch.zeros(T, K)
    wg, wgu = torch.zeros(E, D, dtype=torch.bfloat16), torch.zeros(E, 2 * F, D, dtype=torch.bfloat16)
    wd, gb = torch.zeros(E, D, F, dtype=torch.bfloat16), torch.zeros(E)
    u8 = lambda *s: torch.zeros(*s, dtype=torch.uint8)  # noqa: E731
    calls = [
        (moe.moe_block_permute, permute, range(1, 5)),
        (moe.moe_block_gate_up, gate_up, range(1, 9)),
        (moe.moe_block_down, down, range(1, 8)),
        (moe.moe_select, [plain, torch.zeros(T, E), None, None, idx, w], (1, 4, 5)),
        (moe.moe_route4, [plain, x, wg, gb, None, None, idx, w, ws1], (1, 2, 3, 6, 7, 8)),
        (moe.moe_forward_routed, [plain, x, idx, w, wgu, None, wd, None, out, ws1],
         (1, 2, 3, 4, 6, 8, 9)),
        (moe.moe_forward4, [plain, x, wg, gb, None, None, wgu, None, wd, None, out, ws1],
         (1, 2, 3, 6, 8, 10, 11)),
        (moe.moe_block_quant, [torch.zeros(4, 256, dtype=torch.bfloat16), u8(4, 256),
                               torch.zeros(4, 2)], range(3)),
        (moe.moe_block_gemm, [u8(4, 256), torch.zeros(4, 2), u8(2, 128, 256),
                              torch.zeros(2, 1, 2), torch.zeros(4, 128), u8(256),
                              torch.zeros(3, dtype=torch.int32)], range(7)),
    ]
    for fn, args, at in calls:
        here = [Elsewhere(a, 0) if isinstance(a, torch.Tensor) else a for a in args]
        # all on the current device: past the checks, to the pointers
        with pytest.raises(AssertionError, match="went on"):
            fn(*here, stream=0)
        for i in at:
            refused(fn, *here[:i], Elsewhere(args[i], index), *here[i + 1:])


def test_route_options_keep_their_tensors():
    """The library reads them through pointers: a temporary lives as long as the options."""
    gone = []

    class Watched(torch.Tensor):
        def __del__(self):
            gone.append(1)

    opt = moe.route_options(torch.ones(E).as_subclass(Watched),
                            torch.ones(D).as_subclass(Watched))
    assert not gone and opt.score_bias and opt.norm_weight
    del opt
    assert len(gone) == 2


def test_route_options_refuse_other_types_and_layouts():
    for bad in (torch.ones(E, dtype=torch.bfloat16), torch.ones(E, dtype=torch.float64),
                torch.ones(2 * E)[::2]):
        for kw in (dict(score_bias=bad), dict(norm_weight=bad)):
            with pytest.raises(moe.MoeError) as e:
                moe.route_options(**kw)
            assert e.value.code == moe.MOE_ERR_INVALID_ARG


@pytest.mark.parametrize("index", [0, -1, 1])
def test_options_that_do_not_fit_the_call(monkeypatch, index):
    """A bias of fewer than E experts, a norm weight of fewer than d columns, and (index
    other than 0) options whose tensors are on another device than the call's."""
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    at0 = lambda *s, t=torch.float32: Elsewhere(torch.zeros(*s, dtype=t), 0)  # noqa: E731
    cfg = moe.config(T, D, E, K, F)
    ws = Elsewhere(torch.zeros(moe.moe_workspace_size(cfg), dtype=torch.uint8), 0)
    x, wg = at0(T, D, t=torch.bfloat16), at0(E, D, t=torch.bfloat16)
    idx, w = at0(T, K, t=torch.int32), at0(T, K)
    wgu, wd = at0(E, 2 * F, D, t=torch.bfloat16), at0(E, D, F, t=torch.bfloat16)
    out = at0(T, D, t=torch.bfloat16)
    short = 0 if index else 1
    for kw in (dict(score_bias=torch.zeros(E - short)), dict(norm_weight=torch.zeros(D - short))):
        opt = moe.route_options(**kw)
        opt.tensors = [t if t is None else Elsewhere(t, index) for t in opt.tensors]
        refused(moe.moe_route4, cfg, x, wg, None, opt, None, idx, w, ws)
        refused(moe.moe_forward4, cfg, x, wg, None, opt, None, wgu, None, wd, None, out, ws)
        if "score_bias" in kw:
            refused(moe.moe_select, cfg, at0(T, E), opt, None, idx, w)
