"""Refusals of the calls around the expert layer (balance loss, block norms, combine with norms):
the documented status codes, before anything is enqueued, so they run without a GPU."""
import ctypes
import math

import pytest
import torch

import mixture_experts_layer_logits_amd as m
from test_abi import LIB, MOE_EALIGN, MOE_EINVAL, MOE_ENULL, MOE_EWORKSPACE, Shape

P = ctypes.c_void_p
A = 0x1000          # an aligned address (never followed: every call here is refused)
BIG = 1 << 40


@pytest.fixture(scope="module")
def lib():
    return m.load_library(LIB)


def _shape(T=64, d=128, E=8, k=2, act=m.MOE_BF16):
    return Shape(T, d, 64, E, k, act, 0 if act == m.MOE_F32 else 1, 0)


def _call(lib, name, shape, args):
    """args in order, without shape, sizes and stream; floats as they are, pointers as ints."""
    raw = []
    for a in args:
        raw.append(ctypes.c_float(a) if isinstance(a, float) else
                   ctypes.c_size_t(a[0]) if isinstance(a, tuple) else P(a))
    fn = getattr(ctypes.CDLL(LIB), name)  # own prototype: raw addresses instead of tensors
    return fn(ctypes.byref(shape), *raw, P(0))


BAL_FWD = dict(logits=A, topk_idx=A, mask=0, lse=A, counts=A, prob_mean=A, loss=A, ws=A, ws_bytes=(BIG,))
BAL_BWD = dict(logits=A, lse=A, counts=A, dloss=A, dgates=A, gates=A, topk_idx=A, dlogits=A)
NORM_FWD = dict(x=A, y=A, gate=A, w_post=A, w_pre=A, res_scale=1.0, eps=1e-6, v=A, xn=A, rstd_post=A, rstd_pre=A)
NORM_BWD = dict(dv=A, dxn=A, v=A, y=A, gate=A, w_post=A, w_pre=A, rstd_post=A, rstd_pre=A, res_scale=1.0, dx=A, dy=A,
                dgate=A, dw_post=A, dw_pre=A, ws=A, ws_bytes=(BIG,))
COMB = dict(y_perm=A, gates=A, slot_row=A, y_add=0, x=A, gate=A, w_post=A, w_pre=A, res_scale=1.0, eps=1e-6, v=A, xn=A,
            rstd_post=A, rstd_pre=A)
COMB_BWD = dict(dv=A, dxn=A, v=A, y_perm=A, gates=A, slot_row=A, y_add=0, gate=A, w_post=A, w_pre=A, rstd_post=A,
                rstd_pre=A, res_scale=1.0, dx=A, dy=A, dy_perm=2 * A, dgates=A, dgate=A, dw_post=A, dw_pre=A, ws=A,
                ws_bytes=(BIG,))
CALLS = {"moe_balance_fwd": BAL_FWD, "moe_balance_bwd": BAL_BWD, "moe_block_norm_fwd": NORM_FWD,
         "moe_block_norm_bwd": NORM_BWD, "moe_combine_norm": COMB, "moe_combine_norm_bwd": COMB_BWD}

REFUSED = (
    [("moe_balance_fwd", {n: 0}, MOE_ENULL) for n in BAL_FWD if n not in ("mask", "ws_bytes")] +
    [("moe_balance_fwd", dict(ws_bytes=(16,)), MOE_EWORKSPACE), ("moe_balance_fwd", dict(ws=A + 4), MOE_EALIGN)] +
    [("moe_balance_bwd", {n: 0}, MOE_ENULL) for n in BAL_BWD if n != "dgates"] +
    [("moe_block_norm_fwd", {n: 0}, MOE_ENULL) for n in ("x", "v", "xn", "rstd_post", "rstd_pre")] +
    [("moe_block_norm_fwd", {n: A + 8}, MOE_EALIGN) for n in ("x", "y", "w_post", "w_pre", "v", "xn")] +
    [("moe_block_norm_fwd", dict(eps=e), MOE_EINVAL) for e in (0.0, -1e-6, 1e-40, math.nan, math.inf)] +
    [("moe_block_norm_fwd", dict(res_scale=e), MOE_EINVAL) for e in (math.nan, -math.inf)] +
    # pointers the call has no use for
    [("moe_block_norm_fwd", dict(y=0), MOE_EINVAL), ("moe_block_norm_fwd", dict(w_pre=0), MOE_EINVAL),
     ("moe_block_norm_fwd", dict(w_post=0), MOE_EINVAL),
     ("moe_block_norm_fwd", dict(y=0, gate=0, w_post=0, v=0, rstd_post=0, w_pre=0, xn=0, rstd_pre=0), MOE_EINVAL)] +
    [("moe_block_norm_bwd", {n: 0}, MOE_ENULL) for n in ("dxn", "v", "rstd_post", "rstd_pre", "dx", "dy", "ws")] +
    [("moe_block_norm_bwd", {n: A + 8}, MOE_EALIGN)
     for n in ("dv", "dxn", "v", "y", "w_post", "w_pre", "dx", "dy", "dw_post", "dw_pre", "ws")] +
    [("moe_block_norm_bwd", dict(ws_bytes=(64,)), MOE_EWORKSPACE), ("moe_block_norm_bwd", dict(y=0), MOE_EINVAL),
     ("moe_block_norm_bwd", dict(w_post=0), MOE_EINVAL), ("moe_block_norm_bwd", dict(w_pre=0), MOE_EINVAL),
     ("moe_block_norm_bwd", dict(gate=0), MOE_EINVAL), ("moe_block_norm_bwd", dict(res_scale=math.inf), MOE_EINVAL),
     ("moe_block_norm_bwd", dict(dv=0, w_pre=0, dxn=0, dw_pre=0, rstd_pre=0), MOE_ENULL)] +
    [("moe_combine_norm", {n: 0}, MOE_ENULL) for n in ("y_perm", "gates", "slot_row", "x", "v", "xn", "rstd_post")] +
    [("moe_combine_norm", {n: A + 8}, MOE_EALIGN) for n in ("y_perm", "y_add", "x", "v", "xn")] +
    [("moe_combine_norm", dict(eps=0.0), MOE_EINVAL)] +
    [("moe_combine_norm_bwd", {n: 0}, MOE_ENULL)
     for n in ("dxn", "v", "y_perm", "gates", "slot_row", "dy_perm", "dgates", "dx", "rstd_post", "ws")] +
    [("moe_combine_norm_bwd", {n: A + 8}, MOE_EALIGN) for n in ("y_perm", "dy_perm", "y_add", "dy", "dx")] +
    [("moe_combine_norm_bwd", dict(dy_perm=A), MOE_EINVAL),   # in place: rows are gathered again
     ("moe_combine_norm_bwd", dict(ws_bytes=(64,)), MOE_EWORKSPACE)]
)


@pytest.mark.parametrize("name,change,code", REFUSED, ids=[f"{n[4:]}-{c}" for n, c, _ in REFUSED])
def test_refused_before_launch(lib, name, change, code):
    assert _call(lib, name, _shape(), {**CALLS[name], **change}.values()) == code


@pytest.mark.parametrize("name", CALLS)
@pytest.mark.parametrize("shape", [dict(T=-1), dict(E=4, k=5), dict(E=1025), dict(d=100), dict(k=0)], ids=str)
def test_bad_shapes_refused(lib, name, shape):
    assert _call(lib, name, _shape(**shape), CALLS[name].values()) == MOE_EINVAL


@pytest.mark.parametrize("name", [n for n in CALLS if "norm" in n])
def test_rows_wider_than_the_kernels_hold_are_refused(lib, name):
    assert _call(lib, name, _shape(d=16384 + 64), CALLS[name].values()) == MOE_EINVAL


def test_workspace_covers_the_calls(lib):
    """What moe_workspace_size reports passes each call's own workspace check: one byte less than
    the need is refused, and the need is never more than reported."""
    for T, d, E, k in [(1, 64, 2, 1), (8192, 2048, 128, 4), (65521, 64, 96, 6), (100, 16384, 1024, 8)]:
        s = m.make_shape(T, d, 64, E, k)
        size = m.moe_workspace_size(s)
        assert size >= min(T, 512) * d * 8
        raw = Shape(T, d, 64, E, k, 1, 1, 0)
        need = min(T, 512) * d * 8
        assert _call(lib, "moe_block_norm_bwd", raw, {**NORM_BWD, "ws_bytes": (need - 1,)}.values()) == MOE_EWORKSPACE
        # large enough for the workspace check, then refused for its null output
        assert _call(lib, "moe_block_norm_bwd", raw, {**NORM_BWD, "ws_bytes": (size,), "dx": 0}.values()) == MOE_ENULL


def test_binding_refuses_tensors_off_the_gpu():
    s = m.make_shape(4, 64, 64, 2, 1, m.MOE_F32)
    x, r = torch.zeros(4, 64), torch.zeros(4)
    with pytest.raises(ValueError, match="must live on the GPU"):
        m.moe_block_norm_fwd(s, x, None, None, None, torch.ones(64), 1.0, 1e-6, None, x.clone(), None, r)
    with pytest.raises(ValueError, match="must live on the GPU"):
        m.moe_balance_fwd(s, torch.zeros(4, 2), torch.zeros(4, 1, dtype=torch.int32), None, r,
                          torch.zeros(3, dtype=torch.int32), torch.zeros(2), torch.zeros(2), x)
