"""Python binding of libmoe_mi355x.so (the MI355X MoE expert-layer library).

Argument marshalling only: every function here takes torch tensors that live on the
GPU, checks dtypes/shapes cheaply, and calls the C-ABI entry point of the same name
(declared in include/moe.h) on the current HIP stream.  Every step of the layer runs in
the library's HIP kernels; there is no CPU or PyTorch fallback, and importing this
package fails loudly if the library has not been built.
"""
from __future__ import annotations

import ctypes
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmoe_mi355x.so")

MOE_F32, MOE_BF16, MOE_MXFP8 = 0, 1, 2
MOE_DEVERR_EXPERT_RANGE, MOE_DEVERR_DUPLICATE = 1, 2
# expert GEMMs as bits of moe_shape.mx_scope (include/moe.h)
MOE_MX_GEMM1, MOE_MX_GEMM2, MOE_MX_DGRAD2, MOE_MX_WGRAD2, MOE_MX_DGRAD1, MOE_MX_WGRAD1 = 1, 2, 4, 8, 16, 32
MOE_MX_ALL = 63
MOE_MX_DEFAULT = MOE_MX_GEMM2 | MOE_MX_DGRAD1
MX_BITS = {"gemm1": MOE_MX_GEMM1, "gemm2": MOE_MX_GEMM2, "dgrad2": MOE_MX_DGRAD2, "wgrad2": MOE_MX_WGRAD2,
           "dgrad1": MOE_MX_DGRAD1, "wgrad1": MOE_MX_WGRAD1}


class MoeError(RuntimeError):
    def __init__(self, fn: str, status: int, msg: str):
        super().__init__(f"{fn} failed: {msg} (status {status})")
        self.status = status


class moe_shape(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int32), ("d", ctypes.c_int32), ("f", ctypes.c_int32),
                ("E", ctypes.c_int32), ("k", ctypes.c_int32), ("act", ctypes.c_int32),
                ("gemm", ctypes.c_int32), ("mx_scope", ctypes.c_int32)]

    def __repr__(self):
        return (f"moe_shape(T={self.T}, d={self.d}, f={self.f}, E={self.E}, k={self.k}, "
                f"act={self.act}, gemm={self.gemm}, mx_scope={self.mx_scope})")


def make_shape(T, d, f, E, k, act=MOE_BF16, gemm=None, mx_scope=0) -> moe_shape:
    """mx_scope: MOE_MX_* bits of the expert GEMMs that run MXFP8 when gemm is MOE_MXFP8
    (0: MOE_MX_DEFAULT); must be 0 otherwise."""
    if gemm is None:
        gemm = MOE_F32 if act == MOE_F32 else MOE_BF16
    return moe_shape(T, d, f, E, k, act, gemm, mx_scope)


def mx_scope_bits(shape: moe_shape) -> int:
    """The expert GEMMs that run MXFP8 under `shape`, as MOE_MX_* bits (0 if none)."""
    if shape.gemm != MOE_MXFP8:
        return 0
    return shape.mx_scope or MOE_MX_DEFAULT


_VP = ctypes.c_void_p
_F = ctypes.c_float
_SZ = ctypes.c_size_t
_SHP = ctypes.POINTER(moe_shape)

# entry point -> argument types after the shape pointer (None = no shape argument)
_SIGS = {
    "moe_router_fwd": [_VP, _VP, _VP, _VP, _VP],
    "moe_route": [_VP, _VP, _VP, _VP, _VP, _VP, _VP, _SZ, _VP],
    "moe_route_given": [_VP, _VP, _VP, _VP, _VP, _VP, _SZ, _VP],
    "moe_route_noalloc": [_VP, _VP, _VP, _VP, _VP, _VP, _VP],
    "moe_permute": [_VP, _VP, _VP, _VP, _VP],
    "moe_grouped_ffn_fwd": [_VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _SZ, _VP],
    "moe_ffn_gemm1_fwd": [_VP, _VP, _VP, _VP, _VP, _VP, _VP, _SZ, _VP],
    "moe_ffn_gemm2_fwd": [_VP, _VP, _VP, _VP, _VP, _SZ, _VP],
    "moe_combine": [_VP, _VP, _VP, _VP, _VP, _VP],
    "moe_combine_bwd": [_VP, _VP, _VP, _VP, _VP, _VP, _VP],
    "moe_grouped_ffn_bwd": [_VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _SZ, _VP],
    "moe_ffn_dgrad2": [_VP, _VP, _VP, _VP, _VP, _VP, _SZ, _VP],
    "moe_ffn_wgrad2": [_VP, _VP, _VP, _VP, _VP, _SZ, _VP],
    "moe_ffn_dgrad1": [_VP, _VP, _VP, _VP, _VP, _VP, _SZ, _VP],
    "moe_ffn_wgrad1": [_VP, _VP, _VP, _VP, _VP, _VP, _SZ, _VP],
    "moe_route_bwd": [_VP, _VP, _VP, _VP, _VP],
    "moe_router_bwd": [_VP, _VP, _VP, _VP, _VP, _VP, _SZ, _VP],
    "moe_permute_bwd": [_VP, _VP, _VP, _VP, _VP, _VP],
    "moe_permute_bwd_router": [_VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP],
    # MXFP8 dispatch and the GEMMs that read its quantised rows
    "moe_permute_mx": [_VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP],
    "moe_combine_bwd_mx": [_VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP],
    "moe_ffn_gemm1_fwd_mx": [_VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _SZ, _VP],
    "moe_ffn_dgrad2_mx": [_VP, _VP, _VP, _VP, _VP, _VP, _VP, _SZ, _VP],
    "moe_ffn_wgrad2_mx": [_VP, _VP, _VP, _VP, _VP, _VP, _SZ, _VP],
    "moe_ffn_wgrad1_mx": [_VP, _VP, _VP, _VP, _VP, _VP, _VP, _SZ, _VP],
    # MXFP8 operands written by the producing bf16 GEMM's epilogue
    "moe_ffn_gemm1_fwd_q": [_VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP],
    "moe_ffn_gemm2_fwd_mx": [_VP, _VP, _VP, _VP, _VP, _VP, _SZ, _VP],
    "moe_ffn_dgrad2_q": [_VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP],
    "moe_ffn_dgrad1_mx": [_VP, _VP, _VP, _VP, _VP, _VP, _VP, _SZ, _VP],
    # around the layer: balance loss, block norms, combine with norms
    "moe_balance_fwd": [_VP] * 8 + [_SZ, _VP],
    "moe_balance_bwd": [_VP] * 9,
    "moe_block_norm_fwd": [_VP] * 5 + [_F, _F] + [_VP] * 5,
    "moe_block_norm_bwd": [_VP] * 9 + [_F] + [_VP] * 6 + [_SZ, _VP],
    "moe_combine_norm": [_VP] * 8 + [_F, _F] + [_VP] * 5,
    "moe_combine_norm_bwd": [_VP] * 12 + [_F] + [_VP] * 8 + [_SZ, _VP],
    # expert products with 4-bit weights
    "moe_ffn_gemm1_fwd_w4": [_VP] * 8,
    "moe_ffn_gemm2_fwd_w4": [_VP] * 6,
    # 8-bit activation checkpoints
    "moe_ffn_gemm1_fwd_c8": [_VP] * 8,
    "moe_ffn_dgrad2_c8": [_VP] * 8,
    "moe_combine_c8": [_VP] * 8,
    "moe_combine_bwd_c8": [_VP] * 8,
}
# entry points without a shape argument
_I32T = ctypes.c_int32
_BLOCK_SIGS = {
    "moe_mx4_quantize": [_I32T] * 3 + [_VP] * 4,
    "moe_ckpt8_pack": [_I32T] * 3 + [_VP] * 4,
    "moe_ckpt8_unpack": [_I32T] * 3 + [_VP] * 5,
}
EXPORTED = sorted(list(_SIGS) + list(_BLOCK_SIGS) + ["moe_mx_quantize", "moe_workspace_size", "moe_mx_cols_ld",
                                                     "moe_status_str", "moe_tuning_reload"])

_lib = None


def load_library(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load the built library (raises if it is missing: there is no fallback)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise ImportError(f"{path} is missing: build it with `python -m mixture_experts_layer_logits_amd.build`")
    lib = ctypes.CDLL(path)
    for name, args in _SIGS.items():
        fn = getattr(lib, name)
        fn.argtypes = [_SHP] + args
        fn.restype = ctypes.c_int
    for name, args in _BLOCK_SIGS.items():
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = ctypes.c_int
    lib.moe_mx_quantize.argtypes = [ctypes.c_int32, ctypes.c_int32, ctypes.c_int32, _VP, ctypes.c_int32, _VP, _VP,
                                    _VP, _VP]
    lib.moe_mx_quantize.restype = ctypes.c_int
    lib.moe_workspace_size.argtypes = [_SHP]
    lib.moe_workspace_size.restype = ctypes.c_size_t
    lib.moe_mx_cols_ld.argtypes = [_SHP]
    lib.moe_mx_cols_ld.restype = ctypes.c_size_t
    lib.moe_status_str.argtypes = [ctypes.c_int]
    lib.moe_status_str.restype = ctypes.c_char_p
    lib.moe_tuning_reload.argtypes = []
    lib.moe_tuning_reload.restype = None
    _lib = lib
    return lib


def _p(t):
    if t is None:
        return None
    if isinstance(t, int):
        return t
    if not t.is_cuda:
        raise ValueError("tensor arguments must live on the GPU")
    if not t.is_contiguous():
        raise ValueError("tensor arguments must be contiguous")
    return t.data_ptr()


# the handle and the index alone: a torch Stream object costs a microsecond
_raw_stream, _device = torch._C._cuda_getCurrentRawStream, torch._C._cuda_getDevice


def _stream(stream=None):
    if stream is None:
        return _raw_stream(_device())
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else stream


def _launch(fn, dev, stream, args):
    """fn(*args, stream handle) on GPU `dev` (None: the current one), on that GPU's current stream if
    none is given, whichever GPU is the current one.  args: a list, used up."""
    here = _device()
    if dev is None or dev == here:
        args.append(_raw_stream(here) if stream is None else _stream(stream))
        return fn(*args)
    with torch.cuda.device(dev):
        return fn(*args, _stream(stream))


def _gpu_of(args):
    """The GPU that the first tensor among the arguments lies on (None: raw pointers alone)."""
    for a in args:
        if a is not None and not isinstance(a, (int, ctypes.c_size_t)):
            return a.get_device()
    return None


def _call(name, shape, *args, stream=None):
    lib = load_library()
    st = _launch(getattr(lib, name), _gpu_of(args), stream,
                 [shape, *[_p(a) if not isinstance(a, ctypes.c_size_t) else a for a in args]])
    if st != 0:
        raise MoeError(name, st, lib.moe_status_str(st).decode())


def moe_workspace_size(shape: moe_shape) -> int:
    return int(load_library().moe_workspace_size(ctypes.byref(shape)))


def moe_mx_cols_ld(shape: moe_shape) -> int:
    return int(load_library().moe_mx_cols_ld(ctypes.byref(shape)))


def moe_status_str(status: int) -> str:
    return load_library().moe_status_str(status).decode()


def _ws(ws):
    return ctypes.c_size_t(ws.numel() * ws.element_size())


# ------------------------------------------------------------------ forward
def moe_router_fwd(shape, x, Wr, bias, logits, stream=None):
    _call("moe_router_fwd", shape, x, Wr, bias, logits, stream=stream)


def moe_route(shape, logits, topk_idx, gates, counts, offsets, slot_row, ws, stream=None):
    _call("moe_route", shape, logits, topk_idx, gates, counts, offsets, slot_row, ws, _ws(ws), stream=stream)


def moe_route_noalloc(shape, logits, topk_idx, gates, counts, offsets, slot_row, stream=None):
    _call("moe_route_noalloc", shape, logits, topk_idx, gates, counts, offsets, slot_row, stream=stream)


def moe_route_given(shape, topk_idx, counts, offsets, slot_row, dev_err, ws, stream=None):
    _call("moe_route_given", shape, topk_idx, counts, offsets, slot_row, dev_err, ws, _ws(ws), stream=stream)


def moe_permute(shape, x, slot_row, row_src, x_perm, stream=None):
    _call("moe_permute", shape, x, slot_row, row_src, x_perm, stream=stream)


def moe_grouped_ffn_fwd(shape, x_perm, W1, W3, W2, offsets, ab, h, y_perm, ws, stream=None):
    _call("moe_grouped_ffn_fwd", shape, x_perm, W1, W3, W2, offsets, ab, h, y_perm, ws, _ws(ws), stream=stream)


def moe_ffn_gemm1_fwd(shape, x_perm, W1, W3, offsets, ab, h, ws, stream=None):
    _call("moe_ffn_gemm1_fwd", shape, x_perm, W1, W3, offsets, ab, h, ws, _ws(ws), stream=stream)


def moe_ffn_gemm2_fwd(shape, h, W2, offsets, y_perm, ws, stream=None):
    _call("moe_ffn_gemm2_fwd", shape, h, W2, offsets, y_perm, ws, _ws(ws), stream=stream)


def moe_combine(shape, y_perm, gates, slot_row, y_add, y, stream=None):
    _call("moe_combine", shape, y_perm, gates, slot_row, y_add, y, stream=stream)


# ------------------------------------------------------------------ backward
def moe_combine_bwd(shape, dy, y_perm, gates, slot_row, dy_perm, dgates, stream=None):
    _call("moe_combine_bwd", shape, dy, y_perm, gates, slot_row, dy_perm, dgates, stream=stream)


def moe_grouped_ffn_bwd(shape, dy_perm, x_perm, ab, h, W1, W3, W2, offsets, dab, dx_perm, dW1, dW3, dW2, ws,
                        stream=None):
    _call("moe_grouped_ffn_bwd", shape, dy_perm, x_perm, ab, h, W1, W3, W2, offsets, dab, dx_perm, dW1, dW3, dW2,
          ws, _ws(ws), stream=stream)


def moe_ffn_dgrad2(shape, dy_perm, W2, ab, offsets, dab, ws, stream=None):
    _call("moe_ffn_dgrad2", shape, dy_perm, W2, ab, offsets, dab, ws, _ws(ws), stream=stream)


def moe_ffn_wgrad2(shape, h, dy_perm, offsets, dW2, ws, stream=None):
    _call("moe_ffn_wgrad2", shape, h, dy_perm, offsets, dW2, ws, _ws(ws), stream=stream)


def moe_ffn_dgrad1(shape, dab, W1, W3, offsets, dx_perm, ws, stream=None):
    _call("moe_ffn_dgrad1", shape, dab, W1, W3, offsets, dx_perm, ws, _ws(ws), stream=stream)


def moe_ffn_wgrad1(shape, x_perm, dab, offsets, dW1, dW3, ws, stream=None):
    _call("moe_ffn_wgrad1", shape, x_perm, dab, offsets, dW1, dW3, ws, _ws(ws), stream=stream)


def moe_route_bwd(shape, dgates, gates, topk_idx, dlogits, stream=None):
    _call("moe_route_bwd", shape, dgates, gates, topk_idx, dlogits, stream=stream)


def moe_router_bwd(shape, x, Wr, dlogits, dx_r, dWr, ws, stream=None):
    _call("moe_router_bwd", shape, x, Wr, dlogits, dx_r, dWr, ws, _ws(ws), stream=stream)


def moe_permute_bwd(shape, dx_perm, slot_row, dx_r, dx_add, dx, stream=None):
    _call("moe_permute_bwd", shape, dx_perm, slot_row, dx_r, dx_add, dx, stream=stream)


def moe_permute_bwd_router(shape, dx_perm, slot_row, topk_idx, dlogits, Wr, dx_add, dx, stream=None):
    _call("moe_permute_bwd_router", shape, dx_perm, slot_row, topk_idx, dlogits, Wr, dx_add, dx, stream=stream)


def moe_tuning_reload():
    """Forget the MOE_TILE_* / MOE_GEMM_* / MOE_MX_TILE overrides read so far; each is read
    from the environment again at its next use."""
    load_library().moe_tuning_reload()


# ------------------------------------------------------------------ MXFP8
def moe_mx_quantize(rows, cols, axis, seg_offsets, nseg, src, q, scales, stream=None):
    lib = load_library()
    st = _launch(lib.moe_mx_quantize, _gpu_of((src, q)), stream,
                 [rows, cols, axis, _p(seg_offsets), nseg, _p(src), _p(q), _p(scales)])
    if st != 0:
        raise MoeError("moe_mx_quantize", st, lib.moe_status_str(st).decode())


def moe_permute_mx(shape, x, slot_row, offsets, row_src, q_rows, s_rows, q_cols, s_cols, stream=None):
    _call("moe_permute_mx", shape, x, slot_row, offsets, row_src, q_rows, s_rows, q_cols, s_cols, stream=stream)


def moe_combine_bwd_mx(shape, dy, y_perm, gates, slot_row, row_src, offsets, dgates, q_rows, s_rows, q_cols, s_cols,
                       stream=None):
    _call("moe_combine_bwd_mx", shape, dy, y_perm, gates, slot_row, row_src, offsets, dgates, q_rows, s_rows, q_cols,
          s_cols, stream=stream)


def moe_ffn_gemm1_fwd_mx(shape, xq_rows, xs_rows, W1, W3, offsets, ab, h, ws, stream=None):
    _call("moe_ffn_gemm1_fwd_mx", shape, xq_rows, xs_rows, W1, W3, offsets, ab, h, ws, _ws(ws), stream=stream)


def moe_ffn_dgrad2_mx(shape, dyq_rows, dys_rows, W2, ab, offsets, dab, ws, stream=None):
    _call("moe_ffn_dgrad2_mx", shape, dyq_rows, dys_rows, W2, ab, offsets, dab, ws, _ws(ws), stream=stream)


def moe_ffn_wgrad2_mx(shape, h, dyq_cols, dys_cols, offsets, dW2, ws, stream=None):
    _call("moe_ffn_wgrad2_mx", shape, h, dyq_cols, dys_cols, offsets, dW2, ws, _ws(ws), stream=stream)


def moe_ffn_wgrad1_mx(shape, xq_cols, xs_cols, dab, offsets, dW1, dW3, ws, stream=None):
    _call("moe_ffn_wgrad1_mx", shape, xq_cols, xs_cols, dab, offsets, dW1, dW3, ws, _ws(ws), stream=stream)


def moe_ffn_gemm1_fwd_q(shape, x_perm, W1, W3, offsets, ab, h, hq_rows, hs_rows, stream=None):
    _call("moe_ffn_gemm1_fwd_q", shape, x_perm, W1, W3, offsets, ab, h, hq_rows, hs_rows, stream=stream)


def moe_ffn_gemm2_fwd_mx(shape, hq_rows, hs_rows, W2, offsets, y_perm, ws, stream=None):
    _call("moe_ffn_gemm2_fwd_mx", shape, hq_rows, hs_rows, W2, offsets, y_perm, ws, _ws(ws), stream=stream)


def moe_ffn_dgrad2_q(shape, dy_perm, W2, ab, offsets, dab, dabq_rows, dabs_rows, stream=None):
    _call("moe_ffn_dgrad2_q", shape, dy_perm, W2, ab, offsets, dab, dabq_rows, dabs_rows, stream=stream)


def moe_ffn_dgrad1_mx(shape, dabq_rows, dabs_rows, W1, W3, offsets, dx_perm, ws, stream=None):
    _call("moe_ffn_dgrad1_mx", shape, dabq_rows, dabs_rows, W1, W3, offsets, dx_perm, ws, _ws(ws), stream=stream)


# ------------------------------------------------------------------ around the layer
def _call_checked(name, shape, args, stream=None):
    """Call `name` with shape (None: the call takes none) and args in the C call's order: a tensor as
    (argument name, tensor or None, dtype, number of elements), anything else as it is.  Tensors have to
    lie on one GPU, contiguous, of that type and size (dtype None: a workspace of any type, whose
    size in bytes is passed on behind it).  The call runs on that GPU's current stream if none is
    given, whichever device is the current one."""
    dev = None
    raw = [] if shape is None else [shape]
    put = raw.append
    for a in args:
        if type(a) is not tuple:
            put(a)
            continue
        arg, t, dtype, n = a
        if t is None:
            put(None)
            if dtype is None:
                put(0)
            continue
        at = t.get_device()
        if at != dev:
            if at < 0:
                raise ValueError(f"{name}: {arg} must live on the GPU")
            if dev is not None:
                raise ValueError(f"{name}: {arg} lives on GPU {at}, the arguments before it on GPU {dev}")
            dev = at
        if dtype is None:
            if not t.is_contiguous():
                raise ValueError(f"{name}: {arg} must be contiguous")
            put(t.data_ptr())
            put(t.numel() * t.element_size())
            continue
        if t.dtype is not dtype or t.numel() != n or not t.is_contiguous():
            raise ValueError(f"{name}: {arg} must be contiguous, {dtype}, of {n} elements; got {t.dtype}, shape "
                             f"{tuple(t.shape)}, strides {t.stride()}")
        put(t.data_ptr())
    lib = _lib or load_library()
    st = _launch(getattr(lib, name), dev, stream, raw)
    if st != 0:
        raise MoeError(name, st, lib.moe_status_str(st).decode())


def _act(shape):
    return _F32 if shape.act == MOE_F32 else torch.bfloat16


_F32, _I32, _U8 = torch.float32, torch.int32, torch.uint8


def moe_balance_fwd(shape, logits, topk_idx, mask, lse, counts, prob_mean, loss, ws, stream=None):
    """Balance loss, z-loss and per-expert counts of the kept tokens (mask: bool or uint8 [T], or None)."""
    T, E, k = shape.T, shape.E, shape.k
    if mask is not None and mask.dtype is torch.bool:
        mask = mask.view(_U8)  # the same bytes
    _call_checked("moe_balance_fwd", shape, (
        ("logits", logits, _F32, T * E), ("topk_idx", topk_idx, _I32, T * k), ("mask", mask, _U8, T),
        ("lse", lse, _F32, T), ("counts", counts, _I32, E + 1), ("prob_mean", prob_mean, _F32, E),
        ("loss", loss, _F32, 2), ("ws", ws, None, 0)), stream)


def moe_balance_bwd(shape, logits, lse, counts, dloss, dgates, gates, topk_idx, dlogits, stream=None):
    """dlogits of the losses (weights dloss, a float32 [2] on the GPU) and, with dgates, of the gates."""
    T, E, k = shape.T, shape.E, shape.k
    _call_checked("moe_balance_bwd", shape, (
        ("logits", logits, _F32, T * E), ("lse", lse, _F32, T), ("counts", counts, _I32, E + 1),
        ("dloss", dloss, _F32, 2), ("dgates", dgates, _F32, T * k), ("gates", gates, _F32, T * k),
        ("topk_idx", topk_idx, _I32, T * k), ("dlogits", dlogits, _F32, T * E)), stream)


def moe_block_norm_fwd(shape, x, y, gate, w_post, w_pre, res_scale, eps, v, xn, rstd_post, rstd_pre, stream=None):
    """v = x + res_scale gate (norm(y) w_post), xn = norm(v) w_pre; None leaves a part out."""
    T, d, a = shape.T, shape.d, _act(shape)
    n = T * d
    _call_checked("moe_block_norm_fwd", shape, (
        ("x", x, a, n), ("y", y, a, n), ("gate", gate, _F32, T), ("w_post", w_post, a, d), ("w_pre", w_pre, a, d),
        res_scale, eps, ("v", v, a, n), ("xn", xn, a, n), ("rstd_post", rstd_post, _F32, T),
        ("rstd_pre", rstd_pre, _F32, T)), stream)


def moe_block_norm_bwd(shape, dv, dxn, v, y, gate, w_post, w_pre, rstd_post, rstd_pre, res_scale, dx, dy, dgate,
                       dw_post, dw_pre, ws, stream=None):
    """Gradients of moe_block_norm_fwd; None for what the forward left out or is not wanted."""
    T, d, a = shape.T, shape.d, _act(shape)
    n = T * d
    _call_checked("moe_block_norm_bwd", shape, (
        ("dv", dv, a, n), ("dxn", dxn, a, n), ("v", v, a, n), ("y", y, a, n), ("gate", gate, _F32, T),
        ("w_post", w_post, a, d), ("w_pre", w_pre, a, d), ("rstd_post", rstd_post, _F32, T),
        ("rstd_pre", rstd_pre, _F32, T), res_scale, ("dx", dx, a, n), ("dy", dy, a, n), ("dgate", dgate, _F32, T),
        ("dw_post", dw_post, _F32, d), ("dw_pre", dw_pre, _F32, d), ("ws", ws, None, 0)), stream)


def moe_combine_norm(shape, y_perm, gates, slot_row, y_add, x, gate, w_post, w_pre, res_scale, eps, v, xn, rstd_post,
                     rstd_pre, stream=None):
    """moe_block_norm_fwd of the gated sum of each token's k routed rows (moe_combine), in one pass."""
    T, d, k, a = shape.T, shape.d, shape.k, _act(shape)
    n = T * d
    _call_checked("moe_combine_norm", shape, (
        ("y_perm", y_perm, a, n * k), ("gates", gates, _F32, T * k), ("slot_row", slot_row, _I32, T * k),
        ("y_add", y_add, a, n), ("x", x, a, n), ("gate", gate, _F32, T), ("w_post", w_post, a, d),
        ("w_pre", w_pre, a, d), res_scale, eps, ("v", v, a, n), ("xn", xn, a, n), ("rstd_post", rstd_post, _F32, T),
        ("rstd_pre", rstd_pre, _F32, T)), stream)


def moe_combine_norm_bwd(shape, dv, dxn, v, y_perm, gates, slot_row, y_add, gate, w_post, w_pre, rstd_post, rstd_pre,
                         res_scale, dx, dy, dy_perm, dgates, dgate, dw_post, dw_pre, ws, stream=None):
    """Gradients of moe_combine_norm; None for what the forward left out or is not wanted."""
    T, d, k, a = shape.T, shape.d, shape.k, _act(shape)
    n = T * d
    _call_checked("moe_combine_norm_bwd", shape, (
        ("dv", dv, a, n), ("dxn", dxn, a, n), ("v", v, a, n), ("y_perm", y_perm, a, n * k),
        ("gates", gates, _F32, T * k), ("slot_row", slot_row, _I32, T * k), ("y_add", y_add, a, n),
        ("gate", gate, _F32, T), ("w_post", w_post, a, d), ("w_pre", w_pre, a, d),
        ("rstd_post", rstd_post, _F32, T), ("rstd_pre", rstd_pre, _F32, T), res_scale, ("dx", dx, a, n),
        ("dy", dy, a, n), ("dy_perm", dy_perm, a, n * k), ("dgates", dgates, _F32, T * k), ("dgate", dgate, _F32, T),
        ("dw_post", dw_post, _F32, d), ("dw_pre", dw_pre, _F32, d), ("ws", ws, None, 0)), stream)


# ------------------------------------------------------------------ 4-bit weights
_I8 = torch.int8


def _act_of(name, t, rows, cols):
    """The `act` argument of a call on rows of blocks: the rows' own type."""
    if not (0 <= rows < 1 << 31 and 0 < cols < 1 << 31):  # the call takes 32 bits of each
        raise ValueError(f"{name}: rows {rows} and cols {cols} must fit 32 bits, cols at least 32")
    if t.dtype is not _F32 and t.dtype is not torch.bfloat16:
        raise ValueError(f"{name}: rows must be float32 or bfloat16, got {t.dtype}")
    return MOE_F32 if t.dtype is _F32 else MOE_BF16


def moe_mx4_quantize(rows, cols, src, q, scales, stream=None):
    """MXFP4 of src [rows, cols] (float32 or bfloat16): q uint8 [rows, cols/2], scales uint8 [rows, cols/32]."""
    n = rows * cols
    _call_checked("moe_mx4_quantize", None, (
        rows, cols, _act_of("moe_mx4_quantize", src, rows, cols), ("src", src, src.dtype, n), ("q", q, _U8, n // 2),
        ("scales", scales, _U8, n // 32)), stream)


def moe_ffn_gemm1_fwd_w4(shape, x_perm, W1q, W1s, W3q, W3s, offsets, h, stream=None):
    """h = silu(X_e W1_e^T) (X_e W3_e^T) with MXFP4 weights."""
    d, f, E, a = shape.d, shape.f, shape.E, _act(shape)
    R = shape.T * shape.k
    _call_checked("moe_ffn_gemm1_fwd_w4", shape, (
        ("x_perm", x_perm, a, R * d), ("W1q", W1q, _U8, E * f * d // 2), ("W1s", W1s, _U8, E * f * d // 32),
        ("W3q", W3q, _U8, E * f * d // 2), ("W3s", W3s, _U8, E * f * d // 32), ("offsets", offsets, _I32, E + 1),
        ("h", h, a, R * f)), stream)


def moe_ffn_gemm2_fwd_w4(shape, h, W2q, W2s, offsets, y_perm, stream=None):
    """y_perm = h W2_e^T with MXFP4 weights."""
    d, f, E, a = shape.d, shape.f, shape.E, _act(shape)
    R = shape.T * shape.k
    _call_checked("moe_ffn_gemm2_fwd_w4", shape, (
        ("h", h, a, R * f), ("W2q", W2q, _U8, E * d * f // 2), ("W2s", W2s, _U8, E * d * f // 32),
        ("offsets", offsets, _I32, E + 1), ("y_perm", y_perm, a, R * d)), stream)


# ------------------------------------------------------------------ 8-bit activation checkpoints
def moe_ckpt8_pack(rows, cols, src, q, scales, stream=None):
    """MXINT8 of src [rows, cols] (float32 or bfloat16): q int8 [rows, cols], scales uint8 [rows, cols/32]."""
    n = rows * cols
    _call_checked("moe_ckpt8_pack", None, (
        rows, cols, _act_of("moe_ckpt8_pack", src, rows, cols), ("src", src, src.dtype, n), ("q", q, _I8, n),
        ("scales", scales, _U8, n // 32)), stream)


def moe_ckpt8_unpack(rows, cols, q, scales, dst, h=None, stream=None):
    """The values of MXINT8 rows, in dst's type; with h [rows, cols/2] also silu of each row's first half
    times its second."""
    n = rows * cols
    _call_checked("moe_ckpt8_unpack", None, (
        rows, cols, _act_of("moe_ckpt8_unpack", dst, rows, cols), ("q", q, _I8, n), ("scales", scales, _U8, n // 32),
        ("dst", dst, dst.dtype, n), ("h", h, dst.dtype, n // 2)), stream)


def moe_ffn_gemm1_fwd_c8(shape, x_perm, W1, W3, offsets, h, abq, ab_s, stream=None):
    """moe_ffn_gemm1_fwd (bf16) with [a | b] kept as MXINT8 rows."""
    d, f, E, a = shape.d, shape.f, shape.E, _act(shape)
    R = shape.T * shape.k
    _call_checked("moe_ffn_gemm1_fwd_c8", shape, (
        ("x_perm", x_perm, a, R * d), ("W1", W1, a, E * f * d), ("W3", W3, a, E * f * d),
        ("offsets", offsets, _I32, E + 1), ("h", h, a, R * f), ("abq", abq, _I8, R * 2 * f),
        ("ab_s", ab_s, _U8, R * 2 * f // 32)), stream)


def moe_ffn_dgrad2_c8(shape, dy_perm, W2, abq, ab_s, offsets, dab, h, stream=None):
    """moe_ffn_dgrad2 (bf16) with a and b from MXINT8 rows; writes h again."""
    d, f, E, a = shape.d, shape.f, shape.E, _act(shape)
    R = shape.T * shape.k
    _call_checked("moe_ffn_dgrad2_c8", shape, (
        ("dy_perm", dy_perm, a, R * d), ("W2", W2, a, E * d * f), ("abq", abq, _I8, R * 2 * f),
        ("ab_s", ab_s, _U8, R * 2 * f // 32), ("offsets", offsets, _I32, E + 1), ("dab", dab, a, R * 2 * f),
        ("h", h, a, R * f)), stream)


def moe_combine_c8(shape, y_perm, gates, slot_row, y_add, y, yq, ys, stream=None):
    """moe_combine, with the routed rows also written as MXINT8 rows."""
    T, d, k, a = shape.T, shape.d, shape.k, _act(shape)
    n = T * d
    _call_checked("moe_combine_c8", shape, (
        ("y_perm", y_perm, a, n * k), ("gates", gates, _F32, T * k), ("slot_row", slot_row, _I32, T * k),
        ("y_add", y_add, a, n), ("y", y, a, n), ("yq", yq, _I8, n * k), ("ys", ys, _U8, n * k // 32)), stream)


def moe_combine_bwd_c8(shape, dy, yq, ys, gates, slot_row, dy_perm, dgates, stream=None):
    """moe_combine_bwd with the routed rows read as MXINT8 rows."""
    T, d, k, a = shape.T, shape.d, shape.k, _act(shape)
    n = T * d
    _call_checked("moe_combine_bwd_c8", shape, (
        ("dy", dy, a, n), ("yq", yq, _I8, n * k), ("ys", ys, _U8, n * k // 32), ("gates", gates, _F32, T * k),
        ("slot_row", slot_row, _I32, T * k), ("dy_perm", dy_perm, a, n * k), ("dgates", dgates, _F32, T * k)), stream)


from .layer import MoEBlock, MoEExpertLayer, quantize_weights  # noqa: E402  (re-export)
