"""The MoE expert layer as a sequence of C-ABI calls.

``MoEExpertLayer`` owns the device buffers of one layer shape (allocated once with
torch, which is used only for device memory and the stream) and runs the forward and
backward passes as the library's calls, in order, on the current stream:

  forward   moe_router_fwd -> moe_route        (learned routing)
            or moe_route_given                 (tokens arrive routed)
            -> moe_permute -> moe_grouped_ffn_fwd -> moe_combine
  backward  moe_combine_bwd -> the expert GEMMs' dgrad2, wgrad2, dgrad1
            -> moe_route_bwd -> moe_router_bwd (learned routing; dWr only)
            -> moe_permute_bwd_router (learned routing) or moe_permute_bwd
            -> wgrad1 (last, after the un-permute has read dx_perm)

Router input gradient (``router_dx_fused``, on by default): the gates are a softmax over
each token's k chosen scores, so dlogits is zero outside them and dx_r = dlogits Wr is k
rows of Wr per token.  moe_permute_bwd_router adds those rows while it gathers the token's
routed rows of dx_perm, so no dense dlogits Wr GEMM runs and no dx_r is written or read
(bigchange.ai, section "Что инженер может попробовать на практике", for the learned
router).  ``router_dx_fused=False`` keeps the dense GEMM into ``dx_r`` and the plain
un-permute.

Nothing is copied back to the host between calls; routing counts and offsets stay on
the GPU (unite.ai, "Ai2 κυκλοφορεί το Olmo-Core 3…", section "Παραλληλισμός, Ακρίβεια
και Τεχνικές Μνήμης").  ``MoEExpertFunction`` wraps the same calls as a
torch.autograd.Function.

Shared expert (``shared_f > 0``): one always-on SwiGLU expert of width ``shared_f`` sees
every token (bigchange.ai, "Olmo-core 3 открывает стек обучения MoE…", section "Что
инженер может попробовать на практике": the production rows use top-four routing and
one shared expert).  It runs as a one-group call of the same grouped GEMMs over the T
token rows (E = 1, k = 1, offsets [0, T]); its output enters through moe_combine's
``y_add`` and its input gradient through moe_permute_bwd's ``dx_add``.

MXFP8 scope (``mx_scope``, MOE_MX_* bits; MOE_MX_DEFAULT = GEMM2 and dgrad1): the expert
GEMMs that take E4M3 operands when ``gemm`` is MOE_MXFP8; the others run bf16.

MXFP8 operands from the producing epilogue (``mx_fused_quant``, on by default where it
applies): when GEMM2 runs MXFP8 and GEMM1 bf16 (the default scope), GEMM1's epilogue also
writes h as MXFP8 row blocks and GEMM2 reads those; likewise dgrad2's epilogue writes
[da | db] for an MXFP8 dgrad1.  The bytes are the ones the GEMM would quantise itself, so the
results are bit-identical and two standalone quantiser passes over h and [da | db] go away.

MXFP8 dispatch (``mx_dispatch``; on by default when the scope holds all four GEMMs that
read the dispatched rows: GEMM1 and wgrad1 read x's, dgrad2 and wgrad2 the output
gradient's): moe_permute_mx and moe_combine_bwd_mx write the routed rows of x and of the
output gradient only as E4M3 codes with their block scales, in the row layout (forward /
data-gradient GEMMs) and the per-expert column layout (weight-gradient GEMMs), so no bf16
x_perm or dy_perm exists and the GEMMs quantise neither (MXFP8 for the data moved to the
experts: unite.ai, section "Παραλληλισμός, Ακρίβεια και Τεχνικές Μνήμης").  The results
are bit-identical with the bf16 dispatch.

Activation recompute (``recompute=True``): the forward keeps only ``x_perm`` of the
expert FFN; ``ab = [a | b]`` and ``h`` live in buffers allocated for the forward's GEMM1 /
GEMM2 and released right after, and the backward runs GEMM1 again (same kernel, same
inputs, so bit-identical ``ab`` and ``h``) before the gradient GEMMs.  This trades one
extra GEMM1 per step for R * 3f activation elements held between the passes, the
memory / throughput trade the pages report for recomputing activations (unite.ai,
section "Παραλληλισμός, Ακρίβεια και Τεχνικές Μνήμης").

8-bit checkpoints (``ckpt8=True``): what the backward needs of the expert FFN is kept in 8 bits.
[a | b] leaves GEMM1's epilogue as MXINT8 (moe_ffn_gemm1_fwd_c8) and the dgrad2 epilogue reads it
and writes h again for wgrad2 (moe_ffn_dgrad2_c8); the combine keeps the routed outputs as MXINT8
(moe_combine_c8) and its backward reads them (moe_combine_bwd_c8); x_perm is gathered again from
the layer's input before wgrad1.  Next to ``recompute`` this holds less and runs no GEMM twice, at
the price of the checkpoint's 8 bits in the gradients (the layer's forward is the same, bit for bit; a
block's carries one rounding more, see MoEBlock).  Where GEMM1 or dgrad2 does not run bf16 the rows go
through moe_ckpt8_pack and moe_ckpt8_unpack instead, and an epilogue that writes the checkpoint writes no
MXFP8 operands: a GEMM that takes them quantises them itself (a step at E = 128, T = 8192, d = 2048, f = 1024
takes 2.23 ms against 2.17 in bf16, 2.51 against 2.43 with the default MXFP8 scope, 3.34 against 3.19 with all).

4-bit weights (``weights4=True``, serving: no backward): W1, W3, W2 are given as the (codes, scales)
pairs that ``quantize_weights`` makes, and the expert products are moe_ffn_gemm1_fwd_w4 and
moe_ffn_gemm2_fwd_w4 on the unquantised rows.

Router losses (``balance=(w_balance, w_z)``, learned routing): the forward also runs
moe_balance_fwd, which leaves the balance loss and the z-loss in ``loss``, the kept tokens'
per-expert counts in ``bal_counts`` and the mean probabilities in ``prob_mean``; ``mask`` (bool or
uint8 [T], 0 = padding) leaves tokens out of all of them.  The backward then takes the gradient of
w_balance loss[0] + w_z loss[1] with the gates' (moe_balance_bwd instead of moe_route_bwd).  That
gradient reaches every expert's score, so the router's input gradient is the dense
dlogits Wr (``router_dx_fused`` is off).

``MoEBlock`` puts the layer between its norms: v = h + res_scale gate (norm(y) w_post) with
y = MoE(norm(h) w_pre), and the norm of the next block in the same pass.
"""
from __future__ import annotations

import math

import torch

from . import (MOE_BF16, MOE_F32, MOE_MX_DGRAD1, MOE_MX_DGRAD2, MOE_MX_GEMM1, MOE_MX_GEMM2, MOE_MX_WGRAD1,
               MOE_MX_WGRAD2, MOE_MXFP8, make_shape, moe_combine, moe_ffn_dgrad1_mx, moe_ffn_dgrad2_q,
               moe_ffn_gemm1_fwd_q, moe_ffn_gemm2_fwd_mx, moe_combine_bwd, moe_combine_bwd_mx,
               moe_ffn_dgrad1, moe_ffn_dgrad2, moe_ffn_dgrad2_mx, moe_ffn_gemm1_fwd, moe_ffn_gemm1_fwd_mx,
               moe_ffn_gemm2_fwd, moe_ffn_wgrad1, moe_ffn_wgrad1_mx, moe_ffn_wgrad2, moe_ffn_wgrad2_mx, moe_mx_cols_ld,
               moe_permute, moe_permute_bwd, moe_permute_bwd_router, moe_permute_mx, moe_route, moe_route_bwd,
               moe_route_given, moe_router_bwd, moe_balance_bwd, moe_balance_fwd, moe_block_norm_bwd,
               moe_block_norm_fwd, moe_combine_norm, moe_combine_norm_bwd, moe_ckpt8_pack, moe_ckpt8_unpack,
               moe_combine_bwd_c8, moe_combine_c8, moe_ffn_dgrad2_c8, moe_ffn_gemm1_fwd_c8, moe_ffn_gemm1_fwd_w4,
               moe_ffn_gemm2_fwd_w4, moe_mx4_quantize, moe_router_fwd, moe_workspace_size, mx_scope_bits)

# the GEMMs that read the dispatched rows: all four must run MXFP8 for the MXFP8 dispatch
_DISPATCH_READERS = MOE_MX_GEMM1 | MOE_MX_WGRAD1 | MOE_MX_DGRAD2 | MOE_MX_WGRAD2


def quantize_weights(*weights):
    """The MXFP4 form of expert weights [.., n, K] (float32 or bfloat16, contiguous, on the GPU): for each a
    pair (codes uint8 [.., n, K/2], scales uint8 [.., n, K/32]), as a layer with ``weights4`` takes them."""
    out = []
    for w in weights:
        rows, K = math.prod(w.shape[:-1]), w.shape[-1]
        q = torch.empty(*w.shape[:-1], K // 2, dtype=torch.uint8, device=w.device)
        s = torch.empty(*w.shape[:-1], K // 32, dtype=torch.uint8, device=w.device)
        moe_mx4_quantize(rows, K, w, q, s)
        out.append((q, s))
    return tuple(out)


class MoEExpertLayer:
    def __init__(self, T, d, f, E, k, act=MOE_BF16, gemm=None, device="cuda", recompute=False, shared_f=0,
                 mx_dispatch=None, mx_scope=0, mx_fused_quant=True, router_dx_fused=True, balance=None, ckpt8=False,
                 weights4=False):
        self.shape = make_shape(T, d, f, E, k, act, gemm, mx_scope)
        self.recompute, self.ckpt8, self.weights4 = recompute, bool(ckpt8), bool(weights4)
        if self.ckpt8 and recompute:
            raise ValueError("a layer recomputes its activations or keeps them in 8 bits, not both")
        if self.weights4 and (recompute or ckpt8 or balance is not None or self.shape.gemm == MOE_MXFP8):
            raise ValueError("a layer with 4-bit weights has no backward (no recompute, ckpt8 or router losses), and "
                             "its products are not MXFP8")
        # the router's input gradient folded into the un-permute (k rows of Wr per token)
        # instead of a dense dlogits Wr GEMM written to dx_r and read back
        # (the router losses' gradient is not zero outside the k chosen experts)
        self.router_dx_fused = bool(router_dx_fused) and balance is None
        self.balance = balance
        bits = mx_scope_bits(self.shape)
        # MXFP8 operands written by the producing bf16 GEMM's epilogue (which writes the checkpoint instead)
        fq = bool(mx_fused_quant) and not self.ckpt8
        self.fq_h = fq and bool(bits & MOE_MX_GEMM2) and not bits & MOE_MX_GEMM1
        self.fq_dab = fq and bool(bits & MOE_MX_DGRAD1) and not bits & MOE_MX_DGRAD2
        # the checkpoint written and read by the GEMMs' own epilogues
        self.c8_fwd = self.ckpt8 and act == MOE_BF16 and not bits & MOE_MX_GEMM1
        self.c8_bwd = self.ckpt8 and act == MOE_BF16 and not bits & MOE_MX_DGRAD2
        covers = (bits & _DISPATCH_READERS) == _DISPATCH_READERS
        self.mx_dispatch = covers if mx_dispatch is None else bool(mx_dispatch)
        if self.mx_dispatch and not covers:
            raise ValueError("the MXFP8 dispatch needs GEMM1, wgrad1, dgrad2 and wgrad2 in the MXFP8 scope")
        self.steps = 0   # forwards run so far: the autograd wrapper checks its backward sees its own
        self.shared_f = shared_f
        self.T, self.d, self.f, self.E, self.k = T, d, f, E, k
        self.R = T * k
        dt = torch.float32 if act == MOE_F32 else torch.bfloat16
        self.dtype = dt
        dev = torch.device(device)
        if dev.type == "cuda" and dev.index is None:  # what later passes allocate lies there too
            dev = torch.device("cuda", torch.cuda.current_device())
        e = lambda *s, dtype=dt: torch.empty(*s, dtype=dtype, device=dev)  # noqa: E731
        R = self.R
        i32, f32 = torch.int32, torch.float32
        # forward buffers
        self.logits = e(T, E, dtype=f32)
        self.topk_idx = e(T, k, dtype=i32)
        self.gates = e(T, k, dtype=f32)
        self.counts = e(E, dtype=i32)
        self.offsets = e(E + 1, dtype=i32)
        self.slot_row = e(T, k, dtype=i32)
        self.row_src = e(R, dtype=i32)
        self.dev_err = torch.zeros(1, dtype=i32, device=dev)
        self._e = e
        u8 = torch.uint8
        if self.mx_dispatch:  # routed rows exist only as E4M3 codes, in the row and column layouts
            L = moe_mx_cols_ld(self.shape)
            self.x_perm = self.dy_perm = None
            self.xq_rows, self.xs_rows = e(R, d, dtype=u8), e(R, d // 32, dtype=u8)
            self.xq_cols, self.xs_cols = e(d, L, dtype=u8), e(d, L // 32, dtype=u8)
            self.dyq_rows, self.dys_rows = e(R, d, dtype=u8), e(R, d // 32, dtype=u8)
            self.dyq_cols, self.dys_cols = e(d, L, dtype=u8), e(d, L // 32, dtype=u8)
        else:
            self.x_perm = None if self.ckpt8 else e(R, d)
            self.dy_perm = None if self.weights4 else e(R, d)
        held = not (recompute or self.ckpt8)
        self.ab = e(R, 2 * f) if held and not self.weights4 else None
        self.h = e(R, f) if held else None
        if self.ckpt8:
            i8 = torch.int8
            self.ab_bits = e(R, 2 * f, dtype=i8), e(R, 2 * f // 32, dtype=u8)  # codes and scales
            self.y_bits = e(R, d, dtype=i8), e(R, d // 32, dtype=u8)
        self.hq_rows = self.hs_rows = self.dabq_rows = self.dabs_rows = None
        if self.fq_h:
            self.hq_rows, self.hs_rows = e(R, f, dtype=u8), e(R, f // 32, dtype=u8)
        if self.fq_dab:
            self.dabq_rows, self.dabs_rows = e(R, 2 * f, dtype=u8), e(R, 2 * f // 32, dtype=u8)
        self.y_perm = None if self.ckpt8 else e(R, d)
        self.y = e(T, d)
        self.ws = torch.empty(moe_workspace_size(self.shape), dtype=torch.uint8, device=dev)
        self.learned = True
        self._params = None
        self._shared = None
        if shared_f:
            fs = shared_f
            self.shape_s = make_shape(T, d, fs, 1, 1, act, gemm, mx_scope)
            self.offsets_s = torch.tensor([0, T], dtype=i32, device=dev)
            self.h_s, self.y_s = None if self.ckpt8 else e(T, fs), e(T, d)
        if self.weights4:
            self.dx = None
            return
        # backward buffers
        self.dgates = e(T, k, dtype=f32)
        self.dab = e(R, 2 * f)
        self.dx_perm = e(R, d)
        self.dW1 = e(E, f, d)
        self.dW3 = e(E, f, d)
        self.dW2 = e(E, d, f)
        self.dlogits = e(T, E, dtype=f32)
        self.dx_r = None if self.router_dx_fused else e(T, d)
        self.dWr = e(E, d, dtype=f32)
        if balance is not None:
            w_balance, w_z = (float(w) for w in balance)
            self.dloss = torch.tensor([w_balance, w_z], dtype=f32, device=dev)
            self.lse, self.prob_mean, self.loss = e(T, dtype=f32), e(E, dtype=f32), e(2, dtype=f32)
            self.bal_counts = e(E + 1, dtype=i32)
        self.dx = e(T, d)
        if shared_f:
            self.ab_s = None if self.ckpt8 else e(T, 2 * fs)
            self.ab_bits_s = (e(T, 2 * fs, dtype=i8), e(T, 2 * fs // 32, dtype=u8)) if self.ckpt8 else None
            self.dab_s, self.dx_s = e(T, 2 * fs), e(T, d)
            if self.fq_h:
                self.hq_s, self.hs_s = e(T, fs, dtype=u8), e(T, fs // 32, dtype=u8)
            if self.fq_dab:
                self.dabq_s, self.dabs_s = e(T, 2 * fs, dtype=u8), e(T, 2 * fs // 32, dtype=u8)
            self.dW1s, self.dW3s, self.dW2s = e(1, fs, d), e(1, fs, d), e(1, d, fs)
            self.ws_s = torch.empty(moe_workspace_size(self.shape_s), dtype=torch.uint8, device=dev)

    # -------------------------------------------------------------- forward
    def _check_losses(self, topk_idx, mask):
        if (self.balance is not None and topk_idx is not None) or (self.balance is None and mask is not None):
            raise ValueError("the router losses need learned routing, and a mask needs the router losses")

    def _check_inputs(self, x, weights):
        if any(isinstance(w, (tuple, list)) != self.weights4 for w in weights):
            raise ValueError("a layer with weights4 takes every weight as a (codes, scales) pair, another none")
        if self.ckpt8 and _shares(x, self.y, self.dx):
            raise ValueError("a layer with ckpt8 reads its input again in the backward: it cannot lie in the layer's "
                             "y or dx")

    def route(self, x=None, Wr=None, bias=None, topk_idx=None, mask=None):
        s = self.shape
        self._check_losses(topk_idx, mask)
        if topk_idx is None:
            self.learned = True
            moe_router_fwd(s, x, Wr, bias, self.logits)
            moe_route(s, self.logits, self.topk_idx, self.gates, self.counts, self.offsets, self.slot_row, self.ws)
            if self.balance is not None:
                moe_balance_fwd(s, self.logits, self.topk_idx, mask, self.lse, self.bal_counts, self.prob_mean,
                                self.loss, self.ws)
        else:  # the caller's ids are only read; the layer's own topk_idx buffer is left alone
            self.learned = False
            moe_route_given(s, topk_idx, self.counts, self.offsets, self.slot_row, self.dev_err, self.ws)

    def forward(self, x, W1, W3, W2, Wr=None, bias=None, topk_idx=None, gates=None, shared=None, mask=None):
        """shared: (W1s [1, fs, d], W3s [1, fs, d], W2s [1, d, fs]) of the shared expert.
        mask: bool or uint8 [T], 0 for a token the router losses leave out.
        With weights4 every weight is a (codes, scales) pair.  x and the weights have to stay as they are
        until the backward."""
        y_add = self._experts_forward(x, W1, W3, W2, Wr, bias, topk_idx, gates, shared, mask)
        return self._combine(y_add)

    def _combine(self, y_add):
        s, g = self.shape, self._params[-1]
        if self.ckpt8:  # y_perm itself is not kept for the backward
            moe_combine_c8(s, self.y_perm, g, self.slot_row, y_add, self.y, *self.y_bits)
            self.y_perm = None
        else:
            moe_combine(s, self.y_perm, g, self.slot_row, y_add, self.y)
        return self.y

    def _experts_forward(self, x, W1, W3, W2, Wr, bias, topk_idx, gates, shared, mask):
        """The forward up to the routed rows y_perm; returns the shared expert's output or None."""
        s = self.shape
        self._check_losses(topk_idx, mask)
        self._check_inputs(x, (W1, W3, W2, *(shared or ())))
        self.steps += 1
        self.route(x, Wr, bias, topk_idx, mask)
        g = self.gates if topk_idx is None else gates
        self._params = (x, W1, W3, W2, Wr, g)
        self._shared = shared
        y_add = None
        if shared is not None:
            W1s, W3s, W2s = shared
            ss = self.shape_s
            if self.weights4:
                self._ffn_w4(ss, x, *shared, self.offsets_s, self.h_s, self.y_s)
            elif self.ckpt8:
                h = self._e(self.T, self.shared_f)
                self._gemm1_c8(ss, x, W1s, W3s, self.offsets_s, h, self.ab_bits_s, self.ws_s)
                moe_ffn_gemm2_fwd(ss, h, W2s, self.offsets_s, self.y_s, self.ws_s)
            elif self.fq_h:
                moe_ffn_gemm1_fwd_q(ss, x, W1s, W3s, self.offsets_s, self.ab_s, self.h_s, self.hq_s, self.hs_s)
                moe_ffn_gemm2_fwd_mx(ss, self.hq_s, self.hs_s, W2s, self.offsets_s, self.y_s, self.ws_s)
            else:
                moe_ffn_gemm1_fwd(ss, x, W1s, W3s, self.offsets_s, self.ab_s, self.h_s, self.ws_s)
                moe_ffn_gemm2_fwd(ss, self.h_s, W2s, self.offsets_s, self.y_s, self.ws_s)
            y_add = self.y_s
        if self.ckpt8:
            self.y_perm = self._e(self.R, self.d)
        if self.mx_dispatch:
            moe_permute_mx(s, x, self.slot_row, self.offsets, self.row_src, self.xq_rows, self.xs_rows, self.xq_cols,
                           self.xs_cols)
        else:
            if self.ckpt8:
                self.x_perm = self._e(self.R, self.d)
            moe_permute(s, x, self.slot_row, self.row_src, self.x_perm)
        if self.weights4:
            self._ffn_w4(s, self.x_perm, W1, W3, W2, self.offsets, self.h, self.y_perm)
            return y_add
        if self.ckpt8:
            self.h = self._e(self.R, self.f)
            self._gemm1_c8(s, self.x_perm, W1, W3, self.offsets, self.h, self.ab_bits, self.ws)
            self.x_perm = None  # gathered again where the backward needs it
            moe_ffn_gemm2_fwd(s, self.h, W2, self.offsets, self.y_perm, self.ws)
            self.h = None
            return y_add
        if self.recompute:
            self.ab, self.h = self._e(self.R, 2 * self.f), self._e(self.R, self.f)
        self._gemm1(W1, W3, with_q=True)
        if self.fq_h:
            moe_ffn_gemm2_fwd_mx(s, self.hq_rows, self.hs_rows, W2, self.offsets, self.y_perm, self.ws)
        else:
            moe_ffn_gemm2_fwd(s, self.h, W2, self.offsets, self.y_perm, self.ws)
        if self.recompute:  # the SwiGLU activations are not kept for the backward
            self.ab = self.h = None
        return y_add

    @staticmethod
    def _ffn_w4(s, x, W1, W3, W2, offsets, h, y):
        moe_ffn_gemm1_fwd_w4(s, x, *W1, *W3, offsets, h)
        moe_ffn_gemm2_fwd_w4(s, h, *W2, offsets, y)

    def _gemm1_c8(self, s, x, W1, W3, offsets, h, bits, ws):
        """GEMM1 with [a | b] left in `bits` (codes, scales) instead of bf16 or fp32 rows."""
        if self.c8_fwd:
            moe_ffn_gemm1_fwd_c8(s, x, W1, W3, offsets, h, *bits)
            return
        n = s.T * s.k
        ab = self._e(n, 2 * s.f)
        if self.mx_dispatch and s is self.shape:
            moe_ffn_gemm1_fwd_mx(s, self.xq_rows, self.xs_rows, W1, W3, offsets, ab, h, ws)
        else:
            moe_ffn_gemm1_fwd(s, x, W1, W3, offsets, ab, h, ws)
        moe_ckpt8_pack(n, 2 * s.f, ab, *bits)

    def _dgrad2_c8(self, s, dy, W2, offsets, bits, dab, ws):
        """[da | db] from the 8-bit [a | b]; returns h of the same a and b."""
        n = s.T * s.k
        h = self._e(n, s.f)
        if self.c8_bwd:
            moe_ffn_dgrad2_c8(s, dy, W2, *bits, offsets, dab, h)
            return h
        ab = self._e(n, 2 * s.f)
        moe_ckpt8_unpack(n, 2 * s.f, *bits, ab, h)
        if self.mx_dispatch and s is self.shape:
            moe_ffn_dgrad2_mx(s, self.dyq_rows, self.dys_rows, W2, ab, offsets, dab, ws)
        else:
            moe_ffn_dgrad2(s, dy, W2, ab, offsets, dab, ws)
        return h

    def _check_backward(self):
        if self.weights4:
            raise RuntimeError("a layer with 4-bit weights has no backward")

    # -------------------------------------------------------------- backward
    def backward(self, dy, dloss=None):
        """dloss: float32 [2] on the GPU, the weights of the router losses in place of the layer's."""
        self._check_backward()
        self._combine_bwd(dy)
        self._input_grads(dy, dloss)
        return self._finish_backward()

    def _combine_bwd(self, dy):
        s, g = self.shape, self._params[-1]
        if self.ckpt8 and self.mx_dispatch:
            y_perm = self._e(self.R, self.d)
            moe_ckpt8_unpack(self.R, self.d, *self.y_bits, y_perm)
        elif self.ckpt8:
            moe_combine_bwd_c8(s, dy, *self.y_bits, g, self.slot_row, self.dy_perm, self.dgates)
            return
        else:
            y_perm = self.y_perm
        if self.mx_dispatch:
            moe_combine_bwd_mx(s, dy, y_perm, g, self.slot_row, self.row_src, self.offsets, self.dgates, self.dyq_rows,
                               self.dys_rows, self.dyq_cols, self.dys_cols)
        else:
            moe_combine_bwd(s, dy, y_perm, g, self.slot_row, self.dy_perm, self.dgates)

    def _input_grads(self, dy, dloss=None):
        """The backward behind the combine's, up to dx: dy_perm and dgates are in place, dy is read
        by the shared expert alone.  wgrad1 is left to _finish_backward."""
        s = self.shape
        x, W1, W3, W2, Wr, g = self._params
        if self.recompute:  # regenerate a, b and h from the kept routed rows
            self.ab, self.h = self._e(self.R, 2 * self.f), self._e(self.R, self.f)
            self._gemm1(W1, W3)
        if self.ckpt8:
            h = self._dgrad2_c8(s, self.dy_perm, W2, self.offsets, self.ab_bits, self.dab, self.ws)
            if self.mx_dispatch:
                moe_ffn_wgrad2_mx(s, h, self.dyq_cols, self.dys_cols, self.offsets, self.dW2, self.ws)
            else:
                moe_ffn_wgrad2(s, h, self.dy_perm, self.offsets, self.dW2, self.ws)
            del h
            moe_ffn_dgrad1(s, self.dab, W1, W3, self.offsets, self.dx_perm, self.ws)
        elif self.mx_dispatch:
            moe_ffn_dgrad2_mx(s, self.dyq_rows, self.dys_rows, W2, self.ab, self.offsets, self.dab, self.ws)
            moe_ffn_wgrad2_mx(s, self.h, self.dyq_cols, self.dys_cols, self.offsets, self.dW2, self.ws)
            moe_ffn_dgrad1(s, self.dab, W1, W3, self.offsets, self.dx_perm, self.ws)
        else:
            if self.fq_dab:
                moe_ffn_dgrad2_q(s, self.dy_perm, W2, self.ab, self.offsets, self.dab, self.dabq_rows,
                                 self.dabs_rows)
            else:
                moe_ffn_dgrad2(s, self.dy_perm, W2, self.ab, self.offsets, self.dab, self.ws)
            moe_ffn_wgrad2(s, self.h, self.dy_perm, self.offsets, self.dW2, self.ws)
            if self.fq_dab:
                moe_ffn_dgrad1_mx(s, self.dabq_rows, self.dabs_rows, W1, W3, self.offsets, self.dx_perm, self.ws)
            else:
                moe_ffn_dgrad1(s, self.dab, W1, W3, self.offsets, self.dx_perm, self.ws)
        dx_r = None
        if self.learned:
            if self.balance is not None:
                moe_balance_bwd(s, self.logits, self.lse, self.bal_counts, self.dloss if dloss is None else dloss,
                                self.dgates, g, self.topk_idx, self.dlogits)
            else:
                moe_route_bwd(s, self.dgates, g, self.topk_idx, self.dlogits)
            moe_router_bwd(s, x, Wr, self.dlogits, self.dx_r, self.dWr, self.ws)
            dx_r = self.dx_r
        dx_add = None
        if self._shared is not None:
            W1s, W3s, W2s = self._shared
            ss, off = self.shape_s, self.offsets_s
            h_s = self.h_s
            if self.ckpt8:
                h_s = self._dgrad2_c8(ss, dy, W2s, off, self.ab_bits_s, self.dab_s, self.ws_s)
            elif self.fq_dab:
                moe_ffn_dgrad2_q(ss, dy, W2s, self.ab_s, off, self.dab_s, self.dabq_s, self.dabs_s)
            else:
                moe_ffn_dgrad2(ss, dy, W2s, self.ab_s, off, self.dab_s, self.ws_s)
            moe_ffn_wgrad2(ss, h_s, dy, off, self.dW2s, self.ws_s)
            del h_s
            if self.fq_dab:
                moe_ffn_dgrad1_mx(ss, self.dabq_s, self.dabs_s, W1s, W3s, off, self.dx_s, self.ws_s)
            else:
                moe_ffn_dgrad1(ss, self.dab_s, W1s, W3s, off, self.dx_s, self.ws_s)
            moe_ffn_wgrad1(ss, x, self.dab_s, off, self.dW1s, self.dW3s, self.ws_s)
            dx_add = self.dx_s
        if self.learned and self.router_dx_fused:
            moe_permute_bwd_router(s, self.dx_perm, self.slot_row, self.topk_idx, self.dlogits, Wr, dx_add, self.dx)
        else:
            moe_permute_bwd(s, self.dx_perm, self.slot_row, dx_r, dx_add, self.dx)
        return self.dx

    def _finish_backward(self):
        # wgrad1 goes last: its gradient writes, the largest output of the step, would
        # otherwise push dx_perm out of the memory-side cache before the un-permute reads it
        # (and dx, before a block's first norm does)
        s = self.shape
        if self.mx_dispatch:
            moe_ffn_wgrad1_mx(s, self.xq_cols, self.xs_cols, self.dab, self.offsets, self.dW1, self.dW3, self.ws)
        elif self.ckpt8:
            x_perm = self._e(self.R, self.d)
            moe_permute(s, self._params[0], self.slot_row, None, x_perm)
            moe_ffn_wgrad1(s, x_perm, self.dab, self.offsets, self.dW1, self.dW3, self.ws)
        else:
            moe_ffn_wgrad1(s, self.x_perm, self.dab, self.offsets, self.dW1, self.dW3, self.ws)
        if self.recompute:
            self.ab = self.h = None
        return self.dx

    def _gemm1(self, W1, W3, with_q=False):
        """GEMM1 (with_q: also h's MXFP8 rows, for the forward's MXFP8 GEMM2)."""
        s = self.shape
        if with_q and self.fq_h:
            moe_ffn_gemm1_fwd_q(s, self.x_perm, W1, W3, self.offsets, self.ab, self.h, self.hq_rows, self.hs_rows)
        elif self.mx_dispatch:
            moe_ffn_gemm1_fwd_mx(s, self.xq_rows, self.xs_rows, W1, W3, self.offsets, self.ab, self.h, self.ws)
        else:
            moe_ffn_gemm1_fwd(s, self.x_perm, W1, W3, self.offsets, self.ab, self.h, self.ws)

    def activation_bytes(self):
        """Bytes of expert-FFN activations held from the forward to the backward: the
        routed rows (x_perm, or with the MXFP8 dispatch their two E4M3 layouts with
        scales), y_perm, and ab and h unless they are recomputed.  With ckpt8 the 8-bit ab and
        y_perm in their place (and no bf16 routed rows).  Of the layer alone: a block holds more
        (MoEBlock)."""
        if self.weights4:
            return 0
        eb = self.y.element_size()
        if self.ckpt8:
            n = sum(t.numel() for t in (*self.ab_bits, *self.y_bits))
            return n + (sum(t.numel() for t in (self.xq_rows, self.xs_rows, self.xq_cols, self.xs_cols))
                        if self.mx_dispatch else 0)
        n = self.R * self.d * eb
        if self.mx_dispatch:
            n += sum(t.numel() for t in (self.xq_rows, self.xs_rows, self.xq_cols, self.xs_cols))
        else:
            n += self.R * self.d * eb
        if not self.recompute:
            n += self.R * 3 * self.f * eb
        return n


def _shares(t, *others):
    """Does t lie in the memory of one of `others` (None: a buffer that is not there)?"""
    at = t.untyped_storage().data_ptr()
    return t.numel() > 0 and any(o is not None and at == o.untyped_storage().data_ptr() for o in others)


class MoEBlock:
    """An expert layer between its norms (RMS norms over d, learned scales w_pre and w_post):

      xn = norm(h) w_pre;  y = MoE(xn);  v = h + res_scale gate (norm(y) w_post)
      xn_next = norm(v) w_next      the next block's xn, in the pass that writes v

    forward   moe_block_norm_fwd (unless xn is given) -> the layer's calls up to y_perm
              -> moe_combine_norm
    backward  moe_combine_norm_bwd -> the layer's calls from dy_perm to dx
              -> moe_block_norm_bwd (unless xn was given) -> wgrad1

    y is never stored: the combine's norm takes it from registers and the backward gathers it
    again.  A layer with the MXFP8 dispatch writes its routed gradient rows in E4M3 from dy, and one
    with 8-bit checkpoints keeps its routed outputs in the combine, so there the combine and the norm
    are separate calls and y is stored: v and xn_next follow from y rounded to the layer's type
    instead of from the fp32 sum, and y [T, d] is held until the backward.  Over a layer with 4-bit
    weights the block serves: it has no backward, and no buffers for one.  The block owns its buffers
    and holds one forward at a time, like its layer, and its calls run on the current stream."""

    def __init__(self, layer: MoEExpertLayer, res_scale=1.0, eps=1e-6):
        self.layer, self.res_scale, self.eps = layer, float(res_scale), float(eps)
        self._saved = None
        self._stores_y = layer.mx_dispatch or layer.ckpt8
        e, T, d, f32 = layer._e, layer.T, layer.d, torch.float32
        self.xn, self.v, self.xn_next = e(T, d), e(T, d), e(T, d)
        self.rstd_pre, self.rstd_post, self.rstd_next = e(T, dtype=f32), e(T, dtype=f32), e(T, dtype=f32)
        self.dv = self.dh = self.dy = self.dgate = self.dw_pre = self.dw_post = self.dw_next = None
        if layer.weights4:  # serves: no backward
            return
        self.dv, self.dh, self.dy = e(T, d), e(T, d), e(T, d)
        self.dgate = e(T, dtype=f32)
        self.dw_pre, self.dw_post, self.dw_next = e(d, dtype=f32), e(d, dtype=f32), e(d, dtype=f32)

    def forward(self, h, W1, W3, W2, w_pre=None, w_post=None, gate=None, w_next=None, xn=None, Wr=None, bias=None,
                topk_idx=None, gates=None, shared=None, mask=None):
        """h [T, d]; w_pre, or xn = norm(h) w_pre from the block before (its xn_next); w_post [d] or
        None (no norm behind the layer); gate float32 [T] or None; w_next [d] or None.  The rest
        as MoEExpertLayer.forward.  Returns v; xn_next is left in the block."""
        if (xn is None) == (w_pre is None):
            raise ValueError("a block takes w_pre, or the xn of the block before")
        L, s = self.layer, self.layer.shape
        # written before h or xn is read for the last time: by the norm, the combine, or the backward
        work = (self.v, self.xn_next, self.dv, self.dy, L.dx, *((L.y,) if self._stores_y else ()))
        if _shares(h, *work, *((self.xn,) if xn is None else ())) or (xn is not None and _shares(xn, *work)):
            raise ValueError("a block cannot read its own output or working buffers: this forward or its backward "
                             "overwrites them")
        L._check_losses(topk_idx, mask)
        L._check_inputs(self.xn if xn is None else xn, (W1, W3, W2, *(shared or ())))
        if xn is None:
            xn = self.xn
            moe_block_norm_fwd(s, h, None, None, None, w_pre, 1.0, self.eps, None, xn, None, self.rstd_pre)
        # from here on the forward before this one is overwritten, also if a later call is refused
        self._saved, self._own_pre = None, w_pre is not None
        y_add = L._experts_forward(xn, W1, W3, W2, Wr, bias, topk_idx, gates, shared, mask)
        g = L._params[-1]
        out = (gate, w_post, w_next, self.res_scale, self.eps, self.v, None if w_next is None else self.xn_next,
               None if w_post is None else self.rstd_post, None if w_next is None else self.rstd_next)
        if self._stores_y:
            moe_block_norm_fwd(s, h, L._combine(y_add), *out)
        else:
            moe_combine_norm(s, L.y_perm, g, L.slot_row, y_add, h, *out)
        self._saved = (h, gate, w_pre, w_post, w_next, y_add)
        return self.v

    def backward(self, dv, dxn_next=None, dloss=None):
        """dv [T, d] (None: v was used through xn_next only), dxn_next [T, d] with w_next, dloss as
        MoEExpertLayer.backward.  Returns dh; with a given xn, (dh, dxn) for the block before.
        dw_pre, dw_post, dw_next, dgate and the layer's gradients are left in their buffers."""
        self.layer._check_backward()
        if self._saved is None:
            raise RuntimeError("the block has no forward to go back through (none ran, or the last one was refused)")
        L, s = self.layer, self.layer.shape
        h, gate, w_pre, w_post, w_next, y_add = self._saved
        mid = (gate, w_post, w_next, None if w_post is None else self.rstd_post,
               None if w_next is None else self.rstd_next, self.res_scale, self.dv)
        tail = (None if gate is None else self.dgate, None if w_post is None else self.dw_post,
                None if w_next is None else self.dw_next, L.ws)
        g = L._params[-1]
        if self._stores_y:
            moe_block_norm_bwd(s, dv, dxn_next, self.v, L.y, *mid, self.dy, *tail)
            L._combine_bwd(self.dy)
        else:
            moe_combine_norm_bwd(s, dv, dxn_next, self.v, L.y_perm, g, L.slot_row, y_add, *mid,
                                 None if y_add is None else self.dy, L.dy_perm, L.dgates, *tail)
        dxn = L._input_grads(self.dy, dloss)
        if self._own_pre:
            moe_block_norm_bwd(s, self.dv, dxn, h, None, None, None, w_pre, None, self.rstd_pre, 1.0, self.dh, None,
                               None, None, self.dw_pre, L.ws)
        L._finish_backward()
        return self.dh if self._own_pre else (self.dv, dxn)


class _FirstOrder(torch.autograd.Function):
    """Passes gradients on under create_graph.  They depend on `inputs`, but the kernels have no
    derivative of the backward: going back through them raises, instead of leaving that part out."""

    @staticmethod
    def forward(ctx, n, *grads_and_inputs):
        return grads_and_inputs[:n]

    @staticmethod
    def backward(ctx, *_):
        raise RuntimeError("the expert layer's and the block's gradients have no second derivative")

    @classmethod
    def of(cls, grads, *inputs):
        return cls.apply(len(grads), *grads, *inputs) if torch.is_grad_enabled() else grads


class MoEExpertFunction(torch.autograd.Function):
    """y = MoE(x) with learned routing (optional constant per-expert router bias), by the routed
    experts alone (a layer's shared expert takes no part); gradients for x, Wr, W1, W3, W2.  The
    layer's buffers hold one forward at a time, so each backward must follow its own forward: a
    second forward through the same layer before the first one's backward makes that backward
    raise instead of returning the second forward's gradients.  The inputs are autograd's saved
    tensors: one changed in place before the backward makes it raise too."""

    @staticmethod
    def forward(ctx, x, Wr, W1, W3, W2, layer: MoEExpertLayer, bias=None):
        layer._check_backward()
        x, Wr, W1, W3, W2 = (t.contiguous() for t in (x, Wr, W1, W3, W2))
        y = layer.forward(x, W1, W3, W2, Wr=Wr, bias=None if bias is None else bias.contiguous())
        ctx.save_for_backward(x, Wr, W1, W3, W2)
        ctx.layer = layer
        ctx.step = layer.steps
        return y.clone()

    @staticmethod
    def backward(ctx, dy):
        L = ctx.layer
        if L.steps != ctx.step:
            raise RuntimeError("MoEExpertFunction: the layer ran another forward since this one; its saved "
                               "activations are gone (one layer object per in-flight forward)")
        # raises if one of them was changed in place since; under saved-tensor hooks, what these returned
        x, Wr, W1, W3, W2 = ctx.saved_tensors
        L._params = (x, W1, W3, W2, Wr, L._params[-1])
        L.backward(dy.contiguous())
        grads = L.dx.clone(), L.dWr.to(L.dtype, copy=True), L.dW1.clone(), L.dW3.clone(), L.dW2.clone()
        return (*_FirstOrder.of(grads, dy, x, Wr, W1, W3, W2), None, None)


class MoEBlockFunction(torch.autograd.Function):
    """v, loss = block(h) with learned routing; gradients for h, w_pre, w_post, gate (float32 [T]
    or None), Wr, W1, W3, W2.  loss is the layer's float32 [2] of router losses (balance, z), to
    be weighted into the objective like any other value; its weights in the layer are not used.
    The layer must have been made with ``balance`` and without a shared expert.  One forward at
    a time, as MoEExpertFunction.  The inputs are autograd's saved tensors: one changed in place
    before the backward makes it raise."""

    @staticmethod
    def forward(ctx, h, w_pre, w_post, gate, Wr, W1, W3, W2, block: MoEBlock, bias=None, mask=None):
        L = block.layer
        if L.balance is None:
            raise ValueError("MoEBlockFunction needs a layer with router losses (balance=(w_balance, w_z))")
        if L.shared_f:
            raise ValueError("MoEBlockFunction takes no shared expert's weights: its layer must have none")
        c = lambda t: None if t is None else t.contiguous()  # noqa: E731
        h, w_pre, w_post, gate, Wr, W1, W3, W2 = (c(t) for t in (h, w_pre, w_post, gate, Wr, W1, W3, W2))
        v = block.forward(h, W1, W3, W2, w_pre=w_pre, w_post=w_post, gate=gate, Wr=Wr, bias=c(bias), mask=c(mask))
        ctx.save_for_backward(h, w_pre, w_post, gate, Wr, W1, W3, W2)
        ctx.block, ctx.step = block, L.steps
        return v.clone(), L.loss.clone()

    @staticmethod
    def backward(ctx, dv, dloss):
        B, L = ctx.block, ctx.block.layer
        if L.steps != ctx.step:
            raise RuntimeError("MoEBlockFunction: the layer ran another forward since this one; its saved "
                               "activations are gone (one block object per in-flight forward)")
        # raises if one of them was changed in place since; under saved-tensor hooks, what these returned
        h, w_pre, w_post, gate, Wr, W1, W3, W2 = ctx.saved_tensors
        B._saved = (h, gate, w_pre, w_post, *B._saved[4:])
        L._params = (L._params[0], W1, W3, W2, Wr, L._params[-1])
        dh = B.backward(dv.contiguous(), dloss=dloss.contiguous())
        own = lambda t: t.to(L.dtype, copy=True)  # noqa: E731  (the buffers are the next backward's too)
        grads = (own(dh), own(B.dw_pre), None if w_post is None else own(B.dw_post),
                 None if gate is None else B.dgate.clone(), own(L.dWr), own(L.dW1), own(L.dW3), own(L.dW2))
        return (*_FirstOrder.of(grads, dv, dloss, h, w_pre, w_post, gate, Wr, W1, W3, W2), None, None, None)
