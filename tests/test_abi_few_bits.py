"""Refusals of the calls on 4-bit weights and 8-bit checkpoints: the documented status codes, before
anything is enqueued, so they run without a GPU; and what the layer refuses on the host."""
import ctypes
import os

import pytest
import torch

import mixture_experts_layer_logits_amd as m
from test_abi import LIB, MOE_EALIGN, MOE_EINVAL, MOE_ENULL, MOE_EUNSUPPORTED, MOE_OK, Shape

P = ctypes.c_void_p
A = 0x1000          # an aligned address (never followed: every call here is refused)

IN4 = dict(x_perm=A, W1q=A, W1s=A, W3q=A, W3s=A, offsets=A, h=A)
OUT4 = dict(h=A, W2q=A, W2s=A, offsets=A, y_perm=A)
G1C8 = dict(x_perm=A, W1=A, W3=A, offsets=A, h=A, abq=A, ab_s=A)
D2C8 = dict(dy_perm=A, W2=A, abq=A, ab_s=A, offsets=A, dab=A, h=A)
COMB = dict(y_perm=A, gates=A, slot_row=A, y_add=0, y=A, yq=A, ys=A)
COMB_BWD = dict(dy=A, yq=A, ys=A, gates=A, slot_row=A, dy_perm=A, dgates=A)
CALLS = {"moe_ffn_gemm1_fwd_w4": IN4, "moe_ffn_gemm2_fwd_w4": OUT4, "moe_ffn_gemm1_fwd_c8": G1C8,
         "moe_ffn_dgrad2_c8": D2C8, "moe_combine_c8": COMB, "moe_combine_bwd_c8": COMB_BWD}
QUANT = dict(src=A, q=A, scales=A)
UNPACK = dict(q=A, scales=A, dst=A, h=A)
BLOCK_CALLS = {"moe_mx4_quantize": QUANT, "moe_ckpt8_pack": QUANT, "moe_ckpt8_unpack": UNPACK}


def _shape(T=64, d=128, E=8, k=2, act=m.MOE_BF16, gemm=None, scope=0):
    return Shape(T, d, 64 if gemm != m.MOE_MXFP8 else 128, E, k, act,
                 gemm if gemm is not None else (0 if act == m.MOE_F32 else 1), scope)


def _call(name, head, args):
    fn = getattr(ctypes.CDLL(LIB), name)
    head = [ctypes.byref(head)] if isinstance(head, ctypes.Structure) else [ctypes.c_int32(v) for v in head]
    return fn(*head, *[P(a) for a in args], P(0))


REFUSED = ([(c, {n: 0}, MOE_ENULL) for c, args in CALLS.items() for n in args if n != "y_add"] +
           [(c, {n: A + 8}, MOE_EALIGN) for c, args in CALLS.items() for n in args
            if n not in ("offsets", "gates", "slot_row", "dgates")])


@pytest.mark.parametrize("name,change,code", REFUSED, ids=[f"{n[4:]}-{c}" for n, c, _ in REFUSED])
def test_refused_before_launch(name, change, code):
    assert _call(name, _shape(), {**CALLS[name], **change}.values()) == code


@pytest.mark.parametrize("name", CALLS)
@pytest.mark.parametrize("shape", [dict(T=-1), dict(E=4, k=5), dict(E=1025), dict(d=100), dict(k=0)], ids=str)
def test_bad_shapes_refused(name, shape):
    assert _call(name, _shape(**shape), CALLS[name].values()) == MOE_EINVAL


@pytest.mark.parametrize("name", ["moe_ffn_gemm1_fwd_w4", "moe_ffn_gemm2_fwd_w4"])
def test_rows_past_32_bit_offsets_are_refused(name):
    assert _call(name, _shape(d=(1 << 22) + 64), CALLS[name].values()) == MOE_EINVAL
    ok = {**CALLS[name], "offsets": 0}
    assert _call(name, _shape(d=1 << 22), ok.values()) == MOE_ENULL  # not for its width


def test_the_products_hand_rows_over_behind_a_fence():
    """Lanes of a wave that pass routed rows on through LDS order the accesses with lanes.h's fence."""
    src = open(os.path.join(os.path.dirname(LIB), "csrc", "w4.hip")).read()
    body = src[src.index("st.hand_over"):]
    assert body.index("wave_lds_fence()") < body.index("st.multiply(cur")
    assert "wave_lds_fence()" in body[body.index("st.multiply(cur"):body.index("__syncthreads()")]
    assert "__builtin_amdgcn_wave_barrier" not in src


@pytest.mark.parametrize("name", [n for n in CALLS if n != "moe_ffn_gemm1_fwd_c8" and n != "moe_ffn_dgrad2_c8"])
def test_an_empty_batch_needs_no_rows(name):
    args = {n: 0 if n in ("x_perm", "h", "y_perm", "dy", "dy_perm", "y", "yq", "ys", "gates", "slot_row", "dgates")
            else v for n, v in CALLS[name].items()}
    assert _call(name, _shape(T=0), args.values()) == MOE_OK


def test_the_fused_checkpoint_needs_bf16_gemms():
    for name, bit in (("moe_ffn_gemm1_fwd_c8", m.MOE_MX_GEMM1), ("moe_ffn_dgrad2_c8", m.MOE_MX_DGRAD2)):
        args = CALLS[name].values()
        assert _call(name, _shape(act=m.MOE_F32), args) == MOE_EUNSUPPORTED
        assert _call(name, _shape(gemm=m.MOE_MXFP8, scope=bit), args) == MOE_EUNSUPPORTED
        # the other GEMMs in the scope do not matter: refused for its null offsets only
        other = {**CALLS[name], "offsets": 0}
        assert _call(name, _shape(gemm=m.MOE_MXFP8, scope=m.MOE_MX_ALL & ~bit), other.values()) == MOE_ENULL


@pytest.mark.parametrize("name", BLOCK_CALLS)
def test_block_rows_refused(name):
    args = BLOCK_CALLS[name]
    bf16 = m.MOE_BF16
    for head, code in [((-1, 64, bf16), MOE_EINVAL), ((4, 0, bf16), MOE_EINVAL), ((4, 48, bf16), MOE_EINVAL),
                       ((4, 64, 2), MOE_EUNSUPPORTED), ((4, 64, -1), MOE_EUNSUPPORTED)]:
        assert _call(name, head, args.values()) == code
    for n in args:
        if n != "h":
            assert _call(name, (4, 64, bf16), {**args, n: 0}.values()) == MOE_ENULL
        assert _call(name, (4, 64, bf16), {**args, n: A + 8}.values()) == MOE_EALIGN
        assert _call(name, (0, 64, bf16), dict.fromkeys(args, 0).values()) == MOE_OK
    if "h" in args:  # [a | b] needs two halves of whole blocks
        assert _call(name, (4, 32, bf16), args.values()) == MOE_EINVAL
        assert _call(name, (4, 96, bf16), args.values()) == MOE_EINVAL


def test_binding_refuses_types_and_tensors_off_the_gpu():
    x = torch.zeros(4, 64)
    u8 = torch.zeros(4, 32, dtype=torch.uint8)
    with pytest.raises(ValueError, match="must live on the GPU"):
        m.moe_mx4_quantize(4, 64, x, u8, u8)
    with pytest.raises(ValueError, match="float32 or bfloat16"):
        m.moe_mx4_quantize(4, 64, x.half(), u8, u8)
    with pytest.raises(ValueError, match="float32 or bfloat16"):
        m.moe_ckpt8_unpack(4, 64, u8, u8, x.double())
    for call in (m.moe_mx4_quantize, m.moe_ckpt8_pack):
        with pytest.raises(ValueError, match="fit 32 bits"):  # not wrapped to 4 rows
            call((1 << 32) + 4, 64, x, u8, u8)
    with pytest.raises(ValueError, match="fit 32 bits"):
        m.moe_ckpt8_unpack(4, (1 << 32) + 64, u8, u8, x)
    s = m.make_shape(4, 64, 64, 2, 1, m.MOE_F32)
    with pytest.raises(ValueError, match="must live on the GPU"):
        m.moe_ffn_gemm2_fwd_w4(s, x, u8, u8, torch.zeros(3, dtype=torch.int32), x)


def _layer(**kw):
    return m.MoEExpertLayer(4, 64, 64, 2, 1, device="cpu", **kw)


def test_layer_refuses_what_does_not_go_together():
    with pytest.raises(ValueError, match="not both"):
        _layer(ckpt8=True, recompute=True)
    for kw in (dict(recompute=True), dict(ckpt8=True), dict(balance=(1, 1))):
        with pytest.raises(ValueError, match="no backward"):
            _layer(weights4=True, **kw)
    with pytest.raises(ValueError, match="not MXFP8"):
        m.MoEExpertLayer(4, 128, 128, 2, 1, device="cpu", weights4=True, gemm=m.MOE_MXFP8)


def test_layer_refuses_weights_of_the_other_kind():
    x, w = torch.zeros(4, 64, dtype=torch.bfloat16), torch.zeros(2, 64, 64, dtype=torch.bfloat16)
    pair = (torch.zeros(2, 64, 32, dtype=torch.uint8), torch.zeros(2, 64, 2, dtype=torch.uint8))
    for layer, ws in ((_layer(weights4=True), (pair, w, pair)), (_layer(), (w, w, pair))):
        with pytest.raises(ValueError, match="pair"):
            layer.forward(x, *ws, Wr=w[0, :2])
        assert layer.steps == 0
        with pytest.raises(ValueError, match="pair"):
            m.MoEBlock(layer).forward(x, *ws, w_pre=x[0], Wr=w[0, :2])


def test_a_serving_layer_has_no_backward():
    layer = _layer(weights4=True)
    x, w = torch.zeros(4, 64, dtype=torch.bfloat16), torch.zeros(2, 64, 64, dtype=torch.bfloat16)
    for call in (lambda: layer.backward(x), lambda: m.MoEBlock(layer).backward(x),
                 lambda: m.layer.MoEExpertFunction.apply(x, w[0, :2], w, w, w, layer)):
        with pytest.raises(RuntimeError, match="no backward"):
            call()


def test_a_checkpointing_layer_refuses_its_own_outputs_as_input():
    w = torch.zeros(2, 64, 64, dtype=torch.bfloat16)
    layer = _layer(ckpt8=True)
    for x in (layer.y, layer.dx):
        with pytest.raises(ValueError, match="again in the backward"):
            layer.forward(x, w, w, w, Wr=w[0, :2])


def test_held_bytes():
    """The 8-bit layer holds d + 2 f bytes a routed row, the recomputing one 4 d, the plain one 4 d + 6 f,
    with a scale byte per 32 on top."""
    T, d, f, E, k = 64, 256, 128, 4, 2
    mk = lambda **kw: m.MoEExpertLayer(T, d, f, E, k, device="cpu", **kw).activation_bytes()  # noqa: E731
    R = T * k
    assert mk() == R * (2 * d + 3 * f) * 2
    assert mk(recompute=True) == R * 2 * d * 2
    assert mk(ckpt8=True) == R * (2 * f + d) * 33 // 32
    assert mk(weights4=True) == 0
