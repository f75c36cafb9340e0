"""Paths through the layer with 8-bit checkpoints and with 4-bit weights that a program takes beside the whole
step: a block next to the plain one, autograd through a block, empty batches, other streams."""
import numpy as np
import pytest
import torch

import workloads
from gpu_common import say, to_dev
from test_gpu_few_bits_layer import CASES, GRADS, _forward, _layer, _values

pytestmark = pytest.mark.gpu

STEP = 2.0 ** -23


def _m():
    import mixture_experts_layer_logits_amd as m
    return m


def _f64(t):
    return t.detach().cpu().double().numpy()


@pytest.mark.parametrize("name", ["bf16", "f32"])
def test_block_next_to_the_plain_block(name):
    """Over a checkpointing layer the block stores y between the combine and the norm, so v carries y's
    rounding too.  With t = res_scale gate (y rstd) w_post the branch, y's half step changes t by at most two of
    them (of y itself and of rstd), and the fp32 sums of the combine and the norm by (d / 64 + k + 32) steps of t and of
    the combine's sum of absolute values; each v rounds once by half a step of its own."""
    m = _m()
    w = CASES[name]
    say(f"[gpu] ckpt8 block next to the plain one {name}")
    d = to_dev(workloads.make_inputs(w))
    g = torch.Generator().manual_seed(5)
    wt = lambda: (1 + 0.1 * torch.randn(w.d, generator=g)).to(d["x"].dtype).cuda()  # noqa: E731
    w_pre, w_post = wt(), wt()
    gate = torch.sigmoid(torch.randn(w.T, generator=g)).cuda()
    A, B = m.MoEBlock(_layer(w), res_scale=0.5), m.MoEBlock(_layer(w, ckpt8=True), res_scale=0.5)
    va, vb = (blk.forward(d["x"], d["W1"], d["W3"], d["W2"], w_pre=w_pre, w_post=w_post, gate=gate, Wr=d["Wr"],
                          bias=d["router_bias"]) for blk in (A, B))
    L = A.layer
    assert torch.equal(L.slot_row, B.layer.slot_row) and torch.equal(A.xn, B.xn)
    rows = _f64(L.y_perm)[_f64(L.slot_row).astype(int)] * _f64(L.gates)[..., None]
    y, mag = rows.sum(1), np.abs(rows).sum(1)
    scale = 0.5 * _f64(gate)[:, None] / np.sqrt((y * y).mean(1, keepdims=True) + 1e-6) * _f64(w_post)
    want = _f64(d["x"]) + scale * y
    half = torch.finfo(d["x"].dtype).eps / 2
    few = (w.d / 64 + w.k + 32) * STEP * (np.abs(scale * y) + np.abs(scale) * mag)
    plain = few + half * (np.abs(want) + few)
    assert (np.abs(_f64(va) - want) <= plain).all()
    # two half steps, and what their product and the rounding of v itself add
    stored = few + 2 * (1 + 2 * half) * half * np.abs(scale * y)
    assert (np.abs(_f64(vb) - want) <= stored + half * (np.abs(want) + stored)).all()


def test_checkpointing_block_under_autograd():
    m = _m()
    w = CASES["bf16"]
    d = to_dev(workloads.make_inputs(w))
    mk = lambda: m.MoEBlock(_layer(w, ckpt8=True, balance=(0.01, 0.001)), res_scale=0.5)  # noqa: E731
    one = torch.ones(w.d, dtype=d["x"].dtype, device="cuda")
    gate = torch.linspace(0, 1, w.T, device="cuda")
    leaves = [t.clone().requires_grad_() for t in (d["x"], one, one, gate, d["Wr"], d["W1"], d["W3"], d["W2"])]
    dl = torch.tensor([0.01, 0.001], device="cuda")
    B, C = mk(), mk()
    v, loss = m.layer.MoEBlockFunction.apply(*leaves, B, d["router_bias"])
    torch.autograd.backward([v, loss], [d["dy"], dl])
    v2 = C.forward(d["x"], d["W1"], d["W3"], d["W2"], w_pre=one, w_post=one, gate=gate, Wr=d["Wr"], bias=d["router_bias"])
    dh = C.backward(d["dy"], dloss=dl)
    L = C.layer
    assert torch.equal(v, v2)
    for t, want in zip(leaves, (dh, C.dw_pre, C.dw_post, C.dgate, L.dWr, L.dW1, L.dW3, L.dW2)):
        assert torch.equal(t.grad, want.to(t.dtype))


@pytest.mark.parametrize("name", ["bf16", "bf16_shared", "f32", "mx", "mx_all"])
def test_empty_checkpointing_layer(name):
    w = workloads.scaled(CASES[name], T=0)
    full = to_dev(workloads.make_inputs(CASES[name]))
    cut = lambda n, t: t[:0] if n in ("x", "dy", "topk_idx", "gates") and t is not None else t  # noqa: E731
    d = {n: cut(n, t) for n, t in full.items()}
    L = _layer(w, ckpt8=True)
    y = _forward(L, w, d)
    dx = L.backward(d["dy"])
    torch.cuda.synchronize()
    assert y.shape == dx.shape == (0, w.d)
    for t in (L.dW1, L.dW3, L.dW2):
        assert not t.any()


def test_empty_serving_layer():
    m = _m()
    L = m.MoEExpertLayer(0, 128, 64, 4, 2, weights4=True, shared_f=64)
    e = lambda *n: torch.randn(*n, device="cuda").to(torch.bfloat16)  # noqa: E731
    q, qs = m.quantize_weights(e(4, 64, 128), e(4, 64, 128), e(4, 128, 64)), m.quantize_weights(e(1, 64, 128), e(1, 64, 128),
                                                                                          e(1, 128, 64))
    y = L.forward(e(0, 128), *q, Wr=e(4, 128), shared=qs)
    torch.cuda.synchronize()
    assert y.shape == (0, 128)


def test_two_checkpointing_steps_at_once():
    """Two layers' steps on two streams, whose temporaries come and go, keep each other's results."""
    w = CASES["bf16"]
    d = to_dev(workloads.make_inputs(w))
    ins = [d, {**d, "x": -0.5 * d["x"], "dy": 2 * d["dy"]}]
    layers = [_layer(w, ckpt8=True) for _ in ins]
    want = []
    for L, i in zip(layers, ins):
        _forward(L, w, i)
        L.backward(i["dy"])
        want.append({n: getattr(L, n).clone() for n in GRADS + ("y", "dWr")})
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in layers]
    for _ in range(3):
        for L, i, st in zip(layers, ins, streams):
            with torch.cuda.stream(st):
                _forward(L, w, i)
        for L, i, st in zip(layers, ins, streams):
            with torch.cuda.stream(st):
                L.backward(i["dy"])
    torch.cuda.synchronize()
    for L, wt in zip(layers, want):
        for n, t in wt.items():
            assert torch.equal(t, getattr(L, n)), n


def test_a_second_backward_of_one_forward():
    w = CASES["bf16_shared"]
    d = to_dev(workloads.make_inputs(w))
    L = _layer(w, ckpt8=True)
    _forward(L, w, d)
    L.backward(-d["dy"])
    L.backward(d["dy"])
    C = _layer(w, ckpt8=True)
    _forward(C, w, d)
    C.backward(d["dy"])
    for n in GRADS + ("dW1s", "dW3s", "dW2s"):
        assert torch.equal(getattr(L, n), getattr(C, n)), n


def test_weights_of_any_rank_quantise_alike():
    m = _m()
    w = torch.randn(3, 4, 64, device="cuda")
    (q, s), (q2, s2), (q1, s1) = m.quantize_weights(w, w.view(12, 64), w[2, 3])
    assert q.shape == (3, 4, 32) and s.shape == (3, 4, 2) and q1.shape == (32,) and s1.shape == (2,)
    assert torch.equal(q.view(12, 32), q2) and torch.equal(s.view(12, 2), s2)
    assert torch.equal(q[2, 3], q1) and torch.equal(s[2, 3], s1)
    with pytest.raises(ValueError, match="contiguous"):
        m.quantize_weights(w.transpose(0, 1))
    for bad in (w[..., :48].contiguous(), w[..., :33].contiguous()):
        with pytest.raises((ValueError, RuntimeError)):
            m.quantize_weights(bad)
    empty = m.quantize_weights(w[:0])
    assert empty[0][0].shape == (0, 4, 32)


@pytest.mark.parametrize("shared_f", [0, 128])
@pytest.mark.parametrize("scope", [("GEMM1",), ("DGRAD2",), ("GEMM1", "DGRAD2"), ("GEMM2", "DGRAD1", "WGRAD1"),
                                   ("GEMM1", "DGRAD2", "WGRAD1", "WGRAD2"), ("GEMM1", "GEMM2", "WGRAD2")], ids="_".join)
def test_any_mxfp8_scope(scope, shared_f):
    """Whichever GEMMs run MXFP8: the forward is the plain layer's and the backward the plain one on the values
    that the checkpoint stands for, bit for bit."""
    m = _m()
    say(f"[gpu] ckpt8 scope {scope} shared={shared_f}")
    T, d, f, E, k = 130, 256, 128, 5, 2
    bits = sum(getattr(m, "MOE_MX_" + n) for n in scope)
    g = torch.Generator().manual_seed(bits)
    r = lambda s, *n: (s * torch.randn(*n, generator=g)).to(torch.bfloat16).cuda()  # noqa: E731
    x, dy, Wr, W = r(1, T, d), r(1, T, d), r(.06, E, d), (r(.06, E, f, d), r(.06, E, f, d), r(.09, E, d, f))
    sh = (r(.06, 1, f, d), r(.06, 1, f, d), r(.09, 1, d, f)) if shared_f else None
    kw = dict(gemm=m.MOE_MXFP8, mx_scope=bits, shared_f=shared_f)
    A, B = m.MoEExpertLayer(T, d, f, E, k, **kw), m.MoEExpertLayer(T, d, f, E, k, ckpt8=True, **kw)
    assert torch.equal(A.forward(x, *W, Wr=Wr, shared=sh), B.forward(x, *W, Wr=Wr, shared=sh))
    A.ab, A.h = _values(m, B.ab_bits, A.dtype, h=True)
    A.y_perm = _values(m, B.y_bits, A.dtype)
    if sh:
        A.ab_s, A.h_s = _values(m, B.ab_bits_s, A.dtype, h=True)
    A.backward(dy)
    B.backward(dy)
    for n in GRADS + ("dlogits", "dWr") + (("dW1s", "dW3s", "dW2s") if sh else ()):
        assert torch.equal(getattr(A, n), getattr(B, n)), n
