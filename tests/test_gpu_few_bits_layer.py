"""The layer and the block with 8-bit checkpoints, and serving with 4-bit weights, as whole steps.

The forward with ckpt8 is the plain layer's, bit for bit, and its backward is the plain backward on the
values that the checkpoint stands for, bit for bit; both are compared with the fp64 oracle given those
values, at the layer's tolerances.  Serving is compared with the oracle on the values of the weights."""
import numpy as np
import pytest
import torch

import workloads
from gpu_common import TOL, host, make_layer, mx_scope_bits, normwise_err, oracle_for, say, to_dev
from oracle import block_ref, few_bits_ref, moe_ref

pytestmark = pytest.mark.gpu

W = workloads.WORKLOADS
GRADS = ("dx", "dgates", "dW1", "dW3", "dW2", "dab", "dx_perm")

CASES = {
    "bf16": workloads.scaled(W["e128_k4_t8192"], T=300, d=256, f=192, E=16, k=4),
    "bf16_long": workloads.scaled(W["e8_k4_t8192"], T=1500, d=128, f=64, E=2, k=2),
    "bf16_shared": workloads.scaled(W["e128_k4_t8192_shared"], T=200, d=192, f=128, E=8, k=3, shared_f=128),
    "bf16_given": workloads.scaled(W["e128_k4_t16384_random"], T=257, d=128, f=64, E=40, k=4),
    "f32": W["tiny_fp32"],
    "mx": workloads.scaled(W["e32_k4_t16384_d4096_mxfp8"], T=200, d=256, f=256, E=6, k=2),
    "mx_all": workloads.scaled(W["e32_k4_t16384_d4096_mxfp8_all"], T=200, d=256, f=256, E=6, k=2),
    "one_token": workloads.scaled(W["e128_k4_t8192"], T=1, d=64, f=64, E=8, k=2),
}


def _layer(w, **kw):
    import mixture_experts_layer_logits_amd as m
    act = m.MOE_F32 if w.dtype == "f32" else m.MOE_BF16
    gemm = {"f32": m.MOE_F32, "bf16": m.MOE_BF16, "mxfp8": m.MOE_MXFP8}[w.gemm]
    return m.MoEExpertLayer(w.T, w.d, w.f, w.E, w.k, act=act, gemm=gemm, shared_f=w.shared_f,
                            mx_scope=mx_scope_bits(w), **kw)


def _forward(layer, w, d):
    kw = dict(topk_idx=d["topk_idx"], gates=d["gates"]) if w.routing == "given_uniform" else dict(
        Wr=d["Wr"], bias=d["router_bias"])
    return layer.forward(d["x"], d["W1"], d["W3"], d["W2"], shared=d.get("shared"), **kw)


def _values(m, bits, dtype, h=False):
    """What a layer's (codes, scales) stand for, and for [a | b] its h."""
    rows, cols = bits[0].shape
    v = torch.empty(rows, cols, dtype=dtype, device="cuda")
    hv = torch.empty(rows, cols // 2, dtype=dtype, device="cuda") if h else None
    m.moe_ckpt8_unpack(rows, cols, *bits, v, hv)
    return (v, hv) if h else v


@pytest.mark.parametrize("name", CASES)
def test_checkpointing_layer(name):
    import mixture_experts_layer_logits_amd as m
    w = CASES[name]
    say(f"[gpu] ckpt8 layer {name}")
    inp = workloads.make_inputs(w)
    d = to_dev(inp)
    A, B = _layer(w, mx_fused_quant=False), _layer(w, ckpt8=True)
    ya, yb = _forward(A, w, d), _forward(B, w, d)
    assert torch.equal(ya, yb)
    assert B.x_perm is B.ab is B.h is B.y_perm is None
    assert B.activation_bytes() < A.activation_bytes()
    # the plain layer's backward on what the checkpoint stands for
    ab, h = _values(m, B.ab_bits, A.dtype, h=True)
    step = A.ab.double().abs().reshape(-1, 32).amax(1) / 127
    assert ((ab.double() - A.ab.double()).abs().reshape(-1, 32) <= (1.01 * step + 2.0 ** -100)[:, None] +
            2.0 ** -8 * A.ab.double().abs().reshape(-1, 32)).all()
    A.ab, A.h = ab, h
    A.y_perm = _values(m, B.y_bits, A.dtype)
    if w.shared_f:
        A.ab_s, A.h_s = _values(m, B.ab_bits_s, A.dtype, h=True)
    A.backward(d["dy"])
    B.backward(d["dy"])
    names = GRADS + (("dlogits", "dWr") if A.learned else ()) + (("dW1s", "dW3s", "dW2s") if w.shared_f else ())
    for n in names:
        assert torch.equal(getattr(A, n), getattr(B, n)), n
    if w.gemm == "mxfp8":
        return
    # and the oracle's
    fw, _ = oracle_for(w, inp, gpu_logits=host(B.logits))
    f64 = lambda t: t.cpu().double().numpy()  # noqa: E731
    fw["a"], fw["b"], fw["y_perm"] = f64(ab[:, :w.f]), f64(ab[:, w.f:]), f64(A.y_perm)
    if w.shared_f:
        fw["shared"]["a"], fw["shared"]["b"] = f64(A.ab_s[:, :w.shared_f]), f64(A.ab_s[:, w.shared_f:])
    learned = w.routing != "given_uniform"
    bw = moe_ref.layer_backward(fw, inp["dy"], inp["x"], inp["W1"], inp["W3"], inp["W2"], Wr=inp["Wr"],
                                learned=learned, shared=inp.get("shared"))
    for n in ("dx", "dgates", "dW1", "dW3", "dW2") + (("dWr",) if learned else ()) + (
            ("dW1s", "dW3s", "dW2s") if w.shared_f else ()):
        assert normwise_err(host(getattr(B, n)), bw[n]) <= TOL[w.gemm], n


def test_a_second_forward_replaces_the_checkpoint():
    w = CASES["bf16"]
    inp = workloads.make_inputs(w)
    d = to_dev(inp)
    B, C = _layer(w, ckpt8=True), _layer(w, ckpt8=True)
    _forward(B, w, {**d, "x": -d["x"]})
    B.backward(d["dy"])
    for L in (B, C):
        _forward(L, w, d)
        L.backward(d["dy"])
    for n in GRADS:
        assert torch.equal(getattr(B, n), getattr(C, n)), n


def test_checkpointing_layer_under_autograd():
    import mixture_experts_layer_logits_amd as m
    w = CASES["bf16"]
    d = to_dev(workloads.make_inputs(w))
    L, C = _layer(w, ckpt8=True), _layer(w, ckpt8=True)
    leaves = [d[n].clone().requires_grad_() for n in ("x", "Wr", "W1", "W3", "W2")]
    y = m.layer.MoEExpertFunction.apply(*leaves, L, d["router_bias"])
    y.backward(d["dy"])
    _forward(C, w, d)
    C.backward(d["dy"])
    for t, n in zip(leaves, ("dx", "dWr", "dW1", "dW3", "dW2")):
        assert torch.equal(t.grad, getattr(C, n).to(t.dtype)), n
    y = m.layer.MoEExpertFunction.apply(*leaves, L, d["router_bias"])
    with torch.no_grad():
        leaves[0].add_(1)  # x is read again in the backward
    with pytest.raises(RuntimeError, match="modified by an inplace"):
        y.backward(d["dy"])


@pytest.mark.parametrize("name", ["bf16", "bf16_shared", "f32", "mx_all"])
def test_checkpointing_block(name):
    """A block over a checkpointing layer is the layer's calls between the norms'."""
    import mixture_experts_layer_logits_amd as m
    w = CASES[name]
    say(f"[gpu] ckpt8 block {name}")
    d = to_dev(workloads.make_inputs(w))
    g = torch.Generator().manual_seed(3)
    wt = lambda: (1 + 0.1 * torch.randn(w.d, generator=g)).to(d["x"].dtype).cuda()  # noqa: E731
    w_pre, w_post, w_next = wt(), wt(), wt()
    gate = torch.sigmoid(torch.randn(w.T, generator=g)).cuda()
    gate[::5] = 0
    dxn = torch.randn(w.T, w.d, generator=g).to(d["x"].dtype).cuda()
    kw = dict(topk_idx=d["topk_idx"], gates=d["gates"]) if w.routing == "given_uniform" else dict(
        Wr=d["Wr"], bias=d["router_bias"])
    B = m.MoEBlock(_layer(w, ckpt8=True), res_scale=0.5)
    v = B.forward(d["x"], d["W1"], d["W3"], d["W2"], w_pre=w_pre, w_post=w_post, gate=gate, w_next=w_next,
                  shared=d.get("shared"), **kw)
    dh = B.backward(d["dy"], dxn)
    L = _layer(w, ckpt8=True)
    e = lambda *n, dtype=L.dtype: torch.empty(*n, dtype=dtype, device="cuda")  # noqa: E731
    T, D, f32 = w.T, w.d, torch.float32
    xn, rp = e(T, D), e(T, dtype=f32)
    m.moe_block_norm_fwd(L.shape, d["x"], None, None, None, w_pre, 1.0, 1e-6, None, xn, None, rp)
    y = _forward(L, w, {**d, "x": xn})
    v2, xn2, rq, rn = e(T, D), e(T, D), e(T, dtype=f32), e(T, dtype=f32)
    m.moe_block_norm_fwd(L.shape, d["x"], y, gate, w_post, w_next, 0.5, 1e-6, v2, xn2, rq, rn)
    assert torch.equal(v, v2) and torch.equal(B.xn_next, xn2)
    dv, dy, dg, dwq, dwn = e(T, D), e(T, D), e(T, dtype=f32), e(D, dtype=f32), e(D, dtype=f32)
    m.moe_block_norm_bwd(L.shape, d["dy"], dxn, v2, y, gate, w_post, w_next, rq, rn, 0.5, dv, dy, dg, dwq, dwn, L.ws)
    dx = L.backward(dy)
    dh2, dwp = e(T, D), e(D, dtype=f32)
    m.moe_block_norm_bwd(L.shape, dv, dx, d["x"], None, None, None, w_pre, None, rp, 1.0, dh2, None, None, None, dwp,
                         L.ws)
    for a, b in ((dh, dh2), (B.dgate, dg), (B.dw_post, dwq), (B.dw_next, dwn), (B.dw_pre, dwp),
                 (B.layer.dW1, L.dW1), (B.layer.dW2, L.dW2)):
        assert torch.equal(a, b)


def test_checkpointing_step_replays_in_a_graph():
    w = CASES["bf16"]
    d = to_dev(workloads.make_inputs(w))
    L = _layer(w, ckpt8=True)

    def step():
        _forward(L, w, d)
        L.backward(d["dy"])

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(3):
        d["x"].mul_(-1)
        graph.replay()
        torch.cuda.synchronize()
        got = {n: getattr(L, n).clone() for n in GRADS + ("y", "dWr")}
        step()
        torch.cuda.synchronize()
        for n, t in got.items():
            assert torch.equal(t, getattr(L, n)), (i, n)


# ------------------------------------------------------------------ serving
SERVE = {
    "one_token": workloads.scaled(W["e128_k4_t8192"], T=1, d=256, f=128, E=16, k=4),
    "batch": workloads.scaled(W["e128_k4_t8192"], T=33, d=320, f=192, E=24, k=4),
    "shared": workloads.scaled(W["e128_k4_t8192_shared"], T=9, d=256, f=128, E=8, k=3, shared_f=192),
    "given": workloads.scaled(W["e128_k4_t16384_random"], T=150, d=128, f=64, E=5, k=2),
    "f32": workloads.scaled(W["tiny_fp32"], T=20),
}


@pytest.mark.parametrize("name", SERVE)
def test_serving_block(name):
    import mixture_experts_layer_logits_amd as m
    w = SERVE[name]
    say(f"[gpu] serving {name}")
    inp = workloads.make_inputs(w)
    d = to_dev(inp)
    q = m.quantize_weights(d["W1"], d["W3"], d["W2"])
    sh = d.get("shared")
    qs = m.quantize_weights(*sh) if sh is not None else None
    host_values = lambda pairs: [few_bits_ref.mx4_values(*(t.cpu().numpy() for t in p)) for p in pairs]  # noqa: E731
    v = host_values(q)
    for have, want in zip(v, (inp["W1"], inp["W3"], inp["W2"])):
        code, sc = few_bits_ref.mx4_quantize(want.double().numpy())
        assert np.array_equal(have, few_bits_ref.mx4_values(code, sc))
    L = _layer(w, weights4=True)
    learned = w.routing != "given_uniform"
    kw = dict(Wr=d["Wr"], bias=d["router_bias"]) if learned else dict(topk_idx=d["topk_idx"], gates=d["gates"])
    y = L.forward(d["x"], *q, shared=qs, **kw)
    okw = dict(Wr=inp["Wr"], bias=inp["router_bias"], select_logits=host(L.logits)) if learned else dict(
        topk_idx=inp["topk_idx"].numpy(), gates=inp["gates"])
    fw = moe_ref.layer_forward(inp["x"], *v, w.k, shared=host_values(qs) if qs else None, **okw)
    assert np.array_equal(host(L.slot_row), fw["slot_row"])
    assert normwise_err(host(L.h), fw["h"]) <= TOL[w.gemm]
    assert normwise_err(host(y), fw["y"]) <= TOL[w.gemm]
    # inside a block, with the norm of the next one, from one pass of the same calls
    B = m.MoEBlock(_layer(w, weights4=True), res_scale=0.5)
    wn = torch.linspace(0.5, 1.5, w.d).to(d["x"].dtype)
    out = B.forward(d["x"], *q, w_pre=wn.cuda(), w_next=wn.cuda(), shared=qs, **kw)
    xn = block_ref.norm_fwd(inp["x"], w_pre=wn, eps=1e-6)["xn"]
    okw.update(dict(select_logits=host(B.layer.logits)) if learned else {})
    fw = moe_ref.layer_forward(xn, *v, w.k, shared=host_values(qs) if qs else None, **okw)
    post = block_ref.norm_fwd(inp["x"], y=fw["y"], w_pre=wn, res_scale=0.5, eps=1e-6)
    assert normwise_err(host(out), post["v"]) <= TOL[w.gemm]
    assert normwise_err(host(B.xn_next), post["xn"]) <= TOL[w.gemm]


def test_serving_block_replays_in_a_graph():
    """A decode step is captured once and replayed for every token."""
    import mixture_experts_layer_logits_amd as m
    w = SERVE["batch"]
    d = to_dev(workloads.make_inputs(w))
    q = m.quantize_weights(d["W1"], d["W3"], d["W2"])
    B = m.MoEBlock(_layer(w, weights4=True))
    one = torch.ones(w.d, dtype=d["x"].dtype, device="cuda")
    run = lambda: B.forward(d["x"], *q, w_pre=one, w_next=one, Wr=d["Wr"], bias=d["router_bias"])  # noqa: E731
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for i in range(4):
        d["x"].copy_(torch.roll(d["x"], 1, 0).mul_(-1))
        graph.replay()
        torch.cuda.synchronize()
        v, xn = B.v.clone(), B.xn_next.clone()
        run()
        torch.cuda.synchronize()
        assert torch.equal(B.v, v) and torch.equal(B.xn_next, xn), i
