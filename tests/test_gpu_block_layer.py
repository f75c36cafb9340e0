"""The expert layer between its norms and with its router losses (MoEBlock, balance=...), whole
steps on the GPU against the fp64 oracle composed of the same parts, at the layer's tolerances."""
import numpy as np
import pytest
import torch

import workloads
from gpu_common import TOL, host, make_layer, mx_scope_bits, normwise_err, say, to_dev
from oracle import block_ref, moe_ref

pytestmark = pytest.mark.gpu

W = workloads.WORKLOADS
EPS = 1e-6


def _layer(w, balance, **kw):
    import mixture_experts_layer_logits_amd as m
    act = m.MOE_F32 if w.dtype == "f32" else m.MOE_BF16
    gemm = {"f32": m.MOE_F32, "bf16": m.MOE_BF16, "mxfp8": m.MOE_MXFP8}[w.gemm]
    return m.MoEExpertLayer(w.T, w.d, w.f, w.E, w.k, act=act, gemm=gemm, shared_f=w.shared_f,
                            mx_scope=mx_scope_bits(w), balance=balance, **kw)


def _extra(w, seed, post, gated, nxt):
    """The block's own inputs, host side."""
    g = torch.Generator().manual_seed(seed)
    dt = w.torch_dtype()
    rnd = lambda *n: torch.randn(*n, generator=g)  # noqa: E731
    e = dict(w_pre=(1 + 0.1 * rnd(w.d)).to(dt))
    e["w_post"] = (1 + 0.1 * rnd(w.d)).to(dt) if post else None
    e["gate"] = torch.sigmoid(rnd(w.T)) if gated else None
    if gated:
        e["gate"][::7] = 0.0
    e["w_next"] = (1 + 0.1 * rnd(w.d)).to(dt) if nxt else None
    e["dxn_next"] = rnd(w.T, w.d).to(dt) if nxt else None
    return e


def _run(block, w, inp, e, mask=None, xn=None):
    d, x = to_dev(inp), {k: None if t is None else t.cuda() for k, t in e.items()}
    kw = dict(topk_idx=d["topk_idx"], gates=d["gates"]) if w.routing == "given_uniform" else dict(
        Wr=d["Wr"], bias=d["router_bias"])
    v = block.forward(d["x"], d["W1"], d["W3"], d["W2"], w_pre=x["w_pre"] if xn is None else None, xn=xn,
                      w_post=x["w_post"], gate=x["gate"], w_next=x["w_next"], shared=d.get("shared"),
                      mask=None if mask is None else mask.cuda(), **kw)
    back = block.backward(d["dy"], x["dxn_next"])
    torch.cuda.synchronize()
    return v, back


def _oracle(w, inp, e, scale, logits, balance=None, mask=None, k_dy=1.0):
    """Block forward and backward in fp64 (routing on the GPU's scores)."""
    learned = w.routing != "given_uniform"
    pre = block_ref.norm_fwd(inp["x"], w_pre=e["w_pre"], eps=EPS)
    xn = pre["xn"]
    sh = inp.get("shared")
    fw = moe_ref.layer_forward(xn, inp["W1"], inp["W3"], inp["W2"], w.k, Wr=inp["Wr"], bias=inp["router_bias"],
                               select_logits=logits, shared=sh) if learned else moe_ref.layer_forward(
        xn, inp["W1"], inp["W3"], inp["W2"], w.k, topk_idx=inp["topk_idx"].numpy(), gates=inp["gates"], shared=sh)
    post = block_ref.norm_fwd(inp["x"], y=fw["y"], gate=e["gate"], w_post=e["w_post"], w_pre=e["w_next"],
                              res_scale=scale, eps=EPS)
    bw = block_ref.norm_bwd(dv=inp["dy"], dxn=e["dxn_next"], v=post["v"], y=fw["y"], gate=e["gate"],
                            w_post=e["w_post"], w_pre=e["w_next"], rstd_post=post.get("rstd_post"),
                            rstd_pre=post.get("rstd_pre"), res_scale=scale)
    lb = moe_ref.layer_backward(fw, bw["dy"], xn, inp["W1"], inp["W3"], inp["W2"], Wr=inp["Wr"], learned=learned,
                                shared=sh)
    dxn, dWr = lb["dx"], lb.get("dWr")
    out = dict(fw=fw, xn=xn, v=post["v"], xn_next=post.get("xn"), dgate=bw.get("dgate"), dw_post=bw.get("dw_post"),
               dw_next=bw.get("dw_pre"), dv=bw["dx"], lb=lb)
    if balance is not None:
        bf = block_ref.balance_fwd(fw["logits"], fw["topk_idx"], mask)
        dl = block_ref.balance_bwd(fw["logits"], bf["lse"], bf["counts"], balance)["dlogits"]
        ax, aw = moe_ref.router_bwd(xn, inp["Wr"], dl)
        dxn, dWr = dxn + ax, dWr + aw
        out.update(bal=bf, dlogits=lb["dlogits"] + dl)
    nb = block_ref.norm_bwd(dv=bw["dx"], dxn=dxn, v=inp["x"], w_pre=e["w_pre"], rstd_pre=pre["rstd_pre"])
    out.update(dxn=dxn, dWr=dWr, dh=nb["dx"], dw_pre=nb["dw_pre"])
    return out


CASES = [
    ("tiny_fp32", {}, dict(post=True, gated=True, nxt=True)),
    ("e128_k4_t8192", dict(T=512, d=256, f=192), dict(post=True, gated=False, nxt=True)),
    ("e128_k4_t8192", dict(T=130, d=320, f=64, E=33, k=3), dict(post=False, gated=True, nxt=False)),
    ("e128_k4_t8192_shared", dict(T=300, d=256, f=192, shared_f=128), dict(post=True, gated=True, nxt=False)),
    ("e128_k4_t8192", dict(T=1, d=256, f=64, E=8, k=2), dict(post=True, gated=False, nxt=True)),
]


@pytest.mark.parametrize("wname,over,parts", CASES, ids=lambda x: str(x)[:40])
@pytest.mark.parametrize("balance", [None, (0.5, 0.1)])
def test_block_step_against_oracle(wname, over, parts, balance):
    import mixture_experts_layer_logits_amd as m
    w = workloads.scaled(W[wname], **over) if over else W[wname]
    say(f"[gpu] block step {w.name} {over} {parts} balance={balance}")
    inp, e = workloads.make_inputs(w), _extra(w, 3, **parts)
    mask = None if balance is None or w.T < 4 else (torch.arange(w.T) % 5 != 0).to(torch.uint8)
    block = m.MoEBlock(_layer(w, balance), res_scale=0.7, eps=EPS)
    v, dh = _run(block, w, inp, e, mask)
    L = block.layer
    o = _oracle(w, inp, e, 0.7, host(L.logits), balance, mask)
    assert np.array_equal(host(L.slot_row), o["fw"]["slot_row"])
    got = dict(xn=block.xn, v=v, dh=dh, dw_pre=block.dw_pre, dv=block.dv, dWr=L.dWr, dxn=L.dx)
    if parts["post"]:
        got["dw_post"] = block.dw_post
    if parts["gated"]:
        got["dgate"] = block.dgate
    if parts["nxt"]:
        got.update(xn_next=block.xn_next, dw_next=block.dw_next)
    errs = {n: normwise_err(host(t), o[n]) for n, t in got.items()}
    for n in ("dgates", "dx_perm", "dW1", "dW3", "dW2") + (("dW1s", "dW2s") if w.shared_f else ()):
        errs[n] = normwise_err(host(getattr(L, n)), o["lb"][n])
    if balance is not None:
        assert np.array_equal(host(L.bal_counts), o["bal"]["counts"])
        errs.update(loss=normwise_err(host(L.loss), o["bal"]["loss"]), dlogits=normwise_err(host(L.dlogits), o["dlogits"]))
    print({k: f"{x:.1e}" for k, x in errs.items()})
    assert not {k: x for k, x in errs.items() if x > TOL[w.gemm]}


@pytest.mark.parametrize("wname", ["e32_k4_t16384_d4096_mxfp8", "e32_k4_t16384_d4096_mxfp8_all"])
def test_block_with_mxfp8_experts(wname):
    """The default MXFP8 scope against the unquantised oracle; all six GEMMs (whose dispatch writes
    E4M3 rows, so the combine and the norm are separate calls) against the layer between the same
    norms, called one by one."""
    import mixture_experts_layer_logits_amd as m
    w = workloads.scaled(W[wname], T=300, d=256, f=256, E=8, k=4)
    say(f"[gpu] block step {w.name}")
    inp, e = workloads.make_inputs(w), _extra(w, 4, True, True, True)
    block = m.MoEBlock(_layer(w, None), res_scale=0.7, eps=EPS)
    v, dh = _run(block, w, inp, e)
    L = block.layer
    if not L.mx_dispatch:
        o = _oracle(w, inp, e, 0.7, None)
        errs = {n: normwise_err(host(t), o[n]) for n, t in
                dict(xn=block.xn, v=v, dh=dh, dw_pre=block.dw_pre, dw_post=block.dw_post, dgate=block.dgate,
                     xn_next=block.xn_next, dw_next=block.dw_next).items()}
        print(errs)
        assert not {k: x for k, x in errs.items() if x > TOL["mxfp8"]}
        return
    d, x = to_dev(inp), {k: t.cuda() for k, t in e.items()}
    P = make_layer(w)
    y = P.forward(block.xn, d["W1"], d["W3"], d["W2"], topk_idx=d["topk_idx"], gates=d["gates"])
    assert torch.equal(y, L.y)
    r1, r2 = torch.empty(w.T, device="cuda"), torch.empty(w.T, device="cuda")
    v2, xn2 = torch.empty_like(v), torch.empty_like(v)
    m.moe_block_norm_fwd(P.shape, d["x"], y, x["gate"], x["w_post"], x["w_next"], 0.7, EPS, v2, xn2, r1, r2)
    assert torch.equal(v2, v) and torch.equal(xn2, block.xn_next)
    P.backward(block.dy)
    assert torch.equal(P.dx, L.dx) and torch.equal(P.dW1, L.dW1) and torch.equal(P.dgates, L.dgates)


def test_a_stack_of_blocks_passes_its_norm_on():
    """Two blocks, the second on the first one's xn_next: the same values and gradients as two
    blocks that each norm their own input, up to the rounding of the stream between them."""
    import mixture_experts_layer_logits_amd as m
    w = workloads.scaled(W["e128_k4_t8192"], T=200, d=256, f=128, E=16, k=4)
    say(f"[gpu] two blocks {w}")
    ia, ib = workloads.make_inputs(w), workloads.make_inputs(workloads.scaled(w, seed=w.seed + 1))
    ea, eb = _extra(w, 5, True, True, False), _extra(w, 6, True, False, False)
    da, db = to_dev(ia), to_dev(ib)
    xa, xb = ({k: None if t is None else t.cuda() for k, t in e.items()} for e in (ea, eb))
    a, b = (m.MoEBlock(_layer(w, (0.1, 0.01)), 0.5, EPS) for _ in range(2))
    h = a.forward(da["x"], da["W1"], da["W3"], da["W2"], w_pre=xa["w_pre"], w_post=xa["w_post"], gate=xa["gate"],
                  w_next=xb["w_pre"], Wr=da["Wr"])
    v = b.forward(h, db["W1"], db["W3"], db["W2"], xn=a.xn_next, w_post=xb["w_post"], Wr=db["Wr"])
    dh, dxn = b.backward(db["dy"])
    dx = a.backward(dh, dxn)
    fused = [t.clone() for t in (v, dx, a.dw_next, a.dw_pre, b.layer.dWr)]
    idx = b.layer.topk_idx.clone()
    h = a.forward(da["x"], da["W1"], da["W3"], da["W2"], w_pre=xa["w_pre"], w_post=xa["w_post"], gate=xa["gate"],
                  Wr=da["Wr"])
    v = b.forward(h, db["W1"], db["W3"], db["W2"], w_pre=xb["w_pre"], w_post=xb["w_post"], Wr=db["Wr"])
    dx = a.backward(b.backward(db["dy"]))
    torch.cuda.synchronize()
    moved = int((idx.sort(dim=1).values != b.layer.topk_idx.sort(dim=1).values).any(dim=1).sum())
    assert moved <= 2, moved  # xn differs by a rounding: a near tie may route otherwise
    for n, x, y in zip(("v", "dx", "dw", "dw_pre", "dWr"), fused, (v, dx, b.dw_pre, a.dw_pre, b.layer.dWr)):
        assert normwise_err(host(x), host(y)) <= TOL["bf16"] or moved, n


def test_block_of_no_tokens():
    """An empty batch: zero losses, counts and weight gradients."""
    import mixture_experts_layer_logits_amd as m
    w = workloads.scaled(W["e8_k4_t8192"], T=0, d=128, f=64)
    say("[gpu] block of no tokens")
    inp, e = workloads.make_inputs(w), _extra(w, 2, True, True, True)
    block = m.MoEBlock(_layer(w, (0.5, 0.1)), 0.5, EPS)
    L = block.layer
    for t in (block.dw_pre, block.dw_post, block.dw_next, L.dWr, L.dW1, L.loss):
        t.fill_(7)
    v, dh = _run(block, w, inp, e)
    assert v.shape == dh.shape == (0, 128)
    for t in (block.dw_pre, block.dw_post, block.dw_next, L.dWr, L.dW1, L.loss, L.bal_counts):
        assert not host(t).any()


def test_block_refuses_its_own_output_as_input():
    import mixture_experts_layer_logits_amd as m
    w = workloads.scaled(W["e8_k4_t8192"], T=32, d=128, f=64)
    inp, e = workloads.make_inputs(w), _extra(w, 2, True, False, True)
    block = m.MoEBlock(_layer(w, None), 0.5, EPS)
    v, _ = _run(block, w, inp, e)
    d, x = to_dev(inp), {k: None if t is None else t.cuda() for k, t in e.items()}
    for kw in (dict(h=v, w_pre=x["w_pre"]), dict(h=d["x"], xn=block.xn_next), dict(h=d["x"]),
               dict(h=d["x"], xn=d["x"], w_pre=x["w_pre"])):
        with pytest.raises(ValueError):
            block.forward(kw.pop("h"), d["W1"], d["W3"], d["W2"], Wr=d["Wr"], **kw)


def test_block_step_graph_replays_match_eager():
    import mixture_experts_layer_logits_amd as m
    w = workloads.scaled(W["e128_k4_t8192_shared"], T=256, d=256, f=128, shared_f=64)
    say(f"[gpu] block step in a graph {w}")
    inp, e = workloads.make_inputs(w), _extra(w, 8, True, True, True)
    block = m.MoEBlock(_layer(w, (0.5, 0.1)), 0.7, EPS)
    d, x = to_dev(inp), {k: t.cuda() for k, t in e.items()}
    mask = (torch.arange(w.T, device="cuda") % 3 != 0).to(torch.uint8)

    def step():
        block.forward(d["x"], d["W1"], d["W3"], d["W2"], w_pre=x["w_pre"], w_post=x["w_post"], gate=x["gate"],
                      w_next=x["w_next"], Wr=d["Wr"], shared=d["shared"], mask=mask)
        block.backward(d["dy"], x["dxn_next"])

    outs = lambda: [block.v, block.xn_next, block.dh, block.dw_pre, block.dw_post, block.dw_next, block.dgate,  # noqa: E731
                    block.layer.dWr, block.layer.dW1, block.layer.loss, block.layer.dlogits, block.layer.bal_counts]
    step()
    want = [t.clone() for t in outs()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    torch.cuda.synchronize()
    for rep in range(3):
        for t in outs():
            t.fill_(7)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs(), want)), rep


def test_block_autograd_function():
    import mixture_experts_layer_logits_amd as m
    from mixture_experts_layer_logits_amd.layer import MoEBlockFunction
    w = workloads.scaled(W["e8_k4_t8192"], T=96, d=128, f=64)
    say(f"[gpu] block autograd {w}")
    inp, e = workloads.make_inputs(w), _extra(w, 9, True, True, False)
    d, x = to_dev(inp), {k: None if t is None else t.cuda() for k, t in e.items()}
    block = m.MoEBlock(_layer(w, (0.0, 0.0)), 0.7, EPS)
    leaves = [t.clone().requires_grad_() for t in (d["x"], x["w_pre"], x["w_post"], x["gate"], d["Wr"], d["W1"],
                                                   d["W3"], d["W2"])]
    v, loss = MoEBlockFunction.apply(*leaves, block)
    # the router losses weigh into the objective like any other value
    ((v.float() * d["dy"].float()).sum() + 0.5 * loss[0] + 0.1 * loss[1]).backward()
    o = _oracle(w, inp, e, 0.7, host(block.layer.logits), (0.5, 0.1))
    want = [o["dh"], o["dw_pre"], o["dw_post"], o["dgate"], o["dWr"], o["lb"]["dW1"], o["lb"]["dW3"], o["lb"]["dW2"]]
    for t, r in zip(leaves, want):
        assert t.grad.dtype is t.dtype and normwise_err(host(t.grad), r) <= TOL["bf16"]
    v, _ = MoEBlockFunction.apply(*leaves, block)
    MoEBlockFunction.apply(*leaves, block)
    with pytest.raises(RuntimeError, match="another forward"):
        v.sum().backward()
    plain = m.MoEBlock(_layer(w, None))
    with pytest.raises(ValueError, match="router losses"):
        MoEBlockFunction.apply(*leaves, plain)


def test_layer_router_losses_without_a_block():
    """balance= on the layer alone: the plain backward uses the layer's weights, and refusals."""
    w = workloads.scaled(W["e128_k4_t8192"], T=200, d=128, f=64)
    say(f"[gpu] layer with router losses {w}")
    inp = workloads.make_inputs(w)
    d = to_dev(inp)
    L, P = _layer(w, (0.5, 0.1)), _layer(w, None)
    for layer in (L, P):
        layer.forward(d["x"], d["W1"], d["W3"], d["W2"], Wr=d["Wr"])
        layer.backward(d["dy"])
    fw = moe_ref.layer_forward(inp["x"], inp["W1"], inp["W3"], inp["W2"], w.k, Wr=inp["Wr"], select_logits=host(L.logits))
    bf = block_ref.balance_fwd(host(L.logits), fw["topk_idx"])
    dl = block_ref.balance_bwd(host(L.logits), bf["lse"], bf["counts"], [0.5, 0.1])["dlogits"]
    assert normwise_err(host(L.dlogits) - host(P.dlogits), dl) <= 1e-3
    ax, aw = moe_ref.router_bwd(inp["x"], inp["Wr"], dl)
    assert normwise_err(host(L.dWr), host(P.dWr) + aw) <= TOL["bf16"]
    assert normwise_err(host(L.dx), host(P.dx) + ax) <= TOL["bf16"]
    assert torch.equal(L.y, P.y) and torch.equal(L.dW1, P.dW1)
    L.backward(d["dy"], torch.zeros(2, device="cuda"))  # other weights than the layer's
    assert normwise_err(host(L.dlogits), host(P.dlogits)) <= 1e-6  # the gates' gradient alone, in another order
    steps = L.steps
    with pytest.raises(ValueError, match="learned routing"):
        L.forward(d["x"], d["W1"], d["W3"], d["W2"], topk_idx=L.topk_idx, gates=L.gates)
    with pytest.raises(ValueError, match="router losses"):
        P.forward(d["x"], d["W1"], d["W3"], d["W2"], Wr=d["Wr"], mask=torch.ones(w.T, dtype=torch.uint8, device="cuda"))
    assert L.steps == steps
