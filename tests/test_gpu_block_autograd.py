"""The autograd functions of the layer and of the block: what the caller holds afterwards, what the
backward notices, and what is refused.  Values are the whole steps' (test_gpu_block_layer.py,
test_gpu_parity.py); here two runs of the same calls are compared bit for bit."""
import pytest
import torch

import workloads
from gpu_common import make_layer, say, to_dev

pytestmark = pytest.mark.gpu

W = workloads.WORKLOADS
SMALL = {"f32": workloads.scaled(W["tiny_fp32"], T=48, d=64, f=64, E=8, k=2),
         "bf16": workloads.scaled(W["e8_k4_t8192"], T=48, d=64, f=64)}
BLOCK_LEAVES = ("h", "w_pre", "w_post", "gate", "Wr", "W1", "W3", "W2")
LAYER_LEAVES = ("x", "Wr", "W1", "W3", "W2")


class Block:
    """Leaves, gradients to come in, and the block of one case."""
    names = BLOCK_LEAVES

    def __init__(self, act="bf16", seed=3, **kw):
        import mixture_experts_layer_logits_amd as m
        from mixture_experts_layer_logits_amd.layer import MoEBlockFunction
        w = SMALL[act]
        d = to_dev(workloads.make_inputs(w))
        g = torch.Generator().manual_seed(seed)
        dt = w.torch_dtype()
        rnd = lambda *n: torch.randn(*n, generator=g)  # noqa: E731
        L = m.MoEExpertLayer(w.T, w.d, w.f, w.E, w.k, act=m.MOE_F32 if act == "f32" else m.MOE_BF16,
                             balance=(0.0, 0.0), **kw)
        self.block, self.layer, self.fn = m.MoEBlock(L, 0.7), L, MoEBlockFunction
        make = dict(h=d["x"], w_pre=(1 + 0.1 * rnd(w.d)).to(dt).cuda(), w_post=(1 + 0.1 * rnd(w.d)).to(dt).cuda(),
                    gate=torch.sigmoid(rnd(w.T)).cuda(), Wr=d["Wr"], W1=d["W1"], W3=d["W3"], W2=d["W2"])
        self.leaves = [make[n].clone().requires_grad_() for n in self.names]
        self.dy = [(rnd(w.T, w.d).to(dt) * 0.1).cuda() for _ in range(2)]
        self.owner = self.block

    def loss(self, i=0):
        v, loss = self.fn.apply(*self.leaves, self.owner)
        return (v.float() * self.dy[i].float()).sum() + 0.5 * loss[0] + 0.1 * loss[1]

    def grads(self, i=0):
        return torch.autograd.grad(self.loss(i), self.leaves)

    def buffers(self):
        return [t for o in (self.layer, self.owner) for t in vars(o).values() if torch.is_tensor(t)]


class Layer(Block):
    names = LAYER_LEAVES

    def __init__(self, act="bf16", seed=3, **kw):
        from mixture_experts_layer_logits_amd.layer import MoEExpertFunction
        w = SMALL[act]
        d = to_dev(workloads.make_inputs(w))
        self.layer = self.owner = make_layer(w, **kw)
        self.fn = MoEExpertFunction
        self.leaves = [d[n].clone().requires_grad_() for n in self.names]
        g = torch.Generator().manual_seed(seed)
        self.dy = [(torch.randn(w.T, w.d, generator=g).to(w.torch_dtype()) * 0.1).cuda() for _ in range(2)]

    def loss(self, i=0):
        return (self.fn.apply(*self.leaves, self.owner).float() * self.dy[i].float()).sum()


def _own_gradients(c):
    """The gradients are the caller's own: no buffer of the layer or block among them, and a second
    step leaves the first one's as they were."""
    first = c.grads(0)
    kept = [t.clone() for t in first]
    owned = {t.untyped_storage().data_ptr() for t in c.buffers()}
    second = c.grads(1)
    torch.cuda.synchronize()
    for n, a, k, b in zip(c.names, first, kept, second):
        assert a.untyped_storage().data_ptr() not in owned, n
        assert torch.equal(a, k) and not torch.equal(a, b), n


def _notices(c, at):
    """An input changed in place between the passes: the backward says so instead of computing with it."""
    out = c.loss()
    with torch.no_grad():
        c.leaves[at].mul_(2)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        out.backward()


def _reads_what_was_saved(c):
    """Tensors that saved-tensor hooks put elsewhere are what the backward computes with."""
    want = c.grads()
    with torch.autograd.graph.saved_tensors_hooks(lambda t: t.clone(), lambda t: t):
        out = c.loss()
    with torch.no_grad():
        for t in c.leaves:
            t.mul_(2)
    got = torch.autograd.grad(out, c.leaves)
    for n, a, b in zip(c.names, got, want):
        assert torch.equal(a, b), n


def _no_second_derivative(c):
    """The kernels have no derivative of the backward: asking for one raises, it is not left out.  The
    first derivatives are the same either way."""
    want = c.grads()
    got = torch.autograd.grad(c.loss(), c.leaves, create_graph=True)
    for n, a, b in zip(c.names, got, want):
        assert torch.equal(a, b), n
        with pytest.raises(RuntimeError, match="second derivative"):
            (a.float().square().sum() + c.leaves[0].float().sum()).backward(retain_graph=True)


@pytest.mark.parametrize("act", ["f32", "bf16"])
def test_block_gradients_are_the_callers_own(act):
    say(f"[gpu] block gradients kept over two steps {act}")
    _own_gradients(Block(act))


@pytest.mark.parametrize("act", ["f32", "bf16"])
def test_layer_gradients_are_the_callers_own(act):
    say(f"[gpu] layer gradients kept over two steps {act}")
    _own_gradients(Layer(act))


@pytest.mark.parametrize("name", BLOCK_LEAVES)
def test_block_backward_notices_an_input_changed_in_place(name):
    say(f"[gpu] block, {name} changed in place")
    _notices(Block(), BLOCK_LEAVES.index(name))


@pytest.mark.parametrize("recompute", [False, True])
def test_block_backward_reads_what_was_saved(recompute):
    say(f"[gpu] block under saved-tensor hooks recompute={recompute}")
    _reads_what_was_saved(Block(recompute=recompute))


@pytest.mark.parametrize("name", LAYER_LEAVES)
def test_layer_backward_notices_an_input_changed_in_place(name):
    say(f"[gpu] layer, {name} changed in place")
    _notices(Layer(), LAYER_LEAVES.index(name))


@pytest.mark.parametrize("recompute", [False, True])
def test_layer_backward_reads_what_was_saved(recompute):
    say(f"[gpu] layer under saved-tensor hooks recompute={recompute}")
    _reads_what_was_saved(Layer(recompute=recompute))


def test_block_function_refuses_a_layer_with_a_shared_expert():
    """It takes no shared weights, and v without the shared expert's part is another function."""
    say("[gpu] block autograd with a shared expert's layer")
    c = Block(shared_f=64)
    with pytest.raises(ValueError, match="shared expert"):
        c.loss()
    assert c.layer.steps == 0


@pytest.mark.parametrize("make", [Block, Layer])
def test_second_derivatives_raise(make):
    say(f"[gpu] second derivative of {make.__name__}")
    _no_second_derivative(make())


def test_block_refused_forward_leaves_the_one_before():
    """A forward refused for its routing arguments writes nothing: the backward of the one before it is
    the undisturbed one's.  One refused later has overwritten part of it: then the backward raises."""
    say("[gpu] block forward refused between a forward and its backward")
    c = Block()
    B, L = c.block, c.layer
    h, w_pre, w_post, gate, Wr, W1, W3, W2 = (t.detach() for t in c.leaves)
    outs = lambda: [t.clone() for t in (B.dh, B.dw_pre, B.dw_post, L.dWr, L.dW1, L.dx)]  # noqa: E731
    kw = dict(w_pre=w_pre, w_post=w_post, gate=gate)
    B.forward(h, W1, W3, W2, Wr=Wr, **kw)
    B.backward(c.dy[0])
    want = outs()
    B.forward(h, W1, W3, W2, Wr=Wr, **kw)
    with pytest.raises(ValueError, match="learned routing"):
        B.forward(h * 3, W1, W3, W2, topk_idx=L.topk_idx, gates=L.gates, **kw)
    with pytest.raises(ValueError, match="learned routing"):
        B.forward(h * 3, W1, W3, W2, xn=h, w_post=w_post, topk_idx=L.topk_idx, gates=L.gates)
    B.backward(c.dy[0])
    assert all(torch.equal(a, b) for a, b in zip(outs(), want))
    out = c.loss()
    with pytest.raises(ValueError, match="gate"):
        B.forward(h * 3, W1, W3, W2, Wr=Wr, w_pre=w_pre, w_post=w_post, gate=gate.double())
    with pytest.raises(RuntimeError, match="no forward"):
        B.backward(c.dy[0])
    with pytest.raises(RuntimeError, match="another forward"):
        out.backward()
    B.forward(h, W1, W3, W2, Wr=Wr, **kw)
    B.backward(c.dy[0])
    assert all(torch.equal(a, b) for a, b in zip(outs(), want))


def test_block_refuses_its_working_buffers_as_inputs():
    """What the forward or the backward writes before it reads h or xn for the last time."""
    say("[gpu] block on its own buffers")
    c = Block()
    B, L = c.block, c.layer
    h, w_pre, w_post, _, Wr, W1, W3, W2 = (t.detach() for t in c.leaves)
    B.forward(h, W1, W3, W2, w_pre=w_pre, w_post=w_post, w_next=w_pre, Wr=Wr)
    for own in (B.xn, B.v, B.xn_next, B.dv, B.dy, L.dx):
        with pytest.raises(ValueError, match="its own"):
            B.forward(own, W1, W3, W2, w_pre=w_pre, Wr=Wr)
        if own is not B.xn:
            with pytest.raises(ValueError, match="its own"):
                B.forward(h, W1, W3, W2, xn=own, Wr=Wr)
    # its own norm's output is not written when it is given
    B.forward(h, W1, W3, W2, w_pre=w_pre, w_post=w_post, Wr=Wr)
    B.backward(c.dy[0])
    want = [t.clone() for t in (B.v, B.dv, L.dWr)]
    B.forward(h, W1, W3, W2, xn=B.xn, w_post=w_post, Wr=Wr)
    B.backward(c.dy[0])
    assert all(torch.equal(a, b) for a, b in zip((B.v, B.dv, L.dWr), want))


def test_block_on_the_mxfp8_dispatch_refuses_the_layers_output():
    """There the combine writes y before the norm reads h; elsewhere y is the layer's own forward's."""
    import mixture_experts_layer_logits_amd as m
    say("[gpu] block on its layer's y, MXFP8 dispatch")
    L = m.MoEExpertLayer(16, 128, 128, 8, 2, gemm=m.MOE_MXFP8, mx_scope=m.MOE_MX_ALL)
    B, w = m.MoEBlock(L), torch.ones(128, dtype=torch.bfloat16, device="cuda")
    idx = torch.arange(2, dtype=torch.int32, device="cuda").repeat(16, 1)
    with pytest.raises(ValueError, match="its own"):
        B.forward(L.y, None, None, None, w_pre=w, topk_idx=idx, gates=torch.ones(16, 2, device="cuda"))
    assert L.steps == 0


@pytest.mark.parametrize("create_graph", [False, True])
def test_block_function_without_the_norm_behind_and_the_gate(create_graph):
    """None for w_post and gate: the gradients of the others are the block's own backward's."""
    say(f"[gpu] block autograd, no w_post, no gate, create_graph={create_graph}")
    c = Block("f32")
    c.leaves[2] = c.leaves[3] = None
    given = [t for t in c.leaves if t is not None]
    v, loss = c.fn.apply(*c.leaves, c.block)
    got = torch.autograd.grad([v, loss], given, [c.dy[0], torch.tensor([0.5, 0.1], device="cuda")],
                              create_graph=create_graph)
    h, w_pre, _, _, Wr, W1, W3, W2 = (None if t is None else t.detach() for t in c.leaves)
    B, L = c.block, c.layer
    assert torch.equal(B.forward(h, W1, W3, W2, w_pre=w_pre, Wr=Wr), v.detach())
    B.backward(c.dy[0], dloss=torch.tensor([0.5, 0.1], device="cuda"))
    for a, b in zip(got, (B.dh, B.dw_pre, L.dWr, L.dW1, L.dW3, L.dW2)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("make", [Block, Layer])
def test_functions_under_inference_mode(make):
    say(f"[gpu] {make.__name__} under inference_mode")
    c = make()
    want = c.fn.apply(*c.leaves, c.owner)
    with torch.inference_mode():
        got = c.fn.apply(*c.leaves, c.owner)
    for a, b in zip(want, got):
        assert torch.equal(a.detach(), b)
