"""Paths through the layer with 8-bit checkpoints and with 4-bit weights that a program takes beside the whole
step: a block next to the plain one, autograd through a block, empty batches, other streams."""
import numpy as np
import pytest
import torch

import workloads
from gpu_common import say, to_dev
from test_gpu_few_bits_layer import CASES, GRADS, _forward, _layer

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
