"""What a block over a layer with 4-bit weights holds: the forward's buffers alone."""
import torch

import mixture_experts_layer_logits_amd as m


def _tensors(o):
    return {n: t for n, t in vars(o).items() if isinstance(t, torch.Tensor)}


def test_a_serving_block_holds_no_gradient_buffers():
    mk = lambda **kw: m.MoEBlock(m.MoEExpertLayer(64, 128, 64, 4, 2, device="cpu", **kw))  # noqa: E731
    serve, train = _tensors(mk(weights4=True)), _tensors(mk())
    forward = {"xn", "v", "xn_next", "rstd_pre", "rstd_post", "rstd_next"}
    assert set(serve) == forward
    assert set(train) == forward | {"dv", "dh", "dy", "dgate", "dw_pre", "dw_post", "dw_next"}
