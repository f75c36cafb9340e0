"""The router's weight gradient at expert counts that are no multiple of 8, where a row of score
gradients ends inside a 16-byte load."""
import numpy as np
import pytest
import torch

from gpu_common import host, say

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("E", [1, 2, 7, 12, 33, 97, 130])
@pytest.mark.parametrize("T,d", [(130, 320), (513, 64)])
def test_router_weight_gradient_of_every_expert(E, T, d):
    import mixture_experts_layer_logits_amd as m
    say(f"[gpu] router weight gradient T={T} d={d} E={E}")
    s = m.make_shape(T, d, 64, E, 1)
    g = torch.Generator().manual_seed(E)
    dl = torch.randn(T, E, generator=g).bfloat16().float()  # what its bf16 copy holds exactly
    x, Wr = torch.randn(T, d, generator=g).bfloat16(), torch.randn(E, d, generator=g).bfloat16()
    dWr, dxr = torch.empty(E, d, device="cuda"), torch.empty(T, d, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(m.moe_workspace_size(s), dtype=torch.uint8, device="cuda")
    m.moe_router_bwd(s, x.cuda(), Wr.cuda(), dl.cuda(), dxr, dWr, ws)
    want = dl.double().t() @ x.double()
    # T exact products, each addition rounds by 2^-24 of the sum of magnitudes
    bound = T * 2.0 ** -24 * (dl.abs().double().t() @ x.abs().double())
    assert np.all(np.abs(host(dWr) - want.numpy()) <= bound.numpy())
    want = dl.double() @ Wr.double()
    bound = E * 2.0 ** -24 * (dl.abs().double() @ Wr.abs().double()) + 2.0 ** -8 * want.abs()
    assert np.all(np.abs(host(dxr).astype(np.float64) - want.numpy()) <= bound.numpy() + 1e-30)
