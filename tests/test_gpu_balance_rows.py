"""What the balance loss gives each token, at the precision of a row: no sum over tokens stands
between the scores and lse or dlogits, so the number of tokens is in neither bound."""
import numpy as np
import pytest
import torch

from gpu_common import host, say
from oracle import block_ref as ref
from test_gpu_block import F32, Balance, _balance_inputs

pytestmark = pytest.mark.gpu


def test_ids_out_of_range_have_no_gate_gradient():
    """The forward counts them as the nearest expert; the gates' gradient of such a choice has no
    score to go to and is left out, as in moe_route_bwd.  The others' keep its share of sum_j."""
    import mixture_experts_layer_logits_amd as m
    say("[gpu] balance backward, ids out of range")
    L, idx, gates, dgates = _balance_inputs(30, 8, 2, 3)
    idx[4] = torch.tensor([-5, 8])
    idx[9] = torch.tensor([2 ** 31 - 1, -(2 ** 31)])
    idx[11, 1] = 8
    b = Balance(L, idx, gates, dgates, dloss=(0.0, 0.0)).fwd().bwd()
    want = torch.empty(30, 8, device="cuda")
    m.moe_route_bwd(b.s, b.dgates, b.gates, b.idx, want)
    got = host(b.dlogits.view(30, 8)).astype(np.float64)
    g, dg = gates.double().numpy(), dgates.double().numpy()
    # two orders of two terms: at most two roundings a sum, one of the difference and one of the product
    mag = (g * (np.abs(dg) + (g * np.abs(dg)).sum(1, keepdims=True))).max(1, keepdims=True)
    assert np.all(np.abs(got - host(want)) <= 8 * F32 * mag)
    assert not got[4].any() and not got[9].any() and np.count_nonzero(got[11]) == 1


def test_masks_of_truth_values():
    """A bool mask is the same bytes as the uint8 one, in the calls and through the layer."""
    import mixture_experts_layer_logits_amd as m
    say("[gpu] balance forward, bool mask")
    L, idx, gates, dgates = _balance_inputs(300, 8, 2, 3)
    keep = torch.arange(300) % 3 != 1
    a = Balance(L, idx, gates, dgates, keep.to(torch.uint8)).fwd()
    b = Balance(L, idx, gates, dgates, keep).fwd()
    for n in ("lse", "counts", "prob", "loss"):
        assert torch.equal(getattr(a, n), getattr(b, n)), n
    layer = m.MoEExpertLayer(300, 64, 64, 8, 2, balance=(1.0, 1.0))
    x, Wr = torch.randn(300, 64, device="cuda").bfloat16(), torch.randn(8, 64, device="cuda").bfloat16()
    layer.route(x, Wr, mask=keep.cuda())
    assert int(layer.bal_counts[8]) == 200
    with pytest.raises(ValueError, match="mask"):
        Balance(L, idx, gates, dgates, keep.float()).fwd()
