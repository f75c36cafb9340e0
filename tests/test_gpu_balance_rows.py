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


# Roundings (2^-24 each) between a row's scores and its outputs, whatever T is:
#   exp_neg is within 2 units in the last place, 4 roundings; its argument's own rounding shifts it by
#   |z| more, z = score - top or score - lse
#   a sum over a row: at most 16 terms a lane, then 6 exchanges: 22
#   lse = top + log(sum): log within 2 units (4 log(sum)), one of the addition (|lse|); the sum's relative
#   error is log's absolute one
#   dlogits: p 4 + |z|; c_e / N 2; the inner sum 22 + 4 + |z| + 2 of its terms' own; a 4, b 3, b l 1;
#   difference, fma and product 3; the gate's part: 5 exchanges over 32 choices, 4 operations, the last sum
LSE = 22 + 4
DLOGITS = 22 + (4 + 2) + (4 + 2) + 4 + 3 + 1 + 3 + 5 + 4 + 1


@pytest.mark.parametrize("T,E,k,spread", [
    (300, 8, 2, 1.5), (2000, 128, 4, 1.5), (65, 1024, 32, 1.5), (130, 1000, 4, 8.0), (77, 33, 4, 40.0),
    # the forward's layouts of several loads a lane
    (25001, 96, 6, 1.5), (12500, 513, 8, 1.5), (50003, 40, 1, 4.0), (50021, 37, 3, 1.5)])
def test_rows_are_as_exact_as_their_roundings(T, E, k, spread):
    say(f"[gpu] balance rows T={T} E={E} k={k} spread={spread}")
    L, idx, gates, dgates = _balance_inputs(T, E, k, T + E, spread)
    L[T // 2, ::3] = -float("inf")
    b = Balance(L, idx, gates, dgates, dloss=(0.7, 0.2)).fwd().bwd()
    torch.cuda.synchronize()
    x = L.double().numpy()
    top = x.max(axis=1, keepdims=True)
    e = np.exp(x - top)
    s = e.sum(axis=1, keepdims=True)
    want = (top + np.log(s))[:, 0]
    z = np.where(np.isneginf(x), 0, np.abs(x - top))
    shift = (e / s * z).sum(axis=1)  # what the arguments' roundings do to the sum, weighted as they are
    got = host(b.lse).astype(np.float64)
    bound = (LSE + shift + 4 * np.log(s[:, 0]) + np.abs(want)) * F32
    assert np.all(np.abs(got - want) <= bound), np.max(np.abs(got - want) / bound)
    c = np.bincount(idx.numpy().reshape(-1), minlength=E)
    assert np.array_equal(host(b.counts), np.append(c, T))
    # the backward from the stored lse: rows written out apart from the oracle's loop
    l = got[:, None]
    p = np.exp(x - l)
    z = np.where(np.isneginf(x), 0, np.abs(x - l))
    f = c / T
    w = host(b.dloss).astype(np.float64)
    bal, zl = w[0] * E / (k * T), w[1] * 2 * l / T
    out = p * (bal * (f - (p * f).sum(axis=1, keepdims=True)) + zl)
    mag = p * (abs(bal) * (f + (p * f).sum(axis=1, keepdims=True)) + np.abs(zl))
    far = p * (abs(bal) * (p * f * z).sum(axis=1, keepdims=True)) + z * mag
    g, dg = gates.double().numpy(), dgates.double().numpy()
    at = (np.arange(T)[:, None], idx.numpy().astype(np.int64))
    out[at] += g * (dg - (g * dg).sum(axis=1, keepdims=True))
    mag[at] += g * (np.abs(dg) + (g * np.abs(dg)).sum(axis=1, keepdims=True))
    got = host(b.dlogits.view(T, E)).astype(np.float64)
    bound = (DLOGITS * mag + far) * F32 + 2.0 ** -126  # p below the smallest normal value is zero
    assert np.all(np.abs(got - out) <= bound), np.max(np.abs(got - out) / bound)


def test_probabilities_are_within_two_units():
    """p = e^(score - lse) alone: with lse 1, one kept token counted, loss weights (0, 1/2) and no gates,
    dlogits is p times exactly 1.  The argument is taken as the kernel rounds it."""
    import mixture_experts_layer_logits_amd as m
    say("[gpu] balance backward, the exponential")
    T, E = 4096, 64
    g = torch.Generator().manual_seed(1)
    x = (1 - torch.exp(torch.rand(T, E, generator=g) * 12 - 7)).float()  # z from -1e-3 to -150
    x[0, :4] = torch.tensor([1.0, 1.0 - 2.0 ** -23, -86.0, -400.0])
    s = m.make_shape(T, 64, 64, E, 1, m.MOE_F32)
    counts = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    counts[0] = counts[E] = 1
    out = torch.empty(T, E, device="cuda")
    m.moe_balance_bwd(s, x.cuda(), torch.ones(T, device="cuda"), counts, torch.tensor([0.0, 0.5], device="cuda"), None,
                      None, None, out)
    got = host(out)
    z = x.numpy() - np.float32(1)
    assert z.dtype == np.float32
    want = np.exp(z.astype(np.float64))
    normal = want >= 2.0 ** -126
    unit = np.spacing(want[normal].astype(np.float32)).astype(np.float64)
    worst = np.max(np.abs(got[normal] - want[normal]) / unit)
    assert worst <= 2, worst
    assert np.all(got[~normal] <= 2.0 ** -126) and got[0, 0] == 1 and got[0, 3] == 0
