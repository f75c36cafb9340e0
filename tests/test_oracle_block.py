"""Pins for the CPU oracle of the operators around the expert layer (no GPU): closed forms,
torch's own softmax and logsumexp, and central finite differences for every gradient."""
import numpy as np
import pytest
import torch

from oracle import block_ref as ref
from oracle import moe_ref


def _diff(f, a, h=1e-5):
    """Central differences of the scalar f() in every element of a (changed in place)."""
    out = np.zeros_like(a)
    for i in np.ndindex(a.shape):
        old = a[i]
        a[i] = old + h
        up = f()
        a[i] = old - h
        out[i] = (up - f()) / (2 * h)
        a[i] = old
    return out


def _close(got, want, tol=1e-8):
    np.testing.assert_allclose(got, want, rtol=tol, atol=tol)


# ------------------------------------------------------------------ balance loss
def test_even_routing_has_loss_one_and_a_zero_balance_gradient():
    T, E, k = 12, 6, 2
    L = np.zeros((T, E))
    idx = np.array([[(2 * t) % E, (2 * t + 1) % E] for t in range(T)])
    fw = ref.balance_fwd(L, idx)
    assert fw["counts"].tolist() == [4] * 6 + [12]
    _close(fw["loss"], [1.0, np.log(E) ** 2])
    bw = ref.balance_bwd(L, fw["lse"], fw["counts"], [1.0, 0.0])
    _close(bw["dlogits"], 0.0)


def test_balance_forward_against_torch():
    rng = np.random.default_rng(0)
    L = rng.normal(size=(9, 5)) * 2
    mask = np.array([1, 1, 0, 1, 0, 1, 1, 1, 1])
    idx, _ = moe_ref.topk_gates(L, 2)
    fw = ref.balance_fwd(L, idx, mask)
    rows = torch.from_numpy(L[mask != 0])
    _close(fw["prob_mean"], torch.softmax(rows, 1).mean(0).numpy())
    _close(fw["lse"][mask != 0], torch.logsumexp(rows, 1).numpy())
    assert np.isneginf(fw["lse"][mask == 0]).all()
    chosen = idx[mask != 0].reshape(-1)
    assert fw["counts"].tolist() == [int((chosen == e).sum()) for e in range(5)] + [7]


def test_tokens_left_out_enter_nothing():
    rng = np.random.default_rng(1)
    L = rng.normal(size=(6, 4))
    idx, _ = moe_ref.topk_gates(L, 2)
    alone = ref.balance_fwd(L[:3], idx[:3])
    L[3] = np.nan
    L[4] = np.inf
    L[5] = -np.inf  # no score above -inf: out without a mask
    fw = ref.balance_fwd(L, idx, np.array([1, 1, 1, 0, 0, 1]))
    for key in ("counts", "prob_mean", "loss"):
        _close(fw[key], alone[key])
    bw = ref.balance_bwd(L, fw["lse"], fw["counts"], [1.0, 1.0])
    assert not bw["dlogits"][3:].any() and np.isfinite(bw["dlogits"]).all()
    empty = ref.balance_fwd(L, idx, np.zeros(6))
    assert empty["counts"].tolist() == [0] * 5 and not empty["loss"].any()
    assert not ref.balance_bwd(L, empty["lse"], empty["counts"], [1.0, 1.0])["dlogits"].any()


@pytest.mark.parametrize("T,E,k", [(5, 4, 2), (7, 6, 3), (1, 3, 1)])
def test_balance_gradient_against_differences(T, E, k):
    rng = np.random.default_rng(T)
    L = rng.normal(size=(T, E))
    idx, g = moe_ref.topk_gates(L, k)
    mask = np.ones(T) if T == 1 else (np.arange(T) != 2).astype(float)
    dgates = rng.normal(size=(T, k))
    w = np.array([0.7, -0.3])

    def loss():  # the choices are held: counts have no gradient
        chosen = np.take_along_axis(L, idx, axis=1)
        e = np.exp(chosen - chosen.max(axis=1, keepdims=True))
        return w @ ref.balance_fwd(L, idx, mask)["loss"] + (dgates * e / e.sum(axis=1, keepdims=True)).sum()

    fw = ref.balance_fwd(L, idx, mask)
    bw = ref.balance_bwd(L, fw["lse"], fw["counts"], w, topk=(idx, g, dgates))
    _close(bw["dlogits"], _diff(loss, L), 1e-8)


def test_balance_gradient_over_ranks_adds_up():
    rng = np.random.default_rng(3)
    L = rng.normal(size=(10, 5))
    idx, _ = moe_ref.topk_gates(L, 2)
    whole = ref.balance_fwd(L, idx)
    counts = sum(ref.balance_fwd(L[s], idx[s])["counts"] for s in (slice(0, 4), slice(4, 10)))
    assert np.array_equal(counts, whole["counts"])
    full = ref.balance_bwd(L, whole["lse"], counts, [1.0, 0.5])["dlogits"]
    part = ref.balance_bwd(L[4:], whole["lse"][4:], counts, [1.0, 0.5])["dlogits"]
    _close(part, full[4:])


# ------------------------------------------------------------------ block norms
def test_norm_forward_closed_forms():
    x = np.array([[3.0, 4.0]])
    fw = ref.norm_fwd(x, w_pre=np.array([1.0, 2.0]), eps=1e-30)
    _close(fw["xn"], [[3 / np.sqrt(12.5), 8 / np.sqrt(12.5)]])
    # a row of constant size c: norm gives its sign
    fw = ref.norm_fwd(x, y=np.array([[5.0, -5.0]]), w_post=np.ones(2), res_scale=0.5, gate=np.array([2.0]), eps=1e-30)
    _close(fw["v"], [[4.0, 3.0]])
    shut = ref.norm_fwd(x, y=np.array([[np.nan, np.inf]]), w_post=np.ones(2), gate=np.zeros(1))
    _close(shut["v"], x)
    zero = ref.norm_fwd(np.zeros((1, 4)), w_pre=np.ones(4), eps=0.25)
    _close(zero["rstd_pre"], 2.0)


@pytest.mark.parametrize("branch", ["none", "y", "combine"])
@pytest.mark.parametrize("post", [False, True])
@pytest.mark.parametrize("pre", [False, True])
@pytest.mark.parametrize("gated", [False, True])
def test_norm_gradients_against_differences(branch, post, pre, gated):
    if branch == "none" and (post or gated or not pre):
        pytest.skip("no branch to norm or gate")
    T, d, k = 4, 6, 2
    rng = np.random.default_rng(11)
    a = {"x": rng.normal(size=(T, d))}
    if branch == "y":
        a["y"] = rng.normal(size=(T, d))
    if branch == "combine":
        a["y_perm"], a["gates"], a["y_add"] = rng.normal(size=(T * k, d)), rng.random((T, k)), rng.normal(size=(T, d))
    slot = rng.permutation(T * k).reshape(T, k)
    if post:
        a["w_post"] = 1 + 0.2 * rng.normal(size=d)
    if pre:
        a["w_pre"] = 1 + 0.2 * rng.normal(size=d)
    if gated:
        a["gate"] = rng.normal(size=T)
    dv, dxn = rng.normal(size=(T, d)), rng.normal(size=(T, d))
    scale, eps = 0.8, 1e-3

    def fwd():
        comb = (a["y_perm"], a["gates"], slot, a["y_add"]) if branch == "combine" else None
        return ref.norm_fwd(a["x"], y=a.get("y"), gate=a.get("gate"), w_post=a.get("w_post"), w_pre=a.get("w_pre"),
                            res_scale=scale, eps=eps, combine=comb)

    def loss():
        fw = fwd()
        v = fw["v"] if "v" in fw else a["x"]
        return (dv * v).sum() + ((dxn * fw["xn"]).sum() if pre else 0.0)

    fw = fwd()
    comb = (a["y_perm"], a["gates"], slot, a["y_add"]) if branch == "combine" else None
    bw = ref.norm_bwd(dv=dv, dxn=dxn if pre else None, v=fw["v"] if "v" in fw else a["x"], y=a.get("y"),
                      gate=a.get("gate"), w_post=a.get("w_post"), w_pre=a.get("w_pre"),
                      rstd_post=fw.get("rstd_post"), rstd_pre=fw.get("rstd_pre"), res_scale=scale, combine=comb)
    names = {"x": "dx", "y": "dy", "y_add": "dy", "y_perm": "dy_perm", "gates": "dgates", "w_post": "dw_post",
             "w_pre": "dw_pre", "gate": "dgate"}
    for n, t in a.items():
        _close(bw[names[n]], _diff(loss, t), 2e-8)


def test_a_closed_gate_has_a_gradient_and_passes_none():
    rng = np.random.default_rng(5)
    x, y, dv = (rng.normal(size=(2, 5)) for _ in range(3))
    gate = np.array([0.0, 1.0])
    fw = ref.norm_fwd(x, y=y, gate=gate, w_post=np.ones(5))
    bw = ref.norm_bwd(dv=dv, y=y, gate=gate, w_post=np.ones(5), rstd_post=fw["rstd_post"])
    assert not bw["dy"][0].any() and bw["dy"][1].any()
    _close(bw["dgate"], _diff(lambda: (dv * ref.norm_fwd(x, y=y, gate=gate, w_post=np.ones(5))["v"]).sum(), gate), 1e-7)
