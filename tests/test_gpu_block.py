"""GPU parity of the operators around the expert layer against the fp64 oracle: balance loss,
block norms, combine with norms, each forward and backward.

Tolerances count roundings.  The oracle gives every output's magnitude (the same formula over
absolute values).  A float value is off by at most n 2^-24 of its magnitude, n the roundings on
its path: a lane's share of a row is at most 16 terms, the wave and up to 16 waves of a row add
6 + 16, k <= 32 gathered rows 32, and at most two such row sums with some 20 single operations
follow one another, so n = 2 (16 + 6 + 16) + 32 + 20 = 128.  Sums over tokens add a rounding a
token: n = 128 + T.  A stored row rounds once more, by half a step (finfo.eps / 2) of its value.
For the balance loss p = exp(z) is off by a rounding of z = logit - lse (|z| 2^-24) on top, so n
grows by R = the largest |z| in the case.
"""
import numpy as np
import pytest
import torch

from gpu_common import host, say
from oracle import block_ref as ref
from oracle import moe_ref

pytestmark = pytest.mark.gpu

F32 = 2.0 ** -24
EPS = 1e-6


def _m():
    import mixture_experts_layer_logits_amd as m
    return m


def _check(got, want, mag, n, what):
    """|got - want| <= n 2^-24 mag + half a step of the stored type at want."""
    g = host(got).astype(np.float64)
    half = torch.finfo(got.dtype).eps / 2
    bound = n * F32 * mag + half * np.abs(want) + 1e-37
    assert np.isfinite(g).all(), what
    worst = np.max(np.abs(g - want) / bound)
    assert worst <= 1, (what, worst)


# ------------------------------------------------------------------ balance loss
def _balance_inputs(T, E, k, seed, spread=1.5):
    g = torch.Generator().manual_seed(seed)
    L = torch.randn(T, E, generator=g) * spread + torch.randn(1, E, generator=g)
    idx = torch.topk(L, k, dim=1).indices.to(torch.int32)
    gates = torch.softmax(torch.gather(L, 1, idx.long()), 1)
    return L, idx, gates, torch.randn(T, k, generator=g) * 0.1


class Balance:
    """One pass of both calls on device copies of the inputs; outputs start as junk."""

    def __init__(self, L, idx, gates, dgates, mask=None, dloss=(1e-2, 1e-3), offset=0):
        m = _m()
        T, E = L.shape
        self.s = m.make_shape(T, 64, 64, E, idx.shape[1], m.MOE_F32)
        junk = lambda *n: torch.full(n, float("nan"), device="cuda")  # noqa: E731

        def place(t):  # offset: elements before the first, so a row starts off 16-byte alignment
            buf = junk(t.numel() + offset)
            buf[offset:] = t.reshape(-1).cuda()
            return buf[offset:]
        self.logits = place(L)
        self.idx, self.gates, self.dgates = idx.cuda(), gates.cuda(), dgates.cuda()
        self.mask = None if mask is None else mask.cuda()
        self.dloss = torch.tensor(dloss, device="cuda")
        self.lse, self.prob, self.loss = junk(T), junk(E), junk(2)
        self.counts = torch.full((E + 1,), -7, dtype=torch.int32, device="cuda")
        self.dlogits = junk(T * E + offset)[offset:]
        self.ws = torch.full((m.moe_workspace_size(self.s),), 255, dtype=torch.uint8, device="cuda")

    def fwd(self):
        _m().moe_balance_fwd(self.s, self.logits, self.idx, self.mask, self.lse, self.counts, self.prob, self.loss,
                             self.ws)
        return self

    def bwd(self, gates=True):
        _m().moe_balance_bwd(self.s, self.logits, self.lse, self.counts, self.dloss, self.dgates if gates else None,
                             self.gates if gates else None, self.idx if gates else None, self.dlogits)
        return self


def _check_balance(b, L, idx, gates, dgates, mask, with_gates=True):
    T, E = L.shape
    fw = ref.balance_fwd(L, idx, mask)
    kept = np.isfinite(fw["lse"])
    z = np.abs(np.where(np.isfinite(host(L)), host(L), 0) - np.where(kept, fw["lse"], 0)[:, None])[kept]
    n = 128 + T + (z.max() if kept.any() else 0)
    assert np.array_equal(host(b.counts), fw["counts"])
    lse = host(b.lse).astype(np.float64)
    assert np.array_equal(np.isneginf(lse), ~kept)
    # lse = top + log(sum): a rounding each, the log's argument off by the sum's roundings
    assert np.all(np.abs(lse[kept] - fw["lse"][kept]) <= n * F32 * (1 + np.abs(fw["lse"][kept])))
    _check(b.prob, fw["prob_mean"], fw["prob_mean"], 2 * n, "prob_mean")
    # loss[0]: positive terms; loss[1]: mean of squares whose lse is off as above
    _check(b.loss[:1], fw["loss"][:1], fw["loss"][:1], 2 * n, "balance loss")
    lse_mag = np.mean((1 + np.abs(fw["lse"][kept])) ** 2) if kept.any() else 0.0
    _check(b.loss[1:], fw["loss"][1:], np.array([lse_mag]), 3 * n, "z loss")
    # the backward from the forward's own lse, as stored
    bw = ref.balance_bwd(L, lse, fw["counts"], host(b.dloss), topk=(idx, gates, dgates) if with_gates else None)
    _check(b.dlogits.view(T, E), bw["dlogits"], bw["mag"]["dlogits"], 2 * n, "dlogits")


@pytest.mark.parametrize("T,E,k", [
    (1, 1, 1), (1, 128, 4), (5, 2, 1), (64, 3, 3), (300, 8, 2), (1025, 8, 8), (257, 33, 4), (64, 64, 32), (513, 96, 6),
    (2000, 128, 4), (77, 130, 5), (100, 256, 8), (63, 257, 2), (130, 1000, 4), (65, 1024, 32), (9001, 16, 2),
    # past three rounds of the widest layout: several loads a lane
    (13000, 134, 2), (25001, 96, 6), (12500, 513, 8), (50003, 40, 1)])
@pytest.mark.parametrize("masked", [False, True])
def test_balance_against_oracle(T, E, k, masked):
    say(f"[gpu] balance T={T} E={E} k={k} masked={masked}")
    L, idx, gates, dgates = _balance_inputs(T, E, k, T + E)
    mask = None
    if masked:  # tokens left out hold NaN and infinities
        mask = (torch.arange(T) % 3 != 1).to(torch.uint8)
        L[mask == 0] = float("nan")
        if T > 4:
            L[4] = float("inf")
            mask[4] = 0
    b = Balance(L, idx, gates, dgates, mask).fwd().bwd()
    torch.cuda.synchronize()
    _check_balance(b, L, idx, gates, dgates, mask)
    b.bwd(gates=False)
    _check_balance(b, L, idx, gates, dgates, mask, with_gates=False)


@pytest.mark.parametrize("case", ["all_out", "one_kept", "minus_inf", "far_apart", "unaligned", "one_expert_hot"])
def test_balance_edges(case):
    say(f"[gpu] balance edge {case}")
    T, E, k = 70, 32, 4
    L, idx, gates, dgates = _balance_inputs(T, E, k, 5, spread=40.0 if case == "far_apart" else 1.5)
    mask, offset = None, 0
    if case == "all_out":
        mask = torch.zeros(T, dtype=torch.uint8)
    if case == "one_kept":
        mask = torch.zeros(T, dtype=torch.uint8)
        mask[69] = 1
    if case == "minus_inf":  # experts out of use, and tokens with no score at all
        L[:, 7] = -float("inf")
        L[3] = L[64] = -float("inf")
    if case == "unaligned":
        offset = 1
    if case == "one_expert_hot":
        idx[:, 0] = 9
    b = Balance(L, idx, gates, dgates, mask, offset=offset).fwd().bwd()
    torch.cuda.synchronize()
    _check_balance(b, L, idx, gates, dgates, mask)
    if case == "all_out":
        assert not host(b.loss).any() and not host(b.prob).any()


def test_balance_of_no_tokens():
    L, idx, gates, dgates = _balance_inputs(4, 8, 2, 1)
    b = Balance(L[:0], idx[:0], gates[:0], dgates[:0]).fwd().bwd()
    torch.cuda.synchronize()
    assert not host(b.counts).any() and not host(b.loss).any() and not host(b.prob).any()


def test_balance_nan_of_a_kept_token_reaches_the_loss():
    L, idx, gates, dgates = _balance_inputs(40, 8, 2, 2)
    L[17, 3] = float("nan")
    b = Balance(L, idx, gates, dgates).fwd().bwd()
    assert np.isnan(host(b.loss)).all() and np.isnan(host(b.lse)[17])
    d = host(b.dlogits).reshape(40, 8)
    assert np.isnan(d[17]).any() and np.isfinite(np.delete(d, 17, axis=0)).all()


@pytest.mark.parametrize("T,E,k", [(333, 128, 4), (50, 33, 3), (20, 1024, 32), (31, 4, 4), (9, 40, 32)])
def test_balance_with_zero_weights_is_route_bwd(T, E, k):
    """Both compute g (dg - S), S = sum_j g_j dg_j, in other orders of the k terms: each S is off by at
    most k roundings of its magnitude, the difference and the product add one each on both sides."""
    m = _m()
    L, idx, gates, dgates = _balance_inputs(T, E, k, 7)
    b = Balance(L, idx, gates, dgates, dloss=(0.0, 0.0)).fwd().bwd()
    want = torch.empty(T, E, device="cuda")
    m.moe_route_bwd(b.s, b.dgates, b.gates, b.idx, want)
    got, want = host(b.dlogits.view(T, E)).astype(np.float64), host(want).astype(np.float64)
    g, dg = gates.double().numpy(), dgates.double().numpy()
    mag = np.zeros((T, E))
    np.put_along_axis(mag, idx.numpy().astype(np.int64), g * (np.abs(dg) + (g * np.abs(dg)).sum(1, keepdims=True)), 1)
    assert np.all(np.abs(got - want) <= (2 * k + 4) * F32 * mag)


def test_balance_counts_are_the_routes():
    m = _m()
    L, idx, gates, dgates = _balance_inputs(1000, 96, 6, 8)
    b = Balance(L, idx, gates, dgates).fwd()
    i32 = dict(dtype=torch.int32, device="cuda")
    counts, off, slot = torch.empty(96, **i32), torch.empty(97, **i32), torch.empty(1000, 6, **i32)
    ri, rg = torch.empty(1000, 6, **i32), torch.empty(1000, 6, device="cuda")
    m.moe_route(b.s, b.logits, ri, rg, counts, off, slot, b.ws.clone())
    assert torch.equal(b.counts[:96], counts) and int(b.counts[96]) == 1000


def test_balance_over_ranks():
    """Two ranks' tokens with the counts added up: each rank's rows of the whole batch's gradient."""
    L, idx, gates, dgates = _balance_inputs(500, 64, 4, 9)
    whole = Balance(L, idx, gates, dgates).fwd().bwd()
    parts = [Balance(L[s], idx[s], gates[s], dgates[s]).fwd() for s in (slice(0, 123), slice(123, 500))]
    total = parts[0].counts + parts[1].counts
    for p in parts:
        p.counts.copy_(total)
        p.bwd()
    assert torch.equal(torch.cat([p.dlogits for p in parts]), whole.dlogits)


def test_balance_ids_out_of_range_are_clamped():
    L, idx, gates, dgates = _balance_inputs(30, 8, 2, 3)
    idx[4] = torch.tensor([-5, 8])
    idx[9] = torch.tensor([2 ** 31 - 1, -(2 ** 31)])
    b = Balance(L, idx, gates, dgates).fwd()
    assert np.array_equal(host(b.counts), ref.balance_fwd(L, idx)["counts"])


def test_balance_offsets_past_32_bits():
    m = _m()
    T, E, k = 2 ** 21 + 3, 1024, 1
    say(f"[gpu] balance T={T} E={E} (2^31 scores)")
    s = m.make_shape(T, 64, 64, E, k, m.MOE_F32)
    L = torch.zeros(T, E, device="cuda")
    L[-1, 5], L[0, 3] = 2.0, 1.0
    idx = torch.zeros(T, k, dtype=torch.int32, device="cuda")
    lse, prob, loss = torch.empty(T, device="cuda"), torch.empty(E, device="cuda"), torch.empty(2, device="cuda")
    counts = torch.empty(E + 1, dtype=torch.int32, device="cuda")
    ws = torch.empty(m.moe_workspace_size(s), dtype=torch.uint8, device="cuda")
    m.moe_balance_fwd(s, L, idx, None, lse, counts, prob, loss, ws)
    assert abs(float(lse[-1]) - np.log(1023 + np.exp(2.0))) < 1e-5 and abs(float(lse[0]) - np.log(1023 + np.e)) < 1e-5
    assert int(counts[0]) == T and int(counts[E]) == T
    out = torch.full((T, E), 7.0, device="cuda")
    m.moe_balance_bwd(s, L, lse, counts, torch.tensor([0.0, 1.0], device="cuda"), None, None, None, out)
    want = ref.balance_bwd(host(L[-3:]), host(lse[-3:]), host(counts), [0.0, 1.0])["dlogits"]
    np.testing.assert_allclose(host(out[-3:]), want, rtol=1e-4)
    del L, out


# ------------------------------------------------------------------ block norms
class Norm:
    """Inputs of one case (host copies in c, device copies in d) and the calls on them.  Row buffers
    have GUARD rows behind the last one, which every call has to leave alone."""
    GUARD = 3

    def __init__(self, T, d, act="bf16", branch="y", post=True, pre=True, gated=True, k=2, add=False, seed=0,
                 scale=0.5):
        m = _m()
        dt = torch.float32 if act == "f32" else torch.bfloat16
        self.T, self.d_, self.k, self.dt, self.branch, self.scale = T, d, k, dt, branch, scale
        E = max(k, 4)
        self.s = m.make_shape(T, d, 64, E, k, m.MOE_F32 if act == "f32" else m.MOE_BF16)
        g = torch.Generator().manual_seed(seed)
        rnd = lambda *n: torch.randn(*n, generator=g)  # noqa: E731
        c = dict(x=(rnd(T, d) * torch.exp(0.5 * rnd(1, d))).to(dt))
        c["dv"] = (0.1 * rnd(T, d)).to(dt)
        if pre:
            c["w_pre"], c["dxn"] = (1 + 0.1 * rnd(d)).to(dt), (0.1 * rnd(T, d)).to(dt)
        if branch != "none":
            if post:
                c["w_post"] = (1 + 0.1 * rnd(d)).to(dt)
            if gated:
                c["gate"] = torch.sigmoid(rnd(T))
                c["gate"][1::5] = 0.0
        if branch == "y":
            c["y"] = (0.3 * rnd(T, d)).to(dt)
        if branch == "combine":
            logits = rnd(T, E)
            idx, gates = moe_ref.topk_gates(logits, k)
            c["gates"] = torch.from_numpy(gates).float()
            c["slot_row"] = torch.from_numpy(np.ascontiguousarray(moe_ref.dispatch(idx, E)[2])).to(torch.int32)
            c["y_perm"] = (0.3 * rnd(T * k, d)).to(dt)
            if add:
                c["y_add"] = (0.2 * rnd(T, d)).to(dt)
        self.c = c
        self.d = {n: t.cuda() for n, t in c.items()}
        self.ws = torch.full((m.moe_workspace_size(self.s),), 255, dtype=torch.uint8, device="cuda")
        self.bufs = {}

    def out(self, name, rows, *width, dtype=None):
        buf = torch.full((rows + self.GUARD, *width), -3.0, dtype=dtype or torch.float32, device="cuda")
        self.bufs[name] = buf
        return buf[:rows]

    def get(self, n):
        return self.d.get(n)

    def fwd(self, inplace=False):
        m, T, d = _m(), self.T, self.d_
        pre, post, br = "w_pre" in self.d, "w_post" in self.d, self.branch != "none"
        o = self.o = {}
        x = self.d["x"].clone() if inplace else self.d["x"]
        o["v"] = None if not br else (x if inplace else self.out("v", T, d, dtype=self.dt))
        o["xn"] = self.out("xn", T, d, dtype=self.dt) if pre else None
        o["rstd_post"] = self.out("rstd_post", T) if post else None
        o["rstd_pre"] = self.out("rstd_pre", T) if pre else None
        tail = (self.get("gate"), self.get("w_post"), self.get("w_pre"), self.scale, EPS, o["v"], o["xn"],
                o["rstd_post"], o["rstd_pre"])
        if self.branch == "combine":
            m.moe_combine_norm(self.s, self.d["y_perm"], self.d["gates"], self.d["slot_row"], self.get("y_add"), x, *tail)
        else:
            m.moe_block_norm_fwd(self.s, x, self.get("y"), *tail)
        return {n: t for n, t in o.items() if t is not None}

    def ref_fwd(self):
        c = self.c
        comb = (c["y_perm"], c["gates"], c["slot_row"], c.get("y_add")) if self.branch == "combine" else None
        return ref.norm_fwd(c["x"], y=c.get("y"), gate=c.get("gate"), w_post=c.get("w_post"), w_pre=c.get("w_pre"),
                            res_scale=self.scale, eps=EPS, combine=comb)

    def bwd(self, dv=True, inplace=False, ws=True, dy=None):
        """The backward at the forward's own stored v and rstd (fwd first)."""
        m, T, d, k = _m(), self.T, self.d_, self.k
        pre, post, br = "w_pre" in self.d, "w_post" in self.d, self.branch != "none"
        b = self.b = {}
        dvt = (self.d["dv"].clone() if inplace else self.d["dv"]) if dv else None
        b["dx"] = dvt if inplace else self.out("dx", T, d, dtype=self.dt)
        dy = self.branch == "y" or "y_add" in self.d if dy is None else dy
        b["dy"] = self.out("dy", T, d, dtype=self.dt) if dy else None
        b["dgate"] = self.out("dgate", T) if "gate" in self.d else None
        b["dw_post"] = self.out("dw_post", 1, d)[0] if post and ws else None
        b["dw_pre"] = self.out("dw_pre", 1, d)[0] if pre and ws else None
        v = self.o["v"] if br else self.d["x"]
        mid = (self.get("gate"), self.get("w_post"), self.get("w_pre"), self.o["rstd_post"], self.o["rstd_pre"],
               self.scale)
        if self.branch == "combine":
            b["dy_perm"], b["dgates"] = self.out("dy_perm", T * k, d, dtype=self.dt), self.out("dgates", T, k)
            m.moe_combine_norm_bwd(self.s, dvt, self.get("dxn"), v, self.d["y_perm"], self.d["gates"],
                                   self.d["slot_row"], self.get("y_add"), *mid, b["dx"], b["dy"], b["dy_perm"],
                                   b["dgates"], b["dgate"], b["dw_post"], b["dw_pre"], self.ws if ws else None)
        else:
            m.moe_block_norm_bwd(self.s, dvt, self.get("dxn"), v, self.get("y"), *mid, b["dx"], b["dy"], b["dgate"],
                                 b["dw_post"], b["dw_pre"], self.ws if ws else None)
        return {n: t for n, t in b.items() if t is not None}

    def ref_bwd(self, dv=True):
        c = self.c
        comb = (c["y_perm"], c["gates"], c["slot_row"], c.get("y_add")) if self.branch == "combine" else None
        stored = lambda n: None if self.o[n] is None else self.o[n].cpu()  # noqa: E731
        return ref.norm_bwd(dv=c["dv"] if dv else None, dxn=c.get("dxn"),
                            v=c["x"] if self.branch == "none" else stored("v"), y=c.get("y"), gate=c.get("gate"),
                            w_post=c.get("w_post"), w_pre=c.get("w_pre"), rstd_post=stored("rstd_post"),
                            rstd_pre=stored("rstd_pre"), res_scale=self.scale, combine=comb)

    def check(self, got, want, extra=0):
        for n, t in got.items():
            over_tokens = self.T if n in ("dw_post", "dw_pre") else 0
            _check(t, want[n].reshape(tuple(t.shape)), want["mag"][n].reshape(tuple(t.shape)), 128 + over_tokens, n)
        for n, buf in self.bufs.items():
            assert bool((buf[-self.GUARD:] == -3.0).all()), ("rows behind the last one", n)


FLAGS = [(True, True, True), (True, True, False), (True, False, True), (False, True, True), (False, False, False)]


@pytest.mark.parametrize("act", ["bf16", "f32"])
@pytest.mark.parametrize("T,d", [(1, 64), (1, 2048), (2, 192), (7, 512), (65, 576), (257, 1088), (33, 2048), (9, 2112),
                                 (40, 4096), (30, 5120), (21, 7168), (6, 8256), (5, 16384)])
def test_norm_widths(T, d, act):
    for branch in ("none", "y", "combine"):
        say(f"[gpu] norm T={T} d={d} {act} {branch}")
        n = Norm(T, d, act, branch, seed=d)
        n.check(n.fwd(), n.ref_fwd())
        n.check(n.bwd(), n.ref_bwd())


@pytest.mark.parametrize("branch", ["y", "combine"])
@pytest.mark.parametrize("post,pre,gated", FLAGS)
def test_norm_parts(branch, post, pre, gated):
    say(f"[gpu] norm parts {branch} post={post} pre={pre} gated={gated}")
    n = Norm(130, 320, "bf16", branch, post, pre, gated, k=3, add=True, seed=4)
    n.check(n.fwd(), n.ref_fwd())
    n.check(n.bwd(), n.ref_bwd())
    if pre:  # nothing but xn was used
        n.check(n.bwd(dv=False), n.ref_bwd(dv=False))


@pytest.mark.parametrize("k", [1, 2, 3, 4, 5, 8, 9, 32])
@pytest.mark.parametrize("d,act", [(256, "bf16"), (2048, "bf16"), (2048, "f32"), (5120, "bf16"), (7168, "bf16"),
                                   (16384, "bf16")])
def test_combine_norm_top_k(k, d, act):
    say(f"[gpu] combine norm k={k} d={d} {act}")
    n = Norm(37 if d < 4096 else 7, d, act, "combine", k=k, add=k % 2 == 1, seed=k)
    n.check(n.fwd(), n.ref_fwd())
    n.check(n.bwd(), n.ref_bwd())


@pytest.mark.parametrize("branch", ["none", "y", "combine"])
@pytest.mark.parametrize("T,d,k,act", [(9001, 64, 3, "bf16"), (2049, 128, 6, "bf16"), (5003, 192, 4, "f32"),
                                       (2500, 256, 9, "bf16"), (3001, 320, 2, "bf16"), (2048, 64, 5, "f32")])
def test_norm_many_rows(branch, T, d, k, act):
    """More rows than workgroups: several rows to every wave, narrow ones side by side in it."""
    say(f"[gpu] norm many rows {branch} T={T} d={d} k={k} {act}")
    n = Norm(T, d, act, branch, k=k, seed=6)
    n.check(n.fwd(), n.ref_fwd())
    n.check(n.bwd(), n.ref_bwd())


@pytest.mark.parametrize("branch", ["y", "combine"])
@pytest.mark.parametrize("T,k,post", [(64, 2, True), (64, 6, True), (2100, 3, True), (64, 2, False)])
def test_norm_closed_gates_drop_what_the_branch_holds(branch, T, k, post):
    n = Norm(T, 256, "bf16", branch, k=k, post=post, seed=3)
    shut = torch.nonzero(n.c["gate"] == 0)[:, 0]
    clean = {k: v.clone() for k, v in n.fwd().items()}
    cb = {k: v.clone() for k, v in n.bwd().items()}
    if branch == "y":
        n.d["y"][shut.cuda()] = float("nan")
    else:
        n.d["y_perm"][n.d["slot_row"][shut.cuda()].reshape(-1).long()] = float("inf")
    f = n.fwd()
    assert torch.equal(f["v"], clean["v"]) and torch.equal(f["xn"], clean["xn"])
    assert torch.equal(f["v"][shut.cuda()], n.d["x"][shut.cuda()])
    b = n.bwd()
    assert torch.equal(b["dx"], cb["dx"]) and (not post or torch.equal(b["dw_post"], cb["dw_post"]))
    if branch == "y":
        assert torch.equal(b["dy"], cb["dy"]) and not host(b["dy"][shut.cuda()]).any()
    else:
        assert torch.equal(b["dy_perm"], cb["dy_perm"]) and torch.equal(b["dgates"], cb["dgates"])
        assert not host(b["dgates"][shut.cuda()]).any()


def test_norm_rows_of_zeros():
    n = Norm(12, 128, "bf16", "y", gated=False, seed=2)
    for t in (n.c, n.d):
        t["x"][3] = 0
        t["y"][3] = t["y"][7] = 0
    n.check(n.fwd(), n.ref_fwd())
    assert float(n.o["rstd_post"][7]) == pytest.approx(EPS ** -0.5, rel=1e-6)
    n.check(n.bwd(), n.ref_bwd())


@pytest.mark.parametrize("branch", ["y", "combine"])
@pytest.mark.parametrize("d", [192, 4096])
def test_norm_in_place(branch, d):
    n = Norm(50, d, "bf16", branch, seed=8)
    apart = {k: v.clone() for k, v in n.fwd().items()}
    same = n.fwd(inplace=True)
    for k in apart:
        assert torch.equal(apart[k], same[k]), k
    apart = {k: v.clone() for k, v in n.bwd().items()}
    same = n.bwd(inplace=True)
    for k in apart:
        assert torch.equal(apart[k], same[k]), k


def test_norm_without_weight_gradients_needs_no_workspace():
    n = Norm(20, 256, "bf16", "y", seed=9)
    n.fwd()
    full = {k: v.clone() for k, v in n.bwd().items()}
    part = n.bwd(ws=False)
    assert all(torch.equal(full[k], part[k]) for k in part) and "dw_pre" not in part


def test_combine_norm_dy_is_optional():
    n = Norm(20, 256, "bf16", "combine", k=2, add=True, seed=9)
    n.fwd()
    full = {k: v.clone() for k, v in n.bwd().items()}
    part = n.bwd(dy=False)
    assert "dy" in full and "dy" not in part and all(torch.equal(full[k], part[k]) for k in part)


@pytest.mark.parametrize("branch", ["none", "y"])
def test_norm_of_no_rows(branch):
    m = _m()
    s = m.make_shape(0, 128, 64, 4, 2)
    e = lambda *n: torch.empty(*n, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    x, w, r = e(0, 128), torch.ones(128, dtype=torch.bfloat16, device="cuda"), torch.empty(0, device="cuda")
    y = e(0, 128) if branch == "y" else None
    dw, dw2 = torch.full((128,), 5.0, device="cuda"), torch.full((128,), 5.0, device="cuda")
    ws = torch.empty(m.moe_workspace_size(s), dtype=torch.uint8, device="cuda")
    post = w if branch == "y" else None
    m.moe_block_norm_fwd(s, x, y, None, post, w, 1.0, EPS, e(0, 128) if branch == "y" else None, e(0, 128), r, r)
    m.moe_block_norm_bwd(s, x, x, x, y, None, post, w, r, r, 1.0, e(0, 128), e(0, 128), None,
                         dw2 if branch == "y" else None, dw, ws)
    torch.cuda.synchronize()
    assert not host(dw).any() and (branch == "none" or not host(dw2).any())


def test_norm_offsets_past_32_bits():
    m = _m()
    T, d = 2 ** 20 + 5, 2048 + 64
    say(f"[gpu] norm T={T} d={d} (past 2^31 elements)")
    s = m.make_shape(T, d, 64, 1, 1)
    bf = dict(dtype=torch.bfloat16, device="cuda")
    x = torch.ones(T, d, **bf)
    x[-2:] = torch.randn(2, d, generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
    w = torch.full((d,), 2.0, **bf)
    xn, r = torch.empty(T, d, **bf), torch.empty(T, device="cuda")
    m.moe_block_norm_fwd(s, x, None, None, None, w, 1.0, EPS, None, xn, None, r)
    want = ref.norm_fwd(x[-2:].cpu(), w_pre=w.cpu(), eps=EPS)
    _check(xn[-2:], want["xn"], want["mag"]["xn"], 128, "xn")
    dx, dw = torch.empty(T, d, **bf), torch.empty(d, device="cuda")
    ws = torch.empty(m.moe_workspace_size(s), dtype=torch.uint8, device="cuda")
    m.moe_block_norm_bwd(s, None, x, x, None, None, None, w, None, r, 1.0, dx, None, None, None, dw, ws)
    bw = ref.norm_bwd(dxn=x[-2:].cpu(), v=x[-2:].cpu(), w_pre=w.cpu(), rstd_pre=r[-2:].cpu())
    _check(dx[-2:], bw["dx"], bw["mag"]["dx"], 128, "dx")
    # the rows of ones add (T - 2) * rstd, each off by a rounding
    one = float(r[0]) * (T - 2)
    rest = (host(x[-2:]).astype(np.float64) ** 2 * host(r[-2:]).astype(np.float64)[:, None]).sum(0)
    assert np.all(np.abs(host(dw) - (one + rest)) <= (T // 512 + 600) * F32 * (one + rest))


# ------------------------------------------------------------------ how a program runs them
def test_calls_repeat_bit_for_bit():
    for branch in ("none", "y", "combine"):
        n = Norm(700, 1088, "bf16", branch, k=4, seed=5)
        a = {k: v.clone() for k, v in {**n.fwd(), **n.bwd()}.items()}
        n.ws.fill_(17)
        again = {**n.fwd(), **n.bwd()}
        assert all(torch.equal(a[k], again[k]) for k in a)
    L, idx, gates, dgates = _balance_inputs(5000, 128, 4, 1)
    b = Balance(L, idx, gates, dgates).fwd().bwd()
    first = [t.clone() for t in (b.loss, b.prob, b.lse, b.counts, b.dlogits)]
    b.ws.fill_(3)
    b.fwd().bwd()
    assert all(torch.equal(x, y) for x, y in zip(first, (b.loss, b.prob, b.lse, b.counts, b.dlogits)))


def test_calls_on_a_side_stream_and_in_a_graph():
    """Captured on one stream and replayed between eager work that clobbers every output."""
    n = Norm(300, 576, "bf16", "combine", k=4, add=True, seed=12)
    L, idx, gates, dgates = _balance_inputs(300, 96, 4, 12)
    b = Balance(L, idx, gates, dgates)

    def step():
        o = {**n.fwd(), **n.bwd()}
        b.fwd().bwd()
        return {**o, "loss": b.loss, "prob": b.prob, "lse": b.lse, "counts": b.counts, "dlogits": b.dlogits}

    want = {k: v.clone() for k, v in step().items()}
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = step()
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(got[k], want[k]) for k in want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = step()
    torch.cuda.synchronize()
    for rep in range(3):
        for t in got.values():
            t.fill_(7)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        bad = [k for k in want if not torch.equal(got[k], want[k])]
        assert not bad, (rep, bad)


def test_binding_refuses_wrong_tensors():
    m = _m()
    s = m.make_shape(4, 64, 64, 4, 2)
    bf = dict(dtype=torch.bfloat16, device="cuda")
    x, xn, w, r = torch.zeros(4, 64, **bf), torch.zeros(4, 64, **bf), torch.ones(64, **bf), torch.zeros(4, device="cuda")

    def call(x=x, w=w, xn=xn, r=r):
        m.moe_block_norm_fwd(s, x, None, None, None, w, 1.0, EPS, None, xn, None, r)
    call()
    for change in (dict(x=x.float()), dict(x=x[:3]), dict(x=torch.zeros(4, 128, **bf)[:, ::2]), dict(w=w.cpu()),
                   dict(r=r.bfloat16()), dict(xn=torch.zeros(64, 4, **bf).t())):
        with pytest.raises(ValueError):
            call(**change)
    with pytest.raises(m.MoeError) as e:
        m.moe_block_norm_fwd(s, x, None, r, None, w, 1.0, EPS, None, xn, None, r)
    assert e.value.status == -1
