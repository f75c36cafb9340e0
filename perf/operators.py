"""What is measured of the operators that stand around the expert layer: the router's balance
loss (with z-loss and per-expert counts), the norms before and after a block with its gate and
residual scale, and the layer's combine fused with those norms, forward and backward.

    listed()              the measured cases
    draw(rng)             one more case of the same ranges
    prepare(case, seed)   inputs on the GPU, and the buffers a program keeps
    run(state)            one pass: plain torch (own = False) or the library's calls (own = True)
    work(case)            bytes and operations that a pass cannot do without
    exact(case, seed)     the same outputs from the definitions in 64 bits

Notation: T tokens, d width, E experts, k experts per token, R = T*k routed rows.

Balance (dir fwd / bwd).  Tokens left out by the mask count nowhere.  Over the N kept ones,
p = softmax(logits[t]), c_e = choices of expert e, P_e = mean of p_e:
    loss[0] = E / (k N) sum_e c_e P_e          loss[1] = mean of lse(logits[t])^2
    counts = [c_0 .. c_{E-1}, N]               lse[t] = -inf for a token left out
    dlogits[t, e] = p_e (g0 E / (k N^2) (c_e - sum p c) + 2 g1 lse / N) + gate gradient
The gate gradient, the derivative of the softmax over a token's k chosen scores, enters the same
pass: g_e (dg_e - sum_j g_j dg_j) at the chosen experts.

Norm.  r(z) = 1 / sqrt(mean(z^2) + eps), a = residual scale, g = the token's gate:
    v = x + a g (y r(y) w_post)                xn = v r(v) w_pre
with y (and w_post, gate) left out for a norm before the block only.  A gate of zero drops the
branch.  Backward, with D the gradient of v from both of its uses:
    D = dv + r_v (w_pre dxn - vh mean(vh w_pre dxn)),  vh = v r_v;  dx = D
    dy = a g r_y (w_post D - yh mean(yh w_post D)),    yh = y r_y
    dgate = a sum(D w_post yh)   dw_post = a sum_t g D yh   dw_pre = sum_t dxn vh

Combine.  The same with y = y_add + sum_j gates[t, j] y_perm[slot_row[t, j]]; backward also
    dy_perm[slot_row[t, j]] = gates[t, j] dy[t]        dgates[t, j] = <dy[t], y_perm[slot_row[t, j]]>
"""
import math

import torch

own = False

EPS = 1e-6
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------ cases
def _balance(name, dir, T, E, k, mask):
    return dict(name=name, op="balance", dir=dir, T=T, E=E, k=k, mask=mask)


def _norm(name, dir, T, d, act, post, pre, gate):
    return dict(name=name, op="norm", dir=dir, T=T, d=d, act=act, post=post, pre=pre, gate=gate)


def _combine(name, dir, T, d, E, k, act, add, pre, gate):
    return dict(name=name, op="combine", dir=dir, T=T, d=d, E=E, k=k, act=act, add=add, pre=pre, gate=gate)


def listed():
    return [
        # the fp32 unit configuration's router: a call that is all latency
        _balance("balance_fwd_t256_e8", "fwd", 256, 8, 2, False),
        # one micro-batch of the 128-expert training configuration
        _balance("balance_fwd_t8192_e128", "fwd", 8192, 128, 4, False),
        _balance("balance_bwd_t8192_e128", "bwd", 8192, 128, 4, False),
        # a long padded batch with an expert count that fills no power of two
        _balance("balance_bwd_t65521_e96_pad", "bwd", 65521, 96, 6, True),
        # serving: one token enters a block
        _norm("norm_pre_fwd_t1_d2048", "fwd", 1, 2048, "bf16", False, True, False),
        # training: a block's end and the next block's start in one pass
        _norm("norm_fwd_t8192_d2048", "fwd", 8192, 2048, "bf16", True, True, True),
        _norm("norm_bwd_t8192_d2048", "bwd", 8192, 2048, "bf16", True, True, True),
        # fp32 training with an odd token count and a width off the powers of two
        _norm("norm_bwd_t1531_d1088_f32", "bwd", 1531, 1088, "f32", True, True, False),
        # the norm before the wide MXFP8 configuration's block
        _norm("norm_pre_bwd_t16384_d4096", "bwd", 16384, 4096, "bf16", False, True, False),
        # serving: a decode batch leaves the experts
        _combine("combine_fwd_t32_d2048", "fwd", 32, 2048, 128, 4, "bf16", False, True, False),
        # training: the experts' rows to the residual stream, with a shared expert
        _combine("combine_fwd_t8192_d2048", "fwd", 8192, 2048, 128, 4, "bf16", True, True, False),
        _combine("combine_bwd_t16384_d4096", "bwd", 16384, 4096, 32, 4, "bf16", False, True, True),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["balance", "norm", "combine"])
    c = dict(op=op, dir=rng.choice(["fwd", "bwd"]), T=1024)
    flags = [rng.random() < 0.5 for _ in range(3)]
    if op == "balance":
        c["E"] = _log_int(rng, 2, 1024)
        c.update(k=rng.randint(1, min(8, c["E"])), mask=flags[0])
        most = 55e6
    else:
        c.update(d=64 * _log_int(rng, 1, 128), act=rng.choice(["bf16", "bf16", "f32"]), pre=flags[0])
        if op == "norm":
            c.update(post=flags[1] or not flags[0], gate=flags[2] and (flags[1] or not flags[0]))
            most = 5e8
        else:
            c["E"] = _log_int(rng, 4, 128)
            c.update(k=rng.randint(1, min(8, c["E"])), add=flags[1], gate=flags[2])
            most = 1.6e9
    # from one token to what the largest listed case of the operator moves
    c["T"] = _log_int(rng, 1, min(131072, int(most * 1024 / work(c)["bytes"])))
    return c


# ------------------------------------------------------------------ inputs
def _rand(gen, *shape):
    return torch.randn(*shape, generator=gen, device="cuda")


def _routing(gen, T, E, k):
    """Scores of a skewed router, its k best experts, their gates and the packed row of each choice."""
    logits = 1.5 * _rand(gen, T, E) + _rand(gen, 1, E)
    top, idx = torch.sort(logits, dim=1, descending=True, stable=True)
    top, idx = top[:, :k].contiguous(), idx[:, :k].to(torch.int32).contiguous()
    gates = torch.softmax(top, dim=1)
    order = torch.argsort(idx.reshape(-1), stable=True)
    slot = torch.empty(T * k, dtype=torch.int32, device="cuda")
    slot[order] = torch.arange(T * k, dtype=torch.int32, device="cuda")
    return logits, idx, gates, slot.reshape(T, k)


def _rstd64(z):
    return torch.rsqrt(z.double().square().mean(dim=1) + EPS)


def _inputs(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    T = case["T"]
    s = {}
    if case["op"] == "balance":
        E, k = case["E"], case["k"]
        s["logits"], s["topk_idx"], s["gates"], _ = _routing(gen, T, E, k)
        # padding: about a sixth of the tokens, whose scores are whatever the buffer held
        s["mask"] = None
        if case["mask"]:
            keep = torch.rand(T, generator=gen, device="cuda") < 0.84
            s["mask"] = keep.to(torch.uint8)
            s["logits"] = torch.where(keep[:, None], s["logits"], torch.full_like(s["logits"], float("nan")))
        if case["dir"] == "bwd":
            keep = torch.ones(T, dtype=torch.bool, device="cuda") if s["mask"] is None else s["mask"] != 0
            lse = torch.logsumexp(s["logits"].double(), dim=1).float()
            s["lse"] = torch.where(keep, lse, torch.full_like(lse, -math.inf))
            chosen = s["topk_idx"][keep].reshape(-1).long()
            s["counts"] = torch.cat([torch.bincount(chosen, minlength=E), keep.sum()[None]]).to(torch.int32)
            s["dloss"] = torch.tensor([1e-2, 1e-3], device="cuda")
            s["dgates"] = 1e-3 * _rand(gen, T, k)
        return s
    d, dt = case["d"], DTYPES[case["act"]]
    channel = torch.exp(0.5 * _rand(gen, 1, d))  # a residual stream has loud channels
    x = (_rand(gen, T, d) * channel).to(dt)
    s["w_pre"] = (1 + 0.1 * _rand(gen, d)).to(dt) if case["pre"] else None
    branch = case["op"] == "combine" or case["post"]
    s["w_post"] = (1 + 0.1 * _rand(gen, d)).to(dt) if branch else None
    s["gate"] = None
    if case["gate"]:  # per-token gates, some tokens skip the block
        s["gate"] = torch.sigmoid(_rand(gen, T)) * (torch.rand(T, generator=gen, device="cuda") < 0.9)
    s["res_scale"] = 0.5 if branch else 1.0
    if case["op"] == "combine":
        k = case["k"]
        _, _, s["gates"], s["slot_row"] = _routing(gen, T, case["E"], k)
        s["y_perm"] = (0.3 * _rand(gen, T * k, d)).to(dt)
        s["y_add"] = (0.2 * _rand(gen, T, d)).to(dt) if case["add"] else None
    else:
        s["y"] = (0.3 * _rand(gen, T, d)).to(dt) if branch else None
    if case["dir"] == "fwd":
        s["x"] = x
        return s
    s["v"] = x  # the stream behind the residual sum, as the forward stored it
    s["dv"] = (1e-2 * _rand(gen, T, d)).to(dt)
    s["dxn"] = (1e-2 * _rand(gen, T, d)).to(dt) if case["pre"] else None
    s["rstd_pre"] = _rstd64(x).float() if case["pre"] else None
    s["rstd_post"] = None
    if branch:
        s["rstd_post"] = _rstd64(_branch(s, torch.float64)).float()
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    s["case"] = case
    if own:
        import mixture_experts_layer_logits_amd as m
        s["m"] = m
        T, d, E, k = case["T"], case.get("d", 64), case.get("E", 1), case.get("k", 1)
        act = m.MOE_F32 if case.get("act") == "f32" else m.MOE_BF16
        dt = DTYPES.get(case.get("act"), torch.float32)
        e = lambda *n, dtype=torch.float32: torch.empty(*n, dtype=dtype, device="cuda")  # noqa: E731
        s["shape"] = m.make_shape(T, d, 64, E, k, act)
        s["ws"] = e(m.moe_workspace_size(s["shape"]), dtype=torch.uint8)
        if case["op"] == "balance":
            if case["dir"] == "fwd":
                s["out"] = dict(lse=e(T), counts=e(E + 1, dtype=torch.int32), prob_mean=e(E), loss=e(2))
            else:
                s["out"] = dict(dlogits=e(T, E))
            return s
        pre, post = case["pre"], s["w_post"] is not None
        if case["dir"] == "fwd":
            s["out"] = dict(v=e(T, d, dtype=dt) if post else None, xn=e(T, d, dtype=dt) if pre else None,
                            rstd_post=e(T) if post else None, rstd_pre=e(T) if pre else None)
        else:
            s["out"] = dict(dx=e(T, d, dtype=dt), dgate=e(T) if s["gate"] is not None else None,
                            dw_post=e(d) if post else None, dw_pre=e(d) if pre else None)
            if case["op"] == "combine":
                s["out"].update(dy=e(T, d, dtype=dt) if case["add"] else None, dy_perm=e(T * k, d, dtype=dt),
                                dgates=e(T, k))
            else:
                s["out"].update(dy=e(T, d, dtype=dt) if post else None)
    return s


# ------------------------------------------------------------------ the library's calls
def _run_own(s):
    m, sh, o, c = s["m"], s["shape"], s["out"], s["case"]
    if c["op"] == "balance":
        if c["dir"] == "fwd":
            m.moe_balance_fwd(sh, s["logits"], s["topk_idx"], s["mask"], o["lse"], o["counts"], o["prob_mean"],
                              o["loss"], s["ws"])
        else:
            m.moe_balance_bwd(sh, s["logits"], s["lse"], s["counts"], s["dloss"], s["dgates"], s["gates"],
                              s["topk_idx"], o["dlogits"])
    elif c["op"] == "norm":
        if c["dir"] == "fwd":
            m.moe_block_norm_fwd(sh, s["x"], s["y"], s["gate"], s["w_post"], s["w_pre"], s["res_scale"], EPS, o["v"],
                                 o["xn"], o["rstd_post"], o["rstd_pre"])
        else:
            m.moe_block_norm_bwd(sh, s["dv"], s["dxn"], s["v"], s["y"], s["gate"], s["w_post"], s["w_pre"],
                                 s["rstd_post"], s["rstd_pre"], s["res_scale"], o["dx"], o["dy"], o["dgate"],
                                 o["dw_post"], o["dw_pre"], s["ws"])
    elif c["dir"] == "fwd":
        m.moe_combine_norm(sh, s["y_perm"], s["gates"], s["slot_row"], s["y_add"], s["x"], s["gate"], s["w_post"],
                           s["w_pre"], s["res_scale"], EPS, o["v"], o["xn"], o["rstd_post"], o["rstd_pre"])
    else:
        m.moe_combine_norm_bwd(sh, s["dv"], s["dxn"], s["v"], s["y_perm"], s["gates"], s["slot_row"], s["y_add"],
                               s["gate"], s["w_post"], s["w_pre"], s["rstd_post"], s["rstd_pre"], s["res_scale"],
                               o["dx"], o["dy"], o["dy_perm"], o["dgates"], o["dgate"], o["dw_post"], o["dw_pre"],
                               s["ws"])
    return {n: t for n, t in o.items() if t is not None}


# ------------------------------------------------------------------ the plain forms
def _branch(s, dtype):
    """The block's output y[t] before its norm."""
    if "y_perm" not in s:
        return s["y"].to(dtype)
    T, k = s["slot_row"].shape
    rows = s["y_perm"].to(dtype)
    y = torch.zeros(T, rows.shape[1], dtype=dtype, device=rows.device) if s["y_add"] is None else s["y_add"].to(dtype)
    for j in range(k):
        y = y + s["gates"][:, j:j + 1].to(dtype) * rows[s["slot_row"][:, j].long()]
    return y


def _plain_balance(s):
    logits, idx, E, k = s["logits"], s["topk_idx"].long(), s["case"]["E"], s["case"]["k"]
    if s["case"]["dir"] == "fwd":
        keep = torch.ones(logits.shape[0], dtype=torch.bool, device="cuda") if s["mask"] is None else s["mask"] != 0
        z = torch.where(keep[:, None], logits, torch.zeros_like(logits))
        top = z.max(dim=1, keepdim=True).values
        ex = torch.exp(z - top)
        den = ex.sum(dim=1, keepdim=True)
        p = torch.where(keep[:, None], ex / den, torch.zeros_like(ex))
        lse = (top + torch.log(den))[:, 0]
        c = torch.zeros(E, dtype=torch.int64, device="cuda")
        c.scatter_add_(0, idx.reshape(-1), keep[:, None].expand(-1, k).reshape(-1).long())
        n = keep.sum()
        nf = torch.clamp(n, min=1).double()
        mean = p.double().sum(dim=0) / nf
        bal = (c.double() * mean).sum() * E / (k * nf)
        zl = torch.where(keep, lse, torch.zeros_like(lse)).double().square().sum() / nf
        return dict(lse=torch.where(keep, lse, torch.full_like(lse, -math.inf)),
                    counts=torch.cat([c, n[None]]).to(torch.int32), prob_mean=mean.float(),
                    loss=torch.stack([bal, zl]).float())
    keep = s["lse"] > -math.inf
    lse = torch.where(keep, s["lse"], torch.zeros_like(s["lse"]))[:, None]
    z = torch.where(keep[:, None], logits, torch.zeros_like(logits))
    p = torch.where(keep[:, None], torch.exp(z - lse), torch.zeros_like(z))
    n = torch.clamp(s["counts"][E], min=1).float()
    frac = s["counts"][:E].float() / n
    inner = (p * frac).sum(dim=1, keepdim=True)
    out = p * (s["dloss"][0] * (E / k) / n * (frac - inner) + s["dloss"][1] * 2 * lse / n)
    g, dg = s["gates"], s["dgates"]
    gate_grad = g * (dg - (g * dg).sum(dim=1, keepdim=True))
    return dict(dlogits=out.scatter_add(1, idx, gate_grad))


def _rstd(z):
    return torch.rsqrt((z * z).mean(dim=1, keepdim=True) + EPS)


def _plain_norm(s):
    c = s["case"]
    dt = DTYPES[c["act"]]
    f = torch.float32
    wq = None if s["w_post"] is None else s["w_post"].to(f)
    wp = None if s["w_pre"] is None else s["w_pre"].to(f)
    a = s["res_scale"]
    g = None if s["gate"] is None else s["gate"][:, None]
    out = {}
    if c["dir"] == "fwd":
        v = s["x"].to(f)
        if wq is not None:
            y = _branch(s, f)
            rq = _rstd(y)
            b = a * y * rq * wq
            v = v + (b if g is None else torch.where(g == 0, torch.zeros_like(b), g * b))
            out["v"], out["rstd_post"] = v.to(dt), rq[:, 0]
        if wp is not None:
            rp = _rstd(v)
            out["xn"], out["rstd_pre"] = (v * rp * wp).to(dt), rp[:, 0]
        return out
    D = s["dv"].to(f)
    if wp is not None:
        rp = s["rstd_pre"][:, None]
        vh = s["v"].to(f) * rp
        dxn = s["dxn"].to(f)
        wd = wp * dxn
        D = D + rp * (wd - vh * (vh * wd).mean(dim=1, keepdim=True))
        out["dw_pre"] = (dxn * vh).sum(dim=0)
    out["dx"] = D.to(dt)
    if wq is not None:
        rq = s["rstd_post"][:, None]
        yh = _branch(s, f) * rq
        wd = wq * D
        dy = a * rq * (wd - yh * (yh * wd).mean(dim=1, keepdim=True))
        gd = a * D * yh
        if g is not None:
            out["dgate"] = a * (wd * yh).sum(dim=1)
            dy = torch.where(g == 0, torch.zeros_like(dy), g * dy)
            gd = torch.where(g == 0, torch.zeros_like(gd), g * gd)
        out["dw_post"] = gd.sum(dim=0)
        if c["op"] == "norm" or s["y_add"] is not None:
            out["dy"] = dy.to(dt)
        if c["op"] == "combine":
            T, k = s["slot_row"].shape
            out["dy_perm"] = torch.empty(T * k, c["d"], dtype=dt, device="cuda")
            out["dgates"] = torch.empty(T, k, device="cuda")
            for j in range(k):
                r = s["slot_row"][:, j].long()
                out["dy_perm"][r] = (s["gates"][:, j:j + 1] * dy).to(dt)
                out["dgates"][:, j] = (dy * s["y_perm"][r].to(f)).sum(dim=1)
    return out


_ORDER = ("lse", "counts", "prob_mean", "loss", "dlogits", "v", "xn", "rstd_post", "rstd_pre", "dx", "dy", "dy_perm",
          "dgates", "dgate", "dw_post", "dw_pre")


def run(state):
    if own:
        out = _run_own(state)
    else:
        out = _plain_balance(state) if state["case"]["op"] == "balance" else _plain_norm(state)
    return {n: out[n] for n in _ORDER if n in out}


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    T = case["T"]
    if case["op"] == "balance":
        E, k = case["E"], case["k"]
        if case["dir"] == "fwd":
            b = 4 * T * E + 4 * T * k + 4 * T + (T if case["mask"] else 0) + 8 * E
            return {"bytes": b, "flops": 6 * T * E}
        return {"bytes": 8 * T * E + 4 * T + 12 * T * k + 4 * E, "flops": 8 * T * E}
    d, eb = case["d"], DTYPES[case["act"]].itemsize
    post, pre = case["op"] == "combine" or case["post"], case["pre"]
    row = T * d * eb
    rows = 0.0
    flops = 0
    if case["op"] == "combine":
        k = case["k"]
        rows += k + case["add"] + (k + case["add"] if case["dir"] == "bwd" else 0)  # y_perm, y_add; dy_perm, dy
        flops += (2 if case["dir"] == "fwd" else 5) * k * T * d
    elif post:
        rows += 1 + (case["dir"] == "bwd")  # y; dy
    if case["dir"] == "fwd":
        rows += 1 + post + pre  # x; v, xn
        flops += (6 * post + 5 * pre) * T * d
    else:
        rows += 2 + 2 * pre  # dv, dx; v, dxn
        flops += (12 * post + 10 * pre) * T * d
    small = 4 * T * (post + pre + case["gate"] * (2 if case["dir"] == "bwd" else 1))
    if case["op"] == "combine":
        small += T * case["k"] * (8 if case["dir"] == "fwd" else 12)
    small += d * (post + pre) * (eb + (4 if case["dir"] == "bwd" else 0))
    return {"bytes": int(rows * row + small), "flops": int(flops)}


# ------------------------------------------------------------------ 64-bit definitions
def exact(case, seed):
    s = _inputs(case, seed)
    return _exact_balance(case, s) if case["op"] == "balance" else _exact_norm(case, s)


def _exact_balance(case, s):
    E, k, T = case["E"], case["k"], case["T"]
    logits = s["logits"].double()
    if case["dir"] == "fwd":
        kept = torch.arange(T, device="cuda") if s["mask"] is None else torch.nonzero(s["mask"])[:, 0]
        n = max(1, kept.numel())
        lse = torch.full((T,), -math.inf, dtype=torch.float64, device="cuda")
        rows = logits[kept]
        lse[kept] = torch.logsumexp(rows, dim=1)
        prob = torch.softmax(rows, dim=1).sum(dim=0) / n
        c = torch.bincount(s["topk_idx"][kept].reshape(-1).long(), minlength=E)
        loss = torch.stack([E / (k * n) * torch.dot(c.double(), prob), (lse[kept] ** 2).sum() / n])
        counts = torch.cat([c, torch.tensor([kept.numel()], device="cuda")]).to(torch.int32)
        return dict(lse=lse, counts=counts, prob_mean=prob, loss=loss)
    kept = torch.nonzero(s["lse"] > -math.inf)[:, 0]
    n = max(1, int(s["counts"][E]))
    lse = s["lse"][kept].double().unsqueeze(1)
    p = torch.exp(logits[kept] - lse)
    share = s["counts"][:E].double()
    gb, gz = s["dloss"].double()
    out = torch.zeros(T, E, dtype=torch.float64, device="cuda")
    out[kept] = gb * E / (k * n * n) * p * (share - p @ share.unsqueeze(1)) + gz * 2 / n * lse * p
    g, dg = s["gates"].double(), s["dgates"].double()
    rows = torch.arange(T, device="cuda")
    mean = (g * dg).sum(1)
    for j in range(k):
        out[rows, s["topk_idx"][:, j].long()] += g[:, j] * (dg[:, j] - mean)
    return dict(dlogits=out)


def _exact_norm(case, s):
    f64 = lambda n: None if s.get(n) is None else s[n].double()  # noqa: E731
    d, T = case["d"], case["T"]
    wq, wp, scale = f64("w_post"), f64("w_pre"), s["res_scale"]
    gate = torch.ones(T, dtype=torch.float64, device="cuda") if s["gate"] is None else s["gate"].double()
    y = None
    if case["op"] == "combine":
        w = s["gates"].double()
        y = torch.zeros(T, d, dtype=torch.float64, device="cuda")
        for j in range(case["k"]):
            y.addcmul_(s["y_perm"].index_select(0, s["slot_row"][:, j].long()).double(), w[:, j, None])
        if s["y_add"] is not None:
            y += s["y_add"].double()
    elif wq is not None:
        y = s["y"].double()
    res = {}
    if case["dir"] == "fwd":
        v = s["x"].double()
        if y is not None:
            rq = 1.0 / torch.sqrt(y.pow(2).sum(1) / d + EPS)
            v = v + (scale * gate * rq).unsqueeze(1) * y * wq
            res.update(v=v, rstd_post=rq)
        if wp is not None:
            rp = 1.0 / torch.sqrt(v.pow(2).sum(1) / d + EPS)
            res.update(xn=v * wp * rp.unsqueeze(1), rstd_pre=rp)
        return {n: res[n] for n in _ORDER if n in res}
    D = f64("dv")
    if wp is not None:
        rp, v, dxn = f64("rstd_pre").unsqueeze(1), f64("v"), f64("dxn")
        u = dxn * wp
        D = D + rp * u - rp ** 3 * v * ((u * v).sum(1, keepdim=True) / d)
        res["dw_pre"] = torch.matmul((rp[:, 0]).unsqueeze(0), dxn * v)[0]
    res["dx"] = D
    if y is not None:
        rq = f64("rstd_post").unsqueeze(1)
        u = D * wq
        inner = (u * y).sum(1, keepdim=True)
        dy = (scale * gate).unsqueeze(1) * (rq * u - rq ** 3 * y * (inner / d))
        if s["gate"] is not None:
            res["dgate"] = scale * (rq * inner)[:, 0]
        res["dw_post"] = torch.matmul((scale * gate * rq[:, 0]).unsqueeze(0), D * y)[0]
        if case["op"] == "norm" or s["y_add"] is not None:
            res["dy"] = dy
        if case["op"] == "combine":
            rows, dg = torch.empty(T * case["k"], d, dtype=torch.float64, device="cuda"), []
            for j in range(case["k"]):
                at = s["slot_row"][:, j].long()
                rows.index_copy_(0, at, dy * s["gates"][:, j, None].double())
                dg.append((s["y_perm"].index_select(0, at).double() * dy).sum(1))
            res["dy_perm"], res["dgates"] = rows, torch.stack(dg, dim=1)
    return {n: res[n] for n in _ORDER if n in res}
