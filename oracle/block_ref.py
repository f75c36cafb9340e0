"""CPU oracle for the operators around the expert layer -- TEST INFRASTRUCTURE ONLY.

The balance loss with its gradient, and the norms before and after a block with gate and
residual scale, written out as their plain definitions in NumPy float64.  Like ``moe_ref``
it shares no code with the product path.

Every function also returns, under ``mag``, the sum of the absolute values of the terms of
each output (products of magnitudes, sums of magnitudes, with the saved rstd as given): a
float computation of the same terms is off by at most a count of roundings times 2^-24 times
that, which is what the GPU tests' tolerances are made of.
"""
from __future__ import annotations

import numpy as np

from .moe_ref import f64

__all__ = ["balance_fwd", "balance_bwd", "norm_fwd", "norm_bwd"]


# ------------------------------------------------------------------ balance loss
def _kept(L, mask):
    with np.errstate(invalid="ignore"):
        some = ~(np.isneginf(L).all(axis=1))
    return some if mask is None else some & (np.asarray(mask) != 0)


def balance_fwd(logits, topk_idx, mask=None):
    """counts [E + 1] (the last: kept tokens), prob_mean [E], lse [T], loss [2]."""
    L, idx = f64(logits), np.asarray(topk_idx)
    T, E = L.shape
    k = idx.shape[1]
    keep = _kept(L, mask)
    n = int(keep.sum())
    lse = np.full(T, -np.inf)
    counts = np.zeros(E + 1, dtype=np.int64)
    prob = np.zeros(E)
    z = 0.0
    for t in np.nonzero(keep)[0]:
        top = L[t].max()
        e = np.exp(L[t] - top)
        lse[t] = top + np.log(e.sum())
        prob += e / e.sum()
        z += lse[t] ** 2
        for j in range(k):
            counts[min(max(int(idx[t, j]), 0), E - 1)] += 1
    counts[E] = n
    if n == 0:
        return dict(counts=counts, prob_mean=prob, lse=lse, loss=np.zeros(2))
    prob /= n
    return dict(counts=counts, prob_mean=prob, lse=lse, loss=np.array([E / (k * n) * (counts[:E] @ prob), z / n]))


def balance_bwd(logits, lse, counts, dloss, topk=None):
    """dlogits of dloss . loss, plus the gates' gradient when topk = (topk_idx, gates, dgates)
    is given; k comes from topk or from counts."""
    L, lse, c = f64(logits), f64(lse), np.asarray(counts, dtype=np.float64)
    T, E = L.shape
    n = c[E]
    g0, g1 = f64(dloss)
    out, mag = np.zeros((T, E)), np.zeros((T, E))
    if n > 0:
        k = c[:E].sum() / n
        for t in range(T):
            if np.isneginf(lse[t]):
                continue
            p = np.exp(L[t] - lse[t])
            bal, zl = g0 * E / (k * n) / n, g1 * 2 * lse[t] / n
            out[t] = p * (bal * (c[:E] - p @ c[:E]) + zl)
            mag[t] = p * (abs(bal) * (c[:E] + p @ c[:E]) + abs(zl))
    if topk is not None:
        idx, g, dg = np.asarray(topk[0]), f64(topk[1]), f64(topk[2])
        for t in range(T):
            for j in range(idx.shape[1]):
                out[t, idx[t, j]] += g[t, j] * (dg[t, j] - g[t] @ dg[t])
                mag[t, idx[t, j]] += abs(g[t, j]) * (abs(dg[t, j]) + np.abs(g[t]) @ np.abs(dg[t]))
    return dict(dlogits=out, mag=dict(dlogits=mag))


# ------------------------------------------------------------------ block norms
def _combine(y_perm, gates, slot_row, y_add):
    rows, g = f64(y_perm), f64(gates)
    y = np.zeros((g.shape[0], rows.shape[1])) if y_add is None else f64(y_add).copy()
    m = np.abs(y)
    for j in range(g.shape[1]):
        r = rows[np.asarray(slot_row)[:, j]]
        y += g[:, j:j + 1] * r
        m += np.abs(g[:, j:j + 1] * r)
    return y, m


def norm_fwd(x, y=None, gate=None, w_post=None, w_pre=None, res_scale=1.0, eps=1e-6, combine=None):
    """combine = (y_perm, gates, slot_row, y_add or None) in place of y."""
    v = f64(x).copy()
    mv = np.abs(v)
    out, mag = {}, {}
    if combine is not None or y is not None:
        y, my = _combine(*combine) if combine is not None else (f64(y), np.abs(f64(y)))
        b, mb = y, my
        if w_post is not None:
            r = 1 / np.sqrt((y ** 2).mean(axis=1) + eps)
            out["rstd_post"], mag["rstd_post"] = r, r ** 3 * (my ** 2).mean(axis=1) + r
            b = y * r[:, None] * f64(w_post)
            mb = my * mag["rstd_post"][:, None] * np.abs(f64(w_post))
        g = np.ones(v.shape[0]) if gate is None else f64(gate)
        shut = (g == 0)[:, None]
        v += np.where(shut, 0.0, res_scale * g[:, None] * b)
        mv += np.where(shut, 0.0, np.abs(res_scale * g[:, None]) * mb)
        out["v"], mag["v"] = v, mv
    if w_pre is not None:
        r = 1 / np.sqrt((v ** 2).mean(axis=1) + eps)
        out["rstd_pre"], mag["rstd_pre"] = r, r ** 3 * (mv ** 2).mean(axis=1) + r
        out["xn"] = v * r[:, None] * f64(w_pre)
        mag["xn"] = mv * mag["rstd_pre"][:, None] * np.abs(f64(w_pre))
    out["mag"] = mag
    return out


def norm_bwd(dv=None, dxn=None, v=None, y=None, gate=None, w_post=None, w_pre=None, rstd_post=None, rstd_pre=None,
             res_scale=1.0, combine=None):
    some = dv if dv is not None else dxn
    D = np.zeros(tuple(some.shape)) if dv is None else f64(dv).copy()
    mD = np.abs(D)
    out, mag = {}, {}
    if w_pre is not None:
        r = f64(rstd_pre)[:, None]
        vh, dx = f64(v) * r, f64(dxn)
        u = f64(w_pre) * dx
        D = D + r * (u - vh * (vh * u).mean(axis=1, keepdims=True))
        mD = mD + r * (np.abs(u) + np.abs(vh) * np.abs(vh * u).mean(axis=1, keepdims=True))
        out["dw_pre"], mag["dw_pre"] = (dx * vh).sum(axis=0), np.abs(dx * vh).sum(axis=0)
    out["dx"], mag["dx"] = D, mD
    if combine is None and y is None:
        out["mag"] = mag
        return out
    y, my = _combine(*combine) if combine is not None else (f64(y), np.abs(f64(y)))
    g = np.ones((D.shape[0], 1)) if gate is None else f64(gate)[:, None]
    shut = g == 0
    if w_post is not None:
        r = f64(rstd_post)[:, None]
        yh, mh, u, mu = y * r, my * r, f64(w_post) * D, np.abs(f64(w_post)) * mD
        dy = res_scale * g * r * (u - yh * (yh * u).mean(axis=1, keepdims=True))
        mdy = np.abs(res_scale * g) * r * (mu + mh * (mh * mu).mean(axis=1, keepdims=True))
        dgate, mdgate = res_scale * (u * yh).sum(axis=1), abs(res_scale) * (mu * mh).sum(axis=1)
        out["dw_post"] = np.where(shut, 0.0, res_scale * g * D * yh).sum(axis=0)
        mag["dw_post"] = np.where(shut, 0.0, np.abs(res_scale * g) * mD * mh).sum(axis=0)
    else:
        dy, mdy = res_scale * g * D, np.abs(res_scale * g) * mD
        dgate, mdgate = res_scale * (D * y).sum(axis=1), abs(res_scale) * (mD * my).sum(axis=1)
    dy, mdy = np.where(shut, 0.0, dy), np.where(shut, 0.0, mdy)
    out["dy"], mag["dy"] = dy, mdy
    if gate is not None:
        out["dgate"], mag["dgate"] = dgate, mdgate
    if combine is not None:
        rows, gk, slot = f64(combine[0]), f64(combine[1]), np.asarray(combine[2])
        out["dy_perm"], mag["dy_perm"] = np.zeros_like(rows), np.zeros_like(rows)
        out["dgates"], mag["dgates"] = np.zeros(gk.shape), np.zeros(gk.shape)
        for j in range(gk.shape[1]):
            out["dy_perm"][slot[:, j]] = gk[:, j:j + 1] * dy
            mag["dy_perm"][slot[:, j]] = np.abs(gk[:, j:j + 1]) * mdy
            out["dgates"][:, j] = (dy * rows[slot[:, j]]).sum(axis=1)
            mag["dgates"][:, j] = (mdy * np.abs(rows[slot[:, j]])).sum(axis=1)
    out["mag"] = mag
    return out
