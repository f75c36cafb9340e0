"""fp64 reference of the expert layer in few bits: MXFP4 rows (4-bit weights), MXINT8 rows (8-bit
activation checkpoints) and the products and gradients that use them.  Blocks are 32 consecutive
elements of a row; plain NumPy, written from the definitions in include/moe.h."""
import numpy as np

BLOCK = 32
FP4 = np.array([0, .5, 1, 1.5, 2, 3, 4, 6], dtype=np.float64)


def _blocks(v):
    v = np.asarray(v, dtype=np.float64)
    return v.reshape(*v.shape[:-1], v.shape[-1] // BLOCK, BLOCK)


def _exponent(amax, top, low):
    """Smallest s >= low with amax <= top 2^s (low for a block of zeros)."""
    s = np.full(amax.shape, low, dtype=np.int64)
    pos = amax > 0
    s[pos] = np.ceil(np.log2(amax[pos] / top)).astype(np.int64)
    s = np.where(pos & (amax > top * np.exp2(s)), s + 1, s)      # a logarithm rounded across the border
    s = np.where(pos & (amax <= top * np.exp2(s - 1)), s - 1, s)
    return np.maximum(s, low)


def mx4_quantize(v):
    """(codes uint8 [.., K/2], scale bytes uint8 [.., K/32])"""
    b = _blocks(v)
    bad = ~np.isfinite(b).all(axis=-1)
    b = np.where(bad[..., None], 0.0, b)
    s = _exponent(np.abs(b).max(axis=-1), 6.0, -126)
    u = np.abs(b) / np.exp2(s)[..., None]
    d = np.abs(u[..., None] - FP4)
    near = d == d.min(axis=-1, keepdims=True)
    even = near & (np.arange(8) % 2 == 0)
    mag = np.where(even.any(axis=-1), even.argmax(axis=-1), near.argmax(axis=-1))
    code = (mag | (np.signbit(b) << 3)).astype(np.uint8)
    code[bad] = 0
    code = code.reshape(*np.shape(v)[:-1], -1, 2)
    return code[..., 0] | (code[..., 1] << 4), np.where(bad, 255, s + 127).astype(np.uint8)


def mx4_values(q, s):
    nib = np.stack([q & 15, q >> 4], axis=-1)
    v = np.where(nib >= 8, -1.0, 1.0) * FP4[nib & 7]
    f = np.where(s == 255, np.nan, np.exp2(s.astype(np.float64) - 127))
    return (v.reshape(*s.shape, BLOCK) * f[..., None]).reshape(*q.shape[:-1], -1)


def ck8_pack(v):
    """(codes int8 [.., K], scale bytes uint8 [.., K/32])"""
    b = _blocks(v)
    bad = ~np.isfinite(b).all(axis=-1)
    b = np.where(bad[..., None], 0.0, b)
    s = np.minimum(_exponent(np.abs(b).max(axis=-1), 127 / 64, -120), 127)
    q = np.clip(np.rint(b * np.exp2(6.0 - s)[..., None]), -127, 127)
    return q.astype(np.int8).reshape(np.shape(v)), np.where(bad, 255, s + 127).astype(np.uint8)


def ck8_values(q, s):
    f = np.where(s == 255, np.nan, np.exp2(s.astype(np.float64) - 133))
    return (_blocks(q) * f[..., None]).reshape(q.shape)


def silu(a):
    with np.errstate(over="ignore"):
        return a / (1 + np.exp(-a))


def grouped(x, w, offsets, transpose=True):
    """rows of expert e times w[e]^T (or w[e])"""
    out = np.zeros((x.shape[0], w.shape[1] if transpose else w.shape[2]))
    for e in range(w.shape[0]):
        at = slice(int(offsets[e]), int(offsets[e + 1]))
        out[at] = x[at] @ (w[e].T if transpose else w[e])
    return out


def dswiglu(dh, a, b):
    """[da | db] of h = silu(a) b"""
    with np.errstate(over="ignore"):
        s = 1 / (1 + np.exp(-a))
    return np.concatenate([dh * b * s * (1 + a * (1 - s)), dh * a * s], axis=1)
