"""GPU parity of the calls on 4-bit weights and 8-bit checkpoints against the fp64 reference.

Tolerances count roundings.  A product's sum over K terms is off by at most (K + 16) steps of 2^-23 of
its magnitude (the same sum over absolute values): K additions on the matrix cores and in LDS, each
counted as a whole fp32 step because the cores' adder is not specified to round to nearest, and the
products of bf16 pairs exact.  silu and its parts take some 16 single roundings, and exp(-a) is off by
|a| 2^-24 for its argument's rounding: (16 + |a|) steps of 2^-23 cover them.  |silu'| <= 1.1 and
|d/da (s (1 + a (1 - s)))| <= 1.1 carry an error of a on.  A stored value rounds once more, by half a
step (finfo.eps / 2) of its value.  The sigmoid's smallest number is 2^-126: where exp(-a) > 2^126 (a below
-87.3) the reciprocal is flushed to zero, an absolute error of at most 2^-126 that a b multiplies (FLUSH).
Codes, scale bytes and the values they stand for are equal.
"""
import numpy as np
import pytest
import torch

from gpu_common import host, say
from oracle import few_bits_ref as ref

pytestmark = pytest.mark.gpu

STEP = 2.0 ** -23
FLUSH = 2.0 ** -126
TINY = 2.0 ** -133  # below it a bf16 or fp32 result may be flushed or rounded as a subnormal


def _m():
    import mixture_experts_layer_logits_amd as m
    return m


def _f64(t):
    return t.detach().cpu().double().numpy()


def _half(t):
    return torch.finfo(t.dtype).eps / 2


def _within(got, want, bound, what):
    g = host(got).astype(np.float64)
    bound = bound + TINY
    assert np.isfinite(g).all(), what
    worst = np.max(np.abs(g - want) / bound) if g.size else 0.0
    assert worst <= 1, (what, worst)


def _routing(T, E, k, seed, skew=1.0):
    """slot_row [T, k], offsets [E + 1] and gates of a routing in which some experts get nothing."""
    g = torch.Generator().manual_seed(seed)
    logits = torch.randn(T, E, generator=g) + skew * torch.randn(1, E, generator=g)
    top, idx = torch.topk(logits, k, dim=1)
    flat = idx.reshape(-1)
    slot = torch.empty(T * k, dtype=torch.int32)
    slot[torch.argsort(flat, stable=True)] = torch.arange(T * k, dtype=torch.int32)
    off = torch.zeros(E + 1, dtype=torch.int32)
    off[1:] = torch.bincount(flat, minlength=E).cumsum(0)
    return slot.reshape(T, k), off, torch.softmax(top, 1)


class Guarded:
    """A device buffer between two 64-element guards that a call has to leave alone (and, to the byte,
    16-byte aligned); it starts as junk."""

    def __init__(self, *shape, dtype, junk=None):
        n = int(np.prod(shape))
        junk = (123 if dtype in (torch.uint8, torch.int8) else 77.0) if junk is None else junk
        self.all = torch.full((n + 128,), junk, dtype=dtype, device="cuda")
        self.t = self.all[64:64 + n].view(*shape)
        self.junk = junk

    def check(self):
        assert (self.all[:64] == self.junk).all() and (self.all[-64:] == self.junk).all()
        return self.t


# ------------------------------------------------------------------ formats
def _block_rows(seed, rows, cols, dtype):
    """Rows whose blocks span the type's range, with zeros, ties and values next to the scales' borders."""
    g = torch.Generator().manual_seed(seed)
    v = torch.randn(rows, cols, generator=g, dtype=torch.float64)
    v *= torch.exp2(torch.randint(-20, 21, (rows, cols // 32, 1), generator=g).double()).expand(-1, -1, 32).reshape(
        rows, cols)
    b = v.view(rows, cols // 32, 32)
    edge = torch.tensor([6.0, 6.03125, 127 / 64, 255 / 128, 1.0, 3.0, 1.5, 0.0])
    for i in range(min(rows, 64)):
        b[i, 0] = torch.clamp(b[i, 0], -1, 1) * edge[i % 8].double() / max(1e-9, float(b[i, 0].abs().max()))
        b[i, 0, i % 32] = edge[i % 8].double()
        b[i, 0, (i + 1) % 32] = edge[i % 8].double() * [0.25 / 6, 5 / 6, 0.5 / 127, -2.5 / 127][(i // 8) % 4]
    if rows > 2:
        b[1] = 0
        b[2, -1] = 2.0 ** -126
    return v.to(dtype)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("rows,cols", [(1, 32), (3, 96), (65, 64), (257, 1088)])
def test_formats_match_the_reference(rows, cols, dtype):
    m = _m()
    say(f"[gpu] formats rows={rows} cols={cols} {dtype}")
    v = _block_rows(rows + cols, rows, cols, dtype)
    q = Guarded(rows, cols // 2, dtype=torch.uint8)
    s = Guarded(rows, cols // 32, dtype=torch.uint8)
    m.moe_mx4_quantize(rows, cols, v.cuda(), q.t, s.t)
    wq, ws = ref.mx4_quantize(_f64(v))
    assert np.array_equal(host(s.check()), ws)
    assert np.array_equal(ref.mx4_values(host(q.check()), ws), ref.mx4_values(wq, ws))
    q = Guarded(rows, cols, dtype=torch.int8)
    s = Guarded(rows, cols // 32, dtype=torch.uint8)
    m.moe_ckpt8_pack(rows, cols, v.cuda(), q.t, s.t)
    wq, ws = ref.ck8_pack(_f64(v))
    assert np.array_equal(host(s.check()), ws) and np.array_equal(host(q.check()), wq)
    for out in (torch.bfloat16, torch.float32):
        dst = Guarded(rows, cols, dtype=out)
        m.moe_ckpt8_unpack(rows, cols, q.t, s.t, dst.t)
        assert np.array_equal(_f64(dst.check()), ref.ck8_values(wq, ws))
        if cols % 64 == 0:
            dst, h = Guarded(rows, cols, dtype=out), Guarded(rows, cols // 2, dtype=out)
            m.moe_ckpt8_unpack(rows, cols, q.t, s.t, dst.t, h.t)
            ab = ref.ck8_values(wq, ws)
            assert np.array_equal(_f64(dst.check()), ab)
            a, b = ab[:, :cols // 2], ab[:, cols // 2:]
            want = ref.silu(a) * b
            _within(h.check(), want, ((16 + np.abs(a)) * STEP + _half(h.t)) * np.abs(want) + FLUSH * np.abs(a * b),
                    "h")


def test_every_bf16_value_rounds_as_the_reference():
    """All finite bf16 values below 2^120, one to a block beside the block's largest, 1.0."""
    m = _m()
    bits = torch.arange(0, 1 << 16, dtype=torch.int32).to(torch.int16).view(torch.bfloat16).float()
    bits = bits[torch.isfinite(bits) & (bits.abs() < 2.0 ** 120)]
    v = torch.zeros(bits.numel(), 32)
    v[:, 0], v[:, 5] = 1.0, bits
    v = v.to(torch.bfloat16).cuda()
    n = v.shape[0]
    q, s = torch.empty(n, 16, dtype=torch.uint8, device="cuda"), torch.empty(n, 1, dtype=torch.uint8, device="cuda")
    m.moe_mx4_quantize(n, 32, v, q, s)
    wq, ws = ref.mx4_quantize(_f64(v))
    assert np.array_equal(host(s), ws) and np.array_equal(ref.mx4_values(host(q), ws), ref.mx4_values(wq, ws))
    q = torch.empty(n, 32, dtype=torch.int8, device="cuda")
    m.moe_ckpt8_pack(n, 32, v, q, s)
    wq, ws = ref.ck8_pack(_f64(v))
    assert np.array_equal(host(s), ws) and np.array_equal(host(q), wq)


@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
def test_blocks_with_no_number(bad, dtype):
    m = _m()
    for place in range(0, 32, 5):
        v = torch.ones(2, 96, dtype=dtype)
        v[0, 32 + place] = bad
        q, s = torch.empty(2, 48, dtype=torch.uint8, device="cuda"), torch.empty(2, 3, dtype=torch.uint8, device="cuda")
        m.moe_mx4_quantize(2, 96, v.cuda(), q, s)
        assert host(s).tolist() == [[125, 255, 125], [125, 125, 125]]
        q = torch.empty(2, 96, dtype=torch.int8, device="cuda")
        m.moe_ckpt8_pack(2, 96, v.cuda(), q, s)
        back = torch.empty(2, 96, dtype=dtype, device="cuda")
        m.moe_ckpt8_unpack(2, 96, q, s, back)
        want = torch.ones(2, 96)
        want[0, 32:64] = float("nan")
        assert torch.equal(torch.nan_to_num(back.float().cpu(), 9.0), torch.nan_to_num(want, 9.0))


def test_every_scale_byte_and_code_unpacks():
    m = _m()
    q = torch.arange(-128, 128, dtype=torch.int16).to(torch.int8).reshape(8, 32).repeat(256, 1)
    s = torch.arange(256, dtype=torch.uint8).repeat_interleave(8).reshape(-1, 1)
    dst = torch.empty(2048, 32, device="cuda")
    m.moe_ckpt8_unpack(2048, 32, q.cuda(), s.cuda(), dst)
    with np.errstate(over="ignore"):  # -128 2^121, which no pack writes, is past fp32: -inf
        want = ref.ck8_values(q.numpy(), s.numpy()).astype(np.float32)
    assert np.array_equal(host(dst), want, equal_nan=True)


# ------------------------------------------------------------------ products with 4-bit weights
def _weights4(E, n, K, seed):
    g = torch.Generator().manual_seed(seed)
    return ref.mx4_quantize((0.05 * torch.randn(E, n, K, generator=g)).numpy())


PRODUCTS = [  # T, d, f, E, k
    (1, 64, 64, 1, 1), (1, 256, 128, 8, 4), (1, 2048, 64, 128, 4), (3, 192, 320, 5, 2), (7, 1088, 64, 5, 3),
    (16, 320, 64, 3, 1), (17, 128, 192, 2, 2), (33, 64, 64, 130, 8), (61, 448, 128, 4, 2), (200, 256, 64, 7, 3),
    (515, 192, 64, 2, 1), (300, 64, 64, 1024, 32), (700, 128, 128, 1, 1),
    (512, 128, 1536, 32, 4), (640, 4096, 128, 20, 2),  # tiles of 12 waves: gated, and not
    (40, 128, 1024, 60, 4), (150, 2048, 192, 96, 3), (9, 1280, 448, 31, 7),  # eight, four and two tiles a workgroup
    (342, 1984, 64, 18, 5), (150, 1152, 192, 2, 2), (257, 576, 320, 3, 1), (120, 1664, 192, 13, 4),  # few tiles
    (500, 320, 1024, 40, 4), (400, 448, 512, 64, 4), (512, 192, 1536, 32, 4), (640, 4096, 192, 20, 2),
    (300, 1024, 512, 4, 2), (300, 1088, 512, 4, 2)]


@pytest.mark.parametrize("act", ["bf16", "f32"])
@pytest.mark.parametrize("T,d,f,E,k", PRODUCTS)
def test_products(T, d, f, E, k, act):
    m = _m()
    say(f"[gpu] w4 products T={T} d={d} f={f} E={E} k={k} {act}")
    dt = torch.float32 if act == "f32" else torch.bfloat16
    s = m.make_shape(T, d, f, E, k, m.MOE_F32 if act == "f32" else m.MOE_BF16)
    _, off, _ = _routing(T, E, k, T + d)
    R = T * k
    g = torch.Generator().manual_seed(T)
    x = torch.randn(R, d, generator=g).to(dt)
    w = [_weights4(E, f, d, 1), _weights4(E, f, d, 2), _weights4(E, d, f, 3)]
    v = [ref.mx4_values(*p) for p in w]
    dev = [[torch.from_numpy(t).cuda() for t in p] for p in w]
    offd = off.cuda()
    h = Guarded(R, f, dtype=dt)
    m.moe_ffn_gemm1_fwd_w4(s, x.cuda(), *dev[0], *dev[1], offd, h.t)
    xv = _f64(x)
    a, b = ref.grouped(xv, v[0], off), ref.grouped(xv, v[1], off)
    ma, mb = (ref.grouped(np.abs(xv), np.abs(u), off) for u in v[:2])
    u = (d + 16) * STEP
    want = ref.silu(a) * b
    bound = 1.1 * np.abs(b) * u * ma + np.abs(ref.silu(a)) * u * mb + 1.1 * u * u * ma * mb
    _within(h.check(), want, bound + ((16 + np.abs(a)) * STEP + _half(h.t)) * np.abs(want) +
            FLUSH * np.abs(a * b), "h")
    y = Guarded(R, d, dtype=dt)
    m.moe_ffn_gemm2_fwd_w4(s, h.t, *dev[2], offd, y.t)
    hv = _f64(h.t)
    want = ref.grouped(hv, v[2], off)
    mag = ref.grouped(np.abs(hv), np.abs(v[2]), off)
    _within(y.check(), want, (f + 16) * STEP * mag + _half(y.t) * np.abs(want), "y")


@pytest.mark.parametrize("act", ["bf16", "f32"])
@pytest.mark.parametrize("T,E", [(4, 3), (70, 3)])
def test_numbers_that_are_none_stay_in_their_rows(T, E, act):
    """An infinite element reaches its own routed row alone, a NaN weight block its own output column."""
    m = _m()
    d, f, k = 256, 64, 1
    dt = torch.float32 if act == "f32" else torch.bfloat16
    s = m.make_shape(T, d, f, E, k, m.MOE_F32 if act == "f32" else m.MOE_BF16)
    off = torch.tensor([0, T // 2, T // 2, T], dtype=torch.int32)  # the middle expert has no row
    x = torch.ones(T, d, dtype=dt)
    x[1, 77] = float("inf")
    q, sc = ref.mx4_quantize(np.full((E, f, d), 0.5))
    sc[2, 5, 3] = 255
    q[2, 5, 48:64] = 0
    args = [torch.from_numpy(q).cuda(), torch.from_numpy(sc).cuda()]
    one = ref.mx4_quantize(np.full((E, f, d), 0.25))
    h = torch.zeros(T, f, dtype=dt, device="cuda")
    m.moe_ffn_gemm1_fwd_w4(s, x.cuda(), *args, *(torch.from_numpy(t).cuda() for t in one), off.cuda(), h)
    bad = ~np.isfinite(host(h))
    want = np.zeros((T, f), dtype=bool)
    want[1] = True
    want[T // 2:, 5] = True
    assert np.array_equal(bad, want)


@pytest.mark.parametrize("act", ["bf16", "f32"])
@pytest.mark.parametrize("K", [64, 128, 192, 384, 448])
@pytest.mark.parametrize("T", [6, 70, 200])
def test_a_nan_block_at_a_rows_end_or_begin_stays_in_its_row(T, K, act):
    """Neither the row before (whose last step may reach past its end) nor the one behind sees it."""
    m = _m()
    E, other = 3, 64
    dt = torch.float32 if act == "f32" else torch.bfloat16
    a = m.MOE_F32 if act == "f32" else m.MOE_BF16
    off = torch.tensor([0, T // 2, T // 2, T], dtype=torch.int32).cuda()
    x = torch.ones(T, K, dtype=dt, device="cuda")
    q, sc = ref.mx4_quantize(np.full((E, other, K), 0.5))
    sc[2, 5, 0] = sc[2, 40, -1] = 255
    w = [torch.from_numpy(t).cuda() for t in (q, sc)]
    want = np.zeros((T, other), dtype=bool)
    want[T // 2:, [5, 40]] = True
    h = torch.zeros(T, other, dtype=dt, device="cuda")
    m.moe_ffn_gemm1_fwd_w4(m.make_shape(T, K, other, E, 1, a), x, *w, *w, off, h)
    assert np.array_equal(np.isnan(host(h)), want)
    y = torch.zeros(T, other, dtype=dt, device="cuda")
    m.moe_ffn_gemm2_fwd_w4(m.make_shape(T, other, K, E, 1, a), x, *w, off, y)
    assert np.array_equal(np.isnan(host(y)), want)
    fine = host(y)[~want]
    assert (fine == 0.5 * K).all()


def test_rows_do_not_depend_on_the_expert_that_holds_them():
    """Rows moved to another expert with the same weights come out the same, bit for bit."""
    m = _m()
    T, d, f, E = 6, 512, 64, 4
    s = m.make_shape(T, d, f, E, 1)
    x = torch.randn(T, d, generator=torch.Generator().manual_seed(0)).to(torch.bfloat16).cuda()
    q, sc = (torch.from_numpy(t).cuda() for t in _weights4(E, f, d, 5))
    out = []
    for off in ([0, 6, 6, 6, 6], [0, 0, 6, 6, 6]):
        q1 = q.clone()
        s1 = sc.clone()
        if off[1] == 0:  # the second expert now holds the first one's weights
            q1[1], s1[1] = q[0], sc[0]
        h = torch.empty(T, f, dtype=torch.bfloat16, device="cuda")
        m.moe_ffn_gemm1_fwd_w4(s, x, q1, s1, q1, s1, torch.tensor(off, dtype=torch.int32).cuda(), h)
        out.append(h)
    assert torch.equal(*out)


# ------------------------------------------------------------------ 8-bit checkpoints
FFN = [(1, 64, 64, 1, 1), (5, 128, 64, 4, 2), (40, 192, 320, 6, 3), (130, 256, 128, 3, 1), (257, 64, 192, 5, 2),
       (300, 448, 64, 64, 4), (1100, 64, 64, 1, 1),
       (24700, 64, 128, 2, 1), (3300, 64, 1024, 2, 1), (16320, 64, 1024, 1, 1)]  # each of the larger tiles


def _ffn_inputs(T, d, f, E, k, whole):
    """whole: small whole numbers, so that every sum is exact and the codes have to be equal."""
    g = torch.Generator().manual_seed(T + d + f)
    R = T * k
    _, off, _ = _routing(T, E, k, T + f)
    if whole:
        mk = lambda *n: torch.randint(-2, 3, n, generator=g).float()  # noqa: E731
        x, dy, W1, W3, W2 = mk(R, d), mk(R, d), mk(E, f, d), mk(E, f, d), mk(E, d, f)
    else:
        mk = lambda s, *n: s * torch.randn(*n, generator=g)  # noqa: E731
        x, dy = mk(1.0, R, d), mk(0.1, R, d)
        W1, W3, W2 = mk(d ** -0.5, E, f, d), mk(d ** -0.5, E, f, d), mk(f ** -0.5, E, d, f)
    return off, [t.to(torch.bfloat16) for t in (x, dy, W1, W3, W2)]


@pytest.mark.parametrize("whole", [True, False], ids=["whole", "normal"])
@pytest.mark.parametrize("T,d,f,E,k", FFN)
def test_ffn_checkpoint(T, d, f, E, k, whole):
    m = _m()
    say(f"[gpu] ffn checkpoint T={T} d={d} f={f} E={E} k={k} whole={whole}")
    off, (x, dy, W1, W3, W2) = _ffn_inputs(T, d, f, E, k, whole)
    R = T * k
    s = m.make_shape(T, d, f, E, k)
    offd = off.cuda()
    h, q, sc = (Guarded(R, f, dtype=torch.bfloat16), Guarded(R, 2 * f, dtype=torch.int8),
                Guarded(R, 2 * f // 32, dtype=torch.uint8))
    m.moe_ffn_gemm1_fwd_c8(s, x.cuda(), W1.cuda(), W3.cuda(), offd, h.t, q.t, sc.t)
    xv = _f64(x)
    a, b = ref.grouped(xv, _f64(W1), off), ref.grouped(xv, _f64(W3), off)
    ma, mb = (ref.grouped(np.abs(xv), np.abs(_f64(w)), off) for w in (W1, W3))
    u = 0.0 if whole else (d + 16) * STEP
    want = ref.silu(a) * b
    bound = 1.1 * np.abs(b) * u * ma + np.abs(ref.silu(a)) * u * mb + 1.1 * u * u * ma * mb
    _within(h.check(), want, bound + ((16 + np.abs(a)) * STEP + _half(h.t)) * np.abs(want) +
            FLUSH * np.abs(a * b), "h")
    ab, qv, sv = np.concatenate([a, b], axis=1), host(q.check()), host(sc.check())
    if whole:
        wq, ws = ref.ck8_pack(ab)
        assert np.array_equal(sv, ws) and np.array_equal(qv, wq)
    kept = ref.ck8_values(qv, sv)
    # half a step of the block (at most amax / 127), of sums that are off by delta themselves
    delta = u * np.concatenate([ma, mb], axis=1)
    top = (np.abs(ab) + delta).reshape(R, -1, 32).max(-1).repeat(32, axis=-1)
    assert (np.abs(kept - ab) <= top / 127 + delta + 2.0 ** -127).all()
    # the same h as the plain call's, and its [a | b] within the checkpoint's step of the kept one
    h2, ab2 = torch.empty_like(h.t), torch.empty(R, 2 * f, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(m.moe_workspace_size(s), dtype=torch.uint8, device="cuda")
    m.moe_ffn_gemm1_fwd(s, x.cuda(), W1.cuda(), W3.cuda(), offd, ab2, h2, ws)
    assert torch.equal(h2, h.t)

    dab, h8 = Guarded(R, 2 * f, dtype=torch.bfloat16), Guarded(R, f, dtype=torch.bfloat16)
    m.moe_ffn_dgrad2_c8(s, dy.cuda(), W2.cuda(), q.t, sc.t, offd, dab.t, h8.t)
    dyv, w2 = _f64(dy), _f64(W2)
    dh = ref.grouped(dyv, w2, off, transpose=False)
    ddh = (0.0 if whole else (d + 16) * STEP) * ref.grouped(np.abs(dyv), np.abs(w2), off, transpose=False)
    a8, b8 = kept[:, :f], kept[:, f:]
    want = ref.silu(a8) * b8
    few = (16 + np.abs(a8)) * STEP
    _within(h8.check(), want, (few + _half(h8.t)) * np.abs(want) + FLUSH * np.abs(a8 * b8), "h again")
    want = ref.dswiglu(dh, a8, b8)
    sg = 1 / (1 + np.exp(-np.clip(a8, -700, 700)))
    # 1 + a (1 - s) cancels: its roundings count with the magnitude of its terms
    ba = 1.1 * np.abs(b8) * ddh + 2 * few * (1 + np.abs(a8)) * (np.abs(dh) + ddh) * np.abs(b8) * sg
    bb = np.abs(a8 * sg) * ddh + few * (np.abs(dh) + ddh) * np.abs(a8 * sg)
    ba += FLUSH * (1 + np.abs(a8)) * (np.abs(dh) + ddh) * np.abs(b8)
    bb += FLUSH * (np.abs(dh) + ddh) * np.abs(a8)
    _within(dab.check(), want, np.concatenate([ba, bb], axis=1) + _half(dab.t) * np.abs(want), "dab")


COMBINE = [(1, 64, 1, 1), (3, 192, 5, 4), (65, 320, 8, 3), (129, 2048, 16, 6), (40, 64, 64, 32), (500, 1088, 12, 8)]


@pytest.mark.parametrize("act", ["bf16", "f32"])
@pytest.mark.parametrize("add", [False, True])
@pytest.mark.parametrize("T,d,E,k", COMBINE)
def test_combine_checkpoint(T, d, E, k, add, act):
    m = _m()
    say(f"[gpu] combine checkpoint T={T} d={d} E={E} k={k} add={add} {act}")
    dt = torch.float32 if act == "f32" else torch.bfloat16
    s = m.make_shape(T, d, 64, E, k, m.MOE_F32 if act == "f32" else m.MOE_BF16)
    slot, _, gates = _routing(T, E, k, T + d)
    gates[0, 0] = 0.0
    g = torch.Generator().manual_seed(d)
    R = T * k
    rows = (torch.randn(R, d, generator=g) * torch.exp2(torch.randint(-6, 7, (R, 1), generator=g).float())).to(dt)
    y_add = torch.randn(T, d, generator=g).to(dt).cuda() if add else None
    dy = torch.randn(T, d, generator=g).to(dt)
    args = [t.cuda() for t in (rows, gates, slot)]
    y, q, sc = Guarded(T, d, dtype=dt), Guarded(R, d, dtype=torch.int8), Guarded(R, d // 32, dtype=torch.uint8)
    m.moe_combine_c8(s, *args, y_add, y.t, q.t, sc.t)
    plain = torch.empty(T, d, dtype=dt, device="cuda")
    m.moe_combine(s, *args, y_add, plain)
    assert torch.equal(y.check(), plain)
    wq, ws = ref.ck8_pack(_f64(rows))
    assert np.array_equal(host(q.check()), wq) and np.array_equal(host(sc.check()), ws)
    dyp, dg = Guarded(R, d, dtype=dt), Guarded(T, k, dtype=torch.float32)
    m.moe_combine_bwd_c8(s, dy.cuda(), q.t, sc.t, args[1], args[2], dyp.t, dg.t)
    dyp2, dg2 = torch.empty(R, d, dtype=dt, device="cuda"), torch.empty(T, k, device="cuda")
    m.moe_combine_bwd(s, dy.cuda(), args[0], args[1], args[2], dyp2, dg2)
    assert torch.equal(dyp.check(), dyp2)
    kept = ref.ck8_values(wq, ws)[slot.numpy()]              # [T, k, d]
    dyv = _f64(dy)[:, None]
    # a lane adds d / 64 + 8 products, the wave 6 more times
    _within(dg.check(), (dyv * kept).sum(-1), (d / 64 + 24) * 2.0 ** -24 * (np.abs(dyv) * np.abs(kept)).sum(-1), "dgates")


# ------------------------------------------------------------------ streams, graphs, empty batches
def _pass(m, s, a, out):
    """Every call once, in the order of use: serving, then a training step's."""
    m.moe_ffn_gemm1_fwd_w4(s, a["x"], *a["w"][0], *a["w"][1], a["off"], out["h4"])
    m.moe_ffn_gemm2_fwd_w4(s, out["h4"], *a["w"][2], a["off"], out["y4"])
    m.moe_ffn_gemm1_fwd_c8(s, a["x"], a["W1"], a["W3"], a["off"], out["h"], out["abq"], out["ab_s"])
    m.moe_combine_c8(s, out["y4"], a["gates"], a["slot"], None, out["y"], out["yq"], out["ys"])
    m.moe_combine_bwd_c8(s, a["dy"], out["yq"], out["ys"], a["gates"], a["slot"], out["dyp"], out["dg"])
    m.moe_ffn_dgrad2_c8(s, out["dyp"], a["W2"], out["abq"], out["ab_s"], a["off"], out["dab"], out["h8"])
    m.moe_ckpt8_unpack(s.T * s.k, 2 * s.f, out["abq"], out["ab_s"], out["ab"])
    m.moe_ckpt8_pack(s.T * s.k, s.d, out["dyp"], out["q"], out["qs"])


def _all_inputs(T, d, f, E, k, seed):
    m = _m()
    g = torch.Generator().manual_seed(seed)
    slot, off, gates = _routing(T, E, k, seed)
    R, bf = T * k, torch.bfloat16
    r = lambda s, *n: (s * torch.randn(*n, generator=g)).to(bf).cuda()  # noqa: E731
    a = dict(x=r(1, R, d), dy=r(1, T, d), W1=r(.1, E, f, d), W3=r(.1, E, f, d), W2=r(.1, E, d, f), off=off.cuda(),
             slot=slot.cuda(), gates=gates.cuda())
    a["w"] = m.quantize_weights(a["W1"], a["W3"], a["W2"])
    e = lambda *n, dtype=bf: torch.empty(*n, dtype=dtype, device="cuda")  # noqa: E731
    i8, u8 = torch.int8, torch.uint8
    out = dict(h4=e(R, f), y4=e(R, d), h=e(R, f), abq=e(R, 2 * f, dtype=i8), ab_s=e(R, 2 * f // 32, dtype=u8),
               y=e(T, d), yq=e(R, d, dtype=i8), ys=e(R, d // 32, dtype=u8), dyp=e(R, d),
               dg=e(T, k, dtype=torch.float32), dab=e(R, 2 * f), h8=e(R, f), ab=e(R, 2 * f), q=e(R, d, dtype=i8),
               qs=e(R, d // 32, dtype=u8))
    return m.make_shape(T, d, f, E, k), a, out


def test_repeated_passes_are_bitwise_the_same_and_streams_do_not_mix():
    m = _m()
    sets = [_all_inputs(150, 256, 128, 9, 3, seed) for seed in (1, 2)]
    want = []
    for s, a, out in sets:
        _pass(m, s, a, out)
        want.append({n: t.clone() for n, t in out.items()})
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    for _ in range(3):
        for (s, a, out), st in zip(sets, streams):
            with torch.cuda.stream(st):
                for t in out.values():
                    t.zero_()
                _pass(m, s, a, out)
    torch.cuda.synchronize()
    for (_, _, out), w in zip(sets, want):
        for n in out:
            assert torch.equal(out[n], w[n]), n


def test_captured_passes_replay():
    m = _m()
    s, a, out = _all_inputs(37, 128, 64, 5, 2, 3)
    s2, b, _ = _all_inputs(37, 128, 64, 5, 2, 4)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        _pass(m, s, a, out)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _pass(m, s, a, out)
    for i in range(4):
        src = (b, a)[i % 2]  # other inputs and another routing, in place
        if i:
            for n in ("x", "dy", "off", "slot", "gates"):
                keep = a[n].clone() if i == 1 else None
                if keep is not None:
                    b.setdefault("_" + n, keep)
                a[n].copy_(b[n] if i % 2 else b["_" + n])
        for t in out.values():
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        got = {n: t.clone() for n, t in out.items()}
        _pass(m, s, a, out)
        torch.cuda.synchronize()
        for n in out:
            assert torch.equal(out[n], got[n]), (i, n)
        del src


def test_empty_batch():
    m = _m()
    s, a, out = _all_inputs(4, 64, 64, 3, 1, 5)
    s0 = m.make_shape(0, 64, 64, 3, 1)
    a = {**a, "x": a["x"][:0], "dy": a["dy"][:0], "off": torch.zeros(4, dtype=torch.int32, device="cuda"),
         "slot": a["slot"][:0], "gates": a["gates"][:0]}
    _pass(m, s0, a, {n: t[:0] for n, t in out.items()})
    torch.cuda.synchronize()
