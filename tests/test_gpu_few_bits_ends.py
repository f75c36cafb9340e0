"""The few-bits calls at the ends of their formats, against the fp64 reference: codes, scale bytes and the
values that they stand for are equal."""
import numpy as np
import pytest
import torch

from gpu_common import host, say
from oracle import few_bits_ref as ref

pytestmark = pytest.mark.gpu

TYPES = [torch.bfloat16, torch.float32]
IDS = ["bf16", "f32"]


def _m():
    import mixture_experts_layer_logits_amd as m
    return m


def _f64(t):
    return t.detach().cpu().double().numpy()


def _end_rows(dtype):
    """Blocks whose largest magnitude lies at an end of the formats' scales: the type's smallest number, around
    the lowest scale bytes (6 2^-126 of MXFP4, 127/64 2^-120 of MXINT8), and the highest."""
    low = 2.0 ** -149 if dtype == torch.float32 else 2.0 ** -133
    step = torch.finfo(dtype).eps
    tops = [low, 2.0 ** -130, 2.0 ** -127, 2.0 ** -126, 6 * 2.0 ** -126, 6 * (1 + step) * 2.0 ** -126, 2.0 ** -121, 2.0 ** -120,
            127 / 64 * 2.0 ** -120, 127 / 64 * (1 + step) * 2.0 ** -120, 2.0 ** 127, 1.5 * 2.0 ** 127,
            127 / 64 * 2.0 ** 127, torch.finfo(dtype).max]
    g = torch.Generator().manual_seed(7)
    rows = []
    for top in tops:
        v = (2 * torch.rand(4, 32, generator=g, dtype=torch.float64) - 1) * top
        v[0, 3], v[1, 3], v[2, 30], v[3, 0] = top, -top, top, -top
        v[2, :8] = torch.tensor([0.0, -0.0, top / 2, -top / 4, top / 6, -top / 127, top / 254, -top * 126.5 / 127],
                                dtype=torch.float64)
        v[3, 1:] = 0                                           # the largest alone
        rows.append(v)
    return torch.cat(rows).to(dtype)


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
def test_blocks_at_the_ends_of_the_scales(dtype):
    m = _m()
    say(f"[gpu] format ends {dtype}")
    v = _end_rows(dtype)
    n = v.shape[0]
    assert torch.isfinite(v).all()
    q, s = torch.empty(n, 16, dtype=torch.uint8, device="cuda"), torch.empty(n, 1, dtype=torch.uint8, device="cuda")
    m.moe_mx4_quantize(n, 32, v.cuda(), q, s)
    wq, ws = ref.mx4_quantize(_f64(v))
    assert {1, 253} <= set(ws.ravel().tolist())
    assert np.array_equal(host(s), ws) and np.array_equal(host(q), wq)
    q = torch.empty(n, 32, dtype=torch.int8, device="cuda")
    m.moe_ckpt8_pack(n, 32, v.cuda(), q, s)
    wq, ws = ref.ck8_pack(_f64(v))
    assert {7, 254} <= set(ws.ravel().tolist())
    assert np.array_equal(host(s), ws) and np.array_equal(host(q), wq)
    back = torch.empty(n, 32, dtype=dtype, device="cuda")
    m.moe_ckpt8_unpack(n, 32, q, s, back)
    assert np.array_equal(_f64(back), ref.ck8_values(wq, ws))


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
def test_the_combine_keeps_rows_at_the_ends_of_the_scales(dtype):
    m = _m()
    v = _end_rows(dtype)
    v = v[: v.shape[0] // 2 * 2].reshape(-1, 64)
    T = v.shape[0]
    s = m.make_shape(T, 64, 64, 1, 1, m.MOE_F32 if dtype == torch.float32 else m.MOE_BF16)
    slot = torch.arange(T, dtype=torch.int32, device="cuda").flip(0).reshape(T, 1)
    y, q = torch.empty(T, 64, dtype=dtype, device="cuda"), torch.empty(T, 64, dtype=torch.int8, device="cuda")
    sc = torch.empty(T, 2, dtype=torch.uint8, device="cuda")
    m.moe_combine_c8(s, v.cuda(), torch.zeros(T, 1, device="cuda"), slot, None, y, q, sc)
    wq, ws = ref.ck8_pack(_f64(v))
    assert np.array_equal(host(sc), ws) and np.array_equal(host(q), wq)


@pytest.mark.parametrize("R", [40, 300])
def test_gemm1_keeps_sums_at_the_ends_of_the_scales(R):
    """Row r takes one column of the weights: a and b are the weights' own values."""
    m = _m()
    f = d = 64
    g = torch.Generator().manual_seed(R)
    top = torch.tensor([2.0 ** -121, 2.0 ** -120, 127 / 64 * 2.0 ** -120, 2.0 ** -100, 1.0, 2.0 ** 127, 127 / 64 * 2.0 ** 127,
                        torch.finfo(torch.bfloat16).max], dtype=torch.float64).repeat(8)
    W = [(2 * torch.rand(1, f, d, generator=g, dtype=torch.float64) - 1) * top for _ in range(2)]
    for w in W:
        w[0, 3] = w[0, 40] = top * torch.where(torch.arange(d) % 2 == 0, 1, -1)
        w[:, :, top < 2.0 ** -110] = torch.where(w.abs() < 2.0 ** -126, 0, w)[:, :, top < 2.0 ** -110]  # no subnormals
    W = [w.to(torch.bfloat16) for w in W]
    x = torch.zeros(R, d)
    x[torch.arange(R), torch.arange(R) % d] = 1
    s = m.make_shape(R, d, f, 1, 1)
    off = torch.tensor([0, R], dtype=torch.int32, device="cuda")
    e = lambda *n, dtype=torch.bfloat16: torch.empty(*n, dtype=dtype, device="cuda")  # noqa: E731
    h, q, sc = e(R, f), e(R, 2 * f, dtype=torch.int8), e(R, 2 * f // 32, dtype=torch.uint8)
    m.moe_ffn_gemm1_fwd_c8(s, x.to(torch.bfloat16).cuda(), W[0].cuda(), W[1].cuda(), off, h, q, sc)
    ab = np.concatenate([_f64(w)[0].T[np.arange(R) % d] for w in W], axis=1)
    wq, ws = ref.ck8_pack(ab)
    assert {7, 254} <= set(ws.ravel().tolist())
    assert np.array_equal(host(sc), ws) and np.array_equal(host(q), wq)


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
@pytest.mark.parametrize("T", [8, 96])
def test_products_take_every_scale_byte(T, dtype):
    """One element of a row is 1: the output is one weight.  Below the type's smallest normal number it may be
    zero; from 2^126 on a row of weights holds one number alone, as a larger code would be infinite."""
    m = _m()
    say(f"[gpu] scale bytes T={T} {dtype}")
    K, N = 64, 256
    codes = np.arange(K) % 16
    q = np.tile((codes[0::2] | codes[1::2] << 4).astype(np.uint8), (1, N, 1))
    sc = np.repeat(np.arange(N, dtype=np.uint8)[None, :, None], 2, axis=2)
    q[0, 253:] = 0
    q[0, 253:, [0, 20]] = 2 | 9 << 4                           # 1 and -0.5
    sc[0, 255] = 254
    x = torch.zeros(T, K, dtype=dtype)
    x[torch.arange(T), (torch.arange(T) * 5) % K] = 1
    s = m.make_shape(T, N, K, 1, 1, m.MOE_F32 if dtype == torch.float32 else m.MOE_BF16)
    y = torch.empty(T, N, dtype=dtype, device="cuda")
    m.moe_ffn_gemm2_fwd_w4(s, x.cuda(), torch.from_numpy(q).cuda(), torch.from_numpy(sc).cuda(),
                           torch.tensor([0, T], dtype=torch.int32, device="cuda"), y)
    want = ref.mx4_values(q, sc)[0].T[(np.arange(T) * 5) % K]
    got = _f64(y)
    small = np.abs(want) < 2.0 ** -126
    assert small.any() and np.array_equal(got[~small], want[~small])
    assert ((got[small] == 0) | (got[small] == want[small])).all()
