"""The products with 4-bit weights over many pieces of their reduction, against the fp64 reference.

A sum of whole numbers that stays below 2^24 is exact in fp32 in any order, so a product of such rows and
weights is the exact sum, rounded once to the output's type, and the comparison is for equality.  Other sums
are off by at most (K + 16) steps of 2^-23 of the sum of absolute values, and a stored value by half a step
of its type."""
import numpy as np
import pytest
import torch

from gpu_common import host, say
from oracle import few_bits_ref as ref

pytestmark = pytest.mark.gpu

STEP = 2.0 ** -23
TYPES = [torch.bfloat16, torch.float32]
IDS = ["bf16", "f32"]


def _m():
    import mixture_experts_layer_logits_amd as m
    return m


def _f64(t):
    return t.detach().cpu().double().numpy()


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
@pytest.mark.parametrize("T,K,N,E", [(1, 4096, 256, 1), (8, 2048, 512, 8), (24, 1536, 2048, 24), (5, 1088, 192, 3),
                                     (4, 192, 2048, 40), (200, 2048, 128, 2), (90, 4160, 64, 1), (800, 512, 192, 3)])
def test_each_piece_of_a_row_meets_its_own_weights(T, K, N, E, dtype):
    """The pieces of the reduction (64 elements, and whole runs of them) hold different whole numbers, as do
    neighbouring rows and experts, and every partial sum is exact: an element of another piece, row or
    tile, or one that is left over from the piece before, changes the sum."""
    m = _m()
    say(f"[gpu] pieces T={T} K={K} N={N} E={E} {dtype}")
    k, r = np.arange(K), np.arange(T)
    x = ((k // 64)[None] * 3 + r[:, None] * 7 + k[None] % 5) % 31 + 1                          # 1 .. 31
    u8 = lambda v: np.asarray(v, dtype=np.uint8)  # noqa: E731  (bytes wrap at a multiple of 16)
    n, e = u8(np.arange(N) % 256)[None, :, None], u8(np.arange(E))[:, None, None]
    code = (u8(k // 32 * 5 % 256) + n * u8(3) + e + u8(k % 3)) & u8(15)
    q = code[..., 0::2] | code[..., 1::2] << u8(4)
    sc = u8(127) + ((u8(k[::32] // 32 % 256) + n + e) & u8(1))
    assert 2 * 31 * 12 * K < 2 ** 24  # every sum a whole number of halves below 2^24
    off = np.linspace(0, T, E + 1).astype(np.int32)
    s = m.make_shape(T, N, K, E, 1, m.MOE_F32 if dtype == torch.float32 else m.MOE_BF16)
    y = torch.empty(T, N, dtype=dtype, device="cuda")
    args = [torch.from_numpy(t).cuda() for t in (q, sc, off)]
    xd = torch.from_numpy(x).to(dtype).cuda()
    a = ref.grouped(x.astype(np.float64), ref.mx4_values(q, sc), off)
    want = torch.from_numpy(a).to(dtype)
    for _ in range(3):
        y.fill_(-1)
        m.moe_ffn_gemm2_fwd_w4(s, xd, *args, y)
        assert torch.equal(y.cpu(), want)
    # gated, both projections the same: h = silu(a) a of the exact a
    s1 = m.make_shape(T, K, N, E, 1, m.MOE_F32 if dtype == torch.float32 else m.MOE_BF16)
    h, h2 = torch.empty(T, N, dtype=dtype, device="cuda"), torch.empty(T, N, dtype=dtype, device="cuda")
    m.moe_ffn_gemm1_fwd_w4(s1, xd, *args[:2], *args[:2], args[2], h)
    m.moe_ffn_gemm1_fwd_w4(s1, xd, *args[:2], *args[:2], args[2], h2)
    with np.errstate(over="ignore"):
        hw = ref.silu(a) * a
    tol = ((16 + np.abs(a)) * STEP + torch.finfo(dtype).eps / 2) * np.abs(hw) + 2.0 ** -126 * (a * a + 1)
    assert torch.equal(h, h2) and (np.abs(_f64(h) - hw) <= tol).all()


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
@pytest.mark.parametrize("K,N,E", [(2048, 512, 4), (1088, 192, 3), (4096, 256, 16)])
def test_a_row_in_batches_of_many_sizes(K, N, E, dtype):
    """The products split the reduction by the sizes of the batch, so a row's output is not the same to the bit
    in every batch: each lies within its own bound of the exact sum, and a batch repeats bit for bit."""
    m = _m()
    g = torch.Generator().manual_seed(K)
    x = torch.randn(700 * E, K, generator=g).to(dtype).cuda()
    w = 0.05 * torch.randn(E, N, K, generator=g)
    q, sc = m.quantize_weights(w.cuda())[0]
    v = ref.mx4_values(host(q), host(sc))
    for per in (1, 2, 9, 33, 96, 97, 700):
        say(f"[gpu] batch rows={per} E={E} K={K} {dtype}")
        T = per * E
        rows = x.view(E, 700, K)[:, :per].reshape(T, K).contiguous()
        off = torch.arange(0, T + 1, per, dtype=torch.int32)
        s = m.make_shape(T, N, K, E, 1, m.MOE_F32 if dtype == torch.float32 else m.MOE_BF16)
        y = torch.empty(T, N, dtype=dtype, device="cuda")
        z = torch.full_like(y, 3)
        m.moe_ffn_gemm2_fwd_w4(s, rows, q, sc, off.cuda(), y)
        m.moe_ffn_gemm2_fwd_w4(s, rows, q, sc, off.cuda(), z)
        assert torch.equal(y, z)
        xv = _f64(rows)
        want = ref.grouped(xv, v, off)
        bound = (K + 16) * STEP * ref.grouped(np.abs(xv), np.abs(v), off) + torch.finfo(dtype).eps / 2 * np.abs(want)
        assert (np.abs(_f64(y) - want) <= bound + 2.0 ** -133).all()
