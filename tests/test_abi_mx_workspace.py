"""The workspace that moe_workspace_size reports covers every region the MXFP8 GEMMs carve from it, at row
counts that are no multiple of the 32-element block too (host arithmetic alone)."""
import pytest

import mixture_experts_layer_logits_amd as m


def _regions(*operands):
    """[codes | scales] of each operand (rows, K), every region rounded up to 256 bytes"""
    al = lambda n: (n + 255) // 256 * 256  # noqa: E731
    return sum(al(rows * K) + al(rows * K // 32) for rows, K in operands)


@pytest.mark.parametrize("T,d,f,E,k", [(1100, 256, 384, 2, 2), (16384, 4096, 1536, 32, 4), (33, 128, 128, 5, 1),
                                       (7, 1024, 256, 1, 1), (999, 2048, 1024, 128, 3)])
def test_workspace_covers_the_mx_gemms(T, d, f, E, k):
    R = T * k
    Rp = R + 128 * E
    size = m.moe_workspace_size(m.make_shape(T, d, f, E, k, m.MOE_BF16, m.MOE_MXFP8, m.MOE_MX_ALL))
    for name, need in dict(gemm1=_regions((R, d), (2 * E * f, d)), gemm2=_regions((R, f), (E * d, f)),
                           dgrad2=_regions((R, d), (E * f, d)), dgrad1=_regions((R, 2 * f), (E * d, 2 * f)),
                           wgrad2=_regions((d, Rp), (f, Rp)), wgrad1=_regions((2 * f, Rp), (d, Rp))).items():
        assert size >= need, (name, size, need)
