// Internal declarations: expert products with MXFP4 weights (E2M1 codes, two a byte, one E8M0 scale
// byte per 32 elements along the reduction axis).
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>
#include "gemm.h"

namespace moe {

constexpr int kMx4Block = 32;
constexpr int kW4MaxWidth = 1 << 22;  // d and f: offsets inside a tile's rows are 32-bit

// elem_bytes: 2 (bf16) or 4 (float)
hipError_t mx4_quantize_rows(int elem_bytes, int rows, int cols, const void* src, uint8_t* q, uint8_t* s,
                             hipStream_t st);
// h = silu(X W1^T) (X W3^T)
hipError_t gemm1_fwd_w4(int elem_bytes, const GemmShape& g, const int* offsets, const void* X, const uint8_t* W1q,
                        const uint8_t* W1s, const uint8_t* W3q, const uint8_t* W3s, void* h, hipStream_t st);
// Y = H W2^T
hipError_t gemm2_fwd_w4(int elem_bytes, const GemmShape& g, const int* offsets, const void* H, const uint8_t* W2q,
                        const uint8_t* W2s, void* Y, hipStream_t st);

}  // namespace moe
