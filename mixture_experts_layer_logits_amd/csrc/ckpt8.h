// Internal declarations: 8-bit activation checkpoints (MXINT8 rows: codes [rows][cols], one scale
// byte per 32 columns [rows][cols / 32]).
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>
#include "common.h"
#include "gemm.h"
#include "mxint8.h"

namespace moe {

// elem_bytes: 2 (bf16) or 4 (float)
hipError_t ck8_pack_rows(int elem_bytes, int rows, int cols, const void* src, int8_t* q, uint8_t* s, hipStream_t st);
// h (optional, cols = 2f): silu(first half) * second half of each row
hipError_t ck8_unpack_rows(int elem_bytes, int rows, int cols, const int8_t* q, const uint8_t* s, void* dst, void* h,
                           hipStream_t st);
// moe_combine, with the gathered rows also written as MXINT8
hipError_t combine_rows_c8(int elem_bytes, int T, int d, int k, const void* y_perm, const float* gates,
                           const int32_t* slot_row, const void* y_add, void* y, int8_t* yq, uint8_t* ys,
                           hipStream_t st);
// moe_combine_bwd with the gathered rows read as MXINT8
hipError_t combine_rows_bwd_c8(int elem_bytes, int T, int d, int k, const void* dy, const int8_t* yq,
                               const uint8_t* ys, const float* gates, const int32_t* slot_row, void* dy_perm,
                               float* dgates, hipStream_t st);

// GEMM1 whose epilogue writes [a | b] as MXINT8 instead of bf16; dgrad2 whose epilogue reads it and
// writes h again beside [da | db]
hipError_t gemm1_fwd_c8_bf16(const GemmShape& s, const int* offsets, const bf16_t* X, const bf16_t* W1,
                             const bf16_t* W3, bf16_t* h, int8_t* abq, uint8_t* ab_s, hipStream_t st);
hipError_t dgrad2_c8_bf16(const GemmShape& s, const int* offsets, const bf16_t* dY, const bf16_t* W2,
                          const int8_t* abq, const uint8_t* ab_s, bf16_t* dab, bf16_t* h, hipStream_t st);

}  // namespace moe
