// Reductions inside a wave by register exchange (DPP and the permute-lane swaps) instead of
// shuffles, which go through the LDS crossbar: they stand on the critical path of every row of
// the norms, and the crossbar's throughput bounded the balance loss's backward (20.1 us with
// shuffles, 14.4 without, at 65521 tokens of 96 experts).
#pragma once
#include "common.h"

namespace moe {

template <int CTRL, int ROWS>
__device__ __forceinline__ float dpp(float v) {
  return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, ROWS, 0xF, false));
}

// Sum over the wave, the same in every lane (and known to be): four exchanges inside each row of
// 16 lanes, then the rows' sums passed on to lane 63 and read from there.
__device__ __forceinline__ float wave_total(float v) {
  v += dpp<0xB1, 0xF>(v);   // quad_perm [1,0,3,2]
  v += dpp<0x4E, 0xF>(v);   // quad_perm [2,3,0,1]
  v += dpp<0x141, 0xF>(v);  // row_half_mirror: the other quad of each 8
  v += dpp<0x140, 0xF>(v);  // row_mirror: the other 8 of each 16
  v += dpp<0x142, 0xA>(v);  // row_bcast15 into rows 1 and 3
  v += dpp<0x143, 0xC>(v);  // row_bcast31 into rows 2 and 3
  return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 63));
}

// The value of lane ^ N; for N = 4 a lane of the other quad, which serves a reduction whose quads
// already hold one value each.
template <int N>
__device__ __forceinline__ float other_half(float v) {
  if constexpr (N <= 8) {
    // quad_perm [1,0,3,2], quad_perm [2,3,0,1], row_half_mirror, row_ror:8
    constexpr int ctrl = N == 1 ? 0xB1 : N == 2 ? 0x4E : N == 4 ? 0x141 : 0x128;
    return dpp<ctrl, 0xF>(v);
  } else {
    // swapping the odd halves of one copy with the even halves of another leaves each lane its own
    // value in one of the two and the partner's in the other
    const int x = __float_as_int(v);
    const auto r = N == 16 ? __builtin_amdgcn_permlane16_swap(x, x, false, false)
                           : __builtin_amdgcn_permlane32_swap(x, x, false, false);
    return __int_as_float((threadIdx.x & N) != 0 ? r[0] : r[1]);
  }
}

// Sum over each group of LANES lanes (a power of two), the same in all of them.
template <int LANES, int N = 1>
__device__ __forceinline__ float group_sum(float v) {
  if constexpr (N < LANES) return group_sum<LANES, 2 * N>(v + other_half<N>(v));
  return v;
}

// Between a wave's own writes to LDS and its other lanes' reads: orders them for the compiler (the
// hardware runs a wave's LDS accesses in order, so it costs no instruction).
__device__ __forceinline__ void wave_lds_fence() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

}  // namespace moe
