// Row kernels of the 8-bit activation checkpoints: rows to MXINT8 and back, the combine that keeps
// the routed rows as MXINT8 while it gathers them, and its backward reading them (what the layer
// keeps between the passes instead of recomputing or holding bf16: activation memory of the training
// step, unite.ai, "Ai2 κυκλοφορεί το Olmo-Core 3…", section "Παραλληλισμός, Ακρίβεια και Τεχνικές
// Μνήμης").
//
// All of them move rows once and are bound by HBM.  A lane takes 8 consecutive elements, so the four
// lanes of a quad hold one block of 32 and its largest magnitude takes two register exchanges.
#include "ckpt8.h"
#include "lanes.h"
#include "mxint8.h"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kTokPerBlock = kThreads / kWave;
constexpr int kMaxGrid = 1 << 20;

// Largest magnitude (NaN wins) over the lane's 8 values and its quad
__device__ __forceinline__ float quad_amax(const float (&v)[8]) {
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < 8; i++) m = ck8_max(m, v[i]);
  m = ck8_max(m, other_half<1>(m));
  return ck8_max(m, other_half<2>(m));
}

__device__ __forceinline__ uint2 encode8(const float (&v)[8], int byte) {
  const float inv = ck8_inv_scale(byte);
  return make_uint2(ck8_codes4(v[0], v[1], v[2], v[3], inv), ck8_codes4(v[4], v[5], v[6], v[7], inv));
}

__device__ __forceinline__ void decode8(const uint2& q, int byte, float (&v)[8]) {
  const float sc = ck8_scale(byte);
  float lo[4], hi[4];
  ck8_values4(q.x, sc, lo);
  ck8_values4(q.y, sc, hi);
#pragma unroll
  for (int i = 0; i < 4; i++) v[i] = lo[i], v[4 + i] = hi[i];
}

// rows of whole blocks are one long run of 8-element chunks (chunk c: elements 8c .. 8c + 7, block c / 4)
template <typename T>
__global__ void __launch_bounds__(kThreads) ck8_pack_kernel(int64_t nchunk, const T* __restrict__ src,
                                                            int8_t* __restrict__ q, uint8_t* __restrict__ s) {
  const int64_t step = (int64_t)gridDim.x * kThreads;  // a multiple of 4: quads stay whole
  for (int64_t c = (int64_t)blockIdx.x * kThreads + threadIdx.x; c < nchunk; c += step) {
    float v[8];
    load8<T>(src + c * 8, v);
    const int byte = ck8_scale_byte(quad_amax(v));
    reinterpret_cast<uint2*>(q)[c] = encode8(v, byte);
    if ((threadIdx.x & 3) == 0) s[c >> 2] = (uint8_t)byte;
  }
}

template <typename T>
__global__ void __launch_bounds__(kThreads) ck8_unpack_kernel(int64_t nchunk, const int8_t* __restrict__ q,
                                                              const uint8_t* __restrict__ s, T* __restrict__ dst) {
  const int64_t step = (int64_t)gridDim.x * kThreads;
  for (int64_t c = (int64_t)blockIdx.x * kThreads + threadIdx.x; c < nchunk; c += step) {
    float v[8];
    decode8(reinterpret_cast<const uint2*>(q)[c], s[c >> 2], v);
    store8<T>(dst + c * 8, v);
  }
}

// [a | b] rows and h = silu(a) b: one thread per 8 columns of h
template <typename T>
__global__ void __launch_bounds__(kThreads) ck8_unpack_swiglu_kernel(int64_t n, int fchunk,
                                                                     const int8_t* __restrict__ q,
                                                                     const uint8_t* __restrict__ s, T* __restrict__ dst,
                                                                     T* __restrict__ h) {
  const int64_t step = (int64_t)gridDim.x * kThreads;
  for (int64_t c = (int64_t)blockIdx.x * kThreads + threadIdx.x; c < n; c += step) {
    const int64_t row = c / fchunk, ca = row * 2 * fchunk + (c - row * fchunk), cb = ca + fchunk;
    float a[8], b[8], hv[8];
    decode8(reinterpret_cast<const uint2*>(q)[ca], s[ca >> 2], a);
    decode8(reinterpret_cast<const uint2*>(q)[cb], s[cb >> 2], b);
    store8<T>(dst + ca * 8, a);
    store8<T>(dst + cb * 8, b);
#pragma unroll
    for (int i = 0; i < 8; i++) hv[i] = a[i] * sigmoidf_(a[i]) * b[i];
    store8<T>(h + c * 8, hv);
  }
}

// y[t] = y_add[t] + sum_j gates[t, j] y_perm[slot_row[t, j]] in the order and arithmetic of the plain
// combine (bit for bit its y); every routed row is read by exactly one token, so its codes are
// written on the way.
template <typename T>
__global__ void __launch_bounds__(kThreads) combine_c8_kernel(int ntok, int d, int k, const T* __restrict__ y_perm,
                                                              const float* __restrict__ gates,
                                                              const int32_t* __restrict__ slot_row,
                                                              const T* __restrict__ y_add, T* __restrict__ y,
                                                              int8_t* __restrict__ yq, uint8_t* __restrict__ ys) {
  const int lane = threadIdx.x & 63;
  const int nchunk = d / 8;
  for (int64_t t = (int64_t)blockIdx.x * kTokPerBlock + (threadIdx.x >> 6); t < ntok;
       t += (int64_t)gridDim.x * kTokPerBlock) {
    for (int c = lane; c < nchunk; c += kWave) {  // nchunk is a multiple of 8: quads stay whole
      float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
      if (y_add) load8<T>(y_add + t * d + c * 8, acc);
      for (int j = 0; j < k; j++) {
        const int64_t r = slot_row[t * k + j];
        const float g = gates[t * k + j];
        float v[8];
        load8<T>(y_perm + r * d + c * 8, v);
        const int byte = ck8_scale_byte(quad_amax(v));
        reinterpret_cast<uint2*>(yq + r * d)[c] = encode8(v, byte);
        if ((lane & 3) == 0) ys[r * (d / kCk8Block) + (c >> 2)] = (uint8_t)byte;
#pragma unroll
        for (int i = 0; i < 8; i++) acc[i] = fmaf(g, v[i], acc[i]);
      }
      store8<T>(y + t * d + c * 8, acc);
    }
  }
}

// In the order and arithmetic of the plain backward (its results, bit for bit, on the kept values).
template <typename T>
__global__ void __launch_bounds__(kThreads) combine_bwd_c8_kernel(int ntok, int d, int k, const T* __restrict__ dy,
                                                                  const int8_t* __restrict__ yq,
                                                                  const uint8_t* __restrict__ ys,
                                                                  const float* __restrict__ gates,
                                                                  const int32_t* __restrict__ slot_row,
                                                                  T* __restrict__ dy_perm, float* __restrict__ dgates) {
  const int lane = threadIdx.x & 63;
  const int nchunk = d / 8;
  for (int64_t t = (int64_t)blockIdx.x * kTokPerBlock + (threadIdx.x >> 6); t < ntok;
       t += (int64_t)gridDim.x * kTokPerBlock) {
    for (int j = 0; j < k; j++) {
      const int64_t r = slot_row[t * k + j];
      const float g = gates[t * k + j];
      float dot = 0.f;
      for (int c = lane; c < nchunk; c += kWave) {
        float u[8], v[8], o[8];
        load8<T>(dy + t * d + c * 8, u);
        decode8(reinterpret_cast<const uint2*>(yq + r * d)[c], ys[r * (d / kCk8Block) + (c >> 2)], v);
#pragma unroll
        for (int i = 0; i < 8; i++) {
          dot = fmaf(u[i], v[i], dot);
          o[i] = g * u[i];
        }
        store8<T>(dy_perm + r * d + c * 8, o);
      }
      dot = wave_sum(dot);
      if (lane == 0) dgates[t * k + j] = dot;
    }
  }
}

inline dim3 grid_for(int64_t n, int per_block) {
  const int64_t b = (n + per_block - 1) / per_block;
  return dim3((unsigned)(b < kMaxGrid ? b : kMaxGrid));
}

}  // namespace

hipError_t ck8_pack_rows(int eb, int rows, int cols, const void* src, int8_t* q, uint8_t* s, hipStream_t st) {
  const int64_t n = (int64_t)rows * (cols / 8);
  if (n == 0) return hipSuccess;
  if (eb == 2)
    hipLaunchKernelGGL(ck8_pack_kernel<bf16_t>, grid_for(n, kThreads), dim3(kThreads), 0, st, n, (const bf16_t*)src, q,
                       s);
  else
    hipLaunchKernelGGL(ck8_pack_kernel<float>, grid_for(n, kThreads), dim3(kThreads), 0, st, n, (const float*)src, q, s);
  return hipGetLastError();
}

hipError_t ck8_unpack_rows(int eb, int rows, int cols, const int8_t* q, const uint8_t* s, void* dst, void* h,
                           hipStream_t st) {
  const int64_t n = (int64_t)rows * (cols / 8);
  if (n == 0) return hipSuccess;
  if (h) {
    if (eb == 2)
      hipLaunchKernelGGL(ck8_unpack_swiglu_kernel<bf16_t>, grid_for(n / 2, kThreads), dim3(kThreads), 0, st, n / 2,
                         cols / 16, q, s, (bf16_t*)dst, (bf16_t*)h);
    else
      hipLaunchKernelGGL(ck8_unpack_swiglu_kernel<float>, grid_for(n / 2, kThreads), dim3(kThreads), 0, st, n / 2,
                         cols / 16, q, s, (float*)dst, (float*)h);
    return hipGetLastError();
  }
  if (eb == 2)
    hipLaunchKernelGGL(ck8_unpack_kernel<bf16_t>, grid_for(n, kThreads), dim3(kThreads), 0, st, n, q, s, (bf16_t*)dst);
  else
    hipLaunchKernelGGL(ck8_unpack_kernel<float>, grid_for(n, kThreads), dim3(kThreads), 0, st, n, q, s, (float*)dst);
  return hipGetLastError();
}

hipError_t combine_rows_c8(int eb, int T, int d, int k, const void* y_perm, const float* gates, const int32_t* slot_row,
                           const void* y_add, void* y, int8_t* yq, uint8_t* ys, hipStream_t st) {
  if (T == 0) return hipSuccess;
  if (eb == 2)
    hipLaunchKernelGGL(combine_c8_kernel<bf16_t>, grid_for(T, kTokPerBlock), dim3(kThreads), 0, st, T, d, k,
                       (const bf16_t*)y_perm, gates, slot_row, (const bf16_t*)y_add, (bf16_t*)y, yq, ys);
  else
    hipLaunchKernelGGL(combine_c8_kernel<float>, grid_for(T, kTokPerBlock), dim3(kThreads), 0, st, T, d, k,
                       (const float*)y_perm, gates, slot_row, (const float*)y_add, (float*)y, yq, ys);
  return hipGetLastError();
}

hipError_t combine_rows_bwd_c8(int eb, int T, int d, int k, const void* dy, const int8_t* yq, const uint8_t* ys,
                               const float* gates, const int32_t* slot_row, void* dy_perm, float* dgates,
                               hipStream_t st) {
  if (T == 0) return hipSuccess;
  if (eb == 2)
    hipLaunchKernelGGL(combine_bwd_c8_kernel<bf16_t>, grid_for(T, kTokPerBlock), dim3(kThreads), 0, st, T, d, k,
                       (const bf16_t*)dy, yq, ys, gates, slot_row, (bf16_t*)dy_perm, dgates);
  else
    hipLaunchKernelGGL(combine_bwd_c8_kernel<float>, grid_for(T, kTokPerBlock), dim3(kThreads), 0, st, T, d, k,
                       (const float*)dy, yq, ys, gates, slot_row, (float*)dy_perm, dgates);
  return hipGetLastError();
}

}  // namespace moe
