// Row kernels of the 8-bit activation checkpoints: rows to MXINT8 and back, the combine that keeps
// the routed rows as MXINT8 while it gathers them, and its backward reading them (what the layer
// keeps between the passes instead of recomputing or holding bf16: activation memory of the training
// step, unite.ai, "Ai2 κυκλοφορεί το Olmo-Core 3…", section "Παραλληλισμός, Ακρίβεια και Τεχνικές
// Μνήμης").
//
// All of them move rows once and are bound by HBM.  A lane takes 8 consecutive elements, so the four
// lanes of a quad hold one block of 32 and its largest magnitude takes two register exchanges.  32768 x
// 2048 in bf16: pack 30 us (6.8 TB/s read and written), unpack 32 to 35 us (5.8 to 6.3); combine of T = 8192, k = 4
// 52 us (271 MB, 5.2 TB/s; the plain combine 41); its backward at T = 16384, d = 4096 183 us (949 MB, 5.2 TB/s).
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

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

// Eight elements as loaded; load_last: by their last reader (they leave the caches to what comes next:
// 62 -> 57 us for the combine of T = 8192, k = 4, d = 2048)
template <typename T> struct Raw8;
template <> struct Raw8<bf16_t> {
  u32x4 q;
  __device__ __forceinline__ void load(const bf16_t* p) { q = *reinterpret_cast<const u32x4*>(p); }
  __device__ __forceinline__ void load_last(const bf16_t* p) {
    q = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(p));
  }
  __device__ __forceinline__ void zero() { q = u32x4{0, 0, 0, 0}; }
  __device__ __forceinline__ void widen(float (&v)[8]) const {
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 4; i++) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
};
template <> struct Raw8<float> {
  f32x4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = reinterpret_cast<const f32x4*>(p)[0];
    b = reinterpret_cast<const f32x4*>(p)[1];
  }
  __device__ __forceinline__ void load_last(const float* p) {
    a = __builtin_nontemporal_load(reinterpret_cast<const f32x4*>(p));
    b = __builtin_nontemporal_load(reinterpret_cast<const f32x4*>(p) + 1);
  }
  __device__ __forceinline__ void zero() { a = b = f32x4{0.f, 0.f, 0.f, 0.f}; }
  __device__ __forceinline__ void widen(float (&v)[8]) const {
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  }
};

// A wave a token, whose rows and gates the lanes hold and pass on; U chunks of all k (up to KG) rows are
// loaded before any arithmetic (U = 4: 106 us against 112 with 2, at T = 8192, k = 4, d = 2048 with the
// unpack behind it).  KG = 0: any k, a row at a time.
//
// y[t] = y_add[t] + sum_j gates[t, j] y_perm[slot_row[t, j]] in the order and arithmetic of the plain
// combine (bit for bit its y); every routed row is read by exactly one token, so its codes are
// written on the way.  blockIdx.y: parts of the row, which do not depend on each other.
template <typename T, int KG, int U>
__global__ void __launch_bounds__(kThreads) combine_c8_kernel(int ntok, int d, int k, const T* __restrict__ y_perm,
                                                              const float* __restrict__ gates,
                                                              const int32_t* __restrict__ slot_row,
                                                              const T* __restrict__ y_add, T* __restrict__ y,
                                                              int8_t* __restrict__ yq, uint8_t* __restrict__ ys) {
  const int lane = threadIdx.x & 63;
  const int nchunk = d / 8;  // a multiple of 8: quads stay whole
  auto encode = [&](const float (&v)[8], int64_t r, int c) __attribute__((always_inline)) {
    const int byte = ck8_scale_byte(quad_amax(v));
    const uint2 w = encode8(v, byte);
    // read again only in the backward (111 -> 105 us with the unpack behind it)
    __builtin_nontemporal_store((uint64_t)w.y << 32 | w.x, reinterpret_cast<uint64_t*>(yq + r * d) + c);
    if ((lane & 3) == 0) ys[r * (d / kCk8Block) + (c >> 2)] = (uint8_t)byte;
  };
  for (int64_t t = (int64_t)blockIdx.x * kTokPerBlock + (threadIdx.x >> 6); t < ntok;
       t += (int64_t)gridDim.x * kTokPerBlock) {
    const int my_r = lane < k ? slot_row[t * k + lane] : 0;
    const float my_g = lane < k ? gates[t * k + lane] : 0.f;
    for (int c0 = blockIdx.y * U * kWave + lane; c0 < nchunk; c0 += gridDim.y * U * kWave) {
      if constexpr (KG > 0) {
        Raw8<T> q[U][KG + 1];
#pragma unroll
        for (int u = 0; u < U; u++) {
          const int c = c0 + u * kWave;
          q[u][KG].zero();
          if (y_add && c < nchunk) q[u][KG].load(y_add + t * d + c * 8);
#pragma unroll
          for (int j = 0; j < KG; j++) {
            const int64_t r = __builtin_amdgcn_readlane(my_r, j);
            if (j < k && c < nchunk) q[u][j].load_last(y_perm + r * d + c * 8);
          }
        }
#pragma unroll
        for (int u = 0; u < U; u++) {
          const int c = c0 + u * kWave;
          if (c < nchunk) {
            float acc[8];
            q[u][KG].widen(acc);
#pragma unroll
            for (int j = 0; j < KG; j++) {
              if (j < k) {
                const float g = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(my_g), j));
                float v[8];
                q[u][j].widen(v);
                encode(v, __builtin_amdgcn_readlane(my_r, j), c);
#pragma unroll
                for (int i = 0; i < 8; i++) acc[i] = fmaf(g, v[i], acc[i]);
              }
            }
            store8<T>(y + t * d + c * 8, acc);
          }
        }
      } else {
        float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        if (y_add) load8<T>(y_add + t * d + c0 * 8, acc);
        for (int j = 0; j < k; j++) {
          const int64_t r = __builtin_amdgcn_readlane(my_r, j);
          const float g = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(my_g), j));
          float v[8];
          load8<T>(y_perm + r * d + c0 * 8, v);
          encode(v, r, c0);
#pragma unroll
          for (int i = 0; i < 8; i++) acc[i] = fmaf(g, v[i], acc[i]);
        }
        store8<T>(y + t * d + c0 * 8, acc);
      }
    }
  }
}

// In the order and arithmetic of the plain backward (its results, bit for bit, on the kept values).  A
// wave a routed slot: the k waves that share a token's dy read it from the caches (184 us at T = 16384, k =
// 4, d = 4096, against 195 for a wave a token; 12.9 against 16.5 at T = 1531, k = 6, d = 1088 in fp32).
template <typename T, int U>
__global__ void __launch_bounds__(kThreads) combine_bwd_c8_kernel(int64_t nslot, int d, int k, const T* __restrict__ dy,
                                                                  const int8_t* __restrict__ yq,
                                                                  const uint8_t* __restrict__ ys,
                                                                  const float* __restrict__ gates,
                                                                  const int32_t* __restrict__ slot_row,
                                                                  T* __restrict__ dy_perm, float* __restrict__ dgates) {
  const int lane = threadIdx.x & 63;
  const int nchunk = d / 8;
  for (int64_t i = (int64_t)blockIdx.x * kTokPerBlock + (threadIdx.x >> 6); i < nslot;
       i += (int64_t)gridDim.x * kTokPerBlock) {
    const int64_t t = i / k, r = slot_row[i];
    const float g = gates[i];
    float dot = 0.f;
    for (int c0 = lane; c0 < nchunk; c0 += U * kWave) {
      Raw8<T> e[U];
      uint2 q[U];
      int s[U];
#pragma unroll
      for (int u = 0; u < U; u++) {
        const int c = c0 + u * kWave;
        if (c < nchunk) {
          e[u].load(dy + t * d + c * 8);
          q[u] = reinterpret_cast<const uint2*>(yq + r * d)[c];
          s[u] = ys[r * (d / kCk8Block) + (c >> 2)];
        }
      }
#pragma unroll
      for (int u = 0; u < U; u++) {
        const int c = c0 + u * kWave;
        if (c < nchunk) {
          float x[8], v[8], o[8];
          e[u].widen(x);
          decode8(q[u], s[u], v);
#pragma unroll
          for (int n = 0; n < 8; n++) {
            dot = fmaf(x[n], v[n], dot);
            o[n] = g * x[n];
          }
          store8<T>(dy_perm + r * d + c * 8, o);
        }
      }
    }
    dot = wave_sum(dot);
    if (lane == 0) dgates[i] = dot;
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

template <typename T>
static hipError_t combine_c8(int T_, int d, int k, const T* y_perm, const float* gates, const int32_t* slot_row,
                             const T* y_add, T* y, int8_t* yq, uint8_t* ys, hipStream_t st) {
  constexpr int U = sizeof(T) == 2 ? 4 : 2;  // fp32 rows take twice the registers
  // few tokens: the parts of a row to a wave each, up to what the waves of the device hold
  const int parts = (d / 8 + U * kWave - 1) / (U * kWave);
  const dim3 grid(grid_for(T_, kTokPerBlock).x, T_ * (int64_t)parts <= 4096 ? parts : 1);
  if (k <= 4)
    hipLaunchKernelGGL((combine_c8_kernel<T, 4, U>), grid, dim3(kThreads), 0, st, T_, d, k, y_perm, gates, slot_row,
                       y_add, y, yq, ys);
  else if (k <= 8)
    hipLaunchKernelGGL((combine_c8_kernel<T, 8, U / 2>), grid, dim3(kThreads), 0, st, T_, d, k, y_perm, gates, slot_row,
                       y_add, y, yq, ys);
  else
    hipLaunchKernelGGL((combine_c8_kernel<T, 0, 1>), grid, dim3(kThreads), 0, st, T_, d, k, y_perm, gates, slot_row,
                       y_add, y, yq, ys);
  return hipGetLastError();
}

hipError_t combine_rows_c8(int eb, int T, int d, int k, const void* y_perm, const float* gates, const int32_t* slot_row,
                           const void* y_add, void* y, int8_t* yq, uint8_t* ys, hipStream_t st) {
  if (T == 0) return hipSuccess;
  if (eb == 2)
    return combine_c8(T, d, k, (const bf16_t*)y_perm, gates, slot_row, (const bf16_t*)y_add, (bf16_t*)y, yq, ys, st);
  return combine_c8(T, d, k, (const float*)y_perm, gates, slot_row, (const float*)y_add, (float*)y, yq, ys, st);
}

template <typename T>
static hipError_t combine_bwd_c8(int T_, int d, int k, const T* dy, const int8_t* yq, const uint8_t* ys,
                                 const float* gates, const int32_t* slot_row, T* dy_perm, float* dgates,
                                 hipStream_t st) {
  const int64_t n = (int64_t)T_ * k;
  hipLaunchKernelGGL((combine_bwd_c8_kernel<T, 4>), grid_for(n, kTokPerBlock), dim3(kThreads), 0, st, n, d, k, dy, yq,
                     ys, gates, slot_row, dy_perm, dgates);
  return hipGetLastError();
}

hipError_t combine_rows_bwd_c8(int eb, int T, int d, int k, const void* dy, const int8_t* yq, const uint8_t* ys,
                               const float* gates, const int32_t* slot_row, void* dy_perm, float* dgates,
                               hipStream_t st) {
  if (T == 0) return hipSuccess;
  if (eb == 2) return combine_bwd_c8(T, d, k, (const bf16_t*)dy, yq, ys, gates, slot_row, (bf16_t*)dy_perm, dgates, st);
  return combine_bwd_c8(T, d, k, (const float*)dy, yq, ys, gates, slot_row, (float*)dy_perm, dgates, st);
}

}  // namespace moe
