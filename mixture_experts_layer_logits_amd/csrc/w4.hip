// Expert products with 4-bit weights, for serving: few rows per expert against weights that are read
// once (E experts, k chosen per token; every chosen expert's weights are read for the rows routed to
// it: ettayeb.fr, "Olmo-core 3 ouvre l'entraînement des MoE…", section "Le problème que les MoE n'ont
// jamais tout à fait résolu").
//
// MXFP4 weights: E2M1 codes (0, .5, 1, 1.5, 2, 3, 4, 6 and their negatives, two a byte, the even
// element in the low half) with one power of two per 32 elements of a row.  Each value is a bf16
// number exactly, so the weights widen in registers without a rounding (v_cvt_scalef32_pk_bf16_fp4,
// two elements an instruction) and the bf16 matrix cores multiply them with the unquantised rows,
// summing in fp32: the only roundings are the sums' and the one of each output.  fp32 rows take the
// fp32 matrix cores in the same way.
//
// A tile is 16 weight rows by up to 16 NT routed rows of one expert.  The weights are the matrix
// product's left operand: lane l holds weight row l % 16 and 64 consecutive elements (two blocks, two
// 16-byte loads) of every 256, the block 64 (l / 16) of them; the right operand's lane holds the same
// elements of routed row l % 16.  Which element of the reduction a lane's register stands for is the
// same on both sides, so the order inside a matrix instruction does not matter.  The waves of a
// workgroup share the reduction, 256 elements in turn, and add their sums through LDS in wave order.
#include "lanes.h"
#include "tilemap.h"
#include "w4.h"

namespace moe {
namespace {

// ------------------------------------------------------------------ quantisation
// Exponent s of a block's scale: the smallest with amax <= 6 2^s, not below -126
__device__ __forceinline__ int mx4_scale_exp(float amax) {
  const uint32_t u = __float_as_uint(amax);
  const int s = (int)(u >> 23) - 127 - 2 + ((u & 0x7fffffu) > 0x400000u ? 1 : 0);  // 6 = 1.5 * 2^2
  return s < -126 ? -126 : s;
}

// one thread per block of 32
template <typename T>
__global__ void __launch_bounds__(256) mx4_quantize_kernel(int64_t nblk, const T* __restrict__ src,
                                                           uint8_t* __restrict__ q, uint8_t* __restrict__ s) {
  for (int64_t b = (int64_t)blockIdx.x * 256 + threadIdx.x; b < nblk; b += (int64_t)gridDim.x * 256) {
    float v[4][8];
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 4; i++) {
      load8<T>(src + b * kMx4Block + 8 * i, v[i]);
#pragma unroll
      for (int j = 0; j < 8; j++) {
        const uint32_t m = __float_as_uint(v[i][j]) & 0x7fffffffu;
        top = m > top ? m : top;
      }
    }
    uint32_t w[4] = {0, 0, 0, 0};
    int byte = 255;  // an infinity or NaN: the whole block is NaN
    if (top < 0x7f800000u) {
      const int e = mx4_scale_exp(__uint_as_float(top));
      const float inv = __uint_as_float((uint32_t)(127 - e) << 23);  // e <= 126
      byte = e + 127;
#pragma unroll
      for (int i = 0; i < 4; i++) {
        uint32_t c = 0;
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[i][0] * inv, v[i][1] * inv, 1.f, 0);
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[i][2] * inv, v[i][3] * inv, 1.f, 1);
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[i][4] * inv, v[i][5] * inv, 1.f, 2);
        w[i] = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[i][6] * inv, v[i][7] * inv, 1.f, 3);
      }
    }
    reinterpret_cast<uint4*>(q)[b] = make_uint4(w[0], w[1], w[2], w[3]);
    s[b] = (uint8_t)byte;
  }
}

// ------------------------------------------------------------------ products
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

constexpr int kWaves = 4, kThreads = 64 * kWaves;
constexpr int kChunk = 256;  // elements of the reduction a wave takes at a time
constexpr int kRowsW = 16;   // weight rows of a tile

// 2^s of a scale byte (NaN for 255)
__device__ __forceinline__ float mx4_scale(int byte) {
  return byte == 255 ? __uint_as_float(0x7fc00000u) : __builtin_ldexpf(1.f, byte - 127);
}

// Eight codes as bf16
__device__ __forceinline__ bf16x8 widen_bf16(uint32_t c, float scale) {
  const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, scale, 0);
  const bf16x2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, scale, 1);
  const bf16x2 d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, scale, 2);
  const bf16x2 e = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, scale, 3);
  return bf16x8{a[0], a[1], b[0], b[1], d[0], d[1], e[0], e[1]};
}

struct W4Args {
  int R, K, N, E;           // rows, reduction, weight rows of an expert, experts
  const int* offsets;
  const void* X;            // [R][K]
  const uint8_t *q0, *s0;   // [E][N][K/2], [E][N][K/32]
  const uint8_t *q1, *s1;   // the second projection (gated)
  void* out;                // [R][N]
};

// A lane's 64 elements (two blocks) of one weight row, and of NT routed rows, times each other
template <typename T, int NT>
__device__ __forceinline__ void multiply(const uint4 (&q)[2], const float (&sc)[2], const T* const (&x)[NT],
                                         const bool (&have)[NT], int k, f32x4 (&acc)[NT]) {
#pragma unroll
  for (int b = 0; b < 2; b++) {
    const uint32_t w[4] = {q[b].x, q[b].y, q[b].z, q[b].w};
#pragma unroll
    for (int i = 0; i < 4; i++) {
      if constexpr (sizeof(T) == 2) {
        const bf16x8 a = widen_bf16(w[i], sc[b]);
#pragma unroll
        for (int n = 0; n < NT; n++) {
          uint4 v = make_uint4(0, 0, 0, 0);
          if (have[n]) v = *reinterpret_cast<const uint4*>(x[n] + k + 32 * b + 8 * i);
          acc[n] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, __builtin_bit_cast(bf16x8, v), acc[n], 0, 0, 0);
        }
      } else {
        float v[NT][8];
#pragma unroll
        for (int n = 0; n < NT; n++) {
#pragma unroll
          for (int j = 0; j < 8; j++) v[n][j] = 0.f;
          if (have[n]) load8<float>(x[n] + k + 32 * b + 8 * i, v[n]);
        }
        const f32x2 a[4] = {__builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[i], sc[b], 0),
                            __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[i], sc[b], 1),
                            __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[i], sc[b], 2),
                            __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[i], sc[b], 3)};
#pragma unroll
        for (int j = 0; j < 8; j++)
#pragma unroll
          for (int n = 0; n < NT; n++)
            acc[n] = __builtin_amdgcn_mfma_f32_16x16x4f32(a[j >> 1][j & 1], v[n][j], acc[n], 0, 0, 0);
      }
    }
  }
}

template <typename T, bool GATED, int NT>
__global__ void __launch_bounds__(kThreads) w4_kernel(W4Args p) {
  constexpr int P = GATED ? 2 : 1;  // projections
  constexpr int ROWS = 16 * NT;
  __shared__ int s_map[kMaxExperts + 1];
  __shared__ float s_acc[kWaves][P][ROWS][kRowsW + 1];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int wr = lane & 15, grp = lane >> 4;
  auto seg = [&](int e) { return p.offsets[e]; };
  const int tiles = build_tile_map<Group::M, ROWS, kRowsW, kThreads>(s_map, seg, p.E, p.R, p.N, tid);
  const T* X = static_cast<const T*>(p.X);
  const uint8_t* const qs[2] = {p.q0, p.q1};
  const uint8_t* const ss[2] = {p.s0, p.s1};
  for (int t = blockIdx.x; t < tiles; t += gridDim.x) {
    const TileRange tr = tile_at<Group::M, ROWS, kRowsW, true>(t, s_map, seg, p.E, p.R, p.N, p.K);
    const int64_t wrow = (int64_t)tr.e * p.N + tr.n0 + wr;
    const T* x[NT];
    bool have[NT];
#pragma unroll
    for (int n = 0; n < NT; n++) {
      const int r = tr.m0 + 16 * n + wr;
      have[n] = r < tr.m_end;
      x[n] = X + (int64_t)(have[n] ? r : tr.m0) * p.K;
    }
    f32x4 acc[P][NT] = {};
    for (int k0 = wave * kChunk; k0 < p.K; k0 += kWaves * kChunk) {
      const int k = k0 + 64 * grp;
      const bool in = k < p.K;  // K is a multiple of 64
      bool here[NT];
#pragma unroll
      for (int n = 0; n < NT; n++) here[n] = have[n] && in;
#pragma unroll
      for (int h = 0; h < P; h++) {
        uint4 q[2] = {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
        float sc[2] = {1.f, 1.f};
        if (in) {
          const uint4* src = reinterpret_cast<const uint4*>(qs[h] + wrow * (p.K / 2) + k / 2);
          q[0] = src[0];
          q[1] = src[1];
          const uint32_t two = *reinterpret_cast<const uint16_t*>(ss[h] + wrow * (p.K / kMx4Block) + k / kMx4Block);
          sc[0] = mx4_scale(two & 255);
          sc[1] = mx4_scale(two >> 8);
        }
        multiply<T, NT>(q, sc, x, here, k, acc[h]);
      }
    }
    // lane l holds weight rows 4 (l / 16) .. + 3 of routed row l % 16
#pragma unroll
    for (int h = 0; h < P; h++)
#pragma unroll
      for (int n = 0; n < NT; n++)
#pragma unroll
        for (int i = 0; i < 4; i++) s_acc[wave][h][16 * n + wr][4 * grp + i] = acc[h][n][i];
    __syncthreads();
    for (int o = tid; o < ROWS * kRowsW; o += kThreads) {
      const int r = o / kRowsW, c = o % kRowsW;
      float v[P];
#pragma unroll
      for (int h = 0; h < P; h++) {
        v[h] = s_acc[0][h][r][c];
#pragma unroll
        for (int w = 1; w < kWaves; w++) v[h] += s_acc[w][h][r][c];
      }
      float out = v[0];
      if constexpr (GATED) out = v[0] * sigmoidf_(v[0]) * v[1];
      if (tr.m0 + r < tr.m_end) Elem<T>::store(static_cast<T*>(p.out) + (int64_t)(tr.m0 + r) * p.N + tr.n0 + c, out);
    }
    __syncthreads();  // s_acc is the next tile's too
  }
}

template <typename T, bool GATED>
hipError_t launch_w4(const W4Args& p, hipStream_t st) {
  if (p.R == 0) return hipSuccess;
  const int64_t bound = ((int64_t)p.R / 16 + (p.R < p.E ? p.R : p.E)) * (p.N / kRowsW);
  const int64_t most = (int64_t)device_cu_count() * 64;
  const unsigned grid = (unsigned)(bound < most ? bound : most);
  if (p.R <= 16)
    hipLaunchKernelGGL((w4_kernel<T, GATED, 1>), dim3(grid), dim3(kThreads), 0, st, p);
  else
    hipLaunchKernelGGL((w4_kernel<T, GATED, 2>), dim3(grid), dim3(kThreads), 0, st, p);
  return hipGetLastError();
}

}  // namespace

hipError_t mx4_quantize_rows(int eb, int rows, int cols, const void* src, uint8_t* q, uint8_t* s, hipStream_t st) {
  const int64_t n = (int64_t)rows * (cols / kMx4Block);
  if (n == 0) return hipSuccess;
  const int64_t b = (n + 255) / 256;
  const unsigned grid = (unsigned)(b < (1 << 20) ? b : (1 << 20));
  if (eb == 2)
    hipLaunchKernelGGL(mx4_quantize_kernel<bf16_t>, dim3(grid), dim3(256), 0, st, n, (const bf16_t*)src, q, s);
  else
    hipLaunchKernelGGL(mx4_quantize_kernel<float>, dim3(grid), dim3(256), 0, st, n, (const float*)src, q, s);
  return hipGetLastError();
}

hipError_t gemm1_fwd_w4(int eb, const GemmShape& g, const int* offsets, const void* X, const uint8_t* W1q,
                        const uint8_t* W1s, const uint8_t* W3q, const uint8_t* W3s, void* h, hipStream_t st) {
  const W4Args p{g.R, g.d, g.f, g.E, offsets, X, W1q, W1s, W3q, W3s, h};
  return eb == 2 ? launch_w4<bf16_t, true>(p, st) : launch_w4<float, true>(p, st);
}

hipError_t gemm2_fwd_w4(int eb, const GemmShape& g, const int* offsets, const void* H, const uint8_t* W2q,
                        const uint8_t* W2s, void* Y, hipStream_t st) {
  const W4Args p{g.R, g.f, g.d, g.E, offsets, H, W2q, W2s, nullptr, nullptr, Y};
  return eb == 2 ? launch_w4<bf16_t, false>(p, st) : launch_w4<float, false>(p, st);
}

}  // namespace moe
