// Grouped GEMM on gfx950 matrix cores (bf16 operands, fp32 accumulation).
//
// One kernel template serves every expert GEMM of the layer (and the router GEMMs):
// a grouped GEMM over many small expert computations whose group boundaries live only
// on the device (unite.ai, "Ai2 κυκλοφορεί το Olmo-Core 3…", section "Παραλληλισμός,
// Ακρίβεια και Τεχνικές Μνήμης": grouped GEMM, GPU-resident routing, device-scheduled
// grouped matmuls).  The grid is persistent and sized from host-known shapes only; each
// workgroup rebuilds the tile map from `offsets` in LDS, so the host never learns the
// per-expert counts.
//
//   GROUP_M  rows of A and C are grouped by expert (forward and data-gradient GEMMs):
//            C[r, n] = sum_k A[r, k] * B_e[k, n] for r in [offsets[e], offsets[e+1]).
//   GROUP_K  the reduction is grouped by expert (weight-gradient GEMMs):
//            C_e[m, n] = sum_{r in [offsets[e], offsets[e+1])} A[r, m] * B[r, n].
//
// An operand whose reduction axis is contiguous in memory ("K-contiguous") is kept
// [mn][k] in LDS and read with 16-byte ds_read_b128; an operand contiguous along M or N
// is kept [k][mn] as loaded and read with the gfx950 transpose read ds_read_b64_tr_b16,
// so no operand is ever transposed in HBM.  MFMA: v_mfma_f32_32x32x16_bf16 (lane l holds
// row l%32, k = 8*(l/32)..+7 of A; column l%32 of B; accumulator row 8*(i/4)+4*(l/32)+i%4).
#include "gemm_pipe.h"

namespace moe {

// y_perm = h W2_e^T
struct ProbGemm2 : ProbBase {
  using TA = bf16_t;
  static constexpr Group GROUP = Group::M;
  static constexpr bool A_KC = true, B_KC = true;
  static constexpr Epi EPI = Epi::Store;
  const bf16_t* Hm = nullptr; const bf16_t* W2 = nullptr;
  bf16_t* Y = nullptr;
  __device__ const bf16_t* a_row(int, int m) const { return Hm + (int64_t)m * K; }
  __device__ const bf16_t* b_row(int e, int n) const { return W2 + ((int64_t)e * N + n) * K; }
  static constexpr bool STORE16 = true;
  __device__ bf16_t* out_row(int, int m) const { return Y + (int64_t)m * N; }
  __device__ void epilogue4(int, int m, int n, const float (&v)[4]) const { store_bf16x4(Y + (int64_t)m * N + n, v); }
};

// dW2_e[d, f] = dy_e^T h_e: A[m=d][k=r] = dy[r][d], B[k=r][n=f] = h[r][f]
struct ProbWgrad2 : ProbBase {
  using TA = bf16_t;
  static constexpr Group GROUP = Group::K;
  static constexpr bool A_KC = false, B_KC = false;
  static constexpr Epi EPI = Epi::Store;
  const bf16_t* dY = nullptr; const bf16_t* Hm = nullptr;
  bf16_t* dW2 = nullptr;
  __device__ const bf16_t* a_row(int, int r) const { return dY + (int64_t)r * M; }
  __device__ const bf16_t* b_row(int, int r) const { return Hm + (int64_t)r * N; }
  static constexpr bool STORE16 = true;
  __device__ bf16_t* out_row(int e, int m) const { return dW2 + ((int64_t)e * M + m) * N; }
  __device__ void epilogue4(int e, int m, int n, const float (&v)[4]) const {
    store_bf16x4(dW2 + ((int64_t)e * M + m) * N + n, v);
  }
};

// dx_e = [da | db] [W1_e ; W3_e]: K = 2f, B rows k < f from W1, else W3 (read [k][n=d])
struct ProbDgrad1 : ProbBase {
  using TA = bf16_t;
  static constexpr Group GROUP = Group::M;
  static constexpr bool A_KC = true, B_KC = false;
  static constexpr Epi EPI = Epi::Store;
  int f = 0;
  const bf16_t* dab = nullptr; const bf16_t* W1 = nullptr; const bf16_t* W3 = nullptr;
  bf16_t* dX = nullptr;
  __device__ const bf16_t* a_row(int, int m) const { return dab + (int64_t)m * K; }
  __device__ const bf16_t* b_row(int e, int k) const {
    return k < f ? W1 + ((int64_t)e * f + k) * N : W3 + ((int64_t)e * f + (k - f)) * N;
  }
  static constexpr bool K_SPLIT = true;
  __device__ int k_split() const { return f; }
  static constexpr bool STORE16 = true;
  __device__ bf16_t* out_row(int, int m) const { return dX + (int64_t)m * N; }
  __device__ void epilogue4(int, int m, int n, const float (&v)[4]) const { store_bf16x4(dX + (int64_t)m * N + n, v); }
};

// [dW1_e ; dW3_e] [2f, d] = [da | db]_e^T X_e: A[m][k=r] = dab[r][m], B[k=r][n] = x_perm[r][n]
struct ProbWgrad1 : ProbBase {
  using TA = bf16_t;
  static constexpr Group GROUP = Group::K;
  static constexpr bool A_KC = false, B_KC = false;
  static constexpr Epi EPI = Epi::Store;
  int f = 0;
  const bf16_t* dab = nullptr; const bf16_t* X = nullptr;
  bf16_t* dW1 = nullptr; bf16_t* dW3 = nullptr;
  __device__ const bf16_t* a_row(int, int r) const { return dab + (int64_t)r * M; }
  __device__ const bf16_t* b_row(int, int r) const { return X + (int64_t)r * N; }
  static constexpr bool STORE16 = true;
  __device__ bf16_t* out_row(int e, int m) const {
    return m < f ? dW1 + ((int64_t)e * f + m) * N : dW3 + ((int64_t)e * f + (m - f)) * N;
  }
  __device__ void epilogue4(int e, int m, int n, const float (&v)[4]) const { store_bf16x4(out_row(e, m) + n, v); }
};

// Router scores: logits[t, e] = x[t] . Wr[e] + bias[e]  (single group over T rows)
struct ProbRouterFwd : ProbBase {
  using TA = bf16_t;
  static constexpr Group GROUP = Group::M;
  static constexpr bool A_KC = true, B_KC = true;
  static constexpr Epi EPI = Epi::Store;
  const bf16_t* X = nullptr; const bf16_t* Wr = nullptr; const float* bias = nullptr;
  float* L = nullptr;
  __device__ const bf16_t* a_row(int, int m) const { return X + (int64_t)m * K; }
  __device__ const bf16_t* b_row(int, int n) const { return Wr + (int64_t)n * K; }
  __device__ void epilogue4(int, int m, int n, const float (&v)[4]) const {
#pragma unroll
    for (int c = 0; c < 4; c++)
      if (n + c < N) L[(int64_t)m * N + n + c] = v[c] + (bias ? bias[n + c] : 0.f);
  }
};

// dx_r = dlogits Wr: A = the bf16 copy of dlogits [T][lda] (experts zero-padded to lda),
// B[k=e][n] = Wr[e][n]
struct ProbRouterDx : ProbBase {
  using TA = bf16_t;
  static constexpr Group GROUP = Group::M;
  static constexpr bool A_KC = true, B_KC = false;
  static constexpr Epi EPI = Epi::Store;
  int lda = 0;
  const bf16_t* dL = nullptr; const bf16_t* Wr = nullptr;
  bf16_t* dX = nullptr;
  __device__ const bf16_t* a_row(int, int m) const { return dL + (int64_t)m * lda; }
  __device__ const bf16_t* b_row(int, int k) const { return Wr + (int64_t)k * N; }
  static constexpr bool STORE16 = true;
  __device__ bf16_t* out_row(int, int m) const { return dX + (int64_t)m * N; }
  __device__ void epilogue4(int, int m, int n, const float (&v)[4]) const { store_bf16x4(dX + (int64_t)m * N + n, v); }
};

// Partial router weight gradients: split s of the T rows writes
// part[s][e][i] = sum_{t in split s} dlogits[t, e] x[t, i]; a second kernel sums splits.
struct ProbRouterDwSplit : ProbBase {
  using TA = bf16_t;
  static constexpr Group GROUP = Group::K;
  static constexpr bool A_KC = false, B_KC = false;
  static constexpr Epi EPI = Epi::Store;
  int lda = 0;
  const bf16_t* dL = nullptr; const bf16_t* X = nullptr;
  float* part = nullptr;
  __device__ const bf16_t* a_row(int, int r) const { return dL + (int64_t)r * lda; }
  __device__ const bf16_t* b_row(int, int r) const { return X + (int64_t)r * N; }
  __device__ void epilogue4(int e, int m, int n, const float (&v)[4]) const {
    *reinterpret_cast<float4*>(part + ((int64_t)e * M + m) * N + n) = make_float4(v[0], v[1], v[2], v[3]);
  }
};

// Weight gradient of a single group (E == 1) split over the rows: split s writes
// part[s][m][n] = sum_{r in split s} A[r][m] B[r][n] (A [R][M], B [R][N] bf16)
struct ProbWgradSplit : ProbBase {
  using TA = bf16_t;
  static constexpr Group GROUP = Group::K;
  static constexpr bool A_KC = false, B_KC = false;
  static constexpr Epi EPI = Epi::Store;
  const bf16_t* A = nullptr; const bf16_t* B = nullptr;
  float* part = nullptr;
  __device__ const bf16_t* a_row(int, int r) const { return A + (int64_t)r * M; }
  __device__ const bf16_t* b_row(int, int r) const { return B + (int64_t)r * N; }
  __device__ void epilogue4(int e, int m, int n, const float (&v)[4]) const {
    *reinterpret_cast<float4*>(part + ((int64_t)e * M + m) * N + n) = make_float4(v[0], v[1], v[2], v[3]);
  }
};

namespace {
// out = sum over splits s (in order) of part[s], rounded to bf16; rows m < split_row go
// to O0 + m * N, the others to O1 + (m - split_row) * N.  Four elements per thread.
__global__ void sum_splits_bf16_kernel(int64_t mn, int N, int nsplit, const float* __restrict__ part, int split_row,
                                       bf16_t* __restrict__ O0, bf16_t* __restrict__ O1) {
  const int64_t i = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) * 4;
  if (i >= mn) return;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int s = 0; s < nsplit; s++) {
    const float4 v = *reinterpret_cast<const float4*>(part + (int64_t)s * mn + i);
    acc.x += v.x; acc.y += v.y; acc.z += v.z; acc.w += v.w;
  }
  const int64_t m = i / N, n = i % N;
  bf16_t* o = m < split_row ? O0 + m * N + n : O1 + (m - split_row) * N + n;
  const float a[4] = {acc.x, acc.y, acc.z, acc.w};
  store_bf16x4(o, a);
}

// dlogits [T][E] float -> bf16 [T][lda], experts E..lda-1 zero (round to nearest even, as
// the GEMM operand staging always did)
__global__ void dlogits_bf16_kernel(int T, int E, int lda, const float* __restrict__ src, bf16_t* __restrict__ dst) {
  const int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  if (i >= (int64_t)T * lda) return;
  const int64_t t = i / lda;
  const int e = (int)(i - t * lda);
  dst[i] = e < E ? f2bf(src[t * E + e]) : (bf16_t)0;
}

// dW[i] = sum over splits s (in order) of part[s][i]
__global__ void sum_splits_kernel(int64_t n, int nsplit, const float* __restrict__ part, float* __restrict__ out) {
  const int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  if (i >= n) return;
  float acc = 0.f;
  for (int s = 0; s < nsplit; s++) acc += part[(int64_t)s * n + i];
  out[i] = acc;
}
}  // namespace

template <bool Q>
static hipError_t gemm1_launch(const GemmShape& s, const int* offsets, const bf16_t* X, const bf16_t* W1,
                               const bf16_t* W3, bf16_t* ab, bf16_t* h, uint8_t* hq, uint8_t* hs, hipStream_t st) {
  ProbGemm1T<Q> p;
  p.M = s.R; p.N = 2 * s.f; p.K = s.d; p.E = s.E; p.offsets = offsets; p.f = s.f;
  p.X = X; p.W1 = W1; p.W3 = W3; p.ab = ab; p.h = h; p.hq = hq; p.hs = hs;
  return launch(m_grouped_tile("GEMM1", s, 64), p, st);
}
hipError_t gemm1_fwd_bf16(const GemmShape& s, const int* offsets, const bf16_t* X, const bf16_t* W1,
                          const bf16_t* W3, bf16_t* ab, bf16_t* h, hipStream_t st, uint8_t* hq, uint8_t* hs) {
  if (hq) return gemm1_launch<true>(s, offsets, X, W1, W3, ab, h, hq, hs, st);
  return gemm1_launch<false>(s, offsets, X, W1, W3, ab, h, nullptr, nullptr, st);
}
hipError_t gemm2_fwd_bf16(const GemmShape& s, const int* offsets, const bf16_t* H, const bf16_t* W2, bf16_t* Y,
                          hipStream_t st) {
  ProbGemm2 p;
  p.M = s.R; p.N = s.d; p.K = s.f; p.E = s.E; p.offsets = offsets;
  p.Hm = H; p.W2 = W2; p.Y = Y;
  return launch(m_grouped_tile("GEMM2", s, 64), p, st);
}
// dgrad2 runs with loader waves at every segment length: its epilogue reads the saved a, b
// of every output, and with the compute waves issuing no operand loads those reads wait
// only on each other (at 4096 and 2048 rows per expert 14% and 9% faster than the 256 x 256
// two-stage tiles without them).  Short segments keep 128 x 256 tiles, 64 deep.  Long ones
// (1024 rows per expert or more on average) take 192 x 256 tiles, 32 deep in three stages,
// so each weight block is read by fewer tiles of an expert: alternating runs on one MI355X,
// 0.215 -> 0.192 ms at E = 8, T = 8192 and 0.934 -> 0.907 ms at E = 32, T = 16384, d = 4096;
// at 512 and 256 rows per expert they measured 3% slower and even.  The variant that also
// writes MXFP8 rows of [da | db] keeps the 128 x 256 tiles (on 192 x 256 its epilogue took
// 1.74 ms against 1.02 at E = 32, T = 16384, d = 4096).
template <bool Q>
static hipError_t dgrad2_launch(const GemmShape& s, const int* offsets, const bf16_t* dY, const bf16_t* W2,
                                const bf16_t* ab, bf16_t* dab, uint8_t* dq, uint8_t* ds, hipStream_t st) {
  ProbDgrad2T<Q> p;
  p.M = s.R; p.N = s.f; p.K = s.d; p.E = s.E; p.offsets = offsets;
  p.dY = dY; p.W2 = W2; p.ab = ab; p.dab = dab; p.dq = dq; p.ds = ds;
  if (!Q && (int64_t)s.R >= (int64_t)1024 * s.E)
    return launch(tile_for("DGRAD2", Tile::t192x256w8, 32, 3, 4), p, st);
  return launch(tile_for("DGRAD2", Tile::t128x256w8, 64, 3, 4), p, st);
}
hipError_t dgrad2_bf16(const GemmShape& s, const int* offsets, const bf16_t* dY, const bf16_t* W2,
                       const bf16_t* ab, bf16_t* dab, hipStream_t st, uint8_t* dq, uint8_t* ds) {
  if (dq) return dgrad2_launch<true>(s, offsets, dY, W2, ab, dab, dq, ds, st);
  return dgrad2_launch<false>(s, offsets, dY, W2, ab, dab, nullptr, nullptr, st);
}
// Single-group weight gradients: with one expert the output has few tiles (64 for
// 2048 x 2048 at 256 x 256), so the reduction over the R rows is split to give about two
// tiles per CU of a 256-CU device (splits of at least 512 rows); partial sums go to ws and
// are added in split order.  Host-only arithmetic.
static int wgrad_single_splits(int R, int M, int N) {
  const int tiles = ((M + 255) / 256) * ((N + 255) / 256);
  int s = (512 + tiles - 1) / tiles;
  const int max_s = R / 512;
  if (s > max_s) s = max_s;
  return s < 1 ? 1 : s;
}
size_t wgrad_split_workspace_bytes(const GemmShape& s) {
  if (s.E != 1) return 0;
  const int s1 = wgrad_single_splits(s.R, 2 * s.f, s.d), s2 = wgrad_single_splits(s.R, s.d, s.f);
  const size_t a = s1 > 1 ? (size_t)s1 * 2 * s.f * s.d * sizeof(float) : 0;
  const size_t b = s2 > 1 ? (size_t)s2 * s.d * s.f * sizeof(float) : 0;
  return a > b ? a : b;
}
static hipError_t wgrad_split(int R, int M, int N, int nsplit, const bf16_t* A, const bf16_t* B, float* part,
                              int split_row, bf16_t* O0, bf16_t* O1, hipStream_t st) {
  const int seg_len = (R + nsplit - 1) / nsplit;
  ProbWgradSplit p;
  p.M = M; p.N = N; p.K = R; p.E = (R + seg_len - 1) / seg_len; p.seg_len = seg_len; p.seg_total = R;
  p.A = A; p.B = B; p.part = part;
  hipError_t err = launch(tile_for("WGRAD_SPLIT", Tile::t256x256w8, 32, 4), p, st);
  if (err != hipSuccess) return err;
  const int64_t mn = (int64_t)M * N;
  hipLaunchKernelGGL(sum_splits_bf16_kernel, dim3((unsigned)((mn / 4 + 255) / 256)), dim3(256), 0, st, mn, N, p.E,
                     part, split_row, O0, O1);
  return hipGetLastError();
}

// Weight-gradient tiles: 256 x 256, 32 deep, four stage buffers.  With 512 or more rows per
// expert on average, four loader waves issue every operand load, so the compute waves' gradient
// stores hold back no load wait: 8-10% faster on both weight gradients at 512, 2048 and 4096
// rows per expert (E = 128, T = 16384; E = 32, d = 4096; E = 8); at 256 rows they gain nothing.
static TileChoice wgrad_tile(const char* name, const GemmShape& s) {
  return tile_for(name, Tile::t256x256w8, 32, 4, (int64_t)s.R >= (int64_t)512 * s.E ? 4 : 0);
}

hipError_t wgrad2_bf16(const GemmShape& s, const int* offsets, const bf16_t* H, const bf16_t* dY, bf16_t* dW2,
                       void* ws, hipStream_t st) {
  if (s.E == 1 && ws) {
    const int ns = wgrad_single_splits(s.R, s.d, s.f);
    if (ns > 1) return wgrad_split(s.R, s.d, s.f, ns, dY, H, static_cast<float*>(ws), s.d, dW2, dW2, st);
  }
  ProbWgrad2 p;
  p.M = s.d; p.N = s.f; p.K = s.R; p.E = s.E; p.offsets = offsets;
  p.dY = dY; p.Hm = H; p.dW2 = dW2;
  return launch(wgrad_tile("WGRAD2", s), p, st);
}
// dgrad1 takes 192 x 256 tiles, 32 deep in three stages, with four loader waves, at every
// segment length: each weight block is then read by ceil(rows / 192) tiles of an expert
// instead of ceil(rows / 128), and the compute waves' stores wait on no operand load.
// Against its former tiles (128 x 256 without loaders for short segments, 256 x 256 64 deep
// in two stages for long ones), alternating runs on one MI355X: 0.399 -> 0.393 ms at E = 128,
// T = 8192; 0.669 -> 0.620 at E = 128, T = 16384 (uniform routing); 0.329 -> 0.289 at E = 8;
// 1.626 -> 1.538 at E = 32, T = 16384, d = 4096.
hipError_t dgrad1_bf16(const GemmShape& s, const int* offsets, const bf16_t* dab, const bf16_t* W1,
                       const bf16_t* W3, bf16_t* dX, hipStream_t st) {
  ProbDgrad1 p;
  p.M = s.R; p.N = s.d; p.K = 2 * s.f; p.E = s.E; p.offsets = offsets; p.f = s.f;
  p.dab = dab; p.W1 = W1; p.W3 = W3; p.dX = dX;
  return launch(tile_for("DGRAD1", Tile::t192x256w8, 32, 3, 4), p, st);
}
hipError_t wgrad1_bf16(const GemmShape& s, const int* offsets, const bf16_t* X, const bf16_t* dab, bf16_t* dW1,
                       bf16_t* dW3, void* ws, hipStream_t st) {
  if (s.E == 1 && ws) {
    const int ns = wgrad_single_splits(s.R, 2 * s.f, s.d);
    if (ns > 1) return wgrad_split(s.R, 2 * s.f, s.d, ns, dab, X, static_cast<float*>(ws), s.f, dW1, dW3, st);
  }
  ProbWgrad1 p;
  p.M = 2 * s.f; p.N = s.d; p.K = s.R; p.E = s.E; p.offsets = offsets; p.f = s.f;
  p.dab = dab; p.X = X; p.dW1 = dW1; p.dW3 = dW3;
  return launch(wgrad_tile("WGRAD1", s), p, st);
}
hipError_t router_fwd_bf16(int T, int d, int E, const bf16_t* X, const bf16_t* Wr, const float* bias, float* L,
                           hipStream_t st) {
  ProbRouterFwd p;
  p.M = T; p.N = E; p.K = d; p.E = 1; p.seg_len = T; p.seg_total = T;
  p.X = X; p.Wr = Wr; p.bias = bias; p.L = L;
  return launch(tile_for("ROUTER_FWD", Tile::t32x128, 64, 4), p, st);
}
// Split count of the router weight gradient: about 256 output tiles in flight (one per
// compute unit of a 256-CU device), splits of at least 64 rows.  At T = 8192, d = 2048,
// E = 128 that is 16 splits of 512 rows: the backward took 54.6 us against 61.6 us with
// 32 splits (half the partial sums to write and add).  Host-only arithmetic.
int router_dw_splits(int T, int d, int E) {
  const int tiles = ((E + 127) / 128) * ((d + 127) / 128);
  int s = (256 + tiles - 1) / tiles;
  const int max_s = (T + 63) / 64;
  if (s > max_s) s = max_s;
  return s < 1 ? 1 : s;
}
int router_lda(int E) { return (E + 63) / 64 * 64; }
static size_t al256(size_t b) { return (b + 255) / 256 * 256; }
size_t router_dw_workspace_bytes(int T, int d, int E) {
  return al256((size_t)T * router_lda(E) * sizeof(bf16_t)) + (size_t)router_dw_splits(T, d, E) * E * d * sizeof(float);
}
// dx_r = dlogits Wr (skipped when dX is null) and dWr = dlogits^T x through the bf16 copy of
// dlogits at the start of ws (split partials of dWr after it)
hipError_t router_bwd_bf16(int T, int d, int E, const float* dL, const bf16_t* Wr, const bf16_t* X, bf16_t* dX,
                           float* dW, void* ws, hipStream_t st) {
  const int lda = router_lda(E);
  bf16_t* dLb = static_cast<bf16_t*>(ws);
  float* part = reinterpret_cast<float*>(static_cast<char*>(ws) + al256((size_t)T * lda * sizeof(bf16_t)));
  hipError_t err;
  if (T > 0) {
    const int64_t n = (int64_t)T * lda;
    hipLaunchKernelGGL(dlogits_bf16_kernel, dim3((unsigned)((n + 255) / 256)), dim3(256), 0, st, T, E, lda, dL, dLb);
    if ((err = hipGetLastError()) != hipSuccess) return err;
    if (dX) {  // null: the caller folds dx_r into the un-permute (unpermute_router_rows)
      ProbRouterDx p;
      p.M = T; p.N = d; p.K = E; p.E = 1; p.seg_len = T; p.seg_total = T;
      p.lda = lda; p.dL = dLb; p.Wr = Wr; p.dX = dX;
      if ((err = launch(tile_for("ROUTER_DX", Tile::t128x256w8, 64), p, st)) != hipSuccess) return err;
    }
  }
  int ns = router_dw_splits(T, d, E);
  const int seg_len = ((T + ns - 1) / ns + 63) / 64 * 64;
  ns = T == 0 ? 1 : (T + seg_len - 1) / seg_len;
  ProbRouterDwSplit q;
  q.M = E; q.N = d; q.K = T; q.E = ns; q.seg_len = seg_len; q.seg_total = T;
  q.lda = lda; q.dL = dLb; q.X = X; q.part = ns == 1 ? dW : part;
  if ((err = launch(tile_for("ROUTER_DW", Tile::t128x128, 64), q, st)) != hipSuccess || ns == 1) return err;
  const int64_t n = (int64_t)E * d;
  hipLaunchKernelGGL(sum_splits_kernel, dim3((unsigned)((n + 255) / 256)), dim3(256), 0, st, n, ns, part, dW);
  return hipGetLastError();
}

}  // namespace moe
