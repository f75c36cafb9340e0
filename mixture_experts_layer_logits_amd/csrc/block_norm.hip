// Norms before and after a block, with the block's gate and residual scale, and the layer's
// combine fused with them; forward and backward.
//
//   r(z) = 1 / sqrt(mean(z^2) + eps)
//   v[t]  = x[t] + a g_t (y[t] r(y[t]) w_post)        the residual sum (a: residual scale)
//   xn[t] = v[t] r(v[t]) w_pre                        the next block's input
// backward, with vh = v r_v, yh = y r_y and D the gradient of v from both of its uses:
//   D  = dv + r_v (w_pre dxn - vh mean(vh w_pre dxn));  dx = D
//   dy = a g (r_y (w_post D - yh mean(yh w_post D)));   dgate = a sum(D w_post yh)
//   dw_post = a sum_t g D yh;  dw_pre = sum_t dxn vh
// The combine supplies y[t] = y_add[t] + sum_j gates[t, j] y_perm[slot_row[t, j]] without storing
// it; its backward gathers the k rows again (the gate gradients need them anyway), rebuilds y, and
// writes dy_perm[slot_row[t, j]] = gates[t, j] dy[t] and dgates[t, j] = <dy[t], y_perm[..]>.
//
// HBM-bound: every row is read once and written once.  A row is held in the registers of WPR
// waves, 8 consecutive columns per 16-byte load and C such chunks per lane; row sums are float
// butterflies over the wave, then over the WPR waves through LDS.  Rows and weights round to
// the element type once, at the store: xn is taken from the unrounded v, dy from the unrounded D.
// Weight gradients accumulate in registers over a workgroup's rows, meet across its waves in
// LDS, go to one partial row per workgroup and are added by a second launch, all in a fixed
// order (no atomics).
#include "block.h"
#include "gemm.h"

namespace moe {
namespace {

enum Src { kNone = 0, kLoad = 1, kGather = 2 };  // the branch y: absent, read, gathered from routed rows

// Sums over the WPR waves of a row.  Consecutive sums alternate between two LDS buffers, so one
// barrier each is enough: a buffer is written again only after a later barrier.
template <int WPR, int NWAVES>
struct RowSum {
  float (*buf)[NWAVES];
  int at = 0;
  __device__ __forceinline__ float operator()(float v) {
    v = wave_sum(v);
    if constexpr (WPR > 1) {
      const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
      if (lane == 0) buf[at][wave] = v;
      __syncthreads();
      const int w0 = wave / WPR * WPR;
      v = 0.f;
#pragma unroll
      for (int w = 0; w < WPR; w++) v += buf[at][w0 + w];
      at ^= 1;
    }
    return v;
  }
};

template <int C>
__device__ __forceinline__ void zero(float (&v)[C][8]) {
#pragma unroll
  for (int i = 0; i < C; i++)
#pragma unroll
    for (int c = 0; c < 8; c++) v[i][c] = 0.f;
}

template <int C>
__device__ __forceinline__ float dot(const float (&a)[C][8], const float (&b)[C][8]) {
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < C; i++)
#pragma unroll
    for (int c = 0; c < 8; c++) s = fmaf(a[i][c], b[i][c], s);
  return s;
}

// A lane's share of a row: chunks first + i * step (i < C) of 8 columns, those below nchunk
template <typename T, int C>
struct Lane {
  int first, step, nchunk;
  __device__ __forceinline__ void load(const T* row, float (&v)[C][8]) const {
#pragma unroll
    for (int i = 0; i < C; i++)
      if (first + i * step < nchunk) load8<T>(row + (first + i * step) * 8, v[i]);
  }
  __device__ __forceinline__ void store(T* row, const float (&v)[C][8]) const {
#pragma unroll
    for (int i = 0; i < C; i++)
      if (first + i * step < nchunk) store8<T>(row + (first + i * step) * 8, v[i]);
  }
};

// y[t] = y_add[t] + sum_j gates[t, j] y_perm[slot_row[t, j]], j in order
template <typename T, int C>
__device__ __forceinline__ void gather(const Lane<T, C>& ln, int64_t t, int d, int k, const T* y_perm, const T* y_add,
                                       const float* gates, const int32_t* slot_row, float (&y)[C][8]) {
  zero(y);
  if (y_add) ln.load(y_add + t * d, y);
  for (int j = 0; j < k; j++) {
    const float g = gates[t * k + j];
    float r[C][8];
    zero(r);
    ln.load(y_perm + (int64_t)slot_row[t * k + j] * d, r);
#pragma unroll
    for (int i = 0; i < C; i++)
#pragma unroll
      for (int c = 0; c < 8; c++) y[i][c] = fmaf(g, r[i][c], y[i][c]);
  }
}

template <typename T, int WPR, int C, int NWAVES, int SRC>
__global__ void __launch_bounds__(NWAVES * 64) norm_fwd_kernel(const NormFwd a) {
  constexpr int RPB = NWAVES / WPR;
  __shared__ float s_red[2][NWAVES];
  RowSum<WPR, NWAVES> row_sum{s_red};
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const Lane<T, C> ln{(wave % WPR) * kWave + lane, WPR * kWave, a.d / 8};
  const float inv_d = 1.f / (float)a.d;
  for (int64_t base = (int64_t)blockIdx.x * RPB; base < a.T; base += (int64_t)gridDim.x * RPB) {
    const int64_t t = base + wave / WPR;
    const bool in = t < a.T;
    float v[C][8];
    zero(v);
    if (in) ln.load(static_cast<const T*>(a.x) + t * a.d, v);
    if constexpr (SRC != kNone) {
      float y[C][8];
      zero(y);
      if (in) {
        if constexpr (SRC == kLoad) ln.load(static_cast<const T*>(a.y) + t * a.d, y);
        else
          gather<T, C>(ln, t, a.d, a.k, static_cast<const T*>(a.y_perm), static_cast<const T*>(a.y_add), a.gates,
                       a.slot_row, y);
      }
      const float g = a.gate && in ? a.gate[t] : 1.f;
      float coef = a.res_scale * g;
      if (a.w_post) {
        const float r = rsqrtf(row_sum(dot(y, y)) * inv_d + a.eps);
        coef *= r;
        if (in && ln.first == 0) a.rstd_post[t] = r;
      }
      if (g != 0.f) {  // a closed gate drops the branch, whatever it holds
        float w[C][8];
        zero(w);  // columns past the row must stay zero: they enter the next row sum
        if (a.w_post) ln.load(static_cast<const T*>(a.w_post), w);
#pragma unroll
        for (int i = 0; i < C; i++)
#pragma unroll
          for (int c = 0; c < 8; c++) v[i][c] = fmaf(coef * y[i][c], a.w_post ? w[i][c] : 1.f, v[i][c]);
      }
      if (in) ln.store(static_cast<T*>(a.v) + t * a.d, v);
    }
    if (a.w_pre) {
      const float r = rsqrtf(row_sum(dot(v, v)) * inv_d + a.eps);
      if (in) {
        float w[C][8];
        ln.load(static_cast<const T*>(a.w_pre), w);
#pragma unroll
        for (int i = 0; i < C; i++)
#pragma unroll
          for (int c = 0; c < 8; c++) v[i][c] = v[i][c] * r * w[i][c];
        ln.store(static_cast<T*>(a.xn) + t * a.d, v);
        if (ln.first == 0) a.rstd_pre[t] = r;
      }
    }
  }
}

template <typename T, int WPR, int C, int NWAVES, int SRC>
__global__ void __launch_bounds__(NWAVES * 64) norm_bwd_kernel(const NormBwd a) {
  constexpr int RPB = NWAVES / WPR;
  __shared__ float s_red[2][NWAVES];
  __shared__ float s_acc[RPB > 1 ? NWAVES * kWave * 8 : 1];
  RowSum<WPR, NWAVES> row_sum{s_red};
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const Lane<T, C> ln{(wave % WPR) * kWave + lane, WPR * kWave, a.d / 8};
  const float inv_d = 1.f / (float)a.d;
  float acc_pre[C][8], acc_post[C][8];
  zero(acc_pre);
  zero(acc_post);
  for (int64_t base = (int64_t)blockIdx.x * RPB; base < a.T; base += (int64_t)gridDim.x * RPB) {
    const int64_t t = base + wave / WPR;
    const bool in = t < a.T;
    float D[C][8];
    zero(D);
    if (in && a.dv) ln.load(static_cast<const T*>(a.dv) + t * a.d, D);
    if (a.w_pre) {
      float vh[C][8], u[C][8], w[C][8];
      zero(vh);
      zero(u);
      zero(w);
      if (in) {
        ln.load(static_cast<const T*>(a.v) + t * a.d, vh);
        ln.load(static_cast<const T*>(a.dxn) + t * a.d, u);
        ln.load(static_cast<const T*>(a.w_pre), w);
      }
      const float r = in ? a.rstd_pre[t] : 0.f;
#pragma unroll
      for (int i = 0; i < C; i++)
#pragma unroll
        for (int c = 0; c < 8; c++) {
          vh[i][c] *= r;
          acc_pre[i][c] = fmaf(u[i][c], vh[i][c], acc_pre[i][c]);
          u[i][c] *= w[i][c];
        }
      const float m = row_sum(dot(vh, u)) * inv_d;
#pragma unroll
      for (int i = 0; i < C; i++)
#pragma unroll
        for (int c = 0; c < 8; c++) D[i][c] = fmaf(r, fmaf(-m, vh[i][c], u[i][c]), D[i][c]);
    }
    float y[C][8];
    if constexpr (SRC != kNone) {
      zero(y);
      if (in) {
        if constexpr (SRC == kLoad) ln.load(static_cast<const T*>(a.y) + t * a.d, y);
        else
          gather<T, C>(ln, t, a.d, a.k, static_cast<const T*>(a.y_perm), static_cast<const T*>(a.y_add), a.gates,
                       a.slot_row, y);
      }
    }
    if (in) ln.store(static_cast<T*>(a.dx) + t * a.d, D);
    if constexpr (SRC != kNone) {
      const float g = a.gate && in ? a.gate[t] : 1.f;
      const bool open = g != 0.f;
      const float ag = a.res_scale * g;
      if (a.w_post) {
        const float r = in ? a.rstd_post[t] : 0.f;
        float w[C][8];
        zero(w);
        ln.load(static_cast<const T*>(a.w_post), w);
#pragma unroll
        for (int i = 0; i < C; i++)
#pragma unroll
          for (int c = 0; c < 8; c++) {
            y[i][c] *= r;
            if (open) acc_post[i][c] = fmaf(ag * D[i][c], y[i][c], acc_post[i][c]);
            D[i][c] *= w[i][c];
          }
        const float s = row_sum(dot(D, y));
        if (in && a.dgate && ln.first == 0) a.dgate[t] = a.res_scale * s;
        const float m = s * inv_d, ar = ag * r;
#pragma unroll
        for (int i = 0; i < C; i++)
#pragma unroll
          for (int c = 0; c < 8; c++) D[i][c] = open ? ar * fmaf(-m, y[i][c], D[i][c]) : 0.f;
      } else {
        if (a.dgate) {
          const float s = row_sum(dot(D, y));
          if (in && ln.first == 0) a.dgate[t] = a.res_scale * s;
        }
#pragma unroll
        for (int i = 0; i < C; i++)
#pragma unroll
          for (int c = 0; c < 8; c++) D[i][c] = open ? ag * D[i][c] : 0.f;
      }
      if (in && a.dy) ln.store(static_cast<T*>(a.dy) + t * a.d, D);
      if constexpr (SRC == kGather) {
        for (int j = 0; j < a.k; j++) {
          float p[C][8];
          zero(p);
          if (in) {
            const int64_t row = (int64_t)a.slot_row[t * a.k + j] * a.d;
            ln.load(static_cast<const T*>(a.y_perm) + row, p);
            const float gj = a.gates[t * a.k + j];
            float o[C][8];
#pragma unroll
            for (int i = 0; i < C; i++)
#pragma unroll
              for (int c = 0; c < 8; c++) o[i][c] = gj * D[i][c];
            ln.store(static_cast<T*>(a.dy_perm) + row, o);
          }
          const float s = row_sum(dot(D, p));
          if (in && ln.first == 0) a.dgates[t * a.k + j] = s;
        }
      }
    }
  }
  // weight-gradient partials: the workgroup's RPB rows of waves in order, then one row per
  // workgroup of part [2][G][d] (dw_post, dw_pre)
  auto reduce = [&](float (&acc)[C][8], float* out) {
#pragma unroll
    for (int i = 0; i < C; i++) {
      float sum[8];
      if constexpr (RPB > 1) {
        __syncthreads();
        float* mine = s_acc + (wave * kWave + lane) * 8;
#pragma unroll
        for (int c = 0; c < 8; c++) mine[c] = acc[i][c];
        __syncthreads();
        if (wave < WPR) {
#pragma unroll
          for (int c = 0; c < 8; c++) sum[c] = 0.f;
          for (int r = 0; r < RPB; r++)
#pragma unroll
            for (int c = 0; c < 8; c++) sum[c] += s_acc[((r * WPR + wave) * kWave + lane) * 8 + c];
        }
      } else {
#pragma unroll
        for (int c = 0; c < 8; c++) sum[c] = acc[i][c];
      }
      const int chunk = ln.first + i * ln.step;
      if (wave < WPR && chunk < ln.nchunk) store8<float>(out + chunk * 8, sum);
    }
  };
  if (a.dw_post) reduce(acc_post, a.part + (int64_t)blockIdx.x * a.d);
  if (a.dw_pre) reduce(acc_pre, a.part + ((int64_t)gridDim.x + blockIdx.x) * a.d);
}

// dw[c] = sum over the G workgroups, in order, of part[g][c]: 64 columns per workgroup, 16 runs
// of rows that meet in LDS.  blockIdx.y: dw_post, dw_pre.
__global__ void __launch_bounds__(1024) norm_dw_kernel(int d, int G, const float* __restrict__ part,
                                                       float* __restrict__ dw_post, float* __restrict__ dw_pre) {
  __shared__ float s[16][64];
  float* out = blockIdx.y == 0 ? dw_post : dw_pre;
  if (!out) return;
  const int lane = threadIdx.x & 63, run = threadIdx.x >> 6;
  const int col = blockIdx.x * 64 + lane;
  const float* p = part + (int64_t)blockIdx.y * G * d + col;
  float sum = 0.f;
  for (int g = run; g < G; g += 16) sum += p[(int64_t)g * d];
  s[run][lane] = sum;
  __syncthreads();
  if (run == 0) {
    sum = 0.f;
#pragma unroll
    for (int r = 0; r < 16; r++) sum += s[r][lane];
    out[col] = sum;
  }
}

// Calls f(WPR, C, NWAVES) with the waves per row, chunks per lane and waves per workgroup that
// hold a row of d.
template <class F>
hipError_t for_width(int d, F&& f) {
#define MOE_NORM_CASE(WPR, C, NWAVES)                                                                \
  if (d <= WPR * C * 512)                                                                            \
    return f(std::integral_constant<int, WPR>{}, std::integral_constant<int, C>{}, std::integral_constant<int, NWAVES>{});
  MOE_NORM_CASE(1, 1, 4) MOE_NORM_CASE(1, 2, 4) MOE_NORM_CASE(2, 2, 4) MOE_NORM_CASE(4, 2, 4) MOE_NORM_CASE(8, 2, 8)
  MOE_NORM_CASE(16, 2, 16)
#undef MOE_NORM_CASE
  return hipErrorInvalidValue;
}

// one pass of rows per workgroup; more rows than a launch holds threads for go round again
constexpr int64_t kNormFwdBlocks = 1 << 20;

template <typename T>
hipError_t fwd_t(const NormFwd& a, hipStream_t st) {
  return for_width(a.d, [&](auto wpr, auto c, auto nw) {
    constexpr int RPB = nw() / wpr();
    const int64_t rows = ((int64_t)a.T + RPB - 1) / RPB;
    const dim3 grid((unsigned)(rows < kNormFwdBlocks ? rows : kNormFwdBlocks)), block(nw() * 64);
    if (a.y_perm) hipLaunchKernelGGL((norm_fwd_kernel<T, wpr(), c(), nw(), kGather>), grid, block, 0, st, a);
    else if (a.y) hipLaunchKernelGGL((norm_fwd_kernel<T, wpr(), c(), nw(), kLoad>), grid, block, 0, st, a);
    else hipLaunchKernelGGL((norm_fwd_kernel<T, wpr(), c(), nw(), kNone>), grid, block, 0, st, a);
    return hipGetLastError();
  });
}

int bwd_grid(int T, int rpb) {
  const int64_t g = ((int64_t)T + rpb - 1) / rpb;
  return (int)(g < kNormBlocks ? g : kNormBlocks);
}

template <typename T>
hipError_t bwd_t(const NormBwd& a, hipStream_t st) {
  int G = 0;
  const hipError_t err = for_width(a.d, [&](auto wpr, auto c, auto nw) {
    G = bwd_grid(a.T, nw() / wpr());
    if (G == 0) return hipSuccess;
    const dim3 grid(G), block(nw() * 64);
    if (a.y_perm) hipLaunchKernelGGL((norm_bwd_kernel<T, wpr(), c(), nw(), kGather>), grid, block, 0, st, a);
    else if (a.y) hipLaunchKernelGGL((norm_bwd_kernel<T, wpr(), c(), nw(), kLoad>), grid, block, 0, st, a);
    else hipLaunchKernelGGL((norm_bwd_kernel<T, wpr(), c(), nw(), kNone>), grid, block, 0, st, a);
    return hipGetLastError();
  });
  if (err != hipSuccess || (!a.dw_post && !a.dw_pre)) return err;
  hipLaunchKernelGGL(norm_dw_kernel, dim3(a.d / 64, 2), dim3(1024), 0, st, a.d, G, a.part, a.dw_post, a.dw_pre);
  return hipGetLastError();
}

}  // namespace

size_t norm_workspace_bytes(int T, int d) { return (size_t)bwd_grid(T, 1) * d * 2 * sizeof(float); }

hipError_t block_norm_forward(int elem_bytes, const NormFwd& a, hipStream_t st) {
  if (a.T == 0) return hipSuccess;
  return elem_bytes == 4 ? fwd_t<float>(a, st) : fwd_t<bf16_t>(a, st);
}

hipError_t block_norm_backward(int elem_bytes, const NormBwd& a, hipStream_t st) {
  return elem_bytes == 4 ? bwd_t<float>(a, st) : bwd_t<bf16_t>(a, st);
}

}  // namespace moe
