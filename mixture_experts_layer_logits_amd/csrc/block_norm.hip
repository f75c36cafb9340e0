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
// waves, or for narrow rows of LPR lanes of one (WPR = 1, 64 / LPR rows a wave), 8 consecutive
// columns per 16-byte load and C such chunks per lane; row sums are register exchanges over the
// lanes, then over the WPR waves through LDS.  Rows and weights round to
// the element type once, at the store: xn is taken from the unrounded v, dy from the unrounded D.
// Weight gradients accumulate in registers over a workgroup's rows, meet across its waves in
// LDS, go to one partial row per workgroup and are added by a second launch, all in a fixed
// order (no atomics).
//
// Measured on an MI355X (a 2 + 2 GiB copy runs at 4.97 TB/s, 134 + 134 MB at 7.2 out of the
// memory-side cache), bf16: forward with both norms 22.4 us at T = 8192, d = 2048 (6.0 TB/s), 2.4 us
// for one row; backward 47.8 us (4.2 TB/s; 42 and the second launch); backward of the norm
// before a block 103 us at T = 16384, d = 4096 (5.2 TB/s); combine with both norms at k = 4 58.4 us
// at T = 8192, d = 2048 (4.6 TB/s), backward 336 us at T = 16384, d = 4096 (4.8 TB/s).
#include "block.h"
#include "gemm.h"
#include "lanes.h"

namespace moe {
namespace {

// The branch y: absent, read, or gathered from routed rows (in the backward, from at most kBatch rows
// a token, all held in registers, or from any number).
enum Src { kNone = 0, kLoad = 1, kGather = 2, kGatherMany = 3 };
constexpr bool gathers(int src) { return src == kGather || src == kGatherMany; }

// The lanes that hold one row: LPR of a wave, or WPR whole waves.
constexpr int rows_of(int lpr, int wpr, int nwaves) { return nwaves * (kWave / lpr) / wpr; }

// Sums over the lanes of a row.  Over several waves, consecutive sums alternate between two LDS
// buffers, so one barrier each is enough: a buffer is written again only after a later barrier.
template <int LPR, int WPR, int NWAVES>
struct RowSum {
  float (*buf)[NWAVES][4];
  int wave;
  int at = 0;
  template <int N>
  __device__ __forceinline__ void operator()(float (&v)[N]) {
    static_assert(N <= 4, "a buffer holds 4 sums a wave");
#pragma unroll
    for (int n = 0; n < N; n++) v[n] = LPR == kWave ? wave_total(v[n]) : group_sum<LPR>(v[n]);
    if constexpr (WPR > 1) {
      if ((threadIdx.x & 63) == 0)
#pragma unroll
        for (int n = 0; n < N; n++) buf[at][wave][n] = v[n];
      __syncthreads();
      const int w0 = wave / WPR * WPR;
#pragma unroll
      for (int n = 0; n < N; n++) {
        v[n] = 0.f;
#pragma unroll
        for (int w = 0; w < WPR; w++) v[n] += buf[at][w0 + w][n];
      }
      at ^= 1;
    }
  }
  __device__ __forceinline__ float operator()(float v) {
    float a[1] = {v};
    (*this)(a);
    return a[0];
  }
};

// 8 consecutive elements as they lie in memory; rows are held in this form until used, so a
// bf16 row costs half the registers of its floats.
template <typename T> struct Raw;
template <> struct Raw<bf16_t> {
  uint4 q;
  __device__ __forceinline__ void clear() { q = make_uint4(0, 0, 0, 0); }
  __device__ __forceinline__ void load(const bf16_t* p) { q = *reinterpret_cast<const uint4*>(p); }
  // nothing: the compiler may not carry the floats of an earlier use across this point
  __device__ __forceinline__ void repack() { asm volatile("" : "+v"(q.x), "+v"(q.y), "+v"(q.z), "+v"(q.w)); }
  __device__ __forceinline__ float operator[](int i) const {
    const uint32_t w = i < 2 ? q.x : i < 4 ? q.y : i < 6 ? q.z : q.w;
    return __uint_as_float(i & 1 ? w & 0xffff0000u : w << 16);
  }
};
template <> struct Raw<float> {
  float4 a, b;
  __device__ __forceinline__ void clear() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
  __device__ __forceinline__ void load(const float* p) {
    a = reinterpret_cast<const float4*>(p)[0];
    b = reinterpret_cast<const float4*>(p)[1];
  }
  __device__ __forceinline__ void repack() {}
  __device__ __forceinline__ float operator[](int i) const {
    return i == 0 ? a.x : i == 1 ? a.y : i == 2 ? a.z : i == 3 ? a.w : i == 4 ? b.x : i == 5 ? b.y : i == 6 ? b.z : b.w;
  }
};

#define MOE_EACH(i, c)           \
  _Pragma("unroll") for (int i = 0; i < C; i++) \
  _Pragma("unroll") for (int c = 0; c < 8; c++)

// A lane's share of a row: chunks first + i * step (i < C) of 8 columns.  Chunks past the row
// read as zero (they enter row sums) and are not stored.
template <typename T, int C>
struct Lane {
  int first, step, nchunk;
  __device__ __forceinline__ void load(const void* row0, int64_t at, Raw<T> (&v)[C]) const {
    const T* row = static_cast<const T*>(row0) + at;
#pragma unroll
    for (int i = 0; i < C; i++) {
      v[i].clear();
      if (first + i * step < nchunk) v[i].load(row + (first + i * step) * 8);
    }
  }
  __device__ __forceinline__ void store(void* row0, int64_t at, const float (&v)[C][8]) const {
    T* row = static_cast<T*>(row0) + at;
#pragma unroll
    for (int i = 0; i < C; i++)
      if (first + i * step < nchunk) store8<T>(row + (first + i * step) * 8, v[i]);
  }
};

// Routed rows are loaded kBatch at a time, all loads before the first use; the backward keeps the
// last batch (with k <= kBatch all of them) for the gate gradients.
constexpr int kBatch = 4;
// Rows past 8192 columns take 16 waves at two chunks a lane and at most 128 registers: there the
// backward keeps no weights (they are read again each row), loads no row ahead, and gathers one
// routed row at a time.  With a branch that still spills (registers, bf16 / float: 77 / 188 with y, 99 /
// 248 with routed rows; 2 / 6 without a branch; the float gathering forward 75).
template <int C, int NWAVES> constexpr bool kTight = C == 2 && NWAVES == 16;

template <typename T, int C>
struct Gather {
  const void* y_perm;
  const float* gates;       // of this token
  const int32_t* slot_row;  // of this token
  int k, d;
  Raw<T> rows[kBatch][C];
  __device__ __forceinline__ void load(const Lane<T, C>& ln, int j0) {
#pragma unroll
    for (int j = 0; j < kBatch; j++)
      if (j0 + j < k) ln.load(y_perm, (int64_t)slot_row[j0 + j] * d, rows[j]);
  }
  // y += sum_j gates[j] rows[j], j in order
  __device__ __forceinline__ void sum(int j0, float (&y)[C][8]) const {
#pragma unroll
    for (int j = 0; j < kBatch; j++)
      if (j0 + j < k) {
        const float g = gates[j0 + j];
        MOE_EACH(i, c) y[i][c] = fmaf(g, rows[j][i][c], y[i][c]);
      }
  }
};

template <typename T, int LPR, int WPR, int C, int NWAVES, int SRC>
__global__ void __launch_bounds__(NWAVES * 64) norm_fwd_kernel(const NormFwd a) {
  constexpr int RPB = rows_of(LPR, WPR, NWAVES);
  __shared__ float s_red[2][NWAVES][4];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  RowSum<LPR, WPR, NWAVES> row_sum{s_red, wave};
  const Lane<T, C> ln{(wave % WPR) * kWave + lane % LPR, WPR * LPR, a.d / 8};
  // this lane's row of the workgroup's; the same for a whole wave (in scalar registers) at LPR = 64
  const int mine = LPR == kWave ? wave / WPR : wave * (kWave / LPR) + lane / LPR;
  const float inv_d = 1.f / (float)a.d;
  for (int64_t base = (int64_t)blockIdx.x * RPB; base < a.T; base += (int64_t)gridDim.x * RPB) {
    // waves past the last row repeat it without storing (row sums may hold barriers)
    const bool in = base + mine < a.T;
    const int64_t t = in ? base + mine : a.T - 1;
    const int64_t at = t * a.d;
    float v[C][8];
    Raw<T> x[C], w_post[C], w_pre[C];
    ln.load(a.x, at, x);
    if constexpr (SRC != kNone) {
      float y[C][8];
      if constexpr (SRC == kLoad) {
        Raw<T> raw[C];
        ln.load(a.y, at, raw);
        if (a.w_post) ln.load(a.w_post, 0, w_post);
        if (a.w_pre) ln.load(a.w_pre, 0, w_pre);
        MOE_EACH(i, c) y[i][c] = raw[i][c];
      } else {
        Gather<T, C> ga{a.y_perm, a.gates + t * a.k, a.slot_row + t * a.k, a.k, a.d};
        Raw<T> raw[C];
        ga.load(ln, 0);
        if (a.y_add) ln.load(a.y_add, at, raw);
        if (a.w_post) ln.load(a.w_post, 0, w_post);
        if (a.w_pre) ln.load(a.w_pre, 0, w_pre);
        MOE_EACH(i, c) y[i][c] = a.y_add ? raw[i][c] : 0.f;
        ga.sum(0, y);
        for (int j = kBatch; j < a.k; j += kBatch) {
          ga.load(ln, j);
          ga.sum(j, y);
        }
      }
      const float g = a.gate ? a.gate[t] : 1.f;
      float coef = a.res_scale * g;
      if (a.w_post) {
        float ss = 0.f;
        MOE_EACH(i, c) ss = fmaf(y[i][c], y[i][c], ss);
        const float r = rsqrtf(row_sum(ss) * inv_d + a.eps);
        coef *= r;
        if (in && ln.first == 0) a.rstd_post[t] = r;
        MOE_EACH(i, c) y[i][c] *= w_post[i][c];
      }
      // a closed gate drops the branch, whatever it holds
      MOE_EACH(i, c) v[i][c] = g != 0.f ? fmaf(coef, y[i][c], x[i][c]) : x[i][c];
      if (in) ln.store(a.v, at, v);
    } else {
      ln.load(a.w_pre, 0, w_pre);
      MOE_EACH(i, c) v[i][c] = x[i][c];
    }
    if (a.w_pre) {
      float ss = 0.f;
      MOE_EACH(i, c) ss = fmaf(v[i][c], v[i][c], ss);
      const float r = rsqrtf(row_sum(ss) * inv_d + a.eps);
      MOE_EACH(i, c) v[i][c] = v[i][c] * r * w_pre[i][c];
      if (in) {
        ln.store(a.xn, at, v);
        if (ln.first == 0) a.rstd_pre[t] = r;
      }
    }
  }
}

// Waves per SIMD the registers are held to: 4 (128 registers).  Up to 8192 columns the kernels without
// a gather meet that, the bf16 gathering ones nearly (several rows a wave spill 7 to 10, 4 waves a row
// with k > kBatch 2).  Float rows that gather would spill 44 to 53 registers there, and bf16 ones of
// two chunks a lane too, so those get up to 256: the bf16 ones take 206, float 164 to 178, and float of
// two chunks spills 83 to 95 even so.  12 waves a row have 168 (float gathers spill 4 to 11).
template <typename T, int C, int SRC, int NWAVES>
constexpr int bwd_waves_per_eu() {
  if (NWAVES > 8) return (NWAVES + 3) / 4;  // one workgroup a compute unit
  return gathers(SRC) && (sizeof(T) == 4 || C == 2) ? 2 : 4;
}

template <typename T, int LPR, int WPR, int C, int NWAVES, int SRC>
__global__ void __launch_bounds__(NWAVES * 64)
    __attribute__((amdgpu_waves_per_eu(bwd_waves_per_eu<T, C, SRC, NWAVES>()))) norm_bwd_kernel(const NormBwd a) {
  constexpr int RPB = rows_of(LPR, WPR, NWAVES);
  constexpr int kKeep = kTight<C, NWAVES> ? 1 : kBatch;
  __shared__ float s_red[2][NWAVES][4];
  constexpr int GROUPS = NWAVES / WPR;
  __shared__ float s_acc[GROUPS > 1 ? NWAVES * kWave * 8 : 1];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  RowSum<LPR, WPR, NWAVES> row_sum{s_red, wave};
  const Lane<T, C> ln{(wave % WPR) * kWave + lane % LPR, WPR * LPR, a.d / 8};
  // this lane's row of the workgroup's; the same for a whole wave (in scalar registers) at LPR = 64
  const int mine = LPR == kWave ? wave / WPR : wave * (kWave / LPR) + lane / LPR;
  const float inv_d = 1.f / (float)a.d;
  float acc_pre[C][8], acc_post[C][8];
  MOE_EACH(i, c) acc_pre[i][c] = acc_post[i][c] = 0.f;

  // The gradient at v reads one set of rows (dv, dxn, v), the branch another (y, or the routed
  // rows).  Each set's loads are issued before the other is worked on, the first one's a row
  // ahead, so memory stays busy across the row sums without registers for a second row.
  Raw<T> w_pre[C], w_post[C], dv[C], dxn[C], v[C], y_raw[C];
  Raw<T> rows[gathers(SRC) ? kKeep : 1][C];
  const int64_t stride = (int64_t)gridDim.x * RPB;
  int64_t next = (int64_t)blockIdx.x * RPB + mine;
  // rows past the last one repeat it: nothing of them is stored or added to the weights' sums
  auto clamped = [&](int64_t t) { return t < a.T ? t : (int64_t)a.T - 1; };
  auto load_stream = [&](int64_t t) {
    const int64_t at = clamped(t) * a.d;
    if (a.w_pre) {
      ln.load(a.v, at, v);
      ln.load(a.dxn, at, dxn);
    }
    if (a.dv) ln.load(a.dv, at, dv);
  };
  int32_t slot[gathers(SRC) ? kKeep : 1];  // the first routed rows of the next token
  auto load_slots = [&](int64_t t) {
    if constexpr (gathers(SRC)) {
#pragma unroll
      for (int j = 0; j < kKeep; j++) slot[j] = j < a.k ? a.slot_row[clamped(t) * a.k + j] : 0;
    }
  };
  load_slots(next);
  if constexpr (!kTight<C, NWAVES>) load_stream(next);
  if (!kTight<C, NWAVES> && a.w_pre) ln.load(a.w_pre, 0, w_pre);
  if constexpr (SRC != kNone && !kTight<C, NWAVES>)
    if (a.w_post) ln.load(a.w_post, 0, w_post);
  for (int64_t base = (int64_t)blockIdx.x * RPB; base < a.T; base += stride) {
    const bool in = next < a.T;
    const int64_t t = clamped(next), at = t * a.d;
    const float* gates = a.gates + t * a.k;
    const int32_t* slots = a.slot_row + t * a.k;
    if constexpr (kTight<C, NWAVES>) load_stream(next);
    next += stride;
    if constexpr (gathers(SRC)) {
#pragma unroll
      for (int j = 0; j < kKeep; j++)
        if (j < a.k) ln.load(a.y_perm, (int64_t)slot[j] * a.d, rows[j]);
      if (a.y_add) ln.load(a.y_add, at, y_raw);
      load_slots(next);
    }
    if constexpr (SRC == kLoad) ln.load(a.y, at, y_raw);
    if constexpr (kTight<C, NWAVES>) {
      if (a.w_pre) ln.load(a.w_pre, 0, w_pre);
    } else {
#pragma unroll
      for (int i = 0; i < C; i++) {
        w_pre[i].repack();
        w_post[i].repack();
      }
    }

    float D[C][8];
    MOE_EACH(i, c) D[i][c] = a.dv ? dv[i][c] : 0.f;
    if (a.w_pre) {
      const float r = a.rstd_pre[t];
      float s = 0.f;
      MOE_EACH(i, c) {
        const float q = dxn[i][c] * (v[i][c] * r);
        s = fmaf(q, w_pre[i][c], s);
        acc_pre[i][c] += in ? q : 0.f;
      }
      const float m = row_sum(s) * inv_d * r;  // mean(vh w_pre dxn) r
#pragma unroll
      for (int i = 0; i < C; i++) {
        v[i].repack();
        dxn[i].repack();
        w_pre[i].repack();
      }
      MOE_EACH(i, c) D[i][c] = fmaf(r, fmaf(-m, v[i][c], dxn[i][c] * w_pre[i][c]), D[i][c]);
    }
    if (in) ln.store(a.dx, at, D);
    if constexpr (!kTight<C, NWAVES>) load_stream(next);
    if constexpr (SRC != kNone) {
      // kGather: routed rows j0 .. j0 + kKeep - 1 into `rows`, all loads before the first use; those
      // of the last batch (`held`) serve the gate gradients, the others are gathered again
      int held = 0;
      auto load_rows = [&](int j0) {
#pragma unroll
        for (int j = 0; j < kKeep; j++)
          if (j0 + j < a.k) ln.load(a.y_perm, (int64_t)slots[j0 + j] * a.d, rows[j]);
      };
      auto add_rows = [&](int j0, float (&y)[C][8]) {  // j in order
#pragma unroll
        for (int j = 0; j < kKeep; j++)
          if (j0 + j < a.k) {
            const float gj = gates[j0 + j];
            MOE_EACH(i, c) y[i][c] = fmaf(gj, rows[j][i][c], y[i][c]);
#pragma unroll
            for (int i = 0; i < C; i++) rows[j][i].repack();
          }
      };
      float y[C][8];
      if constexpr (SRC == kLoad) {
        MOE_EACH(i, c) y[i][c] = y_raw[i][c];
      } else {
        MOE_EACH(i, c) y[i][c] = a.y_add ? y_raw[i][c] : 0.f;
        add_rows(0, y);
        if constexpr (SRC == kGatherMany)
          for (int j0 = kKeep; j0 < a.k; j0 += kKeep) {
            load_rows(j0);
            add_rows(j0, y);
            held = j0;
          }
      }
      if constexpr (kTight<C, NWAVES>)
        if (a.w_post) ln.load(a.w_post, 0, w_post);
      const float g = a.gate ? a.gate[t] : 1.f;
      const bool open = g != 0.f;
      const float ag = a.res_scale * g;
      if (a.w_post) {
        const float r = a.rstd_post[t];
        const bool adds = in && open;
        float s = 0.f;
        MOE_EACH(i, c) {
          y[i][c] *= r;
          const float q = D[i][c] * y[i][c];
          acc_post[i][c] += adds ? ag * q : 0.f;
          s = fmaf(q, w_post[i][c], s);
          D[i][c] *= w_post[i][c];
        }
        s = row_sum(s);
        if (in && a.dgate && ln.first == 0) a.dgate[t] = a.res_scale * s;
        const float m = s * inv_d, ar = ag * r;
        MOE_EACH(i, c) D[i][c] = open ? ar * fmaf(-m, y[i][c], D[i][c]) : 0.f;
      } else {
        if (a.dgate) {
          float s = 0.f;
          MOE_EACH(i, c) s = fmaf(D[i][c], y[i][c], s);
          s = row_sum(s);
          if (in && ln.first == 0) a.dgate[t] = a.res_scale * s;
        }
        MOE_EACH(i, c) D[i][c] = open ? ag * D[i][c] : 0.f;
      }
      if (in && a.dy) ln.store(a.dy, at, D);
      if constexpr (gathers(SRC)) {
        auto routed = [&](int j0) {  // the batch's rows of dy_perm, and its dgates
          float s[kKeep];
#pragma unroll
          for (int j = 0; j < kKeep; j++) {
            s[j] = 0.f;
            if (j0 + j >= a.k) continue;
            const float gj = gates[j0 + j];
            float o[C][8];
            MOE_EACH(i, c) {
              s[j] = fmaf(D[i][c], rows[j][i][c], s[j]);
              o[i][c] = gj * D[i][c];
            }
            if (in) ln.store(a.dy_perm, (int64_t)slots[j0 + j] * a.d, o);
          }
          row_sum(s);
          if (in && ln.first == 0)
#pragma unroll
            for (int j = 0; j < kKeep; j++)
              if (j0 + j < a.k) a.dgates[t * a.k + j0 + j] = open ? s[j] : 0.f;  // 0 whatever the rows hold
        };
        if constexpr (SRC == kGather) {
          routed(0);
        } else {
          routed(held);
          for (int j0 = 0; j0 < held; j0 += kKeep) {
            load_rows(j0);
            routed(j0);
          }
        }
      }
    }
  }
  // weight-gradient partials: a wave's rows, the workgroup's waves in order, then one row per
  // workgroup of part [2][G][d] (dw_post, dw_pre)
  auto reduce = [&](float (&acc)[C][8], float* out) {
#pragma unroll
    for (int i = 0; i < C; i++) {
      float sum[8];
#pragma unroll
      for (int c = 0; c < 8; c++) {
        sum[c] = acc[i][c];
        if constexpr (LPR <= 8) sum[c] += other_half<8>(sum[c]);
        if constexpr (LPR <= 16) sum[c] += other_half<16>(sum[c]);
        if constexpr (LPR <= 32) sum[c] += other_half<32>(sum[c]);
      }
      if constexpr (GROUPS > 1) {
        __syncthreads();
        float* at = s_acc + (wave * kWave + lane) * 8;
#pragma unroll
        for (int c = 0; c < 8; c++) at[c] = sum[c];
        __syncthreads();
        if (wave < WPR) {
#pragma unroll
          for (int c = 0; c < 8; c++) sum[c] = 0.f;
          for (int r = 0; r < GROUPS; r++)
#pragma unroll
            for (int c = 0; c < 8; c++) sum[c] += s_acc[((r * WPR + wave) * kWave + lane) * 8 + c];
        }
      }
      const int chunk = ln.first + i * ln.step;
      if (wave < WPR && lane < LPR && chunk < ln.nchunk) store8<float>(out + chunk * 8, sum);
    }
  };
  const bool alone = gridDim.x == 1;  // then the sums are whole
  if (a.dw_post) reduce(acc_post, alone ? a.dw_post : a.part + (int64_t)blockIdx.x * a.d);
  if (a.dw_pre) reduce(acc_pre, alone ? a.dw_pre : a.part + ((int64_t)gridDim.x + blockIdx.x) * a.d);
}

// dw[c] = sum over the G workgroups of part[g][c], in a fixed order: 16 columns per workgroup, 64
// runs of rows that meet in LDS (a launch of d / 16 workgroups keeps every load of a run in
// flight; 64 columns each left most of the chip idle).  blockIdx.y: dw_post, dw_pre.
__global__ void __launch_bounds__(1024) norm_dw_kernel(int d, int G, const float* __restrict__ part,
                                                       float* __restrict__ dw_post, float* __restrict__ dw_pre) {
  constexpr int COLS = 16, RUNS = 64;
  __shared__ float s[RUNS][COLS];
  float* out = blockIdx.y == 0 ? dw_post : dw_pre;
  if (!out) return;
  const int col = threadIdx.x % COLS, run = threadIdx.x / COLS;
  const float* p = part + (int64_t)blockIdx.y * G * d + blockIdx.x * COLS + col;
  float sum = 0.f;
#pragma unroll 4
  for (int g = run; g < G; g += RUNS) sum += p[(int64_t)g * d];
  s[run][col] = sum;
  __syncthreads();
#pragma unroll
  for (int n = RUNS / 2; n > 0; n /= 2) {
    if (run < n) s[run][col] += s[run + n][col];
    __syncthreads();
  }
  if (run == 0) out[blockIdx.x * COLS + col] = s[0][col];
}

// Calls f(LPR, WPR, C, NWAVES) with the lanes and waves per row, chunks per lane and waves per
// workgroup that hold a row of d.  Rows between the steps leave lanes idle: at 1.6 GB the backward of combine
// and norm takes 382 us at d = 2560 on 8 waves a row (347 at 2048, 342 at 4096), and 447 on 5, whose
// workgroups fill a compute unit worse; just past a step, with nearly half of the lanes idle, bf16 rows
// take a quarter more (d = 1088: 447 us against 359 at 1024; float 390 against 343).
#define MOE_NORM_CASE(LPR, WPR, C, NWAVES)                                        \
  if (d <= LPR * WPR * C * 8)                                                     \
    return f(std::integral_constant<int, LPR>{}, std::integral_constant<int, WPR>{}, \
             std::integral_constant<int, C>{}, std::integral_constant<int, NWAVES>{});
// Several narrow rows to a wave (combine and norm forward at T = 57912, d = 64, k = 7: 17 us against
// 56) or, for fewer rows, a wave each, whose slots, gates and row sums are scalars (backward at T = 3,
// d = 256, k = 5: 6.8 us against 9.5).  The backward decides the step: with both norms at d = 128, a wave
// each against several takes 7.2 / 9.2 us against 7.6 / 8.1 at T = 2048 / 4096, and gathering k = 4 rows
// 9.8 / 12.4 against 11.2 / 12.0 (d = 64 and 256 cross there too).  The forward gains from packing at any T
// (4.2 against 3.7 us at T = 2048, d = 128, k = 4; 3.7 against 3.5 at 256) and shares the rule.
constexpr int kPackRows = 2048;
template <class F>
hipError_t for_width_fwd(int T, int d, F&& f) {
  if (T > kPackRows) { MOE_NORM_CASE(8, 1, 1, 4) MOE_NORM_CASE(16, 1, 1, 4) MOE_NORM_CASE(32, 1, 1, 4) }
  MOE_NORM_CASE(64, 1, 1, 4)
  MOE_NORM_CASE(64, 1, 2, 4) MOE_NORM_CASE(64, 2, 2, 4) MOE_NORM_CASE(64, 4, 2, 4) MOE_NORM_CASE(64, 8, 2, 8)
  MOE_NORM_CASE(64, 16, 2, 16)
  return hipErrorInvalidValue;
}
// Backward: one chunk a lane, so a row's accumulators and both sets of rows fit 128 registers.  A
// gathering row of more than 12 waves takes 8 at two chunks instead of 16 at one, whose 128
// registers it overflows (d = 8192, k = 4, T = 8192: 393 against 524 us); without a gather 16
// waves are faster (54 against 59 us).  12 waves keep 168 registers each (d = 5120: 396 us against
// 508 on 8 waves of two chunks).
template <int SRC, class F>
hipError_t for_width_bwd(int T, int d, F&& f) {
  if (T > kPackRows) { MOE_NORM_CASE(8, 1, 1, 8) MOE_NORM_CASE(16, 1, 1, 8) MOE_NORM_CASE(32, 1, 1, 8) }
  MOE_NORM_CASE(64, 1, 1, 8)
  MOE_NORM_CASE(64, 2, 1, 8) MOE_NORM_CASE(64, 4, 1, 8) MOE_NORM_CASE(64, 8, 1, 8) MOE_NORM_CASE(64, 12, 1, 12)
  if constexpr (gathers(SRC)) { MOE_NORM_CASE(64, 8, 2, 8) } else { MOE_NORM_CASE(64, 16, 1, 16) }
  if constexpr (SRC != kGather) { MOE_NORM_CASE(64, 16, 2, 16) }  // kGather: at most 8192 columns
  return hipErrorInvalidValue;
}
#undef MOE_NORM_CASE

// one pass of rows per workgroup; more rows than a launch holds threads for go round again
constexpr int64_t kNormFwdBlocks = 1 << 20;

template <typename T>
hipError_t fwd_t(const NormFwd& a, hipStream_t st) {
  return for_width_fwd(a.T, a.d, [&](auto lpr, auto wpr, auto c, auto nw) {
    constexpr int RPB = rows_of(lpr(), wpr(), nw());
    const int64_t rows = ((int64_t)a.T + RPB - 1) / RPB;
    const dim3 grid((unsigned)(rows < kNormFwdBlocks ? rows : kNormFwdBlocks)), block(nw() * 64);
    if (a.y_perm) hipLaunchKernelGGL((norm_fwd_kernel<T, lpr(), wpr(), c(), nw(), kGather>), grid, block, 0, st, a);
    else if (a.y) hipLaunchKernelGGL((norm_fwd_kernel<T, lpr(), wpr(), c(), nw(), kLoad>), grid, block, 0, st, a);
    else hipLaunchKernelGGL((norm_fwd_kernel<T, lpr(), wpr(), c(), nw(), kNone>), grid, block, 0, st, a);
    return hipGetLastError();
  });
}

// One workgroup where that saves the second launch (2.4 us) that adds up weight gradients: two
// passes of rows take less, two that gather (5 us each) do not.  More rows take every resident
// workgroup, kNormBlocks at most, and as few as need that many passes, for fewer partials.
int bwd_grid(int T, int rpb, int resident, bool gather) {
  const int64_t g = ((int64_t)T + rpb - 1) / rpb;
  if (g <= (gather ? 1 : 2)) return g > 0;
  const int most = resident < kNormBlocks ? resident : kNormBlocks;
  const int64_t passes = (g + most - 1) / most;
  return (int)((g + passes - 1) / passes);
}

template <typename T, int SRC>
hipError_t bwd_t(const NormBwd& a, hipStream_t st) {
  int G = 0;
  const hipError_t err = for_width_bwd<SRC>(a.T, a.d, [&](auto lpr, auto wpr, auto c, auto nw) {
    const auto kern = norm_bwd_kernel<T, lpr(), wpr(), c(), nw(), SRC>;
    G = bwd_grid(a.T, rows_of(lpr(), wpr(), nw()),
                 device_cu_count() * kernel_occupancy(reinterpret_cast<const void*>(kern), nw() * 64, 0),
                 gathers(SRC));
    if (G == 0) return hipSuccess;
    hipLaunchKernelGGL(kern, dim3(G), dim3(nw() * 64), 0, st, a);
    return hipGetLastError();
  });
  if (err != hipSuccess || G == 1 || (!a.dw_post && !a.dw_pre)) return err;
  hipLaunchKernelGGL(norm_dw_kernel, dim3(a.d / 16, 2), dim3(1024), 0, st, a.d, G, a.part, a.dw_post, a.dw_pre);
  return hipGetLastError();
}

}  // namespace

size_t norm_workspace_bytes(int T, int d) {
  return (size_t)(T < kNormBlocks ? T : kNormBlocks) * d * 2 * sizeof(float);
}

hipError_t block_norm_forward(int elem_bytes, const NormFwd& a, hipStream_t st) {
  if (a.T == 0) return hipSuccess;
  return elem_bytes == 4 ? fwd_t<float>(a, st) : fwd_t<bf16_t>(a, st);
}

hipError_t block_norm_backward(int elem_bytes, const NormBwd& a, hipStream_t st) {
  if (a.y_perm && a.k <= kBatch && a.d <= 8192)
    return elem_bytes == 4 ? bwd_t<float, kGather>(a, st) : bwd_t<bf16_t, kGather>(a, st);
  if (a.y_perm) return elem_bytes == 4 ? bwd_t<float, kGatherMany>(a, st) : bwd_t<bf16_t, kGatherMany>(a, st);
  if (a.y) return elem_bytes == 4 ? bwd_t<float, kLoad>(a, st) : bwd_t<bf16_t, kLoad>(a, st);
  return elem_bytes == 4 ? bwd_t<float, kNone>(a, st) : bwd_t<bf16_t, kNone>(a, st);
}

}  // namespace moe
