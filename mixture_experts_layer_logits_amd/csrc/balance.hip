// Balance loss, router z-loss and per-expert counts of a batch's routing, with their gradient.
//
// Over the N kept tokens (a token is left out by its mask byte, or when each of its scores is
// -inf), with p = softmax(logits[t]) over all E experts and c_e the kept tokens' choices
// of expert e:
//   loss[0] = E / (k N) sum_e c_e mean_t p_e     (1 when choices and probabilities are even)
//   loss[1] = mean_t lse(logits[t])^2
//   dlogits[t, e] = p_e (g0 E / (k N) (c_e / N - sum_e' p_e' c_e' / N) + 2 g1 lse_t / N)
// c_e is a count and has no gradient.  Both passes read the scores once.
//
// Measured on an MI355X, inputs in the memory-side cache.  Forward: 4.8 us at T = 256, E = 8, k = 2 (one
// launch), 10.0 us at T = 8192, E = 128, k = 4 (two dependent launches, each latency), 19.2 us at T = 65536:
// 14.6 (2.4 TB/s; its 4.2 M vector instructions issue in 7, and the waves, 16 a compute unit, wait
// through half of their cycles) and 4.7 of the second launch; there the choices' atomics are none of it,
// the exponentials 1.2 us, and twice the workgroups take 20.3.  Backward: 4.4 us at T = 8192 and 13.5 us
// (4.1 TB/s) at T = 65521, E = 96, k = 6, where issuing its vector instructions alone takes about 8.
//
// A token's scores lie across LPT lanes (a power of two, at most a wave, and at least k), 4
// consecutive experts per 16-byte load and NV <= 4 loads per lane, so a wave holds 64 / LPT tokens,
// the softmax takes log2(LPT) exchange steps, and lane j holds the token's choice j.  Column sums stay
// in registers over a wave's tokens and meet in a fixed order: across the wave's tokens, the
// workgroup's waves, then the workgroups (a second launch, in double), so the result is the same
// bits on every run.
#include <cmath>

#include "block.h"
#include "gemm.h"
#include "lanes.h"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / kWave;
constexpr float kNegInf = -INFINITY;

// e^x = 2^t (1 + r ln 2) with t = x log2 e rounded and r what that rounding and the constant's own
// dropped: within 2 units in the last place for x <= 0, values below 2^-126 as 0, NaN as NaN.  The
// backward issues some 140 vector instructions per lane and token, which bound it; expf's handling of
// ranges that p = e^(score - lse) never has was 20 of them.
__device__ __forceinline__ float exp_neg(float x) {
  constexpr float kLog2E = 1.44269502f, kLog2ELow = 1.92596303e-08f, kLn2 = 0.693147182f;
  x = x < -150.f ? -150.f : x;  // -inf: its r would be NaN
  const float t = x * kLog2E;
  const float r = fmaf(x, kLog2ELow, fmaf(x, kLog2E, -t));
  const float p = __builtin_amdgcn_exp2f(t);
  return fmaf(p, r * kLn2, p);
}

template <int LPT, int N = 1>
__device__ __forceinline__ float group_max(float v) {
  if constexpr (N < LPT) {
    const float w = other_half<N>(v);
    return group_max<LPT, 2 * N>((w > v || w != w) ? w : v);  // a NaN score wins, so it reaches lse
  }
  return v;
}

// Column of element c of lane q's load i: 4 consecutive ones where rows are 16-byte aligned (VEC),
// else one of each LPT, so that a wave's 4-byte accesses still fall on whole lines.
template <int LPT, bool VEC>
__device__ __forceinline__ int column(int q, int i, int c) {
  return VEC ? 4 * (q + LPT * i) + c : q + LPT * (4 * i + c);
}
// lane q's scores of load i (columns past E: -inf)
template <int LPT, bool VEC>
__device__ __forceinline__ void load_scores(const float* row, int q, int i, int E, float (&v)[4]) {
  if constexpr (VEC) {
    const int e0 = column<LPT, VEC>(q, i, 0);
    float4 w = make_float4(kNegInf, kNegInf, kNegInf, kNegInf);
    if (e0 < E) w = *reinterpret_cast<const float4*>(row + e0);
    v[0] = w.x; v[1] = w.y; v[2] = w.z; v[3] = w.w;
  } else {
#pragma unroll
    for (int c = 0; c < 4; c++) {
      const int e = column<LPT, VEC>(q, i, c);
      v[c] = e < E ? row[e] : kNegInf;
    }
  }
}

// Workspace: the sum kernel's meeting point, then one row of partial sums per workgroup.
struct BalancePart {
  double* dots;      // [kMaxExperts / kSumCols] a sum workgroup's share of sum_e c_e P_e
  uint32_t* ticket;  // sum workgroups done; zeroed by the forward's first workgroup
  float* prob;       // [G][E]
  int32_t* count;    // [G][E]
  float* z;          // [G]
  int32_t* kept;     // [G]
};
constexpr int kSumCols = 64;
constexpr size_t kPartHeader = 256;
static_assert((kMaxExperts / kSumCols) * sizeof(double) + sizeof(uint32_t) <= kPartHeader, "header holds both");

BalancePart carve(void* ws, int G, int E) {
  BalancePart b;
  b.dots = static_cast<double*>(ws);
  b.ticket = reinterpret_cast<uint32_t*>(b.dots + kMaxExperts / kSumCols);
  b.prob = reinterpret_cast<float*>(static_cast<char*>(ws) + kPartHeader);
  b.count = reinterpret_cast<int32_t*>(b.prob + (size_t)G * E);
  b.z = reinterpret_cast<float*>(b.count + (size_t)G * E);
  b.kept = reinterpret_cast<int32_t*>(b.z + G);
  return b;
}

__device__ __forceinline__ double wave_sum_double(double v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o, kWave);
  return v;
}

// Column e's outputs from its whole sums; returns its term of sum_e c_e P_e.
__device__ __forceinline__ double finish_column(int e, double prob, int count, double inv_n, int32_t* counts,
                                                float* prob_mean) {
  counts[e] = count;
  prob_mean[e] = (float)(prob * inv_n);
  return count * (prob * inv_n);
}
__device__ __forceinline__ void finish_loss(int E, int k, double dot, double z, int n, double inv_n, int32_t* counts,
                                            float* loss) {
  counts[E] = n;
  loss[0] = (float)(dot * inv_n * E / k);
  loss[1] = (float)(z * inv_n);
}

constexpr int kFwdThreads = 1024;
constexpr int kFwdWaves = kFwdThreads / kWave;

// What a lane loads of its token: its scores, its choice (lanes below k) and, a pass earlier, the
// mask byte that decides whether there is anything to load.
template <int LPT, int NV, bool VEC>
__global__ void __launch_bounds__(kFwdThreads) balance_fwd_kernel(int T, int E, int k,
                                                                  const float* __restrict__ logits,
                                                                  const int32_t* __restrict__ topk_idx,
                                                                  const uint8_t* __restrict__ mask,
                                                                  float* __restrict__ lse, const BalancePart part,
                                                                  int32_t* __restrict__ counts,
                                                                  float* __restrict__ prob_mean,
                                                                  float* __restrict__ loss) {
  constexpr int TW = kWave / LPT;  // tokens of a wave
  constexpr int HALF = kFwdWaves / 2;
  __shared__ int s_cnt[kMaxExperts];
  __shared__ float s_p[HALF][kMaxExperts];
  __shared__ float s_z[kFwdWaves];
  __shared__ int s_n[kFwdWaves];
  __shared__ double s_dot[kFwdWaves];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int q = lane % LPT, sub = lane / LPT;
  for (int e = tid; e < E; e += kFwdThreads) s_cnt[e] = 0;
  __syncthreads();
  float acc[NV][4];
#pragma unroll
  for (int i = 0; i < NV; i++)
#pragma unroll
    for (int c = 0; c < 4; c++) acc[i][c] = 0.f;
  float z = 0.f;
  int n = 0;
  const int64_t stride = (int64_t)gridDim.x * kFwdWaves * TW;
  int64_t t = ((int64_t)blockIdx.x * kFwdWaves + wave) * TW + sub;
  auto live_at = [&](int64_t at) { return at < T && (!mask || mask[at] != 0); };
  auto load = [&](int64_t at, bool live, float (&v)[NV][4], int& e) {
    e = 0;
    if (live && q < k) e = topk_idx[at * k + q];
#pragma unroll
    for (int i = 0; i < NV; i++) {
      v[i][0] = v[i][1] = v[i][2] = v[i][3] = kNegInf;
      if (live) load_scores<LPT, VEC>(logits + at * E, q, i, E, v[i]);
    }
  };
  float v[NV][4], ahead[NV][4];
  int e, e_ahead;
  load(t, live_at(t), v, e);
  bool live_ahead = live_at(t + stride);
  for (; t - sub < T; t += stride) {
    load(t + stride, live_ahead, ahead, e_ahead);
    live_ahead = live_at(t + 2 * stride);
    float top = kNegInf;
#pragma unroll
    for (int i = 0; i < NV; i++)
#pragma unroll
      for (int c = 0; c < 4; c++) top = (v[i][c] > top || v[i][c] != v[i][c]) ? v[i][c] : top;
    top = group_max<LPT>(top);
    const bool kept = top != kNegInf;  // a token left out holds -inf throughout
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < NV; i++)
#pragma unroll
      for (int c = 0; c < 4; c++) {
        v[i][c] = kept ? exp_neg(v[i][c] - top) : 0.f;
        sum += v[i][c];
      }
    sum = group_sum<LPT>(sum);
    if (kept) {
      const float inv = 1.f / sum;
#pragma unroll
      for (int i = 0; i < NV; i++)
#pragma unroll
        for (int c = 0; c < 4; c++) acc[i][c] = fmaf(v[i][c], inv, acc[i][c]);
      if (q < k) atomicAdd(&s_cnt[e < 0 ? 0 : (e >= E ? E - 1 : e)], 1);
    }
    if (q == 0 && t < T) {
      const float l = kept ? top + logf(sum) : kNegInf;
      lse[t] = l;
      if (kept) {
        z = fmaf(l, l, z);
        n++;
      }
    }
#pragma unroll
    for (int i = 0; i < NV; i++)
#pragma unroll
      for (int c = 0; c < 4; c++) v[i][c] = ahead[i][c];
    e = e_ahead;
  }
  // the wave's tokens, then the workgroup's waves: the upper half hands its sums to the lower one,
  // whose sums are then added column by column
#pragma unroll
  for (int o = LPT; o < kWave; o <<= 1)
#pragma unroll
    for (int i = 0; i < NV; i++)
#pragma unroll
      for (int c = 0; c < 4; c++) acc[i][c] += __shfl_xor(acc[i][c], o, kWave);
  z = wave_sum(z);
  n = wave_sum_int(n);
  if (lane == 0) {
    s_z[wave] = z;
    s_n[wave] = n;
  }
  auto each_column = [&](auto&& f) {
    if (sub == 0) {
#pragma unroll
      for (int i = 0; i < NV; i++)
#pragma unroll
        for (int c = 0; c < 4; c++) {
          const int col = column<LPT, VEC>(q, i, c);
          if (col < E) f(s_p[wave % HALF][col], acc[i][c]);
        }
    }
  };
  if (wave >= HALF) each_column([](float& s, float a) { s = a; });
  __syncthreads();
  if (wave < HALF) each_column([](float& s, float a) { s += a; });
  __syncthreads();
  z = 0.f;
  n = 0;
#pragma unroll
  for (int w = 0; w < kFwdWaves; w++) {
    z += s_z[w];
    n += s_n[w];
  }
  float p = 0.f;  // thread e < E: the workgroup's sum of column e
  if (tid < E) {
#pragma unroll
    for (int w = 0; w < HALF; w++) p += s_p[w][tid];
  }
  if (gridDim.x == 1) {  // the sums are whole: no second launch
    const double inv_n = n > 0 ? 1.0 / n : 0.0;
    const double dot = wave_sum_double(tid < E ? finish_column(tid, p, s_cnt[tid], inv_n, counts, prob_mean) : 0.0);
    if (lane == 0) s_dot[wave] = dot;
    __syncthreads();
    if (tid == 0) {
      double all = 0.0;
#pragma unroll
      for (int w = 0; w < kFwdWaves; w++) all += s_dot[w];
      finish_loss(E, k, all, z, n, inv_n, counts, loss);
    }
    return;
  }
  if (tid < E) {
    part.prob[(int64_t)blockIdx.x * E + tid] = p;
    part.count[(int64_t)blockIdx.x * E + tid] = s_cnt[tid];
  }
  if (tid == 0) {
    part.z[blockIdx.x] = z;
    part.kept[blockIdx.x] = n;
    if (blockIdx.x == 0) *part.ticket = 0;
  }
}

// The G rows of partial sums added in a fixed order (double): 64 columns per workgroup, 16 runs of
// rows.  The workgroup that comes last (device-wide ticket) adds the workgroups' shares of
// sum_e c_e P_e, in order, and writes the losses.
__global__ void __launch_bounds__(1024) balance_sum_kernel(int E, int k, int G, const BalancePart part,
                                                           int32_t* __restrict__ counts, float* __restrict__ prob_mean,
                                                           float* __restrict__ loss) {
  constexpr int RUNS = 16;
  __shared__ double s_p[RUNS][kSumCols];
  __shared__ int s_c[RUNS][kSumCols];
  __shared__ double s_z;
  __shared__ int s_n;
  const int lane = threadIdx.x & 63, run = threadIdx.x >> 6;
  const int col = blockIdx.x * kSumCols + lane;
  double p = 0.0;
  int c = 0;
  if (col < E) {
#pragma unroll 16
    for (int g = run; g < G; g += RUNS) {
      p += part.prob[(int64_t)g * E + col];
      c += part.count[(int64_t)g * E + col];
    }
  }
  s_p[run][lane] = p;
  s_c[run][lane] = c;
  if (run == RUNS - 1) {
    double z = 0.0;
    int n = 0;
#pragma unroll 4
    for (int g = lane; g < G; g += kWave) {
      z += part.z[g];
      n += part.kept[g];
    }
    z = wave_sum_double(z);
    n = wave_sum_int(n);
    if (lane == 0) {
      s_z = z;
      s_n = n;
    }
  }
  __syncthreads();
  if (run != 0) return;
  const double inv_n = s_n > 0 ? 1.0 / s_n : 0.0;
  double dot = 0.0;
  if (col < E) {
    p = 0.0;
    c = 0;
#pragma unroll
    for (int r = 0; r < RUNS; r++) {
      p += s_p[r][lane];
      c += s_c[r][lane];
    }
    dot = finish_column(col, p, c, inv_n, counts, prob_mean);
  }
  dot = wave_sum_double(dot);
  if (lane != 0) return;
  if (gridDim.x > 1) {
    __hip_atomic_store(&part.dots[blockIdx.x], dot, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    const uint32_t before = __hip_atomic_fetch_add(part.ticket, 1u, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT);
    if (before != gridDim.x - 1) return;
    dot = 0.0;
    for (unsigned b = 0; b < gridDim.x; b++)
      dot += __hip_atomic_load(&part.dots[b], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  }
  finish_loss(E, k, dot, s_z, s_n, inv_n, counts, loss);
}

// dlogits, written in full: the losses' gradient plus, with dgates, the gates' gradient.
template <int LPT, int NV, bool VEC>
__global__ void __launch_bounds__(kThreads) balance_bwd_kernel(int T, int E, int k, const float* __restrict__ logits,
                                                               const float* __restrict__ lse,
                                                               const int32_t* __restrict__ counts,
                                                               const float* __restrict__ dloss,
                                                               const float* __restrict__ dgates,
                                                               const float* __restrict__ gates,
                                                               const int32_t* __restrict__ topk_idx,
                                                               float* __restrict__ dlogits) {
  constexpr int TW = kWave / LPT;
  // the gates' gradient of a group's token by column, zero outside its choices (and between tokens)
  __shared__ __align__(16) float s_gate[kWaves][TW][4 * NV * LPT];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int q = lane % LPT, sub = lane / LPT;
  float* mine = s_gate[wave][sub];
#pragma unroll
  for (int i = 0; i < NV; i++)
    *reinterpret_cast<float4*>(mine + 4 * (q + LPT * i)) = make_float4(0.f, 0.f, 0.f, 0.f);
  wave_lds_fence();
  const int n = counts[E];
  const float inv_n = n > 0 ? 1.f / (float)n : 0.f;
  float share[NV][4];  // c_e / N
#pragma unroll
  for (int i = 0; i < NV; i++)
#pragma unroll
    for (int c = 0; c < 4; c++) {
      const int e = column<LPT, VEC>(q, i, c);
      share[i][c] = e < E ? (float)counts[e] * inv_n : 0.f;
    }
  const float a = dloss[0] * ((float)E / (float)k) * inv_n;
  const float b = 2.f * dloss[1] * inv_n;
  const int64_t stride = (int64_t)gridDim.x * kWaves * TW;
  for (int64_t t = ((int64_t)blockIdx.x * kWaves + wave) * TW + sub; t - sub < T; t += stride) {
    const bool in = t < T;
    const float l = in ? lse[t] : kNegInf;
    const bool kept = l != kNegInf;
    float g = 0.f, dg = 0.f;
    int id = -1;
    if (dgates && in && q < k) {
      g = gates[t * k + q];
      dg = dgates[t * k + q];
      id = topk_idx[t * k + q];
    }
    float p[NV][4];
    float inner = 0.f;
#pragma unroll
    for (int i = 0; i < NV; i++) {
      p[i][0] = p[i][1] = p[i][2] = p[i][3] = 0.f;
      if (kept) {
        load_scores<LPT, VEC>(logits + t * E, q, i, E, p[i]);
#pragma unroll
        for (int c = 0; c < 4; c++) {
          p[i][c] = exp_neg(p[i][c] - l);
          inner = fmaf(p[i][c], share[i][c], inner);
        }
      }
    }
    inner = group_sum<LPT>(inner);
    const float bl = kept ? b * l : 0.f;
#pragma unroll
    for (int i = 0; i < NV; i++)
#pragma unroll
      for (int c = 0; c < 4; c++) p[i][c] = kept ? p[i][c] * fmaf(a, share[i][c] - inner, bl) : 0.f;
    if (dgates) {
      // lane j puts choice j's gradient where the lane that holds its column picks it up
      const float gv = g * (dg - group_sum<LPT>(g * dg));
      if (id >= 0 && id < E) atomicAdd(&mine[id], gv);
      wave_lds_fence();
#pragma unroll
      for (int i = 0; i < NV; i++) {
        if constexpr (VEC) {
          const float4 gate = *reinterpret_cast<const float4*>(mine + column<LPT, VEC>(q, i, 0));
          p[i][0] += gate.x;
          p[i][1] += gate.y;
          p[i][2] += gate.z;
          p[i][3] += gate.w;
        } else {
#pragma unroll
          for (int c = 0; c < 4; c++) p[i][c] += mine[column<LPT, VEC>(q, i, c)];
        }
      }
      wave_lds_fence();
      if (id >= 0 && id < E) mine[id] = 0.f;
      wave_lds_fence();
    }
    if (!in) continue;
    float* o = dlogits + t * E;
#pragma unroll
    for (int i = 0; i < NV; i++) {
      if constexpr (VEC) {
        const int e0 = column<LPT, VEC>(q, i, 0);
        if (e0 < E) *reinterpret_cast<float4*>(o + e0) = make_float4(p[i][0], p[i][1], p[i][2], p[i][3]);
      } else {
#pragma unroll
        for (int c = 0; c < 4; c++) {
          const int e = column<LPT, VEC>(q, i, c);
          if (e < E) o[e] = p[i][c];
        }
      }
    }
  }
}

bool vec_ok(int E, const void* a, const void* b) {
  return E % 4 == 0 && ((reinterpret_cast<uintptr_t>(a) | reinterpret_cast<uintptr_t>(b)) & 15) == 0;
}

// How a token's scores lie in a wave: lanes (a power of two, at least k) and loads a lane.
struct Layout {
  int lanes, loads;
  int tokens() const { return kWave / lanes; }  // of a wave
};
// Wide: one load a lane where a wave holds the row.  Dense: up to four, so that the work per token
// that does not depend on E (reductions, addresses, choices) is shared by more tokens of a wave and
// fewer lanes stay idle.
Layout layout_of(int E, int k, bool dense) {
  const int quads = (E + 3) / 4;
  int l = 1;
  while (l < kWave && (l * (dense ? 4 : 1) < quads || l < k)) l *= 2;
  return Layout{l, (quads + l - 1) / l};
}

// Calls f(LPT, NV) with a layout's constants (DENSE: also those that only a dense layout has).
template <bool DENSE, class F>
hipError_t for_layout(const Layout& y, F&& f) {
  using std::integral_constant;
#define MOE_BAL_CASE(LPT, NV) \
  if (y.lanes == LPT && y.loads == NV) return f(integral_constant<int, LPT>{}, integral_constant<int, NV>{});
  MOE_BAL_CASE(1, 1) MOE_BAL_CASE(2, 1) MOE_BAL_CASE(4, 1) MOE_BAL_CASE(8, 1) MOE_BAL_CASE(16, 1) MOE_BAL_CASE(32, 1)
  MOE_BAL_CASE(64, 1) MOE_BAL_CASE(64, 2) MOE_BAL_CASE(64, 3) MOE_BAL_CASE(64, 4)
  if constexpr (DENSE) {
#define MOE_BAL_DENSE(LPT) MOE_BAL_CASE(LPT, 2) MOE_BAL_CASE(LPT, 3) MOE_BAL_CASE(LPT, 4)
    MOE_BAL_DENSE(1) MOE_BAL_DENSE(2) MOE_BAL_DENSE(4) MOE_BAL_DENSE(8) MOE_BAL_DENSE(16) MOE_BAL_DENSE(32)
#undef MOE_BAL_DENSE
  }
#undef MOE_BAL_CASE
  return hipErrorInvalidValue;
}

// workgroups of `waves` waves that hold all tokens at once, up to `most`
int balance_grid(int T, const Layout& y, int waves, int most) {
  const int64_t per = (int64_t)waves * y.tokens();
  const int64_t g = (T + per - 1) / per;
  return (int)(g < 1 ? 1 : (g > most ? most : g));
}
// Four rounds of tokens or fewer stay in one workgroup instead of a second launch.  One workgroup
// against two launches at 3, 4 and 5 rounds: 6.9 / 7.8 / 8.8 us against 8.0 / 8.2 / 8.0 at E = 128, 6.6 /
// 7.2 / 8.0 against 7.2 / 7.3 / 7.3 at E = 8; at E = 64 and 1024 the fourth round is the second launch's
// already (7.6 against 6.9, 14.3 against 12.6), the third is even.
// More are spread as wide as they go (T = 8192, E = 128, side by side: 9.6 us with 256 workgroups of
// one round, 11.4 with 128 of two, 12.2 with 64 of four).
int balance_fwd_grid(int T, const Layout& y) {
  const int g = balance_grid(T, y, kFwdWaves, kBalanceBlocks);
  return g <= 4 ? 1 : g;
}
// Dense once the wide layout takes more than three rounds: T = 63383, E = 134, k = 2 29.9 -> 21.2 us,
// T = 65521, E = 96, k = 6 19.3 -> 16.6, E = 128 and 256 the same; at two rounds it loses (T = 16384,
// E = 128: 10.9 against 14.6).  The backward stays wide: with four loads a lane it keeps too few in
// flight (T = 65536, E = 128, k = 4: 15.8 us against 19.8).
Layout balance_fwd_layout(int T, int E, int k) {
  const Layout wide = layout_of(E, k, false);
  return (int64_t)T > 3ll * kBalanceBlocks * kFwdWaves * wide.tokens() ? layout_of(E, k, true) : wide;
}

}  // namespace

size_t balance_workspace_bytes(int T, int E, int k) {
  return kPartHeader + (size_t)balance_fwd_grid(T, balance_fwd_layout(T, E, k)) * ((size_t)E * 2 + 2) * sizeof(float);
}

hipError_t balance_forward(int T, int E, int k, const float* logits, const int32_t* topk_idx, const uint8_t* mask,
                           float* lse, int32_t* counts, float* prob_mean, float* loss, void* ws, hipStream_t st) {
  const Layout y = balance_fwd_layout(T, E, k);
  const int G = balance_fwd_grid(T, y);
  const BalancePart part = carve(ws, G, E);
  const bool vec = vec_ok(E, logits, logits);
  const hipError_t err = for_layout<true>(y, [&](auto lpt, auto nv) {
    const auto kern = vec ? balance_fwd_kernel<lpt(), nv(), true> : balance_fwd_kernel<lpt(), nv(), false>;
    hipLaunchKernelGGL(kern, dim3(G), dim3(kFwdThreads), 0, st, T, E, k, logits, topk_idx, mask, lse, part, counts,
                       prob_mean, loss);
    return hipGetLastError();
  });
  if (err != hipSuccess || G == 1) return err;
  hipLaunchKernelGGL(balance_sum_kernel, dim3((E + kSumCols - 1) / kSumCols), dim3(1024), 0, st, E, k, G, part, counts,
                     prob_mean, loss);
  return hipGetLastError();
}

hipError_t balance_backward(int T, int E, int k, const float* logits, const float* lse, const int32_t* counts,
                            const float* dloss, const float* dgates, const float* gates, const int32_t* topk_idx,
                            float* dlogits, hipStream_t st) {
  if (T == 0) return hipSuccess;
  const Layout y = layout_of(E, k, false);
  const int G = balance_grid(T, y, kWaves, device_cu_count() * 8);
  const bool vec = vec_ok(E, logits, dlogits);
  return for_layout<false>(y, [&](auto lpt, auto nv) {
    if (vec)
      hipLaunchKernelGGL((balance_bwd_kernel<lpt(), nv(), true>), dim3(G), dim3(kThreads), 0, st, T, E, k, logits, lse,
                         counts, dloss, dgates, gates, topk_idx, dlogits);
    else
      hipLaunchKernelGGL((balance_bwd_kernel<lpt(), nv(), false>), dim3(G), dim3(kThreads), 0, st, T, E, k, logits,
                         lse, counts, dloss, dgates, gates, topk_idx, dlogits);
    return hipGetLastError();
  });
}

}  // namespace moe
