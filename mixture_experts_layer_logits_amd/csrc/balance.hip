// Balance loss, router z-loss and per-expert counts of a batch's routing, with their gradient.
//
// Over the N kept tokens (a token is left out by its mask byte, or when none of its scores is
// above -inf), with p = softmax(logits[t]) over all E experts and c_e the kept tokens' choices
// of expert e:
//   loss[0] = E / (k N) sum_e c_e mean_t p_e     (1 when choices and probabilities are even)
//   loss[1] = mean_t lse(logits[t])^2
//   dlogits[t, e] = p_e (g0 E / (k N) (c_e / N - sum_e' p_e' c_e' / N) + 2 g1 lse_t / N)
// c_e is a count and has no gradient.  Both passes read the scores once; what bounds them is HBM
// at large T and launch latency below about 4 MB of scores.
//
// A token's scores lie across LPT lanes (a power of two, at most a wave), 4 consecutive experts
// per 16-byte load and NV loads per lane, so a wave holds 64 / LPT tokens and the softmax takes
// log2(LPT) exchange steps.  Column sums stay in registers over a wave's tokens and meet in a
// fixed order: across the wave's tokens, the workgroup's waves, then the workgroups (a second
// launch, in double), so the result is the same bits on every run.
#include <cmath>

#include "block.h"
#include "gemm.h"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / kWave;
constexpr float kNegInf = -INFINITY;

template <int LPT>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
  for (int o = LPT / 2; o > 0; o >>= 1) v += __shfl_xor(v, o, kWave);
  return v;
}
template <int LPT>
__device__ __forceinline__ float group_max(float v) {
#pragma unroll
  for (int o = LPT / 2; o > 0; o >>= 1) {
    const float w = __shfl_xor(v, o, kWave);
    v = (w > v || w != w) ? w : v;  // a NaN score wins, so it reaches lse
  }
  return v;
}

// the 4 scores at columns e0 .. e0+3 of a row (columns past E: -inf)
template <bool VEC>
__device__ __forceinline__ void load_scores(const float* row, int e0, int E, float (&v)[4]) {
  if constexpr (VEC) {
    float4 q = make_float4(kNegInf, kNegInf, kNegInf, kNegInf);
    if (e0 < E) q = *reinterpret_cast<const float4*>(row + e0);
    v[0] = q.x; v[1] = q.y; v[2] = q.z; v[3] = q.w;
  } else {
#pragma unroll
    for (int c = 0; c < 4; c++) v[c] = e0 + c < E ? row[e0 + c] : kNegInf;
  }
}

// Partial sums per workgroup, in ws: prob [G][E] float, then count [G][E] int32, then
// z [G] float and kept [G] int32.
template <int LPT, int NV, bool VEC>
__global__ void __launch_bounds__(kThreads) balance_fwd_kernel(int T, int E, int k, const float* __restrict__ logits,
                                                               const int32_t* __restrict__ topk_idx,
                                                               const uint8_t* __restrict__ mask,
                                                               float* __restrict__ lse, float* __restrict__ part_p,
                                                               int32_t* __restrict__ part_c,
                                                               float* __restrict__ part_z,
                                                               int32_t* __restrict__ part_n) {
  constexpr int TW = kWave / LPT;  // tokens of a wave
  __shared__ int s_cnt[kMaxExperts];
  __shared__ float s_p[kWaves][kMaxExperts];
  __shared__ float s_z[kWaves];
  __shared__ int s_n[kWaves];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int q = lane % LPT, sub = lane / LPT;
  for (int e = tid; e < E; e += kThreads) s_cnt[e] = 0;
  __syncthreads();
  float acc[NV][4];
#pragma unroll
  for (int i = 0; i < NV; i++)
#pragma unroll
    for (int c = 0; c < 4; c++) acc[i][c] = 0.f;
  float z = 0.f;
  int n = 0;
  const int64_t stride = (int64_t)gridDim.x * kWaves * TW;
  for (int64_t t = ((int64_t)blockIdx.x * kWaves + wave) * TW + sub; t - sub < T; t += stride) {
    const bool live = t < T && (!mask || mask[t] != 0);
    float v[NV][4];
    float top = kNegInf;
#pragma unroll
    for (int i = 0; i < NV; i++) {
      v[i][0] = v[i][1] = v[i][2] = v[i][3] = kNegInf;
      if (live) load_scores<VEC>(logits + t * E, 4 * (q + LPT * i), E, v[i]);
#pragma unroll
      for (int c = 0; c < 4; c++) top = (v[i][c] > top || v[i][c] != v[i][c]) ? v[i][c] : top;
    }
    top = group_max<LPT>(top);
    const bool kept = live && top != kNegInf;
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < NV; i++)
#pragma unroll
      for (int c = 0; c < 4; c++) {
        v[i][c] = kept ? expf(v[i][c] - top) : 0.f;
        sum += v[i][c];
      }
    sum = group_sum<LPT>(sum);
    if (kept) {
      const float inv = 1.f / sum;
#pragma unroll
      for (int i = 0; i < NV; i++)
#pragma unroll
        for (int c = 0; c < 4; c++) acc[i][c] = fmaf(v[i][c], inv, acc[i][c]);
      for (int j = q; j < k; j += LPT) {
        int e = topk_idx[t * k + j];
        e = e < 0 ? 0 : (e >= E ? E - 1 : e);
        atomicAdd(&s_cnt[e], 1);
      }
    }
    if (q == 0 && t < T) {
      const float l = kept ? top + logf(sum) : kNegInf;
      lse[t] = l;
      if (kept) {
        z = fmaf(l, l, z);
        n++;
      }
    }
  }
  // the wave's tokens, then the workgroup's waves
#pragma unroll
  for (int o = LPT; o < kWave; o <<= 1)
#pragma unroll
    for (int i = 0; i < NV; i++)
#pragma unroll
      for (int c = 0; c < 4; c++) acc[i][c] += __shfl_xor(acc[i][c], o, kWave);
  z = wave_sum(z);
  n = wave_sum_int(n);
  if (sub == 0) {
#pragma unroll
    for (int i = 0; i < NV; i++)
#pragma unroll
      for (int c = 0; c < 4; c++) {
        const int e = 4 * (q + LPT * i) + c;
        if (e < E) s_p[wave][e] = acc[i][c];
      }
  }
  if (lane == 0) {
    s_z[wave] = z;
    s_n[wave] = n;
  }
  __syncthreads();
  for (int e = tid; e < E; e += kThreads) {
    float p = 0.f;
#pragma unroll
    for (int w = 0; w < kWaves; w++) p += s_p[w][e];
    part_p[(int64_t)blockIdx.x * E + e] = p;
    part_c[(int64_t)blockIdx.x * E + e] = s_cnt[e];
  }
  if (tid == 0) {
    float zs = 0.f;
    int ns = 0;
    for (int w = 0; w < kWaves; w++) {
      zs += s_z[w];
      ns += s_n[w];
    }
    part_z[blockIdx.x] = zs;
    part_n[blockIdx.x] = ns;
  }
}

// One workgroup: the G rows of partial sums added in order (double), then the losses.
__global__ void __launch_bounds__(1024) balance_sum_kernel(int E, int k, int G, const float* __restrict__ part_p,
                                                           const int32_t* __restrict__ part_c,
                                                           const float* __restrict__ part_z,
                                                           const int32_t* __restrict__ part_n,
                                                           int32_t* __restrict__ counts, float* __restrict__ prob_mean,
                                                           float* __restrict__ loss) {
  __shared__ double s_p[1024];
  __shared__ int s_c[1024];
  __shared__ double s_dot[16];
  __shared__ double s_zn[2];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  // thread (part, expert) adds one run of rows of one expert
  const int P = 1024 / E > 0 ? 1024 / E : 1;
  const int part = tid / E, e = tid - part * E;
  double p = 0.0;
  int c = 0;
  if (part < P)
    for (int g = part; g < G; g += P) {
      p += part_p[(int64_t)g * E + e];
      c += part_c[(int64_t)g * E + e];
    }
  s_p[tid] = p;
  s_c[tid] = c;
  if (wave == 0) {
    double z = 0.0;
    int n = 0;
    for (int g = lane; g < G; g += kWave) {
      z += part_z[g];
      n += part_n[g];
    }
    for (int o = 32; o > 0; o >>= 1) z += __shfl_xor(z, o, kWave);
    n = wave_sum_int(n);
    if (lane == 0) {
      s_zn[0] = z;
      s_zn[1] = n;
    }
  }
  __syncthreads();
  const int n = (int)s_zn[1];
  const double inv = n > 0 ? 1.0 / n : 0.0;
  double dot = 0.0;
  if (tid < E) {
    double pe = 0.0;
    int ce = 0;
    for (int r = 0; r < P; r++) {
      pe += s_p[r * E + tid];
      ce += s_c[r * E + tid];
    }
    counts[tid] = ce;
    prob_mean[tid] = (float)(pe * inv);
    dot = ce * (pe * inv);
  }
  for (int o = 32; o > 0; o >>= 1) dot += __shfl_xor(dot, o, kWave);
  if (lane == 0) s_dot[wave] = dot;
  __syncthreads();
  if (tid == 0) {
    double sum = 0.0;
    for (int w = 0; w < 16; w++) sum += s_dot[w];
    counts[E] = n;
    loss[0] = (float)(sum * inv * E / k);
    loss[1] = (float)(s_zn[0] * inv);
  }
}

// dlogits, written in full: the losses' gradient plus, with dgates, the gates' gradient of
// route_backward (same arithmetic, so the two are equal when dloss is zero).
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
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int q = lane % LPT, sub = lane / LPT;
  const int n = counts[E];
  const float inv_n = n > 0 ? 1.f / (float)n : 0.f;
  float share[NV][4];  // c_e / N
#pragma unroll
  for (int i = 0; i < NV; i++)
#pragma unroll
    for (int c = 0; c < 4; c++) {
      const int e = 4 * (q + LPT * i) + c;
      share[i][c] = e < E ? (float)counts[e] * inv_n : 0.f;
    }
  const float a = dloss[0] * ((float)E / (float)k) * inv_n;
  const float b = 2.f * dloss[1] * inv_n;
  const int64_t stride = (int64_t)gridDim.x * kWaves * TW;
  for (int64_t t = ((int64_t)blockIdx.x * kWaves + wave) * TW + sub; t - sub < T; t += stride) {
    const bool in = t < T;
    const float l = in ? lse[t] : kNegInf;
    const bool kept = l != kNegInf;
    float p[NV][4];
    float inner = 0.f;
#pragma unroll
    for (int i = 0; i < NV; i++) {
      p[i][0] = p[i][1] = p[i][2] = p[i][3] = 0.f;
      if (kept) {
        load_scores<VEC>(logits + t * E, 4 * (q + LPT * i), E, p[i]);
#pragma unroll
        for (int c = 0; c < 4; c++) {
          p[i][c] = expf(p[i][c] - l);
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
    if (!in) continue;
    if (dgates) {
      const float* g = gates + t * k;
      const float* dg = dgates + t * k;
      const int32_t* id = topk_idx + t * k;
      float gsum = 0.f;
      for (int j = 0; j < k; j++) gsum = fmaf(g[j], dg[j], gsum);
      float gate[NV][4];
#pragma unroll
      for (int i = 0; i < NV; i++) gate[i][0] = gate[i][1] = gate[i][2] = gate[i][3] = 0.f;
      for (int j = 0; j < k; j++) {
        const float gv = g[j] * (dg[j] - gsum);
#pragma unroll
        for (int i = 0; i < NV; i++) {
          const int r = id[j] - 4 * (q + LPT * i);
#pragma unroll
          for (int c = 0; c < 4; c++)
            if (r == c) gate[i][c] += gv;
        }
      }
#pragma unroll
      for (int i = 0; i < NV; i++)
#pragma unroll
        for (int c = 0; c < 4; c++) p[i][c] += gate[i][c];
    }
#pragma unroll
    for (int i = 0; i < NV; i++) {
      const int e0 = 4 * (q + LPT * i);
      float* o = dlogits + t * E + e0;
      if constexpr (VEC) {
        if (e0 < E) *reinterpret_cast<float4*>(o) = make_float4(p[i][0], p[i][1], p[i][2], p[i][3]);
      } else {
#pragma unroll
        for (int c = 0; c < 4; c++)
          if (e0 + c < E) o[c] = p[i][c];
      }
    }
  }
}

bool vec_ok(int E, const void* a, const void* b) {
  return E % 4 == 0 && ((reinterpret_cast<uintptr_t>(a) | reinterpret_cast<uintptr_t>(b)) & 15) == 0;
}

// Calls f(LPT, NV) with the lanes per token and loads per lane that hold E scores.
template <class F>
hipError_t for_experts(int E, F&& f) {
  using std::integral_constant;
  const int e4 = (E + 3) / 4;
#define MOE_BAL_CASE(LIMIT, LPT, NV) \
  if (e4 <= LIMIT) return f(integral_constant<int, LPT>{}, integral_constant<int, NV>{});
  MOE_BAL_CASE(1, 1, 1) MOE_BAL_CASE(2, 2, 1) MOE_BAL_CASE(4, 4, 1) MOE_BAL_CASE(8, 8, 1) MOE_BAL_CASE(16, 16, 1)
  MOE_BAL_CASE(32, 32, 1) MOE_BAL_CASE(64, 64, 1) MOE_BAL_CASE(128, 64, 2) MOE_BAL_CASE(256, 64, 4)
#undef MOE_BAL_CASE
  return hipErrorInvalidValue;
}

int lanes_per_token(int E) {
  int l = 1;
  while (l < 64 && 4 * l < E) l *= 2;
  return l;
}

// workgroups that give every wave at most one pass, up to `most`
int balance_grid(int T, int E, int most) {
  const int64_t per = (int64_t)kWaves * (kWave / lanes_per_token(E));
  const int64_t g = (T + per - 1) / per;
  return (int)(g < 1 ? 1 : (g > most ? most : g));
}

}  // namespace

size_t balance_workspace_bytes(int T, int E) {
  return (size_t)balance_grid(T, E, kBalanceBlocks) * ((size_t)E * 2 + 2) * sizeof(float);
}

hipError_t balance_forward(int T, int E, int k, const float* logits, const int32_t* topk_idx, const uint8_t* mask,
                           float* lse, int32_t* counts, float* prob_mean, float* loss, void* ws, hipStream_t st) {
  const int G = balance_grid(T, E, kBalanceBlocks);
  float* part_p = static_cast<float*>(ws);
  int32_t* part_c = reinterpret_cast<int32_t*>(part_p + (size_t)G * E);
  float* part_z = reinterpret_cast<float*>(part_c + (size_t)G * E);
  int32_t* part_n = reinterpret_cast<int32_t*>(part_z + G);
  const bool vec = vec_ok(E, logits, logits);
  const hipError_t err = for_experts(E, [&](auto lpt, auto nv) {
    if (vec)
      hipLaunchKernelGGL((balance_fwd_kernel<lpt(), nv(), true>), dim3(G), dim3(kThreads), 0, st, T, E, k, logits,
                         topk_idx, mask, lse, part_p, part_c, part_z, part_n);
    else
      hipLaunchKernelGGL((balance_fwd_kernel<lpt(), nv(), false>), dim3(G), dim3(kThreads), 0, st, T, E, k, logits,
                         topk_idx, mask, lse, part_p, part_c, part_z, part_n);
    return hipGetLastError();
  });
  if (err != hipSuccess) return err;
  hipLaunchKernelGGL(balance_sum_kernel, dim3(1), dim3(1024), 0, st, E, k, G, part_p, part_c, part_z, part_n, counts,
                     prob_mean, loss);
  return hipGetLastError();
}

hipError_t balance_backward(int T, int E, int k, const float* logits, const float* lse, const int32_t* counts,
                            const float* dloss, const float* dgates, const float* gates, const int32_t* topk_idx,
                            float* dlogits, hipStream_t st) {
  if (T == 0) return hipSuccess;
  const int G = balance_grid(T, E, device_cu_count() * 8);
  const bool vec = vec_ok(E, logits, dlogits);
  return for_experts(E, [&](auto lpt, auto nv) {
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
