// The two expert GEMMs that write and read the 8-bit activation checkpoints in their epilogues
// (bf16 operands, the kernel and tiles of the plain GEMMs).
#include "ckpt8.h"
#include "gemm_pipe.h"

namespace moe {

// GEMM1 that keeps [a | b] as MXINT8 (codes abq [R][2f], scale bytes ab_s [R][2f/32]) instead of bf16
struct ProbGemm1C8 : ProbGemm1 {
  static constexpr bool CK8 = true;
  int8_t* abq = nullptr; uint8_t* ab_s = nullptr;
  // 8 columns hcol .. hcol+7 of row m: codes of a and b, packed bf16 h
  __device__ void store_swiglu_c8(int m, int hcol, const uint2& a, const uint2& b, const uint4& hv) const {
    int8_t* qr = abq + (int64_t)m * 2 * f;
    *reinterpret_cast<uint2*>(qr + hcol) = a;
    *reinterpret_cast<uint2*>(qr + f + hcol) = b;
    *reinterpret_cast<uint4*>(h + (int64_t)m * f + hcol) = hv;
  }
  __device__ void store_scales_c8(int m, int hcol, int sa, int sb) const {
    uint8_t* sr = ab_s + (int64_t)m * (2 * f / kCk8Block);
    sr[hcol / kCk8Block] = (uint8_t)sa;
    sr[(f + hcol) / kCk8Block] = (uint8_t)sb;
  }
};

// dgrad2 reading a and b from an MXINT8 [a | b] and writing h = silu(a) b [R][f] again
struct ProbDgrad2C8 : ProbDgrad2 {
  static constexpr bool CK8 = true;
  const int8_t* abq = nullptr; const uint8_t* ab_s = nullptr;
  bf16_t* h = nullptr;
  __device__ Ck8Pair prefetch_c8(int m, int n) const {
    const int8_t* qr = abq + (int64_t)m * 2 * N;
    const uint8_t* sr = ab_s + (int64_t)m * (2 * N / kCk8Block);
    return Ck8Pair{*reinterpret_cast<const uint32_t*>(qr + n), *reinterpret_cast<const uint32_t*>(qr + N + n),
                   sr[n / kCk8Block], sr[(N + n) / kCk8Block]};
  }
  __device__ void store_h16(int m, int n, const uint4& hv) const {
    *reinterpret_cast<uint4*>(h + (int64_t)m * N + n) = hv;
  }
};

// Tiles.  128 x 256 with four loader waves, 64 deep in three stages, where its tiles fill the device
// (the plain GEMMs' choice; 417 us for GEMM1 and 271 us for dgrad2 at E = 128, T = 8192, d = 2048, f =
// 1024).  `tiles` counts them for the worst routing.  Below two a compute unit, or with a row or two per
// expert, smaller tiles give more workgroups:
//   GEMM1   64 x 128 in three stages (four waves of 32 x 64, so that a wave holds a and b of its
//           columns): 12.5 against 22 us at R = 993, E = 6, d = 1088, f = 448; 57 against 65 at R =
//           4000, E = 8 and 117 against 141 at R = 256, E = 128 (d = 2048, f = 1024)
//   dgrad2  32 x 128 up to half a tile a compute unit: 11 against 26 us at R = 993, E = 6; 65 against 81
//           at R = 256, E = 128; from there to two 128 x 128 in two stages: 71 against 79 us at R =
//           32768, E = 8, d = 1024, f = 512
static int64_t c8_tiles(const GemmShape& s, int N) {
  return ((int64_t)s.R / 128 + (s.R < s.E ? s.R : s.E)) * ((N + 255) / 256);
}

hipError_t gemm1_fwd_c8_bf16(const GemmShape& s, const int* offsets, const bf16_t* X, const bf16_t* W1,
                             const bf16_t* W3, bf16_t* h, int8_t* abq, uint8_t* ab_s, hipStream_t st) {
  ProbGemm1C8 p;
  p.M = s.R; p.N = 2 * s.f; p.K = s.d; p.E = s.E; p.offsets = offsets; p.f = s.f;
  p.X = X; p.W1 = W1; p.W3 = W3; p.h = h; p.abq = abq; p.ab_s = ab_s;
  if (c8_tiles(s, p.N) <= 2 * device_cu_count() || s.R <= (int64_t)16 * s.E)
    return launch_pipe<TileCfg<64, 128, 2, 2>, ProbGemm1C8, 64, 3>(p, st);
  return launch_pipe<TileCfg<128, 256, 2, 4>, ProbGemm1C8, 64, 3, 4>(p, st);
}

hipError_t dgrad2_c8_bf16(const GemmShape& s, const int* offsets, const bf16_t* dY, const bf16_t* W2,
                          const int8_t* abq, const uint8_t* ab_s, bf16_t* dab, bf16_t* h, hipStream_t st) {
  ProbDgrad2C8 p;
  p.M = s.R; p.N = s.f; p.K = s.d; p.E = s.E; p.offsets = offsets;
  p.dY = dY; p.W2 = W2; p.dab = dab; p.abq = abq; p.ab_s = ab_s; p.h = h;
  const int64_t tiles = c8_tiles(s, p.N), cus = device_cu_count();
  if (2 * tiles <= cus || s.R <= (int64_t)4 * s.E)
    return launch_pipe<TileCfg<32, 128, 1, 4>, ProbDgrad2C8, 64, 2>(p, st);
  if (tiles <= 2 * cus && s.R > (int64_t)64 * s.E)
    return launch_pipe<TileCfg<128, 128, 2, 2>, ProbDgrad2C8, 64, 2>(p, st);
  return launch_pipe<TileCfg<128, 256, 2, 4>, ProbDgrad2C8, 64, 3, 4>(p, st);
}

}  // namespace moe
