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

hipError_t gemm1_fwd_c8_bf16(const GemmShape& s, const int* offsets, const bf16_t* X, const bf16_t* W1,
                             const bf16_t* W3, bf16_t* h, int8_t* abq, uint8_t* ab_s, hipStream_t st) {
  ProbGemm1C8 p;
  p.M = s.R; p.N = 2 * s.f; p.K = s.d; p.E = s.E; p.offsets = offsets; p.f = s.f;
  p.X = X; p.W1 = W1; p.W3 = W3; p.h = h; p.abq = abq; p.ab_s = ab_s;
  return launch(m_grouped_tile("GEMM1", s, 64), p, st);
}

hipError_t dgrad2_c8_bf16(const GemmShape& s, const int* offsets, const bf16_t* dY, const bf16_t* W2,
                          const int8_t* abq, const uint8_t* ab_s, bf16_t* dab, bf16_t* h, hipStream_t st) {
  ProbDgrad2C8 p;
  p.M = s.R; p.N = s.f; p.K = s.d; p.E = s.E; p.offsets = offsets;
  p.dY = dY; p.W2 = W2; p.dab = dab; p.abq = abq; p.ab_s = ab_s; p.h = h;
  return launch(tile_for("DGRAD2", Tile::t128x256w8, 64, 3, 4), p, st);
}

}  // namespace moe
