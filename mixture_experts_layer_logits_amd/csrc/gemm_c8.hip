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

// Tiles (us below are medians of graph replays in turn, of the named alternatives).  128 x 256 with four loader
// waves, 64 deep in three stages, where they fill the rounds of one tile a compute unit: 432 against 454 with
// 128 x 128 for GEMM1 and 272 against 291 for dgrad2 at E = 128, R = 32768, d = 2048, f = 1024 (the plain calls
// 399 and 272).  Where the last round or the last columns stand empty 128 x 128 (8 waves, two workgroups a compute
// unit) is faster: 57 against 65 for GEMM1 (0.69 filled) and 41 against 52 for dgrad2 (0.52) at R = 16384, E = 4, d =
// 1024, f = 512.  Between the two the thresholds lie on the side of 128 x 128: at E = 8, d = 2048 GEMM1 takes 121
// with it against 112 (0.84 filled, three rounds of f = 256, just below its threshold) and 118 against 115 (0.86,
// just above), dgrad2 113 against 100 (0.72, two rounds of f = 256) and 118 against 106 (0.76).  A launch of at
// most one round takes 128 x 128 at any fill: 128 x 256 measured 1 to 8% less there with E = 1 and from 2% more to 4%
// less with E = 4 (R = 4352 to 15872, d = 2048).
//
// The larger tiles that the plain GEMMs take for 1024 rows an expert and more are not built for these epilogues.
// 256 x 256 (64 deep, two stages): GEMM1 347 against 334 with 128 x 256 at R = 32768, E = 8, d = 2048, f = 1024 (plain
// 309), but 2115 against 2183 at R = 65536, E = 32, d = 4096, f = 2048 (plain 2117); dgrad2 290 against 232 and 1421 against
// 1276.  192 x 256 (32 deep, three stages, loader waves): GEMM1 320 and 2158, dgrad2, which spills 28 registers
// with the codes, 367 and 2336.  There the coded dgrad2 is slower than the plain one, which has those tiles
// (190 and 1189).
//
// Tiles of a launch for the worst routing, and whether 128 x 256 ones use num / den of their rounds
static int64_t c8_tiles(const GemmShape& s, int N, int bm, int bn) {
  return ((int64_t)s.R / bm + (s.R < s.E ? s.R : s.E)) * ((N + bn - 1) / bn);
}
static bool c8_large(const GemmShape& s, int N, int num, int den) {
  const int64_t tiles = c8_tiles(s, N, 128, 256), cus = device_cu_count(), rounds = (tiles + cus - 1) / cus;
  return rounds > 1 && tiles * N * den >= rounds * cus * ((N + 255) / 256 * 256) * num;
}

hipError_t gemm1_fwd_c8_bf16(const GemmShape& s, const int* offsets, const bf16_t* X, const bf16_t* W1,
                             const bf16_t* W3, bf16_t* h, int8_t* abq, uint8_t* ab_s, hipStream_t st) {
  ProbGemm1C8 p;
  p.M = s.R; p.N = 2 * s.f; p.K = s.d; p.E = s.E; p.offsets = offsets; p.f = s.f;
  p.X = X; p.W1 = W1; p.W3 = W3; p.h = h; p.abq = abq; p.ab_s = ab_s;
  // up to 32 rows an expert 64 x 128 (four waves of 32 x 64, so that a wave holds a and b of its columns):
  // 18 against 22 with 128 x 128 at R = 784, E = 43, d = 1344, f = 256, 206 against 221 at R = 4096, E = 128
  if (s.R <= (int64_t)32 * s.E) return launch_pipe<TileCfg<64, 128, 2, 2>, ProbGemm1C8, 64, 3>(p, st);
  if (c8_large(s, p.N, 27, 32)) return launch_pipe<TileCfg<128, 256, 2, 4>, ProbGemm1C8, 64, 3, 4>(p, st);
  return launch_pipe<TileCfg<128, 128, 4, 2>, ProbGemm1C8, 64, 2>(p, st);
}

hipError_t dgrad2_c8_bf16(const GemmShape& s, const int* offsets, const bf16_t* dY, const bf16_t* W2,
                          const int8_t* abq, const uint8_t* ab_s, bf16_t* dab, bf16_t* h, hipStream_t st) {
  ProbDgrad2C8 p;
  p.M = s.R; p.N = s.f; p.K = s.d; p.E = s.E; p.offsets = offsets;
  p.dY = dY; p.W2 = W2; p.dab = dab; p.abq = abq; p.ab_s = ab_s; p.h = h;
  // a row or two an expert: 32 rows a tile (66 against 69 with 64 x 64, R = 256, E = 128, f = 1024)
  if (s.R <= (int64_t)4 * s.E) return launch_pipe<TileCfg<32, 128, 1, 4>, ProbDgrad2C8, 64, 2>(p, st);
  // few tiles, or one column of them: 18 against 20 with 128 x 128 at R = 800, E = 8, f = 2048 (640 tiles; 16 against
  // 15.6 at 893), 24 against 32 at R = 120000, f = 64
  if (p.N <= 64 || c8_tiles(s, p.N, 64, 64) <= 3 * (int64_t)device_cu_count())
    return launch_pipe<TileCfg<64, 64, 2, 2>, ProbDgrad2C8, 64, 2>(p, st);
  // few columns, or a sixth of the last 128 empty: 27 against 29 with 128 x 128 at f = 128, 15 against 21 at 192, 48
  // against 51 at 320
  const int cols = (p.N + 127) / 128 * 128;
  if (cols == 128 || 6 * (cols - p.N) >= cols) return launch_pipe<TileCfg<128, 64, 4, 2>, ProbDgrad2C8, 64, 2>(p, st);
  if (c8_large(s, p.N, 3, 4)) return launch_pipe<TileCfg<128, 256, 2, 4>, ProbDgrad2C8, 64, 3, 4>(p, st);
  return launch_pipe<TileCfg<128, 128, 4, 2>, ProbDgrad2C8, 64, 2>(p, st);
}

}  // namespace moe
