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
#include <type_traits>

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

// one thread per block of 32.  Bound by HBM: 128 x 1024 x 2048 in bf16 takes 117 us (5.8 TB/s read and written)
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

struct W4Args {
  int R, K, N, E;           // rows, reduction, weight rows of an expert, experts
  const int* offsets;
  const void* X;            // [R][K]
  const uint8_t *q0, *s0;   // [E][N][K/2], [E][N][K/32]
  const uint8_t *q1, *s1;   // the second projection (gated)
  void* out;                // [R][N]
  int cus;                  // compute units (for the choice of tiles, on the host)
};

// A scale byte as the widening instructions take it: they read the exponent field alone, 0 as 2^-127
// and 255 as NaN.
__device__ __forceinline__ float mx4_scale(uint32_t byte) { return __uint_as_float(byte << 23); }

// Eight codes as bf16 or float
__device__ __forceinline__ bf16x8 widen_bf16(uint32_t c, float scale) {
  const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, scale, 0);
  const bf16x2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, scale, 1);
  const bf16x2 d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, scale, 2);
  const bf16x2 e = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, scale, 3);
  return bf16x8{a[0], a[1], b[0], b[1], d[0], d[1], e[0], e[1]};
}
__device__ __forceinline__ void widen_f32(uint32_t c, float scale, float (&v)[8]) {
  const f32x2 a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, scale, 0);
  const f32x2 b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, scale, 1);
  const f32x2 d = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, scale, 2);
  const f32x2 e = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, scale, 3);
  v[0] = a[0], v[1] = a[1], v[2] = b[0], v[3] = b[1], v[4] = d[0], v[5] = d[1], v[6] = e[0], v[7] = e[1];
}

// Loads go through buffer resources: a lane whose offset lies past the end (kNowhere: anywhere's) reads
// zeros and fetches nothing, so no load stands under a branch, and the number of loads in flight, which the
// waits count, is known.
constexpr uint32_t kNowhere = 0xffffffffu;
__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer(const void* base, uint32_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), (short)0, (int)bytes, 0x00020000);
}
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

// Sums over the lanes up to and including each
__device__ __forceinline__ int wave_scan(int v) {
  v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xF, 0xF, false);  // row_shr:1, 2, 4, 8
  v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xF, 0xF, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xF, 0xF, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xF, 0xF, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xA, 0xF, false);  // row_bcast15 into rows 1 and 3
  v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xC, 0xF, false);  // row_bcast31 into rows 2 and 3
  return v;
}

// The tiles of a launch: an expert's rows in runs of at most kRowsX where UNIT is 8, of even shares of at most
// `cap` whole 16s where UNIT is 16 (cap_inv: 2^32 / cap, rounded up), its weight rows in ntn tiles; the runs
// that share a weight tile follow one another.  Every wave finds its tiles by itself, so no barrier stands
// before the first load: a lane holds two experts of a window of 128, whose run counts are scanned in
// registers, and as tiles are asked for in ascending order the window only moves forward.
struct W4Tile {
  int e, m0, m_end, nt;  // e < 0: past the last tile
};
template <int UNIT>
struct W4Finder {
  const int* offsets;
  int E, ntn, lane, cap;
  uint32_t cap_inv;
  int e0, at[3], incl;  // at: where the lane's experts e0 + 2 lane, + 1 begin, and the next
  __device__ __forceinline__ int runs(int rows) const {
    const int units = (rows + UNIT - 1) / UNIT;
    if constexpr (UNIT == 8) return units;
    return cap == 1 ? units : (int)__umulhi(units + cap - 1, cap_inv);
  }
  __device__ __forceinline__ void window(int before) {
#pragma unroll
    for (int i = 0; i < 3; i++) {
      const int e = e0 + 2 * lane + i;
      at[i] = offsets[e < E ? e : E];
    }
    incl = before + wave_scan(runs(at[1] - at[0]) + runs(at[2] - at[1]));
  }
  __device__ __forceinline__ W4Finder(const int* off, int E_, int ntn_, int lane_, int cap_ = 1, uint32_t inv = 0)
      : offsets(off), E(E_), ntn(ntn_), lane(lane_), cap(cap_), cap_inv(inv), e0(0) {
    window(0);
  }
  __device__ __forceinline__ W4Tile find(int t) {
    while (true) {
      const int mine = runs(at[1] - at[0]) + runs(at[2] - at[1]);
      const uint64_t hit = __ballot(t >= (incl - mine) * ntn && t < incl * ntn);
      if (hit) {
        const int l = __builtin_ctzll(hit);
        const int a0 = __builtin_amdgcn_readlane(at[0], l), a1 = __builtin_amdgcn_readlane(at[1], l),
                  a2 = __builtin_amdgcn_readlane(at[2], l);
        const int r0 = runs(a1 - a0), r1 = runs(a2 - a1);
        int local = t - (__builtin_amdgcn_readlane(incl, l) - r0 - r1) * ntn;
        const bool second = local >= r0 * ntn;
        if (second) local -= r0 * ntn;
        const int me = second ? r1 : r0, start = second ? a1 : a0, end = second ? a2 : a1;
        const int nt = me == 1 ? local : local / me;
        const int per = UNIT == 8   ? UNIT
                        : me == 1 ? cap * UNIT
                                  : ((end - start + UNIT - 1) / UNIT + me - 1) / me * UNIT;
        const int m0 = start + (local - nt * me) * per;
        return W4Tile{e0 + 2 * l + (second ? 1 : 0), m0, m0 + per < end ? m0 + per : end, nt};
      }
      e0 += 2 * kWave;
      if (e0 >= E) return W4Tile{-1, 0, 0, 0};
      window(__builtin_amdgcn_readlane(incl, kWave - 1));
    }
  }
};

// First tile of a workgroup: workgroups b and b + 8 run on one XCD, which takes 8 neighbouring tiles of
// every 64 (they share weight tiles or routed rows, and so its L2), so that a last round that is not full
// is spread over all XCDs.
__device__ __forceinline__ int first_tile() {
  const int b = blockIdx.x, in = b & 63;
  return gridDim.x % 64 == 0 ? b - in + (in & 7) * 8 + in / 8 : b;
}

// ---- few rows: the weights stream through registers
// A tile is 16 weight rows by up to 8 routed rows of one expert.  The weights are the matrix product's
// left operand, the routed rows its right: lane l holds elements of weight row l % 16 and of routed row
// l % 8 (the upper half of the columns is computed twice), the same ones of the reduction, and which
// they are is free: NB blocks of 32 at 128 apart, block l / 16 of each 128, so that the four lanes of a
// row read 64 bytes of codes side by side.  The 8 waves of a workgroup are
// `tiles` neighbouring tiles by 8 / tiles shares of the reduction, taken piece by piece; the shares' sums
// are added through LDS in order.  Each wave loads its next piece, of this tile or the next, before it
// multiplies the one it has; the routed rows' part comes in whole rows (a load for two of them) and is
// handed to the lanes through LDS of the wave's own.  What bounds it where most experts have a row or two is
// HBM: 34 to 40 us for the 183 MB of T = 32, k = 4, E = 128, d = 2048, f = 1024, gated (4.6 to 5.4 TB/s), 19.4 us for
// the 92 MB of the second product; for one token the launch and two round trips to memory (offsets, then
// weights), 5.3 us.
constexpr int kStreamWaves = 8;
constexpr int kRowsW = 16;          // weight rows of a tile
constexpr int kRowsX = 8;           // routed rows of a tile

// NB: blocks of a lane's piece (1 or 2).  TAIL: the last piece may end inside (NB = 1).
template <typename T, int P, int NB, bool TAIL>
struct Stream {
  static constexpr int Q = 4 * NB;       // code words
  static constexpr int SPAN = 128 * NB;  // elements of the reduction a wave takes at a time
  static constexpr int LPR = SPAN * sizeof(T) / 16;  // lanes (16-byte chunks) of a routed row's piece
  static constexpr int RPL = kWave / LPR;            // rows of a load
  static constexpr int XL = kRowsX / RPL;            // loads
  static constexpr int SB = SPAN / kMx4Block;        // scale bytes of a row's piece
  struct Piece {
    uint32_t q[P][Q];
    bool live;  // the wave has this piece (the same in all lanes)
  };
  // Scale bytes of four pieces that follow one another: lane l holds those of piece l / 16, row l % 16, so
  // that a row's come in one load.  TAIL, where K / 32 is an odd number of pairs: the 8 aligned bytes that hold
  // the 4 (not past the tile's end), until settle
  struct Scales {
    uint32_t w[P][TAIL ? 2 : NB];
  };
  const W4Args& a;
  int lane, wr, grp;

  // Where a tile's weight rows from `col` on and its routed rows lie (past the last tile: nowhere)
  struct Source {
    __amdgpu_buffer_rsrc_t q[P], s[P], x;
  };
  __device__ __forceinline__ Source source(const W4Tile& t, int col) const {
    const uint8_t* const qs[2] = {a.q0, a.q1};
    const uint8_t* const ss[2] = {a.s0, a.s1};
    const bool in = t.e >= 0;
    const int64_t wrow = (int64_t)(in ? t.e : 0) * a.N + col;
    const uint32_t qb = a.K / 2, sb = a.K / kMx4Block, row = a.K * sizeof(T);  // bytes of a row
    Source r;
#pragma unroll
    for (int h = 0; h < P; h++) {
      r.q[h] = buffer(qs[h] + wrow * qb, in ? kRowsW * qb : 0);
      r.s[h] = buffer(ss[h] + wrow * sb, in ? kRowsW * sb : 0);
    }
    r.x = buffer(static_cast<const T*>(a.X) + (int64_t)t.m0 * a.K, in ? (t.m_end - t.m0) * row : 0);
    return r;
  }
  // Past the reduction's end an offset is past any buffer: kFar + a lane's own, without a wrap
  static constexpr uint32_t kFar = 0x80000000u;

  __device__ __forceinline__ void load_codes(Piece& c, const Source& src, bool live, int k) const {
    c.live = live && k < a.K;
    const uint32_t at = k < a.K ? k / 2 : kFar;
    const uint32_t qo = !TAIL || k + 32 * grp < a.K ? wr * (a.K / 2) + 16 * grp + at : kNowhere;
#pragma unroll
    for (int h = 0; h < P; h++) {
#pragma unroll
      for (int b = 0; b < NB; b++) {
        const u32x4 v = __builtin_amdgcn_raw_buffer_load_b128(src.q[h], qo + 64 * b, 0, 0);
        c.q[h][4 * b] = v.x, c.q[h][4 * b + 1] = v.y, c.q[h][4 * b + 2] = v.z, c.q[h][4 * b + 3] = v.w;
      }
    }
  }
  static __device__ __forceinline__ uint32_t aligned(uint32_t so, uint32_t sb) {
    const uint32_t last = kRowsW * sb - 8, down = so & ~3u;
    return down < last ? down : last;
  }
  __device__ __forceinline__ void load_scales(Scales& c, const Source& src, int k) const {
    const uint32_t sb = a.K / kMx4Block, at = k / kMx4Block + SB * grp, so = wr * sb + at;
#pragma unroll
    for (int h = 0; h < P; h++) {
      if constexpr (TAIL) {
        const u32x2 v = __builtin_amdgcn_raw_buffer_load_b64(src.s[h], at < sb ? aligned(so, sb) : kNowhere, 0, 0);
        c.w[h][0] = v.x, c.w[h][1] = v.y;
      } else if constexpr (NB == 2) {
        const u32x2 v = __builtin_amdgcn_raw_buffer_load_b64(src.s[h], so, 0, 0);
        c.w[h][0] = v.x, c.w[h][1] = v.y;
      } else {
        c.w[h][0] = __builtin_amdgcn_raw_buffer_load_b32(src.s[h], so, 0, 0);
      }
    }
  }
  // The loaded scales of the pieces from k on, as `scale` takes them
  __device__ __forceinline__ void settle(Scales& to, const Scales& c, int k) const {
    if constexpr (!TAIL) {
      to = c;
    } else {
      const uint32_t sb = a.K / kMx4Block, at = k / kMx4Block + SB * grp, so = wr * sb + at;
#pragma unroll
      for (int h = 0; h < P; h++) {
        const uint32_t w = (uint32_t)(((uint64_t)c.w[h][1] << 32 | c.w[h][0]) >> (8 * (so - aligned(so, sb)) & 63));
        to.w[h][0] = at + 2 < sb ? w : w & 0xffff;  // past the row's end lies the next row's, which may be NaN
      }
    }
  }
  // The scale of projection h's block b of the p-th of the four pieces, as the widening instructions take it
  __device__ __forceinline__ float scale(const Scales& c, int p, int h, int b) const {
    const uint32_t w = __builtin_amdgcn_ds_bpermute(4 * (16 * p + wr), c.w[h][b]);
    return mx4_scale(w >> (8 * grp) & 255);
  }

  __device__ __forceinline__ void load_rows(u32x4 (&x)[XL], const Source& src, int k) const {
    const uint32_t row = a.K * sizeof(T), o = (lane % LPR) * 16;
    const uint32_t at = (lane / LPR) * row + o + (k < a.K ? k * sizeof(T) : kFar);
#pragma unroll
    for (int i = 0; i < XL; i++)
      x[i] = __builtin_amdgcn_raw_buffer_load_b128(
          src.x, !TAIL || o + k * sizeof(T) < row ? i * RPL * row + at : kNowhere, 0, 0);
  }
  // 16-byte chunks of a row are exchanged by its number: the 8 rows' at one place are on distinct banks
  __device__ __forceinline__ void hand_over(const u32x4 (&x)[XL], u32x4 (*s)[LPR]) const {
#pragma unroll
    for (int i = 0; i < XL; i++) {
      const int r = i * RPL + lane / LPR;
      s[r][(lane % LPR) ^ r] = x[i];
    }
  }

  // fp32: 4 x 4 products of one element, 16 at a time, a lane's with four weight rows' and the four routed
  // rows of set g, so that no column of the product stands empty; the four sixteenths of the wave with one
  // set of weight rows hold parts of the reduction, added at the end.  8 rows an expert: 13.1 us with 16 x
  // 16 products, 11.9 with these (E = 8, K = 1024, N = 2048).
  static constexpr int SETS = sizeof(T) == 4 ? kRowsX / 4 : 1;
  __device__ __forceinline__ void multiply(const Piece& c, const Scales& sc, int p, const u32x4 (*s)[LPR], int rows,
                                           f32x4 (&acc)[P][SETS]) const {
    const int r = wr % kRowsX;
    float f[P][NB];
#pragma unroll
    for (int h = 0; h < P; h++)
#pragma unroll
      for (int b = 0; b < NB; b++) f[h][b] = scale(sc, p, h, b);
#pragma unroll
    for (int i = 0; i < Q; i++) {
      if constexpr (sizeof(T) == 2) {
        const bf16x8 x = __builtin_bit_cast(bf16x8, s[r][(16 * (i / 4) + 4 * grp + i % 4) ^ r]);
#pragma unroll
        for (int h = 0; h < P; h++)
          acc[h][0] =
              __builtin_amdgcn_mfma_f32_16x16x32_bf16(widen_bf16(c.q[h][i], f[h][i / 4]), x, acc[h][0], 0, 0, 0);
      } else {
        float w[P][8];
#pragma unroll
        for (int h = 0; h < P; h++) widen_f32(c.q[h][i], f[h][i / 4], w[h]);
#pragma unroll
        for (int g = 0; g < SETS; g++) {
          if (g > 0 && rows <= 4 * g) break;
          const int rg = 4 * g + lane % 4;
#pragma unroll
          for (int u = 0; u < 2; u++) {
            const float4 x = __builtin_bit_cast(float4, s[rg][(8 * grp + 2 * i + u) ^ rg]);
            const float xv[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
            for (int j = 0; j < 4; j++)
#pragma unroll
              for (int h = 0; h < P; h++)
                acc[h][g] = __builtin_amdgcn_mfma_f32_4x4x1f32(w[h][4 * u + j], xv[j], acc[h][g], 0, 0, 0);
          }
        }
      }
    }
  }
};

template <typename T, int P, int NB, bool TAIL>
__global__ void __launch_bounds__(64 * kStreamWaves, 4) w4_stream_kernel(W4Args a, int tiles) {
  using S = Stream<T, P, NB, TAIL>;
  constexpr int NW = kStreamWaves, ROWS = kRowsX;
  __shared__ __attribute__((aligned(16))) u32x4 s_x[NW][ROWS][S::LPR];
  __shared__ float s_acc[2][NW][P][ROWS][kRowsW + 1];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const S st{a, lane, lane & 15, lane >> 4};
  const int shares = NW / tiles, share = wave % shares, sub = wave / shares;
  const int iters = (a.K + S::SPAN * shares - 1) / (S::SPAN * shares);
  const int width = kRowsW * tiles;  // weight rows of the workgroup's tiles
  int t = first_tile();
  static_assert(ROWS == 8, "runs of the finder");
  W4Finder<ROWS> finder(a.offsets, a.E, a.N / width, lane);
  W4Tile tile = finder.find(t), ahead = tile;  // the tile in hand, and that of the next piece
  if (tile.e < 0) return;
  constexpr int GROUP = 4;  // pieces whose scales are loaded at once
  auto first = [&](int i) { return (share * iters + i) * S::SPAN; };  // element of piece i of a tile
  auto column = [&](const W4Tile& t) { return t.nt * width + kRowsW * sub; };
  int it = 0, buf = 0;
  f32x4 acc[P][S::SETS] = {};
  typename S::Piece even, odd;
  typename S::Scales now, then;  // of the pieces in hand, and of those behind them
  u32x4 x[S::XL];
  typename S::Source src = st.source(tile, column(tile));  // of the tile ahead
  st.load_scales(then, src, first(0));
  st.load_rows(x, src, first(0));
  st.load_codes(even, src, true, first(0));
  // multiplies `cur` while the piece behind it loads into `nxt`; false behind the last tile
  auto step = [&](const typename S::Piece& cur, typename S::Piece& nxt) __attribute__((always_inline)) {
    st.hand_over(x, s_x[wave]);
    const int at = it % GROUP;
    if (at == 0) st.settle(now, then, first(it));  // here, behind the rows, which were loaded after them: the copy waits for nothing else
    const bool last = ++it == iters;
    if (last) {
      it = 0;
      t += gridDim.x;
      ahead = finder.find(t);
      src = st.source(ahead, column(ahead));
    }
    const bool group = it % GROUP == 0;
    if (group) st.load_scales(then, src, first(it));
    st.load_rows(x, src, first(it));
    st.load_codes(nxt, src, ahead.e >= 0, first(it));
    wave_lds_fence();
    if (cur.live) st.multiply(cur, now, at, s_x[wave], tile.m_end - tile.m0, acc);
    wave_lds_fence();
    if (!last) return true;
#pragma unroll
    for (int h = 0; h < P; h++) {
#pragma unroll
      for (int g = 0; g < S::SETS; g++) {
        f32x4& v = acc[h][g];
        if constexpr (sizeof(T) == 2) {
          // lane l holds weight rows 4 (l / 16) .. + 3 of routed row l % 16
          if (st.wr < ROWS) {
#pragma unroll
            for (int i = 0; i < 4; i++) s_acc[buf][wave][h][st.wr][4 * st.grp + i] = v[i];
          }
        } else {
          // lane l holds weight rows 4 (l / 4 % 4) .. + 3 of routed row 4 g + l % 4, a quarter of the sum
#pragma unroll
          for (int i = 0; i < 4; i++) {
            const float half = v[i] + other_half<16>(v[i]);
            const float sum = half + other_half<32>(half);
            if (lane < 16) s_acc[buf][wave][h][4 * g + lane % 4][4 * (lane / 4) + i] = sum;
          }
        }
        v = f32x4{0.f, 0.f, 0.f, 0.f};
      }
    }
    __syncthreads();
    const int rows = tile.m_end - tile.m0;  // at most ROWS
    for (int o = tid; o < rows * width; o += 64 * NW) {
      const int r = o / width, c = o % width;
      const int w0 = (c / kRowsW) * shares;
      float v[P];
#pragma unroll
      for (int h = 0; h < P; h++) {
        auto add = [&](auto n) {  // n shares, read at once and added in order
          float part[decltype(n)::value];
#pragma unroll
          for (int w = 0; w < n; w++) part[w] = s_acc[buf][w0 + w][h][r][c % kRowsW];
          float sum = part[0];
#pragma unroll
          for (int w = 1; w < n; w++) sum += part[w];
          return sum;
        };
        v[h] = shares == 8   ? add(std::integral_constant<int, 8>())
               : shares == 4 ? add(std::integral_constant<int, 4>())
               : shares == 2 ? add(std::integral_constant<int, 2>())
                             : add(std::integral_constant<int, 1>());
      }
      float out = v[0];
      if constexpr (P == 2) out = v[0] * sigmoidf_(v[0]) * v[1];
      Elem<T>::store(static_cast<T*>(a.out) + (int64_t)(tile.m0 + r) * a.N + tile.nt * width + c, out);
    }
    buf ^= 1;  // read until the barrier of the next tile, written again behind it
    tile = ahead;
    return tile.e >= 0;
  };
  while (step(even, odd) && step(odd, even)) {
  }
}

// ---- many rows: the rows in LDS, each weight widened once for up to 96 of them
// A workgroup of NW waves takes 16 NW weight rows of both projections (gated) or 32 NW of one, 2 x 16 a
// wave, by up to 96 routed rows.  256 bytes of every routed row are staged in LDS (16-byte chunks
// exchanged by the row's number, so that 16 rows at one place fall on distinct banks) while the 256
// before are multiplied; rows are loaded into registers two steps ahead, weights three.  In bf16 its time goes
// with the bytes that a compute unit loads, weights or rows, from the L2 or from memory, at some 24 a
// nanosecond; that is this kernel's rate (rows pass through registers, all waves meet at a barrier each step,
// and each 16-byte read of LDS feeds two products), not the memory path's: loads straight to LDS take in 39 to
// 51 from the L2.  In fp32 its products bound it.  choose_tile picks the tile that needs least of both.  61 to
// 72 us at 64 rows an expert, E = 32, K = 4096, N = 1536, gated, in bf16 (237 MB and 52 GFLOP; 318 MB read from HBM),
// 13.7 us at 128 rows, E = 8, K = 1024, N = 2048.  fp32: 93 us at 151 rows, E = 8, K = 2048, N = 1024, gated (10 GFLOP),
// 35 us at 151 rows, E = 13, K = 1664, N = 192.
//
// It is made for the rows of decode batches and short prompts.  us against the bf16 GEMM with bf16 weights, E = 128, d =
// 2048, f = 1024, in (gated) and out: 99 / 224 and 66 / 118 at 64 rows an expert, 172 / 256 and 117 / 132 at 128, 336 /
// 360 and 224 / 177 at 256, 677 / 597 and 466 / 314 at 512; at 4096 (E = 8) 299 / 261 and 196 / 136.
constexpr int kTileRows = 96;

template <typename T>
struct Tile4 {
  static constexpr int KC = 256 / sizeof(T);  // elements of the reduction a step
  static constexpr int EPL = KC / 4;          // a lane's (32 or 16)
  static constexpr int Q = EPL / 8;           // code words of them
};

// A step's products for NTA runs of 16 routed rows
template <typename T, int NTA>
__device__ __forceinline__ void multiply_step(const u32x4 (*x)[16], const uint32_t (&q)[2][Tile4<T>::Q], float s0,
                                              float s1, int wr, int grp, f32x4 (&acc)[2][NTA]) {
#pragma unroll
  for (int i = 0; i < Tile4<T>::Q; i++) {
    if constexpr (sizeof(T) == 2) {
      const bf16x8 w0 = widen_bf16(q[0][i], s0), w1 = widen_bf16(q[1][i], s1);
#pragma unroll
      for (int n = 0; n < NTA; n++) {
        const bf16x8 b = __builtin_bit_cast(bf16x8, x[16 * n + wr][(grp * 4 + i) ^ wr]);
        acc[0][n] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w0, b, acc[0][n], 0, 0, 0);
        acc[1][n] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w1, b, acc[1][n], 0, 0, 0);
      }
    } else {
      float w0[8], w1[8];
      widen_f32(q[0][i], s0, w0);
      widen_f32(q[1][i], s1, w1);
#pragma unroll
      for (int u = 0; u < 2; u++) {
#pragma unroll
        for (int n = 0; n < NTA; n++) {
          const float4 b = __builtin_bit_cast(float4, x[16 * n + wr][(grp * 4 + 2 * i + u) ^ wr]);
          const float bv[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
          for (int j = 0; j < 4; j++) {
            acc[0][n] = __builtin_amdgcn_mfma_f32_16x16x4f32(w0[4 * u + j], bv[j], acc[0][n], 0, 0, 0);
            acc[1][n] = __builtin_amdgcn_mfma_f32_16x16x4f32(w1[4 * u + j], bv[j], acc[1][n], 0, 0, 0);
          }
        }
      }
    }
  }
}

// One tile with NTA runs of 16 routed rows
template <typename T, int P, int NW, int KS, bool TAIL, int NTA>
__device__ __forceinline__ void do_tile(const W4Args& a, const W4Tile& tile, u32x4 (*s_all)[2][kTileRows][16]) {
  using C = Tile4<T>;
  constexpr int KC = C::KC, EPL = C::EPL, Q = C::Q;
  constexpr int BN = 32 * NW / P;                        // weight rows of a tile (per projection)
  constexpr int XN = (NTA * 256 + 64 * NW - 1) / (64 * NW);  // 16-byte chunks of routed rows a thread loads
  const int tid = threadIdx.x % (64 * NW), lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int share = KS == 1 ? 0 : __builtin_amdgcn_readfirstlane(threadIdx.x / (64 * NW));
  u32x4(*s_x)[kTileRows][16] = s_all[share];
  const int wr = lane & 15, grp = lane >> 4;
  const int steps = (a.K + KC * KS - 1) / (KC * KS);  // of this share: KS i + share
  const int xr = tid >> 4, xc = tid & 15;  // row xr + 4 NW n, chunk xc
  const int rows = tile.m_end - tile.m0;
  // the wave's two sets of 16 weight rows: both projections of the same, or 32 of the one
  const uint32_t qb = a.K / 2, sb = a.K / kMx4Block, xb = a.K * sizeof(T);  // bytes of a row
  __amdgpu_buffer_rsrc_t qr[2], sr[2];
  int ncol[2];
#pragma unroll
  for (int h = 0; h < 2; h++) {
    ncol[h] = tile.nt * BN + (P == 2 ? 16 * wave : 32 * wave + 16 * h);
    const int64_t wrow = (int64_t)tile.e * a.N + ncol[h];
    const bool in = ncol[h] < a.N;  // N is a multiple of 16
    qr[h] = buffer((P == 2 && h ? a.q1 : a.q0) + wrow * qb, in ? 16 * qb : 0);
    sr[h] = buffer((P == 2 && h ? a.s1 : a.s0) + wrow * sb, in ? 16 * sb : 0);
  }
  const auto rr = buffer(static_cast<const T*>(a.X) + (int64_t)tile.m0 * a.K, rows * xb);
  constexpr int AHEAD = 3;  // steps that weights are loaded ahead (even + 1: the rows' sets take turns too)
  u32x4 xs[2][XN];
  uint32_t q[AHEAD + 1][2][Q];
  uint32_t sc[2][2], hi[2][2];  // of 4 steps, the lane's of step l / 16; hi: TAIL's second half
  // past the reduction's end both sides are zero
  auto load_x = [&](int step, u32x4(&x)[XN]) __attribute__((always_inline)) {
    const uint32_t o = (step * KS + share) * 256 + xc * 16;
#pragma unroll
    for (int n = 0; n < XN; n++)
      x[n] = __builtin_amdgcn_raw_buffer_load_b128(rr, o < xb ? (xr + 4 * NW * n) * xb + o : kNowhere, 0, 0);
  };
  auto load_w = [&](int step, uint32_t(&w)[2][Q]) __attribute__((always_inline)) {
    const int k = (step * KS + share) * KC + grp * EPL;
    const uint32_t qo = k < a.K ? wr * qb + k / 2 : kNowhere;
#pragma unroll
    for (int h = 0; h < 2; h++) {
      if constexpr (Q == 4) {
        const u32x4 v = __builtin_amdgcn_raw_buffer_load_b128(qr[h], qo, 0, 0);
        w[h][0] = v.x, w[h][1] = v.y, w[h][2] = v.z, w[h][3] = v.w;
      } else {
        const u32x2 v = __builtin_amdgcn_raw_buffer_load_b64(qr[h], qo, 0, 0);
        w[h][0] = v.x, w[h][1] = v.y;
      }
    }
  };
  // a row's scale bytes of four steps come in one load (TAIL: two), a step's to each of its four lanes
  auto load_s = [&](int step, int set) __attribute__((always_inline)) {
#pragma unroll
    for (int h = 0; h < 2; h++) {
      constexpr int SB = KC / kMx4Block;
      const uint32_t at = ((step + grp) * KS + share) * SB;  // past the row's end the next row's, which may be NaN
      const uint32_t o = at < sb ? wr * sb + at : kNowhere;
      if constexpr (SB == 4 && !TAIL) sc[set][h] = __builtin_amdgcn_raw_buffer_load_b32(sr[h], o, 0, 0);
      else sc[set][h] = __builtin_amdgcn_raw_buffer_load_b16(sr[h], o, 0, 0);
      if constexpr (TAIL)
        hi[set][h] = __builtin_amdgcn_raw_buffer_load_b16(sr[h], at + 2 < sb ? o + 2 : kNowhere, 0, 0);
    }
  };
  auto scale = [&](int set, int h, int v) __attribute__((always_inline)) {
    const uint32_t s = TAIL ? sc[set][h] | hi[set][h] << 16 : sc[set][h];
    const uint32_t w = __builtin_amdgcn_ds_bpermute(4 * (16 * v + wr), s);
    return mx4_scale(w >> (8 * (grp * EPL / kMx4Block)) & 255);
  };
  auto stage = [&](int buf) __attribute__((always_inline)) {
#pragma unroll
    for (int n = 0; n < XN; n++) {
      const int r = xr + 4 * NW * n;
      if (16 * NTA % (4 * NW) == 0 || r < 16 * NTA) s_x[buf][r][xc ^ (r & 15)] = xs[buf][n];
    }
  };
  f32x4 acc[2][NTA] = {};
  load_x(0, xs[0]);
#pragma unroll
  for (int v = 0; v < AHEAD; v++) load_w(v, q[v]);
  load_s(0, 0);
  load_x(1, xs[1]);
  stage(0);
  __syncthreads();
  constexpr int N = AHEAD + 1;
  static_assert(N == 4, "steps whose scales come together");
  for (int step = 0; step < steps;) {
    // a register set is loaded again the step after its use: no set is copied, which would wait for it
#pragma unroll
    for (int v = 0; v < 2 * N; v++) {
      load_x(step + 2, xs[v & 1]);
      load_w(step + AHEAD, q[(v + AHEAD) % N]);
      if (v % N == 0) load_s(step + N, v / N ^ 1);
      __builtin_amdgcn_sched_barrier(0);  // the loads go first
      multiply_step<T, NTA>(s_x[v & 1], q[v % N], scale(v / N, 0, v % N), scale(v / N, 1, v % N), wr, grp, acc);
      stage((v & 1) ^ 1);
      __syncthreads();
      if (++step == steps) break;
    }
  }
  if constexpr (KS == 2) {  // the second share's sums go through the LDS of both
    f32x4* s_sum = reinterpret_cast<f32x4*>(s_all);
    if (share == 1) {
#pragma unroll
      for (int h = 0; h < 2; h++)
#pragma unroll
        for (int n = 0; n < NTA; n++) s_sum[(h * NTA + n) * 64 * NW + tid] = acc[h][n];
    }
    __syncthreads();
    if (share == 0) {
#pragma unroll
      for (int h = 0; h < 2; h++)
#pragma unroll
        for (int n = 0; n < NTA; n++) acc[h][n] += s_sum[(h * NTA + n) * 64 * NW + tid];
    }
    __syncthreads();  // the next tile's rows go there
    if (share == 1) return;
  }
#pragma unroll
  for (int n = 0; n < NTA; n++) {
    const int r = 16 * n + wr;
    if (r < rows) {
      T* o = static_cast<T*>(a.out) + (int64_t)(tile.m0 + r) * a.N + 4 * grp;
      auto put = [&](int col, const f32x4& v) {
        if (col >= a.N) return;
        if constexpr (sizeof(T) == 2)
          *reinterpret_cast<uint2*>(o + col) = make_uint2((uint32_t)f2bf(v[0]) | ((uint32_t)f2bf(v[1]) << 16),
                                                          (uint32_t)f2bf(v[2]) | ((uint32_t)f2bf(v[3]) << 16));
        else
          *reinterpret_cast<float4*>(o + col) = make_float4(v[0], v[1], v[2], v[3]);
      };
      if constexpr (P == 2) {
        f32x4 v;
#pragma unroll
        for (int i = 0; i < 4; i++) v[i] = acc[0][n][i] * sigmoidf_(acc[0][n][i]) * acc[1][n][i];
        put(ncol[0], v);
      } else {
        put(ncol[0], acc[0][n]);
        put(ncol[1], acc[1][n]);
      }
    }
  }
}

// KS: shares of the reduction, each NW waves (2 where tiles are few: a compute unit loads for one tile alone)
template <typename T, int P, int NW, int KS, bool TAIL>
__global__ void __launch_bounds__(64 * NW * KS, NW == 12 ? 3 : 2) w4_tile_kernel(W4Args a, int cap, uint32_t cap_inv) {
  constexpr int BN = 32 * NW / P;
  __shared__ __attribute__((aligned(16))) u32x4 s_x[KS][2][kTileRows][16];
  W4Finder<16> finder(a.offsets, a.E, (a.N + BN - 1) / BN, threadIdx.x & 63, cap, cap_inv);
  for (int t = first_tile();; t += gridDim.x) {
    const W4Tile tile = finder.find(t);
    if (tile.e < 0) break;
    switch ((tile.m_end - tile.m0 + 15) / 16) {
      case 1: do_tile<T, P, NW, KS, TAIL, 1>(a, tile, s_x); break;
      case 2: do_tile<T, P, NW, KS, TAIL, 2>(a, tile, s_x); break;
      case 3: do_tile<T, P, NW, KS, TAIL, 3>(a, tile, s_x); break;
      case 4: do_tile<T, P, NW, KS, TAIL, 4>(a, tile, s_x); break;
      case 5: do_tile<T, P, NW, KS, TAIL, 5>(a, tile, s_x); break;
      default: do_tile<T, P, NW, KS, TAIL, 6>(a, tile, s_x);
    }
  }
}

// rows: of a tile, at most
unsigned w4_grid(const W4Args& p, int rows, int ntn, int per_cu) {
  const int64_t bound = ((int64_t)p.R / rows + (p.R < p.E ? p.R : p.E)) * ntn;  // tiles of any routing
  const int64_t most = (int64_t)p.cus * per_cu;
  const int64_t g = bound < most ? bound : most;
  return (unsigned)(g < 64 ? g : (g + 63) / 64 * 64);
}

template <typename T, int P, int NB, bool TAIL>
hipError_t launch_stream(const W4Args& p, int tiles, hipStream_t st) {
  // a wave has a piece in flight: three workgroups a compute unit where it is 1 KB and the registers allow
  // them (T = 32, E = 128, K = 1088, N = 2048 33.7 -> 28.7 us)
  constexpr int PER_CU = sizeof(T) == 2 && P == 1 && NB == 1 ? 3 : 2;
  hipLaunchKernelGGL((w4_stream_kernel<T, P, NB, TAIL>), dim3(w4_grid(p, kRowsX, p.N / (kRowsW * tiles), PER_CU)),
                     dim3(64 * kStreamWaves), 0, st, p, tiles);
  return hipGetLastError();
}

template <typename T, int P, int NW, int KS, bool TAIL>
hipError_t launch_tile(const W4Args& p, int cap, hipStream_t st) {
  constexpr int BN = 32 * NW / P;
  hipLaunchKernelGGL((w4_tile_kernel<T, P, NW, KS, TAIL>), dim3(w4_grid(p, 16 * cap, (p.N + BN - 1) / BN, 64)),
                     dim3(64 * NW * KS), 0, st, p, cap, (uint32_t)(((1ull << 32) + cap - 1) / cap));
  return hipGetLastError();
}

// What the tiles of a launch cost the busiest compute unit, as bytes that this kernel loads in that time (24 a
// nanosecond), for `waves` waves by up to `cap` 16s of rows, `shares` of the reduction: the bytes of its tiles,
// in fp32 their products where these take longer (25 operations a byte, of 12 rows more than there are), and
// 48 KB (2 us) a tile for its first loads and its end, more with two shares or 12 waves; a quarter of the
// largest tile for the last round, and a quarter for 12 waves, of which no two tiles share a compute unit;
// one tile of 4 waves alone loads a fifth slower.  Half of the experts leave a run unfilled, and the fullest
// have 1.6 times the average.  Fitted to 56 shapes (1 to 256 rows an expert): what it chooses takes 2.3%
// more than the fastest choice on average, 22% at worst.
struct TileChoice {
  int waves, shares, cap;
  double cost;
};
template <typename T, int P>
double tile_cost(const W4Args& p, int waves, int shares, int cap) {
  const double k = p.K, bn = 32 * waves / P, experts = p.R < p.E ? p.R : p.E, rows = p.R / experts;
  const double filled = p.R / (16.0 * cap) + experts / 2, runs = filled > experts ? filled : experts;
  const double tiles = runs * ((p.N + (int)bn - 1) / (int)bn);
  auto work = [&](double r) {
    const double units = ((int)r + 15) / 16 * 16;
    const double bytes = r * k * sizeof(T) + bn * P * k * 17 / 32, products = (units + 12) * bn * P * k * 2 / 25;
    return (sizeof(T) == 4 && products > bytes ? products : bytes) + 49152 * (shares == 2 ? 1.5 : waves == 12 ? 2 : 1);
  };
  const double most = 1.6 * rows < 16 * cap ? ((int)(1.6 * rows) + 15) / 16 * 16 : 16 * cap;
  double one = work(most);
  if (shares == 1 && waves == 4) one *= 1.2;
  const double all = tiles * work(p.R / runs) / p.cus + one / 4;
  return (all > one ? all : one) * (waves == 12 ? 1.25 : 1);
}
// The same of streaming: the bytes of its tiles, whose 16 weight rows load the routed rows again, and 72 KB; in
// fp32 its products, 22 bytes an element of 16 weight rows by four routed ones.  A tile's end counts as 128
// elements of the reduction
template <typename T, int P>
double stream_cost(const W4Args& p) {
  const double experts = p.R < p.E ? p.R : p.E, cus = p.cus;
  if (sizeof(T) == 4) return (p.R / 4.0 + experts / 2) * P * (p.N / kRowsW) * (p.K + 128.0) * 22 / cus;
  const double filled = (double)p.R / kRowsX + experts / 2, runs = filled > experts ? filled : experts;
  return runs * (p.N / kRowsW) * (p.K + 128.0) * (8.5 * P + 2 * p.R / runs) / cus + 73728;
}

// us of the alternatives (waves x shares, 16s a tile): 4 x 1, 6: 89, 4 x 1, 3: 97, 12 x 1, 6: 70 (64 rows an expert,
// E = 32, K = 4096, N = 1536, gated); 45, 51, 49 (32 rows, E = 64, K = 2048, N = 1024); 4 x 2, 6: 27, 4 x 2, 2: 17
// (150 rows, E = 4, K = 4096, N = 512); fp32 83 and, 4 x 2, 2: 33 (151 rows, E = 13, K = 1664, N = 192)
template <typename T, int P>
TileChoice choose_tile(const W4Args& p) {
  TileChoice best{4, 1, 6, tile_cost<T, P>(p, 4, 1, 6)};
  auto consider = [&](int waves, int shares, int cap) {
    const double c = tile_cost<T, P>(p, waves, shares, cap);
    if (c < best.cost) best = TileChoice{waves, shares, cap, c};
  };
  for (const int cap : {6, 3, 2, 1}) {
    consider(4, 1, cap);
    consider(4, 2, cap);
  }
  if (sizeof(T) == 2) consider(12, 1, 6);
  return best;
}

template <typename T, int P, bool TAIL>
hipError_t launch_tiles(const W4Args& p, const TileChoice& c, hipStream_t st) {
  if constexpr (sizeof(T) == 2) {
    if (c.waves == 12) return launch_tile<T, P, 12, 1, TAIL>(p, c.cap, st);
  }
  if (c.shares == 2) return launch_tile<T, P, 4, 2, TAIL>(p, c.cap, st);
  return launch_tile<T, P, 4, 1, TAIL>(p, c.cap, st);
}

// Tiles of a streaming workgroup, and so shares of the reduction (8 / tiles): the number that takes the
// fewest rounds of pieces, a tile's end counting as some two of them (barrier and sums of the shares).
// More shares than pieces leave waves idle, fewer tiles than the device holds leave it idle.
// us with 1, 2, 4 tiles: 5.2, 4.3, 5.0 (T = 1, K = 1024, N = 2048, not gated), 9.3, 8.9, 7.5 (T = 10, E = 31, K =
// 1280, N = 448), 16.9, 15.7, 14.4 (T = 8, E = 128, K = 2048, N = 1024); with 2, 4, 8: 20, 12, 9.5 (T = 32, E = 128,
// K = 256, N = 2048).
int stream_tiles(const W4Args& p, int span) {
  const int64_t experts = p.R < p.E ? p.R : p.E, rows = (p.R + experts - 1) / experts;
  const int64_t all = experts * ((rows + kRowsX - 1) / kRowsX) * (p.N / kRowsW), fit = p.cus;
  int best = 1;
  int64_t least = INT64_MAX;
  for (int tiles = 1; tiles <= kStreamWaves; tiles *= 2) {
    const int shares = kStreamWaves / tiles;
    if (p.N % (kRowsW * tiles) != 0 || (shares == 1 && p.K > 256)) break;
    const int64_t cost = ((all / tiles + fit - 1) / fit) * (((int64_t)p.K + span * shares - 1) / (span * shares) + 2);
    if (cost < least) least = cost, best = tiles;
  }
  return best;
}

template <typename T, int P>
hipError_t launch_w4(const W4Args& p, hipStream_t st) {
  if (p.R == 0) return hipSuccess;
  // weights that stream past the rows or tiles of many rows, us: 5 / 8.5 (32 rows, E = 1, K = 2048, N = 1024, gated),
  // 55 / 64 (4 rows, E = 128, the same), 24.5 / 15.3 (8 rows, E = 8, K = 4096, N = 1536), 8.7 / 7.1 (16 rows, E = 8, K =
  // 1024, N = 2048, not gated); fp32 6.5 / 14.5 (30 rows, E = 2), 13.4 / 14.9 (12 rows, E = 8), 17.2 / 15.2 (16
  // rows, E = 8; all three K = 1024, N = 1024 or 2048)
  const TileChoice tile = choose_tile<T, P>(p);
  if (tile.cost < stream_cost<T, P>(p)) {
    if constexpr (sizeof(T) == 2) {
      if (p.K % 128 != 0) return launch_tiles<T, P, true>(p, tile, st);
    }
    return launch_tiles<T, P, false>(p, tile, st);
  }
  const int tiles = stream_tiles(p, sizeof(T) == 2 && p.K % 256 == 0 ? 256 : 128);
  if (p.K % 128 != 0) return launch_stream<T, P, 1, true>(p, tiles, st);
  // two blocks a piece where every share has one of them (fp32 rows would not fit the registers)
  if constexpr (sizeof(T) == 2) {
    if (p.K % 256 == 0 && p.K >= 256 * kStreamWaves / tiles) return launch_stream<T, P, 2, false>(p, tiles, st);
  }
  return launch_stream<T, P, 1, false>(p, tiles, st);
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
  const W4Args p{g.R, g.d, g.f, g.E, offsets, X, W1q, W1s, W3q, W3s, h, device_cu_count()};
  return eb == 2 ? launch_w4<bf16_t, 2>(p, st) : launch_w4<float, 2>(p, st);
}

hipError_t gemm2_fwd_w4(int eb, const GemmShape& g, const int* offsets, const void* H, const uint8_t* W2q,
                        const uint8_t* W2s, void* Y, hipStream_t st) {
  const W4Args p{g.R, g.f, g.d, g.E, offsets, H, W2q, W2s, nullptr, nullptr, Y, device_cu_count()};
  return eb == 2 ? launch_w4<bf16_t, 1>(p, st) : launch_w4<float, 1>(p, st);
}

}  // namespace moe
