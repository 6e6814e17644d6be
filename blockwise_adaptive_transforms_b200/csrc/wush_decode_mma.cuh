// The product core of the few-token operators: rows of 4-bit weights against up to 16 columns
// of fp16 activations on warp-level tensor-core instructions (mma.sync m16n8k16, fp32 sums).
//
// The weights bound these products: one pass over them from memory, 23.5 bytes per clock and
// SM at the measured copy rate, which is 47 weights, against 128 issued lanes per clock.  So
// a weight may cost at most 2.7 issued lanes in all.  E2M1 codes become fp16 pairs with one
// conversion per two weights (measured: conversions and logic operations share 64 lanes per
// clock and SM); INT4 codes with one logic operation and one fp16 subtraction or
// fused multiply-add per two.  Products and sums go to the tensor cores: 256 weights per
// instruction and warp, 8 columns (measured 992 multiply-adds per clock and SM, or 124 weights).
// tcgen05's kind::f16 would need fp16 weights in shared memory, written there by the same conversions; its
// block-scaled kinds take E2M1 weights and their scales as they are, but activations of 8 bits at
// most, so several columns for the 11 bits held here: not built, not measured.
// Measured, all told: 59 weights per clock and SM with four groups per instruction (fp32 results,
// so two columns), 33 with one group and 16 columns, where the warps' chains of instructions are what
// is waited for (602 for 64 rows by 128 channels, half of the issue slots with two warps a scheduler; no
// pipe is full).
//
// Group scales cannot be applied before the sum over a group (E8M0 and fp32 scales do not fit
// fp16), so an instruction's sum must stay inside one group, or keep the groups apart.  Both
// follow from which columns hold what.  Lane 4 g + t of a warp holds weights of rows g and
// g + 8; the order of k inside an instruction is free as long as both operands share it.
//   NG = 4: each lane takes 16 bytes of a row; the four lanes of a row hold four groups of 32.
//           Column 2 j + v holds token v's activations of group j and zeros elsewhere, so one
//           instruction serves 2 tokens and lane t reads its own group's sums.
//   NG = 2: 8 bytes per lane, two groups per instruction, 4 tokens.
//   NG = 1: 4 bytes per lane, one group, 8 tokens (NC = 2 such column tiles: 16).
// NVFP4's E4M3 scales do fit: e2m1 * e4m3 has at most 6 significant bits and stays within
// [2^-10, 2688], so the pair is multiplied by its scale in fp16, exactly, and only the
// activations' scale is applied to the sums.
#pragma once
#include "wush_decode.cuh"

namespace wush {
namespace decode {

// Transformed activations in memory: columns v of fp16 [ld] with one fp32 scale, a power of
// two, per 32 or 128 channels (the kernels' PER_SCALE).  Inside each run of 8 channels the order
// is the one in which the weight conversion delivers them.
struct Columns {
  const __half* y;
  const float* s;
  int ld;   // channels per column, a multiple of 128; s has ld / 32 places per column
};

__device__ __forceinline__ uint32_t h2u(__half2 h) { return *reinterpret_cast<uint32_t*>(&h); }
__device__ __forceinline__ __half2 u2h(uint32_t u) { return *reinterpret_cast<__half2*>(&u); }

// 8 codes -> four fp16 pairs.  E2M1: pair i is codes (2i, 2i + 1).  INT4: codes (i, i + 4).
template <int FMT>
__device__ __forceinline__ void unpack8(uint32_t w, uint32_t (&p)[4]) {
  if constexpr (FMT == kInt) {
    // a nibble in an fp16 mantissa: 0x6400 | n = 1024 + n, and n ^ 8 = q + 8
    const uint32_t hi = w >> 8;
    p[0] = h2u(__hsub2(u2h((w & 0x000F000Fu) ^ 0x64086408u), u2h(0x64086408u)));            // - 1032
    p[1] = h2u(__hfma2(u2h((w & 0x00F000F0u) ^ 0x64806480u), u2h(0x2C002C00u), u2h(0xD480D480u)));   // / 16 - 72
    p[2] = h2u(__hsub2(u2h((hi & 0x000F000Fu) ^ 0x64086408u), u2h(0x64086408u)));
    p[3] = h2u(__hfma2(u2h((hi & 0x00F000F0u) ^ 0x64806480u), u2h(0x2C002C00u), u2h(0xD480D480u)));
  } else {
    asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, a;\n\tcvt.rn.f16x2.e2m1x2 %1, b;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, c;\n\tcvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
        : "=r"(p[0]), "=r"(p[1]), "=r"(p[2]), "=r"(p[3])
        : "r"(w));
  }
}

// where channel k of a run of 8 goes in that order
template <int FMT>
__device__ __forceinline__ int pair_place(int k) {
  return FMT == kInt ? (k < 4 ? 2 * k : 2 * (k - 4) + 1) : k;
}

// c = a b, and c += a b
__device__ __forceinline__ void mma16816_first(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                               uint32_t b0, uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
}
__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// pairs of fp32 in one instruction
__device__ __forceinline__ uint64_t pack2(float a, float b) {
  uint64_t v;
  asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(a), "f"(b));
  return v;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t v;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(v) : "l"(a), "l"(b));
  return v;
}
__device__ __forceinline__ void fma2(uint64_t& c, uint64_t a, uint64_t b) {
  asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(c) : "l"(a), "l"(b));
}
__device__ __forceinline__ float low(uint64_t v) { return __uint_as_float(static_cast<uint32_t>(v)); }
__device__ __forceinline__ float high(uint64_t v) { return __uint_as_float(static_cast<uint32_t>(v >> 32)); }

template <class V>
__device__ __forceinline__ V at(const uint8_t* p) {
  return *reinterpret_cast<const V*>(p);
}

// volatile: in order with the waits and arrivals of a stage, but without a hold on other loads
__device__ __forceinline__ void load_matrix4(uint32_t (&q)[4], uint32_t shared) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(q[0]), "=r"(q[1]), "=r"(q[2]), "=r"(q[3]) : "r"(shared));
}

// Warps that compute: as many as their registers leave room for (12 leave 128 to a thread, where two
// column tiles need up to 168).  64 experts of 4096 x 1536, 32 tokens: 154 us with 8, 141 us with 12.
__host__ __device__ constexpr int compute_warps(int ng) { return ng == 1 ? 8 : 12; }

// Warps that share a stage's channels.  57344 x 8192 with 16 tokens: 88.9 us with two, 82.4 with four.
constexpr int kAlongK = 4;

// A stage of weights in shared memory, which the warps take as WR x kAlongK parts of 64 rows by 128
// channels: ROWS = 64 WR rows by kAlongK / 2 boxes of 128 bytes (256 channels).  In a box, row r has its
// 16-byte unit u at unit u ^ (r & 7) (the 128-byte swizzle of tensor copies): the reads of eight
// rows' equal units then meet in no bank.  Then the rows' scales, SROW bytes each.
// EXACT: rows of K / G one-byte scales start at multiples of a stage's worth of them (INT4: 16
// bytes); else one-byte scales come as the aligned words that hold them.
template <int FMT, int G, int NG, bool EXACT>
struct Stage {
  static constexpr int WARPS = compute_warps(NG), WR = WARPS / kAlongK, ROWS = 64 * WR, STEP = 128 * kAlongK;   // rows and channels
  static constexpr int PER = 128 / G;                                   // groups of a row per warp
  static constexpr int BOX = ROWS * 128, CODES = kAlongK / 2 * BOX;
  static constexpr int SROW = FMT == kInt ? 4 * PER * kAlongK + 16 : PER * kAlongK + (EXACT ? 0 : 4);
  static constexpr int SCALES = (ROWS * SROW + 15) / 16 * 16;

  // scales of channels 128 wk .. of a row (one byte each)
  static __device__ __forceinline__ void byte_scales(const uint8_t* sc, int row, int wk, uint32_t shift, int left,
                                                     uint32_t (&w)[PER / 4]) {
    const uint8_t* a = sc + row * SROW + wk * PER;
    if constexpr (EXACT) {
      if constexpr (PER == 4) {
        w[0] = at<uint32_t>(a);
      } else {
        const uint2 v = at<uint2>(a);
        w[0] = v.x, w[1] = v.y;
      }
    } else {
      uint32_t v[PER / 4 + 1];
#pragma unroll
      for (int j = 0; j <= PER / 4; ++j) v[j] = at<uint32_t>(a + 4 * j);
#pragma unroll
      for (int j = 0; j < PER / 4; ++j) {
        // bytes past the row belong to others; as NaNs they would outlive a product with zero
        const int n = left - 4 * j;
        const uint32_t keep = n >= 4 ? 0xFFFFFFFFu : n <= 0 ? 0u : (1u << (8 * n)) - 1u;
        w[j] = __funnelshift_r(v[j], v[j + 1], shift) & keep;
      }
    }
  }
};

// tokens (columns in memory) that one instruction set of NG serves
__host__ __device__ constexpr int columns_of(int NG, int NC) { return NG == 4 ? 2 : NG == 2 ? 4 : 8 * NC; }

// this lane's column in memory by its g (null where the instruction's column is zero for its t)
template <int NG>
__device__ __forceinline__ int lane_column(int g, int t) {
  if constexpr (NG == 4) return (g >> 1) == t ? (g & 1) : -1;
  if constexpr (NG == 2) return (g >> 2) == (t >> 1) ? (g & 3) : -1;
  return g;
}
// the column of the sums acc[..][j], j = 0, 1
template <int NG>
__device__ __forceinline__ int sum_column(int t, int j) {
  if constexpr (NG == 4) return j;
  if constexpr (NG == 2) return 2 * (t & 1) + j;
  return 2 * t + j;
}

// The activations of a stage in shared memory: columns of STEP channels, 64 bytes apart in the banks
// from their neighbours (so for every NG), then each column's scales.
constexpr int kColumnPitch = 256 * kAlongK + 64;

// two E8M0 bytes -> 2^(b - 127), exactly (bf16 holds them, 2^-127 as a subnormal)
__device__ __forceinline__ void e8m0_pair(uint32_t two, float& lo, float& hi) {
  uint32_t v;
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %1;\n\tcvt.rn.bf16x2.ue8m0x2 %0, a;\n\t}" : "=r"(v) : "r"(two));
  lo = __uint_as_float(v << 16);
  hi = __uint_as_float(v & 0xFFFF0000u);
}
// two E4M3 bytes -> an fp16 pair
__device__ __forceinline__ uint32_t e4m3_pair(uint32_t two) {
  uint32_t v;
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\t}" : "=r"(v) : "r"(two));
  return v;
}

// Sums of one warp: acc[i][c][h] is row g + 8 h, columns 8 c + 2 t (low) and 8 c + 2 t + 1 (high) of
// the instruction (tokens by NG as above).
template <int FMT, int G, int NG, int NC, int PER_SCALE, bool EXACT>
struct Core {
  static_assert(NG == 1 || NC == 1, "one column tile where groups share an instruction");
  using S = Stage<FMT, G, NG, EXACT>;
  static constexpr int MT = 4;   // tiles of 16 rows
  static constexpr int UNITS = NG == 4 ? 1 : NG == 2 ? 2 : 4;   // instruction groups per step
  static constexpr int WORDS = 4 / UNITS;                       // words of 8 codes per lane and unit
  static constexpr int SETS = FMT == kInt && G == 16 ? 2 : 1;   // separate sums per unit
  static constexpr int COLS = columns_of(NG, NC);
  static constexpr int YS = PER_SCALE == 128 ? 1 : 4;           // activation scales of a column per warp
  static constexpr int COLUMN_SCALES = 4 * YS * kAlongK;             // bytes per column and stage
  uint64_t acc[MT][NC][2];
  // Activations of a step where lanes without a column exist: theirs stay zero from the start, so that
  // a step writes the others' alone
  uint4 kept[NG > 1 ? UNITS : 1][NG > 1 ? WORDS : 1];

  __device__ __forceinline__ void begin() {
    if constexpr (NG > 1) {
#pragma unroll
      for (int u = 0; u < UNITS; ++u)
#pragma unroll
        for (int w = 0; w < WORDS; ++w) kept[u][w] = make_uint4(0u, 0u, 0u, 0u);
    }
  }
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int c = 0; c < NC; ++c) acc[i][c][0] = acc[i][c][1] = 0ull;
  }

  // c += a b, in two columns, or (MASKED) in those of them that are on
  template <bool MASKED>
  static __device__ __forceinline__ void accumulate(uint64_t& c, uint64_t a, uint64_t b, const bool (&on)[2]) {
    if constexpr (!MASKED) fma2(c, a, b);
    else c = pack2(on[0] ? fmaf(low(a), low(b), low(c)) : low(c), on[1] ? fmaf(high(a), high(b), high(c)) : high(c));
  }

  // Which row of a tile's 8 is an instruction's row g: the order that keeps the reads of neighbouring
  // lanes in different banks (eight lanes read 16 bytes each of two rows, or sixteen 8 bytes of four).
  static __device__ __forceinline__ int row_of(int g) {
    if constexpr (NG == 4) return (g >> 1) | (g & 1) << 2;
    if constexpr (NG == 2) return (g & 3) << 1 | g >> 2;
    return g;
  }
  static __device__ __forceinline__ int tile_row(int i, int r0, int r1) { return (i < 2 ? r0 : r1) + 16 * (i & 1); }

  // Adds this warp's part of a stage: its rows r0 .. r0 + 31 and r1 .. r1 + 31, channels 128 wk ...
  //   a: codes of the stage; sc: scales; y: columns; ys: their scales
  //   shift: by tile and half, for one-byte scales that are not aligned; left: groups up to K
  //   live: (MASKED) bit v says that column v holds activations.  The others keep their sums: they are left
  //   out of the addition, since a product with zero is a NaN where the weights' scale is not finite; what
  //   the stage holds in their place is multiplied along and reaches no other column
  //   mul: factors on the columns whose sums this lane holds; ts: the tensor scale
  // The scales are multiplied with one another before a sum, NVFP4's tensor scale with the
  // activations' scale: a sum under one of them alone can overflow where the result does not.
  template <bool MASKED>
  __device__ __forceinline__ void add(const uint8_t* a, const uint8_t* sc, const uint8_t* y, const uint8_t* ys, int r0,
                                      int r1, int wk, const uint32_t (&shift)[MT][2], int left, uint32_t live,
                                      const float (&mul)[NC][2], float ts, int lane) {
    const int g = lane >> 2, t = lane & 3, rg = row_of(g);
    uint64_t sy[NC][YS == 1 ? 1 : UNITS];
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      float f2[2][YS == 1 ? 1 : UNITS];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int v = 8 * c + sum_column<NG>(t, j);
        const float f = FMT == kNv ? ts * mul[c][j] : mul[c][j];
        const uint8_t* p = ys + v * COLUMN_SCALES + 4 * YS * wk;
        if constexpr (YS == 1) {
          f2[j][0] = at<float>(p) * f;
        } else if constexpr (NG == 1) {
          const float4 q = at<float4>(p);
          f2[j][0] = q.x * f, f2[j][1] = q.y * f, f2[j][2] = q.z * f, f2[j][3] = q.w * f;
        } else {
#pragma unroll
          for (int u = 0; u < UNITS; ++u) f2[j][u] = at<float>(p + 4 * (NG == 4 ? t : 2 * u + t / 2)) * f;
        }
      }
#pragma unroll
      for (int u = 0; u < (YS == 1 ? 1 : UNITS); ++u) sy[c][u] = pack2(f2[0][u], f2[1][u]);
    }
    const int mine_v = lane_column<NG>(g, t);
    bool on[NC][2];
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
      for (int j = 0; j < 2; ++j) on[c][j] = !MASKED || (live >> (8 * c + sum_column<NG>(t, j)) & 1u);
    // scales of the weights, by unit (and set): MXFP4 and INT4 fp32, NVFP4 an fp16 pair per word
    float sw[MT][2][UNITS * SETS];
    uint32_t sn[MT][2][FMT == kNv ? (NG == 4 ? 2 : UNITS) : 1];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int row = tile_row(i, r0, r1) + 8 * h + rg;
        if constexpr (FMT == kMx) {
          uint32_t w[1];
          if constexpr (NG == 4 && EXACT) {
            // 2^(b - 127); the smallest is subnormal, and the byte 255 is a NaN
            const uint32_t b = sc[row * S::SROW + 4 * wk + t];
            sw[i][h][0] = __uint_as_float(b == 255u ? 0x7FFFFFFFu : max(b << 23, 0x00400000u));
          } else if constexpr (NG == 4) {
            S::byte_scales(sc, row, wk, shift[i][h], left, w);
            float unused;
            e8m0_pair(w[0] >> (8 * t) & 255u, sw[i][h][0], unused);
          } else {
            S::byte_scales(sc, row, wk, shift[i][h], left, w);
            float s0, s1, s2, s3;
            if constexpr (NG == 2) w[0] = t & 2 ? w[0] >> 8 : w[0];   // bytes 0, 2 or 1, 3
            e8m0_pair(w[0], s0, s1);
            e8m0_pair(w[0] >> 16, s2, s3);
            if constexpr (NG == 1) sw[i][h][0] = s0, sw[i][h][1] = s1, sw[i][h][2] = s2, sw[i][h][3] = s3;
            else sw[i][h][0] = s0, sw[i][h][1] = s2;
          }
        } else if constexpr (FMT == kNv) {
          uint32_t w[2];
          S::byte_scales(sc, row, wk, shift[i][h], left, w);
          if constexpr (NG == 4) {   // groups 2 t, 2 t + 1
            const uint32_t p = e4m3_pair((t & 2 ? w[1] : w[0]) >> (16 * (t & 1)));
            sn[i][h][0] = __byte_perm(p, 0u, 0x1010), sn[i][h][1] = __byte_perm(p, 0u, 0x3232);
          } else if constexpr (NG == 2) {   // group 4 u + t
            const uint32_t pick = t & 1 ? 0x3232u : 0x1010u;
            sn[i][h][0] = __byte_perm(e4m3_pair(w[0] >> (8 * (t & 2))), 0u, pick);
            sn[i][h][1] = __byte_perm(e4m3_pair(w[1] >> (8 * (t & 2))), 0u, pick);
          } else {   // group 2 u + t / 2
            const uint32_t pick = t & 2 ? 0x3232u : 0x1010u;
            sn[i][h][0] = __byte_perm(e4m3_pair(w[0]), 0u, pick);
            sn[i][h][1] = __byte_perm(e4m3_pair(w[0] >> 16), 0u, pick);
            sn[i][h][2] = __byte_perm(e4m3_pair(w[1]), 0u, pick);
            sn[i][h][3] = __byte_perm(e4m3_pair(w[1] >> 16), 0u, pick);
          }
        } else {
          const uint8_t* q = sc + row * S::SROW + 4 * S::PER * wk;
          // groups: NG = 4: of this lane's 32 channels; NG = 2: of its half of each unit; NG = 1: all
#pragma unroll
          for (int u = 0; u < UNITS; ++u)
#pragma unroll
            for (int x = 0; x < SETS; ++x) {
              const int gi = SETS * (NG == 4 ? t : NG == 2 ? 2 * u + t / 2 : u) + x;
              sw[i][h][SETS * u + x] = at<float>(q + 4 * gi);
            }
        }
      }
    uint64_t part[MT][NC][2];   // NVFP4 with one activation scale per step: the step's sums
    const int base = 4 * (wk & 1);   // this warp's 16-byte units of a row
    const uint8_t* box = a + (wk >> 1) * S::BOX;
    const uint8_t* ya = y + (NG == 1 || mine_v >= 0 ? mine_v : 0) * kColumnPitch + 256 * wk + 16 * WORDS * t;
#pragma unroll
    for (int u = 0; u < UNITS; ++u) {
      uint4 b[NC][WORDS];
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        // channels of word w: NG = 4: 32 t + 8 w; NG = 2: 64 u + 16 t + 8 w; NG = 1: 32 u + 8 t
#pragma unroll
        for (int w = 0; w < WORDS; ++w) {
          const uint8_t* from = ya + 8 * c * kColumnPitch + (256 / UNITS) * u + 16 * w;
          if constexpr (NG == 1) {
            b[c][w] = at<uint4>(from);
          } else {
            if (mine_v >= 0) kept[u][w] = at<uint4>(from);
            b[c][w] = kept[u][w];
          }
        }
      }
      uint32_t q[MT][2][WORDS];
      if constexpr (NG == 1) {
        // four 8 x 8 matrices of 16-bit places: rows g and g + 8 of two tiles; lane l points at row l of
        // them, and lane 4 g + t receives word t of row g of each
#pragma unroll
        for (int i = 0; i < MT; i += 2) {
          uint32_t m[4];
          const int row = (i ? r1 : r0) + lane;
          load_matrix4(m, static_cast<uint32_t>(__cvta_generic_to_shared(box + row * 128 + 16 * ((base + u) ^ (lane & 7)))));
          q[i][0][0] = m[0], q[i][1][0] = m[1], q[i + 1][0][0] = m[2], q[i + 1][1][0] = m[3];
        }
      } else {
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint8_t* row = box + (tile_row(i, r0, r1) + 8 * h + rg) * 128;
            if constexpr (NG == 4) {
              const uint4 v = at<uint4>(row + 16 * ((base + t) ^ rg));
              q[i][h][0] = v.x, q[i][h][1] = v.y, q[i][h][WORDS - 2] = v.z, q[i][h][WORDS - 1] = v.w;
            } else {
              const uint2 v = at<uint2>(row + 16 * ((base + 2 * u + (t >> 1)) ^ rg) + 8 * (t & 1));
              q[i][h][0] = v.x, q[i][h][WORDS - 1] = v.y;
            }
          }
      }
      // INT4 with two groups per 32 channels: NG = 4: words 0-1 and 2-3 of a lane; NG = 2: even and odd
      // lanes; NG = 1: lanes 0-1 and 2-3.  The other group's activations are zeroed.
      float c4[MT][SETS][NC][4];
#pragma unroll
      for (int w = 0; w < WORDS; ++w) {
#pragma unroll
        for (int i = 0; i < MT; ++i) {
          uint32_t p[4], r[4];
          unpack8<FMT>(q[i][0][w], p);
          unpack8<FMT>(q[i][1][w], r);
          if constexpr (FMT == kNv) {
            const int x = NG == 4 ? w / 2 : u;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              p[j] = h2u(__hmul2(u2h(p[j]), u2h(sn[i][0][x])));
              r[j] = h2u(__hmul2(u2h(r[j]), u2h(sn[i][1][x])));
            }
          }
#pragma unroll
          for (int x = 0; x < SETS; ++x) {
            if (SETS == 2 && NG == 4 && w / 2 != x) continue;
            const bool mine = SETS == 1 || NG == 4 || (NG == 2 ? (t & 1) == x : (t >> 1) == x);
            const bool begins = w == (SETS == 2 && NG == 4 ? 2 * x : 0);
#pragma unroll
            for (int c = 0; c < NC; ++c) {
              const uint32_t b0 = mine ? b[c][w].x : 0u, b1 = mine ? b[c][w].y : 0u;
              const uint32_t b2 = mine ? b[c][w].z : 0u, b3 = mine ? b[c][w].w : 0u;
              if (begins) mma16816_first(c4[i][x][c], p[0], r[0], p[1], r[1], b0, b1);
              else mma16816(c4[i][x][c], p[0], r[0], p[1], r[1], b0, b1);
              mma16816(c4[i][x][c], p[2], r[2], p[3], r[3], b2, b3);
            }
          }
        }
      }
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int x = 0; x < SETS; ++x)
#pragma unroll
          for (int c = 0; c < NC; ++c)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const uint64_t sum = pack2(c4[i][x][c][2 * h], c4[i][x][c][2 * h + 1]);
              if constexpr (FMT == kNv && PER_SCALE == 128) {
                part[i][c][h] = u == 0 ? sum : add2(part[i][c][h], sum);
              } else if constexpr (FMT == kNv) {
                accumulate<MASKED>(acc[i][c][h], sum, sy[c][YS == 1 ? 0 : u], on[c]);
              } else {
                const float w = sw[i][h][SETS * u + x];
                const uint64_t y2 = sy[c][YS == 1 ? 0 : u];
                accumulate<MASKED>(acc[i][c][h], sum, pack2(w * low(y2), w * high(y2)), on[c]);
              }
            }
    }
    if constexpr (FMT == kNv && PER_SCALE == 128) {
      static_assert(!MASKED, "sums per step go to every column");
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int c = 0; c < NC; ++c)
#pragma unroll
          for (int h = 0; h < 2; ++h) fma2(acc[i][c][h], part[i][c][h], sy[c][0]);
    }
  }

  // sums over the lanes of a row that hold different groups of the same column
  __device__ __forceinline__ void join() {
    if constexpr (NG > 1) {
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float v0 = low(acc[i][0][h]), v1 = high(acc[i][0][h]);
          if constexpr (NG == 4) v0 += __shfl_xor_sync(0xffffffffu, v0, 1), v1 += __shfl_xor_sync(0xffffffffu, v1, 1);
          v0 += __shfl_xor_sync(0xffffffffu, v0, 2), v1 += __shfl_xor_sync(0xffffffffu, v1, 2);
          acc[i][0][h] = pack2(v0, v1);
        }
    }
  }

  // to red[column * pitch + row]
  __device__ __forceinline__ void put(float* red, int pitch, int r0, int r1, int lane) const {
    const int rg = row_of(lane >> 2), t = lane & 3;
    if (NG > 1 && t >= 4 / NG) return;   // NG = 4: lane 0 has both columns; NG = 2: lanes 0 and 1
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int c = 0; c < NC; ++c)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int v = 8 * c + sum_column<NG>(t, j);
          red[v * pitch + tile_row(i, r0, r1) + rg] = j ? high(acc[i][c][0]) : low(acc[i][c][0]);
          red[v * pitch + tile_row(i, r0, r1) + rg + 8] = j ? high(acc[i][c][1]) : low(acc[i][c][1]);
        }
  }
};

}  // namespace decode
}  // namespace wush
