// The product core of the few-token operators: rows of 4-bit weights against up to 16 columns
// of fp16 activations on warp-level tensor-core instructions (mma.sync m16n8k16, fp32 sums).
//
// The weights bound these products: one pass over them from memory, 23.5 bytes per clock and
// SM at the measured copy rate, which is 47 weights, against 128 issued lanes per clock.  So
// a weight may cost at most 2.7 issued lanes in all.  E2M1 codes become fp16 pairs with one
// conversion per two weights (measured 64 lanes per clock and SM, against four shifts and
// logic operations by hand); INT4 codes with one logic operation and one fp16 subtraction or
// fused multiply-add per two.  Products and sums go to the tensor cores: 256 weights per
// instruction and warp, 8 columns.  tcgen05 would need fp16 weights in shared memory, written
// there by the same conversions.
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
// activations' scale per 32 channels is applied to the sums.
#pragma once
#include "wush_decode.cuh"

namespace wush {
namespace decode {

// Transformed activations in memory: columns v of fp16 [ld] with one fp32 scale, a power of
// two, per 32 channels.  Inside each run of 8 channels the order is the one in which the
// weight conversion delivers them.
struct Columns {
  const __half* y;
  const float* s;
  int ld;   // channels per column, a multiple of 128; s has ld / 32 per column
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

__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t shared_address(const void* p) {
  return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}
// asynchronous copies to shared memory; `bytes` of them come from memory, the rest are zeros
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void copy8(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void copy4(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

__device__ __forceinline__ uint32_t lds4(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ uint2 lds8(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ uint4 lds16(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
  return v;
}

// A tile of rows of one matrix: rows 0..span from each of two bases, the first and the second
// half of the tile's 16 MT rows (a plain tile has the second base 8 MT rows after the first).
// Rows past span repeat row span; their sums are not used.
struct Tile {
  const uint8_t* c[2];
  const uint8_t* s[2];
  int span[2];
};

template <int FMT, int G, int MT>
__device__ __forceinline__ Tile plain_tile(const Matrix4& w, long long row, long long left) {
  const long long cp = w.K / 2, sp = static_cast<long long>(w.K / G) * (FMT == kInt ? 4 : 1);
  constexpr int half = 8 * MT;
  Tile t;
  t.c[0] = w.codes + row * cp;
  t.s[0] = static_cast<const uint8_t*>(w.scales) + row * sp;
  // a second half that lies past the matrix repeats the first half's last row
  const bool two = left > half;
  const long long second = two ? half : left - 1;
  t.c[1] = t.c[0] + second * cp;
  t.s[1] = t.s[0] + second * sp;
  t.span[0] = static_cast<int>(left > half ? half : left) - 1;
  t.span[1] = two ? static_cast<int>(left > 2 * half ? half : left - half) - 1 : 0;
  return t;
}

// One warp's ring of steps in shared memory.  A step is 16 MT rows by 128 channels: 64 bytes
// of codes per row, in 16-byte units that are exchanged by row so that neither the copies nor the
// reads below meet in a bank, then the scales.  Copies are 16 bytes a lane, four lanes a row, and
// run kStages - 1 steps ahead: at two CTAs of 8 warps per SM that is about 100 KB in flight.
// FULL: K is a multiple of 128 and the scales are aligned to a step's worth of them; else ends
// are zero-filled, rows may start at 8-byte boundaries, and one-byte scales at any.
constexpr int kStages = 4;

template <int FMT, int G, int MT, bool FULL>
struct Ring {
  static constexpr int PER = 128 / G;                                    // groups of a row per step
  static constexpr int SROW = FMT == kInt ? 4 * PER : FULL ? PER : PER + 4 + (FMT == kNv ? 4 : 0);   // bytes of scales per row
  static constexpr int STAGE = MT * 16 * (64 + SROW);
  static constexpr int BYTES = kStages * STAGE;                          // per warp
  static_assert(STAGE % 16 == 0, "16-byte copies");

  static __device__ __forceinline__ void issue(uint32_t st, const Tile& tile, int K, int step, int lane) {
    const int g = lane >> 2, t = lane & 3;
    const int k0 = step * 128;
    const uint32_t dst = st + g * 64 + 16 * (t ^ (g >> 1));
    const int pitch = K / 2;
#pragma unroll
    for (int it = 0; it < 2 * MT; ++it) {
      const int b = it / MT, r = min(8 * (it % MT) + g, tile.span[b]);
      const uint8_t* src = tile.c[b] + static_cast<long long>(r) * pitch + step * 64 + 16 * t;
      if constexpr (FULL) {
        copy16(dst + 512 * it, src, 16);
      } else {
        const int left = K - (k0 + 32 * t);   // channels from this unit's first
        if (K % 32 == 0) {
          copy16(dst + 512 * it, left > 0 ? src : tile.c[b], left > 0 ? 16 : 0);
        } else {
          copy8(dst + 512 * it, left > 0 ? src : tile.c[b], left > 0 ? 8 : 0);
          copy8(dst + 512 * it + 8, left > 16 ? src + 8 : tile.c[b], left > 16 ? 8 : 0);
        }
      }
    }
    const uint32_t sdst = st + MT * 1024;
    const long long sp = static_cast<long long>(K / G) * (FMT == kInt ? 4 : 1);
    constexpr int half = 8 * MT;
#pragma unroll
    for (int r0 = 0; r0 < 16 * MT; r0 += 32) {
      const int row = r0 + lane;
      if (row >= 16 * MT) break;
      const int b = row / half, r = min(row % half, tile.span[b]);
      const uint8_t* src = tile.s[b] + r * sp + step * (FMT == kInt ? 4 * PER : PER);
      const uint32_t d = sdst + row * SROW;
      if constexpr (FULL) {
        if constexpr (FMT == kMx) copy4(d, src, 4);
        else if constexpr (FMT == kNv) copy8(d, src, 8);
        else {
#pragma unroll
          for (int j = 0; j < PER / 4; ++j) copy16(d + 16 * j, src + 16 * j, 16);
        }
      } else if constexpr (FMT == kInt) {
#pragma unroll
        for (int j = 0; j < PER; ++j) {
          const bool in = k0 + j * G < K;
          copy4(d + 4 * j, in ? src + 4 * j : tile.s[b], in ? 4 : 0);
        }
      } else {
        // the aligned words that hold the bytes [src, src + groups)
        const int groups = min(PER, (K - k0) / G + ((K - k0) % G != 0));
        const uint8_t* a = reinterpret_cast<const uint8_t*>(reinterpret_cast<uintptr_t>(src) & ~static_cast<uintptr_t>(3));
        const int bytes = static_cast<int>(src - a) + groups;
#pragma unroll
        for (int j = 0; j < SROW / 4; ++j) copy4(d + 4 * j, 4 * j < bytes ? a + 4 * j : a, 4 * j < bytes ? 4 : 0);
      }
    }
  }

  // the step's one-byte scales of tile row `row`
  static __device__ __forceinline__ void byte_scales(uint32_t st, const Tile& tile, int K, int step, int row,
                                                     uint32_t (&w)[PER / 4]) {
    const uint32_t a = st + MT * 1024 + row * SROW;
    if constexpr (FULL) {
      if constexpr (PER == 4) {
        w[0] = lds4(a);
      } else {
        const uint2 v = lds8(a);
        w[0] = v.x, w[1] = v.y;
      }
    } else {
      constexpr int half = 8 * MT;
      const int b = row / half, r = min(row % half, tile.span[b]);
      const uint32_t low = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(tile.s[b])) +
                           static_cast<uint32_t>(r) * static_cast<uint32_t>(K / G) + static_cast<uint32_t>(step * PER);
      const uint32_t sh = 8 * (low & 3u);
      uint32_t v[PER / 4 + 1];
#pragma unroll
      for (int j = 0; j <= PER / 4; ++j) v[j] = lds4(a + 4 * j);
#pragma unroll
      for (int j = 0; j < PER / 4; ++j) {
        // bytes past the row belong to others; as NaNs they would outlive a product with zero
        const int left = (K - step * 128 + G - 1) / G - 4 * j;
        const uint32_t keep = left >= 4 ? 0xFFFFFFFFu : left <= 0 ? 0u : (1u << (8 * left)) - 1u;
        w[j] = __funnelshift_r(v[j], v[j + 1], sh) & keep;
      }
    }
  }
};

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

// Sums of one warp: acc[i][c][0..1] are row g, columns 8 c + 2 t and 8 c + 2 t + 1 of the
// instruction (tokens by NG as above); [2..3] row g + 8.
template <int FMT, int G, int NG, int MT, int NC, bool FULL>
struct Core {
  static_assert(NG == 1 || NC == 1, "one column tile where groups share an instruction");
  using R = Ring<FMT, G, MT, FULL>;
  static constexpr int UNITS = NG == 4 ? 1 : NG == 2 ? 2 : 4;   // instruction groups per step
  static constexpr int WORDS = 4 / UNITS;                       // words of 8 codes per lane and unit
  static constexpr int SETS = FMT == kInt && G == 16 ? 2 : 1;   // separate sums per unit
  float acc[MT][NC][4];

  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int c = 0; c < NC; ++c)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][c][j] = 0.0f;
  }

  // Adds one step that has arrived at st.  col: this lane's columns in memory (by its g), or
  // null; sc: the scale rows of the two columns whose sums it holds, or null, and mul: factors on them.
  __device__ __forceinline__ void add(uint32_t st, const Tile& tile, int K, int step, const __half* const (&col)[NC],
                                      const float* const (&sc)[NC][2], const float (&mul)[NC][2], float ts, int lane) {
    const int g = lane >> 2, t = lane & 3;
    float sy[NC][2][UNITS];
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const float f = FMT == kNv ? ts * mul[c][j] : mul[c][j];
        if constexpr (NG == 1) {
          const float4 v = sc[c][j] ? *reinterpret_cast<const float4*>(sc[c][j] + step * 4) : make_float4(0.f, 0.f, 0.f, 0.f);
          sy[c][j][0] = v.x * f, sy[c][j][1] = v.y * f, sy[c][j][2] = v.z * f, sy[c][j][3] = v.w * f;
        } else {
#pragma unroll
          for (int u = 0; u < UNITS; ++u)
            sy[c][j][u] = sc[c][j] ? sc[c][j][step * 4 + (NG == 4 ? t : 2 * u + t / 2)] * f : 0.0f;
        }
      }
    // scales of the weights, by unit (and set): MXFP4 and INT4 fp32, NVFP4 an fp16 pair per word
    float sw[MT][2][UNITS * SETS];
    uint32_t sn[MT][2][FMT == kNv ? (NG == 4 ? 2 : UNITS) : 1];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int row = 16 * i + 8 * h + g;
        if constexpr (FMT == kMx) {
          uint32_t w[1];
          R::byte_scales(st, tile, K, step, row, w);
          float s0, s1, s2, s3;
          e8m0_pair(w[0], s0, s1);
          e8m0_pair(w[0] >> 16, s2, s3);
          if constexpr (NG == 1) {
            sw[i][h][0] = s0, sw[i][h][1] = s1, sw[i][h][2] = s2, sw[i][h][3] = s3;
          } else if constexpr (NG == 2) {
            sw[i][h][0] = t & 2 ? s1 : s0, sw[i][h][1] = t & 2 ? s3 : s2;
          } else {
            sw[i][h][0] = t & 2 ? (t & 1 ? s3 : s2) : (t & 1 ? s1 : s0);
          }
        } else if constexpr (FMT == kNv) {
          uint32_t w[2];
          R::byte_scales(st, tile, K, step, row, w);
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
          const uint32_t a = st + MT * 1024 + row * R::SROW;
          // groups: NG = 4: of this lane's 32 channels; NG = 2: of its half of each unit; NG = 1: all
#pragma unroll
          for (int u = 0; u < UNITS; ++u)
#pragma unroll
            for (int x = 0; x < SETS; ++x) {
              const int gi = SETS * (NG == 4 ? t : NG == 2 ? 2 * u + t / 2 : u) + x;
              sw[i][h][SETS * u + x] = __uint_as_float(lds4(a + 4 * gi));
            }
        }
      }
#pragma unroll
    for (int u = 0; u < UNITS; ++u) {
      uint4 b[NC][WORDS];
#pragma unroll
      for (int c = 0; c < NC; ++c)
#pragma unroll
        for (int w = 0; w < WORDS; ++w) {
          // channels of word w: NG = 4: 32 t + 8 w; NG = 2: 64 u + 16 t + 8 w; NG = 1: 32 u + 8 t
          const int k = step * 128 + (128 / UNITS) * u + 8 * WORDS * t + 8 * w;
          b[c][w] = col[c] ? *reinterpret_cast<const uint4*>(col[c] + k) : make_uint4(0u, 0u, 0u, 0u);
        }
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        uint32_t q[2][WORDS];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint32_t a = st + 1024 * i + 512 * h + 64 * g;
          if constexpr (NG == 4) {
            const uint4 v = lds16(a + 16 * (t ^ (g >> 1)));
            q[h][0] = v.x, q[h][1] = v.y, q[h][2] = v.z, q[h][3] = v.w;
          } else if constexpr (NG == 2) {
            const uint2 v = lds8(a + 16 * ((2 * u + (t >> 1)) ^ (g >> 1)) + 8 * (t & 1));
            q[h][0] = v.x, q[h][1] = v.y;
          } else {
            q[h][0] = lds4(a + 16 * (u ^ (g >> 1)) + 4 * t);
          }
        }
        uint32_t p[WORDS][4], r[WORDS][4];
#pragma unroll
        for (int w = 0; w < WORDS; ++w) {
          unpack8<FMT>(q[0][w], p[w]);
          unpack8<FMT>(q[1][w], r[w]);
          if constexpr (FMT == kNv) {
            const int x = NG == 4 ? w / 2 : u;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              p[w][j] = h2u(__hmul2(u2h(p[w][j]), u2h(sn[i][0][x])));
              r[w][j] = h2u(__hmul2(u2h(r[w][j]), u2h(sn[i][1][x])));
            }
          }
        }
#pragma unroll
        for (int x = 0; x < SETS; ++x) {
          // INT4 with two groups per 32 channels: NG = 4: words 0-1 and 2-3 of a lane; NG = 2: even
          // and odd lanes; NG = 1: lanes 0-1 and 2-3.  The other group's activations are zeroed.
          const bool mine = SETS == 1 || NG == 4 || (NG == 2 ? (t & 1) == x : (t >> 1) == x);
          float c4[NC][4];
#pragma unroll
          for (int c = 0; c < NC; ++c)
#pragma unroll
            for (int j = 0; j < 4; ++j) c4[c][j] = 0.0f;
#pragma unroll
          for (int w = 0; w < WORDS; ++w) {
            if (SETS == 2 && NG == 4 && w / 2 != x) continue;
#pragma unroll
            for (int c = 0; c < NC; ++c) {
              mma16816(c4[c], p[w][0], r[w][0], p[w][1], r[w][1], mine ? b[c][w].x : 0u, mine ? b[c][w].y : 0u);
              mma16816(c4[c], p[w][2], r[w][2], p[w][3], r[w][3], mine ? b[c][w].z : 0u, mine ? b[c][w].w : 0u);
            }
          }
          // the weights' and the activations' scales are multiplied first: a sum under one of them
          // alone can overflow where the result does not
#pragma unroll
          for (int c = 0; c < NC; ++c)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const float f = FMT == kNv ? sy[c][j & 1][u] : sw[i][j >> 1][SETS * u + x] * sy[c][j & 1][u];
              acc[i][c][j] = fmaf(c4[c][j], f, acc[i][c][j]);
            }
        }
      }
    }
  }

  // sums over the lanes of a row that hold different groups of the same column
  __device__ __forceinline__ void join() {
    if constexpr (NG > 1) {
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          float v = acc[i][0][j];
          if constexpr (NG == 4) v += __shfl_xor_sync(0xffffffffu, v, 1);
          v += __shfl_xor_sync(0xffffffffu, v, 2);
          acc[i][0][j] = v;
        }
    }
  }

  // to red[column][row]
  template <int PITCH>
  __device__ __forceinline__ void put(float (*red)[PITCH], int lane) const {
    const int g = lane >> 2, t = lane & 3;
    if (NG > 1 && t >= 4 / NG) return;   // NG = 4: lane 0 has both columns; NG = 2: lanes 0 and 1
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int c = 0; c < NC; ++c)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int v = 8 * c + (NG == 4 ? j : NG == 2 ? 2 * (t & 1) + j : 2 * t + j);
          red[v][16 * i + g] = acc[i][c][j];
          red[v][16 * i + g + 8] = acc[i][c][2 + j];
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

}  // namespace decode
}  // namespace wush
