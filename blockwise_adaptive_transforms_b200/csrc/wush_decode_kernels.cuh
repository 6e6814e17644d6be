// Kernels of the few-token operators on the product core: the activations' transform, the
// matrix-vector product, and the two halves of a mixture-of-experts layer.
#pragma once
#include "wush_decode_mma.cuh"

namespace wush {
namespace decode {

// ------------------------------------------------------------------ activations
// One warp writes 32 channels of one vector: lane r holds channel r, Trow its row of the block's
// transform (T null: none).  G = 16: lanes 0-15 and 16-31 are two blocks.
//
// The values leave as fp16 under one power-of-two scale per 32 channels that puts their largest
// magnitude into [2^14, 2^15): 11 significant bits, which for bf16 results is an error 10 times
// below the result's own rounding.  SPLIT (fp32 results) writes the remainder to a second column, 11
// more bits.  The scale is clamped at 2^-114, so values under 2^-139 vanish.
template <int FMT, int G, bool SPLIT>
__device__ __forceinline__ void emit_chunk(float v, bool transform, const float (&Trow)[G], int lane, __half* y,
                                           float* s, __half* y2, float* s2, int chunk) {
  if (transform) {
    float a = 0.0f;
#pragma unroll
    for (int c = 0; c < G; ++c) a = fmaf(Trow[c], __shfl_sync(0xffffffffu, v, G == 16 ? (lane & 16) + c : c), a);
    v = a;
  }
  float m = fabsf(v);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  // exponent field of the maximum, from 27 (an infinity gives 255 and stays one)
  const int e = max(static_cast<int>(__float_as_uint(m) >> 23), 27);
  const float up = __uint_as_float(static_cast<uint32_t>(254 + 14 - e) << 23);   // 2^(14 - (e - 127))
  const float z = v * up;
  const __half hi = __float2half_rn(z);
  const int at = 32 * chunk + (lane & ~7) + pair_place<FMT>(lane & 7);
  y[at] = hi;
  if (lane == 0) s[chunk] = __uint_as_float(static_cast<uint32_t>(e - 14) << 23);
  if constexpr (SPLIT) {
    // a value that is not finite is whole in the first column
    const float rest = fabsf(z) < 65536.0f ? (z - __half2float(hi)) * 2048.0f : 0.0f;
    y2[at] = __float2half_rn(rest);
    if (lane == 0) s2[chunk] = __uint_as_float(static_cast<uint32_t>(e - 14 - 11) << 23);
  }
}

// this lane's row of the transform of the block(s) of a chunk
template <int G>
__device__ __forceinline__ void load_transform_row(float (&Trow)[G], const float* T, int T_stride, int chunk, int lane,
                                                   int K) {
  const int k = 32 * chunk + lane;
  if (T && k < K) {
    const float4* src = reinterpret_cast<const float4*>(T + static_cast<long long>(k / G) * T_stride + (k % G) * G);
#pragma unroll
    for (int c = 0; c < G / 4; ++c) {
      const float4 q = src[c];
      Trow[4 * c] = q.x, Trow[4 * c + 1] = q.y, Trow[4 * c + 2] = q.z, Trow[4 * c + 3] = q.w;
    }
  } else {
#pragma unroll
    for (int c = 0; c < G; ++c) Trow[c] = 0.0f;
  }
}

constexpr int kPrepTokens = 4;   // vectors that one warp takes under one load of its transform rows

// Activations [n][K] -> columns.  One warp per 32 channels (channels past K, up to the padded
// length, are written as zeros) and kPrepTokens vectors.
template <int FMT, int G, bool SPLIT>
__global__ void __launch_bounds__(128) prep_kernel(const __nv_bfloat16* __restrict__ x, const float* __restrict__ T,
                                                   int T_stride, int n, int K, int ld, __half* __restrict__ y,
                                                   float* __restrict__ s) {
  pdl_wait();
  pdl_launch();
  const int lane = threadIdx.x & 31, chunk = blockIdx.x * 4 + (threadIdx.x >> 5);
  if (chunk >= ld / 32) return;
  const int k = 32 * chunk + lane;
  const int t0 = blockIdx.y * kPrepTokens, t1 = min(n, t0 + kPrepTokens);
  float v[kPrepTokens];
#pragma unroll
  for (int j = 0; j < kPrepTokens; ++j)
    v[j] = t0 + j < t1 && k < K ? __bfloat162float(x[static_cast<long long>(t0 + j) * K + k]) : 0.0f;
  float Trow[G];
  load_transform_row<G>(Trow, T, T_stride, chunk, lane, K);
#pragma unroll
  for (int j = 0; j < kPrepTokens; ++j) {
    if (t0 + j >= t1) break;
    const int c0 = SPLIT ? 2 * (t0 + j) : t0 + j;
    emit_chunk<FMT, G, SPLIT>(v[j], T != nullptr, Trow, lane, y + static_cast<long long>(c0) * ld, s + c0 * (ld / 32),
                              y + static_cast<long long>(c0 + 1) * ld, s + (c0 + 1) * (ld / 32), chunk);
  }
}

// ------------------------------------------------------------------ matrix-vector products
constexpr int kGemvWarps = 8;

__device__ __forceinline__ void store(float* p, float v) { *p = v; }
__device__ __forceinline__ void store(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

struct GemvParams {
  Matrix4 w;
  Columns y;
  int columns;   // in memory: tokens, or two per token (split)
  int n;
  int col_groups;   // CTAs per row tile, each with its own columns
  int wk;           // warps along K (a power of two); the others of the CTA take more rows
  bool f32;         // fp32 results, and two columns per token
  void* out;
};

// Steps [first, last) of a tile through the ring, added to core.  The first kStages - 1 steps have
// been issued already (prefetch_tile).
template <class Core, class Ring>
__device__ __forceinline__ void prefetch_tile(uint32_t ring, const Tile& tile, int K, int first, int last, int lane) {
#pragma unroll
  for (int j = 0; j < kStages - 1; ++j) {
    if (first + j < last) Ring::issue(ring + j * Ring::STAGE, tile, K, first + j, lane);
    copies_commit();
  }
}

template <class Core, class Ring, int NC>
__device__ __forceinline__ void run_tile(Core& core, uint32_t ring, const Tile& tile, int K, int first, int last,
                                         const __half* const (&col)[NC], const float* const (&sc)[NC][2],
                                         const float (&mul)[NC][2], float ts, int lane) {
  int stage = 0;
  for (int step = first; step < last; ++step) {
    copies_wait<kStages - 2>();
    __syncwarp();   // the step has arrived for all lanes, and all are done with the one before
    const int ahead = step + kStages - 1, to = stage == 0 ? kStages - 1 : stage - 1;
    if (ahead < last) Ring::issue(ring + to * Ring::STAGE, tile, K, ahead, lane);
    copies_commit();
    core.add(ring + stage * Ring::STAGE, tile, K, step, col, sc, mul, ts, lane);
    stage = stage == kStages - 1 ? 0 : stage + 1;
  }
  __syncwarp();
}

// CTA: (kGemvWarps / wk) row tiles of 16 MT rows, wk warps along K for each.
template <int FMT, int G, int NG, int MT, int NC, bool FULL>
__global__ void __launch_bounds__(32 * kGemvWarps, 2) gemv_kernel(const GemvParams p) {
  constexpr int COLS = columns_of(NG, NC), R = 16 * MT;
  using Ring_ = Ring<FMT, G, MT, FULL>;
  using Core_ = Core<FMT, G, NG, MT, NC, FULL>;
  extern __shared__ __align__(16) uint8_t dyn[];
  __shared__ float red[kGemvWarps][COLS][R + 1];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
  const int wk = warp & (p.wk - 1), wr = warp / p.wk, wrs = kGemvWarps / p.wk;
  const int group = blockIdx.x % p.col_groups;
  const long long row0 = (static_cast<long long>(blockIdx.x / p.col_groups) * wrs + wr) * R;
  const int K = p.w.K, steps = (K + 127) / 128;
  const bool any = row0 < p.w.rows;
  const int first = any ? steps * wk / p.wk : 0, last = any ? steps * (wk + 1) / p.wk : 0;
  const Tile tile = plain_tile<FMT, G, MT>(p.w, any ? row0 : 0, any ? p.w.rows - row0 : 1);
  const uint32_t ring = shared_address(dyn) + warp * Ring_::BYTES;
  // the first weights are asked for while the activations are still being transformed: they
  // were written before the kernel that this one overlaps with began
  prefetch_tile<Core_, Ring_>(ring, tile, K, first, last, lane);
  pdl_wait();
  pdl_launch();

  const __half* col[NC];
  const float* sc[NC][2];
  float mul[NC][2];
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    const int v = lane_column<NG>(g, t), at = group * COLS + 8 * c + v;
    col[c] = v >= 0 && at < p.columns ? p.y.y + static_cast<long long>(at) * p.y.ld : nullptr;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int sv = group * COLS + 8 * c + sum_column<NG>(t, j);
      sc[c][j] = sv < p.columns ? p.y.s + static_cast<long long>(sv) * (p.y.ld / 32) : nullptr;
      mul[c][j] = 1.0f;
    }
  }
  Core_ core;
  core.clear();
  run_tile<Core_, Ring_, NC>(core, ring, tile, K, first, last, col, sc, mul, tensor_scale<FMT>(p.w, 0), lane);
  core.join();
  core.put(red[warp], lane);
  __syncthreads();
  const int per = p.f32 ? 2 : 1, tokens = COLS / per;
  for (int i = threadIdx.x; i < wrs * tokens * R; i += 32 * kGemvWarps) {
    const int r = i % R, tok = i / R % tokens, sub = i / (R * tokens);
    const long long row = (static_cast<long long>(blockIdx.x / p.col_groups) * wrs + sub) * R + r;
    const int token = group * tokens + tok;
    if (row >= p.w.rows || token >= p.n) continue;
    float a = 0.0f;
    for (int w = 0; w < p.wk; ++w) {
      const float(&src)[COLS][R + 1] = red[sub * p.wk + w];
      a += p.f32 ? src[2 * tok][r] + src[2 * tok + 1][r] : src[tok][r];
    }
    const long long at = static_cast<long long>(token) * p.w.rows + row;
    if (p.f32) store(static_cast<float*>(p.out) + at, a);
    else store(static_cast<__nv_bfloat16*>(p.out) + at, a);
  }
}

// ------------------------------------------------------------------ experts
// A call's routing: ids [n][k]; an id outside [0, E) is a dropped slot, and a later slot of the
// same token with the same expert is folded into the first.
struct Routing {
  const int* ids;
  const float* weights;
  int n, k, E;
};

__device__ __forceinline__ bool routed(int e, int E) { return e >= 0 && e < E; }

// bit e % 32 of word e / 32: some slot in [first, first + count) has expert e.  All threads.
__device__ __forceinline__ void active_experts(const Routing& r, int first, int count, uint32_t (&words)[kMaxExperts / 32]) {
  for (int i = threadIdx.x; i < kMaxExperts / 32; i += blockDim.x) words[i] = 0u;
  __syncthreads();
  for (int i = threadIdx.x; i < count; i += blockDim.x) {
    const int e = r.ids[first + i];
    if (routed(e, r.E)) atomicOr(&words[e >> 5], 1u << (e & 31));
  }
  __syncthreads();
}

// the experts of the words in ascending order into list (one warp); returns how many
__device__ __forceinline__ int list_experts(const uint32_t (&words)[kMaxExperts / 32], short* list) {
  const int lane = threadIdx.x & 31;
  uint32_t w = words[lane];
  int at = __popc(w);
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, at, o);
    if (lane >= o) at += v;
  }
  const int total = __shfl_sync(0xffffffffu, at, 31);
  at -= __popc(w);
  while (w) {
    list[at++] = static_cast<short>(32 * lane + __ffs(w) - 1);
    w &= w - 1;
  }
  return total;
}
static_assert(kMaxExperts == 1024, "one word of experts per lane");

constexpr int kMoeWarps = 8;
constexpr int kHidden = 32;   // hidden values of one gate-and-up tile: whole transform blocks

struct GateUpParams {
  Matrix4 w;
  Columns y;
  Routing route;
  int f;
  const float* T;
  int T_stride;
  __half* h;    // columns [n * k][ld], one per slot
  float* hs;
  int ld;
};

// Persistent over (active expert, 32 hidden values): the gate and up rows against the tokens of
// the expert, silu(gate) * up, the down projection's transform of these 32 values, and their
// store as a column per slot.  The warps of a CTA split K.
template <int FMT, int G, int NG, int NC, bool FULL>
__global__ void __launch_bounds__(32 * kMoeWarps, 1) gate_up_kernel(const GateUpParams p) {
  constexpr int MT = 4, COLS = columns_of(NG, NC);
  using Ring_ = Ring<FMT, G, MT, FULL>;
  using Core_ = Core<FMT, G, NG, MT, NC, FULL>;
  extern __shared__ __align__(16) uint8_t dyn[];
  __shared__ float red[kMoeWarps][COLS][2 * kHidden + 1];
  __shared__ uint32_t words[kMaxExperts / 32];
  __shared__ short experts[kMaxExperts];
  __shared__ int s_count, s_slots;
  __shared__ short slots[64 * kMaxTopK];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
  pdl_wait();
  pdl_launch();
  active_experts(p.route, 0, p.route.n * p.route.k, words);
  if (warp == 0) {
    const int c = list_experts(words, experts);
    if (lane == 0) s_count = c;
  }
  __syncthreads();
  const int K = p.w.K, steps = (K + 127) / 128;
  const int first = steps * warp / kMoeWarps, last = steps * (warp + 1) / kMoeWarps;
  const int tiles = (p.f + kHidden - 1) / kHidden;
  const uint32_t ring = shared_address(dyn) + warp * Ring_::BYTES;
  const long long items = static_cast<long long>(s_count) * tiles;
  int had = -1;
  for (long long item = blockIdx.x; item < items; item += gridDim.x) {
    const int rank = static_cast<int>(item / tiles), h0 = static_cast<int>(item % tiles) * kHidden, e = experts[rank];
    Tile tile;
    const long long row = static_cast<long long>(e) * p.w.rows + h0;
    const long long cp = K / 2, sp = static_cast<long long>(K / G) * (FMT == kInt ? 4 : 1);
    tile.c[0] = p.w.codes + row * cp;
    tile.c[1] = tile.c[0] + p.f * cp;
    tile.s[0] = static_cast<const uint8_t*>(p.w.scales) + row * sp;
    tile.s[1] = tile.s[0] + p.f * sp;
    tile.span[0] = tile.span[1] = min(kHidden, p.f - h0) - 1;
    prefetch_tile<Core_, Ring_>(ring, tile, K, first, last, lane);
    if (rank != had) {   // this expert's slots, in order, one per token
      had = rank;
      if (warp == 0) {
        int count = 0;
        const int total = p.route.n * p.route.k;
        for (int i0 = 0; i0 < total; i0 += 32) {
          const int i = i0 + lane;
          bool mine = i < total && p.route.ids[i] == e;
          for (int j = i - 1; mine && j >= i / p.route.k * p.route.k; --j) mine = p.route.ids[j] != e;
          const uint32_t m = __ballot_sync(0xffffffffu, mine);
          if (mine) slots[count + __popc(m & ((1u << lane) - 1u))] = static_cast<short>(i);
          count += __popc(m);
        }
        if (lane == 0) s_slots = count;
      }
    }
    __syncthreads();
    const int count = s_slots;
    const float ts = tensor_scale<FMT>(p.w, e);
    for (int c0 = 0; c0 < count; c0 += COLS) {
      if (c0) prefetch_tile<Core_, Ring_>(ring, tile, K, first, last, lane);
      const __half* col[NC];
      const float* sc[NC][2];
      float mul[NC][2];
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        const int v = lane_column<NG>(g, t), at = c0 + 8 * c + v;
        col[c] = v >= 0 && at < count ? p.y.y + static_cast<long long>(slots[at] / p.route.k) * p.y.ld : nullptr;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int sv = c0 + 8 * c + sum_column<NG>(t, j);
          sc[c][j] = sv < count ? p.y.s + static_cast<long long>(slots[sv] / p.route.k) * (p.y.ld / 32) : nullptr;
          mul[c][j] = 1.0f;
        }
      }
      Core_ core;
      core.clear();
      run_tile<Core_, Ring_, NC>(core, ring, tile, K, first, last, col, sc, mul, ts, lane);
      core.join();
      core.put(red[warp], lane);
      __syncthreads();
      for (int v = warp; v < COLS && c0 + v < count; v += kMoeWarps) {   // one warp per column
        float gate = 0.0f, up = 0.0f;
#pragma unroll
        for (int w = 0; w < kMoeWarps; ++w) gate += red[w][v][lane], up += red[w][v][kHidden + lane];
        const float h = h0 + lane < p.f ? gate / (1.0f + expf(-gate)) * up : 0.0f;
        float Trow[G];
        load_transform_row<G>(Trow, p.T, p.T_stride, h0 / 32, lane, p.f);
        const int slot = slots[c0 + v];
        __half* y = p.h + static_cast<long long>(slot) * p.ld;
        float* s = p.hs + static_cast<long long>(slot) * (p.ld / 32);
        emit_chunk<FMT, G, false>(h, p.T != nullptr, Trow, lane, y, s, nullptr, nullptr, h0 / 32);
        if (h0 + kHidden >= p.f) {   // zeros up to the padded length
          for (int c = h0 / 32 + 1; c < p.ld / 32; ++c) {
            y[32 * c + lane] = __float2half_rn(0.0f);
            if (lane == 0) s[c] = 1.0f;
          }
        }
      }
      __syncthreads();
    }
  }
}

struct DownParams {
  Matrix4 w;
  Columns h;   // one column per slot
  Routing route;
  int rows;    // of the output
  __nv_bfloat16* out;
};

// Row tiles of the output, one CTA each, for up to COLS tokens (blockIdx.y): the sum over the
// experts is taken in the accumulators.  Column v is token v for every expert, with the slot's
// weight in the activations' scale, so one pass runs over (expert, K) of all active experts, split
// evenly over the CTA's warps, and joins once at its end.
template <int FMT, int G, int NG, int MT, int NC, bool FULL>
__global__ void __launch_bounds__(32 * kMoeWarps, 2) down_kernel(const DownParams p) {
  constexpr int COLS = columns_of(NG, NC), R = 16 * MT;
  using Ring_ = Ring<FMT, G, MT, FULL>;
  using Core_ = Core<FMT, G, NG, MT, NC, FULL>;
  extern __shared__ __align__(16) uint8_t dyn[];
  __shared__ float red[kMoeWarps][COLS][R + 1];
  __shared__ uint32_t words[kMaxExperts / 32];
  __shared__ short experts[kMaxExperts];
  __shared__ int s_count;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
  const int token0 = blockIdx.y * COLS, tokens = min(COLS, p.route.n - token0), k = p.route.k;
  pdl_wait();
  pdl_launch();
  active_experts(p.route, token0 * k, tokens * k, words);
  if (warp == 0) {
    const int c = list_experts(words, experts);
    if (lane == 0) s_count = c;
  }
  __syncthreads();
  const int K = p.w.K, steps = (K + 127) / 128;
  const long long total = static_cast<long long>(s_count) * steps;
  long long at = total * warp / kMoeWarps;
  const long long end = total * (warp + 1) / kMoeWarps;
  const int row0 = blockIdx.x * R;
  const uint32_t ring = shared_address(dyn) + warp * Ring_::BYTES;
  Core_ core;
  core.clear();
  while (at < end) {
    const int rank = static_cast<int>(at / steps), e = experts[rank];
    const int first = static_cast<int>(at - static_cast<long long>(rank) * steps);
    const int last = static_cast<int>(min(static_cast<long long>(steps), end - static_cast<long long>(rank) * steps));
    const Tile tile = plain_tile<FMT, G, MT>(p.w, static_cast<long long>(e) * p.w.rows + row0, p.rows - row0);
    prefetch_tile<Core_, Ring_>(ring, tile, K, first, last, lane);
    const float ts = tensor_scale<FMT>(p.w, e);
    const __half* col[NC];
    const float* sc[NC][2];
    float mul[NC][2];
    // the slot of a token with this expert, and the sum of its slots' weights
    auto find = [&](int token, float& weight) {
      int slot = -1;
      weight = 0.0f;
      for (int j = 0; j < k; ++j) {
        const int i = (token0 + token) * k + j;
        if (p.route.ids[i] != e) continue;
        if (slot < 0) slot = i;
        weight += p.route.weights[i];
      }
      return slot;
    };
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      float unused;
      const int v = lane_column<NG>(g, t);
      const int slot = v >= 0 && 8 * c + v < tokens ? find(8 * c + v, unused) : -1;
      col[c] = slot >= 0 ? p.h.y + static_cast<long long>(slot) * p.h.ld : nullptr;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int sv = 8 * c + sum_column<NG>(t, j);
        const int ss = sv < tokens ? find(sv, mul[c][j]) : -1;
        if (ss < 0) mul[c][j] = 0.0f;
        sc[c][j] = ss >= 0 ? p.h.s + static_cast<long long>(ss) * (p.h.ld / 32) : nullptr;
      }
    }
    run_tile<Core_, Ring_, NC>(core, ring, tile, K, first, last, col, sc, mul, ts, lane);
    at += last - first;
  }
  core.join();
  core.put(red[warp], lane);
  __syncthreads();
  for (int i = threadIdx.x; i < tokens * R; i += 32 * kMoeWarps) {
    const int r = i % R, v = i / R;
    if (row0 + r >= p.rows) continue;
    float a = 0.0f;
#pragma unroll
    for (int w = 0; w < kMoeWarps; ++w) a += red[w][v][r];
    store(p.out + static_cast<long long>(token0 + v) * p.rows + row0 + r, a);
  }
}

}  // namespace decode
}  // namespace wush
