// Kernels of the few-token operators on the product core: the activations' transform, the
// matrix-vector product, and the two halves of a mixture-of-experts layer.
#pragma once
#include <cuda.h>

#include <type_traits>

#include "wush_decode_mma.cuh"

namespace wush {
namespace decode {

// ------------------------------------------------------------------ activations
// The values leave as fp16 under one power-of-two scale for some channels that puts their largest
// magnitude into [2^14, 2^15): 11 significant bits, for values down to 2^-28 of the largest, which
// for bf16 results is an error 8 times below the result's own rounding; below that a step of 2^-24,
// half of which is 2^-39 of the largest at most.  fp32 results take the remainder in a second column,
// 11 more bits.  The scale is clamped at 2^-114, so values under 2^-139 vanish.

// T_i of the block(s) of this warp's 32 channels: lane r holds channel r and row r of its block
// (G = 16: lanes 0-15 and 16-31 are two blocks)
template <int G>
__device__ __forceinline__ float transformed(float v, const float (&Trow)[G], int lane) {
  float a = 0.0f;
#pragma unroll
  for (int c = 0; c < G; ++c) a = fmaf(Trow[c], __shfl_sync(0xffffffffu, v, G == 16 ? (lane & 16) + c : c), a);
  return a;
}

__device__ __forceinline__ float warp_max(float m) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  return m;
}

// exponent field of the largest magnitude, from 27 (an infinity gives 255 and stays one)
__device__ __forceinline__ int scale_field(float largest) { return max(static_cast<int>(__float_as_uint(largest) >> 23), 27); }
__device__ __forceinline__ float column_scale(int field) { return __uint_as_float(static_cast<uint32_t>(field - 14) << 23); }
__device__ __forceinline__ float scaled_up(float v, int field) {
  return v * __uint_as_float(static_cast<uint32_t>(254 + 14 - field) << 23);   // 2^(14 - (field - 127))
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

// Activations [n][K] -> columns with one scale per 128 channels.  One CTA of 4 warps per 128
// channels (those past K, up to the padded length, are written as zeros) and kPrepTokens vectors.
// SPLIT: two columns per vector.
//
// Before the wait the CTA asks for its transforms and activations in L2 (no data is delivered, and L2
// is where writes meet): after a product has streamed hundreds of megabytes they are out of every
// cache, and fetching them took 7.7 us of a call with 8192 channels and 16 tokens.
// beside: the kernel before this one is the router, which writes nothing that is read or written here
// and has itself waited for everything earlier before it let this one begin.  So the work needs no
// wait; it comes at the end, and lets the next kernel begin when both are done.
template <int FMT, int G, bool SPLIT>
__global__ void __launch_bounds__(128) prep_kernel(const __nv_bfloat16* x, const float* T,
                                                   int T_stride, int n, int K, int ld, __half* y,
                                                   float* s, unsigned int* arrived,
                                                   int arrivals, int beside) {
  __shared__ float largest[kPrepTokens][4];
  __shared__ __align__(16) float Ts[4][32 * (G + 4)];   // a warp's transform rows, 16 bytes apart in the banks
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, chunk = blockIdx.x * 4 + warp;
  const int k = 32 * chunk + lane;
  if (!beside) {
    if (T && T_stride && k < K) {   // this lane's row of its block: G * 4 bytes
      const float* row = T + static_cast<long long>(k / G) * T_stride + k % G * G;
      asm volatile("prefetch.global.L2 [%0];" ::"l"(row));
    }
    if (threadIdx.x < 2 * kPrepTokens) {   // 256 bytes of each vector
      const int t = blockIdx.y * kPrepTokens + threadIdx.x / 2, c = 128 * blockIdx.x + 64 * (threadIdx.x & 1);
      if (t < n && c < K) asm volatile("prefetch.global.L2 [%0];" ::"l"(x + static_cast<long long>(t) * K + c));
    }
    pdl_wait();
    pdl_launch();
  }
  if (blockIdx.x == 0 && blockIdx.y == 0)
    for (int i = threadIdx.x; i < arrivals; i += 128) arrived[i] = 0u;   // for the kernels that follow
  const int t0 = blockIdx.y * kPrepTokens, t1 = min(n, t0 + kPrepTokens);
  float v[kPrepTokens];
#pragma unroll
  for (int j = 0; j < kPrepTokens; ++j)
    v[j] = t0 + j < t1 && k < K ? __bfloat162float(x[static_cast<long long>(t0 + j) * K + k]) : 0.0f;
  if (T) {
    // 32 rows of G values: one block, or two that are neighbours unless they are the same shared one
    float4 q[G / 4];
#pragma unroll
    for (int i = 0; i < G / 4; ++i) {
      const int at = 4 * (32 * i + lane), row = at / G, kr = 32 * chunk + row;
      q[i] = kr < K ? *reinterpret_cast<const float4*>(T + static_cast<long long>(kr / G) * T_stride + kr % G * G + at % G)
                    : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    }
    float* mine = Ts[warp];
#pragma unroll
    for (int i = 0; i < G / 4; ++i) {
      const int at = 4 * (32 * i + lane);
      *reinterpret_cast<float4*>(mine + at / G * (G + 4) + at % G) = q[i];
    }
    __syncwarp();
    float Trow[G];
#pragma unroll
    for (int c = 0; c < G / 4; ++c) {
      const float4 r = *reinterpret_cast<const float4*>(mine + lane * (G + 4) + 4 * c);
      Trow[4 * c] = r.x, Trow[4 * c + 1] = r.y, Trow[4 * c + 2] = r.z, Trow[4 * c + 3] = r.w;
    }
#pragma unroll
    for (int j = 0; j < kPrepTokens; ++j)
      if (t0 + j < t1) v[j] = transformed<G>(v[j], Trow, lane);
  }
#pragma unroll
  for (int j = 0; j < kPrepTokens; ++j) {
    const float m = warp_max(fabsf(v[j]));
    if (lane == 0) largest[j][warp] = m;
  }
  __syncthreads();
  const int at = 32 * chunk + (lane & ~7) + pair_place<FMT>(lane & 7);
#pragma unroll
  for (int j = 0; j < kPrepTokens; ++j) {
    if (t0 + j >= t1) break;
    const int e = scale_field(fmaxf(fmaxf(largest[j][0], largest[j][1]), fmaxf(largest[j][2], largest[j][3])));
    const float z = scaled_up(v[j], e);
    const __half hi = __float2half_rn(z);
    const int c = SPLIT ? 2 * (t0 + j) : t0 + j;
    y[static_cast<long long>(c) * ld + at] = hi;
    if (threadIdx.x == 0) s[c * (ld / 32) + blockIdx.x] = column_scale(e);
    if constexpr (SPLIT) {
      // a value that is not finite is whole in the first column
      const float rest = fabsf(z) < 65536.0f ? (z - __half2float(hi)) * 2048.0f : 0.0f;
      y[static_cast<long long>(c + 1) * ld + at] = __float2half_rn(rest);
      if (threadIdx.x == 0) s[(c + 1) * (ld / 32) + blockIdx.x] = column_scale(e - 11);
    }
  }
  if (beside) {
    pdl_wait();
    pdl_launch();
  }
}

__device__ __forceinline__ void store(float* p, float v) { *p = v; }
__device__ __forceinline__ void store(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

// ------------------------------------------------------------------ copies and barriers
__device__ __forceinline__ uint32_t shared_address(const void* p) {
  return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}
__device__ __forceinline__ void bar_init(uint32_t bar, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}
__device__ __forceinline__ void bar_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void bar_expect(uint32_t bar, uint32_t bytes) {   // without an arrival
  asm volatile("mbarrier.expect_tx.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}
__device__ __forceinline__ void bar_arrive_expect(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}
// this thread's arrival, once its asynchronous copies so far have landed
__device__ __forceinline__ void bar_arrive_copies(uint32_t bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}

// Waits are bounded in time: on expiry the word of device errors gets bit 256 and *abort rises, after
// which every wait of the CTA returns at once and the kernel runs out with unspecified results.
struct Bound {
  volatile int* abort;
  unsigned int* error;
  unsigned long long limit_ns;
};
__device__ __forceinline__ uint64_t now_ns() {
  uint64_t t;
  asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
  return t;
}
__device__ __forceinline__ bool try_wait(uint32_t bar, uint32_t parity) {
  uint32_t done;
  asm volatile(
      "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(done) : "r"(bar), "r"(parity) : "memory");
  return done != 0;
}
__device__ __noinline__ void wait_long(uint32_t bar, uint32_t parity, const Bound& b) {
  const uint64_t t0 = now_ns();
  while (!*b.abort && !try_wait(bar, parity)) {
    if (now_ns() - t0 > b.limit_ns) {
      atomicOr(b.error, 256u);
      *b.abort = 1;
    }
  }
}
__device__ __forceinline__ void wait(uint32_t bar, uint32_t parity, const Bound& b) {
  if (!try_wait(bar, parity)) wait_long(bar, parity, b);
}
// until copies in flight have landed, however short the caller's limit; two seconds are more than any takes
__device__ __noinline__ void wait_landed(uint32_t bar, uint32_t parity, unsigned int* error) {
  const uint64_t t0 = now_ns();
  while (!try_wait(bar, parity)) {
    if (now_ns() - t0 > 2000000000ull) {
      atomicOr(error, 256u);
      return;
    }
  }
}

// Waits on a barrier that no thread arrives on and no copy signals: the wait must give up, and the next
// one of the block return at once.
__global__ void __launch_bounds__(32) selftest_wait_kernel(unsigned int* error, unsigned long long limit_ns) {
  __shared__ uint64_t bar;
  __shared__ int abort;
  if (threadIdx.x == 0) {
    bar_init(shared_address(&bar), 1);
    abort = 0;
  }
  __syncthreads();
  const Bound bound{&abort, error, limit_ns};
  wait(shared_address(&bar), 0u, bound);
  wait(shared_address(&bar), 0u, bound);
}

__device__ __forceinline__ void tensor_copy(uint32_t dst, const CUtensorMap* map, uint32_t bar, int x, int y) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cta.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4}], [%2];"
      ::"r"(dst), "l"(map), "r"(bar), "r"(x), "r"(y) : "memory");
}
__device__ __forceinline__ void bulk_copy(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cta.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
               ::"r"(dst), "l"(src), "r"(bytes), "r"(bar) : "memory");
}
// asynchronous copies of one thread; `bytes` of them come from memory, the rest are zeros
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void copy8(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void copy4(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}

// ------------------------------------------------------------------ routing
// A call's routing: ids [n][k]; an id outside [0, E) is a dropped slot, and a later slot of the
// same token with the same expert is folded into the first.
struct Routing {
  const int* ids;
  const float* weights;
  int n, k, E;
};

__device__ __forceinline__ bool routed(int e, int E) { return e >= 0 && e < E; }

// The active experts in ascending order and their slots, in shared memory, in passes of at most
// `most` slots:
//   experts[r], first[r] .. first[r + 1] into slots and weights (a slot's weight with those of the
//   token's later slots of the same expert)
struct Table {
  short* experts;
  short* first;
  short* slots;
  float* weights;
  int* count;

  // at most one pass per slot
  static constexpr int bytes(int slots) { return 4 * slots + 16 + 2 * (3 * slots + 1); }
  __device__ __forceinline__ void lay(uint8_t* at, int nslots) {
    weights = reinterpret_cast<float*>(at);
    count = reinterpret_cast<int*>(at + 4 * nslots);
    slots = reinterpret_cast<short*>(at + 4 * nslots + 16);
    experts = slots + nslots;
    first = experts + nslots;
  }
  // all threads; places: E ints of scratch
  __device__ __forceinline__ void build(const Routing& r, int most, int* places) {
    const int lane = threadIdx.x & 31, total = r.n * r.k;
    for (int i = threadIdx.x; i < r.E; i += blockDim.x) places[i] = 0;
    __syncthreads();
    auto mine = [&](int i) {   // the expert of a slot that is the token's first with it, else -1
      const int e = r.ids[i];
      if (!routed(e, r.E)) return -1;
      for (int j = i / r.k * r.k; j < i; ++j)
        if (r.ids[j] == e) return -1;
      return e;
    };
    for (int i = threadIdx.x; i < total; i += blockDim.x) {
      const int e = mine(i);
      if (e >= 0) atomicAdd(&places[e], 1);
    }
    __syncthreads();
    if (threadIdx.x < 32) {
      int rank = 0, sum = 0;
      for (int e0 = 0; e0 < r.E; e0 += 32) {
        const int c = e0 + lane < r.E ? places[e0 + lane] : 0;
        const int np = most > c ? c > 0 : (c + most - 1) / most;   // passes
        int upto = c, pass = np;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int v = __shfl_up_sync(0xffffffffu, upto, o), w = __shfl_up_sync(0xffffffffu, pass, o);
          if (lane >= o) upto += v, pass += w;
        }
        for (int j = 0; j < np; ++j) {
          const int at = rank + pass - np + j;
          experts[at] = static_cast<short>(e0 + lane);
          first[at] = static_cast<short>(sum + upto - c + j * most);
        }
        if (c > 0) places[e0 + lane] = sum + upto - c;
        rank += __shfl_sync(0xffffffffu, pass, 31);
        sum += __shfl_sync(0xffffffffu, upto, 31);
      }
      if (lane == 0) first[rank] = static_cast<short>(sum), *count = rank;
    }
    __syncthreads();
    // in the order of the slots, so that every CTA has the same passes
    if (threadIdx.x < 32) {
      for (int i0 = 0; i0 < total; i0 += 32) {
        const int i = i0 + lane, e = i < total ? mine(i) : -1;
        const uint32_t same = __match_any_sync(0xffffffffu, e);
        const int at = e < 0 ? 0 : places[e] + __popc(same & ((1u << lane) - 1u));
        __syncwarp();
        if (e >= 0) {
          if ((same & ((1u << lane) - 1u)) == 0u) places[e] += __popc(same);
          float w = r.weights[i];
          for (int j = i + 1; j < (i / r.k + 1) * r.k; ++j)
            if (r.ids[j] == e) w += r.weights[j];
          slots[at] = static_cast<short>(i);
          weights[at] = w;
        }
        __syncwarp();
      }
    }
    __syncthreads();
  }
};

// out[t] = the sum of the token's slots in their order.  Bound by the reads of the slots' fp32 products,
// which the kernel before has left in L2: 32 tokens with 4 of 4096 channels, 2 MB, are a launch's latency.
__global__ void __launch_bounds__(256) combine_kernel(const float* part, const Routing r, int rows,
                                                      __nv_bfloat16* out) {
  pdl_wait();
  pdl_launch();
  const int row = blockIdx.x * 256 + threadIdx.x, t = blockIdx.y;
  if (row >= rows) return;
  float a = 0.0f;
  for (int j = 0; j < r.k; ++j) {
    const int e = r.ids[t * r.k + j];
    bool use = routed(e, r.E);
    for (int i = 0; use && i < j; ++i) use = r.ids[t * r.k + i] != e;   // folded into slot i
    if (use) a += part[static_cast<long long>(t * r.k + j) * rows + row];
  }
  store(out + static_cast<long long>(t) * rows + row, a);
}

// ------------------------------------------------------------------ the ring
// One persistent kernel for all products, one CTA per SM: 12 or 8 warps that compute, one that asks for
// codes (tensor copies) and activations (bulk copies), three that ask for scales, and a ring of stages
// between them.  The work is a sequence of units (a stage each) cut into equal shares, whatever the
// shape: a CTA's share may begin or end inside a tile, whose sums then meet through memory.
//
// Measured, streaming 57344 x 4096 bytes: tensor copies of 64 to 256 rows by 128 bytes 6.0 to 6.3 TB/s
// with nothing else in the way, where asynchronous copies issued by the computing warps, three
// steps ahead, reached 2.4 TB/s.
//
// What bounds it: memory reads what the weights hold and no more (145 MB for 65537 x 4096 MXFP4), but
// the computing warps' chains of instructions take as long or longer; no pipe is full.  MXFP4, the kernel of 65537 x 4096 with fp32
// results 29 us (15.7 of computing per warp, 4.3 of waiting for copies, 4.8 of sums and results, the
// rest start and end): 5.0 TB/s; 57344 x 8192 with 16 tokens 82 us with its transform: 3.1 TB/s, tensor
// cores 37 %, issue slots 50 %, two warps a scheduler; 64 experts of 4096 x 1536 with 32 tokens: the gate half 3.7 TB/s, the
// down half 3.3 TB/s.  A register split between the copying and the computing warps was slower.
//
//   kGemv    tiles of ROWS rows, groups of COLS columns; out[token][row]
//   kGate    (expert, COLS of its tokens) by 16 ROWS / 32 hidden values: their gate rows and their up
//            rows; silu(gate) * up, the down projection's transform (whole blocks), a column per slot
//   kSlots   (expert, COLS of its slots) by ROWS rows; the product times the slot's weight, by slot
//   kDense   tiles of ROWS rows; a tile's units run over all active experts, column v is token v for
//            every one of them, the slot's weight is in the activations' scale, and the sum over the
//            experts is taken in the accumulators
enum { kGemv = 0, kGate = 1, kSlots = 2, kDense = 3 };

// columns of a tile whose sums other CTAs need (kDense: tokens are columns, whichever the experts)
__device__ __forceinline__ int cols_used(int mode, int most, int cols) { return mode == kDense ? most : cols; }

constexpr int kMaxCtas = 256;            // of a launch: partial sums have two places for each
constexpr int kSharedBytes = 227 * 1024 - 1024;
constexpr int kTableBytes = 26 * 1024;   // room for the largest routing table
static_assert(Table::bytes(kMaxTokens * kMaxTopK) <= kTableBytes, "");

struct RingParams {
  Matrix4 w;           // rows: of one matrix
  Columns y;
  Routing route;
  int columns;         // kGemv: columns in memory
  int n;               // tokens
  int rows;            // outputs; kGate: hidden values
  const float* T;      // kGate
  int T_stride;
  __half* h;           // kGate: columns [n * k] of h_ld channels, one per slot
  float* hs;
  int h_ld;
  bool f32;            // kGemv: fp32 results, and two columns per token
  void* out;           // kSlots: fp32 [n * k][rows]
  int parts;           // kGemv, kDense: CTAs of a cluster that share a tile, or 1
  float* pieces;       // [kMaxCtas][2][COLS][ROWS], whatever those are
  unsigned int* arrived;   // [kMaxCtas], zero
  unsigned int* error;
  unsigned long long limit_ns;
};

template <int MODE, int FMT, int G, int NG, int NC, bool EXACT, bool TENSOR>
struct RingShape {
  static constexpr int PER_SCALE = MODE == kGemv || MODE == kGate ? 128 : 32;
  using S = Stage<FMT, G, NG, EXACT>;
  static constexpr int WARPS = S::WARPS, COMPUTE = 32 * WARPS;
  using C = Core<FMT, G, NG, NC, PER_SCALE, EXACT>;
  static constexpr int COLS = C::COLS, ROWS = S::ROWS, TILE = MODE == kGate ? ROWS / 2 : ROWS;
  static constexpr int Y = COLS * kColumnPitch, YS = COLS * C::COLUMN_SCALES;
  static constexpr int BYTES = (S::CODES + S::SCALES + Y + YS + 1023) / 1024 * 1024;
  static constexpr int PITCH = ROWS + 1, RED = (kAlongK * COLS * PITCH * 4 + 127) / 128 * 128;
  static constexpr int TABLE = MODE == kGemv ? 0 : kTableBytes;
  static constexpr int FIT = (kSharedBytes - RED - TABLE - 512) / BYTES;
  static constexpr int STAGES = FIT > 6 ? 6 : FIT;
  static constexpr int SMEM = STAGES * BYTES + RED + TABLE + 512 + 1024;
  static_assert(STAGES >= 2, "");
  static constexpr int COPY_WARPS = 3;
  static constexpr int THREADS = COMPUTE + 32 + 32 * COPY_WARPS;
};

// A place in the sequence of units.
struct Unit {
  int key, inner;   // tile, and unit inside the tile
  int e;            // expert
  int row0;         // first row (kGate: hidden value) of the tile
  int col0, cols;   // columns: kGemv: in memory; kGate, kSlots: entries of the table; kDense: the expert's
  int rank, step;
};

template <int MODE, int FMT, int G, int NG, int NC, bool EXACT, bool TENSOR>
__global__ void __launch_bounds__(RingShape<MODE, FMT, G, NG, NC, EXACT, TENSOR>::THREADS, 1)
    ring_kernel(const __grid_constant__ CUtensorMap map, const RingParams p) {
  using Shape = RingShape<MODE, FMT, G, NG, NC, EXACT, TENSOR>;
  using S = typename Shape::S;
  using C = typename Shape::C;
  constexpr int COLS = Shape::COLS, ROWS = Shape::ROWS, TILE = Shape::TILE, STAGES = Shape::STAGES;
  constexpr int kComputeWarps = Shape::WARPS, kComputeThreads = Shape::COMPUTE;
  extern __shared__ uint8_t raw[];
  uint8_t* dyn = raw + (-shared_address(raw) & 1023u);
  float* red = reinterpret_cast<float*>(dyn + STAGES * Shape::BYTES);
  uint64_t* bars = reinterpret_cast<uint64_t*>(dyn + STAGES * Shape::BYTES + Shape::RED + Shape::TABLE);
  volatile int* flags = reinterpret_cast<volatile int*>(bars + 2 * STAGES);   // abort, last, last of an earlier tile, reached
  const uint32_t full = shared_address(bars), empty = full + 8 * STAGES;
  const Bound bound{flags, p.error, p.limit_ns};
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid == 0) {
    for (int i = 0; i < STAGES; ++i) {
      bar_init(full + 8 * i, 1 + 32 * Shape::COPY_WARPS);
      bar_init(empty + 8 * i, kComputeWarps);
    }
    flags[0] = flags[3] = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  Table table;
  int passes = 0;
  if constexpr (MODE != kGemv) {
    // ids were written before the kernel that this one overlaps with began, and so were the
    // weights; the activations were not
    table.lay(reinterpret_cast<uint8_t*>(red) + Shape::RED, p.route.n * p.route.k);
    table.build(p.route, MODE == kDense ? (1 << 30) : COLS, reinterpret_cast<int*>(dyn));
    passes = *table.count;
  }
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");   // the table's scratch becomes the ring
  __syncthreads();
  const int K = p.w.K, steps = (K + S::STEP - 1) / S::STEP;
  const int tiles = (p.rows + TILE - 1) / TILE, groups = MODE == kGemv ? (p.columns + COLS - 1) / COLS : 1;
  // (the host refuses what does not fit 31 bits)
  const int length = MODE == kDense ? passes * steps : steps;   // units of a tile
  const int keys = tiles * (MODE == kGemv ? groups : MODE == kDense ? 1 : passes);
  const int total = keys * length;
  // Shares.  parts > 1: a cluster of CTAs for each tile, whose sums meet in shared memory.  Else equal
  // shares of the units (two at least, so that none between two others is empty), or of whole tiles
  // where that leaves at most a sixth of the CTAs' time unused, about what the shared tiles' joining
  // costs (24576 x 4096, 1 token: 16.3 us with whole tiles, 20.7 with equal shares).
  const int parts = MODE == kGemv || MODE == kDense ? p.parts : 1, grid = static_cast<int>(gridDim.x);
  const bool whole = parts == 1 && keys * 6 >= (keys + grid - 1) / grid * grid * 5;
  const int each = whole ? length : 1, pool = whole ? keys : total;
  const int ctas = max(1, whole ? min(grid, keys) : min(grid, total / 2)), share = pool / ctas, more = pool % ctas;
  auto share_begin = [&](int c) { return (c * share + min(c, more)) * each; };
  auto share_of = [&](int unit) {
    const int larger = more * (share + 1);
    return unit < larger ? unit / (share + 1) : more + (unit - larger) / share;
  };
  int begin = 0, end = 0;
  const int tile_of_cluster = static_cast<int>(blockIdx.x) / parts, rank = static_cast<int>(blockIdx.x) % parts;
  if (parts > 1) {
    begin = tile_of_cluster * length + length * rank / parts;
    end = tile_of_cluster * length + length * (rank + 1) / parts;
  } else if (static_cast<int>(blockIdx.x) < ctas && total > 0) {
    begin = share_begin(blockIdx.x), end = share_begin(blockIdx.x + 1);
  }
  const bool idle = MODE == kDense && total == 0 && parts == 1;   // no expert at all: zeros, below

  auto locate = [&](Unit& u) {
    if constexpr (MODE == kGemv) {
      u.e = 0;
      u.row0 = u.key / groups * TILE;
      u.col0 = u.key % groups * COLS;
      u.cols = min(COLS, p.columns - u.col0);
      u.step = u.inner;
    } else {
      if constexpr (MODE == kDense) {
        u.row0 = u.key * TILE;
        u.rank = u.inner / steps;
        u.step = u.inner - u.rank * steps;
      } else {
        u.rank = u.key / tiles;
        u.row0 = (u.key - u.rank * tiles) * TILE;
        u.step = u.inner;
      }
      u.e = table.experts[u.rank];
      u.col0 = table.first[u.rank];
      u.cols = table.first[u.rank + 1] - u.col0;
    }
  };
  auto start = [&](Unit& u, int i) {
    u.key = i / length;
    u.inner = i - u.key * length;
    locate(u);
  };
  auto advance = [&](Unit& u) {   // to the next unit (of a sequence that has one)
    ++u.inner, ++u.step;
    if (u.inner == length) {
      ++u.key, u.inner = 0;
      if (u.key < keys) locate(u);
    } else if (MODE == kDense && u.step == steps) {
      locate(u);
    }
  };
  // row `r` of a stage among the rows of all matrices; rows past the tile's matrix repeat its last
  auto matrix_row = [&](const Unit& u, int r) {
    const long long base = static_cast<long long>(u.e) * p.w.rows;
    if constexpr (MODE == kGate) return base + (r < TILE ? 0 : p.rows) + min(u.row0 + (r < TILE ? r : r - TILE), p.rows - 1);
    else return base + min(u.row0 + r, p.rows - 1);
  };

  // How the copying warps leave, with a wait of theirs or of a computing warp expired or not: no copy is in
  // flight when the CTA's shared memory is given away.  After an expired wait they may have stopped at
  // different units, at most a ring apart.  They agree on the furthest, and those behind it arrive for the
  // units they have not served; so every barrier of a unit that anyone copied for completes when its
  // copies have landed, and the warp that issues the codes waits for the last ring of them.
  auto furthest = [&](int reached) {
    __syncwarp();
    atomicMax(const_cast<int*>(flags + 3), reached);
    asm volatile("bar.sync 2, %0;" ::"n"(32 * (1 + Shape::COPY_WARPS)) : "memory");
    return flags[3];
  };

  if (warp == kComputeWarps) {
    // -------- codes by tensor copies, activations by bulk copies
    if (TENSOR && lane == 0) asm volatile("prefetch.tensormap [%0];" ::"l"(&map) : "memory");
    if (begin == end) {
      pdl_wait();
      pdl_launch();
      return;
    }
    const int ahead = min(STAGES, end - begin);
    auto codes = [&](const Unit& u, int stage) {
      if constexpr (TENSOR) {
        if (lane == 0) {
          const uint32_t bar = full + 8 * stage, dst = shared_address(dyn) + stage * Shape::BYTES;
          bar_expect(bar, S::CODES);
#pragma unroll
          for (int b = 0; b < kAlongK / 2; ++b) {
            const int x = u.step * (S::STEP / 2) + 128 * b, y = u.e * p.w.rows + u.row0;
            tensor_copy(dst + b * S::BOX, &map, bar, x, y);
            if constexpr (MODE == kGate) tensor_copy(dst + b * S::BOX + TILE * 128, &map, bar, x, y + p.rows);
          }
        }
      }
    };
    auto columns = [&](const Unit& u, int stage) {
      const uint32_t bar = full + 8 * stage, dst = shared_address(dyn) + stage * Shape::BYTES + S::CODES + S::SCALES;
      const int k0 = u.step * S::STEP, bytes = 2 * min(S::STEP, p.y.ld - k0);
      if (lane == 0) bar_arrive_expect(bar, bytes * u.cols);
      __syncwarp();
      for (int j = lane; j < u.cols; j += 32) {
        int v = j;
        long long c = u.col0 + j;
        if constexpr (MODE != kGemv) {
          const int slot = table.slots[u.col0 + j];
          c = MODE == kGate ? slot / p.route.k : slot;
          if (MODE == kDense) v = slot / p.route.k;
        }
        bulk_copy(dst + v * kColumnPitch, p.y.y + c * p.y.ld + k0, bytes, bar);
      }
    };
    Unit u;
    start(u, begin);
    for (int i = 0; i < ahead; ++i) {   // weights before the wait
      codes(u, i);
      advance(u);
    }
    pdl_wait();
    pdl_launch();
    start(u, begin);
    int stage = 0, i = begin;
    uint32_t phase = 0;
    for (; i < end; ++i) {
      if (i - begin >= STAGES) {
        wait(empty + 8 * stage, phase ^ 1u, bound);
        if (__any_sync(0xffffffffu, *bound.abort)) break;   // the warp as one
        codes(u, stage);
      }
      columns(u, stage);
      advance(u);
      if (++stage == STAGES) stage = 0, phase ^= 1u;
    }
    const int upto = furthest(i);
    if (lane == 0) {
      for (; i < upto; ++i) bar_arrive(full + 8 * ((i - begin) % STAGES));
      for (int j = max(begin, upto - STAGES); j < upto; ++j)
        wait_landed(full + 8 * ((j - begin) % STAGES), (j - begin) / STAGES & 1, p.error);
    }
    return;
  }
  if (warp > kComputeWarps) {
    // -------- scales of weights and activations (and codes, without tensor copies) by asynchronous copies
    const int id = tid - kComputeThreads - 32;
    constexpr int THREADS = 32 * Shape::COPY_WARPS;
    if (begin == end) {
      pdl_wait();
      pdl_launch();
      return;
    }
    const int groups_k = K / G;
    // where the tile's rows are: the first row (of each half of a kGate tile) and the last one that
    // counts, which the rows past it repeat
    int had = -1, span = 0;
    long long first_row = 0;
    auto row_of = [&](int r) {   // relative to first_row
      if constexpr (MODE == kGate) return min(r < TILE ? r : r - TILE, span) + (r < TILE ? 0 : p.rows);
      else return min(r, span);
    };
    auto weights = [&](const Unit& u, int stage) {
      const int place = MODE == kDense ? u.key * passes + u.rank : u.key;
      if (place != had) {
        had = place;
        first_row = static_cast<long long>(u.e) * p.w.rows + u.row0;
        span = min(TILE, p.rows - u.row0) - 1;
      }
      const uint32_t st = shared_address(dyn) + stage * Shape::BYTES;
      if constexpr (!TENSOR) {
        const uint8_t* base = p.w.codes + first_row * (K / 2);
        const int left = K / 2 - u.step * (S::STEP / 2);   // bytes
        for (int j = id; j < ROWS * 8 * kAlongK; j += THREADS) {
          const int r = j / (8 * kAlongK), q = j % (8 * kAlongK);   // 8-byte unit q of row r
          const uint8_t* row = base + static_cast<long long>(row_of(r)) * (K / 2) + u.step * (S::STEP / 2);
          const bool in = 8 * q < left;
          copy8(st + q / 16 * S::BOX + r * 128 + 16 * ((q % 16 / 2) ^ (r & 7)) + 8 * (q & 1), in ? row + 8 * q : row, in ? 8 : 0);
        }
      }
      // scales, in pieces of BYTES: a piece is inside the row or past it
      constexpr int ONE = FMT == kInt ? 4 : 1, PER_ROW = S::PER * kAlongK * ONE;   // bytes per row and stage
      const uint8_t* base = static_cast<const uint8_t*>(p.w.scales) + first_row * groups_k * ONE + u.step * PER_ROW;
      const int left = groups_k * ONE - u.step * PER_ROW;
      const uint32_t sc = st + S::CODES;
      auto pieces = [&](auto bytes) {
        constexpr int BYTES = decltype(bytes)::value, EACH = PER_ROW / BYTES;
        for (int j = id; j < ROWS * EACH; j += THREADS) {
          const int r = j / EACH, q = j % EACH * BYTES;
          const uint8_t* src = base + static_cast<long long>(row_of(r)) * (groups_k * ONE);
          const bool in = q < left;
          if (in) src += q;
          if constexpr (BYTES == 16) copy16(sc + r * S::SROW + q, src, in ? 16 : 0);
          else if constexpr (BYTES == 8) copy8(sc + r * S::SROW + q, src, in ? 8 : 0);
          else copy4(sc + r * S::SROW + q, src, in ? 4 : 0);
        }
      };
      if constexpr (FMT == kInt || EXACT) {
        const uintptr_t align = reinterpret_cast<uintptr_t>(p.w.scales) | static_cast<uintptr_t>(groups_k * ONE);
        if (align % 16 == 0) pieces(std::integral_constant<int, 16>{});
        else if (align % 8 == 0) pieces(std::integral_constant<int, 8>{});
        else pieces(std::integral_constant<int, 4>{});
      } else {
        // the aligned words that hold a row's bytes of this stage
        constexpr int WORDS = PER_ROW / 4 + 1;
        const int bytes = min(PER_ROW, left);
        for (int j = id; j < ROWS * WORDS; j += THREADS) {
          const int r = j / WORDS, q = 4 * (j % WORDS);
          const uint8_t* src = base + static_cast<long long>(row_of(r)) * groups_k;
          const int off = static_cast<int>(reinterpret_cast<uintptr_t>(src) & 3u);
          const bool in = q < off + bytes;
          copy4(sc + r * S::SROW + q, src - off + (in ? q : 0), in ? 4 : 0);
        }
      }
    };
    auto columns = [&](const Unit& u, int stage) {
      const uint32_t dst = shared_address(dyn) + stage * Shape::BYTES + S::CODES + S::SCALES + Shape::Y;
      for (int j = id; j < u.cols * kAlongK; j += THREADS) {
        const int i = j / kAlongK, q = j % kAlongK;
        const int at = (u.step * kAlongK + q) * C::YS;
        int v = i;
        long long c = u.col0 + i;
        if constexpr (MODE != kGemv) {
          const int slot = table.slots[u.col0 + i];
          c = MODE == kGate ? slot / p.route.k : slot;
          if (MODE == kDense) v = slot / p.route.k;
        }
        const float* row = p.y.s + c * (p.y.ld / 32);
        const bool in = (u.step * kAlongK + q) * 128 < p.y.ld;
        const uint32_t to = dst + v * C::COLUMN_SCALES + q * 4 * C::YS;
        if constexpr (C::YS == 1) copy4(to, in ? row + at : row, in ? 4 : 0);
        else copy16(to, in ? row + at : row, in ? 16 : 0);
      }
    };
    const int ahead = min(STAGES, end - begin);
    Unit u;
    start(u, begin);
    for (int i = 0; i < ahead; ++i) {
      weights(u, i);
      advance(u);
    }
    pdl_wait();
    pdl_launch();
    start(u, begin);
    int stage = 0, i = begin;
    uint32_t phase = 0;
    for (; i < end; ++i) {
      if (i - begin >= STAGES) {
        wait(empty + 8 * stage, phase ^ 1u, bound);
        if (*bound.abort) break;
        weights(u, stage);
      }
      columns(u, stage);
      bar_arrive_copies(full + 8 * stage);
      advance(u);
      if (++stage == STAGES) stage = 0, phase ^= 1u;
    }
    const int upto = furthest(i);
    for (; i < upto; ++i) bar_arrive(full + 8 * ((i - begin) % STAGES));
    asm volatile("cp.async.wait_all;" ::: "memory");
    return;
  }

  // -------- products
  pdl_wait();
  pdl_launch();
  if (idle) {
    for (long long i = static_cast<long long>(blockIdx.x) * kComputeThreads + tid; i < static_cast<long long>(p.n) * p.rows;
         i += static_cast<long long>(gridDim.x) * kComputeThreads)
      store(static_cast<__nv_bfloat16*>(p.out) + i, 0.0f);
    return;
  }
  auto sync = [] { asm volatile("bar.sync 1, %0;" ::"n"(kComputeThreads) : "memory"); };
  const int wk = warp / S::WR, wr = warp % S::WR, g = lane >> 2, t = lane & 3;
  const int r0 = MODE == kGate ? 32 * wr : 64 * wr, r1 = MODE == kGate ? TILE + r0 : r0 + 32;
  // the tile's pieces, summed in the order of the CTAs, to red
  auto join_pieces = [&](int c0, int c1, int used) {
    auto place = [&](int c) { return p.pieces + (2 * c + (c == c0 ? 1 : 0)) * (COLS * ROWS); };
    // as many loads in flight as there are sums and pieces, eight at most
    constexpr int EACH = (COLS * ROWS + kComputeThreads - 1) / kComputeThreads, ABREAST = EACH >= 8 ? 1 : 8 / EACH;
    float a[EACH];
#pragma unroll
    for (int x = 0; x < EACH; ++x) a[x] = 0.0f;
    for (int c = c0; c <= c1; c += ABREAST) {
      float v[ABREAST][EACH];
#pragma unroll
      for (int y = 0; y < ABREAST; ++y)
#pragma unroll
        for (int x = 0; x < EACH; ++x) {
          const int j = tid + x * kComputeThreads;
          v[y][x] = c + y <= c1 && j < used ? __ldcg(place(c + y) + j) : 0.0f;
        }
#pragma unroll
      for (int y = 0; y < ABREAST; ++y)
#pragma unroll
        for (int x = 0; x < EACH; ++x) a[x] += v[y][x];
    }
#pragma unroll
    for (int x = 0; x < EACH; ++x) {
      const int j = tid + x * kComputeThreads;
      if (j < used) red[j / ROWS * Shape::PITCH + j % ROWS] = a[x];
    }
  };
  // what becomes of a tile's sums in red
  auto finish = [&](int row0, int col0, int cols) {
    if constexpr (MODE == kGemv) {
      const int per = p.f32 ? 2 : 1;
      for (int j = tid; j < COLS / per * ROWS; j += kComputeThreads) {
        const int v = j / ROWS, r = j % ROWS, token = col0 / per + v, row = row0 + r;
        if (row >= p.rows || token >= p.n) continue;
        const long long at = static_cast<long long>(token) * p.rows + row;
        if (p.f32) store(static_cast<float*>(p.out) + at, red[2 * v * Shape::PITCH + r] + red[(2 * v + 1) * Shape::PITCH + r]);
        else store(static_cast<__nv_bfloat16*>(p.out) + at, red[v * Shape::PITCH + r]);
      }
    } else if constexpr (MODE == kGate) {
      for (int j = warp; j < cols * (TILE / 32); j += kComputeWarps) {   // a warp per column and 32 values
        const int v = j / (TILE / 32), b = j % (TILE / 32), h0 = row0 + 32 * b, slot = table.slots[col0 + v];
        if (h0 >= p.rows) continue;
        const float* at = red + v * Shape::PITCH + 32 * b + lane;
        const float gate = at[0], up = at[TILE];
        float h = h0 + lane < p.rows ? gate / (1.0f + expf(-gate)) * up : 0.0f;
        if (p.T) {
          float Trow[G];
          load_transform_row<G>(Trow, p.T, p.T_stride, h0 / 32, lane, p.rows);
          h = transformed<G>(h, Trow, lane);
        }
        const int e = scale_field(warp_max(fabsf(h)));   // one scale per 32 channels here
        __half* y = p.h + static_cast<long long>(slot) * p.h_ld;
        float* s = p.hs + static_cast<long long>(slot) * (p.h_ld / 32);
        y[h0 + (lane & ~7) + pair_place<FMT>(lane & 7)] = __float2half_rn(scaled_up(h, e));
        if (lane == 0) s[h0 / 32] = column_scale(e);
        if (h0 + 32 >= p.rows) {   // zeros up to the padded length
          for (int c = h0 / 32 + 1; c < p.h_ld / 32; ++c) {
            y[32 * c + lane] = __float2half_rn(0.0f);
            if (lane == 0) s[c] = 1.0f;
          }
        }
      }
    } else if constexpr (MODE == kSlots) {
      for (int j = tid; j < cols * ROWS; j += kComputeThreads) {
        const int v = j / ROWS, r = j % ROWS;
        if (row0 + r < p.rows)
          static_cast<float*>(p.out)[static_cast<long long>(table.slots[col0 + v]) * p.rows + row0 + r] =
              red[v * Shape::PITCH + r] * table.weights[col0 + v];
      }
    } else {
      for (int j = tid; j < p.n * ROWS; j += kComputeThreads) {
        const int v = j / ROWS, r = j % ROWS;
        if (row0 + r < p.rows)
          store(static_cast<__nv_bfloat16*>(p.out) + static_cast<long long>(v) * p.rows + row0 + r, red[v * Shape::PITCH + r]);
      }
    }
  };
  int later_key = -1, later_c0 = 0, later_c1 = 0;   // a shared tile that was not the CTA's last
  C core;
  core.begin();
  Unit u{};
  if (begin < end) start(u, begin);
  int stage = 0;
  uint32_t phase = 0;
  bool once = parts > 1;   // a cluster's CTA has one tile, and sums to meet even without units
  for (int i = begin; i < end || once; once = false) {
    if (parts > 1 && begin == end) {
      u.row0 = (MODE == kGemv ? tile_of_cluster / groups : tile_of_cluster) * TILE;
      u.col0 = MODE == kGemv ? tile_of_cluster % groups * COLS : 0;
    }
    const int key = u.key, row0 = u.row0, col0 = u.col0, cols = u.cols;
    const int key_begin = key * length, key_end = key_begin + length, until = min(end, key_end);
    core.clear();
    float ts = 1.0f, mul[NC][2];
    uint32_t live = 0xFFFFFFFFu, shift[C::MT][2] = {};
#pragma unroll
    for (int c = 0; c < NC; ++c) mul[c][0] = mul[c][1] = 1.0f;
    int had = -1;
    for (; i < until; ++i) {
      const int now = MODE == kDense ? u.rank : u.e;
      if (now != had) {
        had = now;
        ts = tensor_scale<FMT>(p.w, u.e);
        if constexpr (FMT != kInt && !EXACT) {
#pragma unroll
          for (int x = 0; x < C::MT; ++x)
#pragma unroll
            for (int h = 0; h < 2; ++h)
              shift[x][h] = 8 * ((static_cast<uint32_t>(reinterpret_cast<uintptr_t>(p.w.scales)) +
                                  static_cast<uint32_t>(matrix_row(u, C::tile_row(x, r0, r1) + 8 * h + C::row_of(g))) * static_cast<uint32_t>(K / G)) & 3u);
        }
        if constexpr (MODE == kDense) {
          live = 0u;
#pragma unroll
          for (int c = 0; c < NC; ++c) mul[c][0] = mul[c][1] = 0.0f;
          for (int j = u.col0; j < u.col0 + u.cols; ++j) {
            const int v = table.slots[j] / p.route.k;
            live |= 1u << v;
#pragma unroll
            for (int c = 0; c < NC; ++c)
#pragma unroll
              for (int x = 0; x < 2; ++x)
                if (v == 8 * c + sum_column<NG>(t, x)) mul[c][x] = table.weights[j];
          }
        }
      }
      wait(full + 8 * stage, phase, bound);
      const int k0 = u.step * S::STEP + 128 * wk;
      if (k0 < K && row0 + r0 < p.rows) {
        const uint8_t* st = dyn + stage * Shape::BYTES;
        core.template add<MODE == kDense>(st, st + S::CODES, st + S::CODES + S::SCALES, st + S::CODES + S::SCALES + Shape::Y,
                                          r0, r1, wk, shift, (K - k0 + G - 1) / G, live, mul, ts, lane);
      }
      __syncwarp();
      if (lane == 0) bar_arrive(empty + 8 * stage);
      if (++stage == STAGES) stage = 0, phase ^= 1u;
      advance(u);
    }
    // the tile's sums: over the warps along K, and over the CTAs that share the tile
    core.join();
    sync();   // the previous tile's sums have been used
    core.put(red + wk * COLS * Shape::PITCH, Shape::PITCH, r0, r1, lane);
    sync();
    auto own_sum = [&](int j) {   // over the warps along K
      const float* from = red + j / ROWS * Shape::PITCH + j % ROWS;
      float a = from[0];
#pragma unroll
      for (int w = 1; w < kAlongK; ++w) a += from[w * COLS * Shape::PITCH];
      return a;
    };
    if constexpr (MODE == kGemv || MODE == kDense) {
      if (parts > 1) {
        for (int j = tid; j < COLS * ROWS; j += kComputeThreads) {
          const float a = own_sum(j);
          red[j / ROWS * Shape::PITCH + j % ROWS] = a;   // this thread alone reads and writes it
        }
        cluster_sync();
        // each CTA writes a share of the tile, summed in the order of the CTAs
        const int per = MODE == kGemv && p.f32 ? 2 : 1;
        for (int j = rank * kComputeThreads + tid; j < COLS / per * ROWS; j += parts * kComputeThreads) {
          const int v = j / ROWS, r = j % ROWS, token = (MODE == kGemv ? col0 / per : 0) + v, row = row0 + r;
          if (row >= p.rows || token >= p.n) continue;
          float a = 0.0f;
          float q[8][2];
#pragma unroll
          for (int c = 0; c < 8; ++c) {   // parts is 8 at most
            q[c][0] = c < parts ? load_remote(red + per * v * Shape::PITCH + r, c) : 0.0f;
            q[c][1] = c < parts && per == 2 ? load_remote(red + (2 * v + 1) * Shape::PITCH + r, c) : 0.0f;
          }
#pragma unroll
          for (int c = 0; c < 8; ++c) a += q[c][0] + q[c][1];
          const long long at = static_cast<long long>(token) * p.rows + row;
          if (MODE == kGemv && p.f32) store(static_cast<float*>(p.out) + at, a);
          else store(static_cast<__nv_bfloat16*>(p.out) + at, a);
        }
        cluster_sync();   // no CTA leaves while others read its sums
        return;
      }
    }
    if (key_begin < begin || key_end > end) {
      // first and last CTA of the tile: the first one's piece is in its second place, the others' are
      // in their first; whoever arrives last adds them up in order
      const int c0 = share_of(key_begin), c1 = share_of(key_end - 1);
      float* to = p.pieces + (2 * static_cast<int>(blockIdx.x) + (static_cast<int>(blockIdx.x) == c0 ? 1 : 0)) * (COLS * ROWS);
      for (int j = tid; j < cols_used(MODE, COLS, cols) * ROWS; j += kComputeThreads) __stcg(to + j, own_sum(j));
      sync();
      if (tid == 0) {
        __threadfence();   // the barrier has ordered the other threads' stores before it
        flags[1] = atomicAdd(&p.arrived[c0], 1u) == static_cast<unsigned int>(c1 - c0);
        __threadfence();
      }
      if (i < end) {
        // not this CTA's last tile: the others go on, and what the arrival says is looked at in the end
        if (tid == 0) flags[2] = flags[1];
        later_key = key, later_c0 = c0, later_c1 = c1;
        continue;
      }
      sync();
      if (flags[1]) {
        join_pieces(c0, c1, cols_used(MODE, COLS, cols) * ROWS);
        sync();
        finish(row0, col0, cols);
      }
    } else {
      for (int j = tid; j < COLS * ROWS; j += kComputeThreads) {
        const float a = own_sum(j);
        red[j / ROWS * Shape::PITCH + j % ROWS] = a;   // this thread alone reads and writes it
      }
      sync();
      finish(row0, col0, cols);
    }
  }
  if (later_key >= 0) {
    sync();
    if (flags[2]) {
      Unit l{};
      start(l, later_key * length);
      join_pieces(later_c0, later_c1, cols_used(MODE, COLS, l.cols) * ROWS);
      sync();
      finish(l.row0, l.col0, l.cols);
    }
  }
}

}  // namespace decode
}  // namespace wush
