// Few-token operators on the library's 4-bit weights: matrix-vector products, the router of
// a mixture-of-experts layer and the layer itself.
//
//   y[t, o] = s_t sum_i s[o, i] sum_r q[o, iG + r] (T_i x_t,i)_r
//
// with the codes q, group scales s and tensor scale s_t that wush_quant_weight writes, and
// the online transform T_i of the activations (paper-graph-ui analysis, section 3.2 "Online
// Activation Transform + Quantize Kernel", without its quantise step: the activations keep
// 16-bit precision, so this is the weight-only form of the layer).
#pragma once
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <math_constants.h>

namespace wush {
namespace decode {

enum { kMx = 0, kNv = 1, kInt = 2 };

__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void pdl_launch() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// A stack of quantised matrices [E][rows][K]: codes u8 [E][rows][K/2], scales [E][rows][K/G],
// tensor scales fp32 [E] (NVFP4).
struct Matrix4 {
  const uint8_t* codes;
  const void* scales;
  const float* ts;
  int rows, K;
};

// the value of a 4-bit code without its scale
template <int FMT>
__device__ __forceinline__ float code_value(uint32_t c) {
  if constexpr (FMT == kInt) {
    return static_cast<float>(static_cast<int>(c ^ 8u) - 8);
  } else {
    // E2M1 under fp16's exponent: the same bits at fp16's place are the value times 2^-14
    const unsigned short h = static_cast<unsigned short>(((c & 8u) << 12) | ((c & 7u) << 9));
    return __half2float(__ushort_as_half(h)) * 16384.0f;
  }
}

template <int FMT>
__device__ __forceinline__ float scale_value(const void* scales, long long i) {
  if constexpr (FMT == kInt) {
    return static_cast<const float*>(scales)[i];
  } else {
    const uint32_t b = static_cast<const uint8_t*>(scales)[i];
    if constexpr (FMT == kMx) return b ? __uint_as_float(b << 23) : __uint_as_float(0x00400000u);   // 2^(b - 127)
    const __half_raw h = __nv_cvt_fp8_to_halfraw(static_cast<__nv_fp8_storage_t>(b), __NV_E4M3);
    return __half2float(__half(h));
  }
}

template <int FMT>
__device__ __forceinline__ float tensor_scale(const Matrix4& w, long long e) {
  return FMT == kNv ? w.ts[e] : 1.0f;
}

// ------------------------------------------------------------------ transform
// y = T_i x per token and block, fp32 [n][ld]; one thread per value.  T_stride: G * G, or 0
// for one matrix shared by all blocks; T null: y = x.
template <int G, class X>
__global__ void transform_kernel(const X* __restrict__ x, const float* __restrict__ T, int T_stride, int n, int K,
                                 float* __restrict__ y, int ld) {
  pdl_wait();
  pdl_launch();
  const int k = blockIdx.x * blockDim.x + threadIdx.x;
  if (k >= K) return;
  const int b = k / G, r = k % G;
  for (int t = blockIdx.y; t < n; t += gridDim.y) {
    const X* xt = x + static_cast<long long>(t) * K;
    float acc;
    if (!T) {
      acc = static_cast<float>(xt[k]);
    } else {
      const float* Tr = T + static_cast<long long>(b) * T_stride + r * G;
      acc = 0.0f;
      for (int c = 0; c < G; ++c) acc = fmaf(Tr[c], static_cast<float>(xt[b * G + c]), acc);
    }
    y[static_cast<long long>(t) * ld + k] = acc;
  }
}

// the dot product of row `row` (under tensor scale ts) with y, summed by a warp (every lane
// gets it).  The two scales are multiplied first: a partial sum under the group scale alone can
// overflow where the result does not.
template <int FMT, int G>
__device__ __forceinline__ float row_dot(const Matrix4& w, long long row, float ts, const float* __restrict__ y,
                                         int lane) {
  const uint8_t* codes = w.codes + row * (w.K / 2);
  const long long s0 = row * (w.K / G);
  float acc = 0.0f;
  for (int k = lane * 8; k < w.K; k += 256) {   // 8 codes, all in one group (G is 16 or 32)
    const uint32_t c = *reinterpret_cast<const uint32_t*>(codes + k / 2);
    float part = 0.0f;
#pragma unroll
    for (int j = 0; j < 8; ++j) part = fmaf(code_value<FMT>((c >> (4 * j)) & 15u), y[k + j], part);
    acc = fmaf(scale_value<FMT>(w.scales, s0 + k / G) * ts, part, acc);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, o);
  return acc;
}

__device__ __forceinline__ void store(float* p, float v) { *p = v; }
__device__ __forceinline__ void store(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

// one warp per output row
template <int FMT, int G, class Y>
__global__ void gemv_kernel(Matrix4 w, const float* __restrict__ y, int ld, int n, Y* __restrict__ out) {
  pdl_wait();
  pdl_launch();
  const int row = blockIdx.x * (blockDim.x / 32) + threadIdx.x / 32, lane = threadIdx.x & 31;
  if (row >= w.rows) return;
  for (int t = 0; t < n; ++t) {
    const float v = row_dot<FMT, G>(w, row, tensor_scale<FMT>(w, 0), y + static_cast<long long>(t) * ld, lane);
    if (lane == 0) store(out + static_cast<long long>(t) * w.rows + row, v);
  }
}

// ------------------------------------------------------------------ router
constexpr int kMaxExperts = 1024, kMaxTopK = 32;

__device__ __forceinline__ double as_double(__nv_bfloat16 v) { return static_cast<double>(__bfloat162float(v)); }
__device__ __forceinline__ double as_double(float v) { return static_cast<double>(v); }

// One CTA per token.  Logits are summed in 64 bits: which experts are chosen hangs on their
// order, and a 32-bit sum over thousands of channels can turn round two logits 1e-6 apart.
template <class R>
__global__ void route_kernel(const __nv_bfloat16* __restrict__ x, const R* __restrict__ router, int n, int d, int E,
                             int k, int renorm, int* __restrict__ ids, float* __restrict__ weights) {
  __shared__ double logit[kMaxExperts];
  pdl_wait();
  pdl_launch();
  const int t = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  for (int e = warp; e < E; e += warps) {
    double a = 0.0;
    for (int c = lane; c < d; c += 32)
      a = fma(as_double(x[static_cast<long long>(t) * d + c]), as_double(router[static_cast<long long>(e) * d + c]), a);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) a += __shfl_xor_sync(0xffffffffu, a, o);
    if (lane == 0) logit[e] = a;
  }
  __syncthreads();
  if (warp != 0) return;
  double best = -CUDART_INF;
  for (int e = lane; e < E; e += 32) best = fmax(best, logit[e]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) best = fmax(best, __shfl_xor_sync(0xffffffffu, best, o));
  double sum = 0.0;   // a NaN logit makes the sum, and with it the token's weights, NaN
  for (int e = lane; e < E; e += 32) sum += exp(logit[e] - best);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  unsigned taken = 0u;   // bit j: this lane's expert lane + 32 j is chosen
  double chosen = 0.0;
  int mine = 0;   // lane j keeps the j-th chosen expert
  for (int j = 0; j < k; ++j) {
    double v = -CUDART_INF;
    int id = 0x7fffffff;
    for (int i = 0, e = lane; e < E; ++i, e += 32) {
      if (taken >> i & 1u) continue;
      const double l = isnan(logit[e]) ? -CUDART_INF : logit[e];   // NaN ranks with -infinity
      if (id == 0x7fffffff || l > v) v = l, id = e;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const double v2 = __shfl_xor_sync(0xffffffffu, v, o);
      const int id2 = __shfl_xor_sync(0xffffffffu, id, o);
      if (id2 != 0x7fffffff && (id == 0x7fffffff || v2 > v || (v2 == v && id2 < id))) v = v2, id = id2;
    }
    if ((id & 31) == lane) taken |= 1u << (id >> 5);
    if (lane == j) mine = id;
    chosen += exp(logit[id] - best);
  }
  if (lane < k) {
    const long long o = static_cast<long long>(t) * k + lane;
    ids[o] = mine;
    weights[o] = static_cast<float>(exp(logit[mine] - best) / (renorm && !isnan(sum) ? chosen : sum));
  }
}

// ------------------------------------------------------------------ experts
__device__ __forceinline__ bool routed(int e, int E) { return e >= 0 && e < E; }

// h[slot][f] = silu(gate) * up for every (token, slot) with an expert; one warp per value
template <int FMT, int G>
__global__ void gate_up_kernel(Matrix4 w, const float* __restrict__ y, int ld, const int* __restrict__ ids, int k,
                               int E, int f, float* __restrict__ h) {
  pdl_wait();
  pdl_launch();
  const int r = blockIdx.x * (blockDim.x / 32) + threadIdx.x / 32, lane = threadIdx.x & 31;
  const int slot = blockIdx.y, e = ids[slot];
  if (r >= f || !routed(e, E)) return;
  const float* yt = y + static_cast<long long>(slot / k) * ld;
  const long long base = static_cast<long long>(e) * w.rows;
  const float ts = tensor_scale<FMT>(w, e);
  const float g = row_dot<FMT, G>(w, base + r, ts, yt, lane);
  const float u = row_dot<FMT, G>(w, base + f + r, ts, yt, lane);
  if (lane == 0) h[static_cast<long long>(slot) * f + r] = g / (1.0f + expf(-g)) * u;
}

template <int FMT, int G>
__global__ void down_kernel(Matrix4 w, const float* __restrict__ y, int ld, const int* __restrict__ ids,
                            const float* __restrict__ weights, int k, int E, __nv_bfloat16* __restrict__ out) {
  pdl_wait();
  pdl_launch();
  const int r = blockIdx.x * (blockDim.x / 32) + threadIdx.x / 32, lane = threadIdx.x & 31, t = blockIdx.y;
  if (r >= w.rows) return;
  float acc = 0.0f;
  for (int j = 0; j < k; ++j) {
    const int slot = t * k + j, e = ids[slot];
    if (!routed(e, E)) continue;
    const float v = row_dot<FMT, G>(w, static_cast<long long>(e) * w.rows + r, tensor_scale<FMT>(w, e),
                                    y + static_cast<long long>(slot) * ld, lane);
    acc = fmaf(weights[slot], v, acc);
  }
  if (lane == 0) store(out + static_cast<long long>(t) * w.rows + r, acc);
}

}  // namespace decode
}  // namespace wush
