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

// No kernel here declares its inputs __restrict__: a load that is known never to change may be moved
// ahead of the wait, and the kernel before writes what is read after it.
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

template <int FMT>
__device__ __forceinline__ float tensor_scale(const Matrix4& w, long long e) {
  return FMT == kNv ? w.ts[e] : 1.0f;
}

// ------------------------------------------------------------------ router
constexpr int kMaxExperts = 1024, kMaxTopK = 32;

__device__ __forceinline__ double as_double(__nv_bfloat16 v) { return static_cast<double>(__bfloat162float(v)); }
__device__ __forceinline__ double as_double(float v) { return static_cast<double>(v); }

// One CTA per token.  Logits are summed in 64 bits: which experts are chosen hangs on their
// order, and a 32-bit sum over thousands of channels can turn round two logits 1e-6 apart.
template <class R>
__global__ void route_kernel(const __nv_bfloat16* x, const R* router, int n, int d, int E,
                             int k, int renorm, int* ids, float* weights) {
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

}  // namespace decode
}  // namespace wush
