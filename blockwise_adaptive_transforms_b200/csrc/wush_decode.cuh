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

// ------------------------------------------------------------------ clusters
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive;\n\tbarrier.cluster.wait;" ::: "memory");
}
// the two halves, for a kernel that has work to do until the others of its cluster are known to run
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.relaxed;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait;" ::: "memory"); }
__device__ __forceinline__ uint32_t remote_address(const void* local, int rank) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(static_cast<uint32_t>(__cvta_generic_to_shared(local))), "r"(rank));
  return a;
}
__device__ __forceinline__ float load_remote(const float* local, int rank) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(remote_address(local, rank)) : "memory");
  return v;
}
__device__ __forceinline__ void store_remote(double* local, int rank, double v) {
  asm volatile("st.shared::cluster.f64 [%0], %1;" ::"r"(remote_address(local, rank)), "d"(v) : "memory");
}

// ------------------------------------------------------------------ router
constexpr int kMaxExperts = 1024, kMaxTopK = 32, kMaxTokens = 64;   // tokens: of a product, the router takes any
constexpr int kRouteCluster = 8, kRouteWarps = 16;

// 8 values from 16 bytes of bf16 or 32 of fp32
__device__ __forceinline__ void load8f(const __nv_bfloat16* p, float (&v)[8]) {
  const uint4 u = *reinterpret_cast<const uint4*>(p);
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) v[2 * j] = __uint_as_float(w[j] << 16), v[2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
}
__device__ __forceinline__ void load8f(const float* p, float (&v)[8]) {
  const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
  v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}

struct RouteParams {
  const __nv_bfloat16* x;
  const void* router;
  int n, d, E, k, renorm;
  int* ids;
  float* weights;
};

// Experts of a warp's tile: four for one or two tokens, eight for eight (matrix instructions).
__host__ __device__ constexpr int route_experts(int tt) { return tt == 8 ? 8 : 4; }

// Shared memory of a CTA: the logits of the token this CTA ranks and their exponentials, and
// partial sums.
template <int TT>
struct RouteShared {
  double logit[kMaxExperts];
  double power[kMaxExperts];
  double part[kRouteWarps][TT][route_experts(TT)];
};

// c += a b for 8 x 4 by 4 x 8 in 64 bits: lane 4 g + t holds a[g][t], b[t][g], c[g][2 t], c[g][2 t + 1]
__device__ __forceinline__ void mma884(double (&c)[2], double a, double b) {
  asm("mma.sync.aligned.m8n8k4.row.col.f64.f64.f64.f64 {%0, %1}, {%2}, {%3}, {%0, %1};"
      : "+d"(c[0]), "+d"(c[1])
      : "d"(a), "d"(b));
}

// an integer that orders as the logit does, NaN with -infinity
__device__ __forceinline__ unsigned long long rank_key(double l) {
  const long long b = __double_as_longlong(isnan(l) ? -CUDART_INF : l + 0.0);   // -0 as 0
  return static_cast<unsigned long long>(b < 0 ? ~b : b ^ (1ll << 63));
}

// The router for TT tokens by a cluster of 8 CTAs: each takes an eighth of the experts, its 16
// warps a group of them and a share of the channels each, and CTA t ranks token t.
//
// Logits are summed in 64 bits: which experts are chosen hangs on their order, and a 32-bit sum
// over thousands of channels can turn round two logits 1e-6 apart.  Every expert's sum takes the
// same order, so equal rows give equal logits and the tie goes to the lower index.
//
// One token of 4096 channels and 64 experts takes 7.3 us, a chain of latencies: launch, the row's
// loads, the cluster's barrier, the ranking (first form, a CTA per token: 48.7 us).  A batch is bound
// by 64-bit multiply-adds, measured at 59 a clock and SM: 129 tokens of 8192 channels with 256 experts
// 55 us, where that rate on all SMs needs 16 (120 tokens: 33 us, 17 clusters do not fit 148 SMs
// side by side).  The matrix instruction takes 8 experts by 8 tokens, with a conversion to 64 bits per
// operand and lane; building the operands from integer fields instead was slower (43 to 31 us with 30
// tokens), so conversions are not the bound; loads further ahead of their use help (34.8 to 33.1 us).
template <class R, int TT>
__device__ __forceinline__ void route_tokens(const RouteParams& p, int token0, int rank, RouteShared<TT>& sh) {
  constexpr int EE = route_experts(TT);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int mine = (p.E + kRouteCluster - 1) / kRouteCluster, e0 = rank * mine, e1 = min(p.E, e0 + mine);
  const int groups = (mine + EE - 1) / EE;
  // as many ways along d as there are warps for, the same for every expert
  const int ways = groups >= kRouteWarps ? 1 : kRouteWarps / groups, at_once = kRouteWarps / ways;
  const int chunks = (p.d + 255) / 256;   // of the channels, to the ways in turn
  const R* router = static_cast<const R*>(p.router);
  for (int g0 = 0; g0 < groups; g0 += at_once) {
    const int group = g0 + warp / ways, way = warp % ways, e = e0 + group * EE;
    const bool works = warp / ways < at_once && e < e1;
    if constexpr (TT == 8) {
      double c[2] = {0.0, 0.0};
      if (works) {
        const int g = lane >> 2, t = lane & 3;
        const R* wr = router + static_cast<long long>(min(e + g, p.E - 1)) * p.d;
        const __nv_bfloat16* xr = p.x + static_cast<long long>(min(token0 + g, p.n - 1)) * p.d;
        for (int ch = way; ch < chunks; ch += ways) {
#pragma unroll 4
          for (int k = 256 * ch + 8 * t; k < 256 * ch + 256; k += 32) {   // 32 channels, 8 per lane, past the row as zeros
            float w[8], x[8];
            const bool in = k < p.d;
            load8f(wr + (in ? k : 0), w);
            load8f(xr + (in ? k : 0), x);
#pragma unroll
            for (int i = 0; i < 8; ++i) mma884(c, in ? static_cast<double>(w[i]) : 0.0, in ? static_cast<double>(x[i]) : 0.0);
          }
        }
        sh.part[warp][2 * t][g] = c[0];
        sh.part[warp][2 * t + 1][g] = c[1];
      }
    } else {
      double acc[TT][EE];
#pragma unroll
      for (int t = 0; t < TT; ++t)
#pragma unroll
        for (int j = 0; j < EE; ++j) acc[t][j] = 0.0;
      if (works) {
        for (int c = way; c < chunks; c += ways) {
          const int k = 256 * c + 8 * lane;
          if (k >= p.d) continue;
          float w[EE][8];
#pragma unroll
          for (int j = 0; j < EE; ++j) load8f(router + static_cast<long long>(min(e + j, p.E - 1)) * p.d + k, w[j]);
          float x[TT][8];
#pragma unroll
          for (int t = 0; t < TT; ++t) load8f(p.x + static_cast<long long>(min(token0 + t, p.n - 1)) * p.d + k, x[t]);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            double wd[EE];
#pragma unroll
            for (int j = 0; j < EE; ++j) wd[j] = static_cast<double>(w[j][i]);
#pragma unroll
            for (int t = 0; t < TT; ++t) {
              const double xd = static_cast<double>(x[t][i]);
#pragma unroll
              for (int j = 0; j < EE; ++j) acc[t][j] = fma(xd, wd[j], acc[t][j]);
            }
          }
        }
      }
#pragma unroll
      for (int t = 0; t < TT; ++t)
#pragma unroll
        for (int j = 0; j < EE; ++j) {
          double a = acc[t][j];
#pragma unroll
          for (int o = 16; o > 0; o >>= 1) a += __shfl_xor_sync(0xffffffffu, a, o);
          if (lane == 0) sh.part[warp][t][j] = a;
        }
    }
    __syncthreads();
    if (g0 == 0) cluster_wait();   // a CTA's shared memory is its own from when it has begun
    // the ways' sums in order, to the CTA that ranks the token
    for (int i = threadIdx.x; i < at_once * EE * TT; i += 32 * kRouteWarps) {
      const int j = i % EE, t = i / EE % TT, gg = i / (EE * TT), to = e0 + (g0 + gg) * EE + j;
      if (to >= e1) continue;
      double a = 0.0;
      for (int w = 0; w < ways; ++w) a += sh.part[gg * ways + w][t][j];
      store_remote(&sh.logit[to], t, a);
    }
    __syncthreads();
  }
  cluster_sync();
  const int t = token0 + rank;
  if (rank >= TT || t >= p.n) return;   // the whole CTA
  double best = -CUDART_INF;
  for (int e = lane; e < p.E; e += 32) best = fmax(best, sh.logit[e]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) best = fmax(best, __shfl_xor_sync(0xffffffffu, best, o));
  for (int e = threadIdx.x; e < p.E; e += 32 * kRouteWarps) sh.power[e] = exp(sh.logit[e] - best);
  __syncthreads();
  if (warp != 0) return;
  double sum = 0.0;   // a NaN logit makes the sum, and with it the token's weights, NaN
  for (int e = lane; e < p.E; e += 32) sum += sh.power[e];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  unsigned taken = 0u;   // bit j: this lane's expert lane + 32 j is chosen
  double chosen = 0.0;
  int kept = 0;   // lane j keeps the j-th chosen expert
  unsigned long long key = 0ull;   // this lane's best expert that is not chosen
  int id = 0x7fffffff;
  auto next = [&] {
    key = 0ull, id = 0x7fffffff;
    for (int i = 0, e = lane; e < p.E; ++i, e += 32) {
      const unsigned long long q = rank_key(sh.logit[e]);
      if (!(taken >> i & 1u) && (id == 0x7fffffff || q > key)) key = q, id = e;
    }
  };
  next();
  for (int j = 0; j < p.k; ++j) {
    // the largest key, then the lowest index that has it; no logit's key is 0
    const unsigned high = static_cast<unsigned>(key >> 32), most = __reduce_max_sync(0xffffffffu, high);
    const unsigned rest = __reduce_max_sync(0xffffffffu, high == most ? static_cast<unsigned>(key) : 0u);
    const bool top = id != 0x7fffffff && high == most && static_cast<unsigned>(key) == rest;
    const int winner = __reduce_min_sync(0xffffffffu, top ? id : 0x7fffffff);
    if (winner == id) {
      taken |= 1u << (id >> 5);
      next();
    }
    if (lane == j) kept = winner;
    if (p.renorm) chosen += sh.power[winner];
  }
  if (lane < p.k) {
    const long long o = static_cast<long long>(t) * p.k + lane;
    p.ids[o] = kept;
    p.weights[o] = static_cast<float>(sh.power[kept] / (p.renorm && !isnan(sum) ? chosen : sum));
  }
}

template <class R, int TT>
__global__ void __cluster_dims__(kRouteCluster) __launch_bounds__(32 * kRouteWarps) route_kernel(const RouteParams p) {
  __shared__ RouteShared<TT> sh;
  cluster_arrive();
  pdl_wait();
  pdl_launch();
  route_tokens<R, TT>(p, static_cast<int>(blockIdx.x) / kRouteCluster * TT, static_cast<int>(blockIdx.x) % kRouteCluster, sh);
}

}  // namespace decode
}  // namespace wush
