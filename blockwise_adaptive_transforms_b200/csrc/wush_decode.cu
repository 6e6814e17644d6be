// Host side of the few-token operators (wush_gemv, wush_moe_route, wush_moe_experts,
// wush_moe_layer): argument checks, workspace layout, kernel selection and launch.
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <climits>
#include <type_traits>
#include <cstdint>

#include "wush.h"
#include "wush_decode_kernels.cuh"
#include "wush_host.h"

namespace {

using wush::is_aligned;
using wush::decode::Matrix4;

#define WUSH_DECODE_CHECK(call)                                                                               \
  do {                                                                                                        \
    const cudaError_t wush_e_ = (call);                                                                       \
    if (wush_e_ != cudaSuccess) return wush::record_cuda_failure(wush_e_, #call, "wush_decode.cu", __LINE__, false); \
  } while (0)

// A launch with programmatic stream serialisation: every kernel here calls
// griddepcontrol.wait before its first read of anything another kernel may have written.
template <typename... KArgs, typename... Args>
int launch(void (*kern)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t s, Args... args) {
  cudaLaunchConfig_t lc = {};
  lc.gridDim = grid;
  lc.blockDim = block;
  lc.dynamicSmemBytes = smem;
  lc.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  lc.attrs = attr;
  lc.numAttrs = WUSH_USE_PDL ? 1 : 0;
  WUSH_DECODE_CHECK(cudaLaunchKernelEx(&lc, kern, args...));
  return WUSH_OK;
}

// The same for a kernel with SMEM bytes of dynamic shared memory, allowed once per device.
template <auto KERN, int SMEM, typename... Args>
int launch_smem(dim3 grid, dim3 block, cudaStream_t s, Args... args) {
  static std::atomic<unsigned long long> configured{0ull};   // one bit per device ordinal
  int dev = 0;
  WUSH_DECODE_CHECK(cudaGetDevice(&dev));
  const unsigned long long bit = 1ull << (dev & 63);
  if (!(configured.load(std::memory_order_acquire) & bit)) {
    WUSH_DECODE_CHECK(cudaFuncSetAttribute(KERN, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM));
    configured.fetch_or(bit, std::memory_order_acq_rel);
  }
  return launch(KERN, grid, block, SMEM, s, args...);
}

constexpr int64_t kMaxTokens = 64;       // rows of one few-token call
constexpr int64_t kMaxDim = 1 << 20;     // channels of one matrix

int64_t round_up(int64_t v, int64_t m) { return (v + m - 1) / m * m; }
int64_t padded(int64_t K) { return round_up(K, 128); }

// transformed activations of `rows` vectors of K channels
int64_t activation_bytes(int64_t rows, int64_t K) { return round_up(rows * padded(K) * 17 / 4, 256); }

int check_format(int G, int fmt) {
  if (fmt < 0 || fmt > 2) return WUSH_ERR_UNSUPPORTED;
  const bool ok = fmt == WUSH_MXFP4 ? G == 32 : fmt == WUSH_NVFP4 ? G == 16 : (G == 16 || G == 32);
  return ok ? WUSH_OK : WUSH_ERR_UNSUPPORTED;
}

int check_matrix(const uint8_t* codes, const void* scales, const float* ts, int fmt) {
  if (!codes || !scales || (fmt == WUSH_NVFP4 && !ts)) return WUSH_ERR_INVALID_ARG;
  if (!is_aligned(codes, 16) || (fmt == WUSH_INT4 && !is_aligned(scales, 4)) ||
      (fmt == WUSH_NVFP4 && !is_aligned(ts, 4)))
    return WUSH_ERR_MISALIGNED;
  return WUSH_OK;
}

using wush::decode::Columns;

// the columns of `rows` vectors of K channels at `ws`: fp16 values, then their scales
Columns columns_at(void* ws, int64_t rows, int64_t K) {
  const int64_t ld = padded(K);
  __half* y = static_cast<__half*>(ws);
  return Columns{y, reinterpret_cast<const float*>(y + rows * ld), static_cast<int>(ld)};
}

template <int FMT, int G, bool SPLIT>
int prep(const __nv_bfloat16* x, const float* T, int shared, int64_t n, int64_t K, const Columns& y, cudaStream_t s) {
  constexpr int per = wush::decode::kPrepTokens;
  const dim3 grid(static_cast<unsigned>(y.ld / 128), static_cast<unsigned>((n + per - 1) / per));
  return launch(wush::decode::prep_kernel<FMT, G, SPLIT>, grid, dim3(128), 0, s, x, T, shared ? 0 : G * G,
                static_cast<int>(n), static_cast<int>(K), y.ld, const_cast<__half*>(y.y), const_cast<float*>(y.s));
}

// whether the kernels' whole-step form takes a matrix: see Ring
bool whole_steps(const Matrix4& w, int fmt, int G) {
  return w.K % 128 == 0 && is_aligned(w.scales, fmt == WUSH_INT4 ? 16 : 128 / G);
}

template <int FMT, int G, int NG, int NC>
int launch_gemv(wush::decode::GemvParams p, cudaStream_t s) {
  constexpr int MT = 2, warps = wush::decode::kGemvWarps;
  constexpr int cols = wush::decode::columns_of(NG, NC);
  const int steps = (p.w.K + 127) / 128;
  p.wk = warps;
  while (p.wk > 1 && p.wk > steps) p.wk /= 2;
  p.col_groups = (p.columns + cols - 1) / cols;
  const int64_t per = static_cast<int64_t>(warps / p.wk) * 16 * MT;
  const int64_t ctas = (p.w.rows + per - 1) / per * p.col_groups;
  if (ctas > INT_MAX) return WUSH_ERR_UNSUPPORTED;
  const dim3 grid(static_cast<unsigned>(ctas)), block(32 * warps);
  if (whole_steps(p.w, FMT, G)) return launch_smem<wush::decode::gemv_kernel<FMT, G, NG, MT, NC, true>, 8 * wush::decode::Ring<FMT, G, MT, true>::BYTES>(grid, block, s, p);
  return launch_smem<wush::decode::gemv_kernel<FMT, G, NG, MT, NC, false>, 8 * wush::decode::Ring<FMT, G, MT, false>::BYTES>(grid, block, s, p);
}

template <int FMT, int G>
int gemv(const __nv_bfloat16* x, const float* T, int shared, const Matrix4& w, int64_t n, void* y, int y_f32, void* ws,
         cudaStream_t s) {
  wush::decode::GemvParams p{};
  p.w = w;
  p.columns = static_cast<int>(y_f32 ? 2 * n : n);
  p.n = static_cast<int>(n);
  p.y = columns_at(ws, p.columns, w.K);
  p.f32 = y_f32 != 0;
  p.out = y;
  const int st = y_f32 ? prep<FMT, G, true>(x, T, shared, n, w.K, p.y, s) : prep<FMT, G, false>(x, T, shared, n, w.K, p.y, s);
  if (st != WUSH_OK) return st;
  if (p.columns <= 2) return launch_gemv<FMT, G, 4, 1>(p, s);
  if (p.columns <= 4) return launch_gemv<FMT, G, 2, 1>(p, s);
  if (p.columns <= 8) return launch_gemv<FMT, G, 1, 1>(p, s);
  return launch_gemv<FMT, G, 1, 2>(p, s);
}

int route(const void* x, const void* router, int router_f32, int64_t n, int64_t d, int E, int k, int renorm, int32_t* ids,
          float* weights, cudaStream_t s) {
  const dim3 grid(static_cast<unsigned>(n));
  const __nv_bfloat16* xb = static_cast<const __nv_bfloat16*>(x);
  if (router_f32)
    return launch(wush::decode::route_kernel<float>, grid, dim3(256), 0, s, xb, static_cast<const float*>(router),
                  static_cast<int>(n), static_cast<int>(d), E, k, renorm, ids, weights);
  return launch(wush::decode::route_kernel<__nv_bfloat16>, grid, dim3(256), 0, s, xb,
                static_cast<const __nv_bfloat16*>(router), static_cast<int>(n), static_cast<int>(d), E, k, renorm, ids,
                weights);
}

struct Moe {
  const __nv_bfloat16* x;
  const int* ids;
  const float* weights;
  const float* T_in;
  const float* T_out;
  int T_in_shared, T_out_shared;
  Matrix4 w_in, w_out;
  int64_t n, d, f;
  int E, k;
  __nv_bfloat16* y;
  char* ws;
};

int sm_count() {
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return 148;
  return sms;
}

template <int FMT, int G, int NG, int NC>
int launch_gate_up(const wush::decode::GateUpParams& p, cudaStream_t s) {
  const int64_t tiles = (p.f + wush::decode::kHidden - 1) / wush::decode::kHidden;
  const int64_t most = tiles * std::min<int64_t>(static_cast<int64_t>(p.route.n) * p.route.k, p.route.E);
  const dim3 grid(static_cast<unsigned>(std::min<int64_t>(most, 2 * sm_count()))), block(32 * wush::decode::kMoeWarps);
  if (whole_steps(p.w, FMT, G)) return launch_smem<wush::decode::gate_up_kernel<FMT, G, NG, NC, true>, 8 * wush::decode::Ring<FMT, G, 4, true>::BYTES>(grid, block, s, p);
  return launch_smem<wush::decode::gate_up_kernel<FMT, G, NG, NC, false>, 8 * wush::decode::Ring<FMT, G, 4, false>::BYTES>(grid, block, s, p);
}

template <int FMT, int G, int NG, int NC>
int launch_down(const wush::decode::DownParams& p, cudaStream_t s) {
  constexpr int MT = 1, cols = wush::decode::columns_of(NG, NC);
  const dim3 grid(static_cast<unsigned>((p.rows + 16 * MT - 1) / (16 * MT)),
                  static_cast<unsigned>((p.route.n + cols - 1) / cols)),
      block(32 * wush::decode::kMoeWarps);
  if (whole_steps(p.w, FMT, G)) return launch_smem<wush::decode::down_kernel<FMT, G, NG, MT, NC, true>, 8 * wush::decode::Ring<FMT, G, MT, true>::BYTES>(grid, block, s, p);
  return launch_smem<wush::decode::down_kernel<FMT, G, NG, MT, NC, false>, 8 * wush::decode::Ring<FMT, G, MT, false>::BYTES>(grid, block, s, p);
}

template <int FMT, int G>
int experts(const Moe& m, cudaStream_t s) {
  const int64_t slots = m.n * m.k;
  const Columns x = columns_at(m.ws, m.n, m.d);
  const Columns h = columns_at(m.ws + activation_bytes(m.n, m.d), slots, m.f);
  int st = prep<FMT, G, false>(m.x, m.T_in, m.T_in_shared, m.n, m.d, x, s);
  if (st != WUSH_OK) return st;
  const wush::decode::Routing route{m.ids, m.weights, static_cast<int>(m.n), m.k, m.E};
  wush::decode::GateUpParams g{};
  g.w = m.w_in;
  g.y = x;
  g.route = route;
  g.f = static_cast<int>(m.f);
  g.T = m.T_out;
  g.T_stride = m.T_out_shared ? 0 : G * G;
  g.h = const_cast<__half*>(h.y);
  g.hs = const_cast<float*>(h.s);
  g.ld = h.ld;
  if (m.n <= 2) st = launch_gate_up<FMT, G, 4, 1>(g, s);
  else if (m.n <= 4) st = launch_gate_up<FMT, G, 2, 1>(g, s);
  else st = launch_gate_up<FMT, G, 1, 1>(g, s);
  if (st != WUSH_OK) return st;
  wush::decode::DownParams d{};
  d.w = m.w_out;
  d.h = h;
  d.route = route;
  d.rows = m.w_out.rows;
  d.out = m.y;
  if (m.n <= 2) return launch_down<FMT, G, 4, 1>(d, s);
  if (m.n <= 4) return launch_down<FMT, G, 2, 1>(d, s);
  if (m.n <= 8) return launch_down<FMT, G, 1, 1>(d, s);
  if (m.n <= 16) return launch_down<FMT, G, 1, 2>(d, s);
  return launch_down<FMT, G, 1, 4>(d, s);
}

template <class F>
int by_format(int fmt, int G, F&& f) {
  using wush::decode::kInt;
  using wush::decode::kMx;
  using wush::decode::kNv;
  if (fmt == WUSH_MXFP4) return f(std::integral_constant<int, kMx>{}, std::integral_constant<int, 32>{});
  if (fmt == WUSH_NVFP4) return f(std::integral_constant<int, kNv>{}, std::integral_constant<int, 16>{});
  if (G == 16) return f(std::integral_constant<int, kInt>{}, std::integral_constant<int, 16>{});
  return f(std::integral_constant<int, kInt>{}, std::integral_constant<int, 32>{});
}

int check_route(const void* x, const void* router, int router_f32, int64_t n, int64_t d, int E, int k,
                const int32_t* ids, const float* weights) {
  if (!x || !router || !ids || !weights) return WUSH_ERR_INVALID_ARG;
  (void)n, (void)d, (void)E, (void)k;
  if (!is_aligned(x, 16) || !is_aligned(router, 16) || !is_aligned(ids, 4) || !is_aligned(weights, 4))
    return WUSH_ERR_MISALIGNED;
  (void)router_f32;
  return WUSH_OK;
}

int check_route_sizes(int64_t n, int64_t d, int E, int k) {
  if (n < 0 || n > INT_MAX || d <= 0 || d > kMaxDim || d % 8 || E <= 0 || k <= 0 || k > E) return WUSH_ERR_INVALID_ARG;
  if (E > wush::decode::kMaxExperts || k > wush::decode::kMaxTopK) return WUSH_ERR_UNSUPPORTED;
  return WUSH_OK;
}

int check_moe_sizes(int64_t n, int64_t d, int64_t f, int E, int k, int G, int fmt) {
  if (n < 0 || d <= 0 || f <= 0 || d > kMaxDim || f > kMaxDim || E <= 0 || k <= 0) return WUSH_ERR_INVALID_ARG;
  const int st = check_format(G, fmt);
  if (st != WUSH_OK) return st;
  if (d % G || f % G) return WUSH_ERR_INVALID_ARG;
  if (n > kMaxTokens || E > wush::decode::kMaxExperts || k > wush::decode::kMaxTopK) return WUSH_ERR_UNSUPPORTED;
  return WUSH_OK;
}

}  // namespace

extern "C" {

int64_t wush_gemv_workspace_bytes(int64_t n_tok, int64_t d_in) {
  if (n_tok < 0 || n_tok > kMaxTokens || d_in <= 0 || d_in > kMaxDim) return -1;
  return activation_bytes(n_tok, d_in);
}

int wush_gemv(const void* x_bf16, const float* T, int T_shared, const uint8_t* codes, const void* scales,
              const float* tensor_scale, int64_t n_tok, int64_t d_out, int64_t d_in, int G, int fmt, void* y,
              int y_f32, void* workspace, int64_t workspace_bytes, wush_stream_t stream) {
  if (n_tok < 0 || d_out <= 0 || d_in <= 0 || d_out > INT_MAX / 2 || d_in > kMaxDim) return WUSH_ERR_INVALID_ARG;
  int st = check_format(G, fmt);
  if (st != WUSH_OK) return st;
  if (d_in % G) return WUSH_ERR_INVALID_ARG;
  if (n_tok > kMaxTokens) return WUSH_ERR_UNSUPPORTED;
  if (n_tok == 0) return WUSH_OK;
  if (!x_bf16 || !y || !workspace) return WUSH_ERR_INVALID_ARG;
  st = check_matrix(codes, scales, tensor_scale, fmt);
  if (st != WUSH_OK) return st;
  if (workspace_bytes < wush_gemv_workspace_bytes(n_tok, d_in)) return WUSH_ERR_INVALID_ARG;
  if (!is_aligned(x_bf16, 16) || (T && !is_aligned(T, 16)) || !is_aligned(y, 16) || !is_aligned(workspace, 16))
    return WUSH_ERR_MISALIGNED;
  const Matrix4 w{codes, scales, tensor_scale, static_cast<int>(d_out), static_cast<int>(d_in)};
  return by_format(fmt, G, [&](auto f, auto g) {
    return gemv<decltype(f)::value, decltype(g)::value>(static_cast<const __nv_bfloat16*>(x_bf16), T, T_shared, w, n_tok,
                                                        y, y_f32, workspace, reinterpret_cast<cudaStream_t>(stream));
  });
}

int wush_moe_route(const void* x_bf16, const void* router, int router_f32, int64_t n_tok, int64_t d, int n_experts,
                   int top_k, int renormalise, int32_t* ids, float* weights, wush_stream_t stream) {
  int st = check_route_sizes(n_tok, d, n_experts, top_k);
  if (st != WUSH_OK || n_tok == 0) return st;
  st = check_route(x_bf16, router, router_f32, n_tok, d, n_experts, top_k, ids, weights);
  if (st != WUSH_OK) return st;
  return route(x_bf16, router, router_f32, n_tok, d, n_experts, top_k, renormalise, ids, weights,
               reinterpret_cast<cudaStream_t>(stream));
}

int64_t wush_moe_workspace_bytes(int64_t n_tok, int64_t d, int64_t f, int top_k) {
  if (n_tok < 0 || n_tok > kMaxTokens || d <= 0 || d > kMaxDim || f <= 0 || f > kMaxDim || top_k <= 0 ||
      top_k > wush::decode::kMaxTopK)
    return -1;
  return activation_bytes(n_tok, d) + 2 * activation_bytes(n_tok * top_k, f);
}

int wush_moe_experts(const void* x_bf16, const int32_t* ids, const float* weights, const float* T_in, int T_in_shared,
                     const uint8_t* in_codes, const void* in_scales, const float* in_tensor_scale, const float* T_out,
                     int T_out_shared, const uint8_t* out_codes, const void* out_scales,
                     const float* out_tensor_scale, int64_t n_tok, int64_t d, int64_t f, int n_experts, int top_k, int G,
                     int fmt, void* y_bf16, void* workspace, int64_t workspace_bytes, wush_stream_t stream) {
  int st = check_moe_sizes(n_tok, d, f, n_experts, top_k, G, fmt);
  if (st != WUSH_OK || n_tok == 0) return st;
  if (!x_bf16 || !ids || !weights || !y_bf16 || !workspace) return WUSH_ERR_INVALID_ARG;
  st = check_matrix(in_codes, in_scales, in_tensor_scale, fmt);
  if (st != WUSH_OK) return st;
  st = check_matrix(out_codes, out_scales, out_tensor_scale, fmt);
  if (st != WUSH_OK) return st;
  if (workspace_bytes < wush_moe_workspace_bytes(n_tok, d, f, top_k)) return WUSH_ERR_INVALID_ARG;
  if (!is_aligned(x_bf16, 16) || !is_aligned(ids, 4) || !is_aligned(weights, 4) || (T_in && !is_aligned(T_in, 16)) ||
      (T_out && !is_aligned(T_out, 16)) || !is_aligned(y_bf16, 16) || !is_aligned(workspace, 16))
    return WUSH_ERR_MISALIGNED;
  Moe m{};
  m.x = static_cast<const __nv_bfloat16*>(x_bf16);
  m.ids = ids;
  m.weights = weights;
  m.T_in = T_in;
  m.T_out = T_out;
  m.T_in_shared = T_in_shared;
  m.T_out_shared = T_out_shared;
  m.w_in = Matrix4{in_codes, in_scales, in_tensor_scale, static_cast<int>(2 * f), static_cast<int>(d)};
  m.w_out = Matrix4{out_codes, out_scales, out_tensor_scale, static_cast<int>(d), static_cast<int>(f)};
  m.n = n_tok;
  m.d = d;
  m.f = f;
  m.E = n_experts;
  m.k = top_k;
  m.y = static_cast<__nv_bfloat16*>(y_bf16);
  m.ws = static_cast<char*>(workspace);
  return by_format(fmt, G, [&](auto f_, auto g_) {
    return experts<decltype(f_)::value, decltype(g_)::value>(m, reinterpret_cast<cudaStream_t>(stream));
  });
}

int wush_moe_layer(const void* x_bf16, const void* router, int router_f32, int renormalise, int32_t* ids,
                   float* weights, const float* T_in, int T_in_shared, const uint8_t* in_codes, const void* in_scales,
                   const float* in_tensor_scale, const float* T_out, int T_out_shared, const uint8_t* out_codes,
                   const void* out_scales, const float* out_tensor_scale, int64_t n_tok, int64_t d, int64_t f,
                   int n_experts, int top_k, int G, int fmt, void* y_bf16, void* workspace, int64_t workspace_bytes,
                   wush_stream_t stream) {
  int st = check_moe_sizes(n_tok, d, f, n_experts, top_k, G, fmt);
  if (st != WUSH_OK) return st;
  st = check_route_sizes(n_tok, d, n_experts, top_k);
  if (st != WUSH_OK || n_tok == 0) return st;
  st = check_route(x_bf16, router, router_f32, n_tok, d, n_experts, top_k, ids, weights);
  if (st != WUSH_OK) return st;
  // every check of the experts' call comes before the first launch
  if (!y_bf16 || !workspace) return WUSH_ERR_INVALID_ARG;
  st = check_matrix(in_codes, in_scales, in_tensor_scale, fmt);
  if (st != WUSH_OK) return st;
  st = check_matrix(out_codes, out_scales, out_tensor_scale, fmt);
  if (st != WUSH_OK) return st;
  if (workspace_bytes < wush_moe_workspace_bytes(n_tok, d, f, top_k)) return WUSH_ERR_INVALID_ARG;
  if ((T_in && !is_aligned(T_in, 16)) || (T_out && !is_aligned(T_out, 16)) || !is_aligned(y_bf16, 16) ||
      !is_aligned(workspace, 16))
    return WUSH_ERR_MISALIGNED;
  st = route(x_bf16, router, router_f32, n_tok, d, n_experts, top_k, renormalise, ids, weights,
             reinterpret_cast<cudaStream_t>(stream));
  if (st != WUSH_OK) return st;
  return wush_moe_experts(x_bf16, ids, weights, T_in, T_in_shared, in_codes, in_scales, in_tensor_scale, T_out,
                          T_out_shared, out_codes, out_scales, out_tensor_scale, n_tok, d, f, n_experts, top_k, G, fmt,
                          y_bf16, workspace, workspace_bytes, stream);
}

}  // extern "C"
