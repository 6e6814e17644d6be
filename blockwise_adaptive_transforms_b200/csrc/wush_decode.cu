// Host side of the few-token operators (wush_gemv, wush_moe_route, wush_moe_experts,
// wush_moe_layer): argument checks, workspace layout, kernel selection and launch.
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <climits>
#include <type_traits>
#include <cstdint>
#include <initializer_list>

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

// Programmatic stream serialisation as the next of a launch's attributes; returns how many there are now.
// Every kernel here calls griddepcontrol.wait before its first read of anything another kernel may have written.
unsigned int with_overlap(cudaLaunchAttribute* attr, unsigned int n) {
  if (!WUSH_USE_PDL) return n;
  attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[n].val.programmaticStreamSerializationAllowed = 1;
  return n + 1;
}

template <typename... KArgs, typename... Args>
int launch(void (*kern)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t s, Args... args) {
  cudaLaunchConfig_t lc = {};
  lc.gridDim = grid;
  lc.blockDim = block;
  lc.dynamicSmemBytes = smem;
  lc.stream = s;
  cudaLaunchAttribute attr[1];
  lc.attrs = attr;
  lc.numAttrs = with_overlap(attr, 0);
  WUSH_DECODE_CHECK(cudaLaunchKernelEx(&lc, kern, args...));
  return WUSH_OK;
}

// The small kernels ask for the ring kernel's division of an SM's memory into L1 and shared memory:
// a kernel that wants another one cannot start on an SM before the last one has left it.
template <typename F>
int same_carveout(F kern, std::atomic<unsigned long long>& configured) {
  int dev = 0;
  WUSH_DECODE_CHECK(cudaGetDevice(&dev));
  const unsigned long long bit = 1ull << (dev & 63);
  if (!(configured.load(std::memory_order_acquire) & bit)) {
    WUSH_DECODE_CHECK(cudaFuncSetAttribute(kern, cudaFuncAttributePreferredSharedMemoryCarveout, cudaSharedmemCarveoutMaxShared));
    configured.fetch_or(bit, std::memory_order_acq_rel);
  }
  return WUSH_OK;
}

using wush::decode::kMaxTokens;
constexpr int64_t kMaxDim = 1 << 20;     // channels of one matrix

// Tokens up to which the down projection sums over experts in place.  Measured against a product per
// slot and a kernel that adds the slots up: 2048 x 1024, 1 token with 8 of 64 experts 30.5 and 32.4 us;
// 4096 x 1024, 8 tokens with 4 of 16 46.1 and 47.1 us; only many experts with few tokens each turn it
// round (4096 x 1536, 8 tokens with 4 of 64: 80.5 and 79.0 us).
constexpr int64_t kDenseDown = 8;
constexpr int64_t kArrivedBytes = 4 * wush::decode::kMaxCtas;
constexpr int64_t kPieceBytes = int64_t{wush::decode::kMaxCtas} * 2 * 16 * 256 * 4;   // sums of shared tiles, 16 columns by 256 rows

int64_t round_up(int64_t v, int64_t m) { return (v + m - 1) / m * m; }
int64_t padded(int64_t K) { return round_up(K, 128); }

// transformed activations of `rows` vectors of K channels
int64_t activation_bytes(int64_t rows, int64_t K) { return round_up(rows * padded(K) * 17 / 4, 256); }

// The kernels count the rows of a stack and the units of a product in 31 bits.  Units: tiles of 64 rows or
// more by stages of 512 channels, for each pass over a tile's channels that the call can come to.
bool countable(int64_t stack_rows, int64_t rows, int64_t K, int64_t passes) {
  return stack_rows <= INT_MAX && (rows + 63) / 64 * ((K + 511) / 512) * passes <= INT_MAX / 2;
}

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

// the transform of x into columns; also clears `arrivals` words at `arrived`
template <int FMT, int G, bool SPLIT>
int prep(const __nv_bfloat16* x, const float* T, int shared, int64_t n, int64_t K, const Columns& y, unsigned int* arrived,
         int arrivals, bool beside, cudaStream_t s) {
  constexpr int per = wush::decode::kPrepTokens;
  const dim3 grid(static_cast<unsigned>(y.ld / 128), static_cast<unsigned>((n + per - 1) / per));
  static std::atomic<unsigned long long> configured{0ull};
  const int st = same_carveout(wush::decode::prep_kernel<FMT, G, SPLIT>, configured);
  if (st != WUSH_OK) return st;
  return launch(wush::decode::prep_kernel<FMT, G, SPLIT>, grid, dim3(128), 0, s, x, T, shared ? 0 : G * G,
                static_cast<int>(n), static_cast<int>(K), y.ld, const_cast<__half*>(y.y), const_cast<float*>(y.s), arrived, arrivals, beside ? 1 : 0);
}

int sm_count(int dev, int* sms) {
  static std::atomic<int> known[64];
  *sms = dev < 64 ? known[dev].load(std::memory_order_relaxed) : 0;
  if (*sms) return WUSH_OK;
  WUSH_DECODE_CHECK(cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev));
  if (dev < 64) known[dev].store(*sms, std::memory_order_relaxed);
  return WUSH_OK;
}

// A tile's units per CTA up to which a cluster shares it.  The sums of a cluster meet in shared memory,
// those of equal shares through L2 in the last CTA to arrive; but a cluster size that divides the SMs
// badly leaves some unused, which a long tile does not make up for.  Measured with clusters and without:
// 4096 x 4096 7.1 and 8.5 us, 4096 x 14336 (3 tokens) 14.5 and 18.5, 8192 x 8192 (8 tokens) 17.0 and 21.3; with
// more units than this 8192 x 65536 64.9 and 54.6, 6144 x 49152 (8 tokens) 54.8 and 43.1.
constexpr int64_t kMostClusterUnits = 16;

// Clusters of c CTAs of a kernel that the device holds at once; asked once per device.
template <auto KERN, int THREADS, int SMEM>
int clusters_that_fit(int dev, int c, int* fit) {
  static std::atomic<int> known[64][9];
  std::atomic<int>* slot = dev < 64 ? &known[dev][c] : nullptr;
  *fit = slot ? slot->load(std::memory_order_relaxed) - 1 : -1;   // 0: not asked yet
  if (*fit >= 0) return WUSH_OK;
  cudaLaunchConfig_t lc = {};
  lc.gridDim = dim3(static_cast<unsigned>(c));
  lc.blockDim = dim3(THREADS);
  lc.dynamicSmemBytes = SMEM;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(c);
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  lc.attrs = attr;
  lc.numAttrs = 1;
  WUSH_DECODE_CHECK(cudaOccupancyMaxActiveClusters(fit, KERN, &lc));
  if (slot) slot->store(*fit + 1, std::memory_order_relaxed);
  return WUSH_OK;
}

// Clusters of the router's size that the device holds at once with an SM for each CTA, asked of a launch
// that wants more than half of an SM's shared memory (the router's own launches want none).
int whole_clusters(int dev, int* fit) {
  constexpr auto kern = wush::decode::route_kernel<float, 1>;
  constexpr int kThreads = 32 * wush::decode::kRouteWarps, kMoreThanHalf = 128 * 1024;   // of an SM's shared memory
  static std::atomic<unsigned long long> configured{0ull};
  const unsigned long long bit = 1ull << (dev & 63);
  if (!(configured.load(std::memory_order_acquire) & bit)) {
    WUSH_DECODE_CHECK(cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kMoreThanHalf));
    configured.fetch_or(bit, std::memory_order_acq_rel);
  }
  return clusters_that_fit<kern, kThreads, kMoreThanHalf>(dev, wush::decode::kRouteCluster, fit);
}

// One CTA per SM, or fewer: every CTA gets at least two units where there are that many.  passes: how
// often a tile's channels are walked, at most: which experts are active is known on the device alone.
template <int MODE, int FMT, int G, int NG, int NC, bool EXACT, bool TENSOR>
int launch_ring_as(wush::decode::RingParams p, int64_t passes, int64_t matrices, cudaStream_t s) {
  using Shape = wush::decode::RingShape<MODE, FMT, G, NG, NC, EXACT, TENSOR>;
  static std::atomic<unsigned long long> configured{0ull};   // one bit per device ordinal
  constexpr auto kern = wush::decode::ring_kernel<MODE, FMT, G, NG, NC, EXACT, TENSOR>;
  int dev = 0, sms = 0;
  WUSH_DECODE_CHECK(cudaGetDevice(&dev));
  const unsigned long long bit = 1ull << (dev & 63);
  if (!(configured.load(std::memory_order_acquire) & bit)) {
    WUSH_DECODE_CHECK(cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Shape::SMEM));
    configured.fetch_or(bit, std::memory_order_acq_rel);
  }
  int st = sm_count(dev, &sms);
  if (st != WUSH_OK) return st;
  st = wush::device_error_word(&p.error);
  if (st != WUSH_OK) return st;
  p.limit_ns = wush::wait_limit_ns();
  CUtensorMap map{};
  if (TENSOR) {
    st = wush::encode_u8_rows(&map, p.w.codes, matrices * p.w.rows, p.w.K / 2, 128, Shape::TILE);
    if (st != WUSH_OK) return st;
  }
  const int64_t tiles = (p.rows + int64_t{Shape::TILE} - 1) / Shape::TILE *
                        (MODE == wush::decode::kGemv ? (p.columns + Shape::COLS - 1) / Shape::COLS : 1);
  const int64_t length = (p.w.K + int64_t{Shape::S::STEP} - 1) / Shape::S::STEP * passes, units = tiles * length;
  int64_t ctas = std::max<int64_t>(1, std::min<int64_t>({units / 2, sms, wush::decode::kMaxCtas}));
  p.parts = 1;
  if (MODE == wush::decode::kGemv || MODE == wush::decode::kDense) {
    // Few tiles with few units each: a cluster per tile, whose sums meet in shared memory, if all of
    // them can be resident at once
    for (int c = 2; c <= 8; ++c) {
      if (tiles * c > sms || c > length) break;
      int fit = 0;
      st = clusters_that_fit<kern, Shape::THREADS, Shape::SMEM>(dev, c, &fit);
      if (st != WUSH_OK) return st;
      if (tiles <= fit) p.parts = c;
    }
    if (length / p.parts > kMostClusterUnits) p.parts = 1;
    if (p.parts > 1) ctas = tiles * p.parts;
  }
  cudaLaunchConfig_t lc = {};
  lc.gridDim = dim3(static_cast<unsigned>(ctas));
  lc.blockDim = dim3(Shape::THREADS);
  lc.dynamicSmemBytes = Shape::SMEM;
  lc.stream = s;
  cudaLaunchAttribute attr[2];
  lc.attrs = attr;
  lc.numAttrs = with_overlap(attr, 0);
  if (p.parts > 1) {
    cudaLaunchAttribute& cluster = attr[lc.numAttrs++];
    cluster.id = cudaLaunchAttributeClusterDimension;
    cluster.val.clusterDim.x = static_cast<unsigned>(p.parts);
    cluster.val.clusterDim.y = cluster.val.clusterDim.z = 1;
  }
  WUSH_DECODE_CHECK(cudaLaunchKernelEx(&lc, kern, map, p));
  return WUSH_OK;
}

// Tensor copies want rows at multiples of 16 bytes (K a multiple of 32).
template <int MODE, int FMT, int G, int NG, int NC>
int launch_ring(const wush::decode::RingParams& p, int64_t passes, int64_t matrices, cudaStream_t s) {
  const bool tensor = p.w.K % 32 == 0;   // always so for G = 32
  if constexpr (FMT == wush::decode::kInt) {
    if constexpr (G == 16) {
      if (!tensor) return launch_ring_as<MODE, FMT, G, NG, NC, true, false>(p, passes, matrices, s);
    }
    return launch_ring_as<MODE, FMT, G, NG, NC, true, true>(p, passes, matrices, s);
  } else {
    if constexpr (G == 16) {   // an odd number of scales per row
      if (!tensor) return launch_ring_as<MODE, FMT, G, NG, NC, false, false>(p, passes, matrices, s);
    }
    if (p.w.K / G % 4 == 0 && is_aligned(p.w.scales, 4)) return launch_ring_as<MODE, FMT, G, NG, NC, true, true>(p, passes, matrices, s);
    return launch_ring_as<MODE, FMT, G, NG, NC, false, true>(p, passes, matrices, s);
  }
}

template <int FMT, int G>
int gemv(const __nv_bfloat16* x, const float* T, int shared, const Matrix4& w, int64_t n, void* y, int y_f32, void* ws,
         cudaStream_t s) {
  wush::decode::RingParams p{};
  p.columns = static_cast<int>(y_f32 ? 2 * n : n);
  p.n = static_cast<int>(n);
  p.y = columns_at(ws, p.columns, w.K);
  p.f32 = y_f32 != 0;
  p.out = y;
  char* rest = static_cast<char*>(ws) + activation_bytes(n, w.K);
  p.w = w;
  p.rows = w.rows;
  p.arrived = reinterpret_cast<unsigned int*>(rest);
  p.pieces = reinterpret_cast<float*>(rest + kArrivedBytes);
  constexpr int arrivals = wush::decode::kMaxCtas;
  const int st = y_f32 ? prep<FMT, G, true>(x, T, shared, n, w.K, p.y, p.arrived, arrivals, false, s)
                       : prep<FMT, G, false>(x, T, shared, n, w.K, p.y, p.arrived, arrivals, false, s);
  if (st != WUSH_OK) return st;
  // As many groups of a row in one instruction as leave room for the columns.  Measured, MXFP4 24576 x
  // 4096: 1 token with 4, 2 and 1 groups 16.5, 16.0 and 22.6 us (NVFP4 18.1, 19.5, 25.3); 4 tokens with 2
  // and 1 16.4 and 24.2 us; 8 tokens with one and two column tiles 23.9 and 30.2 us.
  const int64_t c = p.columns;
  if (c <= 2) return launch_ring<wush::decode::kGemv, FMT, G, 4, 1>(p, 1, 1, s);
  if (c <= 4) return launch_ring<wush::decode::kGemv, FMT, G, 2, 1>(p, 1, 1, s);
  if (c <= 8) return launch_ring<wush::decode::kGemv, FMT, G, 1, 1>(p, 1, 1, s);
  return launch_ring<wush::decode::kGemv, FMT, G, 1, 2>(p, 1, 1, s);
}

template <class R, int TT>
int route_by(const wush::decode::RouteParams& p, cudaStream_t s) {
  return launch(wush::decode::route_kernel<R, TT>, dim3(static_cast<unsigned>((p.n + TT - 1) / TT * wush::decode::kRouteCluster)),
                dim3(32 * wush::decode::kRouteWarps), 0, s, p);
}

template <class R>
int route_as(const wush::decode::RouteParams& p, cudaStream_t s) {
  // Tokens per cluster: as few as leave every cluster SMs of its own (15 clusters on the device measured),
  // then eight on matrix instructions.  Measured with 256 experts of 8192 fp32 channels, 1, 2 and 8
  // tokens per cluster: a batch of 15 23.0, 25.4 and 34 us; of 16 33.1, 25.4 and 34 us (two clusters
  // on the same SMs); of 31 36, 43 and 34 us.
  int dev = 0, fit = 0;
  WUSH_DECODE_CHECK(cudaGetDevice(&dev));
  const int st = whole_clusters(dev, &fit);
  if (st != WUSH_OK) return st;
  if (p.n <= fit) return route_by<R, 1>(p, s);
  if (p.n <= 2 * fit) return route_by<R, 2>(p, s);
  return route_by<R, 8>(p, s);
}

int route(const void* x, const void* router, int router_f32, int64_t n, int64_t d, int E, int k, int renorm, int32_t* ids,
          float* weights, cudaStream_t s) {
  const wush::decode::RouteParams p{static_cast<const __nv_bfloat16*>(x), router, static_cast<int>(n), static_cast<int>(d),
                                    E, k, renorm, ids, weights};
  return router_f32 ? route_as<float>(p, s) : route_as<__nv_bfloat16>(p, s);
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
  bool after_router;   // the kernel launched just before is this call's router
};

template <int MODE, int FMT, int G>
int launch_experts(const wush::decode::RingParams& p, cudaStream_t s) {
  // The groups of an instruction by the columns of an expert: its tokens at most, and where many tokens
  // go to more experts, half the batch's mean or so; an expert with more takes further passes.  Measured
  // with 4096 x 1024, 4 experts a token, 2 and 1 groups: 16 tokens of 64 experts 86.5 and 94.0 us, 40 of 64
  // 128.1 and 140.2, but 64 of 64 178.0 and 162.7, 16 of 16 61.9 and 54.4.
  const int64_t slots = static_cast<int64_t>(p.n) * p.route.k;
  if (p.n <= 2) return launch_ring<MODE, FMT, G, 4, 1>(p, slots, p.route.E, s);
  if (p.n <= 4 || (MODE != wush::decode::kDense && 2 * slots <= 5 * static_cast<int64_t>(p.route.E)))
    return launch_ring<MODE, FMT, G, 2, 1>(p, slots, p.route.E, s);
  return launch_ring<MODE, FMT, G, 1, 1>(p, slots, p.route.E, s);
}

template <int FMT, int G>
int experts(const Moe& m, cudaStream_t s) {
  const int64_t slots = m.n * m.k;
  const Columns x = columns_at(m.ws, m.n, m.d);
  const Columns h = columns_at(m.ws + activation_bytes(m.n, m.d), slots, m.f);
  char* rest = m.ws + activation_bytes(m.n, m.d) + activation_bytes(slots, m.f);
  constexpr int arrivals = wush::decode::kMaxCtas;
  unsigned int* arrived = reinterpret_cast<unsigned int*>(rest);
  int st = prep<FMT, G, false>(m.x, m.T_in, m.T_in_shared, m.n, m.d, x, arrived, 2 * arrivals, m.after_router, s);
  if (st != WUSH_OK) return st;
  const wush::decode::Routing route{m.ids, m.weights, static_cast<int>(m.n), m.k, m.E};
  wush::decode::RingParams g{};
  g.w = m.w_in;
  g.y = x;
  g.route = route;
  g.n = static_cast<int>(m.n);
  g.rows = static_cast<int>(m.f);
  g.T = m.T_out;
  g.T_stride = m.T_out_shared ? 0 : G * G;
  g.h = const_cast<__half*>(h.y);
  g.hs = const_cast<float*>(h.s);
  g.h_ld = h.ld;
  g.arrived = arrived;
  g.pieces = reinterpret_cast<float*>(rest + 2 * kArrivedBytes);
  st = launch_experts<wush::decode::kGate, FMT, G>(g, s);
  if (st != WUSH_OK) return st;
  wush::decode::RingParams d{};
  d.w = m.w_out;
  d.y = h;
  d.route = route;
  d.n = static_cast<int>(m.n);
  d.rows = m.w_out.rows;
  d.arrived = arrived + arrivals;
  d.pieces = g.pieces;
  d.out = m.y;
  if (m.n <= kDenseDown) return launch_experts<wush::decode::kDense, FMT, G>(d, s);
  d.out = rest + 2 * kArrivedBytes + kPieceBytes;
  st = launch_experts<wush::decode::kSlots, FMT, G>(d, s);
  if (st != WUSH_OK) return st;
  return launch(wush::decode::combine_kernel, dim3(static_cast<unsigned>((d.rows + 255) / 256), static_cast<unsigned>(m.n)),
                dim3(256), 0, s, static_cast<const float*>(d.out), route, d.rows, m.y);
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

int check_route(const void* x, const void* router, const int32_t* ids, const float* weights) {
  if (!x || !router || !ids || !weights) return WUSH_ERR_INVALID_ARG;
  if (!is_aligned(x, 16) || !is_aligned(router, 16) || !is_aligned(ids, 4) || !is_aligned(weights, 4))
    return WUSH_ERR_MISALIGNED;
  return WUSH_OK;
}

int check_route_sizes(int64_t n, int64_t d, int E, int k) {
  if (n < 0 || n > INT_MAX / 8 || d <= 0 || d > kMaxDim || d % 8 || E <= 0 || k <= 0 || k > E) return WUSH_ERR_INVALID_ARG;
  if (E > wush::decode::kMaxExperts || k > wush::decode::kMaxTopK) return WUSH_ERR_UNSUPPORTED;
  return WUSH_OK;
}

int check_moe_sizes(int64_t n, int64_t d, int64_t f, int E, int k, int G, int fmt) {
  if (n < 0 || d <= 0 || f <= 0 || d > kMaxDim || f > kMaxDim || E <= 0 || k <= 0) return WUSH_ERR_INVALID_ARG;
  const int st = check_format(G, fmt);
  if (st != WUSH_OK) return st;
  if (d % G || f % G) return WUSH_ERR_INVALID_ARG;
  if (n > kMaxTokens || E > wush::decode::kMaxExperts || k > wush::decode::kMaxTopK) return WUSH_ERR_UNSUPPORTED;
  // an expert has a token once at most, and four tokens a pass at least if it has as many
  const int64_t passes = std::min(n * k, E * ((n + 3) / 4));
  return countable(E * 2 * f, f, d, passes) && countable(E * d, d, f, passes) ? WUSH_OK : WUSH_ERR_UNSUPPORTED;
}

int run_experts(bool after_router, const void* x_bf16, const int32_t* ids, const float* weights, const float* T_in, int T_in_shared,
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
  m.after_router = after_router;
  return by_format(fmt, G, [&](auto f_, auto g_) {
    return experts<decltype(f_)::value, decltype(g_)::value>(m, reinterpret_cast<cudaStream_t>(stream));
  });
}

}  // namespace

extern "C" {

int64_t wush_gemv_workspace_bytes(int64_t n_tok, int64_t d_in) {
  if (n_tok < 0 || n_tok > kMaxTokens || d_in <= 0 || d_in > kMaxDim) return -1;
  return activation_bytes(n_tok, d_in) + kArrivedBytes + kPieceBytes;
}

int wush_gemv(const void* x_bf16, const float* T, int T_shared, const uint8_t* codes, const void* scales,
              const float* tensor_scale, int64_t n_tok, int64_t d_out, int64_t d_in, int G, int fmt, void* y,
              int y_f32, void* workspace, int64_t workspace_bytes, wush_stream_t stream) {
  if (n_tok < 0 || d_out <= 0 || d_in <= 0 || d_out > INT_MAX / 2 || d_in > kMaxDim) return WUSH_ERR_INVALID_ARG;
  int st = check_format(G, fmt);
  if (st != WUSH_OK) return st;
  if (d_in % G) return WUSH_ERR_INVALID_ARG;
  // 16 columns a pass, of which fp32 results take two a token
  if (n_tok > kMaxTokens || !countable(d_out, d_out, d_in, ((y_f32 ? 2 : 1) * n_tok + 15) / 16)) return WUSH_ERR_UNSUPPORTED;
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
  st = check_route(x_bf16, router, ids, weights);
  if (st != WUSH_OK) return st;
  return route(x_bf16, router, router_f32, n_tok, d, n_experts, top_k, renormalise, ids, weights,
               reinterpret_cast<cudaStream_t>(stream));
}

int64_t wush_moe_workspace_bytes(int64_t n_tok, int64_t d, int64_t f, int top_k) {
  if (n_tok < 0 || n_tok > kMaxTokens || d <= 0 || d > kMaxDim || f <= 0 || f > kMaxDim || top_k <= 0 ||
      top_k > wush::decode::kMaxTopK)
    return -1;
  const int64_t parts = n_tok > kDenseDown ? round_up(n_tok * top_k * d * 4, 256) : 0;
  return activation_bytes(n_tok, d) + activation_bytes(n_tok * top_k, f) + 2 * kArrivedBytes + kPieceBytes + parts;
}

int wush_moe_experts(const void* x_bf16, const int32_t* ids, const float* weights, const float* T_in, int T_in_shared,
                     const uint8_t* in_codes, const void* in_scales, const float* in_tensor_scale, const float* T_out,
                     int T_out_shared, const uint8_t* out_codes, const void* out_scales,
                     const float* out_tensor_scale, int64_t n_tok, int64_t d, int64_t f, int n_experts, int top_k, int G,
                     int fmt, void* y_bf16, void* workspace, int64_t workspace_bytes, wush_stream_t stream) {
  return run_experts(false, x_bf16, ids, weights, T_in, T_in_shared, in_codes, in_scales, in_tensor_scale, T_out,
                     T_out_shared, out_codes, out_scales, out_tensor_scale, n_tok, d, f, n_experts, top_k, G, fmt, y_bf16,
                     workspace, workspace_bytes, stream);
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
  st = check_route(x_bf16, router, ids, weights);
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
  return run_experts(true, x_bf16, ids, weights, T_in, T_in_shared, in_codes, in_scales, in_tensor_scale, T_out,
                     T_out_shared, out_codes, out_scales, out_tensor_scale, n_tok, d, f, n_experts, top_k, G, fmt,
                          y_bf16, workspace, workspace_bytes, stream);
}

int wush_selftest_decode_wait_timeout(uint64_t limit_ns, wush_stream_t stream, uint32_t* bits) {
  unsigned int* error = nullptr;
  int st = wush::device_error_word(&error);
  if (st != WUSH_OK) return st;
  wush::decode::selftest_wait_kernel<<<1, 32, 0, reinterpret_cast<cudaStream_t>(stream)>>>(error, limit_ns);
  WUSH_DECODE_CHECK(cudaGetLastError());
  uint32_t word = 0;
  st = wush_device_status(stream, &word);
  if (bits) *bits = word;
  return st;
}

int wush_call_packed(int call, const int64_t* a) {
  if (!a) return WUSH_ERR_INVALID_ARG;
  const auto at = [&](int i) { return reinterpret_cast<void*>(static_cast<intptr_t>(a[i])); };
  const auto num = [&](int i) { return static_cast<int>(a[i]); };
  const auto f32 = [&](int i) { return static_cast<float*>(at(i)); };
  const auto u8 = [&](int i) { return static_cast<const uint8_t*>(at(i)); };
  const auto stream = [&](int i) { return static_cast<wush_stream_t>(at(i)); };
  const auto small = [&](std::initializer_list<int> which) {
    for (int i : which)
      if (a[i] < INT_MIN || a[i] > INT_MAX) return false;
    return true;
  };
  if (call == WUSH_CALL_GEMV)
    return !small({2, 9, 10, 12}) ? WUSH_ERR_INVALID_ARG
                                  : wush_gemv(at(0), f32(1), num(2), u8(3), at(4), f32(5), a[6], a[7], a[8], num(9), num(10),
                                              at(11), num(12), at(13), a[14], stream(15));
  if (call == WUSH_CALL_MOE_ROUTE)
    return !small({2, 5, 6, 7}) ? WUSH_ERR_INVALID_ARG
                                : wush_moe_route(at(0), at(1), num(2), a[3], a[4], num(5), num(6), num(7),
                                                 static_cast<int32_t*>(at(8)), f32(9), stream(10));
  if (call == WUSH_CALL_MOE_EXPERTS)
    return !small({4, 9, 16, 17, 18, 19})
               ? WUSH_ERR_INVALID_ARG
               : wush_moe_experts(at(0), static_cast<const int32_t*>(at(1)), f32(2), f32(3), num(4), u8(5), at(6), f32(7), f32(8),
                                  num(9), u8(10), at(11), f32(12), a[13], a[14], a[15], num(16), num(17), num(18), num(19),
                                  at(20), at(21), a[22], stream(23));
  if (call == WUSH_CALL_MOE_LAYER)
    return !small({2, 3, 7, 12, 19, 20, 21, 22})
               ? WUSH_ERR_INVALID_ARG
               : wush_moe_layer(at(0), at(1), num(2), num(3), static_cast<int32_t*>(at(4)), f32(5), f32(6), num(7), u8(8), at(9),
                                f32(10), f32(11), num(12), u8(13), at(14), f32(15), a[16], a[17], a[18], num(19), num(20),
                                num(21), num(22), at(23), at(24), a[25], stream(26));
  return WUSH_ERR_UNSUPPORTED;
}

}  // extern "C"
