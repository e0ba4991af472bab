// fa_lib.cu -- the C ABI declared in include/fa.h: argument checks, TMA descriptors, launches.
// Host code only decides shapes and launches; every step of the attention itself runs in the
// kernels of fa_prefill.cuh, fa_backward.cuh, fa_decode.cuh, fa_merge.cuh, fa_rope.cuh, fa_cache.cuh
// and fa_q8.cuh.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <climits>
#include <cmath>
#include <cstdint>
#include <cstdlib>
#include <cstring>
#include <mutex>
#include <string>
#include <vector>

#include "fa.h"
#include "fa_backward.cuh"
#include "fa_cache.cuh"
#include "fa_decode.cuh"
#include "fa_merge.cuh"
#include "fa_prefill.cuh"
#include "fa_q8.cuh"
#include "fa_q8_tile.cuh"
#include "fa_rope.cuh"

namespace fa {
// One thread waits on a barrier that nothing arrives at; the bounded wait must give up.
__global__ void selftest_wait_kernel(uint64_t limit_ns) {
  __shared__ uint64_t bar;
  __shared__ int abort_flag;
  if (threadIdx.x != 0) return;
  abort_flag = 0;
  mbar_init(&bar, 1);
  fence_mbar_init();
  mbar_wait(&bar, 0, &abort_flag, limit_ns);  // records FA_ERR_TIMEOUT when it gives up
}

// MUFU throughput probe: every thread runs kEx2Chains independent chains x <- 2^x - 1.5 (which
// stays in [-1.5, 0.5]), so the exponentials, not their latency, bound the kernel.  The sink is
// written only if the sum takes a value it never takes, which keeps the work alive.
constexpr int kEx2Chains = 16;
__global__ void __launch_bounds__(256) ex2_rate_kernel(float *sink, int iters) {
  float x[kEx2Chains];
#pragma unroll
  for (int i = 0; i < kEx2Chains; ++i) x[i] = -1.f + 1e-2f * i + 1e-5f * threadIdx.x;
  for (int it = 0; it < iters; ++it) {
#pragma unroll
    for (int i = 0; i < kEx2Chains; ++i) x[i] = ex2(x[i]) - 1.5f;
  }
  float acc = 0.f;
#pragma unroll
  for (int i = 0; i < kEx2Chains; ++i) acc += x[i];
  if (acc == 1.0e30f) *sink = acc;
}

// HBM read probe: a grid-stride sweep over the buffer with the decode kernel's 16-byte streaming
// loads, four in flight per thread; the words are xor-folded so the loads stay live.
__global__ void __launch_bounds__(512) read_rate_kernel(const uint4 *buf, size_t n16, float *sink) {
  uint32_t acc = 0;
  const size_t stride = static_cast<size_t>(gridDim.x) * blockDim.x;
  size_t i = static_cast<size_t>(blockIdx.x) * blockDim.x + threadIdx.x;
  for (; i + 3 * stride < n16; i += 4 * stride) {
    uint4 a = ld_stream_v4(buf + i), b = ld_stream_v4(buf + i + stride);
    uint4 c = ld_stream_v4(buf + i + 2 * stride), d = ld_stream_v4(buf + i + 3 * stride);
    acc ^= a.x ^ a.y ^ a.z ^ a.w ^ b.x ^ b.y ^ b.z ^ b.w ^ c.x ^ c.y ^ c.z ^ c.w ^ d.x ^ d.y ^ d.z ^ d.w;
  }
  for (; i < n16; i += stride) {
    uint4 a = ld_stream_v4(buf + i);
    acc ^= a.x ^ a.y ^ a.z ^ a.w;
  }
  if (acc == 0x7fc01234u) *sink = __uint_as_float(acc);
}
}  // namespace fa

namespace {

constexpr int kVersion = 100;  // 0.1.0
constexpr int kMaxDevices = 64;

thread_local std::string t_last_error;

fa_status launch_failed(cudaError_t e) {
  t_last_error = cudaGetErrorString(e);
  return FA_ERR_LAUNCH;
}

struct DeviceInfo {
  bool probed = false;
  bool supported = false;
  int num_sms = 0;
  bool prefill_attr[6] = {};  // (d = 64, 128) x (square, paged, key range)
  bool bwd_attr[2] = {false, false};                    // d = 64, 128
  bool q8_attr[16] = {};  // (few, many rows) x (d = 64, 128) x (one, two row tiles) x (e4m3, int8)
};

std::mutex g_mutex;
DeviceInfo g_devices[kMaxDevices];

// Looks up (once per device) whether the current device is an sm_100 part and its SM count.
fa_status current_device(DeviceInfo **out, int *dev_out) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return launch_failed(e);
  if (dev < 0 || dev >= kMaxDevices) return FA_ERR_UNSUPPORTED;
  std::lock_guard<std::mutex> lock(g_mutex);
  DeviceInfo &d = g_devices[dev];
  if (!d.probed) {
    int major = 0, minor = 0, sms = 0;
    if ((e = cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev)) != cudaSuccess ||
        (e = cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev)) != cudaSuccess ||
        (e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess)
      return launch_failed(e);
    d.supported = (major == 10 && minor == 0);
    d.num_sms = sms;
    d.probed = true;
  }
  if (!d.supported) return FA_ERR_UNSUPPORTED;
  *out = &d;
  *dev_out = dev;
  return FA_OK;
}

PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void *ptr = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &ptr, cudaEnableDefault, &q) ==
            cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr);
  });
  return fn;
}

// [BH, N, d] bf16 viewed as a 3-D tensor (d innermost); boxes of 64 x box_rows x 1 with 128-byte
// swizzle, rows past N read as zeros (and not written by stores).
bool encode_bhnd(CUtensorMap *map, const void *base, int d, int N, int BH, int box_rows = 128) {
  auto enc = tensor_map_encoder();
  if (!enc) return false;
  cuuint64_t dims[3] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(N),
                        static_cast<cuuint64_t>(BH)};
  cuuint64_t strides[2] = {static_cast<cuuint64_t>(d) * 2, static_cast<cuuint64_t>(N) * d * 2};
  cuuint32_t box[3] = {64, static_cast<cuuint32_t>(box_rows), 1};
  cuuint32_t estr[3] = {1, 1, 1};
  CUresult r = enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(base), dims,
                   strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                   CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS;
}

// The backward's fp32 dQ accumulator [rows, d] as a 2-D tensor for bulk reductions: boxes of
// 32 features (128 bytes) x box_rows rows, 128-byte swizzle.
bool encode_dq_acc(CUtensorMap *map, float *base, int d, long long rows, int box_rows) {
  auto enc = tensor_map_encoder();
  if (!enc) return false;
  cuuint64_t dims[2] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(rows)};
  cuuint64_t strides[1] = {static_cast<cuuint64_t>(d) * 4};
  cuuint32_t box[2] = {32, static_cast<cuuint32_t>(box_rows)};
  cuuint32_t estr[2] = {1, 1};
  CUresult r = enc(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 2, base, dims, strides, box, estr,
                   CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                   CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS;
}

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

bool overlaps(const void *a, size_t na, const void *b, size_t nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + nb && y < x + na;
}

bool resolve_scale(float scale, int d, float *out) {
  if (std::isnan(scale) || std::isinf(scale)) return false;
  *out = scale > 0.f ? scale : 1.0f / std::sqrt(static_cast<float>(d));
  return true;
}

// The pools [num_blocks, H, 16, d] as a 4-D tensor (d, 16, H, num_blocks) read in 64 x 16 x 1 x 1
// boxes.  Used at d = 64, where that box is a whole 16-token page of one head (2 KB); d = 128 takes
// the 5-D page maps below.
bool encode_pool(CUtensorMap *map, const void *base, int d, int H, int num_blocks) {
  auto enc = tensor_map_encoder();
  if (!enc) return false;
  cuuint64_t dims[4] = {static_cast<cuuint64_t>(d), 16, static_cast<cuuint64_t>(H),
                        static_cast<cuuint64_t>(num_blocks)};
  cuuint64_t strides[3] = {static_cast<cuuint64_t>(d) * 2, static_cast<cuuint64_t>(16) * d * 2,
                           static_cast<cuuint64_t>(H) * 16 * d * 2};
  cuuint32_t box[4] = {64, 16, 1, 1};
  cuuint32_t estr[4] = {1, 1, 1, 1};
  CUresult r = enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void *>(base), dims,
                   strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                   CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS;
}

// The d = 128 V pool as a 5-D tensor (64 columns, 16 tokens, 2 column halves, H, num_blocks) read
// in 64 x 16 x 2 x 1 x 1 boxes: a whole 16-token page of one head (4 KB) per load, landing as
// [half][token][64 columns].  The half stride (128 bytes) is smaller than the token stride (256
// bytes): the box reorders the page so that each half is the 16 x 128-byte K-group pair the P V
// product reads for its 16 keys.
// The d = 128 K pool as a 5-D tensor (64 columns, 8 tokens, 2 column chunks, 2 token groups,
// num_blocks * H pages of one head) read in 64 x 8 x 2 x 2 x 1 boxes: a whole 16-token page of one
// head (4 KB) per load, landing as [token group][chunk][8 tokens][64 columns].  Eight such pages
// make a K tile whose 8-key groups (1 KB swizzle atoms) sit 2 KB apart for each 64-column chunk,
// the layout issue_qk reads for the paged mode.
bool encode_pool_k_pages(CUtensorMap *map, const void *base, int H, int num_blocks) {
  auto enc = tensor_map_encoder();
  if (!enc) return false;
  cuuint64_t dims[5] = {64, 8, 2, 2, static_cast<cuuint64_t>(num_blocks) * H};
  cuuint64_t strides[4] = {256, 128, 8 * 256, 16 * 256};
  cuuint32_t box[5] = {64, 8, 2, 2, 1};
  cuuint32_t estr[5] = {1, 1, 1, 1, 1};
  CUresult r = enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 5, const_cast<void *>(base), dims,
                   strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                   CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS;
}

bool encode_pool_v_pages(CUtensorMap *map, const void *base, int H, int num_blocks) {
  auto enc = tensor_map_encoder();
  if (!enc) return false;
  cuuint64_t dims[5] = {64, 16, 2, static_cast<cuuint64_t>(H), static_cast<cuuint64_t>(num_blocks)};
  cuuint64_t strides[4] = {256, 128, 16 * 256, static_cast<cuuint64_t>(H) * 16 * 256};
  cuuint32_t box[5] = {64, 16, 2, 1, 1};
  cuuint32_t estr[5] = {1, 1, 1, 1, 1};
  CUresult r = enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 5, const_cast<void *>(base), dims,
                   strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                   CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS;
}

// Static unit assignment of a causal square launch (fa::UnitTable).  The units are taken in groups
// of heads whose K and V total at most kGroupKvBytes (a quarter of L2), longest pair level first
// within a group, and each goes to the CTA that frees up first under the cost model "key blocks of
// both tiles + 1.5" (ties to the lowest CTA).  A group keeps at least kMinGroupHeads heads (with
// fewer, dozens of CTAs stream the same head's K/V at once, which measured slower) and there are
// no more groups than full rounds of units.  Returns false when the launch takes no table (d = 64,
// see fa::UnitTableOf; or one group: the level-major snake is then as good).
constexpr double kGroupKvBytes = 32.0 * 1024 * 1024;
constexpr int kMinGroupHeads = 16;

static bool build_unit_table(fa::UnitTable &t, int BH, int N, int num_pairs, int grid, int HD) {
  const int units = BH * num_pairs;
  if (HD != 128 || grid <= 0 || grid > fa::kMaxSchedCtas || units <= grid || units > fa::kMaxSchedUnits)
    return false;
  const double kv_head = 2.0 * N * HD * 2;  // bf16 K and V of one (b, h)
  int groups = static_cast<int>(std::ceil(BH * kv_head / kGroupKvBytes));
  groups = std::min({groups, units / grid, BH / kMinGroupHeads});
  if (groups <= 1) return false;
  auto tile_blocks = [&](int pr, int i) {
    const int q0 = pr * 2 * fa::kBM + i * fa::kBM;
    return q0 >= N ? 0 : (std::min(q0 + fa::kBM, N) - 1) / fa::kBN + 1;
  };
  std::vector<int> owner(units);
  std::vector<int> order;
  order.reserve(units);
  std::vector<std::pair<long, int>> heap;  // (finish time in half blocks, CTA): a min-heap
  for (int c = 0; c < grid; ++c) heap.push_back({0, c});
  auto later = [](const std::pair<long, int> &a, const std::pair<long, int> &b) { return a > b; };
  std::make_heap(heap.begin(), heap.end(), later);
  for (int g = 0, h0 = 0; g < groups; ++g) {
    const int gk = BH / groups + (g < BH % groups ? 1 : 0);
    for (int level = 0; level < num_pairs; ++level) {
      const int pr = num_pairs - 1 - level;
      const long cost = 2L * (tile_blocks(pr, 0) + tile_blocks(pr, 1)) + 3;
      for (int bh = h0; bh < h0 + gk; ++bh) {
        std::pop_heap(heap.begin(), heap.end(), later);
        const int u = level * BH + bh;
        owner[u] = heap.back().second;
        order.push_back(u);
        heap.back().first += cost;
        std::push_heap(heap.begin(), heap.end(), later);
      }
    }
    h0 += gk;
  }
  std::vector<int> count(grid + 1, 0);
  for (int u = 0; u < units; ++u) ++count[owner[u] + 1];
  for (int c = 0; c < grid; ++c) count[c + 1] += count[c];
  for (int c = 0; c <= grid; ++c) t.start[c] = static_cast<uint16_t>(count[c]);
  std::vector<int> fill(count.begin(), count.end() - 1);
  for (int u : order) t.unit[fill[owner[u]]++] = static_cast<uint16_t>(u);  // per CTA in run order
  t.count = units;
  return true;
}

// The table of the last causal square launch made by this thread, reused while the shape repeats.
struct UnitTableCache {
  int BH = -1, N = -1, grid = -1, HD = -1;
  bool valid = false;
  fa::UnitTable table{};
};

static const fa::UnitTable &unit_table(int BH, int N, int num_pairs, int grid, int HD) {
  static thread_local UnitTableCache cache;
  static const fa::UnitTable none{};
  if (cache.BH != BH || cache.N != N || cache.grid != grid || cache.HD != HD) {
    cache.BH = BH, cache.N = N, cache.grid = grid, cache.HD = HD;
    cache.valid = build_unit_table(cache.table, BH, N, num_pairs, grid, HD);
  }
  return cache.valid ? cache.table : none;
}

template <int HD, int kMode>
fa_status launch_prefill(DeviceInfo &dev, const CUtensorMap &tq, const CUtensorMap &tk,
                         const CUtensorMap &tv, fa::PrefillParams p, cudaStream_t stream,
                         const CUtensorMap *to = nullptr) {
  using C = fa::PrefillCfg<HD>;
  p.num_pairs = (p.N + 2 * fa::kBM - 1) / (2 * fa::kBM);
  p.num_units = p.BH * p.num_pairs;
  const int slot = (HD == 128 ? 1 : 0) + 2 * kMode;
  {
    std::lock_guard<std::mutex> lock(g_mutex);
    if (!dev.prefill_attr[slot]) {
      cudaError_t e = cudaFuncSetAttribute(fa::fa_prefill_kernel<HD, kMode>,
                                           cudaFuncAttributeMaxDynamicSharedMemorySize,
                                           static_cast<int>(C::kSmemBytes));
      if (e != cudaSuccess) return launch_failed(e);
      dev.prefill_attr[slot] = true;
    }
  }
  const int grid = p.num_units < dev.num_sms ? p.num_units : dev.num_sms;
  // without an O map (p.o_tma = 0) the kernel never reads its O map argument
  typename fa::UnitTableOf<HD, kMode>::type tab{};
  if constexpr (!std::is_same_v<decltype(tab), fa::NoUnitTable>) {
    if (p.causal) tab = unit_table(p.BH, p.N, p.num_pairs, grid, HD);
  }
  fa::fa_prefill_kernel<HD, kMode><<<grid, fa::kPrefillThreads, C::kSmemBytes, stream>>>(
      tq, tk, tv, to != nullptr ? *to : tq, p, tab);
  cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? FA_OK : launch_failed(e);
}

template <int HD>
fa_status launch_prefill_dense(DeviceInfo &dev, const void *q, const void *k, const void *v,
                               void *o, int o_f32, float *lse, int BH, int N, int causal,
                               float scale, cudaStream_t stream) {
  CUtensorMap tq, tk, tv;
  if (!encode_bhnd(&tq, q, HD, N, BH) || !encode_bhnd(&tk, k, HD, N, BH) ||
      !encode_bhnd(&tv, v, HD, N, BH)) {
    t_last_error = "cuTensorMapEncodeTiled failed";
    return FA_ERR_LAUNCH;
  }
  fa::PrefillParams p{};
  p.o = o;
  p.lse = lse;
  p.o_f32 = o_f32;
  p.BH = BH;
  p.N = N;
  p.causal = causal;
  p.scale_log2 = scale * 1.4426950408889634f;
  p.q_rows = N;
  p.Nk = N;
  // bf16 O leaves through tensor stores of 32-row boxes
  CUtensorMap to;
  p.o_tma = (!o_f32 && encode_bhnd(&to, o, HD, N, BH, 32)) ? 1 : 0;
  return launch_prefill<HD, fa::kModeSquare>(dev, tq, tk, tv, p, stream, p.o_tma ? &to : nullptr);
}

// Backward workspace: dQ accumulator fp32 [BH, Np, d], then LSE2 and D fp32 [BH, Np] each, with
// Np = N rounded up to the 128-row block.
size_t bwd_padded_rows(int BH, int N) {
  return static_cast<size_t>(BH) * ((static_cast<size_t>(N) + fa::kBM - 1) / fa::kBM * fa::kBM);
}

template <int HD>
fa_status launch_bwd(DeviceInfo &dev, const void *q, const void *k, const void *v, const void *o,
                     int o_f32, const void *dout, const float *lse, void *dq, void *dk, void *dv,
                     int g_f32,
                     int BH, int N, int causal, float scale, void *workspace, cudaStream_t stream) {
  using C = fa::BwdCfg<HD>;
  CUtensorMap tq, tk, tv, tdo;
  if (!encode_bhnd(&tq, q, HD, N, BH) || !encode_bhnd(&tk, k, HD, N, BH) ||
      !encode_bhnd(&tv, v, HD, N, BH) || !encode_bhnd(&tdo, dout, HD, N, BH)) {
    t_last_error = "cuTensorMapEncodeTiled failed";
    return FA_ERR_LAUNCH;
  }
  {
    std::lock_guard<std::mutex> lock(g_mutex);
    if (!dev.bwd_attr[HD == 128]) {
      cudaError_t e = cudaFuncSetAttribute(fa::fa_bwd_kernel<HD>,
                                           cudaFuncAttributeMaxDynamicSharedMemorySize,
                                           static_cast<int>(C::kSmemBytes));
      if (e != cudaSuccess) return launch_failed(e);
      dev.bwd_attr[HD == 128] = true;
    }
  }
  const int Np = (N + fa::kBM - 1) / fa::kBM * fa::kBM;
  const size_t prow = static_cast<size_t>(BH) * Np;
  float *dq_acc = static_cast<float *>(workspace);
  float *lse2 = dq_acc + prow * HD;
  float *dvec = lse2 + prow;
  constexpr int kRowThreads = HD / 8;
  const long long prep_threads = static_cast<long long>(prow) * kRowThreads;
  const unsigned prep_blocks = static_cast<unsigned>((prep_threads + 255) / 256);
  if (o_f32)
    fa::fa_bwd_prep_kernel<HD, true><<<prep_blocks, 256, 0, stream>>>(
        o, static_cast<const uint16_t *>(dout), lse, lse2, dvec, dq_acc, BH, N, Np);
  else
    fa::fa_bwd_prep_kernel<HD, false><<<prep_blocks, 256, 0, stream>>>(
        o, static_cast<const uint16_t *>(dout), lse, lse2, dvec, dq_acc, BH, N, Np);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return launch_failed(e);
  fa::BwdParams p{};
  p.lse2 = lse2;
  p.dvec = dvec;
  p.dq_acc = dq_acc;
  p.dk = dk;
  p.dv = dv;
  p.g_f32 = g_f32;
  p.BH = BH;
  p.N = N;
  p.Np = Np;
  p.nkb = Np / fa::kBN;
  p.causal = causal;
  p.scale_log2 = scale * 1.4426950408889634f;
  p.scale = scale;
  CUtensorMap tdq;
  if (!encode_dq_acc(&tdq, dq_acc, HD, static_cast<long long>(prow), C::kBoxRows)) {
    t_last_error = "cuTensorMapEncodeTiled failed";
    return FA_ERR_LAUNCH;
  }
  // persistent: one CTA per SM at most, each taking pairs of key blocks (see the kernel)
  const long long pairs = static_cast<long long>(BH) * ((p.nkb + 1) / 2);
  const unsigned grid = static_cast<unsigned>(pairs < dev.num_sms ? pairs : dev.num_sms);
  fa::fa_bwd_kernel<HD><<<grid, fa::kBwdThreads, C::kSmemBytes, stream>>>(tq, tk, tv, tdo, tdq, p);
  if ((e = cudaGetLastError()) != cudaSuccess) return launch_failed(e);
  const long long post_threads = static_cast<long long>(BH) * N * kRowThreads;
  fa::fa_bwd_dq_kernel<HD><<<static_cast<unsigned>((post_threads + 255) / 256), 256, 0, stream>>>(
      dq_acc, dq, g_f32, scale, BH, N, Np);
  e = cudaGetLastError();
  return e == cudaSuccess ? FA_OK : launch_failed(e);
}

int decode_splits(int max_blocks) {
  return (max_blocks + fa::kDecodeChunkPages - 1) / fa::kDecodeChunkPages;
}

}  // namespace

extern "C" {

fa_status fa_fwd(const void *q, const void *k, const void *v, void *o, fa_out_dtype o_dtype,
                 float *lse, int B, int H, int N, int d, int causal, float scale,
                 fa_stream_t stream) {
  if (!q || !k || !v || !o) return FA_ERR_INVALID_ARG;
  if (B < 1 || H < 1 || N < 1) return FA_ERR_INVALID_ARG;
  if (causal != 0 && causal != 1) return FA_ERR_INVALID_ARG;
  if (o_dtype != FA_OUT_BF16 && o_dtype != FA_OUT_F32) return FA_ERR_INVALID_ARG;
  if (d != 64 && d != 128) return FA_ERR_UNSUPPORTED;
  if (static_cast<long long>(B) * H > INT_MAX) return FA_ERR_INVALID_ARG;
  // work units (pairs of 128-row query tiles) are counted in an int
  if (static_cast<long long>(B) * H * ((static_cast<long long>(N) + 2 * fa::kBM - 1) / (2 * fa::kBM)) >
      INT_MAX)
    return FA_ERR_INVALID_ARG;
  float sc;
  if (!resolve_scale(scale, d, &sc)) return FA_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o)) return FA_ERR_ALIGNMENT;
  if (lse && (reinterpret_cast<uintptr_t>(lse) & 3u)) return FA_ERR_ALIGNMENT;
  const int BH = B * H;
  const size_t rows = static_cast<size_t>(BH) * N;
  const size_t in_bytes = rows * d * 2;
  const size_t o_bytes = rows * d * (o_dtype == FA_OUT_F32 ? 4 : 2);
  if (overlaps(o, o_bytes, q, in_bytes) || overlaps(o, o_bytes, k, in_bytes) ||
      overlaps(o, o_bytes, v, in_bytes))
    return FA_ERR_INVALID_ARG;
  if (lse && (overlaps(lse, rows * 4, q, in_bytes) || overlaps(lse, rows * 4, k, in_bytes) ||
              overlaps(lse, rows * 4, v, in_bytes) || overlaps(lse, rows * 4, o, o_bytes)))
    return FA_ERR_INVALID_ARG;
  DeviceInfo *dev = nullptr;
  int dev_id = 0;
  fa_status st = current_device(&dev, &dev_id);
  if (st != FA_OK) return st;
  const int o_f32 = o_dtype == FA_OUT_F32;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (d == 128) return launch_prefill_dense<128>(*dev, q, k, v, o, o_f32, lse, BH, N, causal, sc, s);
  return launch_prefill_dense<64>(*dev, q, k, v, o, o_f32, lse, BH, N, causal, sc, s);
}

size_t fa_bwd_workspace_size(int B, int H, int N, int d) {
  if (B < 1 || H < 1 || N < 1 || (d != 64 && d != 128)) return 0;
  if (static_cast<long long>(B) * H > INT_MAX) return 0;
  return bwd_padded_rows(B * H, N) * (d + 2) * sizeof(float);
}

fa_status fa_bwd(const void *q, const void *k, const void *v, const void *o, fa_out_dtype o_dtype,
                 const void *dout, const float *lse, void *dq, void *dk, void *dv,
                 fa_out_dtype g_dtype, int B, int H, int N, int d, int causal, float scale,
                 void *workspace, size_t workspace_bytes, fa_stream_t stream) {
  if (!q || !k || !v || !o || !dout || !lse || !dq || !dk || !dv) return FA_ERR_INVALID_ARG;
  if (B < 1 || H < 1 || N < 1) return FA_ERR_INVALID_ARG;
  if (causal != 0 && causal != 1) return FA_ERR_INVALID_ARG;
  if (g_dtype != FA_OUT_BF16 && g_dtype != FA_OUT_F32) return FA_ERR_INVALID_ARG;
  if (o_dtype != FA_OUT_BF16 && o_dtype != FA_OUT_F32) return FA_ERR_INVALID_ARG;
  if (d != 64 && d != 128) return FA_ERR_UNSUPPORTED;
  if (static_cast<long long>(B) * H > INT_MAX) return FA_ERR_INVALID_ARG;
  const int BH = B * H;
  if (static_cast<long long>(BH) * ((N + fa::kBN - 1) / fa::kBN) > INT_MAX) return FA_ERR_INVALID_ARG;
  float sc;
  if (!resolve_scale(scale, d, &sc)) return FA_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o) || !aligned16(dout) ||
      !aligned16(dq) || !aligned16(dk) || !aligned16(dv))
    return FA_ERR_ALIGNMENT;
  if (reinterpret_cast<uintptr_t>(lse) & 3u) return FA_ERR_ALIGNMENT;
  const size_t need = fa_bwd_workspace_size(B, H, N, d);
  if (!workspace || workspace_bytes < need) return FA_ERR_WORKSPACE;
  if (!aligned16(workspace)) return FA_ERR_ALIGNMENT;
  const size_t rows = static_cast<size_t>(BH) * N;
  const size_t in_bytes = rows * d * 2, g_bytes = rows * d * (g_dtype == FA_OUT_F32 ? 4 : 2);
  const size_t o_bytes = rows * d * (o_dtype == FA_OUT_F32 ? 4 : 2);
  const void *ins[6] = {q, k, v, o, dout, lse};
  const size_t in_sizes[6] = {in_bytes, in_bytes, in_bytes, o_bytes, in_bytes, rows * 4};
  void *outs[4] = {dq, dk, dv, workspace};
  const size_t out_sizes[4] = {g_bytes, g_bytes, g_bytes, need};
  for (int a = 0; a < 4; ++a) {
    for (int b = 0; b < 6; ++b)
      if (overlaps(outs[a], out_sizes[a], ins[b], in_sizes[b])) return FA_ERR_INVALID_ARG;
    for (int b = a + 1; b < 4; ++b)
      if (overlaps(outs[a], out_sizes[a], outs[b], out_sizes[b])) return FA_ERR_INVALID_ARG;
  }
  DeviceInfo *dev = nullptr;
  int dev_id = 0;
  fa_status st = current_device(&dev, &dev_id);
  if (st != FA_OK) return st;
  const int g_f32 = g_dtype == FA_OUT_F32, o_f32 = o_dtype == FA_OUT_F32;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (d == 128)
    return launch_bwd<128>(*dev, q, k, v, o, o_f32, dout, lse, dq, dk, dv, g_f32, BH, N, causal,
                           sc, workspace, s);
  return launch_bwd<64>(*dev, q, k, v, o, o_f32, dout, lse, dq, dk, dv, g_f32, BH, N, causal, sc,
                        workspace, s);
}

size_t fa_decode_workspace_size(int num_seqs, int H, int d, int max_blocks_per_seq) {
  if (num_seqs < 1 || H < 1 || max_blocks_per_seq < 1 || (d != 64 && d != 128)) return 0;
  const size_t units = static_cast<size_t>(num_seqs) * H * decode_splits(max_blocks_per_seq);
  return units * (d + 2) * sizeof(float);
}

fa_status fa_decode_paged(const void *q, const void *k_pool, const void *v_pool,
                          const int32_t *block_table, int max_blocks_per_seq,
                          const int32_t *seq_lens, int num_blocks, void *o, fa_out_dtype o_dtype,
                          float *lse, int S, int H, int d, float scale, void *workspace,
                          size_t workspace_bytes, fa_stream_t stream) {
  if (!q || !k_pool || !v_pool || !block_table || !seq_lens || !o) return FA_ERR_INVALID_ARG;
  if (S < 1 || H < 1 || max_blocks_per_seq < 1 || num_blocks < 1) return FA_ERR_INVALID_ARG;
  if (o_dtype != FA_OUT_BF16 && o_dtype != FA_OUT_F32) return FA_ERR_INVALID_ARG;
  if (d != 64 && d != 128) return FA_ERR_UNSUPPORTED;
  if (static_cast<long long>(S) * H > INT_MAX / 4) return FA_ERR_INVALID_ARG;
  if (static_cast<long long>(max_blocks_per_seq) * fa::kPage > INT_MAX) return FA_ERR_INVALID_ARG;
  float sc;
  if (!resolve_scale(scale, d, &sc)) return FA_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k_pool) || !aligned16(v_pool) || !aligned16(o))
    return FA_ERR_ALIGNMENT;
  if ((reinterpret_cast<uintptr_t>(block_table) & 3u) || (reinterpret_cast<uintptr_t>(seq_lens) & 3u))
    return FA_ERR_ALIGNMENT;
  if (lse && (reinterpret_cast<uintptr_t>(lse) & 3u)) return FA_ERR_ALIGNMENT;
  const size_t need = fa_decode_workspace_size(S, H, d, max_blocks_per_seq);
  if (!workspace || workspace_bytes < need) return FA_ERR_WORKSPACE;
  if (!aligned16(workspace)) return FA_ERR_ALIGNMENT;
  const size_t o_bytes = static_cast<size_t>(S) * H * d * (o_dtype == FA_OUT_F32 ? 4 : 2);
  if (overlaps(o, o_bytes, workspace, need) || (lse && overlaps(lse, static_cast<size_t>(S) * H * 4, workspace, need)))
    return FA_ERR_INVALID_ARG;
  DeviceInfo *dev = nullptr;
  int dev_id = 0;
  fa_status st = current_device(&dev, &dev_id);
  if (st != FA_OK) return st;

  fa::DecodeParams p;
  p.q = static_cast<const uint16_t *>(q);
  p.kp = static_cast<const uint16_t *>(k_pool);
  p.vp = static_cast<const uint16_t *>(v_pool);
  p.table = block_table;
  p.lens = seq_lens;
  p.max_blocks = max_blocks_per_seq;
  p.num_blocks = num_blocks;
  p.H = H;
  p.scale_log2 = sc * 1.4426950408889634f;
  p.ws = static_cast<float *>(workspace);
  p.n_split = decode_splits(max_blocks_per_seq);
  p.o = o;
  p.o_f32 = o_dtype == FA_OUT_F32;
  p.lse = lse;
  p.SH = S * H;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const dim3 grid1(p.n_split, H, S);
  const int grid2 = (p.SH + 3) / 4;
  if (d == 128) {
    fa::fa_decode_partial_kernel<128><<<grid1, fa::kDecodeThreads, 0, s>>>(p);
    fa::fa_decode_combine_kernel<128><<<grid2, 128, 0, s>>>(p);
  } else {
    fa::fa_decode_partial_kernel<64><<<grid1, fa::kDecodeThreads, 0, s>>>(p);
    fa::fa_decode_combine_kernel<64><<<grid2, 128, 0, s>>>(p);
  }
  cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? FA_OK : launch_failed(e);
}

}  // extern "C"

// ---------------------------------------------------------------------------------------------
// Allocation-free decode: the split-context scratch lives in a static device array.
// ---------------------------------------------------------------------------------------------
namespace {

// Held by every GPU that loads this library, for the life of the process.
static __device__ __align__(256) unsigned char g_noalloc_scratch[FA_NOALLOC_SCRATCH_BYTES];

std::mutex g_noalloc_mutex;
void *g_noalloc_ptr[kMaxDevices] = {};

// Device address of g_noalloc_scratch on `dev` (the current device), looked up once per device.
// In host code the array's name is only a host-side stand-in, never a device address.
fa_status noalloc_scratch(int dev, void **out) {
  std::lock_guard<std::mutex> lock(g_noalloc_mutex);
  if (!g_noalloc_ptr[dev]) {
    void *ptr = nullptr;
    cudaError_t e = cudaGetSymbolAddress(&ptr, g_noalloc_scratch);
    if (e != cudaSuccess) return launch_failed(e);
    if (!ptr) {
      t_last_error = "cudaGetSymbolAddress returned no address for the decode scratch";
      return FA_ERR_LAUNCH;
    }
    g_noalloc_ptr[dev] = ptr;
  }
  *out = g_noalloc_ptr[dev];
  return FA_OK;
}

}  // namespace

extern "C" {

fa_status fa_decode_paged_noalloc(const void *q, const void *k_pool, const void *v_pool,
                                  const int32_t *block_table, int max_blocks_per_seq,
                                  const int32_t *seq_lens, int num_blocks, void *o,
                                  fa_out_dtype o_dtype, float *lse, int S, int H, int d,
                                  float scale, fa_stream_t stream) {
  if (!q || !k_pool || !v_pool || !block_table || !seq_lens || !o) return FA_ERR_INVALID_ARG;
  if (S < 1 || H < 1 || max_blocks_per_seq < 1 || num_blocks < 1) return FA_ERR_INVALID_ARG;
  if (o_dtype != FA_OUT_BF16 && o_dtype != FA_OUT_F32) return FA_ERR_INVALID_ARG;
  if (d != 64 && d != 128) return FA_ERR_UNSUPPORTED;
  if (static_cast<long long>(S) * H > INT_MAX / 4) return FA_ERR_INVALID_ARG;
  if (static_cast<long long>(max_blocks_per_seq) * fa::kPage > INT_MAX) return FA_ERR_INVALID_ARG;
  float sc;
  if (!resolve_scale(scale, d, &sc)) return FA_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k_pool) || !aligned16(v_pool) || !aligned16(o))
    return FA_ERR_ALIGNMENT;
  if ((reinterpret_cast<uintptr_t>(block_table) & 3u) || (reinterpret_cast<uintptr_t>(seq_lens) & 3u))
    return FA_ERR_ALIGNMENT;
  if (lse && (reinterpret_cast<uintptr_t>(lse) & 3u)) return FA_ERR_ALIGNMENT;
  const size_t need = fa_decode_workspace_size(S, H, d, max_blocks_per_seq);
  if (need > FA_NOALLOC_SCRATCH_BYTES) {
    t_last_error = "fa_decode_paged_noalloc: these sizes need " + std::to_string(need) +
                   " bytes of scratch; the static array holds " +
                   std::to_string(FA_NOALLOC_SCRATCH_BYTES);
    return FA_ERR_WORKSPACE;
  }
  DeviceInfo *dev = nullptr;
  int dev_id = 0;
  fa_status st = current_device(&dev, &dev_id);
  if (st != FA_OK) return st;
  void *scratch = nullptr;
  if ((st = noalloc_scratch(dev_id, &scratch)) != FA_OK) return st;

  fa::DecodeParams p;
  p.q = static_cast<const uint16_t *>(q);
  p.kp = static_cast<const uint16_t *>(k_pool);
  p.vp = static_cast<const uint16_t *>(v_pool);
  p.table = block_table;
  p.lens = seq_lens;
  p.max_blocks = max_blocks_per_seq;
  p.num_blocks = num_blocks;
  p.H = H;
  p.scale_log2 = sc * 1.4426950408889634f;
  p.ws = static_cast<float *>(scratch);
  p.n_split = decode_splits(max_blocks_per_seq);
  p.o = o;
  p.o_f32 = o_dtype == FA_OUT_F32;
  p.lse = lse;
  p.SH = S * H;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const dim3 grid1(p.n_split, H, S);
  const int grid2 = (p.SH + 3) / 4;
  if (d == 128) {
    fa::fa_decode_partial_kernel<128><<<grid1, fa::kDecodeThreads, 0, s>>>(p);
    fa::fa_decode_combine_kernel<128><<<grid2, 128, 0, s>>>(p);
  } else {
    fa::fa_decode_partial_kernel<64><<<grid1, fa::kDecodeThreads, 0, s>>>(p);
    fa::fa_decode_combine_kernel<64><<<grid2, 128, 0, s>>>(p);
  }
  cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? FA_OK : launch_failed(e);
}

// Shared body of fa_prefill_paged and fa_tree_attention (tree_mask null: plain or causal chunk).
static fa_status prefill_paged_impl(const void *q, const void *k_pool, const void *v_pool,
                             const int32_t *block_table, int max_blocks_per_seq,
                                    const int32_t *seq_lens, int num_blocks,
                                    const uint64_t *tree_mask, void *o, fa_out_dtype o_dtype,
                                    float *lse, int S, int H, int Lq, int d, int causal,
                                    float scale, fa_stream_t stream) {
  if (!q || !k_pool || !v_pool || !block_table || !seq_lens || !o) return FA_ERR_INVALID_ARG;
  if (S < 1 || H < 1 || Lq < 1 || max_blocks_per_seq < 1 || num_blocks < 1) return FA_ERR_INVALID_ARG;
  if (causal != 0 && causal != 1) return FA_ERR_INVALID_ARG;
  if (o_dtype != FA_OUT_BF16 && o_dtype != FA_OUT_F32) return FA_ERR_INVALID_ARG;
  if (d != 64 && d != 128) return FA_ERR_UNSUPPORTED;
  if (static_cast<long long>(S) * H * Lq > INT_MAX) return FA_ERR_INVALID_ARG;
  if (static_cast<long long>(max_blocks_per_seq) * fa::kPage > INT_MAX) return FA_ERR_INVALID_ARG;
  if (Lq > max_blocks_per_seq * fa::kPage) return FA_ERR_INVALID_ARG;
  // the d = 128 K map indexes (block, head) pages as block * H + head, block up to num_blocks
  if ((static_cast<long long>(num_blocks) + 1) * H > INT_MAX) return FA_ERR_INVALID_ARG;
  float sc;
  if (!resolve_scale(scale, d, &sc)) return FA_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k_pool) || !aligned16(v_pool) || !aligned16(o))
    return FA_ERR_ALIGNMENT;
  if ((reinterpret_cast<uintptr_t>(block_table) & 3u) || (reinterpret_cast<uintptr_t>(seq_lens) & 3u))
    return FA_ERR_ALIGNMENT;
  if (lse && (reinterpret_cast<uintptr_t>(lse) & 3u)) return FA_ERR_ALIGNMENT;
  const size_t rows = static_cast<size_t>(S) * H * Lq;
  const size_t q_bytes = rows * d * 2, o_bytes = rows * d * (o_dtype == FA_OUT_F32 ? 4 : 2);
  const size_t pool_bytes = static_cast<size_t>(num_blocks) * H * fa::kPage * d * 2;
  if (overlaps(o, o_bytes, q, q_bytes) || overlaps(o, o_bytes, k_pool, pool_bytes) ||
      overlaps(o, o_bytes, v_pool, pool_bytes))
    return FA_ERR_INVALID_ARG;
  if (lse && (overlaps(lse, rows * 4, o, o_bytes) || overlaps(lse, rows * 4, q, q_bytes) ||
              overlaps(lse, rows * 4, k_pool, pool_bytes) || overlaps(lse, rows * 4, v_pool, pool_bytes)))
    return FA_ERR_INVALID_ARG;
  DeviceInfo *dev = nullptr;
  int dev_id = 0;
  fa_status st = current_device(&dev, &dev_id);
  if (st != FA_OK) return st;
  CUtensorMap tq, tk, tv;
  const int BH = S * H;
  // d = 128: K and V pages arrive as one 4 KB box each (see encode_pool_k_pages / _v_pages)
  const bool pages = d == 128;
  if (!encode_bhnd(&tq, q, d, Lq, BH) ||
      !(pages ? encode_pool_k_pages(&tk, k_pool, H, num_blocks)
              : encode_pool(&tk, k_pool, d, H, num_blocks)) ||
      !(pages ? encode_pool_v_pages(&tv, v_pool, H, num_blocks)
              : encode_pool(&tv, v_pool, d, H, num_blocks))) {
    t_last_error = "cuTensorMapEncodeTiled failed";
    return FA_ERR_LAUNCH;
  }
  fa::PrefillParams p{};
  p.o = o;
  p.lse = lse;
  p.o_f32 = o_dtype == FA_OUT_F32;
  p.BH = BH;
  p.N = Lq;
  p.causal = causal;
  p.scale_log2 = sc * 1.4426950408889634f;
  p.seq_lens = seq_lens;
  p.block_table = block_table;
  p.max_blocks = max_blocks_per_seq;
  p.num_blocks = num_blocks;
  p.H = H;
  p.tree_mask = tree_mask;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  p.q_rows = Lq;
  // bf16 O leaves through tensor stores of 32-row boxes ([S * H, Lq, d] view)
  CUtensorMap to;
  p.o_tma = (o_dtype == FA_OUT_BF16 && encode_bhnd(&to, o, d, Lq, BH, 32)) ? 1 : 0;
  const CUtensorMap *top = p.o_tma ? &to : nullptr;
  if (d == 128) return launch_prefill<128, fa::kModePaged>(*dev, tq, tk, tv, p, s, top);
  return launch_prefill<64, fa::kModePaged>(*dev, tq, tk, tv, p, s, top);
}

fa_status fa_prefill_paged(const void *q, const void *k_pool, const void *v_pool,
                           const int32_t *block_table, int max_blocks_per_seq,
                           const int32_t *seq_lens, int num_blocks, void *o, fa_out_dtype o_dtype,
                           float *lse, int S, int H, int Lq, int d, int causal, float scale,
                           fa_stream_t stream) {
  return prefill_paged_impl(q, k_pool, v_pool, block_table, max_blocks_per_seq, seq_lens,
                            num_blocks, nullptr, o, o_dtype, lse, S, H, Lq, d, causal, scale,
                            stream);
}

fa_status fa_tree_attention(const void *q, const void *k_pool, const void *v_pool,
                            const int32_t *block_table, int max_blocks_per_seq,
                            const int32_t *seq_lens, int num_blocks, const uint64_t *tree_mask,
                            void *o, fa_out_dtype o_dtype, float *lse, int S, int H, int T, int d,
                            float scale, fa_stream_t stream) {
  if (!tree_mask) return FA_ERR_INVALID_ARG;
  if (T < 1 || T > 64) return FA_ERR_INVALID_ARG;
  if (reinterpret_cast<uintptr_t>(tree_mask) & 7u) return FA_ERR_ALIGNMENT;
  if (S >= 1 && H >= 1 && (d == 64 || d == 128)) {
    const size_t o_bytes =
        static_cast<size_t>(S) * H * T * d * (o_dtype == FA_OUT_F32 ? 4 : 2);
    if (overlaps(o, o_bytes, tree_mask, static_cast<size_t>(S) * T * 8)) return FA_ERR_INVALID_ARG;
  }
  return prefill_paged_impl(q, k_pool, v_pool, block_table, max_blocks_per_seq, seq_lens,
                            num_blocks, tree_mask, o, o_dtype, lse, S, H, T, d, 0, scale, stream);
}

fa_status fa_fwd_keyrange(const void *q, const void *k, const void *v, void *o, fa_out_dtype o_dtype,
                          float *lse, int B, int H, int Nq, int q_row0, int Nk, int k_pos0, int d,
                          int causal, float scale, fa_stream_t stream) {
  if (!q || !k || !v || !o) return FA_ERR_INVALID_ARG;
  if (B < 1 || H < 1 || Nq < 1 || Nk < 1 || q_row0 < 0 || q_row0 >= Nq || k_pos0 < 0)
    return FA_ERR_INVALID_ARG;
  if (causal != 0 && causal != 1) return FA_ERR_INVALID_ARG;
  if (o_dtype != FA_OUT_BF16 && o_dtype != FA_OUT_F32) return FA_ERR_INVALID_ARG;
  if (d != 64 && d != 128) return FA_ERR_UNSUPPORTED;
  if (static_cast<long long>(B) * H > INT_MAX) return FA_ERR_INVALID_ARG;
  // work units (pairs of 128-row query tiles) are counted in an int
  if (static_cast<long long>(B) * H * ((static_cast<long long>(Nq) + 2 * fa::kBM - 1) / (2 * fa::kBM)) >
      INT_MAX)
    return FA_ERR_INVALID_ARG;
  float sc;
  if (!resolve_scale(scale, d, &sc)) return FA_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o)) return FA_ERR_ALIGNMENT;
  if (lse && (reinterpret_cast<uintptr_t>(lse) & 3u)) return FA_ERR_ALIGNMENT;
  const int BH = B * H;
  const size_t qrows = static_cast<size_t>(BH) * Nq, krows = static_cast<size_t>(BH) * Nk;
  const size_t o_bytes = qrows * d * (o_dtype == FA_OUT_F32 ? 4 : 2);
  if (overlaps(o, o_bytes, q, qrows * d * 2) || overlaps(o, o_bytes, k, krows * d * 2) ||
      overlaps(o, o_bytes, v, krows * d * 2))
    return FA_ERR_INVALID_ARG;
  if (lse && (overlaps(lse, qrows * 4, o, o_bytes) || overlaps(lse, qrows * 4, q, qrows * d * 2) ||
              overlaps(lse, qrows * 4, k, krows * d * 2) || overlaps(lse, qrows * 4, v, krows * d * 2)))
    return FA_ERR_INVALID_ARG;
  DeviceInfo *dev = nullptr;
  int dev_id = 0;
  fa_status st = current_device(&dev, &dev_id);
  if (st != FA_OK) return st;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const int o_f32 = o_dtype == FA_OUT_F32;
  // causal: rows before the range's first key see none of it
  const int q_start = causal ? std::max(q_row0, std::min(k_pos0, Nq)) : q_row0;
  if (q_start > q_row0) {
    const long long threads = static_cast<long long>(BH) * (q_start - q_row0) * (d / 4);
    const unsigned blocks = static_cast<unsigned>((threads + 255) / 256);
    if (d == 128)
      fa::fa_empty_rows_kernel<128><<<blocks, 256, 0, s>>>(o, o_f32, lse, BH, Nq, q_row0, q_start);
    else
      fa::fa_empty_rows_kernel<64><<<blocks, 256, 0, s>>>(o, o_f32, lse, BH, Nq, q_row0, q_start);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return launch_failed(e);
  }
  if (q_start >= Nq) return FA_OK;
  CUtensorMap tq, tk, tv;
  if (!encode_bhnd(&tq, q, d, Nq, BH) || !encode_bhnd(&tk, k, d, Nk, BH) ||
      !encode_bhnd(&tv, v, d, Nk, BH)) {
    t_last_error = "cuTensorMapEncodeTiled failed";
    return FA_ERR_LAUNCH;
  }
  fa::PrefillParams p{};
  p.o = o;
  p.lse = lse;
  p.o_f32 = o_f32;
  p.BH = BH;
  p.N = Nq - q_start;
  p.causal = causal;
  p.scale_log2 = sc * 1.4426950408889634f;
  p.q_row0 = q_start;
  p.q_rows = Nq;
  p.Nk = Nk;
  p.q_off = causal ? q_start - k_pos0 : 0;
  if (d == 128) return launch_prefill<128, fa::kModeRange>(*dev, tq, tk, tv, p, s);
  return launch_prefill<64, fa::kModeRange>(*dev, tq, tk, tv, p, s);
}

fa_status fa_merge_partials(const float *o_parts, const float *lse_parts, int G, long long rows,
                            int d, void *o, fa_out_dtype o_dtype, float *lse, fa_stream_t stream) {
  if (!o_parts || !lse_parts || !o) return FA_ERR_INVALID_ARG;
  if (G < 1 || rows < 1) return FA_ERR_INVALID_ARG;
  if (o_dtype != FA_OUT_BF16 && o_dtype != FA_OUT_F32) return FA_ERR_INVALID_ARG;
  if (d != 64 && d != 128) return FA_ERR_UNSUPPORTED;
  if (rows > (1ll << 40) / d) return FA_ERR_INVALID_ARG;
  if (!aligned16(o_parts) || !aligned16(o) || (reinterpret_cast<uintptr_t>(lse_parts) & 3u))
    return FA_ERR_ALIGNMENT;
  if (lse && (reinterpret_cast<uintptr_t>(lse) & 3u)) return FA_ERR_ALIGNMENT;
  const size_t o_bytes = static_cast<size_t>(rows) * d * (o_dtype == FA_OUT_F32 ? 4 : 2);
  const size_t parts_bytes = static_cast<size_t>(G) * rows * d * 4;
  if (overlaps(o, o_bytes, o_parts, parts_bytes) ||
      overlaps(o, o_bytes, lse_parts, static_cast<size_t>(G) * rows * 4))
    return FA_ERR_INVALID_ARG;
  if (lse && (overlaps(lse, rows * 4, o_parts, parts_bytes) || overlaps(lse, rows * 4, o, o_bytes)))
    return FA_ERR_INVALID_ARG;
  DeviceInfo *dev = nullptr;
  int dev_id = 0;
  fa_status st = current_device(&dev, &dev_id);
  if (st != FA_OK) return st;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const long long threads = rows * (d / 4);
  const unsigned blocks = static_cast<unsigned>((threads + 255) / 256);
  const int o_f32 = o_dtype == FA_OUT_F32;
  if (d == 128)
    fa::fa_merge_kernel<128><<<blocks, 256, 0, s>>>(o_parts, lse_parts, G, rows, o, o_f32, lse);
  else
    fa::fa_merge_kernel<64><<<blocks, 256, 0, s>>>(o_parts, lse_parts, G, rows, o, o_f32, lse);
  cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? FA_OK : launch_failed(e);
}

fa_status fa_get_device_status(fa_stream_t stream) {
  cudaError_t e = cudaStreamSynchronize(reinterpret_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return launch_failed(e);
  int v = 0;
  if ((e = cudaMemcpyFromSymbol(&v, fa::g_device_status, sizeof v)) != cudaSuccess)
    return launch_failed(e);
  if (v != 0) {
    const int zero = 0;
    if ((e = cudaMemcpyToSymbol(fa::g_device_status, &zero, sizeof zero)) != cudaSuccess)
      return launch_failed(e);
  }
  return static_cast<fa_status>(v);
}

fa_status fa_selftest_wait_timeout(unsigned limit_us, fa_stream_t stream) {
  if (limit_us < 1 || limit_us > 2000000u) return FA_ERR_INVALID_ARG;
  DeviceInfo *dev = nullptr;
  int dev_id = 0;
  fa_status st = current_device(&dev, &dev_id);
  if (st != FA_OK) return st;
  fa::selftest_wait_kernel<<<1, 32, 0, reinterpret_cast<cudaStream_t>(stream)>>>(
      static_cast<uint64_t>(limit_us) * 1000ull);
  cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? FA_OK : launch_failed(e);
}

fa_status fa_probe_ex2_rate(float *sink, int iters, long long *exps_out, fa_stream_t stream) {
  if (!sink || !exps_out || iters < 1 || iters > (1 << 24)) return FA_ERR_INVALID_ARG;
  DeviceInfo *dev = nullptr;
  int dev_id = 0;
  fa_status st = current_device(&dev, &dev_id);
  if (st != FA_OK) return st;
  const int blocks = 4 * dev->num_sms;  // 32 warps per SM: 8 per sub-partition
  fa::ex2_rate_kernel<<<blocks, 256, 0, reinterpret_cast<cudaStream_t>(stream)>>>(sink, iters);
  *exps_out = static_cast<long long>(blocks) * 256 * iters * fa::kEx2Chains;
  cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? FA_OK : launch_failed(e);
}

fa_status fa_probe_read_rate(const void *buf, size_t bytes, float *sink, fa_stream_t stream) {
  if (!buf || !sink || bytes < 16 || bytes % 16) return FA_ERR_INVALID_ARG;
  if (!aligned16(buf)) return FA_ERR_ALIGNMENT;
  DeviceInfo *dev = nullptr;
  int dev_id = 0;
  fa_status st = current_device(&dev, &dev_id);
  if (st != FA_OK) return st;
  fa::read_rate_kernel<<<4 * dev->num_sms, 512, 0, reinterpret_cast<cudaStream_t>(stream)>>>(
      static_cast<const uint4 *>(buf), bytes / 16, sink);
  cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? FA_OK : launch_failed(e);
}

const char *fa_status_string(fa_status status) {
  switch (status) {
    case FA_OK: return "FA_OK";
    case FA_ERR_INVALID_ARG: return "FA_ERR_INVALID_ARG: an argument is out of range";
    case FA_ERR_UNSUPPORTED: return "FA_ERR_UNSUPPORTED: head dim must be 64 or 128 on an sm_100 GPU";
    case FA_ERR_ALIGNMENT: return "FA_ERR_ALIGNMENT: tensors must be 16-byte aligned";
    case FA_ERR_LAUNCH: return "FA_ERR_LAUNCH: the CUDA launch failed (see fa_last_error_string)";
    case FA_ERR_TIMEOUT: return "FA_ERR_TIMEOUT: a kernel abandoned a device-side wait";
    case FA_ERR_WORKSPACE: return "FA_ERR_WORKSPACE: decode workspace missing or too small";
  }
  return "unknown fa_status";
}

const char *fa_last_error_string(void) { return t_last_error.c_str(); }

fa_status fa_fwd_schedule(int B, int H, int N, int d, int num_ctas, int *start, int *unit,
                          int capacity, int *count) {
  if (count == nullptr || start == nullptr || unit == nullptr) return FA_ERR_INVALID_ARG;
  *count = 0;
  if (B < 1 || H < 1 || N < 1 || num_ctas < 1 || num_ctas > 1024) return FA_ERR_INVALID_ARG;
  if (d != 64 && d != 128) return FA_ERR_UNSUPPORTED;
  const long long BH = static_cast<long long>(B) * H;
  const long long pairs = (static_cast<long long>(N) + 2 * fa::kBM - 1) / (2 * fa::kBM);
  if (BH * pairs > INT_MAX) return FA_ERR_INVALID_ARG;
  const int units = static_cast<int>(BH * pairs);
  if (capacity < units) return FA_ERR_INVALID_ARG;
  const int grid = std::min(units, num_ctas);
  static thread_local fa::UnitTable t;
  if (!build_unit_table(t, static_cast<int>(BH), N, static_cast<int>(pairs), grid, d)) return FA_OK;
  for (int c = 0; c <= num_ctas; ++c) start[c] = c <= grid ? t.start[c] : units;
  for (int i = 0; i < units; ++i) unit[i] = t.unit[i];
  *count = units;
  return FA_OK;
}

int fa_version(void) { return kVersion; }

}  // extern "C"

// ---------------------------------------------------------------------------------------------
// Rotary positions, the 8-bit paged cache, and the attention that reads it.
// ---------------------------------------------------------------------------------------------
namespace {

bool aligned(const void *p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// The rotation's arguments: rot = 0 turns nothing, and positions and freqs may then be null.
fa_status check_rope(const int32_t *positions, const double *freqs, int rot, fa_rope_layout layout,
                     float amplitude, int d, int inverse, fa::RopeTable *out) {
  if (rot < 0 || rot > d || rot % 16 != 0) return FA_ERR_INVALID_ARG;
  if (layout != FA_ROPE_HALF && layout != FA_ROPE_INTERLEAVED) return FA_ERR_INVALID_ARG;
  if (inverse != 0 && inverse != 1) return FA_ERR_INVALID_ARG;
  if (!std::isfinite(amplitude)) return FA_ERR_INVALID_ARG;
  if (rot > 0 && (!positions || !freqs)) return FA_ERR_INVALID_ARG;
  if (!aligned(positions, 4) || !aligned(freqs, 8)) return FA_ERR_ALIGNMENT;
  *out = fa::RopeTable{freqs, rot, layout == FA_ROPE_INTERLEAVED, amplitude, inverse ? -1.f : 1.f};
  return FA_OK;
}

// The memory from the first to the last element of bf16 rows [T, H, d] with these strides.
struct Span {
  const void *p;
  size_t bytes;
};

Span row_span(const void *x, const long long *strides, int T, int H, int d) {
  const long long n[2] = {T, H};
  long long lo = 0, hi = d;
  for (int a = 0; a < 2; ++a)
    if (n[a] > 1) (strides[a] < 0 ? lo : hi) += (n[a] - 1) * strides[a];
  return Span{static_cast<const char *>(x) + 2 * lo, static_cast<size_t>(hi - lo) * 2};
}

using Wide = __int128;  // strides are the caller's and may be anything

// Strided rows: `bytes` contiguous bytes at p + sum of i_a s_a for all 0 <= i_a < n_a, strides in bytes.
struct Rows {
  const void *p;
  long long bytes, n[3];
  Wide s[3];
};

// Is there a sum r + sum of i_a s_a (0 <= i_a < n_a, s_a >= 0) in (lo, hi)?  Dimensions are taken with the
// largest stride first, where only the i_a that leave the interval in reach of the rest are followed:
// one or two per dimension in layouts whose dimensions lie inside one another, as all dense ones and
// slices of them do.  What is not decided in kRowSteps steps counts as found.
struct RowDim {
  Wide n, s;
};
constexpr int kRowSteps = 1 << 12;

bool sum_within(Wide r, const RowDim *dim, int dims, Wide lo, Wide hi, int *steps) {
  if (++*steps > kRowSteps) return true;
  if (dims == 0) return r > lo && r < hi;
  Wide rest = 0;
  for (int a = 1; a < dims; ++a) rest += (dim[a].n - 1) * dim[a].s;
  auto floor_div = [](Wide a, Wide b) { return a / b - (a % b < 0); };
  const Wide s = dim[0].s;
  const Wide first = std::max<Wide>(0, floor_div(lo - rest - r, s) + 1);
  const Wide last = std::min<Wide>(dim[0].n - 1, floor_div(hi - 1 - r, s));
  for (Wide i = first; i <= last; ++i)
    if (sum_within(r + i * s, dim + 1, dims - 1, lo, hi, steps)) return true;
  return false;
}

// The same with strides of any sign, in any order.
bool any_sum_within(Wide r, const RowDim *in, int count, Wide lo, Wide hi) {
  RowDim dim[6];
  int dims = 0;
  for (int a = 0; a < count; ++a) {
    RowDim x = in[a];
    if (x.s < 0) {  // counted from its other end
      r += (x.n - 1) * x.s;
      x.s = -x.s;
    }
    if (x.n <= 1 || x.s == 0) continue;
    int b = 0;
    while (b < dims && dim[b].s != x.s) ++b;
    if (b < dims) dim[b].n += x.n - 1;  // two indices of one stride are one
    else dim[dims++] = x;
  }
  std::sort(dim, dim + dims, [](const RowDim &a, const RowDim &b) { return a.s > b.s; });
  int steps = 0;
  return sum_within(r, dim, dims, lo, hi, &steps);
}

// Does a row of x share a byte with a row of y?
bool rows_meet(const Rows &x, const Rows &y) {
  const Wide r = static_cast<Wide>(reinterpret_cast<uintptr_t>(x.p)) - static_cast<Wide>(reinterpret_cast<uintptr_t>(y.p));
  Wide lo = r, hi = r;  // of all differences: most tensors lie apart as a whole
  for (int a = 0; a < 3; ++a) {
    const Wide u = (x.n[a] - 1) * x.s[a], v = (y.n[a] - 1) * y.s[a];
    (u < 0 ? lo : hi) += u;
    (v < 0 ? hi : lo) -= v;
  }
  if (hi <= -x.bytes || lo >= y.bytes) return false;
  RowDim dim[6];
  for (int a = 0; a < 3; ++a) {
    dim[a] = RowDim{x.n[a], x.s[a]};
    dim[3 + a] = RowDim{y.n[a], -y.s[a]};
  }
  return any_sum_within(r, dim, 6, -static_cast<Wide>(x.bytes), y.bytes);
}

// Do two different rows of x share a byte?  The first index in which they differ is the larger one's.
bool rows_meet_themselves(const Rows &x) {
  // dimensions that lie inside one another, smallest stride first: no
  Wide size[3], reach = x.bytes;
  int order[3] = {0, 1, 2};
  for (int a = 0; a < 3; ++a) size[a] = x.n[a] < 2 ? 0 : x.s[a] < 0 ? -x.s[a] : x.s[a];
  if (size[order[0]] > size[order[1]]) std::swap(order[0], order[1]);
  if (size[order[1]] > size[order[2]]) std::swap(order[1], order[2]);
  if (size[order[0]] > size[order[1]]) std::swap(order[0], order[1]);
  bool inside = true;
  for (int a : order) {
    if (x.n[a] < 2) continue;
    inside = inside && size[a] >= reach;
    reach += (x.n[a] - 1) * size[a];
  }
  if (inside) return false;
  for (int a = 0; a < 3; ++a) {
    RowDim dim[3];
    Wide r = x.s[a];
    dim[0] = RowDim{static_cast<Wide>(x.n[a]) - 1, x.s[a]};
    if (x.n[a] < 2) continue;
    for (int b = a + 1; b < 3; ++b) {
      r -= (static_cast<Wide>(x.n[b]) - 1) * x.s[b];
      dim[b - a] = RowDim{2 * static_cast<Wide>(x.n[b]) - 1, x.s[b]};
    }
    if (any_sum_within(r, dim, 3 - a, -static_cast<Wide>(x.bytes), x.bytes)) return true;
  }
  return false;
}

// How the heads of a token are split over threads: not at all where the tokens alone give every SM
// kRopeWarps warps, else into as many groups as that takes, down to one head each (a decode step).
// (8191 tokens written as int8 and read back, 48 heads of 128: 45 us with 6 or 12 warps, 47 with 24, 49
// with 48: more threads make the same angles again.  8198 tokens of fp32 gradients, 40 heads of 64: 41 us
// with 6, 31 from 12 on: fewer leave SMs short of loads in flight.)
constexpr int kRopeWarps = 12;

unsigned rope_split(long long tokens, int heads, int d, int num_sms, int *groups, int *per_group) {
  const long long warps = std::max(1LL, tokens * (d / 16) / 32);
  long long g = std::min<long long>(heads, (static_cast<long long>(kRopeWarps) * num_sms + warps - 1) / warps);
  *per_group = static_cast<int>((heads + g - 1) / g);
  *groups = (heads + *per_group - 1) / *per_group;
  return static_cast<unsigned>((tokens * (d / 16) * *groups + fa::kRopeThreads - 1) / fa::kRopeThreads);
}

template <int HD>
cudaError_t launch_rope(const fa::RopeParams &p, int in_f32, int out_f32, unsigned grid, cudaStream_t s) {
  using bf = __nv_bfloat16;
  if (in_f32 && out_f32) fa::fa_rope_kernel<HD, float, float><<<grid, fa::kRopeThreads, 0, s>>>(p);
  else if (in_f32) fa::fa_rope_kernel<HD, float, bf><<<grid, fa::kRopeThreads, 0, s>>>(p);
  else if (out_f32) fa::fa_rope_kernel<HD, bf, float><<<grid, fa::kRopeThreads, 0, s>>>(p);
  else fa::fa_rope_kernel<HD, bf, bf><<<grid, fa::kRopeThreads, 0, s>>>(p);
  return cudaGetLastError();
}

template <int HD>
cudaError_t launch_append(const fa::AppendParams &p, fa_cache_type type, unsigned grid, cudaStream_t s) {
  if (type == FA_CACHE_BF16) fa::fa_cache_append_kernel<HD, fa::kCacheBf16><<<grid, fa::kRopeThreads, 0, s>>>(p);
  else if (type == FA_CACHE_E4M3) fa::fa_cache_append_kernel<HD, fa::kCacheE4m3><<<grid, fa::kRopeThreads, 0, s>>>(p);
  else fa::fa_cache_append_kernel<HD, fa::kCacheInt8><<<grid, fa::kRopeThreads, 0, s>>>(p);
  return cudaGetLastError();
}

template <int HD>
cudaError_t launch_read(const fa::ReadParams &p, fa_cache_type type, unsigned grid, cudaStream_t s) {
  if (type == FA_CACHE_BF16) fa::fa_cache_read_kernel<HD, fa::kCacheBf16><<<grid, fa::kRopeThreads, 0, s>>>(p);
  else if (type == FA_CACHE_E4M3) fa::fa_cache_read_kernel<HD, fa::kCacheE4m3><<<grid, fa::kRopeThreads, 0, s>>>(p);
  else fa::fa_cache_read_kernel<HD, fa::kCacheInt8><<<grid, fa::kRopeThreads, 0, s>>>(p);
  return cudaGetLastError();
}

bool valid_cache(fa_cache_type t) { return t == FA_CACHE_BF16 || t == FA_CACHE_E4M3 || t == FA_CACHE_INT8; }

// The pool's sides shared by the writer and the reader: pointers, scales (8-bit types only), sizes.
fa_status check_pool(const void *k_pool, const void *v_pool, const float *k_scale, const float *v_scale,
                     fa_cache_type type, int num_blocks, int Hk, int d) {
  if (!valid_cache(type) || !k_pool || !v_pool) return FA_ERR_INVALID_ARG;
  if (type != FA_CACHE_BF16 && (!k_scale || !v_scale)) return FA_ERR_INVALID_ARG;
  if (num_blocks < 1 || Hk < 1) return FA_ERR_INVALID_ARG;
  if (d != 64 && d != 128) return FA_ERR_UNSUPPORTED;
  // pages of one head are numbered block * Hk + head in an int
  if ((static_cast<long long>(num_blocks) + 1) * Hk > INT_MAX) return FA_ERR_INVALID_ARG;
  if (!aligned16(k_pool) || !aligned16(v_pool) || !aligned16(k_scale) || !aligned16(v_scale))
    return FA_ERR_ALIGNMENT;
  return FA_OK;
}

// 8-bit pool [num_blocks, Hk, 16, d] as pages of one head, 16 x d bytes each, swizzled so that the
// lanes' 16-byte reads of a page spread over the banks (128-byte rows at d = 128, 64 at d = 64).
bool encode_pool_q8(CUtensorMap *map, const void *base, int d, long long pages) {
  auto enc = tensor_map_encoder();
  if (!enc) return false;
  cuuint64_t dims[3] = {static_cast<cuuint64_t>(d), 16, static_cast<cuuint64_t>(pages)};
  cuuint64_t strides[2] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(d) * 16};
  cuuint32_t box[3] = {static_cast<cuuint32_t>(d), 16, 1};
  cuuint32_t estr[3] = {1, 1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void *>(base), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE,
             d == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// How a call's rows and context are cut.  It depends on the arguments alone, so that the workspace
// can be sized before the call.
struct Q8Plan {
  int R;            // rows of one key head: group * Lq
  bool tile;        // many rows: the tcgen05 kernel
  int nt;           // row tiles of a CTA, 1 or 2 (of 8 rows, or of 128)
  int row_tiles, n_split, split_pages;
  size_t rows;      // S * Hq * Lq
};

// Up to kQ8StreamRows rows fa_q8_stream_kernel, beyond it fa_q8_tile_kernel.  32 sequences of 2048
// tokens, 8 heads of 128: 16 rows per head take the former 58 us and the latter 91; 17 rows 87 and 91;
// 32 rows 89 and 91; 64 rows 140 and 92.  One such sequence: 32 rows 22 and 28, 64 rows 26 and 28.
constexpr int kQ8StreamRows = 32;
// Few rows: chunks enough for two waves of the four CTAs that fit an SM, none longer than 128 pages (so
// that ragged lengths balance: 64 sequences of 512 to 8192 tokens took 397 us in two chunks each and
// 383 in four) and none shorter than 32 (eight to a warp; 4 sequences of 2048 tokens took 18 us at
// least 16 or 32 long and 23 at 64, 8 of 4096 took 31, 27 and 29).
constexpr int kQ8TargetCtas = 148 * 4 * 2;
constexpr int kQ8MinPages = 32, kQ8MaxPages = 128;
// Many rows: chunks only as far as one CTA per SM goes (64 units of 4096 tokens took 111 us in three chunks
// each, more than one round of CTAs, and 79 in two), two token tiles each at least (one sequence of 2048
// tokens, 64 rows per head: 25 us at least one or two long, 27 at four, 31 at eight).
constexpr int kQ8TileTargetCtas = 148;
constexpr int kQ8TileMinPages = 8;
// How the chunks are joined: with a CTA to each row while one round of CTAs covers the rows (128 rows of
// 4 chunks: a call of 18 us, 20 with HD / 4 threads to a row), and always past four chunks (there
// the threads of a row would wait for one chunk after the other).  With more rows of few chunks the CTAs
// come in rounds: 16384 rows of 2 chunks took 104 us that way, 78 with HD / 4 threads to a row.
constexpr int kQ8WideSplit = 4;
constexpr size_t kQ8WideRows = 148 * 8;

bool q8_plan(int S, int Hq, int Hk, int Lq, int d, int max_blocks, Q8Plan *out) {
  if (S < 1 || Hq < 1 || Hk < 1 || Hq % Hk != 0 || Lq < 1 || max_blocks < 1) return false;
  if (d != 64 && d != 128) return false;
  if (static_cast<long long>(S) * Hq * Lq > INT_MAX / 4) return false;
  // token numbers, up to a tile past the last, are ints
  if (static_cast<long long>(max_blocks) * fa::kQ8Page > INT_MAX - 2 * fa::kQ8Tok) return false;
  Q8Plan p{};
  p.R = Hq / Hk * Lq;
  p.tile = p.R > kQ8StreamRows;
  const int tile_rows = p.tile ? 128 : 8;
  p.nt = p.R > tile_rows ? 2 : 1;
  p.row_tiles = (p.R + tile_rows * p.nt - 1) / (tile_rows * p.nt);
  const long long units = static_cast<long long>(S) * Hk * p.row_tiles;
  const int target = p.tile ? kQ8TileTargetCtas : kQ8TargetCtas, least = p.tile ? kQ8TileMinPages : kQ8MinPages;
  long long n = p.tile ? std::max(1LL, target / units) : (target + units - 1) / units;
  if (!p.tile) n = std::max<long long>(n, (max_blocks + kQ8MaxPages - 1) / kQ8MaxPages);
  n = std::min<long long>({n, (max_blocks + least - 1) / least, fa::kQ8MaxSplit});
  p.split_pages = static_cast<int>((max_blocks + n - 1) / n);
  if (p.tile) p.split_pages = (p.split_pages + fa::kQ8TilePages - 1) / fa::kQ8TilePages * fa::kQ8TilePages;
  p.n_split = (max_blocks + p.split_pages - 1) / p.split_pages;
  p.rows = static_cast<size_t>(S) * Hq * Lq;
  if (units * p.n_split > INT_MAX) return false;
  *out = p;
  return true;
}

size_t q8_workspace(const Q8Plan &p, int d) {
  return p.n_split > 1 ? p.rows * p.n_split * (d + 2) * sizeof(float) : 0;
}

// After the kernel that wrote the chunks' partials: joins them where there are several.
template <int HD>
fa_status q8_combine(const fa::Q8Params &p, cudaStream_t s) {
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return launch_failed(e);
  if (p.n_split > 1) {
    const size_t rows = static_cast<size_t>(p.S) * p.Hk * p.R;
    if (p.n_split > kQ8WideSplit || rows <= kQ8WideRows)
      fa::fa_q8_combine_kernel<HD, true><<<static_cast<unsigned>(rows), 256, 0, s>>>(p);
    else
      fa::fa_q8_combine_kernel<HD, false><<<static_cast<unsigned>((rows * (HD / 4) + 255) / 256), 256, 0, s>>>(p);
    if ((e = cudaGetLastError()) != cudaSuccess) return launch_failed(e);
  }
  return FA_OK;
}

template <int HD, int NT, int kType>
fa_status launch_q8_stream(DeviceInfo &dev, const CUtensorMap &tk, const CUtensorMap &tv,
                           const fa::Q8Params &p, cudaStream_t s) {
  using C = fa::Q8Cfg<HD>;
  const int slot = (HD == 128) * 4 + (NT == 2) * 2 + (kType == fa::kQ8Int8);
  {
    std::lock_guard<std::mutex> lock(g_mutex);
    if (!dev.q8_attr[slot]) {
      cudaError_t e = cudaFuncSetAttribute(fa::fa_q8_stream_kernel<HD, NT, kType>,
                                           cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
      if (e != cudaSuccess) return launch_failed(e);
      dev.q8_attr[slot] = true;
    }
  }
  const unsigned grid = static_cast<unsigned>(p.n_split) * p.row_tiles * p.Hk * p.S;
  fa::fa_q8_stream_kernel<HD, NT, kType><<<grid, fa::kQ8Threads, C::kSmem, s>>>(tk, tv, p);
  return q8_combine<HD>(p, s);
}

template <int HD, int kType, bool kTwo>
fa_status launch_q8_tile(DeviceInfo &dev, const fa::Q8Params &p, cudaStream_t s) {
  using C = fa::Q8TileCfg<HD>;
  const int slot = 8 + (HD == 128) * 4 + kTwo * 2 + (kType == fa::kQ8Int8);
  {
    std::lock_guard<std::mutex> lock(g_mutex);
    if (!dev.q8_attr[slot]) {
      cudaError_t e = cudaFuncSetAttribute(fa::fa_q8_tile_kernel<HD, kType, kTwo>,
                                           cudaFuncAttributeMaxDynamicSharedMemorySize,
                                           static_cast<int>(C::kSmem));
      if (e != cudaSuccess) return launch_failed(e);
      dev.q8_attr[slot] = true;
    }
  }
  const unsigned grid = static_cast<unsigned>(p.n_split) * p.row_tiles * p.Hk * p.S;
  fa::fa_q8_tile_kernel<HD, kType, kTwo><<<grid, fa::kQ8TileThreads, C::kSmem, s>>>(p);
  return q8_combine<HD>(p, s);
}

template <int HD, int kType>
fa_status launch_q8(DeviceInfo &dev, const void *k_pool, const void *v_pool, const fa::Q8Params &p,
                    const Q8Plan &plan, cudaStream_t s) {
  if (plan.tile)
    return plan.nt == 2 ? launch_q8_tile<HD, kType, true>(dev, p, s)
                        : launch_q8_tile<HD, kType, false>(dev, p, s);
  CUtensorMap tk, tv;
  const long long pages = static_cast<long long>(p.num_blocks) * p.Hk;
  if (!encode_pool_q8(&tk, k_pool, HD, pages) || !encode_pool_q8(&tv, v_pool, HD, pages)) {
    t_last_error = "cuTensorMapEncodeTiled failed";
    return FA_ERR_LAUNCH;
  }
  return plan.nt == 2 ? launch_q8_stream<HD, 2, kType>(dev, tk, tv, p, s)
                      : launch_q8_stream<HD, 1, kType>(dev, tk, tv, p, s);
}

fa_status q8_attention(const void *q, const void *k_pool, const void *v_pool, const float *k_scale,
                       const float *v_scale, fa_cache_type type, const int32_t *block_table,
                       int max_blocks_per_seq, const int32_t *seq_lens, int num_blocks,
                       const uint64_t *tree_mask, void *o, fa_out_dtype o_dtype, float *lse, int S,
                       int Hq, int Hk, int Lq, int d, int causal, float scale, void *workspace,
                       size_t workspace_bytes, fa_stream_t stream) {
  if (!q || !block_table || !seq_lens || !o) return FA_ERR_INVALID_ARG;
  if (S < 1 || Hq < 1 || Lq < 1 || max_blocks_per_seq < 1) return FA_ERR_INVALID_ARG;
  if (causal != 0 && causal != 1) return FA_ERR_INVALID_ARG;
  if (o_dtype != FA_OUT_BF16 && o_dtype != FA_OUT_F32) return FA_ERR_INVALID_ARG;
  if (type != FA_CACHE_E4M3 && type != FA_CACHE_INT8) return FA_ERR_INVALID_ARG;
  fa_status st = check_pool(k_pool, v_pool, k_scale, v_scale, type, num_blocks, Hk, d);
  if (st != FA_OK) return st;
  if (Lq > static_cast<long long>(max_blocks_per_seq) * fa::kQ8Page) return FA_ERR_INVALID_ARG;
  Q8Plan plan;
  if (!q8_plan(S, Hq, Hk, Lq, d, max_blocks_per_seq, &plan)) return FA_ERR_INVALID_ARG;
  float sc;
  if (!resolve_scale(scale, d, &sc)) return FA_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(o)) return FA_ERR_ALIGNMENT;
  if (!aligned(block_table, 4) || !aligned(seq_lens, 4) || !aligned(lse, 4) || !aligned(tree_mask, 8))
    return FA_ERR_ALIGNMENT;
  const size_t need = q8_workspace(plan, d);
  if (need > 0 && (!workspace || workspace_bytes < need)) return FA_ERR_WORKSPACE;
  if (!aligned16(workspace)) return FA_ERR_ALIGNMENT;
  // nothing that is written may overlap anything that is read, or another output
  const size_t o_bytes = plan.rows * d * (o_dtype == FA_OUT_F32 ? 4 : 2);
  const size_t tokens = static_cast<size_t>(num_blocks) * Hk * fa::kQ8Page;
  const void *ins[8] = {q, k_pool, v_pool, k_scale, v_scale, block_table, seq_lens, tree_mask};
  const size_t in_bytes[8] = {plan.rows * d * 2, tokens * d, tokens * d, tokens * 4, tokens * 4,
                              static_cast<size_t>(S) * max_blocks_per_seq * 4, static_cast<size_t>(S) * 4,
                              tree_mask ? static_cast<size_t>(S) * Lq * 8 : 0};
  const void *outs[3] = {o, lse, workspace};
  const size_t out_bytes[3] = {o_bytes, lse ? plan.rows * 4 : 0, need};
  for (int a = 0; a < 3; ++a) {
    if (out_bytes[a] == 0) continue;
    for (int b = 0; b < 8; ++b)
      if (in_bytes[b] && overlaps(outs[a], out_bytes[a], ins[b], in_bytes[b])) return FA_ERR_INVALID_ARG;
    for (int b = a + 1; b < 3; ++b)
      if (out_bytes[b] && overlaps(outs[a], out_bytes[a], outs[b], out_bytes[b])) return FA_ERR_INVALID_ARG;
  }
  DeviceInfo *dev = nullptr;
  int dev_id = 0;
  if ((st = current_device(&dev, &dev_id)) != FA_OK) return st;
  fa::Q8Params p{};
  p.q = static_cast<const uint16_t *>(q);
  p.k_codes = static_cast<const uint8_t *>(k_pool);
  p.v_codes = static_cast<const uint8_t *>(v_pool);
  p.ks = k_scale;
  p.vs = v_scale;
  p.table = block_table;
  p.lens = seq_lens;
  p.tree = tree_mask;
  p.o = o;
  p.lse = lse;
  p.ws_o = static_cast<float *>(workspace);
  p.ws_ml = reinterpret_cast<float2 *>(static_cast<float *>(workspace) + plan.rows * plan.n_split * d);
  p.S = S;
  p.Hq = Hq;
  p.Hk = Hk;
  p.T = Lq;
  p.R = plan.R;
  p.max_blocks = max_blocks_per_seq;
  p.num_blocks = num_blocks;
  p.row_tiles = plan.row_tiles;
  p.n_split = plan.n_split;
  p.split_pages = plan.split_pages;
  p.causal = causal;
  p.longest_first = plan.tile && S > 1 && S <= fa::kQ8SortSeqs &&
                    static_cast<long long>(S) * Hk * plan.row_tiles * plan.n_split > dev->num_sms;
  p.o_f32 = o_dtype == FA_OUT_F32;
  p.scale_log2 = sc * 1.4426950408889634f;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (type == FA_CACHE_E4M3)
    return d == 128 ? launch_q8<128, fa::kQ8E4m3>(*dev, k_pool, v_pool, p, plan, s)
                    : launch_q8<64, fa::kQ8E4m3>(*dev, k_pool, v_pool, p, plan, s);
  return d == 128 ? launch_q8<128, fa::kQ8Int8>(*dev, k_pool, v_pool, p, plan, s)
                  : launch_q8<64, fa::kQ8Int8>(*dev, k_pool, v_pool, p, plan, s);
}

}  // namespace

extern "C" {

fa_status fa_rope(const void *q, const long long *q_strides, void *q_out,
                  const long long *q_out_strides, const void *k, const long long *k_strides,
                  void *k_out, const long long *k_out_strides, fa_out_dtype in_dtype,
                  fa_out_dtype out_dtype, const int32_t *positions, long long pos_stride,
                  const double *freqs, int rot, fa_rope_layout layout, float amplitude, int inverse,
                  int B, int Hq, int Hk, int N, int d, fa_stream_t stream) {
  if (B < 0 || N < 0 || Hq < 1 || Hk < 0) return FA_ERR_INVALID_ARG;
  if (in_dtype != FA_OUT_BF16 && in_dtype != FA_OUT_F32) return FA_ERR_INVALID_ARG;
  if (out_dtype != FA_OUT_BF16 && out_dtype != FA_OUT_F32) return FA_ERR_INVALID_ARG;
  if (d != 64 && d != 128) return FA_ERR_UNSUPPORTED;
  if (B == 0 || N == 0) return FA_OK;
  fa::RopeParams p{};
  const void *in[2] = {q, k};
  void *out[2] = {q_out, k_out};
  const long long *is[2] = {q_strides, k_strides}, *os[2] = {q_out_strides, k_out_strides};
  const int heads[2] = {Hq, Hk};
  const int in_unit = in_dtype == FA_OUT_F32 ? 4 : 8, out_unit = out_dtype == FA_OUT_F32 ? 4 : 8;
  const long long extent[3] = {B, 0, N};
  for (int i = 0; i < 2; ++i) {
    if (heads[i] == 0) continue;
    if (!in[i] || !out[i] || !is[i] || !os[i]) return FA_ERR_INVALID_ARG;
    if (!aligned16(in[i]) || !aligned16(out[i])) return FA_ERR_ALIGNMENT;
    // in place is the same tensor: a row written elsewhere or wider than it was read meets others
    if (in[i] == out[i]) {
      if (in_dtype != out_dtype) return FA_ERR_INVALID_ARG;
      for (int a = 0; a < 3; ++a)
        if ((a == 1 ? heads[i] : extent[a]) > 1 && is[i][a] != os[i][a]) return FA_ERR_INVALID_ARG;
    }
    p.x[i].in = in[i];
    p.x[i].out = out[i];
    p.x[i].H = heads[i];
    for (int a = 0; a < 3; ++a) {
      if ((a == 1 ? heads[i] : extent[a]) == 1) continue;  // its stride means nothing
      if (is[i][a] % in_unit || os[i][a] % out_unit) return FA_ERR_ALIGNMENT;
      p.x[i].in_s[a] = is[i][a];
      p.x[i].out_s[a] = os[i][a];
    }
  }
  // what is written lies neither on itself nor on anything read (but the same tensor in place) or written
  auto rows_of = [&](const void *x, const long long *strides, int i, fa_out_dtype type) {
    const long long e = type == FA_OUT_F32 ? 4 : 2;
    Rows r{x, d * e, {B, heads[i], N}, {}};
    for (int a = 0; a < 3; ++a) r.s[a] = (a == 1 ? heads[i] : extent[a]) > 1 ? static_cast<Wide>(strides[a]) * e : 0;
    return r;
  };
  for (int i = 0; i < 2; ++i) {
    if (heads[i] == 0) continue;
    const Rows y = rows_of(out[i], os[i], i, out_dtype);
    if (rows_meet_themselves(y)) return FA_ERR_INVALID_ARG;
    for (int j = 0; j < 2; ++j) {
      if (heads[j] == 0) continue;
      if (!(i == j && in[i] == out[i]) && rows_meet(y, rows_of(in[j], is[j], j, in_dtype))) return FA_ERR_INVALID_ARG;
      if (j > i && rows_meet(y, rows_of(out[j], os[j], j, out_dtype))) return FA_ERR_INVALID_ARG;
    }
    if (rot > 0 && rows_meet(y, Rows{positions, 4LL * N, {B, 1, 1}, {4 * static_cast<Wide>(pos_stride), 0, 0}})) return FA_ERR_INVALID_ARG;
    if (rot > 0 && rows_meet(y, Rows{freqs, 4LL * rot, {1, 1, 1}, {}})) return FA_ERR_INVALID_ARG;
  }
  fa_status st = check_rope(positions, freqs, rot, layout, amplitude, d, inverse, &p.table);
  if (st != FA_OK) return st;
  p.positions = positions;
  p.pos_stride = pos_stride;
  p.N = N;
  const long long tokens = static_cast<long long>(B) * N;
  // threads are counted in blocks of an unsigned grid
  if (tokens > INT_MAX || static_cast<long long>(Hq) + Hk > INT_MAX) return FA_ERR_INVALID_ARG;
  p.tokens = static_cast<unsigned>(tokens);
  DeviceInfo *dev = nullptr;
  int dev_id = 0;
  if ((st = current_device(&dev, &dev_id)) != FA_OK) return st;
  const unsigned grid = rope_split(tokens, Hq + Hk, d, dev->num_sms, &p.groups, &p.heads_per_group);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const int inf = in_dtype == FA_OUT_F32, outf = out_dtype == FA_OUT_F32;
  cudaError_t e = d == 128 ? launch_rope<128>(p, inf, outf, grid, s) : launch_rope<64>(p, inf, outf, grid, s);
  return e == cudaSuccess ? FA_OK : launch_failed(e);
}

fa_status fa_cache_append(const void *k, const long long *k_strides, const void *v,
                          const long long *v_strides, void *k_pool, void *v_pool, float *k_scale,
                          float *v_scale, fa_cache_type type, const int64_t *slots, int num_blocks,
                          const void *q, const long long *q_strides, void *q_out,
                          const long long *q_out_strides, const int32_t *positions,
                          const double *freqs, int rot, fa_rope_layout layout, float amplitude,
                          int T, int Hq, int Hk, int d, fa_stream_t stream) {
  if (T < 0 || Hq < 0) return FA_ERR_INVALID_ARG;
  fa_status st = check_pool(k_pool, v_pool, k_scale, v_scale, type, num_blocks, Hk, d);
  if (st != FA_OK) return st;
  fa::AppendParams p{};
  st = check_rope(positions, freqs, rot, layout, amplitude, d, 0, &p.table);
  if (T == 0) return FA_OK;
  if (st != FA_OK) return st;
  if (!k || !v || !slots || !k_strides || !v_strides) return FA_ERR_INVALID_ARG;
  if (Hq > 0 && (!q || !q_out || !q_strides || !q_out_strides)) return FA_ERR_INVALID_ARG;
  if (static_cast<long long>(Hq) + 2LL * Hk > INT_MAX) return FA_ERR_INVALID_ARG;
  if (!aligned16(k) || !aligned16(v) || !aligned(slots, 8)) return FA_ERR_ALIGNMENT;
  if (Hq > 0 && (!aligned16(q) || !aligned16(q_out))) return FA_ERR_ALIGNMENT;
  const long long *strides[4] = {k_strides, v_strides, q_strides, q_out_strides};
  long long *to[4] = {p.k_s, p.v_s, p.q_s, p.qo_s};
  for (int i = 0; i < (Hq > 0 ? 4 : 2); ++i)
    for (int a = 0; a < 2; ++a) {
      if ((a == 0 ? T : i < 2 ? Hk : Hq) == 1) continue;  // its stride means nothing
      if (strides[i][a] % 8) return FA_ERR_ALIGNMENT;
      to[i][a] = strides[i][a];
    }
  p.q = static_cast<const uint16_t *>(q);
  p.k = static_cast<const uint16_t *>(k);
  p.v = static_cast<const uint16_t *>(v);
  p.q_out = static_cast<uint16_t *>(q_out);
  p.k_pool = k_pool;
  p.v_pool = v_pool;
  p.k_scale = k_scale;
  p.v_scale = v_scale;
  p.slots = slots;
  p.positions = positions;
  p.T = T;
  p.Hq = Hq;
  p.Hk = Hk;
  p.num_slots = static_cast<long long>(num_blocks) * fa::kCachePage;
  if (Hq > 0 && q == q_out)  // in place is the same tensor
    for (int a = 0; a < 2; ++a)
      if ((a == 0 ? T : Hq) > 1 && q_strides[a] != q_out_strides[a]) return FA_ERR_INVALID_ARG;
  // q_out is written: like fa_rope's outputs it lies neither on itself nor on anything read, but for q
  // in place
  auto rows_of = [&](const void *x, const long long *st, int heads) {
    return Rows{x, 2LL * d, {T, heads, 1}, {T > 1 ? 2 * static_cast<Wide>(st[0]) : 0,
                                            heads > 1 ? 2 * static_cast<Wide>(st[1]) : 0, 0}};
  };
  if (Hq > 0) {
    const Rows y = rows_of(q_out, q_out_strides, Hq);
    if (rows_meet_themselves(y) || rows_meet(y, rows_of(k, k_strides, Hk)) || rows_meet(y, rows_of(v, v_strides, Hk)))
      return FA_ERR_INVALID_ARG;
    if (q != q_out && rows_meet(y, rows_of(q, q_strides, Hq))) return FA_ERR_INVALID_ARG;
    if (rows_meet(y, Rows{slots, 8LL * T, {1, 1, 1}, {}})) return FA_ERR_INVALID_ARG;
    if (rot > 0 && (rows_meet(y, Rows{positions, 4LL * T, {1, 1, 1}, {}}) ||
                    rows_meet(y, Rows{freqs, 4LL * rot, {1, 1, 1}, {}})))
      return FA_ERR_INVALID_ARG;
  }
  // the pools and scales are written: they may lie neither on one another nor on what is read or
  // written beside them (a strided tensor counts from its first to its last element)
  const size_t rows = static_cast<size_t>(num_blocks) * Hk * fa::kCachePage;
  const size_t pool_bytes = rows * d * (type == FA_CACHE_BF16 ? 2 : 1);
  const size_t scale_bytes = type == FA_CACHE_BF16 ? 0 : rows * 4;
  const void *outs[4] = {k_pool, v_pool, k_scale, v_scale};
  const size_t out_bytes[4] = {pool_bytes, pool_bytes, scale_bytes, scale_bytes};
  const Span kx = row_span(k, k_strides, T, Hk, d), vx = row_span(v, v_strides, T, Hk, d);
  const Span qx = Hq > 0 ? row_span(q, q_strides, T, Hq, d) : Span{nullptr, 0};
  const Span qox = Hq > 0 ? row_span(q_out, q_out_strides, T, Hq, d) : Span{nullptr, 0};
  const void *ins[7] = {slots, positions, freqs, kx.p, vx.p, qx.p, qox.p};
  const size_t in_bytes[7] = {static_cast<size_t>(T) * 8, rot ? static_cast<size_t>(T) * 4 : 0,
                              static_cast<size_t>(rot) * 4, kx.bytes, vx.bytes, qx.bytes, qox.bytes};
  for (int a = 0; a < 4; ++a) {
    if (out_bytes[a] == 0) continue;
    for (int b = 0; b < 7; ++b)
      if (in_bytes[b] && overlaps(outs[a], out_bytes[a], ins[b], in_bytes[b])) return FA_ERR_INVALID_ARG;
    for (int b = a + 1; b < 4; ++b)
      if (out_bytes[b] && overlaps(outs[a], out_bytes[a], outs[b], out_bytes[b])) return FA_ERR_INVALID_ARG;
  }
  DeviceInfo *dev = nullptr;
  int dev_id = 0;
  if ((st = current_device(&dev, &dev_id)) != FA_OK) return st;
  const unsigned grid = rope_split(T, Hq + 2 * Hk, d, dev->num_sms, &p.groups, &p.heads_per_group);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e = d == 128 ? launch_append<128>(p, type, grid, s) : launch_append<64>(p, type, grid, s);
  return e == cudaSuccess ? FA_OK : launch_failed(e);
}

fa_status fa_cache_read(const void *k_pool, const void *v_pool, const float *k_scale,
                        const float *v_scale, fa_cache_type type, const int64_t *slots,
                        int num_blocks, void *k, void *v, int T, int H, int d, fa_stream_t stream) {
  if (T < 0) return FA_ERR_INVALID_ARG;
  fa_status st = check_pool(k_pool, v_pool, k_scale, v_scale, type, num_blocks, H, d);
  if (st != FA_OK) return st;
  if (T == 0) return FA_OK;
  if (!slots || !k || !v) return FA_ERR_INVALID_ARG;
  if (!aligned16(k) || !aligned16(v) || !aligned(slots, 8)) return FA_ERR_ALIGNMENT;
  fa::ReadParams p{};
  p.k_pool = k_pool;
  p.v_pool = v_pool;
  p.k_scale = k_scale;
  p.v_scale = v_scale;
  p.slots = slots;
  p.k = static_cast<uint16_t *>(k);
  p.v = static_cast<uint16_t *>(v);
  p.T = T;
  p.H = H;
  p.num_slots = static_cast<long long>(num_blocks) * fa::kCachePage;
  const size_t out_bytes = static_cast<size_t>(T) * H * d * 2;
  const size_t rows = static_cast<size_t>(num_blocks) * H * fa::kCachePage;
  const size_t pool_bytes = rows * d * (type == FA_CACHE_BF16 ? 2 : 1);
  const void *ins[5] = {k_pool, v_pool, k_scale, v_scale, slots};
  const size_t scale_bytes = type == FA_CACHE_BF16 ? 0 : rows * 4;
  const size_t in_bytes[5] = {pool_bytes, pool_bytes, scale_bytes, scale_bytes, static_cast<size_t>(T) * 8};
  for (int b = 0; b < 5; ++b)
    if (in_bytes[b] && (overlaps(k, out_bytes, ins[b], in_bytes[b]) || overlaps(v, out_bytes, ins[b], in_bytes[b])))
      return FA_ERR_INVALID_ARG;
  if (overlaps(k, out_bytes, v, out_bytes)) return FA_ERR_INVALID_ARG;
  DeviceInfo *dev = nullptr;
  int dev_id = 0;
  if ((st = current_device(&dev, &dev_id)) != FA_OK) return st;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const unsigned grid = rope_split(T, 2 * H, d, dev->num_sms, &p.groups, &p.heads_per_group);
  cudaError_t e = d == 128 ? launch_read<128>(p, type, grid, s) : launch_read<64>(p, type, grid, s);
  return e == cudaSuccess ? FA_OK : launch_failed(e);
}

size_t fa_q8_workspace_size(int S, int Hq, int Hk, int Lq, int d, int max_blocks_per_seq) {
  Q8Plan plan;
  return q8_plan(S, Hq, Hk, Lq, d, max_blocks_per_seq, &plan) ? q8_workspace(plan, d) : 0;
}

fa_status fa_decode_paged_q8(const void *q, const void *k_pool, const void *v_pool,
                             const float *k_scale, const float *v_scale, fa_cache_type type,
                             const int32_t *block_table, int max_blocks_per_seq,
                             const int32_t *seq_lens, int num_blocks, void *o, fa_out_dtype o_dtype,
                             float *lse, int S, int Hq, int Hk, int d, float scale, void *workspace,
                             size_t workspace_bytes, fa_stream_t stream) {
  return q8_attention(q, k_pool, v_pool, k_scale, v_scale, type, block_table, max_blocks_per_seq,
                      seq_lens, num_blocks, nullptr, o, o_dtype, lse, S, Hq, Hk, 1, d, 0, scale,
                      workspace, workspace_bytes, stream);
}

fa_status fa_prefill_paged_q8(const void *q, const void *k_pool, const void *v_pool,
                              const float *k_scale, const float *v_scale, fa_cache_type type,
                              const int32_t *block_table, int max_blocks_per_seq,
                              const int32_t *seq_lens, int num_blocks, void *o,
                              fa_out_dtype o_dtype, float *lse, int S, int Hq, int Hk, int Lq, int d,
                              int causal, float scale, void *workspace, size_t workspace_bytes,
                              fa_stream_t stream) {
  return q8_attention(q, k_pool, v_pool, k_scale, v_scale, type, block_table, max_blocks_per_seq,
                      seq_lens, num_blocks, nullptr, o, o_dtype, lse, S, Hq, Hk, Lq, d, causal,
                      scale, workspace, workspace_bytes, stream);
}

fa_status fa_tree_attention_q8(const void *q, const void *k_pool, const void *v_pool,
                               const float *k_scale, const float *v_scale, fa_cache_type type,
                               const int32_t *block_table, int max_blocks_per_seq,
                               const int32_t *seq_lens, int num_blocks, const uint64_t *tree_mask,
                               void *o, fa_out_dtype o_dtype, float *lse, int S, int Hq, int Hk,
                               int T, int d, float scale, void *workspace, size_t workspace_bytes,
                               fa_stream_t stream) {
  if (!tree_mask || T < 1 || T > 64) return FA_ERR_INVALID_ARG;
  return q8_attention(q, k_pool, v_pool, k_scale, v_scale, type, block_table, max_blocks_per_seq,
                      seq_lens, num_blocks, tree_mask, o, o_dtype, lse, S, Hq, Hk, T, d, 0, scale,
                      workspace, workspace_bytes, stream);
}

}  // extern "C"
