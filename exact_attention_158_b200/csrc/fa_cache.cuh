// fa_cache.cuh -- writing new tokens' keys and values into the paged pool, and reading rows back.
//
// Paging: "LLM study notes" (devocean.sk.com), paged attention.  A token's slot is
// block * 16 + row in the pool [num_blocks, H, 16, d]; scales lie beside it as [num_blocks, H, 16].
//
// 8-bit rows carry one fp32 scale each (per token and head): scale = max|x| / qmax with qmax = 448
// (e4m3) or 127 (int8), code = the value nearest to x / scale, ties to even, and the row stands for
// code * scale.  scale and quotient are fp32 divisions rounded to nearest (bf16 inputs fall on the
// border between two codes too often for a reciprocal's last bit not to matter).  A row whose
// largest magnitude is below 2^-100 is stored as zeros with scale 0; a row that holds an infinity
// or a NaN is stored with scale NaN (and reads back as NaN, as a bf16 row would mostly do).
// Keys are rotated (fa_rope.cuh) and quantised from fp32, with no rounding to bf16 between.
//
// Bound: HBM (and launch latency for a decode step's few rows); everything is read and written once.
#pragma once
#include <cuda_fp8.h>

#include <type_traits>

#include "fa_rope.cuh"

namespace fa {

constexpr int kCachePage = 16;
enum CacheType { kCacheBf16 = 0, kCacheE4m3 = 1, kCacheInt8 = 2 };
constexpr float kCacheTiny = 0x1p-100f;

template <int kType>
__host__ __device__ constexpr float cache_qmax() { return kType == kCacheE4m3 ? 448.f : 127.f; }

struct AppendParams {
  // sources and the q output: [T, H, d] with element strides of token and head
  const uint16_t *q, *k, *v;
  uint16_t *q_out;
  long long q_s[2], k_s[2], v_s[2], qo_s[2];
  void *k_pool, *v_pool;
  float *k_scale, *v_scale;
  const int64_t *slots;
  const int32_t *positions;
  RopeTable table;
  int T, Hq, Hk;
  long long num_slots;
  int groups, heads_per_group;  // of the q, k and v heads, as in RopeParams
};

// x / s rounded to nearest, from r = 1 / s rounded to nearest: one residual step after the product
// (Markstein) gives the correctly rounded quotient; s is a normal number here and |x / s| <= qmax.
__device__ __forceinline__ float div_by_rcp(float x, float s, float r) {
  const float y = x * r;
  return fmaf(fmaf(-y, s, x), r, y);
}

template <int kType>
__device__ __forceinline__ uint32_t cache_code4(const float *f, float s, float r) {
  float y[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) y[i] = div_by_rcp(f[i], s, r);
  if constexpr (kType == kCacheE4m3) {
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(y[0], y[1]), __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(y[2], y[3]), __NV_SATFINITE, __NV_E4M3);
    return lo | (hi << 16);
  } else {
    // |y| <= 127 (1 + 2^-23): adding 1.5 * 2^23 leaves the nearest integer in the low bits, and no clamp
    // is needed (a conversion instruction runs at an eighth of the rate)
    uint32_t b[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) b[i] = __float_as_uint(y[i] + 12582912.f);
    return __byte_perm(__byte_perm(b[0], b[1], 0x0040), __byte_perm(b[2], b[3], 0x0040), 0x5410);
  }
}

__device__ __forceinline__ float max_nan(float a, float b) {  // NaN when either is one
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// Threads as in fa_rope_kernel: one per (head group, token, chunk), the heads of q, k and v counted in
// that order; HD / 16 threads a row, 16 features each, the row maximum by shuffles among them.
// Instructions, not bytes, bound the first form of this kernel (254 per four rows of a warp, 47 us for
// 8191 tokens x 48 heads of 128; 39 with the q, k and v rows walked in loops of their own).  Four rows are
// on their way (with two, written and read back: 52 us for 48).
template <int HD, int kType>
__global__ void __launch_bounds__(kRopeThreads) fa_cache_append_kernel(const AppendParams p) {
  constexpr int kChunks = HD / 16, kUnroll = 4;
  using bf = __nv_bfloat16;
  const unsigned long long gid = static_cast<unsigned long long>(blockIdx.x) * kRopeThreads + threadIdx.x;
  const int chunk = static_cast<int>(gid % kChunks);
  const unsigned long long rest = gid / kChunks;
  const unsigned group = static_cast<unsigned>(rest / static_cast<unsigned>(p.T));
  if (group >= static_cast<unsigned>(p.groups)) return;  // whole rows of threads
  const long long m = rest - static_cast<unsigned long long>(group) * p.T;
  const int first = group * p.heads_per_group;
  const int last = min(first + p.heads_per_group, p.Hq + 2 * p.Hk);
  const RopeCols<8> rcol = rope_cols<HD, 8>(p.table, chunk), vcol{{8 * chunk, HD / 2 + 8 * chunk}};
  long long slot = p.slots[m];
  if (slot >= p.num_slots) {  // caller broke the contract: report, write nothing for the token
    atomicExch(&g_device_status, 1 /* FA_ERR_INVALID_ARG */);
    slot = -1;
  }
  RopeTurn<8> turn;
  // rows [lo, hi) of one kind: four loads on their way ahead of `put`
  auto walk = [&](const uint16_t *src, long long step, int lo, int hi, const RopeCols<8> &col, auto put) {
    Raw16<bf> raw[kUnroll];
    if (lo >= hi) return;
    const bf *row = reinterpret_cast<const bf *>(src) + lo * step;
#pragma unroll
    for (int u = 0; u < kUnroll; ++u)
      if (lo + u < hi) raw_load(raw[u], row + u * step, col);
    for (int h0 = lo; h0 < hi; h0 += kUnroll) {
      row += kUnroll * step;
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        if (h0 + u >= hi) break;
        float f[16];
        raw_floats(raw[u], f);
        if (h0 + u + kUnroll < hi) raw_load(raw[u], row + u * step, col);
        put(h0 + u, f);
      }
    }
  };
  const unsigned mates = ((1u << kChunks) - 1u) << ((threadIdx.x & 31) / kChunks * kChunks);
  const long long row0 = slot < 0 ? 0 : slot / kCachePage * p.Hk * kCachePage + slot % kCachePage;
  auto store = [&](void *pool, float *scales, int h, const RopeCols<8> &col, const float (&f)[16]) {
    const long long row = row0 + static_cast<long long>(h) * kCachePage;
    if constexpr (kType == kCacheBf16) {
      store_pieces(static_cast<bf *>(pool) + row * HD, col, f);
    } else {
      float top = 0.f;  // NaN and infinities come through
#pragma unroll
      for (int e = 0; e < 16; ++e) top = max_nan(top, fabsf(f[e]));
#pragma unroll
      for (int off = kChunks / 2; off > 0; off >>= 1) top = max_nan(top, __shfl_xor_sync(mates, top, off));
      float scale = top >= kCacheTiny ? __fdiv_rn(top, cache_qmax<kType>()) : 0.f;
      float rcp = scale > 0.f ? __frcp_rn(scale) : 0.f;
      if (!(top < INFINITY)) scale = __int_as_float(0x7fc00000), rcp = 0.f;
      uint32_t w[4] = {0u, 0u, 0u, 0u};
      if (rcp > 0.f) {
#pragma unroll
        for (int e = 0; e < 4; ++e) w[e] = cache_code4<kType>(f + 4 * e, scale, rcp);
      }
      uint8_t *dst = static_cast<uint8_t *>(pool) + row * HD;
      *reinterpret_cast<uint2 *>(dst + col.col[0]) = make_uint2(w[0], w[1]);
      *reinterpret_cast<uint2 *>(dst + col.col[1]) = make_uint2(w[2], w[3]);
      if (chunk == 0) scales[row] = scale;
    }
  };
  // (a thread whose heads are all values needs no angles)
  turn.on[0] = turn.on[1] = false;
  if (first < p.Hq + p.Hk) rope_turn(p.table, p.positions + m, rcol, turn);
  walk(p.q + m * p.q_s[0], p.q_s[1], first, min(last, p.Hq), rcol, [&](int h, float (&f)[16]) {
    rope_apply(p.table, turn, f);
    store_pieces(reinterpret_cast<bf *>(p.q_out) + m * p.qo_s[0] + h * p.qo_s[1], rcol, f);
  });
  if (slot < 0) return;
  walk(p.k + m * p.k_s[0], p.k_s[1], max(first - p.Hq, 0), min(last - p.Hq, p.Hk), rcol, [&](int h, float (&f)[16]) {
    rope_apply(p.table, turn, f);
    store(p.k_pool, p.k_scale, h, rcol, f);
  });
  const int v0 = p.Hq + p.Hk;
  walk(p.v + m * p.v_s[0], p.v_s[1], max(first - v0, 0), min(last - v0, p.Hk), vcol,
       [&](int h, float (&f)[16]) { store(p.v_pool, p.v_scale, h, vcol, f); });
}

struct ReadParams {
  const void *k_pool, *v_pool;
  const float *k_scale, *v_scale;
  const int64_t *slots;
  uint16_t *k, *v;  // [T, H, d] contiguous
  int T, H;
  long long num_slots;
  int groups, heads_per_group;  // of the k and v heads, as in RopeParams
};

// Threads as in fa_rope_kernel: one per (head group, token, chunk: features 8 c.. and HD/2 + 8 c..), the
// heads of k and v counted in that order; four rows on their way at once.
template <int HD, int kType>
__global__ void __launch_bounds__(kRopeThreads) fa_cache_read_kernel(const ReadParams p) {
  constexpr int kChunks = HD / 16, kUnroll = 4;
  const unsigned long long gid = static_cast<unsigned long long>(blockIdx.x) * kRopeThreads + threadIdx.x;
  const int chunk = static_cast<int>(gid % kChunks);
  const unsigned long long rest = gid / kChunks;
  const unsigned group = static_cast<unsigned>(rest / static_cast<unsigned>(p.T));
  if (group >= static_cast<unsigned>(p.groups)) return;
  const long long m = rest - static_cast<unsigned long long>(group) * p.T;
  const int first = group * p.heads_per_group, last = min(first + p.heads_per_group, 2 * p.H);
  long long slot = p.slots[m];
  if (slot >= p.num_slots) {
    atomicExch(&g_device_status, 1 /* FA_ERR_INVALID_ARG */);
    slot = -1;
  }
  const long long row0 = slot < 0 ? 0 : slot / kCachePage * p.H * kCachePage + slot % kCachePage;
  using Piece = std::conditional_t<kType == kCacheBf16, uint4, uint2>;  // eight features
  struct Row { Piece c[2]; float scale; } row[kUnroll];
  constexpr int kSize = kType == kCacheBf16 ? 2 : 1;
  for (int h0 = first; h0 < last; h0 += kUnroll) {
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      if (h0 + u >= last || slot < 0) continue;
      const bool is_v = h0 + u >= p.H;
      const long long r = row0 + static_cast<long long>(h0 + u - (is_v ? p.H : 0)) * kCachePage;
      const uint8_t *pool = static_cast<const uint8_t *>(is_v ? p.v_pool : p.k_pool);
      const uint8_t *src = pool + (r * HD + 8 * chunk) * kSize;
      row[u].c[0] = *reinterpret_cast<const Piece *>(src);
      row[u].c[1] = *reinterpret_cast<const Piece *>(src + HD / 2 * kSize);
      if constexpr (kType != kCacheBf16) row[u].scale = (is_v ? p.v_scale : p.k_scale)[r];
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      if (h0 + u >= last) break;
      const bool is_v = h0 + u >= p.H;
      uint16_t *dst = (is_v ? p.v : p.k) + (m * p.H + h0 + u - (is_v ? p.H : 0)) * HD + 8 * chunk;
      uint4 o[2] = {make_uint4(0u, 0u, 0u, 0u), make_uint4(0u, 0u, 0u, 0u)};
      if (slot >= 0) {
        if constexpr (kType == kCacheBf16) {
          o[0] = row[u].c[0];
          o[1] = row[u].c[1];
        } else {
          const uint32_t w[4] = {row[u].c[0].x, row[u].c[0].y, row[u].c[1].x, row[u].c[1].y};
          uint32_t b[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            float x, y;
            if constexpr (kType == kCacheE4m3) {
              const __half2 f = __half2(__nv_cvt_fp8x2_to_halfraw2(
                  static_cast<__nv_fp8x2_storage_t>(w[i / 2] >> (16 * (i % 2))), __NV_E4M3));
              x = __low2float(f);
              y = __high2float(f);
            } else {
              x = static_cast<float>(static_cast<int8_t>(w[i / 2] >> (16 * (i % 2))));
              y = static_cast<float>(static_cast<int8_t>(w[i / 2] >> (16 * (i % 2) + 8)));
            }
            b[i] = pack_bf16x2(x * row[u].scale, y * row[u].scale);
          }
          o[0] = make_uint4(b[0], b[1], b[2], b[3]);
          o[1] = make_uint4(b[4], b[5], b[6], b[7]);
        }
      }
      *reinterpret_cast<uint4 *>(dst) = o[0];
      *reinterpret_cast<uint4 *>(dst + HD / 2) = o[1];
    }
  }
}

}  // namespace fa
