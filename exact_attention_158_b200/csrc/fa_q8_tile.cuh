// fa_q8_tile.cuh -- attention of many rows (a prompt chunk, a draft tree, large groups) over an 8-bit
// paged cache on the tcgen05 tensor cores.  The mathematics is that of fa_q8.cuh; only the values'
// scales sit elsewhere.
//
// One CTA takes up to 256 of the R rows of one (sequence, key head) and a range of its 128-token
// tiles.  Codes cannot feed a 16-bit product, so they are converted once per tile for all of the
// CTA's rows:
//   warps 0-3    one side: a thread holds a row (a TMEM lane).  Scores out of TMEM, p back over
//                them; one thread issues the side's products
//   warps 4-7    the other side
//   warps 8-11   codes: bulk copies into a staging slot, a tile ahead -> fp16 K and V tiles in the
//                swizzled layout the tensor core reads; the tile's key scales and its live tokens
// TMEM (512 columns): S0 [0,128)  S1 [128,256)  O0 [256,256+d)  O1 [256+d,256+2d).
// With more than 128 rows the sides hold two row tiles; with fewer they share one row tile and take
// the tiles of tokens in turn.  Either way one side's products run while the other's softmax does.
// An issuer needs no warp of its own, since its side waits for what it issues; a thirteenth warp
// would leave a thread 128 registers instead of 168.
//
// Scales.  A key's scale multiplies its column of scores in fp32, read from shared memory by every
// row: 32 broadcast 16-byte loads per row and tile, which cost the SM about half as much as the
// exponentials.  A value's scale is folded into V instead (a second set of such loads measured
// 5900 cycles per tile of tokens where this form takes QQQQ): V = code * f in fp16, f = vs 2^a / F
// with F a power of two no smaller than any vs so far; O is rescaled when F has to grow.  f and the
// product are rounded to fp16 (2^-11 each, like p).  V uses fp16 from its top (2^15) down and p from
// 2^6 to 2^15, so a token whose values are 2^20 times the others' and whose weight is 2^-20 takes
// nothing from either.  A value scale that is not finite would reach rows that do not see its token
// as 0 * NaN: V is 0 there, and rows that do see it are marked and written as NaN.
//
// A row's softmax is one pass: p = 2^(s ks - m) against the reference it has, summed and stored;
// where one passes 2^15, and on a row's first tile, the reference moves so that the largest p is 2^6, and
// O is rescaled in TMEM (as it is when F has grown).
//
// Queries go to fp16 against one power of two for all rows of the CTA (q8_q_unit; it is part of the key
// scales).  int8's conversion leaves every four features in the order 0, 2, 1, 3; q is stored in that
// order too, and O's columns are put back when it is written.
//
// Bound: per 128 x 128 scores the products take about 1020 cycles at d = 128 and the exponentials
// 1024 (16 a cycle); the tile's 32 KB of codes take about 1400 cycles of the SM's share of HBM.
// Few rows are bound by HBM, many by the tensor cores and the exponentials together.
#pragma once
#include "fa_q8.cuh"

namespace fa {

constexpr int kQ8TileThreads = 12 * 32;
constexpr int kQ8Tok = 128;                 // tokens of a tile
constexpr float kQ8TileMost = 15.f;         // log2 of the largest p: fp16 ends at 2^16
constexpr float kQ8TileStart = 6.f;         // and after the reference has moved
// f at the largest vs: e4m3 codes are at most 448, int8 codes 127
template <int kType> __device__ constexpr float q8_vtop() { return kType == kQ8E4m3 ? 0x1p6f : 0x1p8f; }

template <int HD>
struct Q8TileCfg {
  static constexpr int kChunks = HD / 64;             // 64-feature (128-byte) swizzle chunks
  static constexpr int kChunkBytes = 128 * 128;       // 128 rows x 128 bytes
  static constexpr int kTileBytes = kChunks * kChunkBytes;
  static constexpr int kScaleBufs = 4;
  static constexpr int kBars = 38;
  // Q (two row tiles), K and V (two tiles of tokens each), the codes of one tile of tokens
  static constexpr int kCodeBytes = kQ8Tok * HD;
  static constexpr size_t kNeed = 6 * kTileBytes + 2 * kCodeBytes + kScaleBufs * (kQ8Tok * 4 + 48) + kBars * 8 + 48;
  static constexpr size_t kSmem = kNeed > 116 * 1024 ? kNeed : 116 * 1024;
  static constexpr uint32_t kColS = 0, kColO = 256;
  // fp16 operands: the type fields of A and B are 0
  static constexpr uint32_t kFp16 = ~((1u << 7) | (1u << 10));
  static constexpr uint32_t kIdescQK = idesc_bf16_f32(128, 128, 0, 0) & kFp16;
  static constexpr uint32_t kIdescPV = idesc_bf16_f32(128, HD, 0, 1) & kFp16;
  static_assert(kSmem <= 227 * 1024, "shared memory budget");
  static_assert(kSmem > 114 * 1024, "one CTA per SM: it takes all of the tensor memory");
};

// Two bf16 features times a power of two, in fp16.
__device__ __forceinline__ uint32_t q8_fp16_of(uint32_t bf16x2, float unit) {
  return pack_fp16x2(__uint_as_float(bf16x2 << 16) * unit, __uint_as_float(bf16x2 & 0xffff0000u) * unit);
}

// 16-byte unit `unit` of row `row` in a 128-byte-swizzled chunk.
__device__ __forceinline__ uint32_t q8_swz(int row, int unit) {
  return static_cast<uint32_t>(row * 128 + ((unit ^ (row & 7)) << 4));
}

__device__ __forceinline__ uint32_t mul_fp16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// Registers a thread: 168 for all at launch (384 x 168 = 64512).  The softmax keeps 128 scores at once
// and spilled around them (reloads from L2: 800 to 2400 cycles a tile), the conversion needs fewer:
// 8 warps x 32 x 200 + 4 x 32 x 104 = 64512.
constexpr int kQ8LaunchRegs = 168, kQ8SoftmaxRegs = 200, kQ8ConvertRegs = 104;
static_assert(256 * kQ8SoftmaxRegs + 128 * kQ8ConvertRegs <= kQ8TileThreads * kQ8LaunchRegs,
              "registers of the launch");
template <int N>
__device__ __forceinline__ void q8_regs_acquire() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N>
__device__ __forceinline__ void q8_regs_release() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }

// Keeps uses of registers that a tcgen05.ld fills behind the wait that precedes this.
__device__ __forceinline__ void q8_pin(float (&x)[32]) {
#pragma unroll
  for (int i = 0; i < 32; ++i) asm volatile("" : "+f"(x[i]));
}

// A row's 128 scores (TMEM) -> p in fp16 (TMEM, over the scores: token pairs in the first 64 columns) and
// the sum of p.  k: the tokens that the row sees (kMasked: not all of them).  m and l are the row's
// reference and sum so far; where the reference has to move, l is brought to the new one and `a` is
// multiplied by what O needs.  All scores are in registers at once and the steps are kept apart
// (arguments, largest, exponentials).
template <bool kMasked>
__device__ __forceinline__ float q8_weigh(uint32_t s_tmem, const uint32_t (&k)[4], const float *ks, float &m,
                                          float &l, float &a) {
  const uint64_t neg2 = f2_pack(-m, -m);
  float x[128];
#pragma unroll
  for (int c = 0; c < 4; ++c) tmem_ld32(s_tmem + 32 * c, reinterpret_cast<uint32_t *>(x) + 32 * c);
  tmem_wait_ld();
#pragma unroll
  for (int i = 0; i < 128; ++i) asm volatile("" : "+f"(x[i]));
  float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
  for (int i = 0; i < 32; ++i) {
    const ulonglong2 f = reinterpret_cast<const ulonglong2 *>(ks)[i];
    f2_unpack(f2_fma(f2_pack(x[4 * i], x[4 * i + 1]), f.x, neg2), x[4 * i], x[4 * i + 1]);
    f2_unpack(f2_fma(f2_pack(x[4 * i + 2], x[4 * i + 3]), f.y, neg2), x[4 * i + 2], x[4 * i + 3]);
    if (kMasked) {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        x[4 * i + e] = (k[i / 8] >> (4 * (i % 8) + e)) & 1 ? x[4 * i + e] : -INFINITY;
    }
    top[i % 4] = fmax3(top[i % 4], fmaxf(x[4 * i], x[4 * i + 1]), fmaxf(x[4 * i + 2], x[4 * i + 3]));
  }
  const float t = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
  // (a row that has seen nothing has l = 0; an infinite score makes its row NaN through inf - inf)
  const bool over = t > kQ8TileMost || (l == 0.f && t != -INFINITY);
  if (__any_sync(0xffffffffu, over)) {
    const float d = over ? t - kQ8TileStart : 0.f;
    const float r = l == 0.f ? 1.f : ex2(-d);
    m += d;
    l *= r;
    a *= r;
    const uint64_t d2 = f2_pack(d, d);
#pragma unroll
    for (int i = 0; i < 64; ++i)
      f2_unpack(f2_sub(f2_pack(x[2 * i], x[2 * i + 1]), d2), x[2 * i], x[2 * i + 1]);
  }
  uint64_t sum[2] = {0, 0};
  uint32_t pk[64];
#pragma unroll
  for (int i = 0; i < 64; ++i) {
    const float p0 = ex2(x[2 * i]), p1 = ex2(x[2 * i + 1]);
    sum[i % 2] = f2_add(sum[i % 2], f2_pack(p0, p1));
    pk[i] = pack_fp16x2(p0, p1);
  }
  tmem_st32(s_tmem, pk);
  tmem_st32(s_tmem + 32, pk + 32);
  tmem_wait_st();
  float u, v;
  f2_unpack(f2_add(sum[0], sum[1]), u, v);
  return u + v;
}

// 32 features of a row, in the conversion's order, from its sums: to the output, or as a partial.
template <int HD, int kType>
__device__ __forceinline__ void q8_write32(const Q8Params &p, size_t row, int split, int c, const float (&o)[32],
                                           float m, float l, bool poison) {
  const float nan = __int_as_float(0x7fc00000);
#pragma unroll
  for (int i = 0; i < 32; i += 4) {
    const float4 v = poison ? make_float4(nan, nan, nan, nan)
                     : kType == kQ8Int8 ? make_float4(o[i], o[i + 2], o[i + 1], o[i + 3])
                                        : make_float4(o[i], o[i + 1], o[i + 2], o[i + 3]);
    if (p.n_split > 1)
      *reinterpret_cast<float4 *>(p.ws_o + (row * p.n_split + split) * HD + c + i) = v;
    else
      q8_write4<HD>(p, row, c + i, v, m, l);
  }
  if (c == 0 && p.n_split > 1) p.ws_ml[row * p.n_split + split] = make_float2(l == 0.f ? -INFINITY : m, l);
}

// Token tiles that the rows [r0, r1) can see: all of them, or up to the last row's own token.
__device__ __forceinline__ int q8_tiles(const Q8Params &p, int L, int r0, int r1) {
  if (r1 <= r0 || L == 0) return 0;
  if (!p.causal) return (L + kQ8Tok - 1) / kQ8Tok;
  const int t0 = r0 % p.T;
  const int t = t0 + (r1 - r0) - 1 < p.T ? t0 + (r1 - r0) - 1 : p.T - 1;
  return (L - p.T + t) / kQ8Tok + 1;
}

// S (TMEM) = Q K^T: both K-major in 64-feature swizzled chunks.
template <int HD>
__device__ __forceinline__ void q8_issue_qk(uint32_t d_tmem, const uint8_t *q, const uint8_t *k) {
  using C = Q8TileCfg<HD>;
  const uint64_t qd = smem_desc_sw128(smem_u32(q), 16, 1024), kd = smem_desc_sw128(smem_u32(k), 16, 1024);
#pragma unroll
  for (int kk = 0; kk < HD / 16; ++kk) {
    const uint64_t off = static_cast<uint64_t>(((kk / 4) * C::kChunkBytes + (kk % 4) * 32) >> 4);
    umma_ss(d_tmem, qd + off, kd + off, C::kIdescQK, kk > 0 ? 1u : 0u);
  }
}

// O (TMEM) (+)= P V: P from TMEM (8 columns per 16 tokens), V MN-major (chunks of 64 features, 8-token
// groups).  P is not staged in shared memory: a 128 x 128 x 16 product with both operands there reads
// the 128 bytes a cycle that shared memory has, and P's stores would come on top.
template <int HD>
__device__ __forceinline__ void q8_issue_pv(uint32_t d_tmem, uint32_t p_tmem, const uint8_t *v, bool accumulate) {
  using C = Q8TileCfg<HD>;
  const uint64_t vd = smem_desc_sw128(smem_u32(v), C::kChunkBytes, 1024);
#pragma unroll
  for (int kk = 0; kk < kQ8Tok / 16; ++kk)
    umma_ts(d_tmem, p_tmem + 8 * kk, vd + static_cast<uint64_t>((kk * 16 * 128) >> 4), C::kIdescPV,
            (accumulate || kk > 0) ? 1u : 0u);
}

// Every thread of warps 0-7 (none of them leaves before it; the waits on the way are bounded).
__device__ __forceinline__ void q8_sides_barrier() { asm volatile("bar.sync 1, 256;" ::: "memory"); }

// kTwo: two tiles of 128 rows, warps 0-3 and 4-7, every tile of tokens.  Else one tile of rows: warps
// 0-3 take the even tiles of tokens and warps 4-7 the odd ones, each with its own S, P, O and row
// sums, joined at the end.  A "side" below is either group of four warps.
template <int HD, int kType, bool kTwo>
__global__ void __launch_bounds__(kQ8TileThreads, 1) fa_q8_tile_kernel(const Q8Params p) {
  using C = Q8TileCfg<HD>;
  extern __shared__ __align__(1024) uint8_t q8_tile_smem[];  // no room for slack: checked below
  uint8_t *sQ = q8_tile_smem;             // [row tile]
  uint8_t *sK = sQ + 2 * C::kTileBytes;   // tile j of tokens is in [j & 1]
  uint8_t *sV = sK + 2 * C::kTileBytes;
  uint8_t *sKc = sV + 2 * C::kTileBytes;  // codes of K as they land, a quarter of the tile to a warp
  uint8_t *sVc = sKc + C::kCodeBytes;     // and of V
  float *sKs = reinterpret_cast<float *>(sVc + C::kCodeBytes);  // [buffer][token]: ks scale log2(e)
  uint32_t *sLive = reinterpret_cast<uint32_t *>(sKs + C::kScaleBufs * kQ8Tok);  // [buffer][4]
  uint32_t *sBad = sLive + C::kScaleBufs * 4;  // [buffer][4]: live tokens whose vs is not finite
  float *sF = reinterpret_cast<float *>(sBad + C::kScaleBufs * 4);  // [buffer][4]: F of the tile
  uint64_t *bars = reinterpret_cast<uint64_t *>(sF + C::kScaleBufs * 4);
  // Barriers of tile j are [j & 1], as its buffers are, so that a side that waits for every other tile of
  // tokens sees each phase of its own.  A buffer is freed by an arrival from each issuer that reads it.
  uint64_t *k_full = bars, *v_full = bars + 2, *k_free = bars + 4, *v_free = bars + 6;  // [2]
  uint64_t *sc_full = bars + 8;                 // [4]
  uint64_t *s_full = bars + 12;                 // [side]
  uint64_t *p_full = bars + 14;                 // [side]
  uint64_t *pv_done = bars + 16;                // [side]
  uint64_t *drain = bars + 18;                  // [side] every product of an issuer has completed
  uint64_t *q_full = bars + 20;                 // [row tile]
  uint64_t *turn = bars + 22;                   // [side][warp]
  uint64_t *landed = bars + 30;                 // [K, V][converter warp]
  float *sTop = reinterpret_cast<float *>(bars + C::kBars);  // [8]: the warps' largest |q|
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(sTop + 8);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);

  unsigned u = blockIdx.x;
  const int split = u % p.n_split;
  u /= p.n_split;
  const int group = u % p.row_tiles;
  u /= p.row_tiles;
  const int kh = u % p.Hk, s = u / p.Hk;
  const int row0 = group * (kTwo ? 256 : 128);
  const size_t row_base = (static_cast<size_t>(s) * p.Hk + kh) * p.R;
  const int L = q8_len(p, s);
  const int tiles_per_split = p.split_pages / (kQ8Tok / kQ8Page);
  const int j0 = split * tiles_per_split;
  if (p.n_split > 1 && j0 * kQ8Tok >= L) return;  // past the sequence's end: the combine skips it
  // tiles of tokens that each side takes, and that the CTA takes in all
  int n[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int r0 = row0 + 128 * i;
    const int all = (i == 1 && !kTwo) ? 0 : q8_tiles(p, L, r0, min(r0 + 128, p.R));
    n[i] = max(0, min(all, j0 + tiles_per_split) - j0);
  }
  const int nmax = max(n[0], n[1]);
  if (!kTwo) n[0] = (nmax + 1) / 2, n[1] = nmax / 2;
  const int both = min(n[0], n[1]);

  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  if (smem_u32(q8_tile_smem) & 1023u) {  // the swizzled tiles need it; the launch gives it
    if (threadIdx.x == 0) atomicExch(&g_device_status, 4 /* FA_ERR_LAUNCH */);
    return;
  }
  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(k_full + i, 4);
      mbar_init(v_full + i, 4);
      mbar_init(k_free + i, kTwo ? 2 : 1);
      mbar_init(v_free + i, kTwo ? 2 : 1);
      mbar_init(s_full + i, 1);
      mbar_init(p_full + i, 4);
      mbar_init(pv_done + i, 1);
      mbar_init(drain + i, 1);
      mbar_init(q_full + i, 4);
    }
    for (int i = 0; i < 4; ++i) mbar_init(sc_full + i, 4);
    for (int i = 0; i < 8; ++i) mbar_init(turn + i, 1), mbar_init(landed + i, 1);
    *abort_flag = 0;
    if (L != p.lens[s] && p.lens[s] > 0) atomicExch(&g_device_status, 1 /* FA_ERR_INVALID_ARG */);
    fence_mbar_init();
  }
  if (warp == 8) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  if (warp < 8) {
    const int row = row0 + (kTwo ? 128 * (warp / 4) : 0) + threadIdx.x % 128;
    float top = 0.f;
    if (row < p.R) {
      const uint4 *src = reinterpret_cast<const uint4 *>(p.q + (row_base + row) * HD);
#pragma unroll
      for (int c = 0; c < HD / 8; ++c) {
        const uint4 v = src[c];
        top = q8_finite_max(q8_finite_max(q8_finite_max(q8_finite_max(top, v.x), v.y), v.z), v.w);
      }
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
    if (lane == 0) sTop[warp] = top;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  float q_top = sTop[0];
#pragma unroll
  for (int i = 1; i < 8; ++i) q_top = fmaxf(q_top, sTop[i]);
  const float q_unit = q8_q_unit(q_top);

  if (warp >= 8) {
    // ------------------------------------------------------------------ codes -> 16-bit tiles
    q8_regs_release<kQ8ConvertRegs>();
    const int w = warp - 8;              // tokens 32 w .. 32 w + 31 of a tile: pages 2 w, 2 w + 1
    constexpr int kPieces = HD / 8;      // 8-code pieces of a token
    constexpr int kRowsPer = 32 / kPieces;  // tokens that a warp-wide load covers
    constexpr int kLoads = 32 / kRowsPer;
    constexpr uint32_t kSlab = kQ8Page * HD;  // a page of one head: contiguous in the pool
    const int piece = lane % kPieces, sub = lane / kPieces;
    const int32_t *trow = p.table + static_cast<size_t>(s) * p.max_blocks;
    const int nblk = (L + kQ8Page - 1) / kQ8Page;
    // lane i < 8: the table's entry for page i of tile j; not looked at before it is needed (named)
    auto entry_of = [&](int j) -> int {
      const int page = (j0 + j) * (kQ8Tok / kQ8Page) + lane;
      return (lane < kQ8Tok / kQ8Page && j < nmax && page < nblk) ? trow[page] : -1;
    };
    auto named = [&](int j, int b) -> int {  // -1 for a page that the table does not name
      const int page = (j0 + j) * (kQ8Tok / kQ8Page) + lane;
      if (b >= 0 && b < p.num_blocks) return b;
      if (lane < kQ8Tok / kQ8Page && j < nmax && page < nblk)
        atomicExch(&g_device_status, 1 /* FA_ERR_INVALID_ARG: the page is left out */);
      return -1;
    };
    uint8_t *kst = sKc + 2 * w * kSlab, *vst = sVc + 2 * w * kSlab;
    uint64_t *k_landed = landed + w, *v_landed = landed + 4 + w;
    // the warp's two pages of a tile into its staging slot: lanes 0 and 1, a page each; one that is left
    // out is not loaded (its tokens are not live)
    auto load_codes = [&](const uint8_t *codes, int blk, uint8_t *dst, uint64_t *bar) {
      const int b = __shfl_sync(0xffffffffu, blk, 2 * w + (lane & 1));
      const uint32_t both_named = __ballot_sync(0xffffffffu, b >= 0) & 3u;
      if (lane == 0) {
        if (both_named) mbar_arrive_expect_tx(bar, (both_named == 3u ? 2 : 1) * kSlab);
        else mbar_arrive(bar);
      }
      if (lane < 2 && b >= 0)
        bulk_load_1d(dst + lane * kSlab, codes + (static_cast<size_t>(b) * p.Hk + kh) * kSlab, kSlab, bar);
    };
    const uint32_t at0 = static_cast<uint32_t>(piece / 8) * C::kChunkBytes;
    const int unit = piece % 8;
    float4 ks, vs;      // of tokens 4 lane .. 4 lane + 3 of the tile (ks: the warp's own tokens only)
    uint32_t live = 0;  // the warp's own 32 tokens
    auto fetch_scales = [&](int j, int blk) {
      const int b = __shfl_sync(0xffffffffu, blk, lane / 4);
      const size_t at = (static_cast<size_t>(max(b, 0)) * p.Hk + kh) * kQ8Page + 4 * (lane % 4);
      ks = vs = make_float4(0.f, 0.f, 0.f, 0.f);
      if (b >= 0) vs = *reinterpret_cast<const float4 *>(p.vs + at);
      if (b >= 0 && lane / 8 == w) ks = *reinterpret_cast<const float4 *>(p.ks + at);
      live = 0;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int left = L - (j0 + j) * kQ8Tok - 32 * w - 16 * h;
        const int bh = __shfl_sync(0xffffffffu, blk, 2 * w + h);
        if (bh >= 0 && left > 0) live |= (left >= 16 ? 0xffffu : (1u << left) - 1u) << (16 * h);
      }
    };
    float F = 0x1p-126f;  // every warp finds the same F, tile by tile
    const float score_scale = p.scale_log2 * q8_inverse(q_unit);
    uint32_t f01 = 0, f23 = 0;  // f of tokens 4 lane ..
    // the scales of tile j (fetched before): key scales, live tokens, F
    auto publish_scales = [&](int j) {
      const int buf = j % C::kScaleBufs;
      const int left = L - (j0 + j) * kQ8Tok - 4 * lane;  // tokens of this lane before the end
      float v[4] = {vs.x, vs.y, vs.z, vs.w};
      float top = 0.f;  // the tile's largest finite vs
      bool bad = false;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        if (c >= left) v[c] = 0.f;  // a slot past the end may hold anything
        const bool fin = fabsf(v[c]) < INFINITY;
        bad = bad || !fin;
        top = fmaxf(top, fin ? v[c] : 0.f);
      }
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
      if (top > F)  // the power of two above it
        F = __uint_as_float(min(((__float_as_uint(top) >> 23) & 0xffu) + 1u, 254u) << 23);
      uint32_t badmask = 0;
      if (__any_sync(0xffffffffu, bad)) {
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const uint32_t m = (__ballot_sync(0xffffffffu, !(fabsf(v[c]) < INFINITY)) >> (8 * w)) & 0xffu;
          for (int i = 0; i < 8; ++i) badmask |= ((m >> i) & 1u) << (4 * i + c);
          if (!(fabsf(v[c]) < INFINITY)) v[c] = 0.f;
        }
      }
      // (vs / F first: neither factor leaves the normal range)
      const float inv = 1.f / F;
      f01 = pack_fp16x2(v[0] * inv * q8_vtop<kType>(), v[1] * inv * q8_vtop<kType>());
      f23 = pack_fp16x2(v[2] * inv * q8_vtop<kType>(), v[3] * inv * q8_vtop<kType>());
      if (lane / 8 == w)
        *reinterpret_cast<float4 *>(sKs + buf * kQ8Tok + 4 * lane) =
            make_float4(ks.x * score_scale, ks.y * score_scale, ks.z * score_scale, ks.w * score_scale);
      if (lane == 0) {
        sLive[buf * 4 + w] = live;
        sBad[buf * 4 + w] = badmask;
        if (w == 0) sF[buf * 4] = F;
      }
    };
    // K runs one tile before V, as the products do
    int blk_k = named(0, entry_of(0)), entry = entry_of(1);
    if (nmax > 0) {
      load_codes(p.k_codes, blk_k, kst, k_landed);
      load_codes(p.v_codes, blk_k, vst, v_landed);
      fetch_scales(0, blk_k);
    }
    // f and the live tokens of the next V tile
    uint32_t f01_v = 0, f23_v = 0, live_v = 0, live_k = 0;
    for (int j = -1; j < nmax; ++j) {
      const int jk = j + 1;
      int blk_next = blk_k;
      f01_v = f01, f23_v = f23, live_v = live_k;
      uint2 c[kLoads];
      if (jk < nmax) {
        if (!__all_sync(0xffffffffu, mbar_wait(k_landed, jk & 1, abort_flag))) break;
#pragma unroll
        for (int i = 0; i < kLoads; ++i)
          c[i] = *reinterpret_cast<const uint2 *>(kst + (i * kRowsPer + sub) * HD + 8 * piece);
        __syncwarp();  // the slot has been read: refill it
        blk_next = named(jk + 1, entry);
        if (jk + 1 < nmax) load_codes(p.k_codes, blk_next, kst, k_landed);
        live_k = live;
        if (jk >= 2 && !__all_sync(0xffffffffu, mbar_wait(k_free + (jk & 1), ((jk >> 1) - 1) & 1, abort_flag))) break;
        publish_scales(jk);
        uint8_t *kt = sK + (jk & 1) * C::kTileBytes + at0;
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
          uint4 o;
          q8_cvt4<kType>(c[i].x, o.x, o.y);
          q8_cvt4<kType>(c[i].y, o.z, o.w);
          *reinterpret_cast<uint4 *>(kt + q8_swz(32 * w + i * kRowsPer + sub, unit)) = o;
        }
        fence_async_smem();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(sc_full + jk % C::kScaleBufs);
          mbar_arrive(k_full + (jk & 1));
        }
        entry = entry_of(jk + 2);
        if (jk + 1 < nmax) fetch_scales(jk + 1, blk_next);
      }
      if (j >= 0) {
        if (!__all_sync(0xffffffffu, mbar_wait(v_landed, j & 1, abort_flag))) break;
#pragma unroll
        for (int i = 0; i < kLoads; ++i)
          c[i] = *reinterpret_cast<const uint2 *>(vst + (i * kRowsPer + sub) * HD + 8 * piece);
        __syncwarp();
        if (j + 1 < nmax) load_codes(p.v_codes, blk_k, vst, v_landed);  // (blk_k: still of tile j + 1)
        if (j >= 2 && !__all_sync(0xffffffffu, mbar_wait(v_free + (j & 1), ((j >> 1) - 1) & 1, abort_flag))) break;
        uint8_t *vt = sV + (j & 1) * C::kTileBytes + at0;
        const bool all = live_v == 0xffffffffu;
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
          const int tok = i * kRowsPer + sub;  // of the warp's 32: f is with lane 8 w + tok / 4
          const uint32_t pair = __shfl_sync(0xffffffffu, (i * kRowsPer) & 2 ? f23_v : f01_v, 8 * w + (i * kRowsPer) / 4);
          // (four tokens to a load at d = 64: the upper two are the other pair's)
          uint32_t fp = pair;
          if (kRowsPer == 4) {
            const uint32_t hi = __shfl_sync(0xffffffffu, f23_v, 8 * w + i);
            fp = sub >= 2 ? hi : pair;
          }
          const uint32_t f = __byte_perm(fp, fp, (sub & 1) ? 0x3232 : 0x1010);
          // a slot that no token holds may have any bytes, and e4m3's NaN would pass through p = 0
          if (kType == kQ8E4m3 && !all && !((live_v >> tok) & 1)) c[i] = make_uint2(0u, 0u);
          uint4 o;
          q8_cvt4<kType>(c[i].x, o.x, o.y);
          q8_cvt4<kType>(c[i].y, o.z, o.w);
          o = make_uint4(mul_fp16x2(o.x, f), mul_fp16x2(o.y, f), mul_fp16x2(o.z, f), mul_fp16x2(o.w, f));
          *reinterpret_cast<uint4 *>(vt + q8_swz(32 * w + tok, unit)) = o;
        }
        fence_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(v_full + (j & 1));
      }
      blk_k = blk_next;
    }
    // abandoned: a copy still on its way lands before the CTA's shared memory goes away
    if (*abort_flag) {
      const uint64_t t0 = globaltimer_ns();
      while (globaltimer_ns() - t0 < 1000000) {
      }
    }
  } else {
    // ------------------------------------------------------------------ softmax, products, epilogue
    q8_regs_acquire<kQ8SoftmaxRegs>();
    const int side = warp / 4;
    const int rtile = kTwo ? side : 0;
    const int lrow = threadIdx.x % 128;
    const int row = row0 + 128 * rtile + lrow;
    const bool mine = row < p.R;
    const int cnt = n[side];
    const uint32_t lane_off = static_cast<uint32_t>((warp % 4) * 32) << 16;
    if (kTwo || side == 0) {  // this thread's row of q, in the layout the tensor core reads
      const uint16_t *src = p.q + (row_base + row) * HD;
      uint8_t *dst = sQ + rtile * C::kTileBytes;
#pragma unroll
      for (int c = 0; c < HD / 8; ++c) {
        uint4 v = make_uint4(0u, 0u, 0u, 0u);
        if (mine) v = *reinterpret_cast<const uint4 *>(src + 8 * c);
        if constexpr (kType == kQ8Int8)
          v = make_uint4(__byte_perm(v.x, v.y, 0x5410), __byte_perm(v.x, v.y, 0x7632),
                         __byte_perm(v.z, v.w, 0x5410), __byte_perm(v.z, v.w, 0x7632));
        v = make_uint4(q8_fp16_of(v.x, q_unit), q8_fp16_of(v.y, q_unit), q8_fp16_of(v.z, q_unit),
                       q8_fp16_of(v.w, q_unit));
        *reinterpret_cast<uint4 *>(dst + (c / 8) * C::kChunkBytes + q8_swz(lrow, c % 8)) = v;
      }
      fence_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(q_full + rtile);
    }
    const uint32_t tS = tmem + C::kColS + 128 * side, tO = tmem + C::kColO + HD * side;
    auto tile_of = [&](int i) { return kTwo ? i : 2 * i + side; };  // the side's i-th tile of tokens
    // The first thread of the side's first warp issues its products.  With two row tiles it also
    // arrives on k_free and v_free for the tiles of tokens that only the other one visits.
    const bool lead = warp % 4 == 0 && lane == 0;
    const int steps = kTwo ? nmax : cnt;
    auto next_scores = [&](int i) -> bool {  // S of the side's tile i, or the word that K is not needed
      if (i >= steps) return true;
      const int j = tile_of(i);
      if (!mbar_wait(k_full + (j & 1), (j >> 1) & 1, abort_flag)) return false;
      if (i < cnt) {
        tc_fence_after();
        q8_issue_qk<HD>(tS, sQ + rtile * C::kTileBytes, sK + (j & 1) * C::kTileBytes);
        umma_commit(s_full + side);
        umma_commit(k_free + (j & 1));
      } else {
        mbar_arrive(k_free + (j & 1));
      }
      return true;
    };
    auto products = [&](int i) -> bool {  // O += P V of the side's tile i, then the next scores
      const int j = tile_of(i);
      if (!mbar_wait(v_full + (j & 1), (j >> 1) & 1, abort_flag)) return false;
      if (i < cnt) {
        if (!mbar_wait(p_full + side, i & 1, abort_flag)) return false;
        tc_fence_after();
        q8_issue_pv<HD>(tO, tS, sV + (j & 1) * C::kTileBytes, i > 0);
        umma_commit(pv_done + side);
        umma_commit(v_free + (j & 1));
        // P lies over S: the next scores may be written once this product has read it
        if (!mbar_wait(pv_done + side, i & 1, abort_flag)) return false;
      } else {
        mbar_arrive(v_free + (j & 1));
      }
      return next_scores(i + 1);
    };
    // Turns: the two sides' warps of an SM sub-partition do their exponentials one after the other, so
    // that one side's products run meanwhile; left alone they fall into step and wait together.
    auto my_turn = [&](int i) -> bool {
      if (i >= both || (side == 0 && i == 0)) return true;
      return __all_sync(0xffffffffu, mbar_wait(turn + warp, (side == 0 ? i - 1 : i) & 1, abort_flag));
    };
    auto pass_turn = [&](int i) {
      __syncwarp();
      if (i < both && lane == 0) mbar_arrive(turn + (warp ^ 4));
    };
    const int t = mine ? row % p.T : 0;
    const int first_own = L - p.T;  // the first of the queries' own tokens
    const uint64_t bits = (p.tree && mine) ? p.tree[static_cast<size_t>(s) * p.T + t] : ~0ull;
    const bool warp_rows = row0 + 128 * rtile + (warp % 4) * 32 < p.R;  // any row in this warp
    float m = 0.f, l = 0.f, F = 0.f;
    bool poison = false;  // the row sees a token whose values are no numbers
    bool ok = __all_sync(0xffffffffu,
                         !lead || ((cnt == 0 || mbar_wait(q_full + rtile, 0, abort_flag)) && next_scores(0)));
    for (int i = 0; ok && i < cnt; ++i) {
      const int j = tile_of(i);
      const int buf = j % C::kScaleBufs;
      const float *ksb = sKs + buf * kQ8Tok;
      // warp-uniform, as the tensor-memory loads below are warp-wide.  P V of the tile before has
      // completed (these scores are issued after it), so O may be rescaled.
      if (!__all_sync(0xffffffffu, mbar_wait(sc_full + buf, (j / C::kScaleBufs) & 1, abort_flag) &&
                                       mbar_wait(s_full + side, i & 1, abort_flag)) ||
          !my_turn(i)) { ok = false; break; }
      tc_fence_after();
      if (!warp_rows) {
        // rows past R: whatever P holds goes to O rows that nobody reads.  (The issuer's warp has
        // rows, or the side has no tiles.)
        pass_turn(i);
        tc_fence_before();
        if (lane == 0) mbar_arrive(p_full + side);
        continue;
      }
      const int tok0 = (j0 + j) * kQ8Tok;
      const float F_old = F;
      F = sF[buf * 4];
      uint32_t k[4];  // the tokens that this row sees
      {
        const uint4 live = *reinterpret_cast<const uint4 *>(sLive + buf * 4);
        k[0] = live.x, k[1] = live.y, k[2] = live.z, k[3] = live.w;
      }
      if ((p.causal || p.tree) && tok0 + kQ8Tok > first_own) {
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const int v0 = tok0 + 32 * c - first_own;  // the chunk's first token among the queries' own
          if (p.tree) {
            k[c] &= v0 >= 64 ? 0u : v0 >= 0 ? static_cast<uint32_t>(bits >> v0)
                    : v0 > -32 ? (static_cast<uint32_t>(bits << -v0) | ((1u << -v0) - 1u)) : ~0u;
          } else {
            const int lim = t - v0 + 1;
            k[c] &= lim >= 32 ? ~0u : lim <= 0 ? 0u : (1u << lim) - 1u;
          }
        }
      }
      const bool all = __all_sync(0xffffffffu, (k[0] & k[1] & k[2] & k[3]) == 0xffffffffu);
      {
        const uint4 bad = *reinterpret_cast<const uint4 *>(sBad + buf * 4);
        poison = poison || ((k[0] & bad.x) | (k[1] & bad.y) | (k[2] & bad.z) | (k[3] & bad.w)) != 0;
      }
      float a = i == 0 ? 1.f : F_old / F;  // what O is to be multiplied by
      const float sum = all ? q8_weigh<false>(tS + lane_off, k, ksb, m, l, a)
                            : q8_weigh<true>(tS + lane_off, k, ksb, m, l, a);
      pass_turn(i);
      if (i > 0 && __any_sync(0xffffffffu, a != 1.f)) {
#pragma unroll 1
        for (int c = 0; c < HD; c += 32) {
          float o[32];
          tmem_ld32(tO + lane_off + c, reinterpret_cast<uint32_t *>(o));
          tmem_wait_ld();
          q8_pin(o);
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] *= a;
          tmem_st32(tO + lane_off + c, reinterpret_cast<uint32_t *>(o));
          tmem_wait_st();
        }
      }
      l += sum;
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(p_full + side);
      ok = __all_sync(0xffffffffu, !lead || products(i));
    }
    if (lead) {
      for (int i = cnt; ok && i < steps; ++i) ok = products(i);
      // every product issued here completes before tensor memory is given back
      umma_commit(drain + side);
      volatile int never = 0;
      mbar_wait(drain + side, 0, &never);
    }
    ok = __all_sync(0xffffffffu, ok && (cnt == 0 || mbar_wait(pv_done + side, (cnt - 1) & 1, abort_flag)));
    tc_fence_after();
    const float f = F / q8_vtop<kType>();  // of this side's O
    if constexpr (!kTwo) {
      // join the sides: the odd tiles' sums go through shared memory, the even side writes.  Both are
      // brought to the larger reference.
      float *xo = reinterpret_cast<float *>(sK);                     // [feature][row]
      float *xm = reinterpret_cast<float *>(sV);                     // m, l, poison of the odd side
      q8_sides_barrier();  // every product has completed: K and V are free
      if (side == 1 && warp_rows && ok) {
        xm[lrow] = m;
        xm[128 + lrow] = l;
        xm[256 + lrow] = poison ? 1.f : 0.f;
#pragma unroll 1
        for (int c = 0; c < HD; c += 32) {
          float o[32];
          if (cnt > 0) {
            tmem_ld32(tO + lane_off + c, reinterpret_cast<uint32_t *>(o));
            tmem_wait_ld();
            q8_pin(o);
          }
#pragma unroll
          for (int e = 0; e < 32; ++e) xo[(c + e) * 128 + lrow] = cnt > 0 && l != 0.f ? o[e] * f : 0.f;
        }
      }
      q8_sides_barrier();
      if (side == 0 && warp_rows && ok) {
        const float m1 = xm[lrow], l1 = xm[128 + lrow];
        poison = poison || xm[256 + lrow] != 0.f;
        const float M = l == 0.f ? m1 : l1 == 0.f ? m : fmaxf(m, m1);
        const float a0 = l == 0.f ? 0.f : ex2(m - M), a1 = l1 == 0.f ? 0.f : ex2(m1 - M);
        const bool none = l == 0.f;
        l = (none ? 0.f : l * a0) + (l1 == 0.f ? 0.f : l1 * a1);
        m = M;
#pragma unroll 1
        for (int c = 0; c < HD; c += 32) {
          float o[32];
          if (cnt > 0) {
            tmem_ld32(tO + lane_off + c, reinterpret_cast<uint32_t *>(o));
            tmem_wait_ld();
            q8_pin(o);
          }
          if (mine) {
#pragma unroll
            for (int e = 0; e < 32; ++e)
              o[e] = (none ? 0.f : o[e] * f * a0) + (l1 == 0.f ? 0.f : xo[(c + e) * 128 + lrow] * a1);
            q8_write32<HD, kType>(p, row_base + row, split, c, o, m, l, poison);
          }
          __syncwarp();
        }
      }
    } else if (ok && warp_rows) {
      const bool none = l == 0.f;
#pragma unroll 1
      for (int c = 0; c < HD; c += 32) {
        float o[32];
        if (cnt > 0) {
          tmem_ld32(tO + lane_off + c, reinterpret_cast<uint32_t *>(o));
          tmem_wait_ld();
          q8_pin(o);
        }
        if (mine) {
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = none ? 0.f : o[e] * f;
          q8_write32<HD, kType>(p, row_base + row, split, c, o, m, l, poison);
        }
        __syncwarp();
      }
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == 8) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

}  // namespace fa
