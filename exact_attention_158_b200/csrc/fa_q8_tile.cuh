// fa_q8_tile.cuh -- attention of many rows (a prompt chunk, a draft tree, large groups) over an 8-bit
// paged cache on the tcgen05 tensor cores.  The mathematics is that of fa_q8.cuh; only the values'
// scales sit elsewhere.
//
// One CTA takes up to 256 of the R rows of one (sequence, key head) and a range of its 64-token
// tiles.  Codes cannot feed a 16-bit product, so they are converted once per tile for all of the
// CTA's rows:
//   warps 0-3    one side: a thread holds a row (a TMEM lane).  Scores out of TMEM, p back over them
//   warps 4-7    the other side
//   warps 8-11   codes -> fp16 K and V tiles in the swizzled layout the tensor core reads
//   warps 12-13  products: one thread issues for each side
//   warp  14     codes out of the pool by bulk copies, three tiles ahead
//   warp  15     a tile's scales and live tokens
// TMEM (512 columns): S [side][2] x 64, then O [side] x d.  With more than 128 rows the sides hold two
// row tiles; with fewer they share one row tile and take the tiles of tokens in turn.  A side's S is
// double, so Q K^T of the next tile and P V of the last run during its softmax.  (128-token tiles fill the
// same columns with one S: softmax, P V and Q K^T of a side then follow one another.  The step away from
// them, with a warp each for loads and scales and the order by length, took trees of 48 nodes from 190
// to 125 us and 512-token chunks from 405 to 304.)
//
// Scales.  A key's scale multiplies its column of scores in fp32, read from shared memory by every
// row (16 broadcast 16-byte loads per row and tile).  A value's scale vs = f 2^e is split: f goes into V =
// code * f in fp16, and the power of two into the exponent of p = 2^(s + e - m), whose reference m then
// follows the largest p vs as in fa_q8.cuh; the row's sum takes p 2^-e.  One e for a tile of tokens (the
// power of two above its largest vs) costs nothing, so that is the form wherever the tile's scales
// lie within 2^8 of one another; f is then 2^-9 at least, and a token loses less than 2^-22 of the row's
// largest p vs.  Else (wide) each token has its own e and p takes a second exponential for the sum: what a
// loud token would take from f and p of the others does not depend on whether a row sees it.  A tile
// far below an earlier one is wide too, since 2^(s + e - m) may leave fp32's range where 2^(s - m), which
// the sum needs, does not.  f, code * f and p are rounded to fp16 (2^-11 each).  A value scale that is not finite would reach rows that do
// not see its token as 0 * NaN: V is 0 there, and rows that do see it are marked and written as NaN.
//
// A row's softmax is one pass over its scores in registers: p = 2^(s ks + e - m) against the reference it
// has; where one passes 2^15, and on a row's first tile, the reference moves so that the largest p is
// 2^6, and O is rescaled in TMEM.
//
// Queries go to fp16 against one power of two for all rows of the CTA (q8_q_unit; it is part of the key
// scales), unless their largest features lie more than 2^12 apart: then each row has its own, and
// every tile is taken in the wide form, which multiplies by it.  int8's conversion leaves every four
// features in the order 0, 2, 1, 3; q is stored in that order too, and O's columns are put back when
// it is written.
//
// Bound: per 128 rows x 64 tokens the products take about 510 cycles at d = 128 and the exponentials
// 512 (16 a cycle); the 16 KB of codes take about 700 cycles of the SM's share of HBM.  Measured, a tile
// of tokens takes 2570 cycles with two row tiles and 1760 with one, and no unit is full: tensor pipe 36%,
// exponentials 37%, issue slots 42%, the softmax warps, two to a scheduler, waiting for one step after
// another.  Start and end of a CTA come on top, once or twice per SM.  512-token chunks of 4 sequences:
// 312 us, 604 TFLOP/s; trees of 48 nodes, 32 sequences: 127 us (DRAM's floor 28 us, the products' 35).
#pragma once
#include "fa_q8.cuh"

namespace fa {

constexpr int kQ8TileThreads = 16 * 32;
constexpr int kQ8Tok = 64;                  // tokens of a tile
constexpr int kQ8TilePages = kQ8Tok / kQ8Page;
constexpr int kQ8KBufs = 4;                 // K tiles in shared memory; V: 2, or 4 with one row tile
constexpr int kQ8MostVBufs = 4;
constexpr int kQ8CodeBufs = 3;              // tiles of codes on their way
constexpr float kQ8TileMost = 15.f;         // log2 of the largest p: fp16 ends at 2^16
constexpr float kQ8TileStart = 6.f;         // and after the reference has moved
constexpr int kQ8TileNear = 8;              // log2 of how far a tile's scales may lie apart and share one e,
constexpr int kQ8TileFar = 64;              // and of how far below an earlier tile's they may lie
// e's range: 2^-89 leaves the smallest scale, 2^-109, f = 2^-20, and a row's sum of p 2^-e in fp32's
// range; 2^126 is the largest whose inverse is a normal number
constexpr int kQ8LeastE = -89, kQ8MostE = 126;
// The largest feature of a row, against the largest of the CTA's rows, from which on they share a power of
// two: it then lies at 2^2 or above in fp16 and loses 2^-27 of it at most.
constexpr float kQ8RowsNear = 0x1p-12f;
// f = 1 as V holds it: e4m3 codes are at most 448, int8 codes 127
template <int kType> __device__ constexpr float q8_vtop() { return kType == kQ8E4m3 ? 0x1p6f : 0x1p8f; }

template <int HD>
struct Q8TileCfg {
  static constexpr int kChunks = HD / 64;             // 64-feature (128-byte) swizzle chunks
  static constexpr int kQChunk = 128 * 128;           // 128 rows x 128 bytes
  static constexpr int kChunk = kQ8Tok * 128;         // 64 tokens x 128 bytes
  static constexpr int kQBytes = kChunks * kQChunk;
  static constexpr int kTileBytes = kChunks * kChunk;
  static constexpr int kCodeBytes = kQ8Tok * HD;      // of K or V of one tile
  static constexpr int kScaleBufs = 8;
  static constexpr int kBars = 2 * kQ8KBufs + 2 * kQ8MostVBufs + 2 * kQ8CodeBufs + 2 * kScaleBufs + 4 + 4 + 4 + 2 + 2;
  // Q (two row tiles, or one and two more V tiles in its place), K and V tiles, codes, scales (ks, f, e, live
  // and bad tokens, the tile's)
  static_assert(kQBytes == 2 * kTileBytes, "two V tiles in the place of a row tile's Q");
  static constexpr size_t kNeed = 1024 + 2 * kQBytes + (kQ8KBufs + 2) * kTileBytes +
                                  2 * kQ8CodeBufs * kCodeBytes + kScaleBufs * (kQ8Tok * 12 + 32) + kBars * 8 + 80 + 1024;
  static constexpr size_t kSmem = kNeed > 116 * 1024 ? kNeed : 116 * 1024;
  static constexpr uint32_t kColO = 256;  // S: [side][2] x 64 columns before it
  // fp16 operands: the type fields of A and B are 0
  static constexpr uint32_t kFp16 = ~((1u << 7) | (1u << 10));
  static constexpr uint32_t kIdescQK = idesc_bf16_f32(128, kQ8Tok, 0, 0) & kFp16;
  static constexpr uint32_t kIdescPV = idesc_bf16_f32(128, HD, 0, 1) & kFp16;
  static_assert(kSmem <= 227 * 1024, "shared memory budget");
  static_assert(kSmem > 114 * 1024, "one CTA per SM: it takes all of the tensor memory");
};

// Up to here every CTA ranks the sequences itself.  128 sequences of 100 to 2000 tokens, 2 key heads, 40 rows:
// 66 us ranked and 82 in the batch's order (all of one length: 68 and 66).  256 would gain as much as
// they lose: 127 us ranked and 137 not when ragged, 131 and 121 when alike; 512 ragged ones 270 and 260.
constexpr int kQ8SortSeqs = 128;

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

// Four columns of a lane's row of tensor memory, and two back.
__device__ __forceinline__ void tmem_ld4(uint32_t taddr, uint32_t *r) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(taddr));
}

__device__ __forceinline__ void tmem_st2(uint32_t taddr, const uint32_t *r) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x2.b32 [%0], {%1,%2};" ::"r"(taddr), "r"(r[0]), "r"(r[1])
               : "memory");
}

// Keeps uses of registers that a tcgen05.ld fills behind the wait that precedes this.
__device__ __forceinline__ void q8_pin(float (&x)[32]) {
#pragma unroll
  for (int i = 0; i < 32; ++i) asm volatile("" : "+f"(x[i]));
}

// The power of two above a scale, as its exponent in e's range.
__device__ __forceinline__ uint32_t q8_exponent(float x) { return (__float_as_uint(x) >> 23) & 0xffu; }
__device__ __forceinline__ int q8_e(uint32_t exponent) {
  return min(max(static_cast<int>(exponent) - 126, kQ8LeastE), kQ8MostE);
}
__device__ __forceinline__ float q8_pow2(int e) { return __uint_as_float(static_cast<uint32_t>(127 + e) << 23); }

// Where a lane's largest p passes 2^15, or its row has seen nothing yet, its reference moves so that the
// largest is 2^6: m and l follow, `a` is multiplied by what O needs, and the step is returned (0: none).
// (a row that has seen nothing has l = 0; an infinite score makes its row NaN through inf - inf)
__device__ __forceinline__ float q8_move(float t, bool over, float &m, float &l, float &a) {
  const float d = over ? t - kQ8TileStart : 0.f;
  if (l != 0.f) {
    l = q8_shift(l, -d);
    a *= ex2(-d);
  }
  m += d;
  return d;
}

// A row's 64 scores (TMEM) -> p in fp16 (TMEM, over the scores: token pairs in the first 32 columns) and
// the sum of p.  k: the tokens that the row sees (kMasked: not all of them).  m and l are the row's
// reference and sum so far, e is the tile's.  All scores are in registers at once and the steps are kept
// apart (arguments, largest, exponentials): taken a few at a time, each few wait for their loads of ks.
template <bool kMasked>
__device__ __forceinline__ float q8_weigh(uint32_t s_tmem, const uint32_t (&k)[2], const float *ks, float e, float &m,
                                          float &l, float &a) {
  const uint64_t off2 = f2_pack(e - m, e - m);
  float x[64];
  tmem_ld32(s_tmem, reinterpret_cast<uint32_t *>(x));
  tmem_ld32(s_tmem + 32, reinterpret_cast<uint32_t *>(x) + 32);
  tmem_wait_ld();
#pragma unroll
  for (int i = 0; i < 64; ++i) asm volatile("" : "+f"(x[i]));
  float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const ulonglong2 f = reinterpret_cast<const ulonglong2 *>(ks)[i];
    f2_unpack(f2_fma(f2_pack(x[4 * i], x[4 * i + 1]), f.x, off2), x[4 * i], x[4 * i + 1]);
    f2_unpack(f2_fma(f2_pack(x[4 * i + 2], x[4 * i + 3]), f.y, off2), x[4 * i + 2], x[4 * i + 3]);
    if (kMasked) {
#pragma unroll
      for (int c = 0; c < 4; ++c)
        x[4 * i + c] = (k[i / 8] >> (4 * (i % 8) + c)) & 1 ? x[4 * i + c] : -INFINITY;
    }
    top[(2 * i) % 4] = fmax3(top[(2 * i) % 4], x[4 * i], x[4 * i + 1]);
    top[(2 * i + 1) % 4] = fmax3(top[(2 * i + 1) % 4], x[4 * i + 2], x[4 * i + 3]);
  }
  const float t = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
  const bool over = t > kQ8TileMost || (l == 0.f && t != -INFINITY);
  if (__any_sync(0xffffffffu, over)) {
    const float d = q8_move(t, over, m, l, a);
    const uint64_t d2 = f2_pack(d, d);
#pragma unroll
    for (int i = 0; i < 32; ++i)
      f2_unpack(f2_sub(f2_pack(x[2 * i], x[2 * i + 1]), d2), x[2 * i], x[2 * i + 1]);
  }
  uint64_t sum[2] = {0, 0};
  uint32_t pk[32];
#pragma unroll
  for (int i = 0; i < 32; ++i) {
    const float p0 = ex2(x[2 * i]), p1 = ex2(x[2 * i + 1]);
    sum[i % 2] = f2_add(sum[i % 2], f2_pack(p0, p1));
    pk[i] = pack_fp16x2(p0, p1);
  }
  tmem_st32(s_tmem, pk);
  tmem_wait_st();
  float u, v;
  f2_unpack(f2_add(sum[0], sum[1]), u, v);
  return u + v;
}

// The same for a wide tile, with an e per token and the row's own power of two; returns the sum of p 2^-e.  This form is rare: it reads
// the scores twice, four at a time in loops, so that neither its registers nor its instructions stand in
// the others' way (unrolled over 32 scores, tree_batch took 6% longer without ever coming here).
__device__ __forceinline__ float q8_weigh_wide(uint32_t s_tmem, const uint32_t (&k)[2], const float *ks,
                                               const float *es, float row_scale, float &m, float &l, float &a) {
  const uint64_t sees = (static_cast<uint64_t>(k[1]) << 32) | k[0];
  auto four = [&](int h, float (&x)[4], float (&e)[4]) {  // s + e - m, and e
    tmem_ld4(s_tmem + h, reinterpret_cast<uint32_t *>(x));
    tmem_wait_ld();
    const float4 f = *reinterpret_cast<const float4 *>(ks + h), g = *reinterpret_cast<const float4 *>(es + h);
    const float fs[4] = {f.x, f.y, f.z, f.w};
    e[0] = g.x, e[1] = g.y, e[2] = g.z, e[3] = g.w;
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      asm volatile("" : "+f"(x[c]));
      x[c] = (sees >> (h + c)) & 1 ? fmaf(x[c], fs[c] * row_scale, e[c] - m) : -INFINITY;
    }
  };
  float t = -INFINITY, sum = 0.f, x[4], e[4];
#pragma unroll 1
  for (int h = 0; h < kQ8Tok; h += 4) {
    four(h, x, e);
    t = fmax3(fmax3(t, x[0], x[1]), x[2], x[3]);
  }
  q8_move(t, t > kQ8TileMost || (l == 0.f && t != -INFINITY), m, l, a);
#pragma unroll 1
  for (int h = 0; h < kQ8Tok; h += 4) {
    four(h, x, e);
    uint32_t pk[2];
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      pk[c] = pack_fp16x2(ex2(x[2 * c]), ex2(x[2 * c + 1]));
      sum += ex2(x[2 * c] - e[2 * c]) + ex2(x[2 * c + 1] - e[2 * c + 1]);
    }
    tmem_st2(s_tmem + h / 2, pk);  // over scores that have been read
    tmem_wait_st();
  }
  return sum;
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

// S (TMEM, 64 columns) = Q K^T: both K-major in 64-feature swizzled chunks.
template <int HD>
__device__ __forceinline__ void q8_issue_qk(uint32_t d_tmem, const uint8_t *q, const uint8_t *k) {
  using C = Q8TileCfg<HD>;
  const uint64_t qd = smem_desc_sw128(smem_u32(q), 16, 1024), kd = smem_desc_sw128(smem_u32(k), 16, 1024);
#pragma unroll
  for (int kk = 0; kk < HD / 16; ++kk)
    umma_ss(d_tmem, qd + static_cast<uint64_t>(((kk / 4) * C::kQChunk + (kk % 4) * 32) >> 4),
            kd + static_cast<uint64_t>(((kk / 4) * C::kChunk + (kk % 4) * 32) >> 4), C::kIdescQK, kk > 0 ? 1u : 0u);
}

// O (TMEM) (+)= P V: P from TMEM (8 columns per 16 tokens), V MN-major (chunks of 64 features, 8-token
// groups).  P is not staged in shared memory: a product with both operands there reads the 128
// bytes a cycle that shared memory has, and P's stores would come on top.
template <int HD>
__device__ __forceinline__ void q8_issue_pv(uint32_t d_tmem, uint32_t p_tmem, const uint8_t *v, bool accumulate) {
  using C = Q8TileCfg<HD>;
  const uint64_t vd = smem_desc_sw128(smem_u32(v), C::kChunk, 1024);
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
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  constexpr int NK = kQ8KBufs, NV = kTwo ? 2 : kQ8MostVBufs, NC = kQ8CodeBufs, NS = C::kScaleBufs;
  uint8_t *sQ = smem;                          // [row tile]
  uint8_t *sK = sQ + (kTwo ? 2 : 1) * C::kQBytes;  // tile j of tokens is in [j % NK]
  uint8_t *sV = sK + NK * C::kTileBytes;       // [j % NV]
  uint8_t *sC = sV + NV * C::kTileBytes;       // [j % NC]: its codes, K then V, as they lie in the pool
  float *sKs = reinterpret_cast<float *>(sC + 2 * NC * C::kCodeBytes);  // [j % NS][token]: ks scale log2(e)
  uint32_t *sFt = reinterpret_cast<uint32_t *>(sKs + NS * kQ8Tok);      // [j % NS][token]: f in fp16, twice
  float *sE = reinterpret_cast<float *>(sFt + NS * kQ8Tok);             // [j % NS][token]: e, of a wide tile
  uint16_t *sLive = reinterpret_cast<uint16_t *>(sE + NS * kQ8Tok);     // [j % NS][page]
  uint16_t *sBad = sLive + NS * 4;             // [j % NS][page]: live tokens whose vs is not finite
  float *sTile = reinterpret_cast<float *>(sBad + NS * 4);  // [j % NS][4]: the tile's e, 2^-e, 1 if it is wide
  uint64_t *bars = reinterpret_cast<uint64_t *>(sTile + NS * 4);
  // Barriers are indexed as the buffers they guard; the counts are even (or every reader takes every
  // tile), so that a side that waits for every other tile of tokens sees each phase of its own.  A
  // buffer is freed by an arrival from each issuer (or converter warp) that reads it.
  uint64_t *k_full = bars, *k_free = k_full + NK, *v_full = k_free + NK, *v_free = v_full + NV;
  uint64_t *code_full = v_free + NV, *code_free = code_full + NC;
  uint64_t *sc_full = code_free + NC, *sc_free = sc_full + NS;
  uint64_t *s_full = sc_free + NS;              // [side][2]: the side's tile i uses [i & 1]
  uint64_t *p_full = s_full + 4;                // [side][2]
  uint64_t *pv_done = p_full + 4;               // [side][2]
  uint64_t *drain = pv_done + 4;                // [side] every product of an issuer has completed
  uint64_t *q_full = drain + 2;                 // [row tile]
  float *sTop = reinterpret_cast<float *>(bars + C::kBars);  // [8]: the warps' largest |q|
  float *sLow = sTop + 8;                       // [8]: and the smallest of their rows' largest, rows of 0 apart
  float *sRow = sLow + 8;                       // [row tile][128]: 1 / the row's own power of two, else 1
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(sRow + 256);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);

  unsigned u = blockIdx.x;
  const int split = u % p.n_split;
  u /= p.n_split;
  const int group = u % p.row_tiles;
  u /= p.row_tiles;
  const int kh = u % p.Hk;
  int s = u / p.Hk;
  if (p.longest_first) {
    // More than one round of CTAs, which start in the order of their index: the s-th longest sequence
    // (ties by index) instead of the s-th, so that the last round is short (32 sequences of 512 to 4096
    // tokens, 8 heads: 175 us in the batch's order, 125 so)
    __shared__ int lens[kQ8SortSeqs], found;
    if (threadIdx.x < p.S) lens[threadIdx.x] = q8_len(p, threadIdx.x);
    __syncthreads();
    if (threadIdx.x < p.S) {
      const int mine = lens[threadIdx.x];
      int rank = 0;
      for (int i = 0; i < p.S; ++i) rank += lens[i] > mine || (lens[i] == mine && i < static_cast<int>(threadIdx.x));
      if (rank == s) found = threadIdx.x;
    }
    __syncthreads();
    s = found;
  }
  const int row0 = group * (kTwo ? 256 : 128);
  const size_t row_base = (static_cast<size_t>(s) * p.Hk + kh) * p.R;
  const int L = q8_len(p, s);
  const int tiles_per_split = p.split_pages / kQ8TilePages;
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

  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  if (threadIdx.x == 0) {
    for (int i = 0; i < NK; ++i) mbar_init(k_full + i, 4), mbar_init(k_free + i, kTwo ? 2 : 1);
    for (int i = 0; i < NV; ++i) mbar_init(v_full + i, 4), mbar_init(v_free + i, kTwo ? 2 : 1);
    for (int i = 0; i < NC; ++i) mbar_init(code_full + i, 1), mbar_init(code_free + i, 4);
    // read by the four converter warps and by the softmax warps of each side
    for (int i = 0; i < NS; ++i) mbar_init(sc_full + i, 1), mbar_init(sc_free + i, kTwo ? 12 : 8);
    for (int i = 0; i < 4; ++i) {
      mbar_init(s_full + i, 1);
      mbar_init(p_full + i, 4);
      mbar_init(pv_done + i, 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(drain + i, 1);
      mbar_init(q_full + i, 4);
    }
    *abort_flag = 0;
    if (L != p.lens[s] && p.lens[s] > 0) atomicExch(&g_device_status, 1 /* FA_ERR_INVALID_ARG */);
    fence_mbar_init();
  }
  if (warp == 8) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  float row_top = 0.f;
  if (warp < 8) {
    const int row = row0 + (kTwo ? 128 * (warp / 4) : 0) + threadIdx.x % 128;
    if (row < p.R) {
      const uint4 *src = reinterpret_cast<const uint4 *>(p.q + (row_base + row) * HD);
#pragma unroll
      for (int c = 0; c < HD / 8; ++c) {
        const uint4 v = src[c];
        row_top = q8_finite_max(q8_finite_max(q8_finite_max(q8_finite_max(row_top, v.x), v.y), v.z), v.w);
      }
    }
    float top = row_top, low = row_top > 0.f ? row_top : INFINITY;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
      low = fminf(low, __shfl_xor_sync(0xffffffffu, low, off));
    }
    if (lane == 0) sTop[warp] = top, sLow[warp] = low;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  float q_top = sTop[0], q_low = sLow[0];
#pragma unroll
  for (int i = 1; i < 8; ++i) q_top = fmaxf(q_top, sTop[i]), q_low = fminf(q_low, sLow[i]);
  const bool rows_apart = q_low < q_top * kQ8RowsNear;
  const float q_unit = q8_q_unit(rows_apart && warp < 8 ? row_top : q_top);  // the CTA's or this thread's row's

  if (warp >= 8 && warp < 12) {
    // ------------------------------------------------------------------ codes -> fp16 tiles
    const int w = warp - 8;              // page w of a tile: tokens 16 w .. 16 w + 15
    constexpr int kPieces = HD / 8;      // 8-code pieces of a token
    constexpr int kRowsPer = 32 / kPieces;  // tokens that a warp-wide load covers
    constexpr int kLoads = kQ8Page / kRowsPer;
    constexpr int kSlab = kQ8Page * HD;
    const int piece = lane % kPieces, sub = lane / kPieces;
    const uint32_t at0 = static_cast<uint32_t>(piece / 8) * C::kChunk;
    const int unit = piece % 8;
    const uint8_t *mine_c = sC + w * kSlab + sub * HD + 8 * piece;
    // K runs one tile before V, as the products do
    for (int j = -1; j < nmax; ++j) {
      const int jk = j + 1;
      uint2 c[kLoads];
      if (jk < nmax) {
        if (!__all_sync(0xffffffffu, mbar_wait(code_full + jk % NC, (jk / NC) & 1, abort_flag) &&
                                         (jk < NK || mbar_wait(k_free + jk % NK, (jk / NK - 1) & 1, abort_flag)))) break;
        const uint8_t *src = mine_c + 2 * (jk % NC) * C::kCodeBytes;
#pragma unroll
        for (int i = 0; i < kLoads; ++i) c[i] = *reinterpret_cast<const uint2 *>(src + i * kRowsPer * HD);
        uint8_t *kt = sK + (jk % NK) * C::kTileBytes + at0;
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
          uint4 o;
          q8_cvt4<kType>(c[i].x, o.x, o.y);
          q8_cvt4<kType>(c[i].y, o.z, o.w);
          *reinterpret_cast<uint4 *>(kt + q8_swz(16 * w + i * kRowsPer + sub, unit)) = o;
        }
        fence_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(k_full + jk % NK);
      }
      if (j >= 0) {
        const int buf = j % NS;
        if (!__all_sync(0xffffffffu, mbar_wait(sc_full + buf, (j / NS) & 1, abort_flag) &&
                                         (j < NV || mbar_wait(v_free + j % NV, (j / NV - 1) & 1, abort_flag)))) break;
        const uint8_t *src = mine_c + (2 * (j % NC) + 1) * C::kCodeBytes;
        uint32_t f[kLoads];
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
          c[i] = *reinterpret_cast<const uint2 *>(src + i * kRowsPer * HD);
          f[i] = sFt[buf * kQ8Tok + 16 * w + i * kRowsPer + sub];
        }
        const uint32_t live = sLive[buf * 4 + w];
        __syncwarp();  // the tile's codes and scales have been read
        if (lane == 0) mbar_arrive(code_free + j % NC), mbar_arrive(sc_free + buf);
        // a slot that no token holds may have any bytes, and e4m3's NaN would pass through p = 0
        if (kType == kQ8E4m3 && live != 0xffffu) {
#pragma unroll
          for (int i = 0; i < kLoads; ++i)
            if (!((live >> (i * kRowsPer + sub)) & 1)) c[i] = make_uint2(0u, 0u);
        }
        uint8_t *vt = sV + (j % NV) * C::kTileBytes + at0;
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
          uint4 o;
          q8_cvt4<kType>(c[i].x, o.x, o.y);
          q8_cvt4<kType>(c[i].y, o.z, o.w);
          o = make_uint4(mul_fp16x2(o.x, f[i]), mul_fp16x2(o.y, f[i]), mul_fp16x2(o.z, f[i]), mul_fp16x2(o.w, f[i]));
          *reinterpret_cast<uint4 *>(vt + q8_swz(16 * w + i * kRowsPer + sub, unit)) = o;
        }
        fence_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(v_full + j % NV);
      }
    }
  } else if (warp >= 14) {
    // ------------------------------------------------------------------ codes and scales of the tiles
    const int32_t *trow = p.table + static_cast<size_t>(s) * p.max_blocks;
    const int nblk = (L + kQ8Page - 1) / kQ8Page;
    // lane i < 4: the table's entry for page i of tile j; not looked at before it is needed (named)
    auto has_page = [&](int j) {
      return lane < kQ8TilePages && j < nmax && (j0 + j) * kQ8TilePages + lane < nblk;
    };
    auto entry_of = [&](int j) -> int { return has_page(j) ? trow[(j0 + j) * kQ8TilePages + lane] : -1; };
    auto named = [&](int j, int b) -> int {  // -1 for a page that the table does not name
      if (b >= 0 && b < p.num_blocks) return b;
      if (has_page(j)) atomicExch(&g_device_status, 1 /* FA_ERR_INVALID_ARG: the page is left out */);
      return -1;
    };
    if (warp == 14) {
      // codes: lanes 0-3 a page of K each, lanes 4-7 of V; a page left out is not loaded (its tokens are
      // not live)
      constexpr uint32_t kSlab = kQ8Page * HD;  // a page of one head: contiguous in the pool
      int entry = entry_of(0);
      for (int j = 0; j < nmax; ++j) {
        const int blk = named(j, entry);
        entry = entry_of(j + 1);
        if (j >= NC && !__all_sync(0xffffffffu, mbar_wait(code_free + j % NC, (j / NC - 1) & 1, abort_flag))) break;
        const int pages = __popc(__ballot_sync(0xffffffffu, blk >= 0) & 0xfu);
        if (lane == 0) {
          if (pages > 0) mbar_arrive_expect_tx(code_full + j % NC, 2 * pages * kSlab);
          else mbar_arrive(code_full + j % NC);
        }
        __syncwarp();
        const int b = __shfl_sync(0xffffffffu, blk, lane & 3), is_v = (lane >> 2) & 1;
        if (lane < 8 && b >= 0)
          bulk_load_1d(sC + (2 * (j % NC) + is_v) * C::kCodeBytes + (lane & 3) * kSlab,
                       (is_v ? p.v_codes : p.k_codes) + (static_cast<size_t>(b) * p.Hk + kh) * kSlab, kSlab,
                       code_full + j % NC);
      }
      // abandoned: a copy still on its way lands before the CTA's shared memory goes away
      if (*abort_flag) {
        const uint64_t t0 = globaltimer_ns();
        while (globaltimer_ns() - t0 < 1000000) {
        }
      }
    } else {
      // scales: lane i < 16 has tokens 4 i .. 4 i + 3 of the tile
      const float score_scale = rows_apart ? p.scale_log2 : p.scale_log2 * q8_inverse(q_unit);
      float4 ks, vs;
      bool has = false;  // this lane's page is named
      int e_most = kQ8LeastE;
      int blk = named(0, entry_of(0)), entry = entry_of(1);
      auto fetch = [&](int b4) {
        const int b = __shfl_sync(0xffffffffu, b4, (lane / 4) & 3);
        const size_t at = (static_cast<size_t>(max(b, 0)) * p.Hk + kh) * kQ8Page + 4 * (lane % 4);
        ks = vs = make_float4(0.f, 0.f, 0.f, 0.f);
        has = b >= 0 && lane < 16;
        if (has) {
          ks = *reinterpret_cast<const float4 *>(p.ks + at);
          vs = *reinterpret_cast<const float4 *>(p.vs + at);
        }
      };
      fetch(blk);
      for (int j = 0; j < nmax; ++j) {
        const int buf = j % NS;
        const int left4 = L - (j0 + j) * kQ8Tok - 4 * lane;  // tokens from this lane's on, before the end
        float v[4] = {vs.x, vs.y, vs.z, vs.w};
        const float4 k4 = make_float4(ks.x * score_scale, ks.y * score_scale, ks.z * score_scale, ks.w * score_scale);
        const int left = L - (j0 + j) * kQ8Tok - kQ8Page * lane;  // and for lane i < 4, of page i
        const uint32_t live = blk < 0 || left <= 0 ? 0u : left >= 16 ? 0xffffu : (1u << left) - 1u;
        // The exponents of the tile's largest finite vs, and of its smallest (as 255 less it), in one word: 0
        // counts as the smallest, its token's weight would set the others' reference
        uint32_t range = 0;
        bool bad = false;  // a live token's vs is not finite
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const bool alive = has && c < left4;
          if (!alive) v[c] = 0.f;  // a slot past the end may hold anything
          const uint32_t x = q8_exponent(v[c]);
          bad = bad || x == 255u;
          range = __vmaxu2(range, alive && x != 255u ? (x << 16) + 255u - x : 0u);
        }
        blk = named(j + 1, entry);
        entry = entry_of(j + 2);
        fetch(blk);  // of tile j + 1
        if constexpr (!kTwo) {
          // and tile j + 2's as far as L2: this warp sets the pace where one row tile is all the work (128 rows
          // by 8192 tokens, one to an SM: 170 us without, 150 so; with two row tiles it does not)
          const int b = __shfl_sync(0xffffffffu, entry, (lane / 4) & 3);
          if (lane < 16 && lane % 4 == 0 && b >= 0 && b < p.num_blocks) {
            const size_t at = (static_cast<size_t>(b) * p.Hk + kh) * kQ8Page;
            asm volatile("prefetch.global.L2 [%0];" ::"l"(p.ks + at));
            asm volatile("prefetch.global.L2 [%0];" ::"l"(p.vs + at));
          }
        }
#pragma unroll
        for (int off = 8; off > 0; off >>= 1) range = __vmaxu2(range, __shfl_xor_sync(0xffffffffu, range, off));
        const int e_tile = q8_e(range >> 16);
        e_most = max(e_most, e_tile);
        const bool wide = q8_e(255u - (range & 0xffffu)) < e_tile - kQ8TileNear || e_tile < e_most - kQ8TileFar || rows_apart;
        uint32_t badmask = 0;  // of page `lane`
        if (__any_sync(0xffffffffu, bad)) {
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const uint32_t m = (__ballot_sync(0xffffffffu, !(fabsf(v[c]) < INFINITY)) >> (4 * (lane & 3))) & 0xfu;
            // lane i's token c is token 4 i + c of the page
            badmask |= ((m & 1u) | (m & 2u) << 3 | (m & 4u) << 6 | (m & 8u) << 9) << c;
            if (!(fabsf(v[c]) < INFINITY)) v[c] = 0.f;
          }
        }
        const float unit = q8_pow2(-e_tile) * q8_vtop<kType>();
        float x[4] = {v[0] * unit, v[1] * unit, v[2] * unit, v[3] * unit}, e4[4];
        if (wide) {
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const int e = q8_e(q8_exponent(v[c]));
            x[c] = v[c] * q8_pow2(-e) * q8_vtop<kType>();
            e4[c] = static_cast<float>(e);
          }
        }
        // A wait by parity must not be overtaken by a phase: the barrier's next one needs these scales.
        // (k_free of tile j - 4 would say as much, but Q K^T of tile j can complete before this wait.)
        if (j >= NS && !__all_sync(0xffffffffu, mbar_wait(sc_free + buf, (j / NS - 1) & 1, abort_flag))) break;
        if (lane < 16) {
          *reinterpret_cast<float4 *>(sKs + buf * kQ8Tok + 4 * lane) = k4;
          *reinterpret_cast<uint4 *>(sFt + buf * kQ8Tok + 4 * lane) = make_uint4(
              pack_fp16x2(x[0], x[0]), pack_fp16x2(x[1], x[1]), pack_fp16x2(x[2], x[2]), pack_fp16x2(x[3], x[3]));
          if (wide) *reinterpret_cast<float4 *>(sE + buf * kQ8Tok + 4 * lane) = make_float4(e4[0], e4[1], e4[2], e4[3]);
        }
        if (lane < kQ8TilePages) {
          sLive[buf * 4 + lane] = static_cast<uint16_t>(live);
          sBad[buf * 4 + lane] = static_cast<uint16_t>(badmask);
        }
        if (lane == 0)
          *reinterpret_cast<float4 *>(sTile + buf * 4) =
              make_float4(static_cast<float>(e_tile), q8_pow2(-e_tile), wide ? 1.f : 0.f, 0.f);
        __syncwarp();
        if (lane == 0) mbar_arrive(sc_full + buf);
      }
    }
  } else if (warp >= 12) {
    // ------------------------------------------------------------------ products: a thread per side
    const int side = warp - 12;
    if (side < 2 && lane == 0) {
      const int cnt = n[side], steps = kTwo ? nmax : cnt, rtile = kTwo ? side : 0;
      const uint32_t tS = tmem + 128 * side, tO = tmem + C::kColO + HD * side;
      // S of the side's tile i; with two row tiles an issuer also takes part for the tiles of tokens
      // that only the other one visits, by freeing them
      auto scores = [&](int i) -> bool {
        if (i >= steps) return true;
        const int j = kTwo ? i : 2 * i + side;
        if (!mbar_wait(k_full + j % NK, (j / NK) & 1, abort_flag)) return false;
        if (i < cnt) {
          tc_fence_after();
          q8_issue_qk<HD>(tS + 64 * (i & 1), sQ + rtile * C::kQBytes, sK + (j % NK) * C::kTileBytes);
          umma_commit(s_full + 2 * side + (i & 1));
          umma_commit(k_free + j % NK);
        } else {
          mbar_arrive(k_free + j % NK);
        }
        return true;
      };
      bool ok = (cnt == 0 || mbar_wait(q_full + rtile, 0, abort_flag)) && scores(0) && scores(1);
      for (int i = 0; ok && i < steps; ++i) {
        const int j = kTwo ? i : 2 * i + side;
        ok = mbar_wait(v_full + j % NV, (j / NV) & 1, abort_flag);
        if (!ok) break;
        if (i < cnt) {
          const int b = 2 * side + (i & 1);
          ok = mbar_wait(p_full + b, (i >> 1) & 1, abort_flag);
          if (!ok) break;
          tc_fence_after();
          q8_issue_pv<HD>(tO, tS + 64 * (i & 1), sV + (j % NV) * C::kTileBytes, i > 0);
          umma_commit(pv_done + b);
          umma_commit(v_free + j % NV);
          // P lies over S: tile i + 2's scores may be written once this product has read it
          ok = i + 2 >= cnt || mbar_wait(pv_done + b, (i >> 1) & 1, abort_flag);
        } else {
          mbar_arrive(v_free + j % NV);
          for (int w = 0; w < 4; ++w) mbar_arrive(sc_free + j % NS);  // for the side's softmax warps
        }
        ok = ok && scores(i + 2);
      }
      // every product issued here completes before tensor memory is given back
      umma_commit(drain + side);
      volatile int never = 0;
      mbar_wait(drain + side, 0, &never);
    }
  } else {
    // ------------------------------------------------------------------ softmax, epilogue
    const int side = warp / 4;
    const int rtile = kTwo ? side : 0;
    const int lrow = threadIdx.x % 128;
    const int row = row0 + 128 * rtile + lrow;
    const bool mine = row < p.R;
    const int cnt = n[side];
    const uint32_t lane_off = static_cast<uint32_t>((warp % 4) * 32) << 16;
    sRow[128 * rtile + lrow] = rows_apart ? q8_inverse(q_unit) : 1.f;  // (two threads of a row write the same)
    if (kTwo || side == 0) {  // this thread's row of q, in the layout the tensor core reads
      const uint16_t *src = p.q + (row_base + row) * HD;
      uint8_t *dst = sQ + rtile * C::kQBytes;
#pragma unroll
      for (int c = 0; c < HD / 8; ++c) {
        uint4 v = make_uint4(0u, 0u, 0u, 0u);
        if (mine) v = *reinterpret_cast<const uint4 *>(src + 8 * c);
        if constexpr (kType == kQ8Int8)
          v = make_uint4(__byte_perm(v.x, v.y, 0x5410), __byte_perm(v.x, v.y, 0x7632),
                         __byte_perm(v.z, v.w, 0x5410), __byte_perm(v.z, v.w, 0x7632));
        v = make_uint4(q8_fp16_of(v.x, q_unit), q8_fp16_of(v.y, q_unit), q8_fp16_of(v.z, q_unit),
                       q8_fp16_of(v.w, q_unit));
        *reinterpret_cast<uint4 *>(dst + (c / 8) * C::kQChunk + q8_swz(lrow, c % 8)) = v;
      }
      fence_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(q_full + rtile);
    }
    const uint32_t tS = tmem + 128 * side, tO = tmem + C::kColO + HD * side;
    const int t = mine ? row % p.T : 0;
    const int first_own = L - p.T;  // the first of the queries' own tokens
    const uint64_t bits = (p.tree && mine) ? p.tree[static_cast<size_t>(s) * p.T + t] : ~0ull;
    const bool warp_rows = row0 + 128 * rtile + (warp % 4) * 32 < p.R;  // any row in this warp
    float m = 0.f, l = 0.f;
    bool poison = false;  // the row sees a token whose values are no numbers
    bool ok = true;
    for (int i = 0; i < cnt; ++i) {
      const int j = kTwo ? i : 2 * i + side;  // the side's i-th tile of tokens
      const int buf = j % C::kScaleBufs, b = 2 * side + (i & 1);
      const float *ksb = sKs + buf * kQ8Tok;
      // warp-uniform, as the tensor-memory loads below are warp-wide
      if (!__all_sync(0xffffffffu, mbar_wait(sc_full + buf, (j / C::kScaleBufs) & 1, abort_flag) &&
                                       mbar_wait(s_full + b, (i >> 1) & 1, abort_flag))) { ok = false; break; }
      tc_fence_after();
      if (!warp_rows) {
        // rows past R: whatever P holds goes to O rows that nobody reads
        tc_fence_before();
        if (lane == 0) mbar_arrive(p_full + b), mbar_arrive(sc_free + buf);
        continue;
      }
      const int tok0 = (j0 + j) * kQ8Tok;
      const float4 tile = *reinterpret_cast<const float4 *>(sTile + buf * 4);
      uint32_t k[2];  // the tokens that this row sees
      {
        const uint2 live = *reinterpret_cast<const uint2 *>(sLive + buf * 4);
        k[0] = live.x, k[1] = live.y;
      }
      if ((p.causal || p.tree) && tok0 + kQ8Tok > first_own) {
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const int v0 = tok0 + 32 * c - first_own;  // the 32 tokens' first among the queries' own
          if (p.tree) {
            k[c] &= v0 >= 64 ? 0u : v0 >= 0 ? static_cast<uint32_t>(bits >> v0)
                    : v0 > -32 ? (static_cast<uint32_t>(bits << -v0) | ((1u << -v0) - 1u)) : ~0u;
          } else {
            const int lim = t - v0 + 1;
            k[c] &= lim >= 32 ? ~0u : lim <= 0 ? 0u : (1u << lim) - 1u;
          }
        }
      }
      const bool wide = tile.z != 0.f, all = __all_sync(0xffffffffu, (k[0] & k[1]) == 0xffffffffu && !wide);
      {
        const uint2 bad = *reinterpret_cast<const uint2 *>(sBad + buf * 4);
        poison = poison || ((k[0] & bad.x) | (k[1] & bad.y)) != 0;
      }
      float a = 1.f;  // what O is to be multiplied by
      const uint32_t ts = tS + lane_off + 64 * (i & 1);
      float sum;
      if (__builtin_expect(all, 1)) sum = tile.y * q8_weigh<false>(ts, k, ksb, tile.x, m, l, a);
      else if (__builtin_expect(!wide, 1)) sum = tile.y * q8_weigh<true>(ts, k, ksb, tile.x, m, l, a);
      else sum = q8_weigh_wide(ts, k, ksb, sE + buf * kQ8Tok, sRow[128 * rtile + lrow], m, l, a);
      if (i > 0 && __any_sync(0xffffffffu, a != 1.f)) {
        // the side's previous product must be in O before it is rescaled
        const int pb = 2 * side + ((i - 1) & 1);
        if (!__all_sync(0xffffffffu, mbar_wait(pv_done + pb, ((i - 1) >> 1) & 1, abort_flag))) { ok = false; break; }
        tc_fence_after();
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
      if (lane == 0) mbar_arrive(p_full + b), mbar_arrive(sc_free + buf);
    }
    const int last = cnt - 1;
    ok = __all_sync(0xffffffffu, ok && (cnt == 0 || mbar_wait(pv_done + 2 * side + (last & 1), (last >> 1) & 1,
                                                              abort_flag)));
    tc_fence_after();
    const float f = 1.f / q8_vtop<kType>();  // of O
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
      ok = ok && *abort_flag == 0;  // the other side's waits too
      if (side == 0 && warp_rows && ok) {
        const float m1 = xm[lrow], l1 = xm[128 + lrow];
        poison = poison || xm[256 + lrow] != 0.f;
        const float M = l == 0.f ? m1 : l1 == 0.f ? m : fmaxf(m, m1);
        const float a0 = l == 0.f ? 0.f : ex2(m - M), a1 = l1 == 0.f ? 0.f : ex2(m1 - M);
        const bool none = l == 0.f;
        l = (none ? 0.f : q8_shift(l, m - M)) + (l1 == 0.f ? 0.f : q8_shift(l1, m1 - M));
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
    // given up (and reported): nothing is written but what makes the joined rows NaN
    if (!ok && mine && p.n_split > 1) p.ws_ml[(row_base + row) * p.n_split + split] = q8_no_partial();
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
