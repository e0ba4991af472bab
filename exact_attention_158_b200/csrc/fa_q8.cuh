// fa_q8.cuh -- attention of few queries per sequence over an 8-bit paged cache (fa_cache.cuh), query
// heads sharing key/value heads: the decode step, and any call whose rows are few.
//
// The rows of one (sequence, key head) are its group = Hq / Hk query heads times T queries, R in
// all, numbered head * T + t: consecutive in q and o.  With K_j = ks_j k_j, V_j = vs_j v_j (codes k,
// v, one scale per token) and everything in log2 units,
//     s_rj = scale log2(e) ks_j (q_r . k_j),   p_rj = 2^(s_rj - m_r),
//     O_r = sum_j (p_rj vs_j) v_j / sum_j p_rj,   LSE_r = ln 2 (m_r + log2 sum_j p_rj):
// the codes go to the tensor cores exactly and the scales stay in fp32, the keys' on the scores and
// the values' on the probabilities.  For the second product p vs is rounded to fp16 (2^-11, against
// bf16's 2^-8); sums and statistics are fp32.
// The reference m_r is chosen for that product: the largest s + log2 vs so far, so that the largest
// p vs lies near 1 and fp16 loses 2^-25 of it at most, whatever the scales are.  It moves only when a
// p vs passes 2^10 (fp16 ends at 2^16) or the sum of p 2^112 (it is fp32, and a warp may add 2^16
// tokens).  A score holds the reference no further below itself than 2^96, which leaves the smallest
// scale the cache keeps, 2^-109, a p vs of 2^-13; a value of scale 0, which asks for no reference,
// 2^60: the further away, the coarser a score's fp32 difference to it (2^-19 there).
//
// Bound: HBM.  Each warp walks its own pages (16 tokens of one head: 16 d bytes of K, as many of V,
// 64 bytes of scales each), kept a few ahead in shared memory by TMA; a chunk of the context is
// shared by the four warps of a CTA and its partials are merged in shared memory.  The scores
// are computed transposed, S^T = K Q^T: 16 tokens are the rows and 8 query rows the columns of an
// m16n8k16 product, so a group of up to 8 query heads costs one product per 16 features where the
// direct form would pad the heads to 16.  O^T = V^T P^T likewise.  (The sm_100 tensor-core path
// wants 64 or 128 rows per product; with 1 to 32 rows it would multiply padding, and its operands
// would have to be converted through shared memory.)  64 sequences of 512 to 8192 tokens, 32 heads of
// 128: 372 us, 6500 GB/s, what a copy reaches; about 370 instructions per page and warp keep the
// schedulers half busy (52% of issue slots), so a power-capped clock shows (404 to 426 us back to back).
#pragma once
#include "sm100_ptx.cuh"

namespace fa {

constexpr int kQ8Page = 16;
constexpr int kQ8Warps = 4;
constexpr int kQ8Threads = 32 * kQ8Warps;
constexpr float kQ8MostPv = 0x1p10f, kQ8MostP = 0x1p112f;  // past these the reference moves
constexpr uint32_t kQ8MostPvBits = 0x6400u;                // 2^10 in fp16
constexpr float kQ8Far = 96.f, kQ8FarZero = 60.f;          // log2: how far below a score the reference may lie

enum Q8Type { kQ8E4m3 = 1, kQ8Int8 = 2 };

struct Q8Params {
  const uint16_t *q;
  const uint8_t *k_codes, *v_codes;  // [num_blocks, Hk, 16, d] (the tile kernel's; else tensor maps)
  const float *ks, *vs;              // [num_blocks, Hk, 16]
  const int32_t *table, *lens;
  const uint64_t *tree;  // [S, T] or null
  void *o;
  float *lse;
  float *ws_o;    // [S * Hk * R, n_split, d]: sum of p vs v, in units of the partial's own maximum
  float2 *ws_ml;  // [S * Hk * R, n_split]: m (log2 units) and the sum of p
  int S, Hq, Hk, T, R;
  int max_blocks, num_blocks;
  int row_tiles, n_split, split_pages;
  int causal, o_f32;
  int longest_first;  // the tile kernel's CTAs take the sequences by length
  float scale_log2;
};

// ---- codes to fp16 pairs ---------------------------------------------------------------------
// Both types are exact in fp16.  e4m3: the hardware's conversion, a pair at a time: lo takes bytes 0, 1
// of the word and hi bytes 2, 3.  int8: c is fp16's 1024 + (c + 128) less 1152; lo takes bytes 0, 2
// and hi bytes 1, 3.  q8_pick picks from two words what makes lo pair byte 0 (or 2) of the first with
// that of the second, and hi byte 1 (or 3).
__device__ __forceinline__ void q8_fp16_e4m3(uint32_t x, uint32_t &lo, uint32_t &hi) {
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(x));
}
__device__ __forceinline__ uint32_t q8_fp16_int8(uint32_t x) {
  uint32_t r;
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"((x & 0x00ff00ffu) ^ 0x64806480u), "r"(0x64806480u));
  return r;
}
template <int kType>
__device__ __forceinline__ void q8_cvt4(uint32_t x, uint32_t &lo, uint32_t &hi) {
  if constexpr (kType == kQ8E4m3) {
    q8_fp16_e4m3(x, lo, hi);
  } else {
    lo = q8_fp16_int8(x);
    hi = q8_fp16_int8(x >> 8);
  }
}
template <int kType>
__device__ __forceinline__ uint32_t q8_pick(uint32_t a, uint32_t b, int half) {
  if constexpr (kType == kQ8E4m3) return __byte_perm(a, b, half ? 0x7362 : 0x5140);
  return __byte_perm(a, b, half ? 0x7632 : 0x5410);
}

// Queries in fp16: a power of two, the row's own, brings its largest feature to 2^14, so that bf16's 8
// bits stay exact over 28 binades below it (and lose 2^-39 of it beyond); scores are divided by it.
__device__ __forceinline__ float q8_q_unit(float top) {  // of the largest finite |q|
  const uint32_t e = min(max((__float_as_uint(top) >> 23) & 0xffu, 15u), 254u);
  return __uint_as_float((254u + 14u - e) << 23);
}
__device__ __forceinline__ float q8_inverse(float u) {  // of a power of two
  return __uint_as_float((254u << 23) - __float_as_uint(u));
}
__device__ __forceinline__ float q8_finite_max(float top, uint32_t bf16x2) {
  const float a = fabsf(__uint_as_float(bf16x2 << 16)), b = fabsf(__uint_as_float(bf16x2 & 0xffff0000u));
  return fmaxf(top, fmaxf(a < INFINITY ? a : 0.f, b < INFINITY ? b : 0.f));
}

__device__ __forceinline__ void mma_fp16_16x8x16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                                 uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t pack_fp16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t max_fp16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t movmatrix_trans(uint32_t x) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}

__device__ __forceinline__ int q8_len(const Q8Params &p, int s) {
  const int hi = p.max_blocks * kQ8Page;
  int L = p.lens[s];
  if (L <= 0) return 0;  // an empty slot of a padded batch
  return L < p.T ? min(p.T, hi) : (L > hi ? hi : L);
}

template <int HD>
struct Q8Cfg {
  static constexpr int kSlab = kQ8Page * HD;              // bytes of one page of one head
  static constexpr int kStage = 2 * kSlab;
  // d = 128: three stages let four CTAs share an SM (16 warps, 200 KB in flight); with four stages
  // and three CTAs the same bytes are in flight but fewer warps compute (125 us against 118 for 16 x
  // 4096 tokens, 32 heads)
  static constexpr int kStages = HD == 128 ? 3 : 4;
  static constexpr int kRing = kQ8Warps * kStages * kStage;
  static constexpr int kScales = kQ8Warps * kStages * 2 * kQ8Page * 4;
  static constexpr int kBars = kQ8Warps * kStages * 8;
  static constexpr int kSmem = kRing + kScales + kBars + 1024;  // + alignment of the ring
};

// x 2^d for d <= 0.  For the sums l: they count scores against references that hold the values' scales too,
// so a reference may move by more than 2^126 (from values of scale 0 to loud ones) under a sum that stays a
// normal number, where 2^d alone does not.  (The output's sums follow the references: ex2(d) serves them.)
__device__ __forceinline__ float q8_shift(float x, float d) {
  const float half = ex2(0.5f * d);
  return x * half * half;
}

// ln 2 (M + log2 l).  M holds the values' log2 vs, which l undoes: l's exponent is added to M first
// (small numbers of opposite sign), and only the fraction's logarithm is approximated.
__device__ __forceinline__ float q8_lse(float M, float l) {
  if (l == 0.f) return -INFINITY;
  const int k = static_cast<int>((__float_as_uint(l) >> 23) & 0xffu) - 127;
  if (k == -127 || k == 128) return (M + lg2(l)) * 0.6931471805599453f;  // not a normal number
  const float f = __uint_as_float((__float_as_uint(l) & 0x007fffffu) | 0x3f800000u);
  return ((M + static_cast<float>(k)) + lg2(f)) * 0.6931471805599453f;
}

// (m, l) of a chunk whose CTA gave up a wait: it makes the rows that it is joined into NaN.
__device__ __forceinline__ float2 q8_no_partial() {
  const float nan = __int_as_float(0x7fc00000);
  return make_float2(nan, nan);
}

// Four features of an output row from its sums: O = a / l, LSE = ln 2 (M + log2 l); a row that saw
// no token has l = 0 and gets O = 0, LSE = -inf.
template <int HD>
__device__ __forceinline__ void q8_write4(const Q8Params &p, size_t row, int e0, const float4 &a, float M,
                                          float l) {
  const float inv = l == 0.f ? 0.f : 1.f / l;
  if (p.o_f32)
    *reinterpret_cast<float4 *>(static_cast<float *>(p.o) + row * HD + e0) =
        make_float4(a.x * inv, a.y * inv, a.z * inv, a.w * inv);
  else
    *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(p.o) + row * HD + e0) =
        make_uint2(pack_bf16x2(a.x * inv, a.y * inv), pack_bf16x2(a.z * inv, a.w * inv));
  if (e0 == 0 && p.lse) p.lse[row] = q8_lse(M, l);
}

// One CTA: one chunk of the context of one (sequence, key head), 8 NT query rows.  NT = 2 at d = 128 is held
// to 168 registers, three CTAs to an SM, and spills 20 bytes: 32 sequences of 2048 tokens, 8 key heads,
// 17 rows take 84 us so and 102 with two CTAs of 211 registers.
template <int HD, int NT, int kType>
__global__ void __launch_bounds__(kQ8Threads, (HD == 128 ? 5 : 6) - NT)
    fa_q8_stream_kernel(const __grid_constant__ CUtensorMap tk, const __grid_constant__ CUtensorMap tv,
                        const Q8Params p) {
  using C = Q8Cfg<HD>;
  constexpr int kUnits = HD / 64;   // 16-byte units of a K row that one lane takes
  constexpr int kVW = HD / 32;      // 4-byte words of a V row that one lane takes
  constexpr int kMT = HD / 16;      // 16-feature tiles of O^T
  constexpr int kRows = 8 * NT;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *ring = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  float *scales = reinterpret_cast<float *>(ring + C::kRing);
  uint64_t *bars = reinterpret_cast<uint64_t *>(ring + C::kRing + C::kScales);
  __shared__ int abort_flag;
  __shared__ float sm_m[kQ8Warps][kRows], sm_l[kQ8Warps][kRows];

  unsigned u = blockIdx.x;
  const int split = u % p.n_split;
  u /= p.n_split;
  const int tile = u % p.row_tiles;
  u /= p.row_tiles;
  const int kh = u % p.Hk, s = u / p.Hk;
  const int row0 = tile * kRows;
  const size_t row_base = (static_cast<size_t>(s) * p.Hk + kh) * p.R;  // of q, o, lse, partials

  const int L = q8_len(p, s);
  const int nblk = (L + kQ8Page - 1) / kQ8Page;
  const int pg0 = split * p.split_pages;
  const int pg1 = min(nblk, pg0 + p.split_pages);
  if (pg0 >= pg1 && !(split == 0 && p.n_split == 1)) return;  // past the sequence's end

  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int g = lane / 4, c = lane % 4;
  if (threadIdx.x == 0) {
    abort_flag = 0;
    if (L != p.lens[s] && p.lens[s] > 0) atomicExch(&g_device_status, 1 /* FA_ERR_INVALID_ARG */);
    for (int i = 0; i < kQ8Warps * C::kStages; ++i) mbar_init(bars + i, 1);
    fence_mbar_init();
  }
  __syncthreads();

  // q: column n = g of the score tile is row row0 + 8 nt + g; this lane holds the features that it
  // reads of K (units kUnits c + i, words w), paired as the conversion pairs codes
  uint32_t qb[NT][4 * kUnits][2];
  float sc[NT][2];  // score scale of the two rows (columns 2c, 2c + 1) whose scores this lane holds
  int tq[NT][2];    // and their query index t
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const int row = row0 + 8 * nt + g;
    const uint16_t *src = p.q + (row_base + row) * HD + 16 * kUnits * c;
    uint2 v[4 * kUnits];
    float top = 0.f;
#pragma unroll
    for (int k = 0; k < 4 * kUnits; ++k) {
      v[k] = make_uint2(0u, 0u);
      if (row < p.R) v[k] = *reinterpret_cast<const uint2 *>(src + 4 * k);
      top = q8_finite_max(q8_finite_max(top, v[k].x), v[k].y);
    }
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
    const float unit = q8_q_unit(top);
#pragma unroll
    for (int k = 0; k < 4 * kUnits; ++k) {
      const float f0 = __uint_as_float(v[k].x << 16) * unit, f1 = __uint_as_float(v[k].x & 0xffff0000u) * unit;
      const float f2 = __uint_as_float(v[k].y << 16) * unit, f3 = __uint_as_float(v[k].y & 0xffff0000u) * unit;
      qb[nt][k][0] = kType == kQ8E4m3 ? pack_fp16x2(f0, f1) : pack_fp16x2(f0, f2);
      qb[nt][k][1] = kType == kQ8E4m3 ? pack_fp16x2(f2, f3) : pack_fp16x2(f1, f3);
    }
    const float inv = p.scale_log2 * q8_inverse(unit);  // of row g: lane 4 g holds it
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      sc[nt][e] = __shfl_sync(0xffffffffu, inv, 4 * (2 * c + e));
      tq[nt][e] = (row0 + 8 * nt + 2 * c + e) % p.T;
    }
  }

  float acc[NT][kMT][4];
  float m[NT][2], l[NT][2];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
    for (int j = 0; j < kMT; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[nt][j][e] = 0.f;
    m[nt][0] = m[nt][1] = -INFINITY;
    l[nt][0] = l[nt][1] = 0.f;
  }

  uint8_t *my_ring = ring + warp * C::kStages * C::kStage;
  float *my_scales = scales + warp * C::kStages * 2 * kQ8Page;
  uint64_t *my_bars = bars + warp * C::kStages;
  const int32_t *trow = p.table + static_cast<size_t>(s) * p.max_blocks;
  const int n_mine = pg1 - pg0 > warp ? (pg1 - pg0 - warp + kQ8Warps - 1) / kQ8Warps : 0;

  // lane i holds the block of this warp's page (batch of 32) + i; bad entries become -1
  int tab = -1;
  auto fetch_table = [&](int first) {
    tab = -1;
    const int i = first + lane;
    if (i < n_mine) {
      tab = trow[pg0 + warp + kQ8Warps * i];
      if (tab < 0 || tab >= p.num_blocks) {
        atomicExch(&g_device_status, 1 /* FA_ERR_INVALID_ARG */);
        tab = -1;
      }
    }
  };
  // loads a page into a stage: lane 0 its K and key scales, lane 1 V; a page left out (-1) loads block 0
  auto issue = [&](int st, int blk) {
    if (lane < 2) {
      const int page = max(blk, 0) * p.Hk + kh;
      uint64_t *bar = my_bars + st;
      if (lane == 0) mbar_arrive_expect_tx(bar, C::kStage + 2 * kQ8Page * 4);
      tma_load_3d(my_ring + st * C::kStage + lane * C::kSlab, lane ? &tv : &tk, bar, 0, 0, page);
      bulk_load_1d(my_scales + (st * 2 + lane) * kQ8Page, (lane ? p.vs : p.ks) + static_cast<size_t>(page) * kQ8Page,
                   kQ8Page * 4, bar);
    }
  };
  // Blocks are fetched 32 pages at a time into `tab`, one batch ahead of the loads; `live` keeps a
  // bit per stage for pages that the table really names.
  fetch_table(0);
  uint32_t live = 0;
#pragma unroll 1
  for (int i = 0; i < C::kStages; ++i) {
    if (i < n_mine) {
      const int blk = __shfl_sync(0xffffffffu, tab, i);
      issue(i, blk);
      if (blk >= 0) live |= 1u << i;
    }
  }

  int st = 0;
  uint32_t phase = 0;
#pragma unroll 1
  for (int i = 0; i < n_mine; ++i) {
    if (!__all_sync(0xffffffffu, mbar_wait(my_bars + st, phase, &abort_flag))) {
      // given up: the pages asked for land (or this gives up too) before their memory is used again
      if (lane == 0) {
        volatile int never = 0;
        for (int k = i; k < min(i + C::kStages, n_mine); ++k) {
          mbar_wait(my_bars + st, phase, &never);
          if (++st == C::kStages) st = 0, phase ^= 1;
        }
      }
      break;
    }
    const uint8_t *kp = my_ring + st * C::kStage, *vp = kp + C::kSlab;
    const float *sp = my_scales + st * 2 * kQ8Page;
    const bool named = (live >> st) & 1;
    const int tok0 = (pg0 + warp + kQ8Warps * i) * kQ8Page;

    // K rows g and g + 8: unit kUnits c + i of a row lies at its swizzled place
    uint4 kr[2][kUnits];
#pragma unroll
    for (int r = 0; r < 2; ++r)
#pragma unroll
      for (int k = 0; k < kUnits; ++k) {
        const int row = g + 8 * r, unit = kUnits * c + k;
        const int at = HD == 128 ? (unit ^ (row & 7)) : (unit ^ ((row >> 1) & 3));
        kr[r][k] = *reinterpret_cast<const uint4 *>(kp + row * HD + 16 * at);
      }
    float kss[2], vss[2];
    bool in[2];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      in[r] = named && tok0 + g + 8 * r < L;
      kss[r] = in[r] ? sp[g + 8 * r] : 0.f;
      vss[r] = in[r] ? sp[kQ8Page + g + 8 * r] : 0.f;
    }
    float sa[NT][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 4; ++e) sa[nt][e] = 0.f;
#pragma unroll
    for (int k = 0; k < kUnits; ++k) {
      const uint32_t w0[4] = {kr[0][k].x, kr[0][k].y, kr[0][k].z, kr[0][k].w};
      const uint32_t w1[4] = {kr[1][k].x, kr[1][k].y, kr[1][k].z, kr[1][k].w};
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        uint32_t a0, a1, a2, a3;
        q8_cvt4<kType>(w0[w], a0, a2);
        q8_cvt4<kType>(w1[w], a1, a3);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
          mma_fp16_16x8x16(sa[nt], a0, a1, a2, a3, qb[nt][4 * k + w][0], qb[nt][4 * k + w][1]);
      }
    }
    // V: tokens 2c, 2c+1, 2c+8, 2c+9, features (HD / 8) g ..
    uint32_t vw[4][kVW];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int row = 2 * c + (r & 1) + 8 * (r >> 1);
      if constexpr (HD == 128) {
        const uint4 x = *reinterpret_cast<const uint4 *>(vp + row * HD + 16 * (g ^ (row & 7)));
        vw[r][0] = x.x, vw[r][1] = x.y, vw[r][2] = x.z, vw[r][3] = x.w;
      } else {
        const uint2 x = *reinterpret_cast<const uint2 *>(vp + row * HD + 16 * ((g >> 1) ^ ((row >> 1) & 3)) + 8 * (g & 1));
        vw[r][0] = x.x, vw[r][1] = x.y;
      }
    }
    // a slot past the sequence's end may hold any bytes, and e4m3's NaN would pass through p = 0
    if (kType == kQ8E4m3 && (!named || tok0 + kQ8Page > L)) {
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const bool keep = named && tok0 + 2 * c + (r & 1) + 8 * (r >> 1) < L;
#pragma unroll
        for (int w = 0; w < kVW; ++w) vw[r][w] = keep ? vw[r][w] : 0u;
      }
    }
    __syncwarp();  // every lane has read the stage: refill it
    {
      const int next = i + C::kStages;
      if ((next & 31) == 0) fetch_table(next);
      const int blk = __shfl_sync(0xffffffffu, tab, next & 31);
      live &= ~(1u << st);
      if (next < n_mine) {
        issue(st, blk);
        if (blk >= 0) live |= 1u << st;
      }
      if (++st == C::kStages) st = 0, phase ^= 1;
    }

    // scores: sa[nt][2 r + e] is token g + 8 r against query row 8 nt + 2 c + e
    // the page reaches the queries' own tokens, where the masks apply
    const bool edge = (p.causal || p.tree) && tok0 + kQ8Page > L - p.T;
    // most pages lie whole inside what every row sees: no masks
    const bool plain = named && tok0 + kQ8Page <= L && !edge;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int r = 0; r < 2; ++r)
#pragma unroll
        for (int e = 0; e < 2; ++e) sa[nt][2 * r + e] *= kss[r] * sc[nt][e];
    if (!plain) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            bool see = in[r];
            if (edge) {
              const int v = tok0 + g + 8 * r - (L - p.T);  // the token's place among the queries
              if (v >= 0 && see) {
                if (p.tree) see = (p.tree[static_cast<size_t>(s) * p.T + tq[nt][e]] >> (v & 63)) & 1;
                else if (p.causal) see = v <= tq[nt][e];
              }
            }
            if (!see) sa[nt][2 * r + e] = -INFINITY;
          }
    }
    float pv[NT][4], pw[NT][4], ln[NT][2];
    uint32_t pb[NT][2];
    auto weigh = [&]() {  // p and p vs against the present references; true when one passes its limit
      bool over = false;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          pw[nt][q] = ex2(sa[nt][q] - m[nt][q % 2]);
          pv[nt][q] = pw[nt][q] * vss[q / 2];
        }
        if (!plain) {
          // a token that a row does not see has no part in its sums, whatever its scales are
#pragma unroll
          for (int q = 0; q < 4; ++q)
            if (sa[nt][q] == -INFINITY) pw[nt][q] = pv[nt][q] = 0.f;
        }
        pb[nt][0] = pack_fp16x2(pv[nt][0], pv[nt][1]);
        pb[nt][1] = pack_fp16x2(pv[nt][2], pv[nt][3]);
        const uint32_t big = max_fp16x2(pb[nt][0], pb[nt][1]);
        over = over || (big & 0xffffu) > kQ8MostPvBits || (big >> 16) > kQ8MostPvBits;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          ln[nt][e] = l[nt][e] + (pw[nt][e] + pw[nt][2 + e]);
          over = over || ln[nt][e] > kQ8MostP;
        }
      }
      return over;
    };
    if (__any_sync(0xffffffffu, weigh())) {
      const float lv[2] = {lg2(vss[0]), lg2(vss[1])};  // -inf for scale 0
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const bool mine = ln[nt][e] > kQ8MostP || pv[nt][e] > kQ8MostPv || pv[nt][2 + e] > kQ8MostPv;
          float x = -INFINITY;
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const float y = sa[nt][2 * r + e];
            if (y != -INFINITY) x = fmaxf(x, lv[r] == -INFINITY ? y - kQ8FarZero : y + fmaxf(lv[r], -kQ8Far));
          }
          float go = mine ? 1.f : 0.f;
#pragma unroll
          for (int off = 4; off < 32; off <<= 1) {
            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, off));
            go = fmaxf(go, __shfl_xor_sync(0xffffffffu, go, off));
          }
          if (go == 0.f) continue;
          const float mn = fmaxf(m[nt][e], x);
          const bool first = m[nt][e] == -INFINITY;
          const float a = first ? 0.f : ex2(m[nt][e] - mn);
          l[nt][e] = first ? l[nt][e] * 0.f : q8_shift(l[nt][e], m[nt][e] - mn);
          m[nt][e] = mn;
#pragma unroll
          for (int j = 0; j < kMT; ++j) {
            acc[nt][j][e] *= a;
            acc[nt][j][2 + e] *= a;
          }
        }
      weigh();
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      l[nt][0] = ln[nt][0];
      l[nt][1] = ln[nt][1];
      pb[nt][0] = movmatrix_trans(pb[nt][0]);
      pb[nt][1] = movmatrix_trans(pb[nt][1]);
    }
#pragma unroll
    for (int w = 0; w < kVW; ++w) {
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        uint32_t a0, a1, a2, a3;
        q8_cvt4<kType>(q8_pick<kType>(vw[0][w], vw[1][w], half), a0, a1);
        q8_cvt4<kType>(q8_pick<kType>(vw[2][w], vw[3][w], half), a2, a3);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
          mma_fp16_16x8x16(acc[nt][2 * w + half], a0, a1, a2, a3, pb[nt][0], pb[nt][1]);
      }
    }
  }

  // merge the warps: lanes of the same c hold the same rows, their l parts over different tokens
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float x = l[nt][e];
#pragma unroll
      for (int off = 4; off < 32; off <<= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
      if (g == 0) {
        sm_m[warp][8 * nt + 2 * c + e] = m[nt][e];
        sm_l[warp][8 * nt + 2 * c + e] = x;
      }
    }
  __syncthreads();  // (no load is on its way any more: the ring is free)
  if (const volatile int *gave_up = &abort_flag; *gave_up) {
    // reported already; nothing is written but what makes the joined rows NaN
    if (p.n_split > 1 && threadIdx.x < kRows && row0 + static_cast<int>(threadIdx.x) < p.R)
      p.ws_ml[(row_base + row0 + threadIdx.x) * p.n_split + split] = q8_no_partial();
    return;
  }
  float *part = reinterpret_cast<float *>(ring);  // [warp][row][HD]
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int row = 8 * nt + 2 * c + e;
      float M = -INFINITY;
#pragma unroll
      for (int w = 0; w < kQ8Warps; ++w) M = fmaxf(M, sm_m[w][row]);
      // a warp that saw no token has l = 0 and takes no part; a NaN stays one
      const bool none = sm_l[warp][row] == 0.f;
      const float f = ex2(m[nt][e] - M);
      float *dst = part + (warp * kRows + row) * HD + (HD / 8) * g;
#pragma unroll
      for (int j = 0; j < kMT; ++j) {
        dst[2 * j] = none ? 0.f : acc[nt][j][e] * f;
        dst[2 * j + 1] = none ? 0.f : acc[nt][j][2 + e] * f;
      }
    }
  __syncthreads();
  constexpr int kPer = HD / 4;  // threads per row, 4 features each
  for (int i = threadIdx.x; i < kRows * kPer; i += kQ8Threads) {
    const int row = i / kPer, e0 = 4 * (i % kPer);
    if (row0 + row >= p.R) continue;
    float M = -INFINITY, sum = 0.f;
#pragma unroll
    for (int w = 0; w < kQ8Warps; ++w) M = fmaxf(M, sm_m[w][row]);
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < kQ8Warps; ++w) {
      if (sm_l[w][row] != 0.f) sum += q8_shift(sm_l[w][row], sm_m[w][row] - M);
      const float4 x = *reinterpret_cast<const float4 *>(part + (w * kRows + row) * HD + e0);
      a.x += x.x, a.y += x.y, a.z += x.z, a.w += x.w;
    }
    const size_t out = row_base + row0 + row;
    if (p.n_split > 1) {
      *reinterpret_cast<float4 *>(p.ws_o + (out * p.n_split + split) * HD + e0) = a;
      if (e0 == 0) p.ws_ml[out * p.n_split + split] = make_float2(M, sum);
      continue;
    }
    q8_write4<HD>(p, out, e0, a, M, sum);
  }
}

// Joins the chunks of every row: M = max m_c, l = sum 2^(m_c - M) l_c (q8_shift), O = sum 2^(m_c - M) O_c / l; a
// chunk without a visible token has l = 0 and takes no part.
//
// kWide: a CTA per row, for few rows or many chunks (one long context), where a thread that walked the
// chunks one after the other would wait for each (111 chunks: 60 us of a 175 us call).  The
// chunks' weights are made by all threads at once, then each warp sums every eighth chunk.
// Otherwise HD / 4 threads per row, each over all chunks.
constexpr int kQ8MaxSplit = 512;

template <int HD, bool kWide>
__global__ void __launch_bounds__(256) fa_q8_combine_kernel(const Q8Params p) {
  constexpr int kPer = HD / 4;
  const size_t rows = static_cast<size_t>(p.S) * p.Hk * p.R;
  const size_t row = kWide ? blockIdx.x : (static_cast<size_t>(blockIdx.x) * 256 + threadIdx.x) / kPer;
  if (row >= rows) return;
  const int s = static_cast<int>(row / (static_cast<size_t>(p.Hk) * p.R));
  const int nblk = (q8_len(p, s) + kQ8Page - 1) / kQ8Page;
  const int n = (nblk + p.split_pages - 1) / p.split_pages;
  const float2 *ml = p.ws_ml + row * p.n_split;
  const int e0 = 4 * static_cast<int>(threadIdx.x % kPer);
  const float *po = p.ws_o + row * p.n_split * HD + e0;
  float M = -INFINITY, sum = 0.f;
  float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
  auto add = [&](float f, const float4 &v) {
    a.x = fmaf(f, v.x, a.x), a.y = fmaf(f, v.y, a.y), a.z = fmaf(f, v.z, a.z), a.w = fmaf(f, v.w, a.w);
  };
  if constexpr (!kWide) {
    for (int i = 0; i < n; ++i) M = fmaxf(M, ml[i].x);
    for (int i = 0; i < n; ++i) {
      const float2 x = ml[i];
      if (x.y == 0.f) continue;
      const float f = ex2(x.x - M);
      sum += q8_shift(x.y, x.x - M);
      add(f, *reinterpret_cast<const float4 *>(po + static_cast<size_t>(i) * HD));
    }
    q8_write4<HD>(p, row, e0, a, M, sum);
  } else {
    constexpr int kGroups = 256 / kPer;  // groups of threads, each a whole row of features
    __shared__ float weight[kQ8MaxSplit], red[2][8];
    __shared__ float4 part[256];
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    for (int i = threadIdx.x; i < n; i += 256) M = fmaxf(M, ml[i].x);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, off));
    if (lane == 0) red[0][warp] = M;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < 8; ++w) M = fmaxf(M, red[0][w]);
    for (int i = threadIdx.x; i < n; i += 256) {
      const float2 x = ml[i];
      const float f = x.y == 0.f ? 0.f : ex2(x.x - M);
      weight[i] = f;
      if (x.y != 0.f) sum += q8_shift(x.y, x.x - M);
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
    if (lane == 0) red[1][warp] = sum;
    __syncthreads();
    sum = 0.f;
#pragma unroll
    for (int w = 0; w < 8; ++w) sum += red[1][w];
    // (a chunk with l = 0 wrote zeros: its weight of 0 does no harm)
#pragma unroll 4
    for (int i = threadIdx.x / kPer; i < n; i += kGroups)
      add(weight[i], *reinterpret_cast<const float4 *>(po + static_cast<size_t>(i) * HD));
    part[threadIdx.x] = a;
    __syncthreads();
    if (threadIdx.x < kPer) {
#pragma unroll
      for (int g = 1; g < kGroups; ++g) {
        const float4 x = part[threadIdx.x + g * kPer];
        a.x += x.x, a.y += x.y, a.z += x.z, a.w += x.w;
      }
      q8_write4<HD>(p, row, e0, a, M, sum);
    }
  }
}

}  // namespace fa
