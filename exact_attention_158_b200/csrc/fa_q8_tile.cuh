// fa_q8_tile.cuh -- attention of many rows (a prompt chunk, a draft tree, large groups) over an 8-bit
// paged cache on the tcgen05 tensor cores.  The mathematics, the scales' places and the row reference
// are those of fa_q8.cuh.
//
// One CTA takes up to 256 of the R rows of one (sequence, key head) and a range of its 128-token
// tiles.  Codes cannot feed a 16-bit product, so they are converted once per tile for all of the
// CTA's rows:
//   warps 0-3    row tile 0: one TMEM lane = one row.  Scores out of TMEM, p and p vs, P to shared
//   warps 4-7    row tile 1: the same; idle with one row tile (kTwo = false)
//   warps 8-11   codes: global (two 16-bit-wide tiles ahead in registers) -> bf16 K / fp16 V tiles in
//                the swizzled layout the tensor core reads; the tile's scales and its live tokens
//   warp  12     tensor-memory owner and issuer of every product (one thread)
// The conversion leaves every four features in the order 0, 2, 1, 3; q is stored in that order too, and
// O's columns are put back when it is written.
// TMEM (512 columns): S0 [0,128)  S1 [128,256)  O0 [256,256+d)  O1 [256+d,256+2d).
// With two row tiles the products of one run while the other's softmax does.  With one, its tiles
// alternate between the two S and P buffers: Q K^T of tile j + 1 runs during the softmax of tile j.
//
// A row's softmax is one pass: p = 2^(s ks - m) with the reference it has, summed and multiplied by vs
// on the way to P; only when a limit is passed (always on a row's first tile) the warp goes back to S,
// moves the references, rescales O in TMEM and does the pass again.
//
// Bound: per 128 x 128 scores the products take about 1020 cycles at d = 128, the exponentials 1020
// (16 a cycle), the conversion's instructions 600 per tile of tokens and the softmax's 550 per row
// tile on each of the SM's four schedulers, and the tile's 32 KB of codes about 1400 cycles of the
// SM's share of HBM: few rows are bound by HBM, many by the tensor cores and the exponentials.
#pragma once
#include "fa_q8.cuh"

namespace fa {

constexpr int kQ8TileThreads = 13 * 32;
constexpr int kQ8Tok = 128;  // tokens of a tile

template <int HD>
struct Q8TileCfg {
  static constexpr int kChunks = HD / 64;             // 64-feature (128-byte) swizzle chunks
  static constexpr int kChunkBytes = 128 * 128;       // 128 rows x 128 bytes
  static constexpr int kTileBytes = kChunks * kChunkBytes;
  static constexpr int kPBytes = 2 * kChunkBytes;     // 128 x 128 fp16
  static constexpr int kScaleBufs = 4;
  static constexpr int kBars = 24;
  static constexpr size_t kSmem = 1024 + 2 * kTileBytes + 2 * kTileBytes + 2 * kPBytes +
                                  kScaleBufs * (2 * kQ8Tok * 4 + 16) + kBars * 8 + 16;
  static constexpr uint32_t kColS = 0, kColO = 256;
  static constexpr uint32_t kIdescQK = idesc_bf16_f32(128, 128, 0, 0);
  // fp16 operands: the type fields of A and B are 0
  static constexpr uint32_t kIdescPV = idesc_bf16_f32(128, HD, 0, 1) & ~((1u << 7) | (1u << 10));
  static_assert(kSmem <= 227 * 1024, "shared memory budget");
  static_assert(kSmem > 114 * 1024, "one CTA per SM: it takes all of the tensor memory");
};

// 16-byte unit `unit` of row `row` in a 128-byte-swizzled chunk.
__device__ __forceinline__ uint32_t q8_swz(int row, int unit) {
  return static_cast<uint32_t>(row * 128 + ((unit ^ (row & 7)) << 4));
}

// Keeps uses of registers that a tcgen05.ld fills behind the wait that precedes this.
__device__ __forceinline__ void q8_pin(float (&x)[32]) {
#pragma unroll
  for (int i = 0; i < 32; ++i) asm volatile("" : "+f"(x[i]));
}

// Token tiles that the rows [r0, r1) can see: all of them, or up to the last row's own token.
__device__ __forceinline__ int q8_tiles(const Q8Params &p, int L, int r0, int r1) {
  if (r1 <= r0 || L == 0) return 0;
  if (!p.causal) return (L + kQ8Tok - 1) / kQ8Tok;
  const int t0 = r0 % p.T;
  const int t = t0 + (r1 - r0) - 1 < p.T ? t0 + (r1 - r0) - 1 : p.T - 1;
  return (L - p.T + t) / kQ8Tok + 1;
}

template <int HD, int kType, bool kTwo>
__global__ void __launch_bounds__(kQ8TileThreads, 1) fa_q8_tile_kernel(const Q8Params p) {
  using C = Q8TileCfg<HD>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint8_t *sQ = smem;
  uint8_t *sK = sQ + 2 * C::kTileBytes;
  uint8_t *sV = sK + C::kTileBytes;
  uint8_t *sP = sV + C::kTileBytes;
  float *sKs = reinterpret_cast<float *>(sP + 2 * C::kPBytes);  // [buffer][token]: ks scale log2(e)
  float *sVs = sKs + C::kScaleBufs * kQ8Tok;
  uint32_t *sLive = reinterpret_cast<uint32_t *>(sVs + C::kScaleBufs * kQ8Tok);  // [buffer][4]
  uint64_t *bars = reinterpret_cast<uint64_t *>(sLive + C::kScaleBufs * 4);
  uint64_t *q_full = bars, *k_full = bars + 1, *k_free = bars + 2, *v_full = bars + 3, *v_free = bars + 4;
  uint64_t *sc_full = bars + 5;            // [4]
  uint64_t *s_full = bars + 9;             // [2]
  uint64_t *p_full = bars + 11;            // [2]
  uint64_t *pv_done = bars + 13;           // [2]
  uint64_t *drain = bars + 15;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + C::kBars);
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
  int n[2];  // tiles of this range that each row tile visits
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int r0 = row0 + 128 * i;
    const int all = (i == 1 && !kTwo) ? 0 : q8_tiles(p, L, r0, min(r0 + 128, p.R));
    n[i] = max(0, min(all, j0 + tiles_per_split) - j0);
  }
  const int nmax = max(n[0], n[1]);

  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  if (threadIdx.x == 0) {
    mbar_init(q_full, kTwo ? 8 : 4);
    mbar_init(k_full, 4);
    mbar_init(k_free, 1);
    mbar_init(v_full, 4);
    mbar_init(v_free, 1);
    for (int i = 0; i < 4; ++i) mbar_init(sc_full + i, 4);
    for (int i = 0; i < 2; ++i) {
      mbar_init(s_full + i, 1);
      mbar_init(p_full + i, 4);
      mbar_init(pv_done + i, 1);
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    if (L != p.lens[s] && p.lens[s] > 0) atomicExch(&g_device_status, 1 /* FA_ERR_INVALID_ARG */);
    fence_mbar_init();
  }
  if (warp == 12) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (warp >= 8 && warp < 12) {
    // ------------------------------------------------------------------ codes -> 16-bit tiles
    const int w = warp - 8;              // tokens 32 w .. 32 w + 31 of a tile: pages 2 w, 2 w + 1
    constexpr int kPieces = HD / 8;      // 8-code pieces of a token
    constexpr int kRowsPer = 32 / kPieces;  // tokens that a warp-wide load covers
    constexpr int kLoads = 32 / kRowsPer;
    const int piece = lane % kPieces, sub = lane / kPieces;
    const int32_t *trow = p.table + static_cast<size_t>(s) * p.max_blocks;
    const int nblk = (L + kQ8Page - 1) / kQ8Page;
    auto block_of = [&](int j) -> int {  // lanes 0-15: the warp's first page, 16-31: its second
      const int page = (j0 + j) * (kQ8Tok / kQ8Page) + 2 * w + lane / 16;
      if (j >= nmax || page >= nblk) return -1;
      int b = trow[page];
      if (b < 0 || b >= p.num_blocks) {
        atomicExch(&g_device_status, 1 /* FA_ERR_INVALID_ARG: the page is left out */);
        b = -1;
      }
      return b;
    };
    const uint8_t *kcodes = p.k_codes + static_cast<size_t>(kh) * kQ8Page * HD;
    const uint8_t *vcodes = p.v_codes + static_cast<size_t>(kh) * kQ8Page * HD;
    const size_t block_stride = static_cast<size_t>(p.Hk) * kQ8Page * HD;
    uint2 kc[kLoads], vc[kLoads];
    // a page left out reads block 0: its tokens are not live
    auto fetch = [&](const uint8_t *codes, int blk, uint2 (&c)[kLoads]) {
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const int b = max(__shfl_sync(0xffffffffu, blk, 16 * half), 0);
        const uint8_t *src = codes + static_cast<size_t>(b) * block_stride + sub * HD + 8 * piece;
#pragma unroll
        for (int k = 0; k < kLoads / 2; ++k) {
          asm volatile("ld.global.nc.L1::no_allocate.v2.u32 {%0,%1}, [%2];"
                       : "=r"(c[half * (kLoads / 2) + k].x), "=r"(c[half * (kLoads / 2) + k].y)
                       : "l"(src + k * kRowsPer * HD));
        }
      }
    };
    const uint32_t chunk_at = static_cast<uint32_t>(piece / 8) * C::kChunkBytes;
    const int unit = piece % 8;
    float ks = 0.f, vs = 0.f;
    bool in = false;
    auto fetch_scales = [&](int j, int blk) {  // token 32 w + lane, of the page that its half warp holds
      in = blk >= 0 && (j0 + j) * kQ8Tok + 32 * w + lane < L;
      ks = vs = 0.f;
      if (in) {
        const size_t at = (static_cast<size_t>(blk) * p.Hk + kh) * kQ8Page + lane % 16;
        ks = p.ks[at];
        vs = p.vs[at];
      }
    };
    const float score_scale = p.scale_log2 * q8_score_unit<kType>();
    int blk = block_of(0), blk_next = block_of(1);
    if (nmax > 0) {
      fetch(kcodes, blk, kc);
      fetch_scales(0, blk);
      fetch(vcodes, blk, vc);
    }
    for (int j = 0; j < nmax; ++j) {
      if (j > 0 && !__all_sync(0xffffffffu, mbar_wait(k_free, (j - 1) & 1, abort_flag))) break;
      const int buf = j % C::kScaleBufs;
      sKs[buf * kQ8Tok + 32 * w + lane] = ks * score_scale;
      sVs[buf * kQ8Tok + 32 * w + lane] = vs;
      const uint32_t live = __ballot_sync(0xffffffffu, in);
      if (lane == 0) sLive[buf * 4 + w] = live;
#pragma unroll
      for (int k = 0; k < kLoads; ++k) {
        const int row = 32 * w + k * kRowsPer + sub;
        uint4 o;
        q8_key4<kType>(kc[k].x, o.x, o.y);
        q8_key4<kType>(kc[k].y, o.z, o.w);
        *reinterpret_cast<uint4 *>(sK + chunk_at + q8_swz(row, unit)) = o;
      }
      fence_async_smem();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(sc_full + buf);
        mbar_arrive(k_full);
      }
      blk = blk_next;
      blk_next = block_of(j + 2);
      if (j + 1 < nmax) {
        fetch(kcodes, blk, kc);
        fetch_scales(j + 1, blk);
      }
      if (j > 0 && !__all_sync(0xffffffffu, mbar_wait(v_free, (j - 1) & 1, abort_flag))) break;
#pragma unroll
      for (int k = 0; k < kLoads; ++k) {
        const int row = 32 * w + k * kRowsPer + sub;
        uint4 o;
        q8_value4<kType>(vc[k].x, o.x, o.y);
        q8_value4<kType>(vc[k].y, o.z, o.w);
        *reinterpret_cast<uint4 *>(sV + chunk_at + q8_swz(row, unit)) = o;
      }
      fence_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(v_full);
      if (j + 1 < nmax) fetch(vcodes, blk, vc);
    }
  } else if (warp == 12) {
    // ------------------------------------------------------------------ products (one thread)
    if (lane == 0) {
      const uint64_t kd = smem_desc_sw128(smem_u32(sK), 16, 1024);
      const uint64_t vd = smem_desc_sw128(smem_u32(sV), C::kChunkBytes, 1024);
      auto qk = [&](int tile, int slot) {
        const uint64_t qd = smem_desc_sw128(smem_u32(sQ + tile * C::kTileBytes), 16, 1024);
#pragma unroll
        for (int kk = 0; kk < HD / 16; ++kk) {
          const uint64_t off = static_cast<uint64_t>(((kk / 4) * C::kChunkBytes + (kk % 4) * 32) >> 4);
          umma_ss(tmem + C::kColS + 128 * slot, qd + off, kd + off, C::kIdescQK, kk > 0 ? 1u : 0u);
        }
        umma_commit(s_full + slot);
      };
      auto pv = [&](int tile, int slot, bool accumulate) {
        const uint64_t pd = smem_desc_sw128(smem_u32(sP + slot * C::kPBytes), 16, 1024);
#pragma unroll
        for (int kk = 0; kk < kQ8Tok / 16; ++kk) {
          const uint64_t off = static_cast<uint64_t>(((kk / 4) * C::kChunkBytes + (kk % 4) * 32) >> 4);
          umma_ss(tmem + C::kColO + HD * tile, pd + off, vd + static_cast<uint64_t>((kk * 16 * 128) >> 4),
                  C::kIdescPV, (accumulate || kk > 0) ? 1u : 0u);
        }
        umma_commit(pv_done + slot);
      };
      bool ok = nmax > 0 && mbar_wait(q_full, 0, abort_flag) && mbar_wait(k_full, 0, abort_flag);
      if (ok) {
        tc_fence_after();
#pragma unroll
        for (int i = 0; i < (kTwo ? 2 : 1); ++i)
          if (n[i] > 0) qk(i, i);
        umma_commit(k_free);
      }
      for (int j = 0; ok && j < nmax; ++j) {
        if constexpr (kTwo) {
          for (int i = 0; ok && i < 2; ++i) {
            if (j >= n[i]) continue;
            ok = mbar_wait(p_full + i, j & 1, abort_flag) && mbar_wait(v_full, j & 1, abort_flag);
            if (!ok) break;
            tc_fence_after();
            pv(i, i, j > 0);
            if (j + 1 < n[i]) {  // S_i has been read: its P is here
              ok = mbar_wait(k_full, (j + 1) & 1, abort_flag);
              if (!ok) break;
              tc_fence_after();
              qk(i, i);
            }
          }
          if (!ok) break;
          umma_commit(v_free);
          if (j + 1 < nmax) umma_commit(k_free);
        } else {
          if (j + 1 < nmax) {  // S of the other slot was read when P_{j-1} came
            ok = mbar_wait(k_full, (j + 1) & 1, abort_flag);
            if (!ok) break;
            tc_fence_after();
            qk(0, (j + 1) & 1);
            umma_commit(k_free);
          }
          ok = mbar_wait(p_full + (j & 1), (j >> 1) & 1, abort_flag) && mbar_wait(v_full, j & 1, abort_flag);
          if (!ok) break;
          tc_fence_after();
          pv(0, j & 1, j > 0);
          umma_commit(v_free);
        }
      }
      // every product issued here completes before tensor memory is given back
      umma_commit(drain);
      volatile int never = 0;
      mbar_wait(drain, 0, &never);
    }
  } else if (kTwo || warp < 4) {
    // ------------------------------------------------------------------ softmax, epilogue
    const int tile = warp / 4;
    const int lrow = threadIdx.x % 128;
    const int row = row0 + 128 * tile + lrow;
    const bool mine = row < p.R;
    const int nt = n[tile];
    const uint32_t lane_off = static_cast<uint32_t>((warp % 4) * 32) << 16;
    {  // this thread's row of q, in the layout the tensor core reads
      const uint16_t *src = p.q + (row_base + row) * HD;
      uint8_t *dst = sQ + tile * C::kTileBytes;
#pragma unroll
      for (int c = 0; c < HD / 8; ++c) {
        uint4 v = make_uint4(0u, 0u, 0u, 0u);
        if (mine) v = *reinterpret_cast<const uint4 *>(src + 8 * c);
        v = make_uint4(__byte_perm(v.x, v.y, 0x5410), __byte_perm(v.x, v.y, 0x7632),
                       __byte_perm(v.z, v.w, 0x5410), __byte_perm(v.z, v.w, 0x7632));
        if constexpr (kType == kQ8E4m3)
          v = make_uint4(q8_scale_q(v.x), q8_scale_q(v.y), q8_scale_q(v.z), q8_scale_q(v.w));
        *reinterpret_cast<uint4 *>(dst + (c / 8) * C::kChunkBytes + q8_swz(lrow, c % 8)) = v;
      }
      fence_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(q_full);
    }
    const int t = mine ? row % p.T : 0;
    const int first_own = L - p.T;  // the first of the queries' own tokens
    const uint64_t bits = (p.tree && mine) ? p.tree[static_cast<size_t>(s) * p.T + t] : ~0ull;
    const bool warp_rows = row0 + 128 * tile + (warp % 4) * 32 < p.R;  // any row in this warp
    float m = -INFINITY, l = 0.f;
    const uint32_t tO = tmem + lane_off + C::kColO + HD * tile;
    bool ok = true;
    for (int j = 0; j < nt; ++j) {
      const int slot = kTwo ? tile : (j & 1);
      const uint32_t use = kTwo ? j : (j >> 1);  // how often the slot was used before
      const uint32_t tS = tmem + lane_off + C::kColS + 128 * slot;
      uint8_t *pt = sP + slot * C::kPBytes;
      const int buf = j % C::kScaleBufs;
      const float *ksb = sKs + buf * kQ8Tok, *vsb = sVs + buf * kQ8Tok;
      // warp-uniform, as the tensor-memory loads below are warp-wide
      if (!__all_sync(0xffffffffu, mbar_wait(sc_full + buf, (j / C::kScaleBufs) & 1, abort_flag) &&
                                       mbar_wait(s_full + slot, use & 1, abort_flag))) { ok = false; break; }
      if (use > 0 && !__all_sync(0xffffffffu, mbar_wait(pv_done + slot, (use - 1) & 1, abort_flag))) { ok = false; break; }
      tc_fence_after();
      if (!warp_rows) {
        // rows past R: whatever P holds goes to O rows that nobody reads
        tc_fence_before();
        if (lane == 0) mbar_arrive(p_full + slot);
        continue;
      }
      const int tok0 = (j0 + j) * kQ8Tok;
      // which of the 32 tokens from tok0 + 32 c this row sees
      auto seen = [&](int c) -> uint32_t {
        uint32_t k = sLive[buf * 4 + c];
        const int v0 = tok0 + 32 * c - first_own;
        if (v0 + 31 >= 0) {
          if (p.tree) {
            const uint32_t b = v0 >= 64 ? 0u : v0 >= 0 ? static_cast<uint32_t>(bits >> v0)
                                                       : (static_cast<uint32_t>(bits << -v0) | ((1u << -v0) - 1u));
            k &= b;
          } else if (p.causal) {
            const int lim = t - v0 + 1;
            k &= lim >= 32 ? ~0u : lim <= 0 ? 0u : (1u << lim) - 1u;
          }
        }
        return k;
      };
      float sum, most;
      auto pass = [&]() {  // p and p vs of the tile against the present reference; P to shared memory
        const float neg = -m;
        const uint64_t neg2 = f2_pack(neg, neg);
        uint64_t sum2 = 0;
        most = 0.f;
        float sc[2][32];
        tmem_ld32(tS, reinterpret_cast<uint32_t *>(sc[0]));
        tmem_wait_ld();
        q8_pin(sc[0]);
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          if (c < 3) tmem_ld32(tS + 32 * (c + 1), reinterpret_cast<uint32_t *>(sc[(c + 1) & 1]));
          const float(&x)[32] = sc[c & 1];
          const uint32_t k = seen(c);
          const bool some = __any_sync(0xffffffffu, k != 0xffffffffu);
#pragma unroll
          for (int e8 = 0; e8 < 4; ++e8) {
            uint32_t pk[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int i = 8 * e8 + 2 * e;
              const ulonglong2 ks4 = *reinterpret_cast<const ulonglong2 *>(ksb + 32 * c + (i & ~3));
              const ulonglong2 vs4 = *reinterpret_cast<const ulonglong2 *>(vsb + 32 * c + (i & ~3));
              const uint64_t ks2 = e & 1 ? ks4.y : ks4.x, vs2 = e & 1 ? vs4.y : vs4.x;
              float y0, y1;
              f2_unpack(f2_fma(f2_pack(x[i], x[i + 1]), ks2, neg2), y0, y1);
              if (some) {
                y0 = (k >> i) & 1 ? y0 : -INFINITY;
                y1 = (k >> (i + 1)) & 1 ? y1 : -INFINITY;
              }
              const uint64_t w2 = f2_pack(ex2(y0), ex2(y1));
              sum2 = f2_add(sum2, w2);
              float v0, v1;
              f2_unpack(f2_mul(w2, vs2), v0, v1);
              if (some) {  // a token that is not seen may hold a scale that is not a number
                v0 = (k >> i) & 1 ? v0 : 0.f;
                v1 = (k >> (i + 1)) & 1 ? v1 : 0.f;
              }
              most = fmax3(most, v0, v1);
              pk[e] = pack_fp16x2(v0, v1);
            }
            *reinterpret_cast<uint4 *>(pt + (c / 2) * C::kChunkBytes + q8_swz(lrow, 4 * (c & 1) + e8)) =
                make_uint4(pk[0], pk[1], pk[2], pk[3]);
          }
          if (c < 3) {
            tmem_wait_ld();
            q8_pin(sc[(c + 1) & 1]);
          }
        }
        float s0, s1;
        f2_unpack(sum2, s0, s1);
        sum = s0 + s1;
      };
      bool over = true;
      if (j > 0) {
        pass();
        over = sum > kQ8MostP || most > kQ8MostPv;
      }
      if (__any_sync(0xffffffffu, over)) {
        float x = -INFINITY;
#pragma unroll 1
        for (int c = 0; c < 4; ++c) {
          float sc[32];
          tmem_ld32(tS + 32 * c, reinterpret_cast<uint32_t *>(sc));
          const uint32_t k = seen(c);
          tmem_wait_ld();
          q8_pin(sc);
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            const float y = sc[i] * ksb[32 * c + i];
            if ((k >> i) & 1) x = fmaxf(x, fmaxf(y - kQ8Slack, y + lg2(vsb[32 * c + i])));
          }
        }
        const float a = !over ? 1.f : m == -INFINITY ? 0.f : ex2(m - x);
        if (over) m = x;
        l *= a;
        if (j > 0) {
          // the previous tile's product must be in O before it is rescaled
          const int ps = kTwo ? tile : ((j - 1) & 1);
          const uint32_t pu = kTwo ? j - 1 : ((j - 1) >> 1);
          if (!__all_sync(0xffffffffu, mbar_wait(pv_done + ps, pu & 1, abort_flag))) { ok = false; break; }
          tc_fence_after();
#pragma unroll 1
          for (int c = 0; c < HD; c += 32) {
            float o[32];
            tmem_ld32(tO + c, reinterpret_cast<uint32_t *>(o));
            tmem_wait_ld();
            q8_pin(o);
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] *= a;
            tmem_st32(tO + c, reinterpret_cast<uint32_t *>(o));
            tmem_wait_st();
          }
        }
        pass();
      }
      l += sum;
      tc_fence_before();
      fence_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(p_full + slot);
    }
    if (ok && nt > 0) {
      const int last = nt - 1;
      const int ps = kTwo ? tile : (last & 1);
      const uint32_t pu = kTwo ? last : (last >> 1);
      ok = __all_sync(0xffffffffu, mbar_wait(pv_done + ps, pu & 1, abort_flag));
      tc_fence_after();
    }
    if (ok && warp_rows) {
      const size_t out = row_base + row;
      const bool none = l == 0.f;
      const float f = none ? 0.f : q8_o_unit<kType>();
#pragma unroll 1
      for (int c = 0; c < HD; c += 32) {
        float o[32];
        if (nt > 0) {
          tmem_ld32(tO + c, reinterpret_cast<uint32_t *>(o));
          tmem_wait_ld();
          q8_pin(o);
        }
        if (mine) {
#pragma unroll
          for (int i = 0; i < 32; i += 4) {
            const float4 v = none ? make_float4(0.f, 0.f, 0.f, 0.f)
                                  : make_float4(o[i] * f, o[i + 2] * f, o[i + 1] * f, o[i + 3] * f);
            if (p.n_split > 1)
              *reinterpret_cast<float4 *>(p.ws_o + (out * p.n_split + split) * HD + c + i) = v;
            else
              q8_write4<HD>(p, out, c + i, v, m, l);
          }
        }
        __syncwarp();
      }
      if (mine && p.n_split > 1) p.ws_ml[out * p.n_split + split] = make_float2(m, l);
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == 12) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

}  // namespace fa
