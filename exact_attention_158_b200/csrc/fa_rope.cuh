// fa_rope.cuh -- rotary positions: every pair (a, b) of a head's rotated features turns by the
// angle p * f_j of its token's position p and the pair's frequency f_j,
//     y_a = amp (x_a cos - x_b sin),  y_b = amp (x_b cos + x_a sin),
// so that q . k depends on the distance of their positions alone.  Pairs are (j, j + rot/2) in the
// half layout and (2j, 2j + 1) in the interleaved one; features from rot on pass through.  The
// gradient is the transposed rotation: sin with its sign changed, the same amplitude.
//
// Angles.  At position 10^6 an fp32 product p * f_j is off by up to 0.06 rad, so p * f_j / (2 pi) is
// formed in fp64 and only its fraction, in [-1/2, 1/2], goes to fp32, the rest (2^-26 turns) as a
// first-order correction of the sine and cosine.
//
// Bound: HBM, each element read and written once.  A thread keeps one token and eight pairs
// for all the heads it takes, so the eight angles it needs are made once, in registers, and
// nothing is shared: no table, no barrier, every warp runs by itself.  (With a table in shared memory,
// made by the CTA behind a barrier, B8 H16+16 N2048 d128 took 57 to 78 us, 45 this
// way: 6000 GB/s.)
// 16-byte accesses, whole rows of 128 to 512 bytes by the HD / 16 threads of a row; the four or eight
// tokens of a warp are neighbours, so the head-major side moves 1 to 2 KB at a time.
#pragma once
#include <cuda_bf16.h>

#include "sm100_ptx.cuh"

namespace fa {

constexpr int kRopeThreads = 128;

// What turns a row: shared by fa_rope and by the cache writer.
struct RopeTable {
  const double *freqs;  // [rot / 2] radians per position
  int rot;              // rotated features, a multiple of 16 (0: nothing is rotated)
  int interleaved;
  float amplitude;
  float sign;           // -1 for the transposed rotation
};

// amp * (cos, sign * sin) of position * freq.
__device__ __forceinline__ float2 rope_cos_sin(const RopeTable &t, int position, int pair) {
  const double turns = static_cast<double>(position) * t.freqs[pair] * 0.15915494309189535;
  const double part = turns - rint(turns);
  const float frac = static_cast<float>(part);
  const float rest = static_cast<float>(part - frac) * 6.2831853f;  // radians that fp32 left out
  float s, c;
  sincospif(2.f * frac, &s, &c);
  const float c0 = c;
  c = fmaf(-s, rest, c);
  s = fmaf(c0, rest, s);
  return make_float2(t.amplitude * c, t.amplitude * t.sign * s);
}

// A thread's 16 features of one row, f[0..15], are 16 / P pieces of P features, 16 bytes each as they are
// read: P = 8 in bf16, 4 in fp32.  The HD / 16 threads of a row take neighbouring pieces, so each of
// their accesses is whole sectors (32 contiguous bytes to a thread instead, two accesses to a sector:
// 55 us where this takes 45, B8 H16+16 N2048 d128 bf16 interleaved).  In the half layout
// the pieces come in twos, those of pairs j in features j.. and rot/2 + j.., and the part passed
// through is split in the same way.
template <int P> struct RopeCols {
  int col[16 / P];
};
template <int HD, int P>
__device__ __forceinline__ RopeCols<P> rope_cols(const RopeTable &t, int chunk) {
  constexpr int kMates = HD / 16;
  RopeCols<P> r;
  if (t.interleaved) {
#pragma unroll
    for (int i = 0; i < 16 / P; ++i) r.col[i] = P * (chunk + i * kMates);
  } else {
#pragma unroll
    for (int k = 0; k < 8 / P; ++k) {
      const int x = P * (chunk + k * kMates), over = x - t.rot / 2;
      r.col[2 * k] = over < 0 ? x : t.rot + over;
      r.col[2 * k + 1] = over < 0 ? t.rot / 2 + x : t.rot + (HD - t.rot) / 2 + over;
    }
  }
  return r;
}

// The cosines and sines of a thread's eight pairs at a token's position: of f[2i], f[2i + 1] in the
// interleaved layout, of features i of the two pieces in the half one.
template <int P> struct RopeTurn {
  float2 w[8];
  bool on[16 / P];  // piece i is turned (in the half layout, pieces 2k and 2k + 1 alike), not passed through
};
template <int P>
__device__ __forceinline__ void rope_turn(const RopeTable &t, const int32_t *position, const RopeCols<P> &c,
                                          RopeTurn<P> &r) {
  bool any = false;
#pragma unroll
  for (int i = 0; i < 16 / P; ++i) {
    r.on[i] = (t.interleaved ? c.col[i] : c.col[i / 2 * 2]) < t.rot;
    any = any || r.on[i];
  }
  if (!any) return;
  // all eight in one go (a piece passed through makes pair 0's and drops them): the sines of one pair
  // run in the latency of the others'
  const int p = *position;
  int pair[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int i = j / (P / 2), e = j % (P / 2);
    pair[j] = !r.on[i] ? 0 : e + (t.interleaved ? c.col[i] / 2 : c.col[i / 2 * 2] + i % 2 * (P / 2));
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) r.w[j] = rope_cos_sin(t, p, pair[j]);
}

__device__ __forceinline__ void rope_pair(float2 w, float &a, float &b) {
  const float x = a;
  a = fmaf(x, w.x, -b * w.y);
  b = fmaf(b, w.x, x * w.y);
}

template <int P>
__device__ __forceinline__ void rope_apply(const RopeTable &t, const RopeTurn<P> &r, float (&f)[16]) {
  if (t.interleaved) {
#pragma unroll
    for (int i = 0; i < 16 / P; ++i)
      if (r.on[i]) {
#pragma unroll
        for (int j = i * (P / 2); j < (i + 1) * (P / 2); ++j) rope_pair(r.w[j], f[2 * j], f[2 * j + 1]);
      }
  } else {
#pragma unroll
    for (int k = 0; k < 8 / P; ++k)
      if (r.on[2 * k]) {
#pragma unroll
        for (int e = 0; e < P; ++e) rope_pair(r.w[P * k + e], f[2 * P * k + e], f[2 * P * k + P + e]);
      }
  }
}

// Sixteen features as they lie in memory: loaded early, converted when their turn comes.
template <class T> struct Raw16;
template <> struct Raw16<__nv_bfloat16> { uint4 v[2]; };
template <> struct Raw16<float> { float4 v[4]; };
template <class T> constexpr int kRopePiece = 16 / sizeof(T);  // features
__device__ __forceinline__ void raw_load(Raw16<__nv_bfloat16> &r, const __nv_bfloat16 *row, const RopeCols<8> &c) {
#pragma unroll
  for (int i = 0; i < 2; ++i) r.v[i] = *reinterpret_cast<const uint4 *>(row + c.col[i]);
}
__device__ __forceinline__ void raw_load(Raw16<float> &r, const float *row, const RopeCols<4> &c) {
#pragma unroll
  for (int i = 0; i < 4; ++i) r.v[i] = *reinterpret_cast<const float4 *>(row + c.col[i]);
}
__device__ __forceinline__ void raw_floats(const Raw16<__nv_bfloat16> &r, float (&f)[16]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t w[4] = {r.v[i].x, r.v[i].y, r.v[i].z, r.v[i].w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      f[8 * i + 2 * j] = __uint_as_float(w[j] << 16);
      f[8 * i + 2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
    }
  }
}
__device__ __forceinline__ void raw_floats(const Raw16<float> &r, float (&f)[16]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[4 * i] = r.v[i].x, f[4 * i + 1] = r.v[i].y, f[4 * i + 2] = r.v[i].z, f[4 * i + 3] = r.v[i].w;
  }
}

__device__ __forceinline__ void store8(float *dst, const float *f) {
  reinterpret_cast<float4 *>(dst)[0] = make_float4(f[0], f[1], f[2], f[3]);
  reinterpret_cast<float4 *>(dst)[1] = make_float4(f[4], f[5], f[6], f[7]);
}
__device__ __forceinline__ void store8(__nv_bfloat16 *dst, const float *f) {
  *reinterpret_cast<uint4 *>(dst) = make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]),
                                               pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
}

__device__ __forceinline__ void store4(float *dst, const float *f) {
  *reinterpret_cast<float4 *>(dst) = make_float4(f[0], f[1], f[2], f[3]);
}
__device__ __forceinline__ void store4(__nv_bfloat16 *dst, const float *f) {
  *reinterpret_cast<uint2 *>(dst) = make_uint2(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]));
}
template <class T, int P>
__device__ __forceinline__ void store_pieces(T *row, const RopeCols<P> &c, const float (&f)[16]) {
#pragma unroll
  for (int i = 0; i < 16 / P; ++i) {
    if constexpr (P == 8) store8(row + c.col[i], f + 8 * i);
    else store4(row + c.col[i], f + 4 * i);
  }
}

// One tensor [B, H, N, d] of the call: element strides of b, h and n on both sides.
struct RopeTensor {
  const void *in;
  void *out;
  long long in_s[3], out_s[3];
  int H;
};

struct RopeParams {
  RopeTensor x[2];  // q, k (k.H = 0 without k)
  const int32_t *positions;
  long long pos_stride;  // between batch rows (0: one row of positions for all)
  RopeTable table;
  int N;
  unsigned tokens;  // B * N
  int groups, heads_per_group;  // the heads are split over `groups` threads where tokens are few
};

// One thread per (head group, token, chunk of features), the chunk fastest, then the token.
template <int HD, class In, class Out>
__global__ void __launch_bounds__(kRopeThreads) fa_rope_kernel(const RopeParams p) {
  constexpr int kChunks = HD / 16, P = kRopePiece<In>;
  // rows on their way at once: four of fp32 cost registers, so warps (8198 tokens, 40 heads of 64: 35 us
  // where two take 31); of bf16 they hide more (B8 H16+16 N2048 d128 back to back: 49 us, two 51)
  constexpr int kUnroll = sizeof(In) == 4 ? 2 : 4;
  const unsigned long long gid = static_cast<unsigned long long>(blockIdx.x) * kRopeThreads + threadIdx.x;
  const int chunk = static_cast<int>(gid % kChunks);
  const unsigned long long rest = gid / kChunks;
  const unsigned group = static_cast<unsigned>(rest / p.tokens);
  if (group >= static_cast<unsigned>(p.groups)) return;
  const unsigned m = static_cast<unsigned>(rest - static_cast<unsigned long long>(group) * p.tokens);
  const long long b = m / static_cast<unsigned>(p.N), n = m % static_cast<unsigned>(p.N);
  const int first = group * p.heads_per_group;
  const int last = min(first + p.heads_per_group, p.x[0].H + p.x[1].H);
  const RopeCols<P> col = rope_cols<HD, P>(p.table, chunk);
  auto in_row = [&](int h) {
    const RopeTensor &x = p.x[h >= p.x[0].H];
    if (h >= p.x[0].H) h -= p.x[0].H;
    return static_cast<const In *>(x.in) + b * x.in_s[0] + h * x.in_s[1] + n * x.in_s[2];
  };
  Raw16<In> raw[kUnroll];
#pragma unroll
  for (int u = 0; u < kUnroll; ++u)
    if (first + u < last) raw_load(raw[u], in_row(first + u), col);
  RopeTurn<P> turn;
  rope_turn(p.table, p.positions + b * p.pos_stride + n, col, turn);
  for (int h0 = first; h0 < last; h0 += kUnroll) {
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      int h = h0 + u;
      if (h >= last) break;
      float f[16];
      raw_floats(raw[u], f);
      // in place, a row is read before it is written: a thread writes the features it has read
      if (h + kUnroll < last) raw_load(raw[u], in_row(h + kUnroll), col);
      rope_apply(p.table, turn, f);
      const RopeTensor &x = p.x[h >= p.x[0].H];
      if (h >= p.x[0].H) h -= p.x[0].H;
      Out *dst = static_cast<Out *>(x.out) + b * x.out_s[0] + h * x.out_s[1] + n * x.out_s[2];
      store_pieces(dst, col, f);
    }
  }
}

}  // namespace fa
