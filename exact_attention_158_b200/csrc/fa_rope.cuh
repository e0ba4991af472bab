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
// Bound: HBM, each element read and written once.  A thread keeps one token and one chunk of eight
// pairs for all the heads it takes, so the eight angles it needs are made once, in registers, and
// nothing is shared: no table, no barrier, every warp runs by itself.  (With a table in shared memory,
// made by the CTA behind a barrier, B8 H16+16 N2048 d128 took 57 to 78 us, 45 this
// way: 5960 GB/s.)
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

// A thread's 16 features of one row: f[0..7] and f[8..15] start at columns rope_cols().  In the
// half layout chunk c of the rotated part is features 8c.. and rot/2 + 8c.. (eight whole pairs);
// every other chunk is 16 features in a row (eight interleaved pairs, or the part passed through).
__device__ __forceinline__ int2 rope_cols(const RopeTable &t, int chunk) {
  if (!t.interleaved && 16 * chunk < t.rot) return make_int2(8 * chunk, t.rot / 2 + 8 * chunk);
  return make_int2(16 * chunk, 16 * chunk + 8);
}

// The cosines and sines of a chunk's eight pairs at a token's position.
struct RopeTurn {
  float2 w[8];
  bool any;  // a chunk of the part passed through turns nothing
};
__device__ __forceinline__ void rope_turn(const RopeTable &t, const int32_t *position, int chunk, RopeTurn &r) {
  r.any = 16 * chunk < t.rot;
  if (r.any) {
    const int p = *position;
#pragma unroll
    for (int j = 0; j < 8; ++j) r.w[j] = rope_cos_sin(t, p, 8 * chunk + j);
  }
}

__device__ __forceinline__ void rope_apply(const RopeTable &t, const RopeTurn &r, float (&f)[16]) {
  if (!r.any) return;
  if (t.interleaved) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float a = f[2 * j], b = f[2 * j + 1];
      f[2 * j] = fmaf(a, r.w[j].x, -b * r.w[j].y);
      f[2 * j + 1] = fmaf(b, r.w[j].x, a * r.w[j].y);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float a = f[j], b = f[8 + j];
      f[j] = fmaf(a, r.w[j].x, -b * r.w[j].y);
      f[8 + j] = fmaf(b, r.w[j].x, a * r.w[j].y);
    }
  }
}

// Sixteen features as they lie in memory: loaded early, converted when their turn comes.
template <class T> struct Raw16;
template <> struct Raw16<__nv_bfloat16> { uint4 v[2]; };
template <> struct Raw16<float> { float4 v[4]; };
__device__ __forceinline__ void raw_load(Raw16<__nv_bfloat16> &r, const __nv_bfloat16 *row, int2 col) {
  r.v[0] = *reinterpret_cast<const uint4 *>(row + col.x);
  r.v[1] = *reinterpret_cast<const uint4 *>(row + col.y);
}
__device__ __forceinline__ void raw_load(Raw16<float> &r, const float *row, int2 col) {
  r.v[0] = reinterpret_cast<const float4 *>(row + col.x)[0];
  r.v[1] = reinterpret_cast<const float4 *>(row + col.x)[1];
  r.v[2] = reinterpret_cast<const float4 *>(row + col.y)[0];
  r.v[3] = reinterpret_cast<const float4 *>(row + col.y)[1];
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

__device__ __forceinline__ void load8(const float *src, float *f) {
  const float4 a = reinterpret_cast<const float4 *>(src)[0], b = reinterpret_cast<const float4 *>(src)[1];
  f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w, f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
}
__device__ __forceinline__ void load8(const __nv_bfloat16 *src, float *f) {
  const uint4 v = *reinterpret_cast<const uint4 *>(src);
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
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
  constexpr int kChunks = HD / 16;
  constexpr int kUnroll = sizeof(In) == 4 ? 2 : 4;  // rows on their way at once
  const unsigned long long gid = static_cast<unsigned long long>(blockIdx.x) * kRopeThreads + threadIdx.x;
  const int chunk = static_cast<int>(gid % kChunks);
  const unsigned long long rest = gid / kChunks;
  const unsigned group = static_cast<unsigned>(rest / p.tokens);
  if (group >= static_cast<unsigned>(p.groups)) return;
  const unsigned m = static_cast<unsigned>(rest - static_cast<unsigned long long>(group) * p.tokens);
  const long long b = m / static_cast<unsigned>(p.N), n = m % static_cast<unsigned>(p.N);
  const int first = group * p.heads_per_group;
  const int last = min(first + p.heads_per_group, p.x[0].H + p.x[1].H);
  const int2 col = rope_cols(p.table, chunk);
  auto in_row = [&](int h) {
    const RopeTensor &x = p.x[h >= p.x[0].H];
    if (h >= p.x[0].H) h -= p.x[0].H;
    return static_cast<const In *>(x.in) + b * x.in_s[0] + h * x.in_s[1] + n * x.in_s[2];
  };
  Raw16<In> raw[kUnroll];
#pragma unroll
  for (int u = 0; u < kUnroll; ++u)
    if (first + u < last) raw_load(raw[u], in_row(first + u), col);
  RopeTurn turn;
  rope_turn(p.table, p.positions + b * p.pos_stride + n, chunk, turn);
  for (int h0 = first; h0 < last; h0 += kUnroll) {
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      int h = h0 + u;
      if (h >= last) break;
      float f[16];
      raw_floats(raw[u], f);
      // in place, a row is read before it is written: it has one thread per chunk of pairs
      if (h + kUnroll < last) raw_load(raw[u], in_row(h + kUnroll), col);
      rope_apply(p.table, turn, f);
      const RopeTensor &x = p.x[h >= p.x[0].H];
      if (h >= p.x[0].H) h -= p.x[0].H;
      Out *dst = static_cast<Out *>(x.out) + b * x.out_s[0] + h * x.out_s[1] + n * x.out_s[2];
      store8(dst + col.x, f);
      store8(dst + col.y, f + 8);
    }
  }
}

}  // namespace fa
