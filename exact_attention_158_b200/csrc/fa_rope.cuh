// fa_rope.cuh -- rotary positions: every pair (a, b) of a head's rotated features turns by the
// angle p * f_j of its token's position p and the pair's frequency f_j,
//     y_a = amp (x_a cos - x_b sin),  y_b = amp (x_b cos + x_a sin),
// so that q . k depends on the distance of their positions alone.  Pairs are (j, j + rot/2) in the
// half layout and (2j, 2j + 1) in the interleaved one; features from rot on pass through.  The
// gradient is the transposed rotation: sin with its sign changed, the same amplitude.
//
// Angles.  At position 10^6 an fp32 product p * f_j is off by up to 0.06 rad, so p * f_j / (2 pi) is
// formed in fp64 and only its fraction, in [-1/2, 1/2], goes to fp32, the rest (2^-26 turns) as a
// first-order correction of the sine and cosine.  One sine and cosine serve every head of the token: a CTA takes kTok tokens, makes their tables in
// shared memory once, and applies them to all heads of q and k.
//
// Bound: HBM, each element read and written once.  16-byte accesses; the strided side (a
// projection's [B, N, heads, d]) and the head-major side are both whole rows of 128 to 512 bytes.
#pragma once
#include <cuda_bf16.h>

#include "sm100_ptx.cuh"

namespace fa {

constexpr int kRopeThreads = 256;
constexpr int kRopeMaxTok = 32;
constexpr int kRopeMaxPairs = 64;  // rot / 2 at d = 128

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

// Turns a thread's 16 features by the token's table cs[rot / 2].
__device__ __forceinline__ void rope_apply(const RopeTable &t, const float2 *cs, int chunk,
                                           float (&f)[16]) {
  if (16 * chunk >= t.rot) return;
  if (t.interleaved) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float2 w = cs[8 * chunk + j];
      const float a = f[2 * j], b = f[2 * j + 1];
      f[2 * j] = fmaf(a, w.x, -b * w.y);
      f[2 * j + 1] = fmaf(b, w.x, a * w.y);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float2 w = cs[8 * chunk + j];
      const float a = f[j], b = f[8 + j];
      f[j] = fmaf(a, w.x, -b * w.y);
      f[8 + j] = fmaf(b, w.x, a * w.y);
    }
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
  long long tokens;  // B * N
  int log_tok;       // tokens per CTA (a power of two)
};

// grid: ceil(tokens / kTok).  A CTA's rows are numbered head by head, its tokens side by side, so
// neighbouring thread groups move neighbouring rows of the head-major side; HD / 16 threads a row.
template <int HD, class In, class Out>
__global__ void __launch_bounds__(kRopeThreads) fa_rope_kernel(const RopeParams p) {
  __shared__ float2 cs[kRopeMaxTok * kRopeMaxPairs];
  __shared__ long long base[2][2][kRopeMaxTok];  // tensor, side: the token's row of head 0
  constexpr int kChunks = HD / 16;
  const int tok_n = 1 << p.log_tok;
  const long long m0 = static_cast<long long>(blockIdx.x) << p.log_tok;
  const int live = static_cast<int>(min(static_cast<long long>(tok_n), p.tokens - m0));
  const int pairs = p.table.rot / 2;
  for (int t = threadIdx.x; t < live; t += kRopeThreads) {
    const long long b = (m0 + t) / p.N, n = (m0 + t) % p.N;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      base[i][0][t] = b * p.x[i].in_s[0] + n * p.x[i].in_s[2];
      base[i][1][t] = b * p.x[i].out_s[0] + n * p.x[i].out_s[2];
    }
  }
  for (int i = threadIdx.x; i < live * pairs; i += kRopeThreads) {
    const int t = i / pairs, j = i % pairs;
    const long long b = (m0 + t) / p.N, n = (m0 + t) % p.N;
    cs[t * pairs + j] = rope_cos_sin(p.table, p.positions[b * p.pos_stride + n], j);
  }
  __syncthreads();
  const int rows = (p.x[0].H + p.x[1].H) << p.log_tok;
  const int chunk = threadIdx.x % kChunks;
  const int2 col = rope_cols(p.table, chunk);
  for (int r = threadIdx.x / kChunks; r < rows; r += kRopeThreads / kChunks) {
    const int t = r & (tok_n - 1);
    int h = r >> p.log_tok;
    if (t >= live) continue;
    const int which = h >= p.x[0].H;
    if (which) h -= p.x[0].H;
    const RopeTensor &x = p.x[which];
    const In *src = static_cast<const In *>(x.in) + base[which][0][t] + h * x.in_s[1];
    Out *dst = static_cast<Out *>(x.out) + base[which][1][t] + h * x.out_s[1];
    float f[16];
    load8(src + col.x, f);
    load8(src + col.y, f + 8);
    rope_apply(p.table, cs + t * pairs, chunk, f);
    store8(dst + col.x, f);
    store8(dst + col.y, f + 8);
  }
}

}  // namespace fa
