// Rotary positions: the turn of each frequency pair and its application to 16 head dims.
//
// A head's first rot_dim dims form rot_dim / 2 pairs; pair i of a token at position p is
// turned by the angle p * inv_freq[i] and scaled by `amplitude`:
//   a' = amplitude (a cos - b sin),   b' = amplitude (b cos + a sin).
// Half layout: the pair is (dim i, dim i + rot_dim / 2); interleaved: (dim 2i, dim 2i + 1).
//
// A thread of the vector path owns 8 frequencies (8g .. 8g + 7) and the 16 dims they turn:
// in the half layout the 16-byte vectors g and g + rot_dim / 16, in the interleaved one the
// vectors 2g and 2g + 1. Groups past rot_dim / 16 copy the vectors 2g and 2g + 1. Both dims
// of a pair belong to one thread, so a call may write over its input.
#pragma once

#include <cuda_bf16.h>
#include <stdint.h>

#include "pa_ptx.cuh"

namespace pa {

struct RopeParams {
  const float* inv_freq;  // [rot_dim / 2]
  int rot_dim;            // 0: nothing is rotated
  int interleaved;
  float amplitude;
};

// A frequency as turns per position in 64-bit fixed point (2^64 = one turn): positions then
// multiply it modulo a turn, without rounding (an fp32 product pos * freq is off by whole
// radians at positions past 2^24). The table's fp32 value is exact, 1 / (2 pi) is a sum of
// two doubles and the first product's rounding error is kept, so the rate is good to its last
// bits and any int32 position to 2^-32 of a turn.
__device__ __forceinline__ unsigned long long rope_rate(float freq) {
  constexpr double kHi = 0.15915494309189535, kLo = -9.839338337591243e-18;  // 1 / (2 pi)
  constexpr double kTurn = 18446744073709551616.0;                            // 2^64
  const double f = static_cast<double>(freq);
  const double p = f * kHi;
  const double err = fma(f, kHi, -p) + f * kLo;
  return __double2ull_rn((p - floor(p)) * kTurn) +
         static_cast<unsigned long long>(__double2ll_rn(err * kTurn));
}

// cos and sin of 2 pi * (pos * rate). The product's top 32 bits are the angle to 2^-32 of a
// turn; its nearest quarter turn is split off, the rest (at most pi / 4) goes through the
// Taylor series of sine (to x^9, next term below 2^-29) and cosine (to x^10, next below 2^-33).
__device__ __forceinline__ float2 rope_circle(int pos, unsigned long long rate) {
  const unsigned long long t = static_cast<unsigned long long>(static_cast<long long>(pos)) * rate;
  const unsigned h = static_cast<unsigned>(t >> 32);
  const unsigned quarter = (h + 0x20000000u) >> 30;
  const float x = static_cast<float>(static_cast<int>(h - (quarter << 30))) *
                  1.46291807926715968e-9f;  // 2 pi / 2^32
  const float z = x * x;
  float s = fmaf(z, 2.75573192e-6f, -1.98412698e-4f);  // 1 / 9!, -1 / 7!
  s = fmaf(z, s, 8.33333333e-3f);                      // 1 / 5!
  s = fmaf(z, s, -1.66666667e-1f);                     // -1 / 3!
  s = fmaf(x * z, s, x);
  float c = fmaf(z, -2.75573192e-7f, 2.48015873e-5f);  // -1 / 10!, 1 / 8!
  c = fmaf(z, c, -1.38888889e-3f);                     // -1 / 6!
  c = fmaf(z, c, 4.16666667e-2f);                      // 1 / 4!
  c = fmaf(z, c, -0.5f);
  c = fmaf(z, c, 1.f);
  // quarter q: (c, s), (-s, c), (-c, -s), (s, -c)
  const bool odd = quarter & 1u;
  const float cc = odd ? s : c, ss = odd ? c : s;
  const unsigned cneg = ((quarter + 1u) & 2u) << 30, sneg = (quarter & 2u) << 30;
  return make_float2(__uint_as_float(__float_as_uint(cc) ^ cneg),
                     __uint_as_float(__float_as_uint(ss) ^ sneg));
}

// The turn of a position is the product of two: of the position with its low four bits
// cleared, times the amplitude, and of those four bits. Kernels that turn the same frequency
// at many neighbouring positions keep both factors in tables (a 28-instruction series becomes
// a packed product); every kernel computes the product in this order, so all agree bit for
// bit. Two roundings more, each 2^-24.
constexpr int kRopeLow = 16;
__device__ __forceinline__ float2 rope_high(int pos, unsigned long long rate, float amplitude) {
  const float2 t = rope_circle(pos & ~(kRopeLow - 1), rate);
  return make_float2(amplitude * t.x, amplitude * t.y);
}
__device__ __forceinline__ float2 rope_low(int pos, unsigned long long rate) {
  return rope_circle(pos & (kRopeLow - 1), rate);
}
__device__ __forceinline__ float2 rope_turn(int pos, unsigned long long rate, float amplitude) {
  const float2 a = rope_high(pos, rate, amplitude), b = rope_low(pos, rate);
  return make_float2(fmaf(a.y, -b.y, a.x * b.x), fmaf(a.y, b.x, a.x * b.y));
}

// One pair, in fp32, rounded once to bf16 by the caller. Every path computes it in this order
// (the vector path on two pairs at a time), so they agree bit for bit.
__device__ __forceinline__ float2 rope_pair(float a, float b, float2 t) {
  return make_float2(fmaf(b, -t.y, a * t.x), fmaf(a, t.y, b * t.x));
}

// The turns of one group: cosines and sines of its 8 frequencies, two to a register pair.
struct RopeTurns {
  float2 c[4], s[4];
};

__device__ __forceinline__ void set_turn(RopeTurns& t, int i, float2 cs) {
  (i & 1 ? t.c[i >> 1].y : t.c[i >> 1].x) = cs.x;
  (i & 1 ? t.s[i >> 1].y : t.s[i >> 1].x) = cs.y;
}

// The two vectors of one group (see the top of the file), turned in place.
__device__ __forceinline__ void rope_group(uint4& va, uint4& vb, const RopeTurns& t,
                                           bool interleaved) {
  uint32_t* a = &va.x;
  uint32_t* b = &vb.x;
  if (interleaved) {
    // word i holds the pair of one frequency: (x0, x1) (c, c) + (x1, x0) (-s, s)
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      uint32_t& w = i < 4 ? a[i] : b[i - 4];
      const float c = i & 1 ? t.c[i >> 1].y : t.c[i >> 1].x;
      const float s = i & 1 ? t.s[i >> 1].y : t.s[i >> 1].x;
      const float x0 = bf16lo_to_f32(w), x1 = bf16hi_to_f32(w);
      const float2 y = __ffma2_rn(make_float2(x1, x0), make_float2(-s, s),
                                  __fmul2_rn(make_float2(x0, x1), make_float2(c, c)));
      w = pack_bf16x2(y.x, y.y);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 x = make_float2(bf16lo_to_f32(a[i]), bf16hi_to_f32(a[i]));
      const float2 y = make_float2(bf16lo_to_f32(b[i]), bf16hi_to_f32(b[i]));
      const float2 ns = make_float2(-t.s[i].x, -t.s[i].y);
      const float2 p = __ffma2_rn(y, ns, __fmul2_rn(x, t.c[i]));
      const float2 q = __ffma2_rn(x, t.s[i], __fmul2_rn(y, t.c[i]));
      a[i] = pack_bf16x2(p.x, p.y);
      b[i] = pack_bf16x2(q.x, q.y);
    }
  }
}

// Indices of the two 16-byte vectors of group g within a head.
__device__ __forceinline__ int2 rope_vectors(int g, const RopeParams& r) {
  const int ng = r.rot_dim >> 4;
  return (g < ng && !r.interleaved) ? make_int2(g, g + ng) : make_int2(2 * g, 2 * g + 1);
}

// Where frequency f of HALF sits in a row of a table: the first four of every group of eight,
// then the second four, so that the eight threads of a head read a group's 16-byte halves
// from consecutive addresses (no bank conflicts).
template <int HALF>
__device__ __forceinline__ int rope_place(int f) {
  return ((f >> 2) & 1) * (HALF / 2) + (f >> 3) * 4 + (f & 3);
}

// A table of ROWS rows of cosines and sines (apart) in shared memory.
template <int ROWS, int HALF>
struct RopeTable {
  alignas(16) float c[ROWS][HALF];
  alignas(16) float s[ROWS][HALF];

  __device__ __forceinline__ void put(int row, int f, float2 t) {
    c[row][rope_place<HALF>(f)] = t.x;
    s[row][rope_place<HALF>(f)] = t.y;
  }
  // the eight frequencies of group g
  __device__ __forceinline__ RopeTurns group(int row, int g) const {
    RopeTurns t;
    const float4 c0 = *reinterpret_cast<const float4*>(&c[row][4 * g]);
    const float4 c1 = *reinterpret_cast<const float4*>(&c[row][HALF / 2 + 4 * g]);
    const float4 s0 = *reinterpret_cast<const float4*>(&s[row][4 * g]);
    const float4 s1 = *reinterpret_cast<const float4*>(&s[row][HALF / 2 + 4 * g]);
    t.c[0] = make_float2(c0.x, c0.y);
    t.c[1] = make_float2(c0.z, c0.w);
    t.c[2] = make_float2(c1.x, c1.y);
    t.c[3] = make_float2(c1.z, c1.w);
    t.s[0] = make_float2(s0.x, s0.y);
    t.s[1] = make_float2(s0.z, s0.w);
    t.s[2] = make_float2(s1.x, s1.y);
    t.s[3] = make_float2(s1.z, s1.w);
    return t;
  }
  // row i: the turns of token t0 + i
  __device__ __forceinline__ void fill_tokens(int tid, int threads, int64_t t0, int num_tokens,
                                              const int32_t* positions, const RopeParams& r) {
    const int half = r.rot_dim >> 1;
    if (half == 0) return;
    // one frequency per thread, rows `step` apart
    const int step = threads / half, row0 = tid / half, f = tid - row0 * half;
    if (row0 >= step) return;
    const unsigned long long rate = rope_rate(__ldg(r.inv_freq + f));
    for (int row = row0; row < ROWS && t0 + row < num_tokens; row += step)
      put(row, f, rope_turn(__ldg(positions + t0 + row), rate, r.amplitude));
  }
};

// Products of two groups' turns, as rope_turn forms them.
__device__ __forceinline__ RopeTurns rope_product(const RopeTurns& a, const RopeTurns& b) {
  RopeTurns t;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 nb = make_float2(-b.s[i].x, -b.s[i].y);
    t.c[i] = __ffma2_rn(a.s[i], nb, __fmul2_rn(a.c[i], b.c[i]));
    t.s[i] = __ffma2_rn(a.s[i], b.c[i], __fmul2_rn(a.c[i], b.s[i]));
  }
  return t;
}

}  // namespace pa
