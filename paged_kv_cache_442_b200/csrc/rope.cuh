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

// cos and sin of pos * freq, times the amplitude. The angle is reduced as a number of whole
// turns in 64 bits (an fp32 product is off by whole radians at positions past 2^24). The
// remainder, at most half a turn, goes through the fp32 sine and cosine of pi x as its fp32
// rounding; what the rounding left out (2^-25 of it) turns the result by its first-order term.
__device__ __forceinline__ float2 rope_turn(int pos, float freq, float amplitude) {
  constexpr double kInvTwoPi = 0.15915494309189533577;
  const double u = static_cast<double>(pos) * (static_cast<double>(freq) * kInvTwoPi);
  const double r = 2.0 * (u - rint(u));
  const float rh = static_cast<float>(r);
  const float rest = 3.14159265f * static_cast<float>(r - static_cast<double>(rh));
  float s, c;
  sincospif(rh, &s, &c);
  return make_float2(amplitude * fmaf(-s, rest, c), amplitude * fmaf(c, rest, s));
}

// One pair, in fp32, rounded once to bf16 by the caller.
__device__ __forceinline__ float2 rope_pair(float a, float b, float2 t) {
  return make_float2(fmaf(a, t.x, -b * t.y), fmaf(b, t.x, a * t.y));
}

// The two vectors of one group (see the top of the file), turned in place.
__device__ __forceinline__ void rope_group(uint4& va, uint4& vb, const float2 (&t)[8],
                                           bool interleaved) {
  uint32_t* a = &va.x;
  uint32_t* b = &vb.x;
  if (interleaved) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 ya = rope_pair(bf16lo_to_f32(a[i]), bf16hi_to_f32(a[i]), t[i]);
      const float2 yb = rope_pair(bf16lo_to_f32(b[i]), bf16hi_to_f32(b[i]), t[4 + i]);
      a[i] = pack_bf16x2(ya.x, ya.y);
      b[i] = pack_bf16x2(yb.x, yb.y);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 y0 = rope_pair(bf16lo_to_f32(a[i]), bf16lo_to_f32(b[i]), t[2 * i]);
      const float2 y1 = rope_pair(bf16hi_to_f32(a[i]), bf16hi_to_f32(b[i]), t[2 * i + 1]);
      a[i] = pack_bf16x2(y0.x, y1.x);
      b[i] = pack_bf16x2(y0.y, y1.y);
    }
  }
}

// Indices of the two 16-byte vectors of group g within a head.
__device__ __forceinline__ int2 rope_vectors(int g, const RopeParams& r) {
  const int ng = r.rot_dim >> 4;
  return (g < ng && !r.interleaved) ? make_int2(g, g + ng) : make_int2(2 * g, 2 * g + 1);
}

}  // namespace pa
