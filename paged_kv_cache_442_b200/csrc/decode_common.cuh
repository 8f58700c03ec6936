// Device helpers shared by the persistent tensor-core decodes: epoch-tagged counters,
// named barriers, tensor-memory column loads and the e4m3 term split.
#pragma once

#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "pa_internal.h"
#include "pa_ptx.cuh"

namespace pa {

constexpr unsigned kCountBits = 24;
constexpr unsigned long long kCountMask = (1ull << kCountBits) - 1;

// Add one to an epoch-tagged counter and return the count before the add; a counter
// carrying another epoch's tag counts as zero. The tag is installed first (count 0):
// a thread that reads a stale tag swaps in (tag, 0), and stops as soon as it sees this
// call's tag, whoever installed it. After that only atomicAdds touch the counter, and
// they keep the tag, so the common case is one atomicAdd with no retries even with one
// producer per SM on one address. Bounded number of attempts.
__device__ __forceinline__ unsigned tagged_fetch_add(unsigned long long* ctr,
                                                     unsigned long long tag, unsigned* err,
                                                     bool* ok) {
  unsigned long long v = *reinterpret_cast<volatile unsigned long long*>(ctr);
  int it = 0;
  while ((v >> kCountBits) != tag) {
    if (++it > 4096) {
      flag_error(err, PA_DEV_ERR_TIMEOUT);
      *ok = false;
      return 0;
    }
    const unsigned long long prev = atomicCAS(ctr, v, tag << kCountBits);
    v = (prev == v) ? (tag << kCountBits) : prev;
  }
  const unsigned long long old = atomicAdd(ctr, 1ull);
  if ((old >> kCountBits) != tag) {  // the count ran into the tag bits
    flag_error(err, PA_DEV_ERR_TIMEOUT);
    *ok = false;
    return 0;
  }
  *ok = true;
  return static_cast<unsigned>(old & kCountMask);
}

// Give a counter this call's tag with count 0 unless it has the tag already. Everyone who
// finds a stale value swaps in the same one, so a failed swap means that another thread
// (or one of its adds, at most one per thread) came first: no two can keep each other busy.
__device__ __forceinline__ bool tagged_install(unsigned long long* ctr, unsigned long long v,
                                               unsigned long long tag, unsigned* err) {
  int it = 0;
  while ((v >> kCountBits) != tag) {
    if (++it > 4096) {
      flag_error(err, PA_DEV_ERR_TIMEOUT);
      return false;
    }
    const unsigned long long prev = atomicCAS(ctr, v, tag << kCountBits);
    if (prev == v) return true;
    v = prev;
  }
  return true;
}

// Same contract as tagged_fetch_add for the arrivals of an item's parts: add first (one atomic
// once the tag is there); with a stale tag that add lands on a value that the installation
// replaces, and is made again. (Adding and swapping in (tag, 1) in turn until one of the two
// holds let sixteen simultaneous arrivals disturb one another for thousands of rounds.)
__device__ __forceinline__ unsigned tagged_arrive(unsigned long long* ctr,
                                                  unsigned long long tag, unsigned* err,
                                                  bool* ok) {
  unsigned long long old = atomicAdd(ctr, 1ull);
  *ok = true;
  if ((old >> kCountBits) != tag) {
    *ok = tagged_install(ctr, old + 1, tag, err);
    old = atomicAdd(ctr, 1ull);
  }
  return static_cast<unsigned>(old & kCountMask);
}

__device__ __forceinline__ void named_bar_sync(int id, int n) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(n) : "memory");
}

// named barrier that also ORs a flag over the participating threads
__device__ __forceinline__ bool bar_or(int id, int n, bool v) {
  unsigned r;
  asm volatile(
      "{\n\t.reg .pred q, p;\n\t"
      "setp.ne.u32 q, %1, 0;\n\t"
      "bar.red.or.pred p, %2, %3, q;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(r)
      : "r"(v ? 1u : 0u), "r"(id), "r"(n)
      : "memory");
  return r != 0;
}

// 16 consecutive fp32 columns of this thread's TMEM lane.
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, float (&v)[16]) {
  uint32_t r[16];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
}

// N consecutive fp32 columns of this thread's TMEM lane (N = 1, 2, 4, 8 or 16; the
// score columns a softmax thread needs are the group's G heads).
template <int N>
__device__ __forceinline__ void tmem_ld_cols(uint32_t taddr, float (&v)[N]) {
  static_assert(N == 1 || N == 2 || N == 4 || N == 8 || N == 16, "tcgen05.ld column count");
  uint32_t r[16];
  if constexpr (N == 1) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];" : "=r"(r[0]) : "r"(taddr) : "memory");
  } else if constexpr (N == 2) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x2.b32 {%0,%1}, [%2];"
                 : "=r"(r[0]), "=r"(r[1]) : "r"(taddr) : "memory");
  } else if constexpr (N == 4) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(taddr) : "memory");
  } else if constexpr (N == 8) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]),
                   "=r"(r[6]), "=r"(r[7])
                 : "r"(taddr)
                 : "memory");
  } else {
    float t[16];
    tmem_ld16(taddr, t);
#pragma unroll
    for (int i = 0; i < 16; ++i) r[i] = __float_as_uint(t[i]);
  }
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = __uint_as_float(r[i]);
}

__device__ __forceinline__ void tmem_st16(uint32_t taddr, const float (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "r"(__float_as_uint(v[0])), "r"(__float_as_uint(v[1])), "r"(__float_as_uint(v[2])),
      "r"(__float_as_uint(v[3])), "r"(__float_as_uint(v[4])), "r"(__float_as_uint(v[5])),
      "r"(__float_as_uint(v[6])), "r"(__float_as_uint(v[7])), "r"(__float_as_uint(v[8])),
      "r"(__float_as_uint(v[9])), "r"(__float_as_uint(v[10])), "r"(__float_as_uint(v[11])),
      "r"(__float_as_uint(v[12])), "r"(__float_as_uint(v[13])), "r"(__float_as_uint(v[14])),
      "r"(__float_as_uint(v[15]))
      : "memory");
}


// Two values -> their e4m3 codes (round to nearest even, saturated to +-448), packed
// with a in the low byte, and the values those codes stand for.
__device__ __forceinline__ uint32_t e4m3x2(float a, float b, float2& back) {
  const __nv_fp8x2_storage_t c =
      __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(c, __NV_E4M3);
  back = __half22float2(*reinterpret_cast<const __half2*>(&h));
  return static_cast<uint32_t>(c);
}

// The same for e5m2 (saturated to +-57344); an e5m2 code is the upper byte of an fp16 number.
__device__ __forceinline__ uint32_t e5m2x2(float a, float b, float2& back) {
  const uint32_t c = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E5M2);
  const uint32_t h = __byte_perm(c, 0u, 0x1404);
  back = __half22float2(*reinterpret_cast<const __half2*>(&h));
  return c;
}

// hi / lo e4m3 terms of two values: hi = e4m3(v), lo = e4m3(lo_scale * (v - hi)),
// as two packed byte pairs (value a in the low byte of each).
__device__ __forceinline__ void split_e4m3x2(float a, float b, float lo_scale, uint32_t& hi,
                                             uint32_t& lo) {
  float2 h, unused;
  hi = e4m3x2(a, b, h);
  lo = e4m3x2((a - h.x) * lo_scale, (b - h.y) * lo_scale, unused);
}

}  // namespace pa
