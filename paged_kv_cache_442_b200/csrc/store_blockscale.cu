// Append of new K/V rows to e4m3 pools that hold one scale for each (block, kv head), with
// the rotary positions of q and k in the same call (for many tokens the queries take a launch of
// their own, beside whose end the rows' one may start).
//
// The scale of a (block, kv head) is the smallest power of two s >= 2^-126 with
// max |x| <= 448 s over the rows the block has taken since its first one (position
// offset 0 starts a block afresh), never smaller than it was. e4m3 codes are themselves
// floating point, so a power of two costs no precision, and when a later row makes the
// scale grow, the stored codes move by an exact power of two: only codes that fall into
// e4m3's subnormal range are rounded again.
//
// Work: one unit per (sequence, block its new rows reach, or 64 positions of small blocks, K or
// V, kv head or heads), 16 dims per thread and row (two 16-byte loads). A unit loads its new
// rows into registers, turns them (K), takes the largest finite magnitude on the bf16 bits,
// agrees on the scale and writes the codes; rows already in the block are rewritten only when
// the scale grew. No unit shares a (block, head) with another, so there are no global atomics
// and the result does not depend on the order. HBM-bound: a bf16 row in, half of it out.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include <cooperative_groups.h>

#include "pa_internal.h"
#include "pa_ptx.cuh"
#include "rope.cuh"

namespace cg = cooperative_groups;

namespace pa {
namespace {

constexpr int kThreads = 256;
constexpr int kFewRows = 16;     // most new rows of a block that one warp takes ...
constexpr int kVeryFewRows = 8;  // ... and of a kernel that keeps half the registers for them
constexpr int kWindow = 1024;    // sequences whose units are counted at a time
constexpr int kMaxCluster = 8;   // CTAs that share a block of 1024 rows
constexpr int kQTokens = 2;      // tokens of a CTA that turns queries

struct AppendParams {
  const __nv_bfloat16* q;
  const __nv_bfloat16* k;
  const __nv_bfloat16* v;
  __nv_bfloat16* q_out;
  int64_t q_stride, k_stride, v_stride, q_out_stride;  // elements between tokens
  uint8_t* k_codes;
  uint8_t* v_codes;
  float* k_scales;  // [num_blocks, Hkv]
  float* v_scales;
  const int32_t* block_tables;
  const int32_t* cu_seqlens;
  const int32_t* context_lens;
  const int32_t* positions;
  RopeParams rope;
  int num_seqs;
  int num_tokens;
  int max_new;
  int max_blocks;
  int num_blocks;
  int bs_log2;
  int num_q_heads;
  int num_kv_heads;
  int q_ctas;
  bool behind_queries;  // may start beside the queries' kernel, whose outputs it does not read
  int span;     // blocks that max_new consecutive positions can reach
  int cluster;  // CTAs per block of many rows
  unsigned* err;
};

// Exponent k of the smallest power of two >= 2^-126 with value <= 448 * 2^k, for a finite
// non-negative bf16 given as bits: 448 = 1.75 * 2^8, and 1.75 has the mantissa bits 0x60.
__device__ __forceinline__ int scale_exponent(unsigned bits) {
  const int k = static_cast<int>(bits >> 7) - 127 - 8 + ((bits & 0x7f) > 0x60 ? 1 : 0);
  return max(k, -126);
}

__device__ __forceinline__ float exp2_int(int k) {  // 2^k, k in [-126, 127]
  return __uint_as_float(static_cast<unsigned>(k + 127) << 23);
}

// Larger magnitude of both halves, kept per half (as bits, which order as the values do).
__device__ __forceinline__ unsigned abs_max2(unsigned acc, unsigned w) {
  return __vmaxu2(acc, w & 0x7fff7fffu);
}
// The same with infinities and NaN counted as 0 (bits from 0x7f80 on).
__device__ __forceinline__ unsigned finite_max2(unsigned acc, unsigned w) {
  const unsigned m = w & 0x7fff7fffu;
  return __vmaxu2(acc, m & __vcmpltu2(m, 0x7f807f80u));
}
constexpr unsigned kInfBits = 0x7f80u;

// Eight bf16 values times inv -> eight codes.
__device__ __forceinline__ uint2 quantise8(const uint4& w, float inv) {
  const uint32_t* x = &w.x;
  uint32_t c[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    c[i] = __nv_cvt_float2_to_fp8x2(__fmul2_rn(make_float2(bf16lo_to_f32(x[i]), bf16hi_to_f32(x[i])),
                                               make_float2(inv, inv)),
                                    __NV_SATFINITE, __NV_E4M3);
  return make_uint2(__byte_perm(c[0], c[1], 0x5410), __byte_perm(c[2], c[3], 0x5410));
}

// Sixteen codes to the codes of the same values over a scale that is 1 / factor as large.
__device__ __forceinline__ uint4 requantise16(uint4 w, float factor) {
  uint32_t* x = &w.x;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t r = 0;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(
          static_cast<__nv_fp8x2_storage_t>(x[i] >> (16 * j)), __NV_E4M3);
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
      r |= static_cast<uint32_t>(__nv_cvt_float2_to_fp8x2(
               make_float2(__fmul_rn(f.x, factor), __fmul_rn(f.y, factor)), __NV_SATFINITE,
               __NV_E4M3))
           << (16 * j);
    }
    x[i] = r;
  }
  return w;
}

// The first `rows` rows of a block's head, to a scale 1 / factor as large.
template <int D>
__device__ __forceinline__ void requantise_rows(uint8_t* codes, int64_t row_bytes, int rows,
                                                float factor, int first, int step) {
  constexpr int VPR = D / 16;  // 16-byte vectors of codes per row
  constexpr int U = 4;         // vectors in flight per thread
  auto at = [&](int i) {
    return reinterpret_cast<uint4*>(codes + (i / VPR) * row_bytes) + i % VPR;
  };
#pragma unroll 1
  for (int i = first; i < rows * VPR; i += U * step) {
    uint4 w[U];
#pragma unroll
    for (int k = 0; k < U; ++k)
      if (i + k * step < rows * VPR) w[k] = *at(i + k * step);
#pragma unroll
    for (int k = 0; k < U; ++k)
      if (i + k * step < rows * VPR) *at(i + k * step) = requantise16(w[k], factor);
  }
}

// The queries of kQTokens tokens (as in rope.cu).
template <int D>
__device__ __forceinline__ void turn_queries(const AppendParams& p,
                                             RopeTable<kQTokens, D / 2>& table) {
  constexpr int NG = D / 16;
  constexpr int HL = kThreads / (NG * kQTokens);
  const int tid = threadIdx.x;
  const int g = tid % NG, tk = (tid / NG) % kQTokens, hl = tid / (NG * kQTokens);
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * kQTokens;
  const int64_t t = t0 + tk;
  const int heads = t < p.num_tokens ? p.num_q_heads : 0;
  const int2 at = rope_vectors(g, p.rope);
  const uint4* src = reinterpret_cast<const uint4*>(p.q + t * p.q_stride);
  uint4* dst = reinterpret_cast<uint4*>(p.q_out + t * p.q_out_stride);
  uint4 a[2], b[2];
  auto load = [&](int h0) {
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int h = h0 + u * HL;
      if (h < heads) {
        a[u] = __ldcs(src + h * (D / 8) + at.x);
        b[u] = __ldcs(src + h * (D / 8) + at.y);
      }
    }
  };
  load(hl);
  table.fill_tokens(tid, kThreads, t0, p.num_tokens, p.positions, p.rope);
  __syncthreads();
  const bool in_rot = g < (p.rope.rot_dim >> 4);
  const RopeTurns cs = table.group(tk, in_rot ? g : 0);
  for (int h0 = hl; h0 < heads; h0 += 2 * HL) {
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int h = h0 + u * HL;
      if (h >= heads) continue;
      if (in_rot) rope_group(a[u], b[u], cs, p.rope.interleaved != 0);
      __stcs(dst + h * (D / 8) + at.x, a[u]);
      __stcs(dst + h * (D / 8) + at.y, b[u]);
    }
    load(h0 + 2 * HL);
  }
}

// A sequence's new rows: n rows from token `begin` on, the last one at position ctx - 1.
struct Seq {
  int begin, n, ctx;
};

// Lengths of sequence s; n = 0 (and an error, if `report`) when they do not fit.
__device__ __forceinline__ Seq seq_of(const AppendParams& p, int s, bool report) {
  Seq q;
  q.begin = __ldg(p.cu_seqlens + s);
  const int end = __ldg(p.cu_seqlens + s + 1);
  q.ctx = __ldg(p.context_lens + s);
  q.n = end - q.begin;
  if (q.begin < 0 || end < q.begin || end > p.num_tokens || q.n > p.max_new || q.ctx < q.n ||
      static_cast<int64_t>(q.ctx) > (static_cast<int64_t>(p.max_blocks) << p.bs_log2)) {
    if (report) flag_error(p.err, PA_DEV_ERR_BAD_INDEX);
    q.n = 0;
  }
  return q;
}

// Blocks that a sequence's new rows reach.
__device__ __forceinline__ int blocks_of(const AppendParams& p, const Seq& q) {
  return q.n ? ((q.ctx - 1) >> p.bs_log2) - ((q.ctx - q.n) >> p.bs_log2) + 1 : 0;
}

// The rows of sequence s that go to the j-th block they reach: `rows` rows from offset r0 of
// the block, tokens tok0 ...
struct Span {
  int id;  // physical block, unchecked
  int rows, r0;
  int64_t tok0;
};

__device__ __forceinline__ Span span_of(const AppendParams& p, const Seq& q, int s, int j) {
  const int pos0 = q.ctx - q.n;
  const int blk = (pos0 >> p.bs_log2) + j;
  const int64_t start = static_cast<int64_t>(blk) << p.bs_log2;
  const int64_t stop = start + (1ll << p.bs_log2);
  const int lo = start > pos0 ? static_cast<int>(start) : pos0;
  const int hi = stop < q.ctx ? static_cast<int>(stop) : q.ctx;
  Span u;
  // read while the rows' loads are on their way; checked by the caller after issuing them
  u.id = __ldg(p.block_tables + static_cast<int64_t>(s) * p.max_blocks + blk);
  u.rows = hi - lo;
  u.r0 = lo & ((1 << p.bs_log2) - 1);
  u.tok0 = q.begin + (lo - pos0);
  return u;
}

// Largest finite magnitude (bits) of N vectors.
template <int N>
__device__ __forceinline__ unsigned top_of(const uint4 (&a)[N], const uint4 (&b)[N]) {
  unsigned top = 0;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    top = abs_max2(abs_max2(top, a[i].x), a[i].y);
    top = abs_max2(abs_max2(top, a[i].z), a[i].w);
    top = abs_max2(abs_max2(top, b[i].x), b[i].y);
    top = abs_max2(abs_max2(top, b[i].z), b[i].w);
  }
  if (max(top & 0xffffu, top >> 16) >= kInfBits) {  // rare: only finite values set the scale
    top = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      top = finite_max2(finite_max2(top, a[i].x), a[i].y);
      top = finite_max2(finite_max2(top, a[i].z), a[i].w);
      top = finite_max2(finite_max2(top, b[i].x), b[i].y);
      top = finite_max2(finite_max2(top, b[i].z), b[i].w);
    }
  }
  return max(top & 0xffffu, top >> 16);
}

// At most one new row per sequence (a decode step). CTA i takes the queries of token i and the
// K and V rows of sequence i, a head per D / 16 threads: one table holds the turns of both
// tokens (the same one, as a rule), and the few dependent reads (lengths, block id, old scale)
// run beside the rows'.
template <int D>
__global__ void __launch_bounds__(kThreads) append_one_kernel(const AppendParams p) {
  constexpr int NG = D / 16;             // threads per head
  constexpr int HL = kThreads / NG;      // heads side by side
  __shared__ RopeTable<2, D / 2> table;  // row 0: the queries' token, row 1: the keys'
  __shared__ int grown[HL];              // K or V heads of a pass whose scale grew
  __shared__ float factor[HL];
  __shared__ int num_grown[2];           // of even and odd passes
  const int tid = threadIdx.x;
  const int i = blockIdx.x;
  const int grp = tid % NG, hl = tid / NG;
  const int2 at = rope_vectors(grp, p.rope);
  const bool in_rot = grp < (p.rope.rot_dim >> 4);
  Seq seq{};
  if (i < p.num_seqs) seq = seq_of(p, i, tid == 0);
  const bool stored = seq.n > 0;
  Span u{};
  if (stored) u = span_of(p, seq, i, 0);
  const int q_heads = i < p.num_tokens ? p.num_q_heads : 0;
  const int kv_heads = stored ? 2 * p.num_kv_heads : 0;  // K heads, then V heads
  const int heads = q_heads + kv_heads;

  // the first pass's vectors, then the turns
  auto source = [&](int h) -> const uint4* {
    if (h < q_heads) return reinterpret_cast<const uint4*>(p.q + i * p.q_stride + h * D);
    h -= q_heads;
    return h < p.num_kv_heads
               ? reinterpret_cast<const uint4*>(p.k + u.tok0 * p.k_stride + h * D)
               : reinterpret_cast<const uint4*>(p.v + u.tok0 * p.v_stride + (h - p.num_kv_heads) * D);
  };
  const bool good = stored && u.id >= 0 && u.id < p.num_blocks;
  auto scale_of = [&](int kv) {  // kv: K head, or num_kv_heads + V head
    return (kv < p.num_kv_heads ? p.k_scales + kv : p.v_scales + kv - p.num_kv_heads) +
           static_cast<int64_t>(u.id) * p.num_kv_heads;
  };
  uint4 a = make_uint4(0, 0, 0, 0), b = a;
  float old = 0.f;  // of a block that starts here
  auto fetch = [&](int h) {
    if (h >= heads) return;
    a = __ldg(source(h) + at.x);
    b = __ldg(source(h) + at.y);
    old = h >= q_heads && good && u.r0 ? __ldcg(scale_of(h - q_heads)) : 0.f;
  };
  fetch(hl);
  if (stored && !good && tid == 0) flag_error(p.err, PA_DEV_ERR_BAD_INDEX);
  const int half = p.rope.rot_dim >> 1;
  if (half > 0) {
    // one (row, frequency) per thread and pass
    for (int k = tid; k < 2 * half; k += kThreads) {
      const int row = k / half, f = k - row * half;
      if (row == 0 ? q_heads > 0 : good) {
        const int pos = __ldg(p.positions + (row == 0 ? i : u.tok0));
        table.put(row, f, rope_turn(pos, rope_rate(__ldg(p.rope.inv_freq + f)), p.rope.amplitude));
      }
    }
  }
  if (tid < 2) num_grown[tid] = 0;
  __syncthreads();
  const int64_t row_bytes = static_cast<int64_t>(p.num_kv_heads) * D;
  auto codes_of = [&](int kv) {
    const bool is_v = kv >= p.num_kv_heads;
    return (is_v ? p.v_codes : p.k_codes) +
           ((static_cast<int64_t>(u.id) << p.bs_log2) * p.num_kv_heads + (is_v ? kv - p.num_kv_heads : kv)) * D;
  };
  int odd = 0;
  for (int h0 = 0; h0 < heads; h0 += HL, odd ^= 1) {
    const int h = h0 + hl, kv = h - q_heads;
    const bool is_q = h < q_heads;
    const bool row = h < heads && !is_q && good;
    if (in_rot && (is_q || (row && kv < p.num_kv_heads)))
      rope_group(a, b, table.group(is_q ? 0 : 1, grp), p.rope.interleaved != 0);
    if (is_q) {
      uint4* dst = reinterpret_cast<uint4*>(p.q_out + i * p.q_out_stride + h * D);
      dst[at.x] = a;
      dst[at.y] = b;
    }
    // the head's threads agree on its scale
    const uint4 va[1] = {a}, vb[1] = {b};
    unsigned amax = row ? top_of(va, vb) : 0;
#pragma unroll
    for (int o = NG / 2; o > 0; o >>= 1) amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    __syncwarp();  // every thread of a head has read its old scale
    if (row) {
      const float need = exp2_int(scale_exponent(amax));
      const float scale = old >= need ? old : need;
      const float inv = __frcp_rn(scale);
      uint8_t* dst = codes_of(kv) + u.r0 * row_bytes;
      *reinterpret_cast<uint2*>(dst + at.x * 8) = quantise8(a, inv);
      *reinterpret_cast<uint2*>(dst + at.y * 8) = quantise8(b, inv);
      if (scale != old && grp == 0) {
        *scale_of(kv) = scale;
        if (u.r0 > 0) {
          const int n = atomicAdd(&num_grown[odd], 1);
          grown[n] = kv;
          factor[n] = __fdiv_rn(old, scale);
        }
      }
    }
    fetch(h + HL);
    // rows that were in the block before, when its scale grew: by the whole CTA
    __syncthreads();
    // the next pass counts in the other word, last read before the barrier that ended its pass
    if (tid == 0) num_grown[odd ^ 1] = 0;
    for (int n = 0; n < num_grown[odd]; ++n)
      requantise_rows<D>(codes_of(grown[n]), row_bytes, u.r0, factor[n], tid, kThreads);
    __syncthreads();
  }
}

// The new rows of a block that takes at most ROWS, of head g of K or V, by one warp.
template <int D, int ROWS>
__device__ __forceinline__ void append_few(const AppendParams& p, const Span& u, bool is_v, int g,
                                           int lane) {
  constexpr int NG = D / 16;         // threads per row
  constexpr int RL = 32 / NG;        // rows side by side
  constexpr int RT = ROWS / RL;      // rows a thread keeps in registers
  const int grp = lane % NG, rl = lane / NG;
  const int2 at = rope_vectors(grp, p.rope);
  const bool turned = !is_v && grp < (p.rope.rot_dim >> 4);
  const int64_t vstride = (is_v ? p.v_stride : p.k_stride) / 8;
  const uint4* src = reinterpret_cast<const uint4*>(is_v ? p.v : p.k) + (u.tok0 + rl) * vstride +
                     g * (D / 8);
  uint4 a[RT], b[RT];
#pragma unroll
  for (int i = 0; i < RT; ++i) {
    a[i] = b[i] = make_uint4(0, 0, 0, 0);
    if (rl + i * RL < u.rows) {
      a[i] = __ldg(src + i * (RL * vstride) + at.x);
      b[i] = __ldg(src + i * (RL * vstride) + at.y);
    }
  }
  if (u.id < 0 || u.id >= p.num_blocks) {
    if (lane == 0) flag_error(p.err, PA_DEV_ERR_BAD_INDEX);
    return;
  }
  float* scale_at = (is_v ? p.v_scales : p.k_scales) + static_cast<int64_t>(u.id) * p.num_kv_heads + g;
  // read by the lane that writes it below, so that no other lane can see the new one
  float old = 0.f;
  if (lane == 0 && u.r0) old = __ldcg(scale_at);
  if (turned) {
    unsigned long long rate[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) rate[e] = rope_rate(__ldg(p.rope.inv_freq + 8 * grp + e));
#pragma unroll
    for (int i = 0; i < RT; ++i) {
      if (rl + i * RL < u.rows) {
        const int pos = __ldg(p.positions + u.tok0 + rl + i * RL);
        RopeTurns cs;
#pragma unroll
        for (int e = 0; e < 8; ++e) set_turn(cs, e, rope_turn(pos, rate[e], p.rope.amplitude));
        rope_group(a[i], b[i], cs, p.rope.interleaved != 0);
      }
    }
  }
  const unsigned amax = __reduce_max_sync(0xffffffffu, top_of(a, b));
  old = __shfl_sync(0xffffffffu, old, 0);
  const float need = exp2_int(scale_exponent(amax));
  const float scale = old >= need ? old : need;  // old is 0 for a block that starts here
  const float inv = __frcp_rn(scale);
  if (lane == 0 && scale != old) *scale_at = scale;
  uint8_t* codes = (is_v ? p.v_codes : p.k_codes) +
                   ((static_cast<int64_t>(u.id) << p.bs_log2) * p.num_kv_heads + g) * D;
  const int64_t row_bytes = static_cast<int64_t>(p.num_kv_heads) * D;
#pragma unroll
  for (int i = 0; i < RT; ++i) {
    if (rl + i * RL < u.rows) {
      uint8_t* dst = codes + (u.r0 + rl + i * RL) * row_bytes;
      *reinterpret_cast<uint2*>(dst + at.x * 8) = quantise8(a[i], inv);
      *reinterpret_cast<uint2*>(dst + at.y * 8) = quantise8(b[i], inv);
    }
  }
  // rows that were in the block before, when its scale grew
  if (u.r0 > 0 && scale != old)
    requantise_rows<D>(codes, row_bytes, u.r0, __fdiv_rn(old, scale), lane, 32);
}

// Both factors (rope.cuh) of the turns at ROWS consecutive positions; a position that does not
// follow is turned by the series.
template <int D, int ROWS>
struct TurnTables {
  static constexpr int HIGH = ROWS / kRopeLow + 1;
  RopeTable<HIGH, D / 2> high;
  RopeTable<kRopeLow, D / 2> low;

  // base: the first position, its low bits cleared
  __device__ __forceinline__ void fill(const RopeParams& r, unsigned base) {
    // one frequency per thread, rows `apart` apart
    const int half = r.rot_dim >> 1, tid = threadIdx.x;
    const int apart = kThreads / half, row0 = tid / half, f = tid - row0 * half;
    if (row0 < apart) {
      const unsigned long long rate = rope_rate(__ldg(r.inv_freq + f));
      for (int row = row0; row < kRopeLow; row += apart) low.put(row, f, rope_low(row, rate));
      for (int row = row0; row < HIGH; row += apart)
        high.put(row, f, rope_high(static_cast<int>(base + row * kRopeLow), rate, r.amplitude));
    }
  }
  __device__ __forceinline__ RopeTurns at(const RopeParams& r, unsigned base, int pos, int grp) const {
    const unsigned row = (static_cast<unsigned>(pos) - base) / kRopeLow;
    RopeTurns cs;
    if (row < HIGH) {
      cs = rope_product(high.group(row, grp), low.group(pos & (kRopeLow - 1), grp));
    } else {
#pragma unroll 1
      for (int e = 0; e < 8; ++e) {
        const float2 t = rope_turn(pos, rope_rate(__ldg(r.inv_freq + 8 * grp + e)), r.amplitude);
#pragma unroll
        for (int k = 0; k < 8; ++k)
          if (k == e) set_turn(cs, k, t);
      }
    }
    return cs;
  }
};

// Chunks in blocks of 16 or 32: a CTA takes the new rows of 64 aligned positions (two or four
// blocks) of HT heads, as below, with a largest magnitude for every block: a row's threads
// agree by shuffles, the rows of a block by a maximum in shared memory.
template <int D, int HT>
struct TileShared {
  static constexpr int kRows = 64;
  static constexpr int kBlocks = 4;  // of 16 rows
  TurnTables<D, kRows> turns;
  unsigned top[kBlocks][HT];
};

template <int D, int HT>
__device__ __forceinline__ void append_tile(const AppendParams& p, const Seq& q, int s, int j, bool is_v,
                                            int g, TileShared<D, HT>& sm) {
  constexpr int NG = D / 16, RL = kThreads / NG, RT = TileShared<D, HT>::kRows / RL;
  constexpr int TILE = TileShared<D, HT>::kRows, NB = TileShared<D, HT>::kBlocks;
  const int tid = threadIdx.x, grp = tid % NG, rl = tid / NG;
  const int2 at = rope_vectors(grp, p.rope);
  const int pos0 = q.ctx - q.n;
  const int64_t start = static_cast<int64_t>(pos0 / TILE + j) * TILE;
  const int lo = start > pos0 ? static_cast<int>(start) : pos0;
  const int rows = static_cast<int>(min(start + TILE, static_cast<int64_t>(q.ctx)) - lo);
  const int off = lo - static_cast<int>(start);  // of the first row
  const int64_t tok0 = q.begin + (lo - pos0);
  const int bs_mask = (1 << p.bs_log2) - 1;
  const int32_t* ids = p.block_tables + static_cast<int64_t>(s) * p.max_blocks + (start >> p.bs_log2);
  auto id_of = [&](int sub) { return __ldg(ids + sub); };
  auto good = [&](int id) { return id >= 0 && id < p.num_blocks; };
  const int64_t vstride = (is_v ? p.v_stride : p.k_stride) / 8;
  const uint4* src = reinterpret_cast<const uint4*>(is_v ? p.v : p.k) + (tok0 + rl) * vstride + g * (D / 8);
  uint4 a[RT][HT], b[RT][HT];
  int id[RT];
#pragma unroll
  for (int i = 0; i < RT; ++i) {
    const uint4* row = src + i * (RL * vstride);
    const int r = rl + i * RL;
    id[i] = r < rows ? id_of((off + r) >> p.bs_log2) : 0;
#pragma unroll
    for (int h = 0; h < HT; ++h) {
      a[i][h] = b[i][h] = make_uint4(0, 0, 0, 0);
      if (r < rows) {
        a[i][h] = __ldg(row + h * (D / 8) + at.x);
        b[i][h] = __ldg(row + h * (D / 8) + at.y);
      }
    }
  }
  // the first block may hold rows already
  const int sub0 = off >> p.bs_log2, r0 = off & bs_mask;
  const int id0 = id_of(sub0);
  float* scales = (is_v ? p.v_scales : p.k_scales) + g;
  float old[HT];
#pragma unroll
  for (int h = 0; h < HT; ++h)
    old[h] = r0 && good(id0) ? __ldcg(scales + static_cast<int64_t>(id0) * p.num_kv_heads + h) : 0.f;
  if (tid < NB * HT) sm.top[tid / HT][tid % HT] = 0;
  const bool turns = !is_v && p.rope.rot_dim > 0;
  const int32_t* pos = p.positions + tok0;
  unsigned base = 0;
  if (turns) {
    base = static_cast<unsigned>(__ldg(pos)) & ~(kRopeLow - 1u);
    sm.turns.fill(p.rope, base);
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < RT; ++i) {
    const int r = rl + i * RL;
    if (turns && r < rows && grp < (p.rope.rot_dim >> 4)) {
      const RopeTurns cs = sm.turns.at(p.rope, base, __ldg(pos + r), grp);
#pragma unroll
      for (int h = 0; h < HT; ++h) rope_group(a[i][h], b[i][h], cs, p.rope.interleaved != 0);
    }
    __syncwarp();
#pragma unroll
    for (int h = 0; h < HT; ++h) {
      const uint4 va[1] = {a[i][h]}, vb[1] = {b[i][h]};
      unsigned t = top_of(va, vb);
#pragma unroll
      for (int o = NG / 2; o > 0; o >>= 1) t = max(t, __shfl_xor_sync(0xffffffffu, t, o));
      if (grp == 0 && r < rows) atomicMax(&sm.top[(off + r) >> p.bs_log2][h], t);
    }
  }
  __syncthreads();
  auto scale_of = [&](int sub, int h, float before) {
    const float need = exp2_int(scale_exponent(sm.top[sub][h]));
    return sub == sub0 && before >= need ? before : need;
  };
  uint8_t* pool = is_v ? p.v_codes : p.k_codes;
  const int64_t row_bytes = static_cast<int64_t>(p.num_kv_heads) * D;
#pragma unroll
  for (int i = 0; i < RT; ++i) {
    const int r = rl + i * RL;
    if (r >= rows) continue;
    if (!good(id[i])) {
      if (grp == 0) flag_error(p.err, PA_DEV_ERR_BAD_INDEX);
      continue;
    }
    uint8_t* dst = pool + ((static_cast<int64_t>(id[i]) << p.bs_log2) + ((off + r) & bs_mask)) * row_bytes + g * D;
#pragma unroll
    for (int h = 0; h < HT; ++h) {
      const float inv = __frcp_rn(scale_of((off + r) >> p.bs_log2, h, old[h]));
      *reinterpret_cast<uint2*>(dst + h * D + at.x * 8) = quantise8(a[i][h], inv);
      *reinterpret_cast<uint2*>(dst + h * D + at.y * 8) = quantise8(b[i][h], inv);
    }
  }
  if (r0 > 0 && good(id0)) {  // rows that were in the first block before, when its scale grew
#pragma unroll
    for (int h = 0; h < HT; ++h) {
      const float scale = scale_of(sub0, h, old[h]);
      if (scale != old[h])
        requantise_rows<D>(pool + (static_cast<int64_t>(id0) << p.bs_log2) * row_bytes + (g + h) * D, row_bytes, r0,
                           __fdiv_rn(old[h], scale), tid, kThreads);
    }
  }
  const int sub = sub0 + tid / HT, h = tid % HT;
  if (sub <= (off + rows - 1) >> p.bs_log2 && good(id_of(sub))) {  // a thread per block and head
    float* to = scales + static_cast<int64_t>(id_of(sub)) * p.num_kv_heads + h;
    const float before = sub == sub0 && r0 ? __ldcg(to) : 0.f;
    const float scale = scale_of(sub, h, before);
    if (scale != before) *to = scale;
  }
}

// Many new rows per block. A thread keeps RH (row, head) pairs in registers (8: 64 registers),
// so a CTA takes RL * RH / HT rows of HT heads (RH 8: 64 rows of 4 heads, 128 of 2 or 256 of
// one at 128 dims), all in registers between the scan for the largest magnitude and the
// quantising; a block with more rows is shared by a cluster of CTAs, which exchange their
// largest magnitudes through distributed shared memory. HT is the largest that holds a block's
// rows in one CTA: the turns of a row are then formed once for HT heads, and a row's HT heads
// (256 bytes each) are read together. (Clusters of 64 rows of 4 heads for blocks of 256
// measured 37.5 us without turns against 25 for one CTA of 256 rows of one head, 16384 tokens
// of 8 kv heads: a cluster waits for its slowest load. With the turns that case's launch takes
// 40 us, 2.5 TB/s: bound by each CTA's loads and stores not overlapping.)
template <int D, int HT, int RH>
struct ManyShared {
  static constexpr int RL = kThreads / (D / 16);  // rows side by side
  static constexpr int RT = RH / HT;              // rows per thread
  static constexpr int CAP = RL * RT;             // rows of a CTA
  TurnTables<D, CAP> turns;
  unsigned warp_top[kThreads / 32][HT];
  unsigned cta_top[kMaxCluster][HT];
};

template <int D, int HT, int RH>
__device__ __forceinline__ void append_many(const AppendParams& p, const Span& u, bool is_v, int g,
                                            ManyShared<D, HT, RH>& tables) {
  using M = ManyShared<D, HT, RH>;
  constexpr int NG = D / 16, RL = M::RL, RT = M::RT, CAP = M::CAP;
  cg::cluster_group cluster = cg::this_cluster();
  const int ranks = p.cluster, rank = static_cast<int>(cluster.block_rank());
  const int tid = threadIdx.x;
  const int grp = tid % NG, rl = tid / NG;
  const int2 at = rope_vectors(grp, p.rope);
  const bool turned = !is_v && grp < (p.rope.rot_dim >> 4);
  const int64_t vstride = (is_v ? p.v_stride : p.k_stride) / 8;
  const int mine = rank * CAP + rl;  // first row of this thread
  const uint4* src = reinterpret_cast<const uint4*>(is_v ? p.v : p.k) + (u.tok0 + mine) * vstride +
                     g * (D / 8);
  uint4 a[RT][HT], b[RT][HT];
#pragma unroll
  for (int i = 0; i < RT; ++i) {
    const uint4* row = src + i * (RL * vstride);
    const bool in = mine + i * RL < u.rows;
#pragma unroll
    for (int h = 0; h < HT; ++h) {
      a[i][h] = b[i][h] = make_uint4(0, 0, 0, 0);
      if (in) {
        a[i][h] = __ldg(row + h * (D / 8) + at.x);
        b[i][h] = __ldg(row + h * (D / 8) + at.y);
      }
    }
  }
  if (u.id < 0 || u.id >= p.num_blocks) {  // so for the whole cluster
    if (tid == 0 && rank == 0) flag_error(p.err, PA_DEV_ERR_BAD_INDEX);
    return;
  }
  if (ranks > 1) cluster.barrier_arrive();  // this CTA is here: its shared memory may be written
  const int64_t scale_row = static_cast<int64_t>(u.id) * p.num_kv_heads + g;
  float* scales = is_v ? p.v_scales : p.k_scales;
  float old[HT];
#pragma unroll
  for (int h = 0; h < HT; ++h) old[h] = u.r0 ? __ldcg(scales + scale_row + h) : 0.f;

  const int half = p.rope.rot_dim >> 1;
  if (!is_v && half > 0 && rank * CAP < u.rows) {
    // both factors of the CTA's positions, while its rows are on their way
    const int32_t* pos = p.positions + u.tok0;
    const unsigned base = static_cast<unsigned>(__ldg(pos + rank * CAP)) & ~(kRopeLow - 1u);
    tables.turns.fill(p.rope, base);
    __syncthreads();
    if (turned) {
#pragma unroll
      for (int i = 0; i < RT; ++i) {
        if (mine + i * RL >= u.rows) continue;
        const RopeTurns cs = tables.turns.at(p.rope, base, __ldg(pos + mine + i * RL), grp);
#pragma unroll
        for (int h = 0; h < HT; ++h) rope_group(a[i][h], b[i][h], cs, p.rope.interleaved != 0);
      }
    }
  }

#pragma unroll
  for (int h = 0; h < HT; ++h) {
    uint4 ah[RT], bh[RT];
#pragma unroll
    for (int i = 0; i < RT; ++i) {
      ah[i] = a[i][h];
      bh[i] = b[i][h];
    }
    const unsigned t = __reduce_max_sync(0xffffffffu, top_of(ah, bh));
    if ((tid & 31) == 0) tables.warp_top[tid >> 5][h] = t;
  }
  __syncthreads();
  if (ranks > 1) {
    cluster.barrier_wait();
    if (tid < ranks * HT) {  // this CTA's maximum of head h to rank r
      const int r = tid / HT, h = tid % HT;
      unsigned t = 0;
#pragma unroll
      for (int w = 0; w < kThreads / 32; ++w) t = max(t, tables.warp_top[w][h]);
      *cluster.map_shared_rank(&tables.cta_top[rank][h], r) = t;
    }
    cluster.sync();
  }
  uint8_t* codes = (is_v ? p.v_codes : p.k_codes) +
                   ((static_cast<int64_t>(u.id) << p.bs_log2) * p.num_kv_heads + g) * D;
  const int64_t row_bytes = static_cast<int64_t>(p.num_kv_heads) * D;
  uint8_t* first = codes + (u.r0 + mine) * row_bytes;
#pragma unroll
  for (int h = 0; h < HT; ++h) {
    unsigned t = 0;
    if (ranks > 1) {
      for (int r = 0; r < ranks; ++r) t = max(t, tables.cta_top[r][h]);
    } else {
#pragma unroll
      for (int w = 0; w < kThreads / 32; ++w) t = max(t, tables.warp_top[w][h]);
    }
    const float need = exp2_int(scale_exponent(t));
    const float scale = old[h] >= need ? old[h] : need;  // old is 0 for a block that starts here
    if (tid == 0 && rank == 0 && scale != old[h]) scales[scale_row + h] = scale;
    const float inv = __frcp_rn(scale);
#pragma unroll
    for (int i = 0; i < RT; ++i) {
      if (mine + i * RL < u.rows) {
        uint8_t* dst = first + i * (RL * row_bytes) + h * D;
        *reinterpret_cast<uint2*>(dst + at.x * 8) = quantise8(a[i][h], inv);
        *reinterpret_cast<uint2*>(dst + at.y * 8) = quantise8(b[i][h], inv);
      }
    }
    // rows that were in the block before, when its scale grew
    if (u.r0 > 0 && scale != old[h])
      requantise_rows<D>(codes + h * D, row_bytes, u.r0, __fdiv_rn(old[h], scale),
                         rank * kThreads + tid, ranks * kThreads);
  }
}

// The units as the host bounds them: max_new rows' blocks for every sequence, of which those
// past a sequence's own have nothing to do. Few rows a block: a warp per unit.
template <int D, int ROWS>
__global__ void __launch_bounds__(kThreads) append_few_kernel(const AppendParams p) {
  __shared__ RopeTable<kQTokens, D / 2> table;
  if (blockIdx.x < static_cast<unsigned>(p.q_ctas)) {
    turn_queries<D>(p, table);
    return;
  }
  const int lane = threadIdx.x & 31;
  const int64_t unit =
      static_cast<int64_t>(blockIdx.x - p.q_ctas) * (kThreads / 32) + (threadIdx.x >> 5);
  const int64_t per_seq = static_cast<int64_t>(p.span) * 2 * p.num_kv_heads;
  if (unit >= per_seq * p.num_seqs) return;
  const int s = static_cast<int>(unit / per_seq);
  int rest = static_cast<int>(unit - s * per_seq);
  const int g = rest % p.num_kv_heads;
  rest /= p.num_kv_heads;
  const Seq q = seq_of(p, s, lane == 0);
  if ((rest >> 1) < blocks_of(p, q))
    append_few<D, ROWS>(p, span_of(p, q, s, rest >> 1), rest & 1, g, lane);
}

// The same with a CTA or a cluster per unit of HT heads. (BEHIND at compile time: the wait in the
// code took calls of a few tokens 0.15 us.)
template <int D, int HT, int RH, bool BEHIND>
__global__ void __launch_bounds__(kThreads, RH == 8 ? 2 : 3) append_many_kernel(const AppendParams p) {
  __shared__ union {
    RopeTable<kQTokens, D / 2> queries;
    ManyShared<D, HT, RH> many;
  } sm;
  if (blockIdx.x < static_cast<unsigned>(p.q_ctas)) {  // whole clusters
    turn_queries<D>(p, sm.queries);
    return;
  }
  const int64_t unit = (blockIdx.x - p.q_ctas) / p.cluster;
  const int hgroups = p.num_kv_heads / HT;
  const int64_t per_seq = static_cast<int64_t>(p.span) * 2 * hgroups;
  const int s = static_cast<int>(unit / per_seq);
  int rest = static_cast<int>(unit - s * per_seq);
  const int g = rest % hgroups * HT;
  rest /= hgroups;
  const Seq q = seq_of(p, s, threadIdx.x == 0);
  if ((rest >> 1) < blocks_of(p, q))
    append_many<D, HT, RH>(p, span_of(p, q, s, rest >> 1), rest & 1, g, sm.many);
  // complete, for what follows in the stream, only once the queries' kernel is
  if (BEHIND && blockIdx.x == 0) asm volatile("griddepcontrol.wait;" ::: "memory");
}

// A CTA per 64 positions and HT heads.
template <int D, int HT, bool BEHIND>
__global__ void __launch_bounds__(kThreads, HT == 4 ? 2 : 3) append_tile_kernel(const AppendParams p) {
  __shared__ union {
    RopeTable<kQTokens, D / 2> queries;
    TileShared<D, HT> tile;
  } sm;
  if (blockIdx.x < static_cast<unsigned>(p.q_ctas)) {
    turn_queries<D>(p, sm.queries);
    return;
  }
  const int64_t unit = blockIdx.x - p.q_ctas;
  const int hgroups = p.num_kv_heads / HT;
  const int64_t per_seq = static_cast<int64_t>(p.span) * 2 * hgroups;
  const int s = static_cast<int>(unit / per_seq);
  int rest = static_cast<int>(unit - s * per_seq);
  const int g = rest % hgroups * HT;
  rest /= hgroups;
  const Seq q = seq_of(p, s, threadIdx.x == 0);
  constexpr int TILE = TileShared<D, HT>::kRows;
  if (q.n > 0 && (rest >> 1) <= (q.ctx - 1) / TILE - (q.ctx - q.n) / TILE)
    append_tile<D, HT>(p, q, s, rest >> 1, rest & 1, g, sm.tile);
  // complete, for what follows in the stream, only once the queries' kernel is
  if (BEHIND && blockIdx.x == 0) asm volatile("griddepcontrol.wait;" ::: "memory");
}

// Batches whose sequences' new rows differ much, one long chunk beside many single tokens: most
// of the units above would have nothing to do. Here every CTA (or cluster) counts the
// sequences' own units, a scan over 1024 sequences at a time, and the CTAs that fit the GPU take
// them in turn; in a block that takes few rows, eight heads are one unit, a warp each (MANY:
// some take more). The scan costs 2 - 3 us.
template <int D, bool MANY>
__global__ void __launch_bounds__(kThreads, 2) append_ragged_kernel(const AppendParams p) {
  constexpr int kEach = kWindow / kThreads;
  constexpr int FEW = MANY ? kVeryFewRows : kFewRows;
  __shared__ union {
    RopeTable<kQTokens, D / 2> queries;
    ManyShared<D, 1, 8> many;
  } sm;
  __shared__ long long first_unit[kWindow];
  __shared__ Seq seqs[kWindow];
  __shared__ long long warp_sum[kThreads / 32];
  if (blockIdx.x < static_cast<unsigned>(p.q_ctas)) {  // whole clusters
    turn_queries<D>(p, sm.queries);
    return;
  }
  const int ranks = p.cluster, rank = blockIdx.x % ranks;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int few_units = (2 * p.num_kv_heads + 8 * ranks - 1) / (8 * ranks);  // of a block
  const int many_units = 2 * p.num_kv_heads;
  // a sequence's blocks, and whether its first and its last one take few rows
  struct Blocks {
    int n;
    bool first, last;
  };
  auto counted = [&](const Seq& q) {
    const int mask = (1 << p.bs_log2) - 1;
    const int left = mask + 1 - ((q.ctx - q.n) & mask);  // rows to the first block's end
    Blocks b;
    b.n = blocks_of(p, q);
    b.first = b.n > 0 && min(q.n, left) <= FEW;
    b.last = b.n > 1 && ((q.ctx - 1) & mask) < FEW;
    return b;
  };
  const int stride = (gridDim.x - p.q_ctas) / ranks;
  int64_t unit = (blockIdx.x - p.q_ctas) / ranks;  // counted from the window's first
  for (int s0 = 0; s0 < p.num_seqs; s0 += kWindow) {
    const int count = min(kWindow, p.num_seqs - s0);
    long long mine[kEach], sum = 0;
#pragma unroll
    for (int e = 0; e < kEach; ++e) {
      const int i = tid * kEach + e;
      mine[e] = sum;
      if (i < count) {
        const Seq q = seq_of(p, s0 + i, blockIdx.x == static_cast<unsigned>(p.q_ctas));
        seqs[i] = q;
        const Blocks b = counted(q);
        const int few = MANY ? b.first + b.last : b.n;
        sum += static_cast<long long>(few) * few_units + static_cast<long long>(b.n - few) * many_units;
      }
    }
    long long upto = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long up = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += up;
    }
    if (lane == 31) warp_sum[warp] = upto;
    __syncthreads();
    long long before = upto - sum, total = 0;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) {
      if (w < warp) before += warp_sum[w];
      total += warp_sum[w];
    }
#pragma unroll
    for (int e = 0; e < kEach; ++e)
      if (tid * kEach + e < count) first_unit[tid * kEach + e] = before + mine[e];
    __syncthreads();
    for (; unit < total; unit += stride) {
      int i = 0;  // the last sequence whose first unit is not after this one
      for (int n = count; n > 1;) {
        const int half = n >> 1;
        if (first_unit[i + half] <= unit) i += half, n -= half;
        else n = half;
      }
      const Seq q = seqs[i];
      const Blocks b = counted(q);
      // a sequence's units: of its blocks with many rows, then of those with few
      int64_t at = unit - first_unit[i];
      if constexpr (MANY) {
        const int64_t many = static_cast<int64_t>(b.n - b.first - b.last) * many_units;
        if (at < many) {
          const int j = static_cast<int>(at / many_units), rest = static_cast<int>(at - j * static_cast<int64_t>(many_units));
          const bool is_v = rest >= p.num_kv_heads;
          __syncthreads();  // the tables are free
          append_many<D, 1, 8>(p, span_of(p, q, s0 + i, j + b.first), is_v,
                            is_v ? rest - p.num_kv_heads : rest, sm.many);
          continue;
        }
        at -= many;
      }
      const int f = static_cast<int>(at / few_units);
      const int pair = (static_cast<int>(at - f * static_cast<int64_t>(few_units)) * ranks + rank) * (kThreads / 32) + warp;
      if (pair < 2 * p.num_kv_heads) {
        const bool is_v = pair >= p.num_kv_heads;
        append_few<D, FEW>(p, span_of(p, q, s0 + i, !MANY ? f : f == 0 && b.first ? 0 : b.n - 1), is_v,
                           is_v ? pair - p.num_kv_heads : pair, lane);
      }
    }
    unit -= total;
    __syncthreads();  // before the next window's lists
  }
}

template <class Kernel>
cudaError_t launch(Kernel kernel, const AppendParams& p, int64_t grid, cudaStream_t stream) {
  if (grid > INT32_MAX) return cudaErrorInvalidValue;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(grid));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  cfg.attrs = attr;
  if (p.cluster > 1) {  // clusters of one CTA took longer (512 tokens in blocks of 16: 10.7 us against 8.8)
    cudaLaunchAttribute& c = attr[cfg.numAttrs++];
    c.id = cudaLaunchAttributeClusterDimension;
    c.val.clusterDim.x = static_cast<unsigned>(p.cluster);
    c.val.clusterDim.y = 1;
    c.val.clusterDim.z = 1;
  }
  if (p.behind_queries) {
    cudaLaunchAttribute& c = attr[cfg.numAttrs++];
    c.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    c.val.programmaticStreamSerializationAllowed = 1;
  }
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

template <int D>
cudaError_t launch_d(AppendParams p, bool q_here, cudaStream_t stream) {
  const int bs = 1 << p.bs_log2;
  const int rows = p.max_new < bs ? p.max_new : bs;  // most new rows of one block
  if (!q_here) p.num_q_heads = 0;
  p.q_ctas = p.num_q_heads > 0 ? (p.num_tokens + kQTokens - 1) / kQTokens : 0;
  p.cluster = 1;
  if (p.max_new == 1) {
    p.behind_queries = false;
    const int grid = p.num_q_heads > 0 && p.num_tokens > p.num_seqs ? p.num_tokens : p.num_seqs;
    return launch(append_one_kernel<D>, p, grid, stream);
  }
  constexpr int CAP = ManyShared<D, 1, 8>::CAP;  // rows of one head that a CTA holds
  // heads and CTAs of a unit of many rows, when a thread keeps rh (row, head) pairs
  int ht, cluster;
  int64_t ctas;
  const int64_t spans = static_cast<int64_t>(p.num_seqs) * p.span;
  auto shape = [&](int rh) {
    const int cap = CAP * rh / 8;
    ht = p.num_kv_heads % 4 == 0 && rh == 8 && rows <= cap / 4 ? 4 : p.num_kv_heads % 2 == 0 && rows <= cap / 2 ? 2 : 1;
    cluster = 1;
    while (cluster * cap < rows * ht) cluster *= 2;
    ctas = spans * 2 * (p.num_kv_heads / ht) * cluster;
  };
  static_assert(kMaxCluster * CAP / 2 >= 1024, "the largest block");
  shape(8);
  const int64_t sms = sm_count();
  // A warp forms its rows' turns for one head, a CTA for all of its heads, but a CTA waits for its
  // rows together: warps up to 8 rows, or up to 16 when the CTAs would fill four waves. Warps /
  // CTAs, us: 64 sequences of 16 rows 11.6 / 9.0, 256 of 12 20.2 / 24.3; 64 of 30 21.0 (with registers
  // for 32 rows) / 11.5.
  const bool few = rows <= kVeryFewRows || (rows <= kFewRows && ctas > 8 * sms);
  const bool behind = p.behind_queries;
  if (few) {
    p.behind_queries = false;
    ctas = (spans * 2 * p.num_kv_heads + kThreads / 32 - 1) / (kThreads / 32);
  }
  // Counting pays beyond four waves of CTAs, when the blocks would hold an eighth of the most
  // rows on average. Without / with it, us (32 q and 8 kv heads): 255 single tokens and a chunk
  // of 8192, blocks of 256, 400 / 58; 63 and 2048 47 / 21; 15 and 2048 24.1 / 20.5; 63 and 512,
  // blocks of 16, 15.7 / 12.4; on the other side 63 and 40, blocks of 64 (1.7 waves) 7.5 / 8.5, 98
  // ragged of up to 45 (a quarter full) 15.2 / 20.5, 64 even chunks of 256 82 / 97.
  auto set_cluster = [&]() {
    p.cluster = cluster;
    p.q_ctas = (p.q_ctas + cluster - 1) / cluster * cluster;  // whole clusters
  };
  if (ctas > 8 * sms && static_cast<int64_t>(p.num_tokens) * 8 < spans * rows) {
    // as many CTAs as are resident (not beside the queries' kernel: 63 and 2048 took 22.5 us)
    p.behind_queries = false;
    set_cluster();
    const int64_t grid = p.q_ctas + 2 * sms / p.cluster * p.cluster;
    return few ? launch(append_ragged_kernel<D, false>, p, grid, stream)
               : launch(append_ragged_kernel<D, true>, p, grid, stream);
  }
  // Several small blocks a CTA. A unit a block / tiles, us: 8 sequences of 2000 rows and 8 heads in
  // blocks of 16 61.7 / 48.5, of 32 52.9 / 48.4, of 500 in blocks of 16 24.5 / 17.3, 100 rows 4.1 / 4.5.
  constexpr int TILE = TileShared<D, 1>::kRows;
  if (bs < TILE && p.max_new > kFewRows) {
    p.behind_queries = behind;
    p.span = static_cast<int>((static_cast<int64_t>(p.max_new) + TILE - 2) / TILE) + 1;
    const int64_t heads = static_cast<int64_t>(p.num_seqs) * p.span * 2 * p.num_kv_heads;
    // the most heads that leave no SM idle
    ht = p.num_kv_heads % 4 == 0 && heads > 4 * sms ? 4 : p.num_kv_heads % 2 == 0 && heads > 2 * sms ? 2 : 1;
    const int64_t grid = p.q_ctas + heads / ht;
    auto tiles = [&](auto plain, auto beside) {
      return behind ? launch(beside, p, grid, stream) : launch(plain, p, grid, stream);
    };
    if (ht == 4) return tiles(append_tile_kernel<D, 4, false>, append_tile_kernel<D, 4, true>);
    if (ht == 2) return tiles(append_tile_kernel<D, 2, false>, append_tile_kernel<D, 2, true>);
    return tiles(append_tile_kernel<D, 1, false>, append_tile_kernel<D, 1, true>);
  }
  if (few)
    return rows <= kVeryFewRows ? launch(append_few_kernel<D, kVeryFewRows>, p, p.q_ctas + ctas, stream)
                                : launch(append_few_kernel<D, kFewRows>, p, p.q_ctas + ctas, stream);
  // Half the pairs a thread (three CTAs an SM) when the units of eight leave SMs idle, or hold one
  // head's rows twice over. With eight / four, us: 1024 tokens of 8 heads, blocks of 256, 10.1 / 8.8,
  // of 64 8.9 / 8.1; 16384 of 3 heads, blocks of 64, 37.7 / 31.0; 4096 of 8, blocks of 256, 17.4 / 19.5.
  const bool half = ctas <= sms || (ht == 1 && rows <= CAP / 2);
  if (half) shape(4);
  set_cluster();
  auto many = [&](auto plain, auto behind) {
    return p.behind_queries ? launch(behind, p, p.q_ctas + ctas, stream)
                            : launch(plain, p, p.q_ctas + ctas, stream);
  };
  if (half)
    return ht == 2 ? many(append_many_kernel<D, 2, 4, false>, append_many_kernel<D, 2, 4, true>)
                   : many(append_many_kernel<D, 1, 4, false>, append_many_kernel<D, 1, 4, true>);
  if (ht == 4) return many(append_many_kernel<D, 4, 8, false>, append_many_kernel<D, 4, 8, true>);
  if (ht == 2) return many(append_many_kernel<D, 2, 8, false>, append_many_kernel<D, 2, 8, true>);
  return many(append_many_kernel<D, 1, 8, false>, append_many_kernel<D, 1, 8, true>);
}

}  // namespace

cudaError_t launch_append_blockscale(const AppendLaunch& a, cudaStream_t stream) {
  AppendParams p;
  p.q = static_cast<const __nv_bfloat16*>(a.q);
  p.k = static_cast<const __nv_bfloat16*>(a.k);
  p.v = static_cast<const __nv_bfloat16*>(a.v);
  p.q_out = static_cast<__nv_bfloat16*>(a.q_out);
  p.q_stride = a.q_stride;
  p.k_stride = a.k_stride;
  p.v_stride = a.v_stride;
  p.q_out_stride = a.q_out_stride;
  p.k_codes = static_cast<uint8_t*>(a.k_codes);
  p.v_codes = static_cast<uint8_t*>(a.v_codes);
  p.k_scales = a.k_scales;
  p.v_scales = a.v_scales;
  p.block_tables = a.block_tables;
  p.cu_seqlens = a.cu_seqlens;
  p.context_lens = a.context_lens;
  p.positions = a.positions;
  p.rope = RopeParams{a.rope.inv_freq, a.rope.rot_dim, a.rope.interleaved, a.rope.amplitude};
  p.num_seqs = a.num_seqs;
  p.num_tokens = a.num_tokens;
  p.max_new = a.max_new;
  p.bs_log2 = 31 - __builtin_clz(static_cast<unsigned>(a.cache.block_size));
  p.span = static_cast<int>((static_cast<int64_t>(a.max_new) + a.cache.block_size - 2) /
                            a.cache.block_size) + 1;
  p.max_blocks = a.max_blocks_per_seq;
  p.num_blocks = a.cache.num_blocks;
  p.num_q_heads = a.num_q_heads;
  p.num_kv_heads = a.cache.num_kv_heads;
  p.err = device_error_word();
  // Few tokens: one launch, whose first CTAs turn the queries. Many: the queries' own kernel
  // (64 registers against the units' 128, so twice the warps stream them), beside whose last
  // CTAs the units of many rows may start (16384 tokens 82.7 -> 80.0 us, 3010 16.6 -> 15.6).
  const bool q_here = a.num_tokens <= 8 * sm_count();
  p.behind_queries = !q_here && a.num_q_heads > 0;
  if (!q_here && a.num_q_heads > 0) {
    RopeStoreLaunch q{};
    q.q_out = a.q_out;
    q.q = a.q;
    q.q_out_stride = a.q_out_stride;
    q.q_stride = a.q_stride;
    q.positions = a.positions;
    q.rope = a.rope;
    q.num_tokens = a.num_tokens;
    q.num_q_heads = a.num_q_heads;
    q.head_dim = a.cache.head_dim;
    const cudaError_t e = launch_rope_store(q, stream);
    if (e != cudaSuccess) return e;
  }
  return a.cache.head_dim == 128 ? launch_d<128>(p, q_here, stream)
                                 : launch_d<64>(p, q_here, stream);
}

}  // namespace pa
