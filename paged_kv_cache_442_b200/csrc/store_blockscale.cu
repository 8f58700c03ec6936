// Append of new K/V rows to e4m3 pools that hold one scale for each (block, kv head), with
// the rotary positions of q and k in the same launch.
//
// The scale of a (block, kv head) is the smallest power of two s >= 2^-126 with
// max |x| <= 448 s over the rows the block has taken since its first one (position
// offset 0 starts a block afresh), never smaller than it was. e4m3 codes are themselves
// floating point, so a power of two costs no precision, and when a later row makes the
// scale grow, the stored codes move by an exact power of two: only codes that fall into
// e4m3's subnormal range are rounded again.
//
// Work: one unit per (sequence, block its new rows reach, K or V, kv head); a unit of W
// warps loads its new rows (16 dims per thread and row: two 16-byte loads) into registers,
// turns them (K), takes the largest finite magnitude on the bf16 bits, agrees on the scale
// and writes the codes; rows already in the block are rewritten only when the scale grew.
// No unit shares a (block, head) with another, so there are no atomics and the result does
// not depend on the order. HBM-bound: a bf16 row in, half of it out. Blocks of up to 256
// rows (512 at head dim 64) stay in registers between the two steps; larger ones are read
// twice (the second time from L2).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "pa_internal.h"
#include "pa_ptx.cuh"
#include "rope.cuh"

namespace pa {
namespace {

constexpr int kThreads = 256;
constexpr int kRowsPerThread = 8;  // rows a thread keeps in registers (64 registers)
constexpr int kQTokens = 2;        // tokens of a CTA that turns queries

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
  int span;  // blocks that max_new consecutive positions can reach
  int max_blocks;
  int num_blocks;
  int bs_log2;
  int num_q_heads;
  int num_kv_heads;
  int q_ctas;
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

// Largest finite magnitude of both halves, kept per half (as bits).
__device__ __forceinline__ unsigned finite_max2(unsigned acc, unsigned w) {
  const unsigned m = w & 0x7fff7fffu;
  return __vmaxu2(acc, m & __vcmpltu2(m, 0x7f807f80u));
}

// Eight bf16 values times inv -> eight codes.
__device__ __forceinline__ uint2 quantise8(const uint4& w, float inv) {
  const uint32_t* x = &w.x;
  uint32_t c[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    c[i] = __nv_cvt_float2_to_fp8x2(
        make_float2(__fmul_rn(bf16lo_to_f32(x[i]), inv), __fmul_rn(bf16hi_to_f32(x[i]), inv)),
        __NV_SATFINITE, __NV_E4M3);
  return make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
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
  table.fill(tid, kThreads, t0, p.num_tokens, p.positions, p.rope);
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

template <int D, int W>
__global__ void __launch_bounds__(kThreads) append_kernel(const AppendParams p) {
  constexpr int NG = D / 16;               // threads per row
  constexpr int UT = W * 32;               // threads per unit
  constexpr int RL = UT / NG;              // rows side by side
  constexpr int CAP = RL * kRowsPerThread;  // rows held in registers
  __shared__ RopeTable<kQTokens, D / 2> table;
  __shared__ unsigned warp_max[kThreads / 32];
  if (blockIdx.x < static_cast<unsigned>(p.q_ctas)) {
    turn_queries<D>(p, table);
    return;
  }
  const int tid = threadIdx.x;
  const int64_t unit = static_cast<int64_t>(blockIdx.x - p.q_ctas) * (kThreads / UT) + tid / UT;
  const int ut = tid % UT;
  const int64_t per_seq = static_cast<int64_t>(p.span) * 2 * p.num_kv_heads;
  if (unit >= per_seq * p.num_seqs) return;
  const int s = static_cast<int>(unit / per_seq);
  int rest = static_cast<int>(unit - s * per_seq);
  const int g = rest % p.num_kv_heads;
  rest /= p.num_kv_heads;
  const bool is_v = rest & 1;
  const int j = rest >> 1;

  // ---- the unit's rows: [r0, r0 + rows) of the block, tokens tok0 .. --------------------
  const int begin = __ldg(p.cu_seqlens + s), end = __ldg(p.cu_seqlens + s + 1);
  const int ctx = __ldg(p.context_lens + s);
  const int bs = 1 << p.bs_log2;
  const int n = end - begin;
  if (begin < 0 || n < 0 || end > p.num_tokens || n > p.max_new || ctx < n ||
      static_cast<int64_t>(ctx) > (static_cast<int64_t>(p.max_blocks) << p.bs_log2)) {
    if (ut == 0) flag_error(p.err, PA_DEV_ERR_BAD_INDEX);
    return;
  }
  if (n == 0) return;
  const int pos0 = ctx - n;
  const int blk = (pos0 >> p.bs_log2) + j;
  const int lo = max(pos0, blk << p.bs_log2);
  const int64_t blk_end = (static_cast<int64_t>(blk) + 1) << p.bs_log2;
  const int hi = blk_end < ctx ? static_cast<int>(blk_end) : ctx;
  if (lo >= hi) return;
  // the block's id and old scale are read while the rows' loads are on their way
  const int id = __ldg(p.block_tables + static_cast<int64_t>(s) * p.max_blocks + blk);
  const int rows = hi - lo;
  const int r0 = lo & (bs - 1);
  const int64_t tok0 = begin + (lo - pos0);
  const int grp = ut % NG, rl = ut / NG;
  const int2 at = rope_vectors(grp, p.rope);
  const bool turned = !is_v && grp < (p.rope.rot_dim >> 4);
  const int64_t stride = is_v ? p.v_stride : p.k_stride;
  const uint4* src = reinterpret_cast<const uint4*>((is_v ? p.v : p.k) + tok0 * stride + g * D);
  const int64_t vstride = stride / 8;

  unsigned long long rate[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) rate[e] = turned ? rope_rate(__ldg(p.rope.inv_freq + 8 * grp + e)) : 0;

  uint4 a[kRowsPerThread], b[kRowsPerThread];
  auto fetch = [&](int base) {
#pragma unroll
    for (int i = 0; i < kRowsPerThread; ++i) {
      const int r = base + rl + i * RL;
      a[i] = b[i] = make_uint4(0, 0, 0, 0);
      if (r < rows) {
        a[i] = __ldg(src + r * vstride + at.x);
        b[i] = __ldg(src + r * vstride + at.y);
      }
    }
  };
  auto turn = [&](int base) {
    if (turned) {
#pragma unroll
      for (int i = 0; i < kRowsPerThread; ++i) {
        const int r = base + rl + i * RL;
        if (r < rows) {
          const int pos = __ldg(p.positions + tok0 + r);
          RopeTurns cs;
#pragma unroll
          for (int e = 0; e < 8; ++e) set_turn(cs, e, rope_turn(pos, rate[e], p.rope.amplitude));
          rope_group(a[i], b[i], cs, p.rope.interleaved != 0);
        }
      }
    }
  };

  // ---- largest finite magnitude of the new rows, and the block's scale -------------------
  const int chunks = (rows + CAP - 1) / CAP;
  unsigned acc = 0;
  float* scale_at = nullptr;
  float old = 0.f;
  for (int c = 0; c < chunks; ++c) {
    fetch(c * CAP);
    if (c == 0) {
      if (id < 0 || id >= p.num_blocks) {  // the same for the whole unit
        if (ut == 0) flag_error(p.err, PA_DEV_ERR_BAD_INDEX);
        return;
      }
      scale_at = (is_v ? p.v_scales : p.k_scales) + static_cast<int64_t>(id) * p.num_kv_heads + g;
      old = r0 ? __ldcg(scale_at) : 0.f;
    }
    turn(c * CAP);
#pragma unroll
    for (int i = 0; i < kRowsPerThread; ++i) {
      acc = finite_max2(finite_max2(acc, a[i].x), a[i].y);
      acc = finite_max2(finite_max2(acc, a[i].z), a[i].w);
      acc = finite_max2(finite_max2(acc, b[i].x), b[i].y);
      acc = finite_max2(finite_max2(acc, b[i].z), b[i].w);
    }
  }
  unsigned amax = __reduce_max_sync(0xffffffffu, max(acc & 0xffffu, acc >> 16));
  if constexpr (W > 1) {
    if ((tid & 31) == 0) warp_max[tid >> 5] = amax;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < W; ++w) amax = max(amax, warp_max[w]);
  }
  const float need = exp2_int(scale_exponent(amax));
  const float scale = old >= need ? old : need;  // old is 0 for a block that starts here
  const float inv = __frcp_rn(scale);
  if (ut == 0 && scale != old) *scale_at = scale;

  // ---- codes of the new rows -------------------------------------------------------------
  uint8_t* codes = (is_v ? p.v_codes : p.k_codes) +
                   ((static_cast<int64_t>(id) << p.bs_log2) * p.num_kv_heads + g) * D;
  const int64_t row_bytes = static_cast<int64_t>(p.num_kv_heads) * D;
  for (int c = chunks - 1;; --c) {
#pragma unroll
    for (int i = 0; i < kRowsPerThread; ++i) {
      const int r = c * CAP + rl + i * RL;
      if (r < rows) {
        uint8_t* dst = codes + (r0 + r) * row_bytes;
        *reinterpret_cast<uint2*>(dst + at.x * 8) = quantise8(a[i], inv);
        *reinterpret_cast<uint2*>(dst + at.y * 8) = quantise8(b[i], inv);
      }
    }
    if (c == 0) break;
    fetch((c - 1) * CAP);
    turn((c - 1) * CAP);
  }

  // ---- rows that were in the block before, when its scale grew ------------------------------
  if (r0 > 0 && scale != old) {
    const float factor = __fdiv_rn(old, scale);
    constexpr int VPR = D / 16;  // 16-byte vectors of codes per row
    for (int i = ut; i < r0 * VPR; i += UT) {
      uint4* at_row = reinterpret_cast<uint4*>(codes + (i / VPR) * row_bytes) + i % VPR;
      *at_row = requantise16(*at_row, factor);
    }
  }
}

template <int D>
cudaError_t launch_d(AppendParams p, bool q_here, cudaStream_t stream) {
  const int bs = 1 << p.bs_log2;
  const int rows = p.max_new < bs ? p.max_new : bs;  // most new rows of one unit
  const int64_t units = static_cast<int64_t>(p.num_seqs) * p.span * 2 * p.num_kv_heads;
  if (!q_here) p.num_q_heads = 0;
  p.q_ctas = p.num_q_heads > 0 ? (p.num_tokens + kQTokens - 1) / kQTokens : 0;
  // a warp holds 32 rows of 128 dims in registers: units of up to 32 rows take one warp
  // (a decode step's single row, blocks of 16 and 32), larger ones eight
  if (rows <= 32) {
    const int64_t grid = p.q_ctas + (units + kThreads / 32 - 1) / (kThreads / 32);
    if (grid > INT32_MAX) return cudaErrorInvalidValue;
    append_kernel<D, 1><<<static_cast<unsigned>(grid), kThreads, 0, stream>>>(p);
  } else {
    const int64_t grid = p.q_ctas + units;
    if (grid > INT32_MAX) return cudaErrorInvalidValue;
    append_kernel<D, 8><<<static_cast<unsigned>(grid), kThreads, 0, stream>>>(p);
  }
  return cudaGetLastError();
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
  // (64 registers against the units' 128, so twice the warps stream them).
  const bool q_here = a.num_tokens <= 8 * sm_count();
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
