// Rotary positions of queries and keys, with the keys and values scattered into the bf16
// pools in the same pass (mini-vllm page, section 2 "KVCache": the block table decides
// where in the pre-allocated tensor K/V are written; the rotation comes before it).
//
// HBM-bound: every q, k and v value is read once and written once. A CTA takes TB tokens,
// computes their rot_dim / 2 turns each once into shared memory (angles in fixed point),
// then its threads walk over the tokens' heads, one group of 16 dims per thread and head
// (two 16-byte loads, two 16-byte stores); a thread keeps its 8 turns in registers across
// the heads. The first loads are issued before the turns are computed, so the two
// latencies overlap.
#include <cuda_bf16.h>

#include "pa_internal.h"
#include "pa_ptx.cuh"
#include "rope.cuh"

namespace pa {
namespace {

constexpr int kThreads = 256;

struct RopeStoreParams {
  const __nv_bfloat16* q;
  const __nv_bfloat16* k;
  const __nv_bfloat16* v;
  __nv_bfloat16* q_out;
  int64_t q_stride, k_stride, v_stride, q_out_stride;  // elements between tokens
  __nv_bfloat16* k_cache;
  __nv_bfloat16* v_cache;
  const int32_t* slot_mapping;
  const int32_t* positions;
  RopeParams rope;
  int num_tokens;
  int num_q_heads;
  int num_kv_heads;
  int64_t num_slots;
  unsigned* err;
};

// Where head h of token t (q heads, then k heads, then v heads) is read and written;
// dst NULL: skipped.
template <int D>
struct Head {
  const uint4* src;
  uint4* dst;
  bool turned;
};

template <int D>
__device__ __forceinline__ Head<D> head_of(const RopeStoreParams& p, int64_t t, int h,
                                           int64_t slot) {
  Head<D> r;
  r.turned = true;
  if (h < p.num_q_heads) {
    r.src = reinterpret_cast<const uint4*>(p.q + t * p.q_stride + h * D);
    r.dst = reinterpret_cast<uint4*>(p.q_out + t * p.q_out_stride + h * D);
    return r;
  }
  h -= p.num_q_heads;
  const bool is_v = h >= p.num_kv_heads;
  if (is_v) h -= p.num_kv_heads;
  r.turned = !is_v;
  r.src = reinterpret_cast<const uint4*>((is_v ? p.v + t * p.v_stride : p.k + t * p.k_stride) +
                                         h * D);
  r.dst = slot < 0 ? nullptr
                   : reinterpret_cast<uint4*>((is_v ? p.v_cache : p.k_cache) +
                                              (slot * p.num_kv_heads + h) * D);
  return r;
}

// The slot of token t: -1 when it is not stored; a slot past the pool is recorded.
__device__ __forceinline__ int64_t slot_of(const RopeStoreParams& p, int t) {
  if (p.num_kv_heads == 0) return -1;
  const int64_t slot = __ldg(p.slot_mapping + t);
  if (slot >= p.num_slots) {
    flag_error(p.err, PA_DEV_ERR_BAD_INDEX);
    return -1;
  }
  return slot;
}

// rot_dim a multiple of 16 (and every row 16-byte aligned): U heads at a time per thread.
template <int D, int TB, int U>
__global__ void __launch_bounds__(kThreads) rope_store_kernel(const RopeStoreParams p) {
  constexpr int NG = D / 16;                   // groups of 16 dims per head
  constexpr int HL = kThreads / (NG * TB);     // heads walked side by side
  __shared__ RopeTable<TB, D / 2> table;
  const int tid = threadIdx.x;
  // a kernel launched behind this one that does not read its outputs may start when every CTA
  // of this one has (the append of the same step's keys and values)
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int g = tid % NG;
  const int tk = (tid / NG) % TB;
  const int hl = tid / (NG * TB);
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * TB;
  const int64_t t = t0 + tk;
  const int heads = t < p.num_tokens ? p.num_q_heads + 2 * p.num_kv_heads : 0;
  const int64_t slot = heads ? slot_of(p, static_cast<int>(t)) : -1;
  const int2 at = rope_vectors(g, p.rope);

  Head<D> hd[U];
  uint4 a[U], b[U];
  auto load = [&](int h0) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int h = h0 + u * HL;
      hd[u].dst = nullptr;
      if (h < heads) hd[u] = head_of<D>(p, t, h, slot);
      if (hd[u].dst) {
        a[u] = __ldcs(hd[u].src + at.x);
        b[u] = __ldcs(hd[u].src + at.y);
      }
    }
  };
  load(hl);

  table.fill_tokens(tid, kThreads, t0, p.num_tokens, p.positions, p.rope);
  __syncthreads();
  const bool in_rot = g < (p.rope.rot_dim >> 4);
  const RopeTurns cs = table.group(tk, in_rot ? g : 0);

  for (int h0 = hl; h0 < heads; h0 += U * HL) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (!hd[u].dst) continue;
      if (in_rot && hd[u].turned) rope_group(a[u], b[u], cs, p.rope.interleaved != 0);
      __stcs(hd[u].dst + at.x, a[u]);
      __stcs(hd[u].dst + at.y, b[u]);
    }
    load(h0 + U * HL);
  }
}

// Any even rot_dim: one thread per (token, head, pair of dims); pairs past rot_dim / 2 copy
// two neighbouring dims. Every thread computes its own turn.
__global__ void __launch_bounds__(kThreads) rope_store_any_kernel(const RopeStoreParams p, int D) {
  const int heads = p.num_q_heads + 2 * p.num_kv_heads;
  const int pairs = D / 2;
  const int64_t total = static_cast<int64_t>(p.num_tokens) * heads * pairs;
  const int64_t step = static_cast<int64_t>(gridDim.x) * kThreads;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x; i < total; i += step) {
    const int64_t th = i / pairs;
    const int f = static_cast<int>(i - th * pairs);
    const int64_t t = th / heads;
    int h = static_cast<int>(th - t * heads);
    const int half = p.rope.rot_dim >> 1;
    const bool in_rot = f < half;
    const int ia = in_rot && !p.rope.interleaved ? f : 2 * f;
    const int ib = in_rot && !p.rope.interleaved ? f + half : 2 * f + 1;
    const __nv_bfloat16* src;
    __nv_bfloat16* dst;
    bool turned = in_rot;
    if (h < p.num_q_heads) {
      src = p.q + t * p.q_stride + h * D;
      dst = p.q_out + t * p.q_out_stride + h * D;
    } else {
      h -= p.num_q_heads;
      const bool is_v = h >= p.num_kv_heads;
      if (is_v) h -= p.num_kv_heads;
      const int64_t slot = slot_of(p, static_cast<int>(t));
      if (slot < 0) continue;
      src = (is_v ? p.v + t * p.v_stride : p.k + t * p.k_stride) + h * D;
      dst = (is_v ? p.v_cache : p.k_cache) + (slot * p.num_kv_heads + h) * D;
      turned = turned && !is_v;
    }
    const __nv_bfloat16 a = src[ia], b = src[ib];
    if (turned) {
      const float2 y = rope_pair(__bfloat162float(a), __bfloat162float(b),
                                 rope_turn(__ldg(p.positions + t),
                                           rope_rate(__ldg(p.rope.inv_freq + f)),
                                           p.rope.amplitude));
      dst[ia] = __float2bfloat16_rn(y.x);
      dst[ib] = __float2bfloat16_rn(y.y);
    } else {
      dst[ia] = a;
      dst[ib] = b;
    }
  }
}

template <int D>
cudaError_t launch_d(const RopeStoreParams& p, cudaStream_t stream) {
  // Tokens a CTA takes: one while they leave SMs free (64 tokens: 2.3 us against 2.5 with two).
  // Beyond four CTAs an SM two of many heads (1159 tokens of 32 q and 8 kv heads 6.8 us against 8.5
  // with one and 7.9 with four), four of fewer, whose heads do not fill a CTA (4000 tokens of 4 and 2
  // heads 5.7 against 7.9 with two) and eight when they are fewest (4.7 against 5.7 with four; 24 heads
  // 12.1 against 11.5). Four for long chunks, whose set-up then weighs least (16384 tokens: 69.3 us
  // against 69.9 with two and 92 with one).
  const int64_t sms = sm_count();
  auto launch = [&](auto kernel, int tb) {
    kernel<<<static_cast<unsigned>((p.num_tokens + tb - 1) / tb), kThreads, 0, stream>>>(p);
  };
  const int64_t wide = (p.num_q_heads + 2 * static_cast<int64_t>(p.num_kv_heads)) * D;  // values of a token
  if (p.num_tokens <= 4 * sms) {
    launch(rope_store_kernel<D, 1, 2>, 1);
  } else if (wide >= 4096 && p.num_tokens <= 32 * sms) {
    launch(rope_store_kernel<D, 2, 2>, 2);
  } else if (wide <= 1024 && p.num_tokens > 16 * sms) {
    launch(rope_store_kernel<D, 8, 2>, 8);
  } else {
    launch(rope_store_kernel<D, 4, 2>, 4);
  }
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_rope_store(const RopeStoreLaunch& a, cudaStream_t stream) {
  RopeStoreParams p;
  p.q = static_cast<const __nv_bfloat16*>(a.q);
  p.k = static_cast<const __nv_bfloat16*>(a.k);
  p.v = static_cast<const __nv_bfloat16*>(a.v);
  p.q_out = static_cast<__nv_bfloat16*>(a.q_out);
  p.q_stride = a.q_stride;
  p.k_stride = a.k_stride;
  p.v_stride = a.v_stride;
  p.q_out_stride = a.q_out_stride;
  p.k_cache = static_cast<__nv_bfloat16*>(a.k_cache);
  p.v_cache = static_cast<__nv_bfloat16*>(a.v_cache);
  p.slot_mapping = a.slot_mapping;
  p.positions = a.positions;
  p.rope = RopeParams{a.rope.inv_freq, a.rope.rot_dim, a.rope.interleaved, a.rope.amplitude};
  p.num_tokens = a.num_tokens;
  p.num_q_heads = a.num_q_heads;
  p.num_kv_heads = a.num_kv_heads;
  p.num_slots = a.num_slots;
  p.err = device_error_word();
  if (a.rope.rot_dim % 16 != 0) {
    const int64_t total = static_cast<int64_t>(a.num_tokens) *
                          (a.num_q_heads + 2 * a.num_kv_heads) * (a.head_dim / 2);
    int64_t blocks = (total + kThreads - 1) / kThreads;
    const int64_t cap = static_cast<int64_t>(sm_count()) * 16;
    if (blocks > cap) blocks = cap;
    rope_store_any_kernel<<<static_cast<unsigned>(blocks), kThreads, 0, stream>>>(p, a.head_dim);
    return cudaGetLastError();
  }
  return a.head_dim == 128 ? launch_d<128>(p, stream) : launch_d<64>(p, stream);
}

}  // namespace pa
