// Paged decode attention over e4m3 pools with one scale per (block, kv head), on the tcgen05
// tensor cores (head dim 128), persistent, with the work split evenly ahead of time.
//
// Mathematics. For a query head with kv head g and position j in block b:
//   x_j = scale * log2(e) * ks[b] * (q . code_k,j),   out = sum_j 2^(x_j - m) vs[b] code_v,j / l,
//   l = sum_j 2^(x_j - m). The tensor cores multiply the stored codes themselves
//   (kind::f8f6f4, fp32 accumulation): S = K Q^T per 128 positions (M = positions, N = rows
//   of q terms) and O^T += V^T P^T (M = head dims, N = rows of P terms).
//   * q (bf16) is three e4m3 terms of one power of two per head, y = q 2^-k with the head's
//     largest |y| in (224, 448]: hi = e4m3(y), mid = e4m3(16 (y - hi)), lo = e4m3(2^22 (y - hi -
//     mid / 16)). A power of two leaves bf16's 8 bits as they are: hi and mid hold them where
//     hi is normal, lo what hi's and mid's steps leave of smaller elements. So q is exact down
//     to 2^-18 of the head's largest element, and off by at most 2^-25 of that one below. Row
//     3h + t of the B operand is term t of head h, so a softmax thread reads its 3 G columns in
//     one load.
//   * the V scale of a block multiplies its probabilities, as a logarithm: y_j = x_j +
//     log2(vs[b]), P'_j = 2^(y_j - u), with the reference u set from the largest product.
//     (Bounding the two factors apart, by the largest x and the largest V scale, lost the
//     answer when they belonged to different positions: a large scale that nothing attends to
//     pushed all weights below the codes' range.) P' <= 2^kBound; a tile that would pass it
//     moves u and rescales O^T in tensor memory.
//   * l has a reference m of its own, set with u: m = (largest y) - (largest log2(vs) so far),
//     never lower than it was. In choosing u a scale counts as 2^-kSpread of the largest one
//     at least, so that x - m <= kSpread + kBound - kTarget: fp32 holds the sum, and one
//     maximum a head serves both. (With a second maximum, of x, 256 ragged contexts took 1.7 us
//     more.)
//   * P' is three e5m2 terms, hi = e5m2(P'), mid = e5m2(16 (P' - hi)) and lo = e5m2(256 (P' -
//     hi - mid / 16)) in rows 3h .. 3h + 2 (kind::f8f6f4 takes its operands' formats apart).
//     Three bits each: 2^-9 of P' from 2^15 down to 2^-14, 2^-8 to 2^-15, and at most 2^-23
//     below. The largest P' is 2^12 or more when the reference is set, so 2^-27 of the part's
//     largest product keeps its bits. (Two e4m3 terms reach over 22 bits in all: a position of
//     weight and no value, as the first one of a context often is, cost the thousands behind
//     it their weights.) O = (O_hi + O_mid / 16 + O_lo / 256) 2^(u - m) / l.
//
// Work. CTAs work in groups of 4, 2 or 1 (the largest that divides the kv heads): the members
// of a group walk the same tiles of 256 positions for neighbouring kv heads, so rows of
// several heads (128 bytes each) are fetched together (one head per group: 82 us against
// 59.5 on batch 64). All tiles, ordered by (sequence, head group, position), are cut into
// runs of equal cost, one per group: a tile costs 8, a context's last tile as many eighths as
// it has positions (4 at least), every item 5 more (fitted to the CTAs' times; without the 5,
// 256 ragged contexts took 105 us instead of 100). So a CTA takes at most two partial items,
// its first and its last, and every CTA knows how many parts an item is in; the CTA that
// completes the last part merges them, sixteen parts at a time. (A share of the tiles left in
// short chunks for the CTAs that are done first gained nothing: batch 64 59.6 - 61.5 us with
// an eighth to a quarter of them in chunks of 2 to 5, 70 us in chunks of one; an item's
// epilogue takes longer than a tile.)
//
// Bound: HBM (every K/V code is read once). Roles, as in the bf16 decode but streaming whole
// runs: warps 0-7 softmax (two groups, one position of a 256-position tile per thread),
// 8-11 epilogue, 12 K (loads and score products), 13 V (loads and value products), 14
// scheduler, 15 q terms.
// The scheduler publishes each tile's block ids and scales through a ring of tile records.
//
// Waits name an mbarrier phase by its parity, so a wait for phase n must know that phase
// n - 1 is complete. Every ring here is waited on phase after phase by the same role; the
// one exception, the softmax clearing V rows, holds because NP <= NV (the P buffer's wait
// covers the V slot's previous tile).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include <cfloat>

#include "decode_common.cuh"
#include "pa_internal.h"
#include "pa_ptx.cuh"

namespace pa {
namespace {

constexpr int TT = 256;        // positions per tile
constexpr int TM = 128;        // positions per product
constexpr int HD = 128;        // head dim
constexpr int NV = 3;          // V ring
constexpr int ND = 8;          // tile records ahead
constexpr int QN = 2;          // q slots (one per item in flight)
constexpr int NO = 2;          // O^T accumulators
constexpr int kMaxBlk = 16;    // blocks of one tile (block size 16)
constexpr int kTileBytes = TT * HD;
constexpr int kHalf = TM * HD;
constexpr int kThreads = 512;
constexpr int kSoftThreads = 256;
constexpr int kFan = 16;       // parts merged at a time
constexpr int kTileCost = 8;   // of a full tile, in units of 32 positions
constexpr int kTailCost = 4;   // least of a context's last tile
// Longest context, in tiles, that is left whole when every item can have a group of its own: the
// merge of a split item costs about a tile's time. Whole against split, us: 4 sequences of 512
// positions, 2 q heads a kv head 8.0 / 9.0, 16 of 512 8.7 / 10.4; at 768 positions the two are
// equal (10.0 / 10.1), at 1024 four sequences want the split (11.1 / 10.4, 8 q heads 13.0 / 11.3).
constexpr int kWholeTiles = 2;
constexpr int kItemCost = 5;   // an item's own (its q terms, first reference and epilogue)
constexpr float kTarget = 12.f;  // a new reference puts the largest P' at 2^kTarget ...
constexpr float kBound = 15.f;   // ... and it moves when one would pass 2^kBound (the scaled
                                 // rests of P' are then at most 2^15, inside e5m2's 57344)
constexpr float kTermScale = 16.f;  // of each term over the one before
constexpr float kQLoScale = 4194304.f;  // 2^22: of q's third term
constexpr float kSpread = 80.f;      // octaves of V scales that count in choosing u
constexpr float kNoScale = -1000.f;  // the largest log2 of a V scale while all have been 0
constexpr float kLog2eF = 1.4426950408889634f;

constexpr int round_up(int x, int a) { return (x + a - 1) / a * a; }

struct TileRec {
  int ids[kMaxBlk];
  float ks[kMaxBlk];
  float lvs[kMaxBlk];  // log2 of the V scales
  float lmax;          // the largest one of the item so far
  int n;               // positions of the tile inside the context
  int first;           // first tile of its item
  int last;            // last tile of its item
  int stop;            // no more tiles
  int row_in_blk;      // first row within ids[0] (blocks larger than a tile)
  int item_s, item_g;  // item: sequence, kv head
  int part, nparts;    // this item's part of the (sequence, kv head)
  int group0;          // group holding part 0
  int pad[5];
};
static_assert(sizeof(TileRec) == 256, "tile record");

// what the epilogue needs of an item
struct ItemRec {
  int s, g, part, nparts, group0, stop, pad[2];
};
static_assert(sizeof(ItemRec) == 32, "item record");

template <int G>
struct Cfg {
  static constexpr int NSR = round_up(3 * G, 16);   // rows of q terms (the MMA's N)
  static constexpr int NPR = round_up(3 * G, 16);   // rows of P terms
  static constexpr int NP = 3;              // P buffers
  // K ring (tiles of 32 KB): from 8 heads on shared memory holds three P buffers or three K tiles
  // (8 heads: 4 sequences of 30000 50.0 us with two K tiles, 50.9 with two P buffers).
  static constexpr int NK = G >= 8 ? 2 : 3;
  static constexpr int NS = 4;                      // S buffers in tensor memory
  static constexpr int kQBytes = NSR * 128;
  static constexpr int kPChunk = NPR * 128;         // P terms of 128 positions
  static constexpr int kPBytes = 2 * kPChunk;
  static constexpr int kOffK = 0;
  static constexpr int kOffV = NK * kTileBytes;
  static constexpr int kOffQ = kOffV + NV * kTileBytes;
  static constexpr int kOffP = kOffQ + QN * kQBytes;
  static constexpr int kOffRec = kOffP + NP * kPBytes;
  static constexpr int kOffRed = kOffRec + ND * static_cast<int>(sizeof(TileRec));
  // [2][G][8] maxima, [8][G] sums
  static constexpr int kOffQs = round_up(kOffRed + 3 * 8 * G * 4, 16);
  static constexpr int kEpiBytes = 32 + 64 * 4;  // item record, m, l and two factors per head
  static constexpr int kOffEpi = round_up(kOffQs + QN * G * 4, 16);
  // heads shared by several epilogue warps meet here when parts are merged
  static constexpr int kOffMerge = round_up(kOffEpi + NO * kEpiBytes, 16);
  static constexpr int kOffBar = kOffMerge + (G < 4 ? 4 * HD * 4 : 0);
  static constexpr int kNumBars = 3 * ND + 2 * NK + 2 * NV + 2 * NS + 2 * NP + 2 * QN + 4 * NO + 2;
  static constexpr int kOffMisc = round_up(kOffBar + 8 * kNumBars, 16);
  static constexpr int kSmemBytes = kOffMisc + 64 + 1024;
  static constexpr uint32_t kSCols = 2 * NSR;  // two products of 128 positions
  static constexpr uint32_t kTmemO = NS * kSCols;
  static constexpr uint32_t kTmemUsed = kTmemO + NO * NPR;
  static constexpr uint32_t kTmemCols = kTmemUsed <= 256 ? 256 : 512;
  static_assert(kTmemUsed <= 512, "tensor memory");
  static_assert(kSmemBytes <= 227 * 1024, "shared memory per CTA");
  static_assert(kOffQ % 1024 == 0 && kOffP % 1024 == 0 && kQBytes % 1024 == 0 && kPChunk % 1024 == 0,
                "swizzled operands");
  static_assert(kOffRec % 16 == 0 && kOffBar % 8 == 0 && kOffEpi % 16 == 0 && kOffMerge % 16 == 0,
                "alignment");
  static_assert(NP <= NV, "the softmax's wait for a V tile relies on it (see the top)");
};

struct BsParams {
  __nv_bfloat16* out;
  const __nv_bfloat16* q;
  const float* k_scales;  // [num_blocks, Hkv]
  const float* v_scales;
  const int32_t* block_tables;
  const int32_t* context_lens;
  unsigned long long* counters;  // [2 * slots] arrivals
  float* ws_o;                   // [slots][G][128] partials, slots = 2 * grid
  float* ws_ml;                  // [slots][G][2]
  unsigned* err;
  unsigned long long tag;
  unsigned long long wait_ns;
  int num_seqs;
  int num_kv_heads;
  int members;  // CTAs of a group
  int groups;
  int max_blocks;
  int num_blocks;
  int bs_log2;
  int max_context_len;
  float scale_log2;
};

__device__ __forceinline__ unsigned long long load_acquire(const unsigned long long* at) {
  unsigned long long v;
  asm volatile("ld.acquire.gpu.global.u64 %0, [%1];" : "=l"(v) : "l"(at) : "memory");
  return v;
}

__device__ __forceinline__ void fence_acq_rel_gpu() {
  asm volatile("fence.acq_rel.gpu;" ::: "memory");
}

__device__ __forceinline__ float warp_max(float v) {
  float r;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
  return r;
}

// The first 3 G fp32 columns at taddr, rounded up to a load's size.
template <int N>
__device__ __forceinline__ void tmem_ld_n(uint32_t taddr, float (&v)[N]) {
  static_assert(N == 4 || N == 8 || N == 16 || N == 32 || N == 48, "columns");
  if constexpr (N <= 16) {
    tmem_ld_cols<N>(taddr, v);
  } else {
    float t[32];
    tmem_ld32(taddr, t);
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = t[i];
    if constexpr (N == 48) {
      float u[16];
      tmem_ld16(taddr + 32, u);
#pragma unroll
      for (int i = 0; i < 16; ++i) v[32 + i] = u[i];
    }
  }
}
constexpr int load_cols(int n) { return n <= 4 ? 4 : n <= 8 ? 8 : n <= 16 ? 16 : n <= 32 ? 32 : 48; }

// One merge step over cnt <= kFan parts by the four epilogue warps. A part's record is its own
// attention output (divided by its sum) with its maximum and sum; part i's is at slot
// first + i * step, but part 0's at `slot0`. A warp takes whole heads (G >= 4) or a head's
// parts in turn with 4 / G - 1 other warps. Lane i reads part i's maximum and sum; the lanes
// hold 4 output dims each, so a part's row is one 16-byte load per lane, and all of a head's
// loads are in flight together. Reads bypass L1 (the parts were written by other SMs).
// The sums' order and roundings do not depend on who arrives last; products are rounded before
// they are added, so that for two parts either may come first (the epilogue's short way).
// out non-NULL: the rows' outputs; NULL: the result replaces part 0's record (read and written
// by the same warps).
template <int G>
__device__ __forceinline__ void merge_parts(float* ws_o, float* ws_ml, int cnt, int slot0, int first,
                                         int step, int warp4, int lane, float* buf,
                                         __nv_bfloat16* out) {
  constexpr int S = G >= 4 ? 1 : 4 / G;  // warps that share a head
  constexpr int N = kFan / S;            // parts of one warp
  const int sub = G >= 4 ? 0 : warp4 / G;
  auto slot_of = [&](int i) -> int64_t { return i == 0 ? slot0 : first + i * step; };
#pragma unroll 1
  for (int h = G >= 4 ? warp4 : warp4 % G; h < G; h += 4) {
    const float2 ml = lane < cnt ? __ldcg(reinterpret_cast<const float2*>(ws_ml) + slot_of(lane) * G + h)
                                 : make_float2(-INFINITY, 0.f);
    float4 o[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
      o[i] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (i * S + sub < cnt)
        o[i] = __ldcg(reinterpret_cast<const float4*>(ws_o + (slot_of(i * S + sub) * G + h) * HD) + lane);
    }
    const float M = warp_max(ml.x);
    const float f = M > -INFINITY ? __fmul_rn(ml.y, ex2_approx(ml.x - M)) : 0.f;
    float L = f;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) L = __fadd_rn(L, __shfl_xor_sync(0xffffffffu, L, off));
    float4 A = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float fi = __shfl_sync(0xffffffffu, f, i * S + sub);
      A.x = __fadd_rn(A.x, __fmul_rn(fi, o[i].x));
      A.y = __fadd_rn(A.y, __fmul_rn(fi, o[i].y));
      A.z = __fadd_rn(A.z, __fmul_rn(fi, o[i].z));
      A.w = __fadd_rn(A.w, __fmul_rn(fi, o[i].w));
    }
    if constexpr (S > 1) {
      // the warps of a head meet in shared memory; the first one finishes
      float* mine = buf + warp4 * HD;
      reinterpret_cast<float4*>(mine)[lane] = A;
      named_bar_sync(2, 128);
      if (sub == 0) {
#pragma unroll
        for (int w = 1; w < S; ++w) {
          const float4 B = reinterpret_cast<const float4*>(buf + (warp4 + w * G) * HD)[lane];
          A = make_float4(A.x + B.x, A.y + B.y, A.z + B.z, A.w + B.w);
        }
      }
      named_bar_sync(2, 128);  // before the buffer's next use
    }
    if (sub == 0) {
      const float r = __fdividef(1.f, L);
      A = make_float4(A.x * r, A.y * r, A.z * r, A.w * r);
      if (out) {
        *reinterpret_cast<uint2*>(out + h * HD + 4 * lane) =
            make_uint2(pack_bf16x2(A.x, A.y), pack_bf16x2(A.z, A.w));
      } else {
        const int64_t to = static_cast<int64_t>(slot0) * G + h;
        reinterpret_cast<float4*>(ws_o + to * HD)[lane] = A;
        if (lane == 0) *reinterpret_cast<float2*>(ws_ml + to * 2) = make_float2(M, L);
      }
    }
  }
}

template <int G>
__global__ void __launch_bounds__(kThreads, 1)
    decode_blockscale_kernel(const __grid_constant__ CUtensorMap tmK,
                             const __grid_constant__ CUtensorMap tmV,
                             const __grid_constant__ CUtensorMap tmKt,
                             const __grid_constant__ CUtensorMap tmVt, const BsParams p) {
  using C = Cfg<G>;
  constexpr int NS = C::NS, NP = C::NP, NK = C::NK, NSR = C::NSR, NPR = C::NPR;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const int tid = threadIdx.x;
  const int warp = tid >> 5;
  const int lane = tid & 31;
  const int Hq = p.num_kv_heads * G;
  const int bs = 1 << p.bs_log2;
  const unsigned long long wl = p.wait_ns;

  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::kOffBar);
  uint64_t* rec_full = bars;            // [ND] a tile's place -> K, V and q warps, softmax
  uint64_t* scl_full = rec_full + ND;   // [ND] its scales -> softmax
  uint64_t* rec_empty = scl_full + ND;  // [ND] K, V and q warps and softmax are done with it
  uint64_t* k_full = rec_empty + ND;    // [NK] K landed
  uint64_t* k_empty = k_full + NK;      // [NK] score product done
  uint64_t* v_full = k_empty + NK;      // [NV] V landed (also the softmax's on a last tile)
  uint64_t* v_empty = v_full + NV;      // [NV] value product done
  uint64_t* s_full = v_empty + NV;      // [NS] score product done -> softmax
  uint64_t* s_free = s_full + NS;       // [NS] softmax has read S
  uint64_t* p_full = s_free + NS;       // [NP] P written -> V warp
  uint64_t* pv_done = p_full + NP;      // [NP] value product done -> softmax
  uint64_t* q_ready = pv_done + NP;     // [QN] q terms and scales written
  uint64_t* q_empty = q_ready + QN;     // [QN] score products of the item done, scales read
  uint64_t* o_full = q_empty + QN;      // [NO] item's value products done -> epilogue
  uint64_t* o_free = o_full + NO;       // [NO] epilogue has read O
  uint64_t* epi_full = o_free + NO;     // [NO] softmax hand-off
  uint64_t* epi_empty = epi_full + NO;  // [NO] epilogue has read it
  uint64_t* mma_drain = epi_empty + NO;  // [2] every product of the K / V warp has finished
  TileRec* recs = reinterpret_cast<TileRec*>(smem + C::kOffRec);
  float* red = reinterpret_cast<float*>(smem + C::kOffRed);
  float* qscale = reinterpret_cast<float*>(smem + C::kOffQs);  // [QN][G]
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::kOffMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::kOffMisc + 8);
  volatile int* last_flag = reinterpret_cast<volatile int*>(smem + C::kOffMisc + 16);

  const int member = blockIdx.x % p.members;
  const int group = blockIdx.x / p.members;
  const int hgroups = p.num_kv_heads / p.members;

  // Scheduler warp state. The costs of 32 sequences at a time (one head group's) sit in the
  // lanes (sequence seq0 + lane) with their running sums; runs only move forward, so the
  // window does too.
  int seq0 = 0, wctx = 0;
  unsigned wcost = 0, winc = 0, wtotal = 0, wbase = 0;  // wbase: cost before the window
  auto context = [&](int s) -> int {
    if (s >= p.num_seqs) return 0;
    const int ctx = __ldg(p.context_lens + s);
    if (ctx > p.max_context_len) {
      flag_error(p.err, PA_DEV_ERR_BAD_INDEX);
      return p.max_context_len;
    }
    return ctx > 0 ? ctx : 0;
  };
  bool whole = false;  // no item is split
  auto cost_of = [&](int ctx) -> unsigned {
    if (ctx == 0) return 0;
    if (whole) return kTileCost;
    const int tiles = (ctx + TT - 1) / TT;
    const int tail = (ctx - (tiles - 1) * TT + 31) / 32;
    return static_cast<unsigned>((tiles - 1) * kTileCost + (tail > kTailCost ? tail : kTailCost) + kItemCost);
  };
  auto window = [&]() {
    wctx = context(seq0 + lane);
    wcost = winc = cost_of(wctx);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const unsigned up = __shfl_up_sync(0xffffffffu, winc, o);
      if (lane >= o) winc += up;
    }
    wtotal = __shfl_sync(0xffffffffu, winc, 31) * hgroups;
  };
  // an item: sequence, head group, context, its cost and the cost before it
  struct Item {
    int s, hg, ctx;
    unsigned cost, cum;
  };
  auto pick = [&](unsigned c) -> Item {  // the item that holds cost c
    while (wbase + wtotal <= c) {
      wbase += wtotal;
      seq0 += 32;
      window();
    }
    const int at = __ffs(__ballot_sync(0xffffffffu, wbase + winc * hgroups > c)) - 1;
    Item it;
    it.cost = __shfl_sync(0xffffffffu, wcost, at);
    it.ctx = __shfl_sync(0xffffffffu, wctx, at);
    const unsigned before = wbase + (__shfl_sync(0xffffffffu, winc, at) - it.cost) * hgroups;
    it.s = seq0 + at;
    it.hg = static_cast<int>((c - before) / it.cost);
    it.cum = before + it.hg * it.cost;
    return it;
  };
  // group i takes the tiles that start in [run_start(i), run_start(i + 1))
  unsigned cost = 0, run_q = 0, run_r = 0;
  auto run_start = [&](unsigned i) { return i * run_q + (i < run_r ? i : run_r); };
  auto group_of = [&](unsigned c) -> int {
    const unsigned wide = run_r * (run_q + 1);
    return c < wide ? c / (run_q + 1) : run_r + (c - wide) / run_q;
  };
  // block ids of an item's 32 blocks from b0 on, one per lane
  auto load_ids = [&](const Item& it, int b0) -> int {
    const int b = b0 + lane;
    return (b << p.bs_log2) < it.ctx && b < p.max_blocks
               ? __ldg(p.block_tables + static_cast<int64_t>(it.s) * p.max_blocks + b)
               : -1;
  };
  // The scheduler counts the costs and reads its first block ids before the set-up barrier,
  // so that these dependent reads overlap the set-up.
  unsigned run_end = 0;
  Item next{};         // the scheduler's next item, with its first tile, first block and ids
  int next_ta = 0, next_bb = 0, next_ids = -1;
  if (warp == 14) {
    const int second = context(32 + lane);  // read beside the window's
    window();
    cost = wtotal;
    unsigned items = __popc(__ballot_sync(0xffffffffu, wctx > 0));
    int longest = wctx;
    if (p.num_seqs > 32) {
      unsigned sum = cost_of(second), count = second > 0;
      longest = max(longest, second);
#pragma unroll 1
      for (int s = 64 + lane; s < p.num_seqs; s += 32) {
        const int ctx = context(s);
        sum += cost_of(ctx);
        count += ctx > 0;
        longest = max(longest, ctx);
      }
      cost += __reduce_add_sync(0xffffffffu, sum) * hgroups;
      items += __reduce_add_sync(0xffffffffu, count);
    }
    items *= hgroups;
    longest = __reduce_max_sync(0xffffffffu, longest);
    unsigned groups;
    if (items > 0 && items <= static_cast<unsigned>(p.groups) && longest <= kWholeTiles * TT) {
      // few short contexts: a group each (every item counts as one tile in the split)
      whole = true;
      groups = items;
      cost = items * kTileCost;
      window();
    } else {
      // runs at least a tile long: no run is skipped between two tiles of an item
      const unsigned most = cost / kTileCost;
      groups = most < static_cast<unsigned>(p.groups) ? (most ? most : 1) : p.groups;
    }
    if (cost > 0 && static_cast<unsigned>(group) < groups) {
      run_q = cost / groups;
      run_r = cost - run_q * groups;
      const unsigned start = run_start(group);
      run_end = run_start(group + 1);
      unsigned c = start;
#pragma unroll 1
      while (true) {
        next = pick(c);
        next_ta = c == start ? static_cast<int>((start - next.cum + kTileCost - 1) / kTileCost) : 0;
        if (next_ta * TT < next.ctx) break;
        c = next.cum + next.cost;  // the run starts inside the item's last tile
        if (c >= run_end) {
          run_end = 0;
          break;
        }
      }
      if (run_end) {
        next_bb = (next_ta * TT) >> p.bs_log2;
        next_ids = load_ids(next, next_bb);
      }
    }
  }

  if (tid == 12 * 32) {
    prefetch_tensormap(&tmK);
    prefetch_tensormap(&tmKt);
  }
  if (tid == 13 * 32) {
    prefetch_tensormap(&tmV);
    prefetch_tensormap(&tmVt);
  }
  // q slots and P buffers start at zero: rows that no head uses stay zero
#pragma unroll 1
  for (int i = tid; i < (QN * C::kQBytes + NP * C::kPBytes) / 16; i += kThreads)
    reinterpret_cast<uint4*>(smem + C::kOffQ)[i] = make_uint4(0, 0, 0, 0);
  fence_proxy_async_smem();
  if (tid < C::kNumBars) {
    uint64_t* bar = bars + tid;
    auto in = [&](uint64_t* first, int n) { return bar >= first && bar < first + n; };
    const unsigned count = in(rec_empty, ND)                      ? 3 + kSoftThreads / 32
                           : in(s_free, NS) || in(p_full, NP)     ? kSoftThreads / 32
                           : in(q_empty, QN)                      ? 2
                           : in(o_free, NO)                       ? 4
                                                                  : 1;
    mbar_init(bar, count);
    if (tid == 0) *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 13) {
    tmem_alloc(tmem_slot, C::kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (warp == 12 || warp == 13) {
    // ======================================================== K warp (12) and V warp (13)
    // Each loads its tiles into its ring and issues the products that read them: an event loop
    // over a load cursor and a product cursor, loads first. (One warp issuing both products,
    // beside two loading ones, took 2400 of a tile's 2860 cycles and held the rings full.)
    const bool is_v = warp == 13;
    const CUtensorMap* map = is_v ? &tmV : &tmK;
    const CUtensorMap* map_tail = is_v ? &tmVt : &tmKt;
    uint8_t* ring = smem + (is_v ? C::kOffV : C::kOffK);
    uint64_t* full = is_v ? v_full : k_full;
    uint64_t* empty = is_v ? v_empty : k_empty;
    constexpr uint32_t idS = idesc_e4m3_f32(TM, NSR, 0, 0);  // K K-major, q terms K-major
    // V^T MN-major, P terms (e5m2) K-major
    constexpr uint32_t idO = idesc_e4m3_e5m2_f32(HD, NPR, 1, 0);
    const uint64_t ring_desc = smem_desc_sw128(smem_u32(ring), is_v ? kHalf : 16, 1024);
    const uint64_t b_desc = smem_desc_sw128(smem_u32(smem + (is_v ? C::kOffP : C::kOffQ)), 16, 1024);
    const int rows_log2 = bs < TT ? p.bs_log2 : 8;   // rows per box of a full tile
    const int trows_log2 = bs < 32 ? p.bs_log2 : 5;  // of a context's last tile (none past it)
    unsigned jl = 0, jm = 0;              // tiles whose load / product was issued
    int item = 0;                         // of the product cursor
    bool ended = false;                   // the stop record was seen
    // load of tile jl (false: no record yet, or no free slot)
    auto load = [&]() -> bool {
      const int rs = jl % ND, slot = is_v ? jl % NV : jl % NK, lap = is_v ? jl / NV : jl / NK;
      if (!__all_sync(0xffffffffu,
                      mbar_test_wait(&rec_full[rs], (jl / ND) & 1) &&
                          (lap == 0 || mbar_test_wait(&empty[slot], (lap - 1) & 1))))
        return false;
      const TileRec& rec = recs[rs];
      if (rec.stop) {
        ended = true;
        return false;
      }
      const bool whole = rec.n == TT;
      const int br_log2 = whole ? rows_log2 : trows_log2;
      const int nbox = (rec.n + (1 << br_log2) - 1) >> br_log2;
      // lane b: the pool row of box b (counted from the first block's start)
      const int r = (lane << br_log2) + rec.row_in_blk;
      const int row = lane < nbox ? (rec.ids[r >> p.bs_log2] << p.bs_log2) + (r & (bs - 1)) : 0;
      const int g = rec.item_g;
      const CUtensorMap* m = whole ? map : map_tail;
      uint8_t* dst = ring + slot * kTileBytes;
      mbar_arrive_expect_tx_w(&full[slot], (nbox << br_log2) * HD);
#pragma unroll 1
      for (int b = 0; b < nbox; ++b)
        tma_load_3d_w(dst + ((b << br_log2) * HD), m, &full[slot], 0, g,
                      __shfl_sync(0xffffffffu, row, b));
      ++jl;
      return true;
    };
    // S of tile jm (false: its q, K tile or S buffer is not ready)
    auto score = [&]() -> bool {
      const int slot = jm % NK, sb = jm % NS, qs = item % QN;
      const TileRec& rec = recs[jm % ND];
      if (!__all_sync(0xffffffffu,
                      mbar_test_wait(&k_full[slot], (jm / NK) & 1) &&
                          (jm < NS || mbar_test_wait(&s_free[sb], ((jm / NS) - 1) & 1)) &&
                          (!rec.first || mbar_test_wait(&q_ready[qs], (item / QN) & 1))))
        return false;
      tc_fence_after();
      const uint64_t aK = desc_advance(ring_desc, slot * kTileBytes);
      const uint64_t bQ = desc_advance(b_desc, qs * C::kQBytes);
      const uint32_t dS = tmem + sb * C::kSCols;
#pragma unroll
      for (int kk = 0; kk < HD / 32; ++kk)
        tc_mma_f8_ss(dS, desc_advance(aK, kk * 32), desc_advance(bQ, kk * 32), idS, kk > 0 ? 1u : 0u);
      if (rec.n > TM) {
#pragma unroll
        for (int kk = 0; kk < HD / 32; ++kk)
          tc_mma_f8_ss(dS + NSR, desc_advance(aK, kHalf + kk * 32), desc_advance(bQ, kk * 32), idS,
                       kk > 0 ? 1u : 0u);
      }
      tc_commit(&s_full[sb]);
      tc_commit(&k_empty[slot]);
      if (rec.last) {
        tc_commit(&q_empty[qs]);
        ++item;
      }
      return true;
    };
    // O += V^T P^T of tile jm (false: P, V or the accumulator is not ready)
    auto value = [&]() -> bool {
      const int pb = jm % NP, slot = jm % NV, ob = item % NO;
      const TileRec& rec = recs[jm % ND];
      const bool first = rec.first != 0;
      if (!__all_sync(0xffffffffu,
                      mbar_test_wait(&p_full[pb], (jm / NP) & 1) &&
                          mbar_test_wait(&v_full[slot], (jm / NV) & 1) &&
                          (!first || item < NO || mbar_test_wait(&o_free[ob], ((item / NO) - 1) & 1))))
        return false;
      tc_fence_after();
      const uint64_t aV = desc_advance(ring_desc, slot * kTileBytes);
      const uint64_t bP = desc_advance(b_desc, pb * C::kPBytes);
      const uint32_t dO = tmem + C::kTmemO + ob * NPR;
      const int steps = (rec.n + 31) >> 5;  // 32 positions each; none past the context
#pragma unroll
      for (int kk = 0; kk < TT / 32; ++kk)
        if (kk < steps)
          tc_mma_f8_ss(dO, desc_advance(aV, kk * 32 * 128),
                       desc_advance(bP, (kk >> 2) * C::kPChunk + (kk & 3) * 32), idO,
                       (first && kk == 0) ? 0u : 1u);
      tc_commit(&pv_done[pb]);
      tc_commit(&v_empty[slot]);
      if (rec.last) {
        tc_commit(&o_full[ob]);
        ++item;
      }
      return true;
    };
    unsigned long long idle_since = 0;
    unsigned idle = 0;
    while (true) {
      bool progressed = !ended && load();
      if (jm < jl && (is_v ? value() : score())) {
        if (lane == 0) mbar_arrive(&rec_empty[jm % ND]);
        ++jm;
        progressed = true;
      }
      if (ended && jm == jl) break;
      if (progressed) {
        idle = 0;
        continue;
      }
      if ((++idle & 3) != 1) continue;  // polls; the timer is read at the first and then now and then
      const unsigned long long now = globaltimer_ns();
      if (idle == 1) idle_since = now;
      const bool give_up = *abort_flag || now - idle_since > wl;
      if (__any_sync(0xffffffffu, give_up)) {
        if (!*abort_flag) {
          if (lane == 0) flag_error(p.err, PA_DEV_ERR_TIMEOUT);
          *abort_flag = 1;
        }
        break;
      }
    }
    // Before the CTA ends: every copy this warp started has landed (per slot only its last one
    // can still be in flight), every product it issued has finished.
    if (lane == 0) {
      const unsigned depth = is_v ? NV : NK;
#pragma unroll 1
      for (unsigned t = jl > depth ? jl - depth : 0; t < jl; ++t)
        mbar_wait(&full[t % depth], (t / depth) & 1, p.err);
    }
    __syncwarp();
    tc_commit(&mma_drain[is_v]);
    mbar_wait(&mma_drain[is_v], 0, p.err);
  } else if (warp == 14) {
    // ======================================================== scheduler
    unsigned j = 0;  // tile records published
    bool alive = true;
    const int per_tile = bs >= TT ? 1 : TT >> p.bs_log2;
    bool more = run_end > 0;
    while (alive && more) {
      // item: its tiles from ta on that start before run_end
      const Item it = next;
      const int ta = next_ta;
      int bb = next_bb, bid = next_ids;  // first block and ids of the batch the lanes hold
      const int g = it.hg * p.members + member;
      const int tiles = (it.ctx + TT - 1) / TT;
      const int upto = static_cast<int>((run_end - it.cum + kTileCost - 1) / kTileCost);
      const int tb = tiles < upto || whole ? tiles : upto;
      more = it.cum + it.cost < run_end;
      float lmax = kNoScale;
      float ksc = 0.f, lvs = 0.f;
      bool fresh = true;  // the batch's scales have not been read
      for (int t = ta; t < tb; ++t) {
        const int slot = j % ND;
        if (j >= ND &&
            !warp_wait_or_abort(&rec_empty[slot], ((j / ND) - 1) & 1, p.err, abort_flag, wl)) {
          alive = false;
          break;
        }
        TileRec& rec = recs[slot];
        const int b0 = (t * TT) >> p.bs_log2;
        if (b0 >= bb + 32) {
          bb = b0;
          bid = load_ids(it, b0);
          fresh = true;
        }
        if (fresh && (bid < 0 || bid >= p.num_blocks)) {
          if (((bb + lane) << p.bs_log2) < it.ctx) flag_error(p.err, PA_DEV_ERR_BAD_INDEX);
          bid = 0;  // in-bounds stand-in
        }
        const int l0 = b0 - bb;
        const bool mine = lane >= l0 && lane < l0 + per_tile;
        if (mine) rec.ids[lane - l0] = bid;
        if (lane == 0) {
          rec.n = it.ctx - t * TT < TT ? it.ctx - t * TT : TT;
          rec.first = t == ta;
          rec.last = t == tb - 1;
          rec.stop = 0;
          rec.row_in_blk = bs > TT ? (t * TT) & (bs - 1) : 0;
          rec.item_s = it.s;
          rec.item_g = g;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&rec_full[slot]);
        // the scales follow (the tile's loads do not wait for them)
        if (fresh) {
          fresh = false;
          const int64_t at = static_cast<int64_t>(bid) * p.num_kv_heads + g;
          ksc = __ldg(p.k_scales + at);
          lvs = __log2f(__ldg(p.v_scales + at));
        }
        const bool used = mine && ((b0 + lane - l0) << p.bs_log2) < it.ctx;
        lmax = fmaxf(lmax, warp_max(used ? lvs : kNoScale));
        if (mine) {
          rec.ks[lane - l0] = ksc;
          rec.lvs[lane - l0] = lvs;
        }
        if (lane == 0) {
          rec.lmax = lmax;
          if (t == tb - 1) {  // what the epilogue needs
            const int group0 = group_of(it.cum);
            rec.group0 = group0;
            rec.part = group - group0;
            rec.nparts = whole ? 1 : group_of(it.cum + (tiles - 1) * kTileCost) - group0 + 1;
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&scl_full[slot]);
        ++j;
        // the next item's ids are on their way while this one's other tiles are published
        if (t == ta && more) {
          next = pick(it.cum + it.cost);
          next_ta = next_bb = 0;
          next_ids = load_ids(next, 0);
        }
      }
    }
    if (alive) {
      const int slot = j % ND;
      if (j < ND ||
          warp_wait_or_abort(&rec_empty[slot], ((j / ND) - 1) & 1, p.err, abort_flag, wl)) {
        if (lane == 0) {
          recs[slot].stop = 1;
          recs[slot].first = recs[slot].last = recs[slot].n = 0;
          mbar_arrive(&rec_full[slot]);
        }
      }
    }
  } else if (warp == 15) {
    // ======================================================== q warp
    // The q terms of every item, from its first tile's record on: lane L holds dims 4L .. 4L + 3.
    int k = 0;
    for (unsigned j = 0;; ++j) {
      const int rs = j % ND;
      if (!warp_wait_or_abort(&rec_full[rs], (j / ND) & 1, p.err, abort_flag, wl)) break;
      const TileRec& rec = recs[rs];
      if (rec.stop) break;
      if (rec.first) {
        const uint2* src = reinterpret_cast<const uint2*>(
            p.q + (static_cast<int64_t>(rec.item_s) * Hq + rec.item_g * G) * HD);
        uint2 raw[G];
#pragma unroll
        for (int h = 0; h < G; ++h) raw[h] = __ldg(src + h * (HD / 4) + lane);
        const int qs = k % QN;
        if (k >= QN &&
            !warp_wait_or_abort(&q_empty[qs], ((k / QN) - 1) & 1, p.err, abort_flag, wl))
          break;
        uint8_t* qd = smem + C::kOffQ + qs * C::kQBytes;
#pragma unroll
        for (int h = 0; h < G; ++h) {
          const float f0 = bf16lo_to_f32(raw[h].x), f1 = bf16hi_to_f32(raw[h].x);
          const float f2 = bf16lo_to_f32(raw[h].y), f3 = bf16hi_to_f32(raw[h].y);
          const float amax = warp_max(fmaxf(fmaxf(fabsf(f0), fabsf(f1)), fmaxf(fabsf(f2), fabsf(f3))));
          // the smallest k >= -126 with amax <= 448 2^k (448 = 1.75 2^8)
          const unsigned bits = __float_as_uint(amax);
          const int up = static_cast<int>(bits >> 23) - 127 - 8 + ((bits & 0x7fffffu) > 0x600000u ? 1 : 0);
          const int e = up > -126 ? up : -126;
          const float inv = __uint_as_float(static_cast<unsigned>(127 - e) << 23);
          float y[4] = {f0 * inv, f1 * inv, f2 * inv, f3 * inv};
#pragma unroll
          for (int term = 0; term < 3; ++term) {
            const int row = 3 * h + term;
            float2 b01, b23;
            const uint32_t c01 = e4m3x2(y[0], y[1], b01);
            const uint32_t c23 = e4m3x2(y[2], y[3], b23);
            *reinterpret_cast<uint32_t*>(qd + row * 128 + ((((lane >> 2) ^ row) & 7) << 4) +
                                         (lane & 3) * 4) = c01 | (c23 << 16);
            const float by = term == 0 ? kTermScale : kQLoScale / kTermScale;
            y[0] = (y[0] - b01.x) * by;
            y[1] = (y[1] - b01.y) * by;
            y[2] = (y[2] - b23.x) * by;
            y[3] = (y[3] - b23.y) * by;
          }
          // an infinite element makes its head's scores NaN
          if (lane == 0)
            qscale[qs * G + h] = amax <= FLT_MAX ? __uint_as_float(static_cast<unsigned>(127 + e) << 23) : NAN;
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&q_ready[qs]);
        ++k;
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&rec_empty[rs]);
    }
  } else if (warp < 8) {
    // ======================================================== softmax
    // Thread r of group sg owns position 128 sg + r of each tile. Control flow is uniform
    // over the 256 threads: a failed wait only marks `failed`, and the vote that every tile
    // has settles it before anything of the tile's record decides a branch around a barrier.
    const int sg = warp >> 2;
    const int quad = warp & 3;
    const int r = quad * 32 + lane;
    const int pos = sg * TM + r;  // within the tile
    const uint32_t lane_off = static_cast<uint32_t>(quad * 32) << 16;
    const int blk = bs >= TT ? 0 : pos >> p.bs_log2;  // block of the tile
    constexpr int SC = load_cols(3 * G);
    unsigned j = 0;
    int k = 0;
    float m[G], l[G], u[G], fs[G];
    auto restart = [&]() {  // for an item's first tile: any reference is above these
#pragma unroll
      for (int h = 0; h < G; ++h) {
        m[h] = u[h] = -INFINITY;
        l[h] = 0.f;
      }
    };
    restart();
#pragma unroll
    for (int h = 0; h < G; ++h) fs[h] = 0.f;
    bool failed = false;
    while (true) {
      const int rs = j % ND, sb = j % NS;
      failed |= !wait_or_abort(&rec_full[rs], (j / ND) & 1, p.err, abort_flag, wl);
      const TileRec& rec = recs[rs];
      const bool stop = rec.stop != 0;
      float x[G];
      bool valid = false, first = false, exceeds = false;
      float lvs = 0.f, lc = 0.f, lmax = 0.f;
      // warp-uniform: the loads below are warp-wide
      const bool go = __all_sync(0xffffffffu, !failed && !stop);
      if (go) {
        first = rec.first != 0;
        valid = pos < rec.n;
        failed |= !wait_or_abort(&scl_full[rs], (j / ND) & 1, p.err, abort_flag, wl);
        if (first) {
          const int qs = k % QN;
          failed |= !wait_or_abort(&q_ready[qs], (k / QN) & 1, p.err, abort_flag, wl);
#pragma unroll
          for (int h = 0; h < G; ++h) fs[h] = p.scale_log2 * qscale[qs * G + h];
        }
        const float ksc = rec.ks[blk];
        lvs = valid ? rec.lvs[blk] : 0.f;
        lmax = rec.lmax;
        lc = fmaxf(lvs, lmax - kSpread);
        failed |= !wait_or_abort(&s_full[sb], (j / NS) & 1, p.err, abort_flag, wl);
        tc_fence_after();
        float sv[SC];
        tmem_ld_n<SC>(tmem + sb * C::kSCols + sg * NSR + lane_off, sv);
        tc_wait_ld();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&s_free[sb]);
        exceeds = first;
#pragma unroll
        for (int h = 0; h < G; ++h) {
          const float d = fmaf(sv[3 * h + 2], 1.f / kQLoScale, fmaf(sv[3 * h + 1], 1.f / kTermScale, sv[3 * h]));
          x[h] = valid ? d * (fs[h] * ksc) : -INFINITY;
          exceeds |= x[h] > u[h] + (kBound - lc);
        }
      }
      // One vote a tile: nothing to do (the reference holds for every position), or the
      // reference must move, or the loop ends.
      float alpha[G], pp[G];
      bool moved = false;
      if (bar_or(1, kSoftThreads, failed || stop || exceeds)) {
        float* rb = red + (j & 1) * 8 * G;
        if (go) {
#pragma unroll
          for (int h = 0; h < G; ++h) {
            const float v = warp_max(x[h] + lc);
            if (lane == 0) rb[h * 8 + warp] = v;
          }
        }
        if (bar_or(1, kSoftThreads, failed || stop)) {
          if (tid == 0 && stop && !failed) {  // tell the epilogue there are no more items
            const int b = k % NO;
            if (k < NO || wait_or_abort(&epi_empty[b], ((k / NO) - 1) & 1, p.err, abort_flag, wl)) {
              reinterpret_cast<ItemRec*>(smem + C::kOffEpi + b * C::kEpiBytes)->stop = 1;
              mbar_arrive(&epi_full[b]);
            }
          }
          break;
        }
#pragma unroll
        for (int h = 0; h < G; ++h) {
          const float4 w0 = *reinterpret_cast<const float4*>(rb + h * 8);
          const float4 w1 = *reinterpret_cast<const float4*>(rb + h * 8 + 4);
          const float my = fmaxf(fmax3(fmaxf(w0.x, w0.y), w0.z, w0.w),
                                 fmax3(fmaxf(w1.x, w1.y), w1.z, w1.w));
          // without branches (with them: 47.5 us, not 42, at 16 heads a kv head)
          const bool passed = my > u[h] + kBound;
          const float un = passed ? my - kTarget : u[h], mn = fmaxf(m[h], my - lmax);
          alpha[h] = ex2_approx(u[h] - un);
          l[h] *= ex2_approx(m[h] - mn);
          u[h] = un;
          m[h] = mn;
          moved |= passed;
        }
        moved = moved && !first;  // a first tile's product overwrites O
      }
      // from here the record is known to be sound for every thread
      if (first && tid == 0) mbar_arrive(&q_empty[k % QN]);  // every thread has its q scales
      const int n = rec.n;
      const bool last = rec.last != 0;
#pragma unroll
      for (int h = 0; h < G; ++h) {
        l[h] += ex2_approx(x[h] - m[h]);  // x is -inf past the context
        pp[h] = ex2_approx((x[h] + lvs) - u[h]);
      }
      // this P buffer was last read by the value product of tile j - NP
      const int pb = j % NP;
      if (j >= NP)
        failed |= !wait_or_abort(&pv_done[pb], ((j / NP) - 1) & 1, p.err, abort_flag, wl);
      {
        uint8_t* pt = smem + C::kOffP + pb * C::kPBytes + sg * C::kPChunk + (r & 15);
        const int c = r >> 4;
        auto put = [&](int row, uint32_t code) {
          pt[row * 128 + (((c ^ row) & 7) << 4)] = static_cast<uint8_t>(code);
        };
#pragma unroll
        for (int h = 0; h < G; h += 2) {
          float2 rest = make_float2(pp[h], h + 1 < G ? pp[h + 1] : 0.f);
#pragma unroll
          for (int term = 0; term < 3; ++term) {
            float2 held;
            const uint32_t code = e5m2x2(rest.x, rest.y, held);
            put(3 * h + term, code);
            if (h + 1 < G) put(3 * h + 3 + term, code >> 8);
            rest = make_float2((rest.x - held.x) * kTermScale, (rest.y - held.y) * kTermScale);
          }
        }
      }
      if (n < TT) {
        // rows past the context may hold anything, and 0 * NaN is NaN: clear those that the
        // value product's steps of 32 positions read
        if (!valid && pos < ((n + 31) & ~31)) {
          const int vs = j % NV;
          failed |= !wait_or_abort(&v_full[vs], (j / NV) & 1, p.err, abort_flag, wl);
          uint8_t* v = smem + C::kOffV + vs * kTileBytes + pos * HD;
#pragma unroll
          for (int c = 0; c < 8; ++c) *reinterpret_cast<uint4*>(v + c * 16) = make_uint4(0, 0, 0, 0);
        }
      }
      if (sg == 0 && moved) {
        // uniform over the group; O holds the products up to tile j - 1
        const unsigned t = j - 1;
        failed |= !wait_or_abort(&pv_done[t % NP], (t / NP) & 1, p.err, abort_flag, wl);
        tc_fence_after();
#pragma unroll
        for (int c = 0; c < NPR; c += 16) {  // three columns per head
          float o[16];
          const uint32_t at = tmem + C::kTmemO + (k % NO) * NPR + c + lane_off;
          tmem_ld16(at, o);
          tc_wait_ld();
#pragma unroll
          for (int i = 0; i < 16; ++i)
            if (c + i < 3 * G) o[i] *= alpha[(c + i) / 3];
          tmem_st16(at, o);
        }
        tc_wait_st();
      }
      fence_proxy_async_smem();
      tc_fence_before();
      const ItemRec it{rec.item_s, rec.item_g, rec.part, rec.nparts, rec.group0, 0, {0, 0}};
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&p_full[pb]);
        mbar_arrive(&rec_empty[rs]);
      }
      ++j;
      if (last) {
        // hand the item to the epilogue: l over the 256 positions, m, the outputs' factors
        float* lb = red + 2 * 8 * G;
#pragma unroll
        for (int h = 0; h < G; ++h) {
          float v = l[h];
#pragma unroll
          for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
          if (lane == 0) lb[warp * G + h] = v;
        }
        named_bar_sync(1, kSoftThreads);
        if (warp == 0) {  // a lane per head
          const int b = k % NO;
          if (k >= NO)
            failed |= !wait_or_abort(&epi_empty[b], ((k / NO) - 1) & 1, p.err, abort_flag, wl);
          if (__all_sync(0xffffffffu, !failed)) {
            uint8_t* es = smem + C::kOffEpi + b * C::kEpiBytes;
            if (lane == 0) *reinterpret_cast<ItemRec*>(es) = it;
            float mine = 0.f, shift = 0.f;
#pragma unroll
            for (int h = 0; h < G; ++h) {
              mine = lane == h ? m[h] : mine;
              shift = lane == h ? u[h] - m[h] : shift;
            }
            if (lane < G) {
              float L = 0.f;
#pragma unroll
              for (int w = 0; w < 8; ++w) L += lb[w * G + lane];
              // O's factor 2^(u - m) / l in two, which stay in fp32's range
              const float half = ex2_approx(0.5f * shift);
              float* em = reinterpret_cast<float*>(es + 32) + lane;
              em[0] = mine;
              em[16] = L;
              em[32] = __fdividef(half, L);
              em[48] = half;
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&epi_full[b]);
          }
        }
        restart();
        ++k;
      }
    }
  } else {
    // ======================================================== epilogue (warps 8-11)
    const int dl = ((warp & 3) << 5) | lane;  // output dim = tensor-memory lane
    const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const bool leader = tid == 8 * 32;
    // this CTA's four counters get this call's tag ahead of the arrivals
    if (dl < 4) {
      unsigned long long* ctr = p.counters + 4 * blockIdx.x + dl;
      tagged_install(ctr, *reinterpret_cast<volatile unsigned long long*>(ctr), p.tag, p.err);
    }
    // empty contexts: a zero row for every head
#pragma unroll 1
    for (int s = blockIdx.x; s < p.num_seqs; s += gridDim.x)
      if (p.max_context_len == 0 || __ldg(p.context_lens + s) <= 0)
#pragma unroll 1
        for (int i = dl; i < Hq * HD / 2; i += 128)
          reinterpret_cast<uint32_t*>(p.out + static_cast<int64_t>(s) * Hq * HD)[i] = 0u;
    int k = 0;
    while (true) {
      const int b = k % NO;
      bool failed = !wait_or_abort(&epi_full[b], (k / NO) & 1, p.err, abort_flag, wl);
      const uint8_t* es = smem + C::kOffEpi + b * C::kEpiBytes;
      const ItemRec it = *reinterpret_cast<const ItemRec*>(es);
      float m[G], L[G], f0[G], f1[G];
#pragma unroll
      for (int h = 0; h < G; ++h) {
        const float* em = reinterpret_cast<const float*>(es + 32) + h;
        m[h] = em[0];
        L[h] = em[16];
        f0[h] = em[32];
        f1[h] = em[48];
      }
      // part i of an item lives in CTA (group0 + i, member): a CTA's first item in slot 0 when
      // it began in an earlier group, its last item in slot 1 when it goes on in a later one
      auto slot_of = [&](int i) -> int64_t {
        return 2 * (static_cast<int64_t>(it.group0 + i) * p.members + member) + (i == 0 ? 1 : 0);
      };
      // Is the other part of two there already? Then it is read while this one's last products
      // run, and this one goes straight into the output, with the bits that merge_parts gives
      // (most split items are in two parts; the code for more of them took 0.8 us longer).
      if (leader && !failed && !it.stop && it.nparts == 2)
        *last_flag = load_acquire(p.counters + 2 * slot_of(0)) == ((p.tag << kCountBits) | 1u);
      if (bar_or(2, 128, failed)) break;  // every thread has read the hand-off
      if (leader) mbar_arrive(&epi_empty[b]);
      if (it.stop) break;
      const bool finish = it.nparts == 2 && *last_flag != 0;
      // this part's weight and the parts' sum, the other one's row times its weight
      float wo[G], sum[G], po[G];
      if (finish) {
        const int64_t at = slot_of(it.part ^ 1) * G;
        float2 ml[G];
#pragma unroll
        for (int h = 0; h < G; ++h) {
          ml[h] = __ldcg(reinterpret_cast<const float2*>(p.ws_ml) + at + h);
          po[h] = __ldcg(p.ws_o + (at + h) * HD + dl);
        }
#pragma unroll
        for (int h = 0; h < G; ++h) {
          const float mx = fmaxf(m[h], ml[h].x);
          const float f = __fmul_rn(ml[h].y, ex2_approx(ml[h].x - mx));
          wo[h] = __fmul_rn(L[h], ex2_approx(m[h] - mx));
          sum[h] = __fadd_rn(wo[h], f);
          po[h] = fmaf(po[h], f, 0.f);  // as in merge_parts, never -0
        }
      }
      failed |= !wait_or_abort(&o_full[b], (k / NO) & 1, p.err, abort_flag, wl);
      tc_fence_after();
      constexpr int OC = load_cols(3 * G);
      float oc[OC], o[G];
      tmem_ld_n<OC>(tmem + C::kTmemO + b * NPR + lane_off, oc);
      tc_wait_ld();
#pragma unroll
      for (int h = 0; h < G; ++h) {
        const float sum = fmaf(fmaf(oc[3 * h + 2], 1.f / kTermScale, oc[3 * h + 1]), 1.f / kTermScale, oc[3 * h]);
        o[h] = sum * f0[h] * f1[h];
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&o_free[b]);
      const int64_t row0 = static_cast<int64_t>(it.s) * Hq + it.g * G;
      if (it.nparts == 1 || finish) {
        if (finish) {
#pragma unroll
          for (int h = 0; h < G; ++h)
            o[h] = __fadd_rn(fmaf(wo[h], o[h], 0.f), po[h]) * __fdividef(1.f, sum[h]);
          if (leader) *reinterpret_cast<volatile unsigned long long*>(p.counters + 2 * slot_of(0)) = 0ull;
        }
        if (!failed) {
#pragma unroll
          for (int h = 0; h < G; ++h)
            p.out[(row0 + h) * HD + dl] = __float2bfloat16_rn(o[h]);
        }
      } else {
        const int64_t mine = slot_of(it.part);
#pragma unroll
        for (int h = 0; h < G; ++h) {
          p.ws_o[(mine * G + h) * HD + dl] = o[h];
          if (dl == 0) *reinterpret_cast<float2*>(p.ws_ml + (mine * G + h) * 2) = make_float2(m[h], L[h]);
        }
        // arrive: written by all 128 threads, one release by the leader
        auto arrive = [&](unsigned long long* ctr, int total) -> bool {
          named_bar_sync(2, 128);
          if (leader) {
            fence_acq_rel_gpu();
            bool okc = true;
            const unsigned before = tagged_arrive(ctr, p.tag, p.err, &okc);
            const bool is_last = okc && before == static_cast<unsigned>(total - 1);
            if (is_last) *reinterpret_cast<volatile unsigned long long*>(ctr) = 0ull;
            *last_flag = is_last;
            fence_acq_rel_gpu();
          }
          named_bar_sync(2, 128);
          return *last_flag != 0;
        };
        const int sub = it.part / kFan, nsub = (it.nparts + kFan - 1) / kFan;
        const int in_sub = it.nparts - sub * kFan < kFan ? it.nparts - sub * kFan : kFan;
        // arrivals of sixteen parts count at the first one's slot; when there are more parts,
        // each sixteen's result replaces its first part, and those arrive at part 0's second
        // counter
        const int base = static_cast<int>(slot_of(0)) - 1, per = 2 * p.members;  // of part 0 in slot 0
        int from = sub * kFan, step = 1, cnt = in_sub;
        bool top = nsub == 1;
        unsigned long long* ctr = p.counters + 2 * slot_of(from);
#pragma unroll 1
        while (arrive(ctr, cnt)) {
          merge_parts<G>(p.ws_o, p.ws_ml, cnt, static_cast<int>(slot_of(from)), base + from * per,
                         step * per, warp - 8, lane, reinterpret_cast<float*>(smem + C::kOffMerge),
                         top ? p.out + row0 * HD : nullptr);
          if (top) break;
          top = true;
          from = 0;
          step = kFan;
          cnt = nsub;
          ctr = p.counters + 2 * slot_of(0) + 1;
        }
      }
      if (bar_or(2, 128, failed)) break;  // also orders last_flag's reuse
      ++k;
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 13) {
    tc_fence_after();
    tmem_dealloc(tmem, C::kTmemCols);
  }
}

// CTAs of a group: neighbouring kv heads walked side by side.
int group_members(int num_kv_heads) {
  return num_kv_heads % 4 == 0 ? 4 : num_kv_heads % 2 == 0 ? 2 : 1;
}

template <int G>
cudaError_t launch_g(const DecodeLaunch& a, BsParams p, cudaStream_t stream) {
  const int bs = a.cache.block_size;
  const uint64_t slots = static_cast<uint64_t>(a.cache.num_blocks) * bs;
  const uint64_t dims[3] = {HD, static_cast<uint64_t>(a.cache.num_kv_heads), slots};
  const uint32_t box[3] = {HD, 1, static_cast<uint32_t>(bs < TT ? bs : TT)};
  const uint32_t tail[3] = {HD, 1, static_cast<uint32_t>(bs < 32 ? bs : 32)};
  CUtensorMap tmK, tmV, tmKt, tmVt;
  const CUtensorMapDataType u8 = CU_TENSOR_MAP_DATA_TYPE_UINT8;
  if (!encode_tensor_map(&tmK, a.k_cache, u8, 1, 3, dims, box, true) ||
      !encode_tensor_map(&tmV, a.v_cache, u8, 1, 3, dims, box, true) ||
      !encode_tensor_map(&tmKt, a.k_cache, u8, 1, 3, dims, tail, true) ||
      !encode_tensor_map(&tmVt, a.v_cache, u8, 1, 3, dims, tail, true))
    return cudaErrorInvalidValue;
  constexpr int smem_bytes = Cfg<G>::kSmemBytes;
  const cudaError_t e = ensure_max_dynamic_smem(
      reinterpret_cast<const void*>(decode_blockscale_kernel<G>), smem_bytes);
  if (e != cudaSuccess) return e;
  decode_blockscale_kernel<G>
      <<<p.groups * p.members, kThreads, smem_bytes, stream>>>(tmK, tmV, tmKt, tmVt, p);
  return cudaGetLastError();
}

}  // namespace

// Slots of partials: two per CTA (its first and its last item); two counters per slot.
namespace {
size_t counter_bytes(size_t slots) { return (2 * slots * 8 + 255) / 256 * 256; }
}  // namespace

size_t decode_blockscale_workspace(int32_t num_q_heads, int32_t num_kv_heads) {
  const int members = group_members(num_kv_heads);
  const size_t slots = 2 * static_cast<size_t>(sm_count() / members * members);
  return counter_bytes(slots) +
         slots * static_cast<size_t>(num_q_heads / num_kv_heads) * (HD + 2) * sizeof(float);
}

cudaError_t launch_decode_blockscale(const DecodeLaunch& a, void* workspace, cudaStream_t stream) {
  BsParams p;
  p.out = static_cast<__nv_bfloat16*>(a.out);
  p.q = static_cast<const __nv_bfloat16*>(a.q);
  p.k_scales = a.k_scales;
  p.v_scales = a.v_scales;
  p.block_tables = a.block_tables;
  p.context_lens = a.context_lens;
  p.err = device_error_word();
  p.tag = next_call_tag();
  p.wait_ns = wait_limit_ns();
  p.num_seqs = a.num_seqs;
  p.num_kv_heads = a.cache.num_kv_heads;
  p.members = group_members(a.cache.num_kv_heads);
  // no more groups than there can be tiles of a head group
  const int64_t tiles = static_cast<int64_t>(a.num_seqs) *
                        (a.max_context_len > 0 ? (a.max_context_len + TT - 1) / TT : 1) *
                        (a.cache.num_kv_heads / p.members);
  p.groups = sm_count() / p.members;
  if (p.groups < 1) return cudaErrorInvalidValue;
  if (tiles < p.groups) p.groups = static_cast<int>(tiles);
  p.max_blocks = a.max_blocks_per_seq;
  p.num_blocks = a.cache.num_blocks;
  p.bs_log2 = 31 - __builtin_clz(static_cast<unsigned>(a.cache.block_size));
  p.max_context_len = a.max_context_len;
  p.scale_log2 = a.scale * kLog2eF;
  const int G = a.num_q_heads / a.cache.num_kv_heads;
  const size_t slots = 2 * static_cast<size_t>(p.groups * p.members);
  p.counters = static_cast<unsigned long long*>(workspace);
  p.ws_o = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + counter_bytes(slots));
  p.ws_ml = p.ws_o + slots * G * HD;
  switch (G) {
    case 1: return launch_g<1>(a, p, stream);
    case 2: return launch_g<2>(a, p, stream);
    case 4: return launch_g<4>(a, p, stream);
    case 8: return launch_g<8>(a, p, stream);
    case 16: return launch_g<16>(a, p, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace pa
