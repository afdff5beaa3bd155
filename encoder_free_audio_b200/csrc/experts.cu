// The experts' gated products of the decoder's mixture-of-experts block ("Inside Inkling: Audio
// Design", Part 3 · Inference: 256 routed and 2 shared experts, 6 chosen per token):
//     out[t] = sum_j weights[t, j] (silu(x[t] G_e) * (x[t] U_e)) D_e,   e = ids[t, j].
//
// Four steps: a plan (the slots ordered by expert, cut into tiles of tokens), the gate and up
// products with the gating in the epilogue, the down product, and each token's weighted sum. With more
// than kSmallSlots slots each has a launch. Up to that, the last block of the down product to finish
// some columns sums them, and every block of the first product makes the plan itself: two launches;
// or three, with the plan's own, where K of the first product is split.
//
// Both products run on the tensor cores with the roles swapped: an expert's weights are the M
// side (256 weight columns per pair of CTAs) and its tokens the N side, whose size an MMA takes in
// steps of 16. So an expert with 5 tokens costs a 16-wide MMA and streams its weights once, one
// with 700 costs three tiles of about 240, and no tile is padded by more than 15 tokens.
//
// A product kernel is persistent, one CTA pair per two SMs: a TMA warp loads weight boxes (64
// columns x 64 K, MN-major, 128-byte swizzle) and, for the down product, the gated rows, which lie in
// expert order; two or eight gather warps of the first product load token rows four at a time
// (K-major) by their index, so tokens are never copied into that order; an elected lane of one warp
// issues M = 256, K = 16 MMAs into TMEM, which holds two tiles' accumulators (or one tall tile's: its
// two halves are the two sets of columns); eight warps, in two groups of four, move finished
// accumulators (a lane per weight column) through shared memory into rows.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math_constants.h>
#include <stdint.h>

#include "common.cuh"
#include "internal.h"

namespace dmel {
namespace {

constexpr unsigned kAll = 0xffffffffu;

// One tile of tokens: rows [row0, row0 + rows) of the expert-ordered slots, all of one expert;
// `width` is rows rounded up to the MMA's step of 16.
struct TokenTile {
  int expert, row0, rows, width;
};

// ---------------------------------------------------------------- plan
//
// The slots in expert order, stable, by counting: a warp counts its chunk of slots per expert, a
// scan over (expert, block, warp) turns the counts into row numbers, and the same walk hands them
// out. Bound by the matching of 32 slots at a time (about 190 cycles of a scheduler each): one
// block for few slots, else a cluster of eight that read each other's counts (24,576 slots: 10 us,
// with one block 48).
constexpr int kPlanThreads = 1024;
constexpr int kAhead = 8;  // slots per lane whose ids are loaded before any is counted

struct PlanOut {
  int *n_tiles;      // [1]
  TokenTile *tiles;
  int *token;        // [n_slots] row -> token
  int *row;          // [n_slots] slot -> row, -1 for a slot without an expert
};

// What a call's kernels share beside the operands of the products.
struct Shared {
  const int32_t *ids;
  const float *weights;
  int n_slots, slots, n_experts;
  int splits;           // of the first product's K, joined by the last block of a tile to finish
  int n_counters;       // per 128 columns of the output: token tiles done; then, with splits, per
  int *counters;        //   tile and CTA of the first product: splits done
  float *partial;       // with splits: [tile][split][CTA of the pair][tokens][128]
  float *scales;        // of the slots' output rows
  __nv_bfloat16 *out;
  PlanOut plan;
};

__global__ void __launch_bounds__(kPlanThreads) experts_plan_kernel(const Shared call, int tile_tokens,
                                                                    uint32_t *err) {
  const int32_t *const ids = call.ids;
  const int n_slots = call.n_slots, slots = call.slots, E = call.n_experts;
  const PlanOut &out = call.plan;
  extern __shared__ int hist[];  // [32 warps][E], the block's totals [E], the experts' first rows [E]
  __shared__ unsigned long long warp_sum[32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int *total = hist + 32 * E, *first = total + E;
  const unsigned block = cluster_ctarank(), blocks = gridDim.x;  // one cluster
  wait_for_predecessors();
  launch_dependents();
  if (block == 0)
    for (int i = threadIdx.x; i < call.n_counters; i += kPlanThreads) call.counters[i] = 0;
  // slots per warp, a multiple of 32 (n_slots <= 2^30)
  const int walkers = 32 * (int)blocks, chunk = ((n_slots + walkers - 1) / walkers + 31) / 32 * 32;
  const int walker = (int)block * 32 + warp;
  const int begin = (int64_t)walker * chunk < n_slots ? walker * chunk : n_slots;
  const int end = n_slots - begin < chunk ? n_slots : begin + chunk;
  // warps of this block that have slots (with few slots most have none, nor counts to add up)
  const int64_t mine = n_slots - (int64_t)block * 32 * chunk;
  const int used = mine <= 0 ? 0 : mine >= 32 * (int64_t)chunk ? 32 : (int)((mine + chunk - 1) / chunk);
  for (int i = threadIdx.x; i < used * E; i += kPlanThreads) hist[i] = 0;
  __syncthreads();
  auto expert_at = [&](int i) {
    if (i >= end) return -1;
    const int e = ids[i];
    return e >= 0 && e < E ? e : -1;
  };
  int e[kAhead], rank[kAhead];  // of a batch's slots: the expert, and the warp's slots of it before
  auto count_batch = [&](int i) {
#pragma unroll
    for (int a = 0; a < kAhead; ++a) e[a] = expert_at(i + 32 * a + lane);
#pragma unroll
    for (int a = 0; a < kAhead; ++a) {
      if (i + 32 * a >= end) break;
      const unsigned peers = __match_any_sync(kAll, e[a]);
      rank[a] = e[a] >= 0 ? hist[warp * E + e[a]] + __popc(peers & ((1u << lane) - 1u)) : 0;
      __syncwarp();
      if (e[a] >= 0 && lane == __ffs(peers) - 1) hist[warp * E + e[a]] += __popc(peers);
      __syncwarp();
    }
  };
  for (int i = begin; i < end; i += 32 * kAhead) count_batch(i);
  __syncthreads();
  // counts -> exclusive row offsets within the expert, per warp of this block; then over the blocks
  int count = 0, tiles = 0, before_block = 0;
  const int e_mine = threadIdx.x;  // E <= 1024
  if (e_mine < E) {
    for (int w = 0; w < used; ++w) {
      const int c = hist[w * E + e_mine];
      hist[w * E + e_mine] = count;
      count += c;
    }
    total[e_mine] = count;
  }
  __syncwarp();
  if (blocks > 1) {
    cluster_sync();
    if (e_mine < E) {
      count = 0;
      for (unsigned q = 0; q < blocks; ++q) {
        if (q == block) before_block = count;
        count += (int)ld_cluster_u32(mapa_shared(smem_addr(total + e_mine), q));
      }
    }
    __syncwarp();
    cluster_sync();  // (no block leaves, or reuses its totals, while another reads them)
  }
  tiles = (count + tile_tokens - 1) / tile_tokens;
  // exclusive scan of {tiles, rows} over the experts
  const unsigned long long own = ((unsigned long long)tiles << 32) | (unsigned)count;
  unsigned long long run = own;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const unsigned long long up = __shfl_up_sync(kAll, run, o);
    if (lane >= o) run += up;
  }
  if (lane == 31) warp_sum[warp] = run;
  __syncthreads();
  if (warp == 0) {
    unsigned long long v = warp_sum[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const unsigned long long up = __shfl_up_sync(kAll, v, o);
      if (lane >= o) v += up;
    }
    warp_sum[lane] = v;
  }
  __syncthreads();
  const unsigned long long before = run - own + (warp > 0 ? warp_sum[warp - 1] : 0ull);
  if (e_mine < E) {
    const int row0 = (int)(unsigned)before, tile0 = (int)(before >> 32);
    first[e_mine] = row0 + before_block;
    if (tiles > 0 && block == 0) {
      const int width = ((count + tiles - 1) / tiles + 15) / 16 * 16;
      for (int m = 0; m < tiles; ++m) {
        const int left = count - m * width, rows = left < width ? left : width;
        TokenTile t;
        t.expert = e_mine;
        t.row0 = row0 + m * width;
        t.rows = rows;
        t.width = (rows + 15) / 16 * 16;
        out.tiles[tile0 + m] = t;
      }
    }
  }
  if (threadIdx.x == kPlanThreads - 1 && block == 0) *out.n_tiles = (int)((before + own) >> 32);
  __syncthreads();
  // hist now has the rows before the warp's own. The last batch's ranks are still there: with one
  // batch per warp (65,536 slots) no slot is matched twice.
  for (int i = begin; i < end; i += 32 * kAhead) {
    if (chunk > 32 * kAhead) count_batch(i);  // (on from the offset, so these ranks include it)
#pragma unroll
    for (int a = 0; a < kAhead; ++a) {
      const int slot = i + 32 * a + lane;
      if (slot >= end) break;
      int pos = -1;
      if (e[a] >= 0) {
        pos = first[e[a]] + rank[a] + (chunk > 32 * kAhead ? 0 : hist[warp * E + e[a]]);
        out.token[pos] = slot / slots;
      } else if (ids[slot] != -1) {
        record_error(err, DMEL_DEVERR_EXPERT);
      }
      out.row[slot] = pos;
    }
  }
}

// The same for at most kSmallSlots slots, by every block of the first product for itself in shared
// memory, by comparing each slot with all others. The `writer` block also leaves it in memory for
// the second product, and clears its counters. With the sums in the second product that saves two
// launches, which both cost more than with many slots: the comparisons, and a fence per work item. 6
// slots a token on 32 experts, 6144 x 1024: 6 slots 46 us against 49, 24 slots 110 against 111, 60 slots
// 185 against 181, 66 slots 190 against 184, 192 slots 220 against 202; 128 slots on 8 experts,
// 2048 x 512: 32 against 23. (Up to here the slots' rows stay in fp32 as well.)
constexpr int kSmallSlots = 64;

struct SmallPlan {
  TokenTile tiles[kSmallSlots];
  int token[kSmallSlots];
  int n_tiles;
};

__device__ __forceinline__ void make_small_plan(const Shared &c, int tile_tokens, SmallPlan *p, int *expert,
                                                int *starts, bool writer, uint32_t *err) {
  const int n = c.n_slots;
  for (int i = threadIdx.x; i < n; i += blockDim.x) {
    const int e = c.ids[i];
    const bool valid = e >= 0 && e < c.n_experts;
    if (!valid && e != -1) record_error(err, DMEL_DEVERR_EXPERT);
    expert[i] = valid ? e : INT32_MAX;
  }
  if (threadIdx.x == 0) p->n_tiles = 0;
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += blockDim.x) {
    const int e = expert[i];
    int first = 0, count = 0, before = 0;  // slots of lower experts, of this one, of this one before i
    for (int j = 0; j < n; ++j) {
      const int o = expert[j];
      first += o < e;
      count += o == e;
      before += o == e && j < i;
    }
    int rows = 0;  // of the tile that starts with this slot
    if (e != INT32_MAX) {
      const int tiles = (count + tile_tokens - 1) / tile_tokens, width = ((count + tiles - 1) / tiles + 15) / 16 * 16;
      p->token[first + before] = i / c.slots;
      if (before % width == 0) {
        rows = count - before < width ? count - before : width;
        atomicAdd(&p->n_tiles, 1);
      }
    }
    starts[i] = rows;
    if (writer) c.plan.row[i] = e != INT32_MAX ? first + before : -1;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += blockDim.x) {
    if (starts[i] == 0) continue;
    const int e = expert[i];
    int at = 0, row0 = 0;  // tiles before this one, and its first row
    for (int j = 0; j < n; ++j) {
      const bool earlier = expert[j] < e || (expert[j] == e && j < i);
      row0 += earlier;
      at += earlier && starts[j] != 0;
    }
    TokenTile t;
    t.expert = e;
    t.row0 = row0;
    t.rows = starts[i];
    t.width = (starts[i] + 15) / 16 * 16;
    p->tiles[at] = t;
    if (writer) c.plan.tiles[at] = t;
  }
  if (writer) {
    for (int i = threadIdx.x; i < c.n_counters; i += blockDim.x) c.counters[i] = 0;
    if (threadIdx.x == 0) *c.plan.n_tiles = p->n_tiles;
  }
  __syncthreads();
}

// ---------------------------------------------------------------- products (tcgen05, CTA pairs)
//
// kGate: D[columns x tokens] of both the gate's and the up product: each CTA's 128 M rows are 64 of
// the gate's columns and the 64 up columns beside them, the epilogue writes bf16(silu(g) u) to
// h [rows x hidden]. (bf16 is what the next MMA takes beside bf16 weights, at fp32's range. This
// rounding and the output's are of one size: 0.0024 of the output's norm together, 0.0017 alone.) Otherwise: 128 columns of the down product per CTA, written as a slot's row in
// fp16 with a power-of-two scale per 128 columns, or in fp32 in a small call. (fp32 rows, written
// and read back, cost a prompt of 4,096 tokens 50 us of 937. 11 bits beside the scale are off
// by 2^-11 at most, an eighth of the rounding of the gated row and of the output to bf16; the
// tokens' sums are fp32.)
template <int kTokens, bool kSmall = false, bool kTall = false>
struct EX {
  static constexpr int SETS = kTall ? 2 : 1;           // accumulators per tile, of 256 M rows per pair
  static constexpr int ACCS = 2 / SETS;                // tiles in TMEM at a time
  static constexpr int BK = 64;                        // K per stage: 128 bytes of a token row
  static constexpr int BOX = 64 * BK * 2;              // 64 columns x 64 K rows of weights: 8 KB
  static constexpr int A_STAGE = SETS * 2 * BOX;       // this CTA's 128 M rows of each set
  static constexpr int B_STAGE = kTokens / 2 * BK * 2; // this CTA's half of the tokens
  static constexpr int EPI_GROUPS = 2, EPI_WARPS = 4 * EPI_GROUPS;
  static constexpr int STG_TOKENS = 32;
  static constexpr int STG = STG_TOKENS * 128 * 4;     // 32 tokens x 128 columns, fp32
  static constexpr int IDX = kTokens / 2 * 4;          // row numbers of the half, for the gather warps
  static constexpr int PLAN = kSmall ? (int)((sizeof(SmallPlan) + 15) / 16 * 16) : 0;
  static constexpr int BUDGET = 227 * 1024 - 1024 - 512 - IDX - PLAN - EPI_GROUPS * STG;
  static constexpr int STAGES = BUDGET / (A_STAGE + B_STAGE);
  static constexpr int OFF_B = STAGES * A_STAGE;
  static constexpr int OFF_STG = OFF_B + STAGES * B_STAGE;
  static constexpr int OFF_BAR = OFF_STG + EPI_GROUPS * STG;
  static constexpr int N_BARS = 2 * STAGES + 4 + 1;
  static constexpr int OFF_LAST = OFF_BAR + 504;
  static constexpr int OFF_IDX = OFF_BAR + 512;
  static constexpr int OFF_PLAN = OFF_IDX + IDX;
  static constexpr int SMEM_BYTES = OFF_PLAN + PLAN + 1024;
  // warp 0 TMA, warp 1 MMA, warps 2..9 epilogue, and for the gate and up products gather warps. What
  // bounds a gather of up to 128 rows per stage is how fast its loads are issued: 4,096 tokens of 6
  // slots, 6144 x 2 x 1024: 780 us with two warps, 584 with four, 517 with eight (393 without any
  // rows loaded). Copies by threads (16 bytes each) came to 1,350 us: the fence between them and the
  // tensor cores takes about a microsecond per stage.
  static constexpr int GATHER_WARPS = kTokens > 64 ? 8 : 2;
  static constexpr int THREADS = 32 * (2 + EPI_WARPS);
  static constexpr int THREADS_GATE = THREADS + 32 * GATHER_WARPS;
  static constexpr uint32_t TMEM_COLS = 2 * kTokens < 32 ? 32 : 2 * kTokens;
  static_assert(kTokens % 32 == 0 && kTokens <= 256 && (TMEM_COLS & (TMEM_COLS - 1)) == 0, "token tile");
  static_assert(B_STAGE % 1024 == 0 && STAGES >= 4 && STAGES <= 24, "stages");
  static_assert(N_BARS * 8 + 8 <= 504 && SMEM_BYTES <= 227 * 1024, "shared memory budget");
};

// Barrier of an epilogue group's 128 threads; and one that also ANDs a flag, so that all take the same branch.
__device__ __forceinline__ void group_bar(int group) { asm volatile("bar.sync %0, 128;" ::"r"(1 + group) : "memory"); }
__device__ __forceinline__ bool group_bar_and(int group, bool v) {
  return group == 0 ? group_and<1, 128>(v) : group_and<2, 128>(v);
}

__device__ __forceinline__ float4 silu_times(float4 g, float4 u) {
  // __expf and __fdividef are within a few fp32 ulps here; the result is rounded to bf16
  return make_float4(__fdividef(g.x, 1.0f + __expf(-g.x)) * u.x, __fdividef(g.y, 1.0f + __expf(-g.y)) * u.y,
                     __fdividef(g.z, 1.0f + __expf(-g.z)) * u.z, __fdividef(g.w, 1.0f + __expf(-g.w)) * u.w);
}

// The power of two that takes a block's largest magnitude to [2^14, 2^15), inside fp16's range with
// 28 binades of normal numbers below. Between 2^-112 and 2^112, so that it and its reciprocal are
// normal fp32 numbers. A warp's lanes hold the block; what is not finite does not enter and stays so.
__device__ __forceinline__ float row_scale_up(float4 r) {
  float top = warp_max(fmaxf(fmaxf(fabsf(r.x), fabsf(r.y)), fmaxf(fabsf(r.z), fabsf(r.w))));
  if (!(top < CUDART_INF_F)) {
    auto finite = [](float v) { return fabsf(v) < CUDART_INF_F ? fabsf(v) : 0.0f; };
    top = warp_max(fmaxf(fmaxf(finite(r.x), finite(r.y)), fmaxf(finite(r.z), finite(r.w))));
  }
  const int up = 127 + 14 + 127 - (int)(__float_as_uint(top) >> 23);  // (of the biased exponent)
  return __uint_as_float((uint32_t)min(max(up, 127 - 112), 127 + 112) << 23);
}

// Four values of a slot's row.
__device__ __forceinline__ float4 row4(const uint2 u, float scale) {
  const float2 a = __half22float2(*reinterpret_cast<const __half2 *>(&u.x));
  const float2 b = __half22float2(*reinterpret_cast<const __half2 *>(&u.y));
  return make_float4(a.x * scale, a.y * scale, b.x * scale, b.y * scale);
}

// Called by the 256 epilogue threads after their writes of a work item: whether this is the last of n
// items to come here (whatever the order), whose threads then see the others' writes. Nothing waits.
// (One thread's fences after the barrier cover the others' writes; a fence in each costs a
// microsecond more per call.)
__device__ __forceinline__ bool last_of(int n, int *counter, int *flag) {
  asm volatile("bar.sync 3, 256;" ::: "memory");
  if (threadIdx.x == 64) {
    __threadfence();
    *flag = atomicAdd(counter, 1) == n - 1;
    __threadfence();
  }
  asm volatile("bar.sync 3, 256;" ::: "memory");
  return *flag != 0;
}

// The gated rows of a tile whose K was split: the splits' partial sums in order.
template <int kTokens>
__device__ __forceinline__ void join_splits(const Shared &c, __nv_bfloat16 *h, int64_t tile, int rank, const TokenTile &tt,
                                            int hidden, int col) {
  const int et = threadIdx.x - 64, q = 4 * (et & 15);
  if (col + q >= hidden) return;
  const float *base = c.partial + (tile * c.splits * 2 + rank) * kTokens * 128 + q;
  for (int k = et >> 4; k < tt.rows; k += 16) {
    float4 g = make_float4(0.0f, 0.0f, 0.0f, 0.0f), u = g;
#pragma unroll 4
    for (int s = 0; s < c.splits; ++s) {
      const float *p = base + ((int64_t)s * 2 * kTokens + k) * 128;
      const float4 a = __ldcg(reinterpret_cast<const float4 *>(p)), b = __ldcg(reinterpret_cast<const float4 *>(p + 64));
      g.x += a.x; g.y += a.y; g.z += a.z; g.w += a.w;
      u.x += b.x; u.y += b.y; u.z += b.z; u.w += b.w;
    }
    const float4 y = silu_times(g, u);
    *reinterpret_cast<uint2 *>(h + (int64_t)(tt.row0 + k) * hidden + col + q) =
        make_uint2(pack_bf16(y.x, y.y), pack_bf16(y.z, y.w));
  }
}

// The slots' rows and weights in shared memory, for small_sum: read by the 256 epilogue threads while
// the products run.
struct SmallSlots {
  int row[kSmallSlots];
  float weight[kSmallSlots];
};
__device__ __forceinline__ void load_slots(const Shared &c, SmallSlots *s) {
  const int i = threadIdx.x - 64;
  if (i >= c.n_slots) return;
  const int r = c.plan.row[i];
  s->row[i] = r;
  s->weight[i] = r < 0 ? 0.0f : c.weights[i];
}

// 128 columns from `col` on of every token's weighted sum, by the 256 epilogue threads: the rows y
// (dim columns each, other blocks' work among them) in slot order.
__device__ __forceinline__ void small_sum(const Shared &c, const SmallSlots &s, const float *y, int dim, int col) {
  const int et = threadIdx.x - 64, q = col + 4 * (et & 31), n_tokens = c.n_slots / c.slots;
  if (q >= dim) return;
  for (int t = et >> 5; t < n_tokens; t += 8) {
    float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
    for (int j = 0; j < c.slots; ++j) {
      const int r = s.row[t * c.slots + j];
      if (r < 0) continue;
      const float w = s.weight[t * c.slots + j];
      const float4 v = __ldcg(reinterpret_cast<const float4 *>(y + (int64_t)r * dim + q));
      acc.x = fmaf(w, v.x, acc.x);
      acc.y = fmaf(w, v.y, acc.y);
      acc.z = fmaf(w, v.z, acc.z);
      acc.w = fmaf(w, v.w, acc.w);
    }
    *reinterpret_cast<uint2 *>(c.out + (int64_t)t * dim + q) =
        make_uint2(pack_bf16(acc.x, acc.y), pack_bf16(acc.z, acc.w));
  }
}

// kSmall: the gate's kernel makes the plan, the down product's kernel the tokens' sums (Shared).
// kSplit: K in parts (of the gate's kernel).
// kTall: tiles of twice the columns (of the gate's kernel), with both halves of TMEM for one tile. What
// bounds wide tiles is the loads from L2 (12 TB/s, 6.7 GB for 4,096 tokens of 6 slots, 6144 x 2 x
// 1024, the tensor pipe 58 % active); a tall tile needs three quarters of the bytes, and more than
// makes up for an epilogue that nothing runs under where K is long (the whole call: 924 us to 863).
template <int kTokens, bool kGate, bool kSmall, bool kSplit, bool kTall>
__global__ void __launch_bounds__(kGate ? EX<kTokens, kSmall, kTall>::THREADS_GATE : EX<kTokens, kSmall, kTall>::THREADS, 1)
    experts_product_kernel(const __grid_constant__ CUtensorMap wmap, const __grid_constant__ CUtensorMap xmap,
                           const __grid_constant__ CUtensorMap xmap8, const int *n_tiles,
                           const TokenTile *tiles, const int *token, int K, int cols, void *out, const Shared shared,
                           uint32_t *err) {
  using X = EX<kTokens, kSmall, kTall>;
  constexpr int STAGES = X::STAGES, BK = X::BK;
  constexpr int SET_COLS = kGate ? 64 : 128, COLS = SET_COLS * X::SETS;  // columns of the output per CTA
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t *smem = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const bool leader = rank == 0;
  const uint32_t bar0 = smem_addr(smem + X::OFF_BAR);
  auto full = [&](int s) { return bar0 + 8u * s; };
  auto empty = [&](int s) { return bar0 + 8u * (STAGES + s); };
  auto tfull = [&](int a) { return bar0 + 8u * (2 * STAGES + a); };
  auto tempty = [&](int a) { return bar0 + 8u * (2 * STAGES + 2 + a); };
  const uint32_t done_bar = bar0 + 8u * (2 * STAGES + 4);
  uint32_t *tmem_holder = reinterpret_cast<uint32_t *>(smem + X::OFF_BAR + X::N_BARS * 8);

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(full(s), 1);   // the even CTA's expect-tx for both CTAs' loads
      mbar_init(empty(s), 1);  // the even CTA's commit, to both
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(tfull(a), 1);
      mbar_init(tempty(a), 2 * X::EPI_WARPS);  // the epilogue warps of both CTAs (even CTA's barrier)
    }
    mbar_init(done_bar, 1);
    mbar_fence_init();
  }
  if (warp == 1) {
    tmem_alloc_pair(smem_addr(tmem_holder), X::TMEM_COLS);
    tmem_relinquish_pair();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&wmap);
    tma_prefetch_desc(&xmap);
  }
  tc_fence_before();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_holder;
  // (Letting the down product load its first weights before this wait measured the same.)
  wait_for_predecessors();
  launch_dependents();
  int token_tiles;
  if (kSmall && kGate) {
    SmallPlan *p = reinterpret_cast<SmallPlan *>(smem + X::OFF_PLAN);
    int *scratch = reinterpret_cast<int *>(smem + X::OFF_STG);  // (the epilogue's, not yet in use)
    make_small_plan(shared, kTokens, p, scratch, scratch + kSmallSlots, blockIdx.x == 0, err);
    token_tiles = p->n_tiles;
    tiles = p->tiles;
    token = p->token;
  } else {
    token_tiles = *n_tiles;
  }

  const int n_ct = (cols + 2 * COLS - 1) / (2 * COLS);  // column tiles
  const int splits = kSplit ? shared.splits : 1;
  const int64_t total = (int64_t)token_tiles * n_ct * splits;
  const int KB = (K + BK - 1) / BK;
  const int64_t step = gridDim.x >> 1;
  // Work item u: split u % splits of K (blocks kb0 .. kb1 - 1) of tile u / splits. Consecutive pairs
  // take the column tiles of one token tile (its rows stay in L2).
  auto tile_of = [&](int64_t u) { return kSplit ? u / splits : u; };
  auto token_tile = [&](int64_t u) { return tiles[tile_of(u) / n_ct]; };
  auto column = [&](int64_t u) { return (int)(tile_of(u) % n_ct) * 2 * COLS + (int)rank * COLS; };
  // The rows of a tile that CTA r loads: those of its half that are there, to a whole load of 4 (gathered)
  // or 8. What lies behind them in shared memory is multiplied into columns that nobody stores. (One
  // token's 6 experts: 49.2 us, with the token's row gathered into all 16 places 55.)
  constexpr int LOAD = kGate ? 4 : 8;
  auto rows_of = [&](const TokenTile &tt, int r) {
    const int half = tt.width / 2, left = tt.rows - r * half;
    return (min(max(left, 0), half) + LOAD - 1) / LOAD * LOAD;
  };
  auto kb_begin = [&](int64_t u) { return kSplit ? KB * (int)(u % splits) / splits : 0; };
  auto kb_end = [&](int64_t u) { return kSplit ? KB * ((int)(u % splits) + 1) / splits : KB; };

  if (warp == 0) {
    // ------------------------------------------------ TMA: weight boxes, and consecutive rows
    int stage = 0;
    uint32_t phase = 0, pending = 0, pending_phase = 0;
    bool ok = true;
    for (int64_t t = blockIdx.x >> 1; ok && t < total; t += step) {
      const TokenTile tt = token_tile(t);
      const int col = column(t), kb1 = kb_end(t);
      const int rows = rows_of(tt, (int)rank);
      const uint32_t bytes = 2u * X::A_STAGE + 128u * (uint32_t)(rows_of(tt, 0) + rows_of(tt, 1));
      for (int kb = kb_begin(t); kb < kb1; ++kb) {
        if (!__all_sync(kAll, mbar_wait(empty(stage), phase ^ 1u, err))) { ok = false; break; }
        if (elect_one()) {
          if (leader) mbar_arrive_expect_tx(full(stage), bytes);
          const uint32_t fb = mapa_shared(full(stage), 0);
          const uint32_t a_dst = smem_addr(smem + stage * X::A_STAGE);
#pragma unroll
          for (int set = 0; set < X::SETS; ++set) {
            // kGate: the gate's box, then the up box `cols` further on
            const int c0 = col + SET_COLS * set;
            tma_load_3d_pair(a_dst + 2 * set * X::BOX, &wmap, c0, kb * BK, tt.expert, fb);
            tma_load_3d_pair(a_dst + (2 * set + 1) * X::BOX, &wmap, c0 + (kGate ? cols : 64), kb * BK, tt.expert, fb);
          }
          if (!kGate) {
            // rows past the tile in its last box are the next expert's, or zeros past the last
            const uint32_t b_dst = smem_addr(smem + X::OFF_B + stage * X::B_STAGE);
            const int row = tt.row0 + (int)rank * (tt.width / 2);
            int r = 0;
            for (; r + 32 <= rows; r += 32) tma_load_2d_pair(b_dst + r * 128, &xmap, kb * BK, row + r, fb);
            for (; r < rows; r += 8) tma_load_2d_pair(b_dst + r * 128, &xmap8, kb * BK, row + r, fb);
          }
        }
        __syncwarp();
        pending |= 1u << stage;
        pending_phase = (pending_phase & ~(1u << stage)) | (phase << stage);
        if (++stage == STAGES) { stage = 0; phase ^= 1u; }
      }
    }
    // the even CTA's barriers count every load; it waits for the last ones before leaving
    if (leader)
      for (int s = 0; s < STAGES; ++s)
        if (pending & (1u << s)) mbar_wait(full(s), (pending_phase >> s) & 1u, err);
  } else if (warp == 1) {
    // ------------------------------------------------ MMA issuer (even CTA)
    if (leader) {
      int stage = 0;
      uint32_t phase = 0, i = 0;
      bool ok = true;
      for (int64_t t = blockIdx.x >> 1; ok && t < total; t += step, ++i) {
        const uint32_t acc = i % X::ACCS, use = i / X::ACCS;
        const uint32_t idesc = idesc_bf16_f32(256, (uint32_t)token_tile(t).width, 0, 1);
        const int kb0 = kb_begin(t), kb1 = kb_end(t);
        if (!__all_sync(kAll, mbar_wait(tempty(acc), (use & 1u) ^ 1u, err))) break;
        tc_fence_after();
        const uint32_t d = tmem_base + acc * kTokens;
        for (int kb = kb0; kb < kb1; ++kb) {
          if (!__all_sync(kAll, mbar_wait(full(stage), phase, err))) { ok = false; break; }
          tc_fence_after();
          const uint32_t a0 = smem_addr(smem + stage * X::A_STAGE);
          const uint32_t b0 = smem_addr(smem + X::OFF_B + stage * X::B_STAGE);
          if (elect_one()) {
#pragma unroll
            for (int set = 0; set < X::SETS; ++set) {
#pragma unroll
              for (int k = 0; k < BK / 16; ++k) {
                // weights: MN-major, 64-column boxes BOX apart, 8 K-rows 1024 B apart, 16 (2 KB) per step
                const uint64_t adesc = smem_desc(a0 + 2 * set * X::BOX + 2048u * k, (uint32_t)X::BOX, 1024u, kSwizzle128B);
                // tokens: K-major, 8-row groups 1024 B apart, 32 B per step
                const uint64_t bdesc = smem_desc(b0 + 32u * k, 16u, 1024u, kSwizzle128B);
                tc_mma_f16_pair(d + set * kTokens, adesc, bdesc, idesc, kb > kb0 || k > 0 ? 1u : 0u);
              }
            }
            tc_commit_pair_both(empty(stage), 3);
          }
          __syncwarp();
          if (++stage == STAGES) { stage = 0; phase ^= 1u; }
        }
        if (!ok) break;
        if (elect_one()) tc_commit_pair_both(tfull(acc), 3);
        __syncwarp();
      }
      if (elect_one()) tc_commit_pair(done_bar);
      __syncwarp();
      mbar_wait(done_bar, 0, err);
    }
  } else if (kGate && warp >= 2 + X::EPI_WARPS) {
    // ------------------------------------------------ gather: token rows four at a time, by number
    // Gather warp w takes the groups of four rows w, w + GATHER_WARPS, ... of this CTA's half.
    const int w = warp - 2 - X::EPI_WARPS;
    int4 *idx = reinterpret_cast<int4 *>(smem + X::OFF_IDX);
    int stage = 0;
    uint32_t phase = 0;
    bool ok = true;
    for (int64_t t = blockIdx.x >> 1; ok && t < total; t += step) {
      const TokenTile tt = token_tile(t);
      const int kb1 = kb_end(t), groups = rows_of(tt, (int)rank) / 4;
      __syncwarp();                     // the last tile's numbers have been read
      for (int g = w + X::GATHER_WARPS * lane; g < groups; g += X::GATHER_WARPS * 32) {
        int r[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int q = (int)rank * (tt.width / 2) + 4 * g + i;  // past the tile: its last row again
          r[i] = token[tt.row0 + (q < tt.rows ? q : tt.rows - 1)];
        }
        idx[g] = make_int4(r[0], r[1], r[2], r[3]);
      }
      __syncwarp();
      for (int kb = kb_begin(t); kb < kb1; ++kb) {
        if (!__all_sync(kAll, mbar_wait(empty(stage), phase ^ 1u, err))) { ok = false; break; }
        if (elect_one()) {
          const uint32_t fb = mapa_shared(full(stage), 0);
          const uint32_t b_dst = smem_addr(smem + X::OFF_B + stage * X::B_STAGE);
#pragma unroll 4
          for (int g = w; g < groups; g += X::GATHER_WARPS) {
            const int4 r = idx[g];
            tma_gather4_pair(b_dst + g * 512, &xmap, kb * BK, r.x, r.y, r.z, r.w, fb);
          }
        }
        __syncwarp();
        if (++stage == STAGES) { stage = 0; phase ^= 1u; }
      }
    }
  } else {
    // ------------------------------------------------ epilogue: lane = one M row (weight column)
    // EPI_GROUPS groups of four warps (one per TMEM lane quarter) take chunks of 32 tokens in turn,
    // each through a staging buffer of its own.
    const int quad = warp & 3, group = (warp - 2) >> 2, et = (threadIdx.x - 64) & 127;
    float *const buf = reinterpret_cast<float *>(smem + X::OFF_STG + group * X::STG);
    int *last = reinterpret_cast<int *>(smem + X::OFF_LAST);
    SmallSlots *const slots = reinterpret_cast<SmallSlots *>(smem + X::OFF_PLAN);  // (last_of's barrier is between)
    static_assert(sizeof(SmallSlots) <= sizeof(SmallPlan), "shared memory of the small plan");
    if (kSmall && !kGate) load_slots(shared, slots);
    uint32_t i = 0;
    bool ok = true;
    for (int64_t t = blockIdx.x >> 1; t < total; t += step, ++i) {
      const uint32_t acc = i % X::ACCS, use = i / X::ACCS;
      const TokenTile tt = token_tile(t);
      const int first_col = column(t);
      ok = group_bar_and(group, ok && mbar_wait(tfull(acc), use & 1u, err));
      tc_fence_after();
      // chunks of both sets, the sets one after the other
      const int per_set = (tt.width + X::STG_TOKENS - 1) / X::STG_TOKENS;
      for (int n = group; ok && n < per_set * X::SETS; n += X::EPI_GROUPS) {
        const int set = X::SETS > 1 && n >= per_set ? 1 : 0, c = X::STG_TOKENS * (n - set * per_set);
        const int col = first_col + SET_COLS * set;
        const uint32_t tb = tmem_base + ((uint32_t)(32 * quad) << 16) + (acc + set) * kTokens;
        // 32 tokens (16 where the tile ends) of this lane's column into the staging rows
        const bool wide = tt.width - c >= 32;
        uint32_t v[2][16];
        tmem_ld16(tb + c, v[0]);
        if (wide) tmem_ld16(tb + c + 16, v[1]);
        tmem_wait_ld();
        const int m = 32 * quad + lane;
#pragma unroll
        for (int k = 0; k < 16; ++k) buf[k * 128 + m] = __uint_as_float(v[0][k]);
        if (wide) {
#pragma unroll
          for (int k = 0; k < 16; ++k) buf[(16 + k) * 128 + m] = __uint_as_float(v[1][k]);
        }
        group_bar(group);
        const int n_tok = tt.rows - c < 32 ? tt.rows - c : 32;
        if (kSplit) {
          float *part = shared.partial + ((t * 2 + rank) * kTokens + c) * 128 + 4 * (et & 31);
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const int k = (et >> 5) + 4 * j;
            const float4 r = *reinterpret_cast<const float4 *>(buf + k * 128 + 4 * (et & 31));
            if (k < n_tok) *reinterpret_cast<float4 *>(part + k * 128) = r;
          }
        } else if (kGate) {
          __nv_bfloat16 *h = static_cast<__nv_bfloat16 *>(out) + (int64_t)(tt.row0 + c) * cols + col;
          const int q = et & 15, k0 = et >> 4;  // 4 columns, a token per 16 threads
          if (col + 4 * q < cols) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const int k = k0 + 8 * j;
              const float4 g = *reinterpret_cast<const float4 *>(buf + k * 128 + 4 * q);
              const float4 u = *reinterpret_cast<const float4 *>(buf + k * 128 + 64 + 4 * q);
              const float4 y = silu_times(g, u);
              if (k < n_tok)
                *reinterpret_cast<uint2 *>(h + (int64_t)k * cols + 4 * q) =
                    make_uint2(pack_bf16(y.x, y.y), pack_bf16(y.z, y.w));
            }
          }
        } else {
          const int64_t row0 = tt.row0 + c;
          const int q = et & 31, k0 = et >> 5;  // 4 columns, a token per warp
          float4 r[8];                          // every read (and reduction) before any store
#pragma unroll
          for (int j = 0; j < 8; ++j) r[j] = *reinterpret_cast<const float4 *>(buf + (k0 + 4 * j) * 128 + 4 * q);
          if (kSmall) {
            float *y = static_cast<float *>(out) + row0 * cols + col + 4 * q;
#pragma unroll
            for (int j = 0; j < 8; ++j)
              if (k0 + 4 * j < n_tok && col + 4 * q < cols)
                *reinterpret_cast<float4 *>(y + (int64_t)(k0 + 4 * j) * cols) = r[j];
          } else {
            __half *y = static_cast<__half *>(out) + row0 * cols + col + 4 * q;
            const int n_blocks = (cols + 127) / 128;
            float *scales = shared.scales + row0 * n_blocks + col / 128;
            float up[8];
            // (columns past the last are zeros: the weights' fill)
#pragma unroll
            for (int j = 0; j < 8; ++j) up[j] = row_scale_up(r[j]);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const int k = k0 + 4 * j;
              if (k < n_tok && col + 4 * q < cols) {
                const __half2 lo = __floats2half2_rn(r[j].x * up[j], r[j].y * up[j]);
                const __half2 hi = __floats2half2_rn(r[j].z * up[j], r[j].w * up[j]);
                *reinterpret_cast<uint2 *>(y + (int64_t)k * cols) =
                    make_uint2(*reinterpret_cast<const uint32_t *>(&lo), *reinterpret_cast<const uint32_t *>(&hi));
                if (q == 0)  // 1 / up, a power of two as well
                  scales[(int64_t)k * n_blocks] = __uint_as_float(0x7f000000u - __float_as_uint(up[j]));
              }
            }
          }
        }
        group_bar(group);  // the buffer has been read
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_remote(mapa_shared(tempty(acc), 0));
      if (kSplit) {
        if (last_of(splits, shared.counters + 2 * ((K + 255) / 256) + 2 * tile_of(t) + rank, last))
          join_splits<kTokens>(shared, static_cast<__nv_bfloat16 *>(out), tile_of(t), (int)rank, tt, cols, first_col);
      }
      if (kSmall && !kGate) {
        // these columns of all tokens, when every token tile has been through them
        if (last_of(token_tiles, shared.counters + 2 * (t % n_ct) + rank, last))
          small_sum(shared, *slots, static_cast<const float *>(out), cols, first_col);
      }
    }
    if (kSmall && !kGate && token_tiles == 0) {  // no token has an expert: zeros
      asm volatile("bar.sync 3, 256;" ::: "memory");
      for (int64_t ct = blockIdx.x >> 1; ct < n_ct; ct += step)
        small_sum(shared, *slots, static_cast<const float *>(out), cols, (int)ct * 2 * COLS + (int)rank * COLS);
    }
  }

  tc_fence_before();
  cluster_sync();  // every MMA into either CTA's TMEM has completed (the even CTA waited above)
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem_base, X::TMEM_COLS);
  }
}

// ---------------------------------------------------------------- the tokens' weighted sums
//
// Reads each chosen slot's row once: HBM bound (or L2, where the rows still lie there).
__global__ void __launch_bounds__(256) experts_sum_kernel(const __half *y, const float *scales, const int *row,
                                                          const float *weights, int64_t n_tokens, int slots, int dim,
                                                          __nv_bfloat16 *out) {
  wait_for_predecessors();
  launch_dependents();
  const int pieces = dim / 8, n_blocks = (dim + 127) / 128;
  const int64_t total = n_tokens * pieces;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
    const int64_t t = i / pieces;
    const int p = (int)(i - t * pieces);
    float acc[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 4
    for (int j = 0; j < slots; ++j) {
      const int r = row[t * slots + j];
      if (r < 0) continue;
      const float w = weights[t * slots + j];
      const uint4 u = *reinterpret_cast<const uint4 *>(y + (int64_t)r * dim + 8 * p);
      const float scale = scales[(int64_t)r * n_blocks + p / 16];
      const float4 a = row4(make_uint2(u.x, u.y), scale), b = row4(make_uint2(u.z, u.w), scale);
      acc[0] = fmaf(w, a.x, acc[0]); acc[1] = fmaf(w, a.y, acc[1]);
      acc[2] = fmaf(w, a.z, acc[2]); acc[3] = fmaf(w, a.w, acc[3]);
      acc[4] = fmaf(w, b.x, acc[4]); acc[5] = fmaf(w, b.y, acc[5]);
      acc[6] = fmaf(w, b.z, acc[6]); acc[7] = fmaf(w, b.w, acc[7]);
    }
    *reinterpret_cast<uint4 *>(out + t * dim + 8 * p) = make_uint4(
        pack_bf16(acc[0], acc[1]), pack_bf16(acc[2], acc[3]), pack_bf16(acc[4], acc[5]), pack_bf16(acc[6], acc[7]));
  }
}

// ---------------------------------------------------------------- host

size_t r256(size_t x) { return (x + 255) / 256 * 256; }

constexpr int kPairs = 74;  // pairs of a B200's 148 SMs, for rules that a workspace's size depends on

// How a call is run, from its sizes alone.
struct Config {
  bool small;         // plan and sums inside the products
  int tile_tokens;    // the products' token tiles
  int splits;         // of the first product's K
  int64_t max_tiles;  // token tiles at most
  int n_counters;
};

Config config(int64_t n_tokens, int slots, const dmel_expert_weights &w) {
  Config c;
  const int64_t n = n_tokens * slots;
  // Tiles of 32 tokens (ten stages of weights in flight) where an expert has few on average: the
  // weights' bytes and latency bound such calls. Wider ones share a pass over the weights between
  // their tokens. 6 slots a token on 32 experts, 6144 / 1024, tiles of 32, 128 and 256: 1,536 slots 320,
  // 213 and 213 us; 6,144 slots 1,008, 383 and 258. Since a tile loads only the rows that are there,
  // 32 gains little over 128 (128 slots on 8 experts, 2048 / 512: 23 us each), and it loses where the
  // mean is no guide: 8 slots a token on 258 experts, two of them shared by all tokens, 64 tokens 1,137
  // us for 1,078, 512 tokens 1,624 for 1,436.
  c.tile_tokens = n <= kSmallSlots || n <= 16 * (int64_t)w.n_experts ? 32 : n <= 64 * (int64_t)w.n_experts ? 128 : 256;
  c.max_tiles = n / c.tile_tokens + (n < w.n_experts ? n : w.n_experts);
  // The first product's K in up to 8 parts of 16 blocks or more where its tiles would leave half of
  // the pairs of CTAs without work
  const int64_t tiles = c.max_tiles * ((w.hidden + 127) / 128);
  int64_t splits = kPairs / tiles, most = (w.dim + 63) / 64 / 16;
  if (splits > 8) splits = 8;
  if (splits > most) splits = most;
  c.splits = splits > 1 ? (int)splits : 1;
  c.small = n <= kSmallSlots;
  c.n_counters = (w.dim + 255) / 256 * 2 + (c.splits > 1 ? 2 * (int)tiles : 0);
  return c;
}

struct Layout {
  size_t n_tiles, counters, tiles, token, row, h, y, scales, partial, total;
};
Layout layout(int64_t n_tokens, int slots, const dmel_expert_weights &w) {
  const Config c = config(n_tokens, slots, w);
  const size_t n = (size_t)n_tokens * slots;
  Layout L;
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t here = at;
    at += r256(bytes);
    return here;
  };
  L.n_tiles = take(4);
  L.counters = take((size_t)c.n_counters * 4);
  L.tiles = take((size_t)c.max_tiles * sizeof(TokenTile));
  L.token = take(n * 4);
  L.row = take(n * 4);
  L.h = take(n * w.hidden * 2);
  L.y = take(n * w.dim * (c.small ? 4 : 2));
  L.scales = take(n * ((w.dim + 127) / 128) * 4);
  L.partial = take(c.splits > 1 ? (size_t)c.max_tiles * ((w.hidden + 127) / 128) * c.splits * 2 * c.tile_tokens * 128 * 4 : 0);
  L.total = at;
  return L;
}

// An expert weight stack [E][K][N] (N contiguous) in boxes of 64 columns x 64 K.
bool weight_map(CUtensorMap *map, EncodeTiledFn enc, const void *base, int E, int K, int64_t N) {
  const cuuint64_t dims[3] = {(cuuint64_t)N, (cuuint64_t)K, (cuuint64_t)E};
  const cuuint64_t strides[2] = {(cuuint64_t)N * 2, (cuuint64_t)N * K * 2};
  const cuuint32_t box[3] = {64, 64, 1};
  const cuuint32_t estr[3] = {1, 1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(base), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Rows [R][K] (K contiguous) in boxes of 64 values of box_rows rows (1 for gathering).
bool row_map(CUtensorMap *map, EncodeTiledFn enc, const void *base, int64_t R, int K, unsigned box_rows) {
  const cuuint64_t dims[2] = {(cuuint64_t)K, (cuuint64_t)R};
  const cuuint64_t strides[1] = {(cuuint64_t)K * 2};
  const cuuint32_t box[2] = {64, box_rows};
  const cuuint32_t estr[2] = {1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void *>(base), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// What the two products of a call need.
struct Call {
  CUtensorMap in_w, in_x, out_w, out_h, out_h8;
  int dim, hidden;
  void *h, *y;
  Shared shared;
  bool tall;
  int64_t max_tiles;
  uint32_t *err;
  int num_sms;
  cudaStream_t stream;
};

template <int kTokens, bool kGate, bool kSmall, bool kSplit, bool kTall = false>
cudaError_t launch_product(const Call &c) {
  using X = EX<kTokens, kSmall, kTall>;
  static std::atomic<bool> attr[256];
  const auto kernel = experts_product_kernel<kTokens, kGate, kSmall, kSplit, kTall>;
  const cudaError_t e = set_smem_attr_once(kernel, X::SMEM_BYTES, attr);
  if (e != cudaSuccess) return e;
  const int cols = kGate ? c.hidden : c.dim, per_pair = (kGate ? 128 : 256) * X::SETS;
  const int64_t work = c.max_tiles * ((cols + per_pair - 1) / per_pair) * (kGate ? c.shared.splits : 1);
  const int64_t pairs = c.num_sms / 2 > 0 ? c.num_sms / 2 : 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(2 * (work < pairs ? work : pairs)));
  cfg.blockDim = dim3(kGate ? X::THREADS_GATE : X::THREADS);
  cfg.dynamicSmemBytes = X::SMEM_BYTES;
  cfg.stream = c.stream;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = 2;
  at[0].val.clusterDim.y = 1;
  at[0].val.clusterDim.z = 1;
  at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 2;
  const PlanOut &p = c.shared.plan;
  return cudaLaunchKernelEx(&cfg, kernel, kGate ? c.in_w : c.out_w, kGate ? c.in_x : c.out_h, c.out_h8,
                            (const int *)p.n_tiles, (const TokenTile *)p.tiles, (const int *)p.token,
                            kGate ? c.dim : c.hidden, cols, kGate ? c.h : c.y, c.shared, c.err);
}

template <int kTokens, bool kSmallGate, bool kSmallDown>
cudaError_t launch_products(const Call &c, int *launches) {
  cudaError_t e;
  if constexpr (kTokens == 256)
    e = c.tall                ? launch_product<kTokens, true, false, false, true>(c)
        : c.shared.splits > 1 ? launch_product<kTokens, true, false, true>(c)
                              : launch_product<kTokens, true, false, false>(c);
  else if constexpr (!kSmallGate)
    e = c.shared.splits > 1 ? launch_product<kTokens, true, false, true>(c) : launch_product<kTokens, true, false, false>(c);
  else
    e = launch_product<kTokens, true, true, false>(c);
  if (e != cudaSuccess) return e;
  ++*launches;
  e = launch_product<kTokens, false, kSmallDown, false>(c);
  if (e == cudaSuccess) ++*launches;
  return e;
}

cudaError_t launch_plan(const Call &c, int tile_tokens, int *launches) {
  static std::atomic<bool> attr[256];
  cudaError_t e = set_smem_attr_once(experts_plan_kernel, 34 * 1024 * 4, attr);
  if (e != cudaSuccess) return e;
  const Shared &s = c.shared;
  const unsigned blocks = s.n_slots > 1024 ? 8 : 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(blocks);
  cfg.blockDim = dim3(kPlanThreads);
  cfg.dynamicSmemBytes = (size_t)34 * s.n_experts * 4;
  cfg.stream = c.stream;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = blocks;
  at[0].val.clusterDim.y = 1;
  at[0].val.clusterDim.z = 1;
  at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 2;
  e = cudaLaunchKernelEx(&cfg, experts_plan_kernel, s, tile_tokens, c.err);
  if (e == cudaSuccess) ++*launches;
  return e;
}

cudaError_t launch_sum(const Call &c, int64_t n_tokens, int *launches) {
  const int64_t blocks = (n_tokens * (c.dim / 8) + 255) / 256, cap = (int64_t)c.num_sms * 32;
  cudaLaunchAttribute at;
  const cudaLaunchConfig_t cfg = programmatic_launch(dim3((unsigned)(blocks < cap ? blocks : cap)), dim3(256), 0, c.stream, &at);
  const cudaError_t e = cudaLaunchKernelEx(&cfg, experts_sum_kernel, (const __half *)c.y, (const float *)c.shared.scales, (const int *)c.shared.plan.row,
                                           c.shared.weights, n_tokens, c.shared.slots, c.dim, c.shared.out);
  if (e == cudaSuccess) ++*launches;
  return e;
}

}  // namespace

size_t experts_workspace_need(int64_t n_tokens, int slots, const dmel_expert_weights &w) {
  return layout(n_tokens, slots, w).total;
}

// A call of fewer tokens may need more: rows in fp32 up to kSmallSlots, partial sums of a split K. While a
// call is run the same way its bytes grow with the tokens, so the largest counts of each way are enough.
// From one way to the next the tiles grow or, with the same tiles, the splits get fewer: each way is
// one range of counts, and its end is found by halving.
size_t experts_workspace_bytes(int64_t n_tokens, int slots, const dmel_expert_weights &w) {
  auto same = [&](const Config &a, int64_t t) {
    const Config b = config(t, slots, w);
    return a.small == b.small && a.tile_tokens == b.tile_tokens && a.splits == b.splits;
  };
  size_t most = 0;
  for (int64_t first = 1; first <= n_tokens;) {
    const Config c = config(first, slots, w);
    int64_t last = first, beyond = n_tokens + 1;
    while (beyond - last > 1) {
      const int64_t mid = last + (beyond - last) / 2;
      if (same(c, mid)) last = mid;
      else beyond = mid;
    }
    const size_t need = experts_workspace_need(last, slots, w);
    if (need > most) most = need;
    first = last + 1;
  }
  return most;
}

cudaError_t launch_experts(const void *x, int64_t n_tokens, const int32_t *ids, const float *weights, int slots,
                           const dmel_expert_weights &w, void *out, void *workspace, uint32_t *err, int num_sms,
                           cudaStream_t stream, int *launches) {
  EncodeTiledFn enc = encode_tiled_fn();
  if (!enc) return cudaErrorNotSupported;
  const Config cf = config(n_tokens, slots, w);
  const Layout L = layout(n_tokens, slots, w);
  uint8_t *base = static_cast<uint8_t *>(workspace);
  const int n_slots = (int)(n_tokens * slots);
  Call c;
  c.dim = w.dim;
  c.hidden = w.hidden;
  c.h = base + L.h;
  c.y = base + L.y;
  c.err = err;
  c.num_sms = num_sms;
  c.stream = stream;
  Shared &s = c.shared;
  s.ids = ids;
  s.weights = weights;
  s.n_slots = n_slots;
  s.slots = slots;
  s.n_experts = w.n_experts;
  s.splits = cf.splits;
  s.n_counters = cf.n_counters;
  s.partial = reinterpret_cast<float *>(base + L.partial);
  s.counters = reinterpret_cast<int *>(base + L.counters);
  s.scales = reinterpret_cast<float *>(base + L.scales);
  s.out = static_cast<__nv_bfloat16 *>(out);
  s.plan.n_tiles = reinterpret_cast<int *>(base + L.n_tiles);
  s.plan.tiles = reinterpret_cast<TokenTile *>(base + L.tiles);
  s.plan.token = reinterpret_cast<int *>(base + L.token);
  s.plan.row = reinterpret_cast<int *>(base + L.row);
  if (!weight_map(&c.in_w, enc, w.w_in, w.n_experts, w.dim, 2 * (int64_t)w.hidden) ||
      !row_map(&c.in_x, enc, x, n_tokens, w.dim, 1) || !weight_map(&c.out_w, enc, w.w_out, w.n_experts, w.hidden, w.dim) ||
      !row_map(&c.out_h, enc, c.h, n_slots, w.hidden, 32) || !row_map(&c.out_h8, enc, c.h, n_slots, w.hidden, 8))
    return cudaErrorInvalidValue;
  c.max_tiles = cf.max_tiles;
  // tall tiles where they still make several rounds over the pairs, and K is 32 blocks or more
  c.tall = cf.max_tiles * ((w.hidden + 255) / 256) >= 3 * kPairs && w.dim >= 2048;
  cudaError_t e = cudaSuccess;
  // the splits' counters are cleared by the plan's kernel
  if (cf.small && cf.splits == 1) return launch_products<32, true, true>(c, launches);
  if ((e = launch_plan(c, cf.tile_tokens, launches)) != cudaSuccess) return e;
  if (cf.small) return launch_products<32, false, true>(c, launches);
  e = cf.tile_tokens == 32    ? launch_products<32, false, false>(c, launches)
      : cf.tile_tokens == 128 ? launch_products<128, false, false>(c, launches)
                              : launch_products<256, false, false>(c, launches);
  return e == cudaSuccess ? launch_sum(c, n_tokens, launches) : e;
}

}  // namespace dmel
