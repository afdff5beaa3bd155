// Routing of tokens to experts ("Inside Inkling: Audio Design", Part 3 · Inference: a sigmoid
// router over 256 routed experts with 6 chosen per token, 2 shared experts always, and a joint
// normalisation over the chosen and the shared).
//
// One warp per token: lane l holds experts l, l + 32, ... in registers, so a row is read once,
// coalesced, and no value leaves the warp before the ids and weights are written. With many tokens
// the kernel is bound by its instructions, not by the row's 1 KB: each lane orders its experts by a
// network of comparisons on values whose last bits give way to the expert's place, and top_k rounds
// take the largest head of the 32 lanes with one reduction each. (8 lanes per token with their best
// 16 merged, so that four tokens share the rounds, needs more registers than fit beside enough warps:
// 48 us for 24,000 tokens of 256 experts, where this takes 21.)
//
// The order is that of 64-bit arithmetic, although the scores are fp32 and cut short: the lanes check
// that each winner is above the next by more than the two can be off. A token where one is not (about
// one in five hundred of ordinary logits) has the winners and what is near the last of them ordered
// by their scores in fp64, one candidate a lane: 1.5 us with sigmoids, 2.7 with a softmax, whose sum
// is wanted too. All experts are chosen again in fp64 (6 to 8 us) only where two groups are that near
// or more than 32 candidates are. So the time goes by the logits: 12,800 bf16 rows of 256 in 8 groups
// without a bias take 25 us where they are normal draws and 68 where all are zeros, as padding is;
// 24,000 fp32 rows without groups or bias 17 and 34.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math_constants.h>
#include <stdint.h>

#include "common.cuh"
#include "internal.h"

namespace dmel {
namespace {

constexpr int kWarps = 4;  // per block
constexpr unsigned kAll = 0xffffffffu;
constexpr float kNone = -__builtin_huge_valf();  // "not to be chosen"

// (Plain loads: what a launch reads may be written until wait_for_predecessors, above which the
// compiler may take loads of read-only memory.)
__device__ __forceinline__ float logit(const float *p) { return *p; }
__device__ __forceinline__ float logit(const __nv_bfloat16 *p) { return __bfloat162float(*p); }

// A logit as the choice sees it: NaN is -inf (never chosen; fmaxf drops it), +inf the largest finite
// value.
__device__ __forceinline__ float clean(float l) { return fminf(fmaxf(l, kNone), 3.402823466e38f); }

// What a kernel is given of a dmel_router, with the experts per group and 2^20 / that, rounded up
// (e / per = e * inv_per >> 20 for e < 1024), and the shared memory per warp.
struct Settings {
  dmel_router r;
  int per, inv_per, warp_doubles;
};

// A key: an fp32 value whose last bits give way to the place i of N (a power of two), such that equal
// values put lower places first. Keys are compared as floats.
template <int N>
__device__ __forceinline__ float key_of(float v, int i) {
  const uint32_t u = __float_as_uint(fminf(v, 3.402823466e38f) + 0.0f);  // (no infinity, no -0)
  const uint32_t low = u >> 31 ? (uint32_t)i : (uint32_t)(N - 1 - i);
  return v > kNone ? __uint_as_float((u & ~(uint32_t)(N - 1)) | low) : kNone;
}
template <int N>
__device__ __forceinline__ int place_of(float k) {
  const uint32_t u = __float_as_uint(k), low = u & (N - 1);
  return (int)(u >> 31 ? low : N - 1 - low);
}
template <int N>
__device__ __forceinline__ float value_of(float k) {  // cut towards -inf, by less than N units
  const uint32_t u = __float_as_uint(k);
  return __uint_as_float(u >> 31 ? u | (N - 1) : u & ~(uint32_t)(N - 1));
}

// Bounds on the fp32 scores' errors, from ex2.approx's 2^-22 and rcp.approx's 2^-23 of the result and
// the roundings around them. A sigmoid's: 3e-7 (the exponential's error counts s (1 - s) at most). A
// softmax's, with its sum of up to 1,056 terms by pairs: 1.8e-6 of the token's largest score, 1 / z.
constexpr float kSigmoidOff = 3.5e-7f, kSoftmaxOff = 2e-6f;

// Two choice values' keys, a above b, stand as in 64-bit arithmetic where they are further apart than
// twice the scores' error (0 for logits) and this share of the larger: the rounding of the sums with
// the bias, and what key_of<N> may have cut off b.
__host__ __device__ constexpr float cut_of(int N) { return (N + 2) * 1.2e-7f; }

// exp and 1 / x on the special-function unit (a few ulps, results below the normal range zero).
__device__ __forceinline__ float fast_exp(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x * 1.4426950408889634f));
  return y;
}
__device__ __forceinline__ float fast_rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

template <typename F>
__device__ __forceinline__ F warp_sum(F v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
  return v;
}

// Descending order by a network of comparisons (Batcher's odd-even merge sort; N a power of two).
template <int N>
__device__ __forceinline__ void sort_down(float (&v)[N]) {
#pragma unroll
  for (int p = 1; p < N; p <<= 1) {
#pragma unroll
    for (int k = p; k > 0; k >>= 1) {
#pragma unroll
      for (int j = k % p; j + k < N; j += 2 * k) {
#pragma unroll
        for (int i = 0; i < k; ++i) {
          if (i + j + k < N && (i + j) / (2 * p) == (i + j + k) / (2 * p)) {
            const float a = v[i + j], b = v[i + j + k];
            v[i + j] = fmaxf(a, b);
            v[i + j + k] = fminf(a, b);
          }
        }
      }
    }
  }
}

// Sum by pairs: an error of log2 N roundings.
template <int N>
__device__ __forceinline__ float pair_sum(float (&v)[N]) {
#pragma unroll
  for (int k = N / 2; k > 0; k >>= 1) {
#pragma unroll
    for (int i = 0; i < k; ++i) v[i] += v[i + k];
  }
  return v[0];
}

// Lanes that walk a group together: a power of two, and up to 32 groups fit the warp.
__device__ __forceinline__ int lanes_per_group(int groups) {
  return groups > 16 ? 1 : groups > 8 ? 2 : groups > 4 ? 4 : groups > 2 ? 8 : 16;
}

// The groups kept, a bit each. A group is rated by the sum of its two largest values (one where
// there is only one). The values lie in shared memory, group g's from v + g (per + lanes_per_group):
// that far apart, the lanes that walk the groups use different banks. *worst, *best: the lowest
// rating kept, the highest left out. *size (where asked for): the largest sum of the magnitudes of a
// group's two values, which bounds what their roundings move its rating by; the rating itself does
// not, since a bias of each sign may cancel in it.
template <typename F>
__device__ __forceinline__ unsigned keep_groups(const F *v, const Settings &q, F *worst, F *best, F *size = nullptr) {
  const int groups = q.r.n_groups, lane = threadIdx.x & 31, share = lanes_per_group(groups), mine = lane / share;
  F m1 = kNone, m2 = kNone;
  if (mine < groups) {
    const F *p = v + mine * (q.per + share);
#pragma unroll 4
    for (int j = lane & (share - 1); j < q.per; j += share) {
      const F x = p[j];
      m2 = max(m2, min(m1, x));
      m1 = max(m1, x);
    }
  }
  __syncwarp();
  for (int o = share >> 1; o > 0; o >>= 1) {
    const F o1 = __shfl_xor_sync(kAll, m1, o), o2 = __shfl_xor_sync(kAll, m2, o);
    m2 = max(max(m2, o2), min(m1, o1));
    m1 = max(m1, o1);
  }
  F rated = __shfl_sync(kAll, m2 > kNone ? m1 + m2 : m1, (lane * share) & 31);  // group `lane`'s
  if (lane >= groups) rated = kNone;
  int before = 0;
  for (int h = 0; h < groups; ++h) {
    const F o = __shfl_sync(kAll, rated, h);
    before += o > rated || (o == rated && h < lane);
  }
  const bool in = lane < groups && before < q.r.topk_groups;
  F lo = in ? rated : -(F)kNone, hi = in ? (F)kNone : rated;
  *worst = -warp_max(-lo);
  *best = warp_max(hi);
  if (size) *size = warp_max((m1 > kNone ? abs(m1) : (F)0) + (m2 > kNone ? abs(m2) : (F)0));
  return __ballot_sync(kAll, in);
}

// A double as an unsigned number of the same order.
__device__ __forceinline__ unsigned long long order_of(double v) {
  const unsigned long long u = (unsigned long long)__double_as_longlong(v + 0.0);
  return u >> 63 ? ~u : u | (1ull << 63);
}

// The choice in fp64: the id of slot `lane`, -1 for none. `top` is the token's largest logit, v the
// warp's shared memory. Apart from the kernel, since few tokens come here; written for a short way
// through, since the last of them may end the launch.
template <typename T, int EPL>
__device__ __noinline__ int choose_fp64(const T *row, const float *bias, const Settings &q, float top, double *v) {
  const dmel_router &r = q.r;
  const int lane = threadIdx.x & 31, E = r.n_experts;
  const bool softmax = r.scoring == DMEL_ROUTE_SOFTMAX;
  constexpr int STEP = EPL < 8 ? EPL : 8;
  double c[EPL], z = 0.0;
#pragma unroll STEP
  for (int i = 0; i < EPL; ++i) {
    const int e = lane + 32 * i;
    const double l = e < E ? (double)clean(logit(row + e)) : kNone;
    c[i] = l;
    if (bias || r.n_groups > 1) {
      const double x = exp(softmax ? l - (double)top : -l);
      c[i] = softmax ? x : 1.0 / (1.0 + x);
      z += x;
    }
  }
  if (bias || r.n_groups > 1) {
    if (softmax) {
      for (int e = E + lane; e < E + r.n_shared; e += 32) z += exp((double)clean(logit(row + e)) - (double)top);
      z = 1.0 / warp_sum(z);
    }
#pragma unroll STEP
    for (int i = 0; i < EPL; ++i) {
      const int e = lane + 32 * i;
      double x = softmax ? c[i] * z : c[i];
      if (bias && e < E) x += (double)bias[e];
      c[i] = e < E && clean(logit(row + e)) > kNone && x == x ? x : (double)kNone;
    }
  }
  if (r.n_groups > 1) {
    const int share = lanes_per_group(r.n_groups);
#pragma unroll STEP
    for (int i = 0; i < EPL; ++i)
      if (lane + 32 * i < E) v[lane + 32 * i + (((lane + 32 * i) * q.inv_per) >> 20) * share] = c[i];
    __syncwarp();
    double worst, best;
    const unsigned kept = keep_groups(v, q, &worst, &best);
#pragma unroll STEP
    for (int i = 0; i < EPL; ++i) {
      const int e = lane + 32 * i;
      if (!((kept >> ((e * q.inv_per) >> 20)) & 1u)) c[i] = kNone;
      else if (!bias && c[i] > kNone) c[i] = (double)clean(logit(row + e));
    }
  }
  int my_id = -1;
  for (int k = 0; k < r.top_k; ++k) {
    double m = kNone;
    int at = 0;
#pragma unroll
    for (int i = 0; i < EPL; ++i)
      if (c[i] > m) { m = c[i]; at = i; }
    // the largest of the warp, its high word first, then the lowest index among equals
    const unsigned long long u = order_of(m);
    const uint32_t hi = __reduce_max_sync(kAll, (uint32_t)(u >> 32));
    const uint32_t lo = __reduce_max_sync(kAll, (uint32_t)(u >> 32) == hi ? (uint32_t)u : 0u);
    const bool held = u == ((unsigned long long)hi << 32 | lo);
    const int idx = (int)__reduce_min_sync(kAll, held && m > kNone ? (uint32_t)(lane + 32 * at) : 0x7fffffffu);
    if (idx == 0x7fffffff) break;  // nothing left
    if (lane == k) my_id = idx;
    if (lane == (idx & 31)) {
#pragma unroll
      for (int i = 0; i < EPL; ++i)
        if (i == idx >> 5) c[i] = kNone;
    }
  }
  return my_id;
}

// An expert's score in fp32, of its logit l; z: the softmax's sum.
__device__ __forceinline__ float score_of(bool sigmoid, float l, float top, float inv_z) {
  return sigmoid ? fast_rcp(1.0f + fast_exp(-l)) : __fmul_rn(fast_exp(l - top), inv_z);
}

// The experts chosen in fp32 (lane k: slot k's id) where `close` has a bit for each slot whose key is
// near the next one's (the last slot's: the next that is not chosen), put right: the id of slot
// `lane`, or kTooMany in all lanes. `top` is the token's largest logit, z the softmax's sum, `least` the
// last slot's value; values a >= b are near within off + cut max(|a|, |b|). Two experts alike are a tie,
// which the keys settle by index; with the last of the chosen they do where no other expert is near it
// and not alike. Else the chosen, with all that are near the last of them, are ordered as logits, or
// with a bias as scores in fp64, one candidate a lane. Short code rather than overlapped: an SM that
// comes here rarely waits for the instructions.
constexpr int kTooMany = -2;  // candidates for the lanes of a warp

template <typename T>
__device__ __noinline__ int settle(const T *row, const float *bias, const Settings &q, float top, float z, unsigned kept,
                                   float least, float off, float cut, unsigned close, int id, int *list) {
  const dmel_router &r = q.r;
  const int lane = threadIdx.x & 31, E = r.n_experts, K = r.top_k;
  const bool softmax = r.scoring == DMEL_ROUTE_SOFTMAX;
  auto alike = [&](int e, int f) {
    return clean(logit(row + e)) == clean(logit(row + f)) && (!bias || bias[e] == bias[f]);
  };
  const int next_id = __shfl_down_sync(kAll, id, 1), least_id = __shfl_sync(kAll, id, K - 1);
  bool open = lane < K - 1 && ((close >> lane) & 1u) && !alike(id, next_id);
  int n = K;
  const bool edge = (close >> (K - 1)) & 1u;
  if (edge) {
    n = 0;
    const float inv_z = fast_rcp(z);
#pragma unroll 1
    for (int e0 = 0; e0 < E; e0 += 32) {
      const int e = min(e0 + lane, E - 1);
      const float l = clean(logit(row + e));
      float v = bias ? __fadd_rn(score_of(!softmax, l, top, inv_z), bias[e]) : l;
      bool in = e == e0 + lane && l > kNone && v > kNone && ((kept >> ((e * q.inv_per) >> 20)) & 1u);
      v = fminf(v, 3.402823466e38f);
      const float gap = least - v, wide = off + cut * fmaxf(fabsf(least), fabsf(v));
      in = in && !(gap > wide);
      if (in && !(-gap > wide) && !alike(e, least_id)) open = true;
      const unsigned all = __ballot_sync(kAll, in);
      const int place = n + __popc(all & ((1u << lane) - 1u));
      if (in && place < 32) list[place] = e;
      n += __popc(all);
    }
  }
  if (!__any_sync(kAll, open)) return id;
  if (n > 32) return kTooMany;
  if (edge) {
    __syncwarp();
    id = lane < n ? list[lane] : -1;
    __syncwarp();  // (read before the next token's are written)
  }
  double x = id >= 0 ? (double)clean(logit(row + id)) : (double)kNone;
  if (bias) {
    const int end = softmax ? E + r.n_shared : 0;
    double own = 0.0, sum = 0.0;
#pragma unroll 1
    for (int e = lane - 32; e < end; e += 32) {  // first the candidate, then the token's sum
      const double l = e < 0 ? x : (double)clean(logit(row + e));
      const double a = exp(softmax ? l - (double)top : -l);
      if (e < 0) own = a;
      else sum += a;
    }
    __syncwarp();
    sum = softmax ? warp_sum(sum) : 1.0 + own;
    x = (softmax ? own : 1.0) / sum + (double)bias[max(id, 0)];
  }
  int before = 0;
  for (int j = 0; j < n; ++j) {
    const double o = __shfl_sync(kAll, x, j);
    const int other = __shfl_sync(kAll, id, j);
    before += other >= 0 && (o > x || (o == x && other < id));
  }
  int mine = -1;
  for (int j = 0; j < n; ++j) {
    const int place = __shfl_sync(kAll, before, j), other = __shfl_sync(kAll, id, j);
    if (place == lane && other >= 0) mine = other;
  }
  return mine;
}

// Registers for a lane's experts: 64 hold 8 of them beside a few spilled values (24,000 tokens of 256
// experts: 21.3 us, with 72 registers 23.3); 32 want 128 (8,192 tokens of 1,024 experts: 58 us, with 64
// 78; in 16 groups 63 and 121).
constexpr int blocks_per_sm(int epl) { return epl >= 32 ? 4 : epl >= 16 ? 6 : 8; }

// kScored: the choice compares scores (a bias, or groups), else the logits themselves.
template <typename T, int EPL, bool kScored, bool kGroups>
__global__ void __launch_bounds__(32 * kWarps, blocks_per_sm(EPL)) route_kernel(const T *logits, int64_t n_tokens,
                                                            const float *bias, const __grid_constant__ Settings q,
                                                            int32_t *ids, float *weights) {
  wait_for_predecessors();
  launch_dependents();
  const dmel_router &r = q.r;
  const int lane = threadIdx.x & 31, E = r.n_experts, S = r.n_shared, K = r.top_k;
  const int cols = E + S, slots = K + S;
  const unsigned lanes_below = (1u << lane) - 1u;
  const bool sigmoid = r.scoring == DMEL_ROUTE_SIGMOID;
  constexpr float kCut = cut_of(EPL);
  __shared__ int list[kWarps][32];  // settle's
  extern __shared__ double smem[];  // with groups: a token's values per warp
  double *const wide = smem + (threadIdx.x >> 5) * q.warp_doubles;
  const int64_t step = (int64_t)gridDim.x * kWarps;
  for (int64_t t = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5); t < n_tokens; t += step) {
    const T *row = logits + t * cols;
    auto at = [&](int e) { return clean(logit(row + e)); };
    float l[EPL];
#pragma unroll
    for (int i = 0; i < EPL; ++i) l[i] = lane + 32 * i < E ? logit(row + lane + 32 * i) : kNone;
    const float ls = lane < S ? at(E + lane) : kNone;  // shared expert `lane`
#pragma unroll
    for (int i = 0; i < EPL; ++i) l[i] = clean(l[i]);
    float top = 0.0f, z = 1.0f;  // softmax: the largest logit, and the sum of exp(l - top)
    if (!sigmoid) {
      top = ls;
#pragma unroll
      for (int i = 0; i < EPL; ++i) top = fmaxf(top, l[i]);
      top = warp_max(top);
      if (!(top > kNone)) top = 0.0f;
      if (kScored || !r.renormalise) {
        float x[EPL];
#pragma unroll
        for (int i = 0; i < EPL; ++i) x[i] = fast_exp(l[i] - top);
        z = warp_sum(pair_sum<EPL>(x) + fast_exp(ls - top));
      }
    }
    // what the choice compares, -inf for what is not to be chosen
    bool unsure = false;
    unsigned kept = ~0u;  // groups
    float v[EPL];
    float off = 0.0f;  // the scores' error
    if (kScored) {
      const float inv_z = fast_rcp(z);
      off = sigmoid ? kSigmoidOff : kSoftmaxOff * inv_z;
#pragma unroll
      for (int i = 0; i < EPL; ++i) {
        const float s = score_of(sigmoid, l[i], top, inv_z);
        v[i] = l[i] > kNone ? s : kNone;
      }
      if (bias) {
#pragma unroll
        for (int i = 0; i < EPL; ++i)
          if (lane + 32 * i < E) v[i] += bias[lane + 32 * i];
      }
    } else {
#pragma unroll
      for (int i = 0; i < EPL; ++i) v[i] = l[i];
    }
    if (kGroups) {
      float *const narrow = reinterpret_cast<float *>(wide);
      const int share = lanes_per_group(r.n_groups);
#pragma unroll
      for (int i = 0; i < EPL; ++i) {
        const int e = lane + 32 * i;
        if (e < E) narrow[e + ((e * q.inv_per) >> 20) * share] = fmaxf(v[i], kNone);  // (NaN: -inf)
      }
      __syncwarp();
      float worst, best, size;
      kept = keep_groups(narrow, q, &worst, &best, &size);
      // Two ratings, each of two values that are off by a score's error and half a unit of their own, and
      // a sum off by half a unit of itself: 4 off + 4 2^-24 size.
      unsure = best > kNone && !(worst - best > 4.0f * off + cut_of(1) * size);
#pragma unroll
      for (int i = 0; i < EPL; ++i) {
        const float x = bias ? v[i] : l[i];
        v[i] = (kept >> (((lane + 32 * i) * q.inv_per) >> 20)) & 1u ? x : kNone;
      }
      __syncwarp();  // (read before the next token's values are written)
    }
    float key[EPL];
#pragma unroll
    for (int i = 0; i < EPL; ++i) key[i] = key_of<EPL>(v[i], i);
    sort_down<EPL>(key);
    // top_k rounds: the largest head, the lowest lane among equals; slot k's key and lanes stay in lane k
    float mine = kNone;
    unsigned holders = 1;
    for (int k = 0; k < K; ++k) {
      const float best = warp_max(key[0]);
      if (!(best > kNone)) break;  // nothing left
      const bool held = key[0] == best;
      const unsigned heads = __ballot_sync(kAll, held);
      if (lane == k) {
        mine = best;
        holders = heads;
      }
      if (held && !(heads & lanes_below)) {
#pragma unroll
        for (int i = 0; i + 1 < EPL; ++i) key[i] = key[i + 1];
        key[EPL - 1] = kNone;
      }
    }
    int my_id = mine > kNone ? __ffs(holders) - 1 + 32 * place_of<EPL>(mine) : -1;  // of slot `lane`
    // keys that may stand the other way round in 64 bits
    const float rest = warp_max(key[0]), below = __shfl_down_sync(kAll, mine, 1);
    const float next = lane == K - 1 ? rest : below, a = value_of<EPL>(mine), b = value_of<EPL>(next);
    const float wide_off = bias ? 2.0f * off : 0.0f;
    const bool near = lane < K && next > kNone && !(a - b > wide_off + kCut * fmaxf(fabsf(a), fabsf(b)));
    const unsigned close = __ballot_sync(kAll, near);
    if (close)
      my_id = settle(row, bias, q, top, z, kept, __shfl_sync(kAll, a, K - 1), wide_off, kCut, close, my_id,
                     list[threadIdx.x >> 5]);
    if (unsure || my_id == kTooMany) my_id = choose_fp64<T, EPL>(row, bias, q, top, wide);
    float x = lane < K && my_id >= 0 ? at(my_id) : kNone;  // slot `lane`'s logit
    if (lane >= K) my_id = -1;
    if (S > 0) {  // shared experts in slots K .. K + S - 1
      const float s = __shfl_sync(kAll, ls, (lane - K) & 31);
      if (lane >= K && lane < slots && s > kNone) {
        my_id = E + lane - K;
        x = s;
      }
    }
    // weights. Renormalised: s / sum(s) from values scaled by exp(-m), m the largest chosen logit
    // (sigmoid: where it is negative), so that scores too small for a float keep their ratios. All in
    // fp32, with expf (a unit or two) and a division by approximate reciprocal (two units) of a number
    // in (1, 2]: the weights are fp32, and what they order is settled above.
    float m = sigmoid ? 0.0f : top;
    if (r.renormalise) {
      m = warp_max(x);
      if (sigmoid) m = fminf(m, 0.0f);
    }
    float w = 0.0f;
    if (x > kNone) {
      w = expf(sigmoid ? fminf(x, 0.0f) - m : x - m);
      if (sigmoid) w = __fdividef(w, 1.0f + expf(-fabsf(x)));
    }
    if (r.renormalise) z = warp_sum(w);
    if (lane < slots) {
      ids[t * slots + lane] = my_id;
      weights[t * slots + lane] = z > 0.0f ? w / z * r.scale : 0.0f;
    }
  }
}

template <typename T>
cudaError_t launch_typed(const void *logits, int64_t n_tokens, const float *bias, const dmel_router &r, int32_t *ids,
                         float *weights, int num_sms, cudaStream_t stream) {
  const int E = r.n_experts;
  Settings q;
  q.r = r;
  q.per = E / r.n_groups;
  q.inv_per = ((1 << 20) + q.per - 1) / q.per;
  q.warp_doubles = r.n_groups > 1 ? E + 32 : 0;  // groups and the lanes per group: at most 32 together
  const T *lt = static_cast<const T *>(logits);
  const size_t smem = (size_t)kWarps * q.warp_doubles * sizeof(double);
  const int64_t blocks = (n_tokens + kWarps - 1) / kWarps, cap = (int64_t)num_sms * 64;
  const unsigned grid = (unsigned)(blocks < cap ? blocks : cap);
  cudaLaunchAttribute at;
  const cudaLaunchConfig_t cfg = programmatic_launch(grid, dim3(32 * kWarps), smem, stream, &at);
#define DMEL_ROUTE(EPL)                                                                                      \
  return r.n_groups > 1 ? cudaLaunchKernelEx(&cfg, route_kernel<T, EPL, true, true>, lt, n_tokens, bias, q,   \
                                             ids, weights)                                                    \
         : bias         ? cudaLaunchKernelEx(&cfg, route_kernel<T, EPL, true, false>, lt, n_tokens, bias, q,  \
                                             ids, weights)                                                    \
                        : cudaLaunchKernelEx(&cfg, route_kernel<T, EPL, false, false>, lt, n_tokens, bias, q, \
                                             ids, weights)
  // a lane's experts, to the next power of two (8,192 tokens of 384 experts: 21 us, as if 1,024: 49)
  if (E <= 64) DMEL_ROUTE(2);
  else if (E <= 128) DMEL_ROUTE(4);
  else if (E <= 256) DMEL_ROUTE(8);
  else if (E <= 512) DMEL_ROUTE(16);
  else DMEL_ROUTE(32);
#undef DMEL_ROUTE
}

}  // namespace

cudaError_t launch_route(const void *logits, int64_t n_tokens, dmel_dtype dtype, const float *bias,
                         const dmel_router &r, int32_t *ids, float *weights, int num_sms, cudaStream_t stream,
                         int *launches) {
  const cudaError_t e = dtype == DMEL_BF16
                            ? launch_typed<__nv_bfloat16>(logits, n_tokens, bias, r, ids, weights, num_sms, stream)
                            : launch_typed<float>(logits, n_tokens, bias, r, ids, weights, num_sms, stream);
  if (e == cudaSuccess) ++*launches;
  return e;
}

}  // namespace dmel
