// Routing of tokens to experts ("Inside Inkling: Audio Design", Part 3 · Inference: a sigmoid
// router over 256 routed experts with 6 chosen per token, 2 shared experts always, and a joint
// normalisation over the chosen and the shared).
//
// One warp per token: lane l holds the logits of experts l, l + 32, ... in registers, so a row is
// read once, coalesced, and no value leaves the warp before the ids and weights are written. The
// choice is top_k rounds of a warp-wide maximum over (value, lower index).
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math_constants.h>
#include <stdint.h>

#include "common.cuh"
#include "internal.h"

namespace dmel {
namespace {

constexpr int kWarps = 4;  // tokens per block
constexpr unsigned kAll = 0xffffffffu;

__device__ __forceinline__ float logit(const float *p) { return __ldg(p); }
__device__ __forceinline__ float logit(const __nv_bfloat16 *p) { return __bfloat162float(*p); }

// A logit as the choice sees it: NaN is -inf (never chosen), +inf the largest finite value.
__device__ __forceinline__ float clean(float l) { return l == l ? fminf(l, 3.402823466e38f) : -CUDART_INF_F; }

// Largest value of the warp and the lowest index that holds it (idx differs between lanes).
__device__ __forceinline__ void warp_best(double &v, int &idx) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const double ov = __shfl_xor_sync(kAll, v, o);
    const int oi = __shfl_xor_sync(kAll, idx, o);
    if (ov > v || (ov == v && oi < idx)) { v = ov; idx = oi; }
  }
}

template <typename T, int EPL>
__global__ void __launch_bounds__(32 * kWarps) route_kernel(const T *__restrict__ logits, int64_t n_tokens,
                                                            const float *__restrict__ bias, dmel_router r,
                                                            int32_t *__restrict__ ids, float *__restrict__ weights) {
  const int lane = threadIdx.x & 31;
  const int E = r.n_experts, S = r.n_shared, K = r.top_k;
  const int cols = E + S, slots = K + S;
  extern __shared__ double group_smem[];  // [kWarps][E] choice values, with groups
  const int64_t warps = (int64_t)gridDim.x * kWarps;
  for (int64_t t = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5); t < n_tokens; t += warps) {
    const T *row = logits + t * cols;
    float l[EPL];
    float top = -CUDART_INF_F;
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      const int e = lane + 32 * i;
      l[i] = e < E ? clean(logit(row + e)) : -CUDART_INF_F;
      top = fmaxf(top, l[i]);
    }
    const float ls = lane < S ? clean(logit(row + E + lane)) : -CUDART_INF_F;  // shared expert `lane`
    top = fmaxf(top, ls);
    double z = 0.0;  // softmax: sum of exp(l - top) over every logit of the token
    if (r.scoring == DMEL_ROUTE_SOFTMAX) {
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(kAll, top, o));
      if (top > -CUDART_INF_F) {
#pragma unroll
        for (int i = 0; i < EPL; ++i) z += exp((double)l[i] - top);
        z += exp((double)ls - top);
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) z += __shfl_xor_sync(kAll, z, o);
    }
    auto score = [&](float x) -> double {
      if (!(x > -CUDART_INF_F)) return 0.0;
      return r.scoring == DMEL_ROUTE_SIGMOID ? 1.0 / (1.0 + exp(-(double)x)) : exp((double)x - top) / z;
    };
    // c[i]: what the choice compares. Without a bias the scores rise with the logits, so the
    // logits themselves are compared (exactly); the groups' ratings need the scores.
    double c[EPL];
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      const int e = lane + 32 * i;
      const float b = bias && e < E ? __ldg(bias + e) : 0.0f;
      c[i] = l[i] > -CUDART_INF_F && b == b ? (bias || r.n_groups > 1 ? score(l[i]) + (double)b : (double)l[i])
                                            : -CUDART_INF;
    }
    if (r.n_groups > 1) {
      const int per = E / r.n_groups;
      double *cs = group_smem + (threadIdx.x >> 5) * E;
#pragma unroll
      for (int i = 0; i < EPL; ++i)
        if (lane + 32 * i < E) cs[lane + 32 * i] = c[i];
      __syncwarp();
      double rated = -CUDART_INF;
      if (lane < r.n_groups) {
        double m1 = -CUDART_INF, m2 = -CUDART_INF;
        for (int j = 0; j < per; ++j) {
          const double v = cs[lane * per + j];
          if (v > m1) { m2 = m1; m1 = v; } else if (v > m2) { m2 = v; }
        }
        rated = m2 > -CUDART_INF ? m1 + m2 : m1;
      }
      __syncwarp();
      int before = 0;  // groups better than this lane's
      for (int g = 0; g < r.n_groups; ++g) {
        const double o = __shfl_sync(kAll, rated, g);
        before += o > rated || (o == rated && g < lane);
      }
      const unsigned kept = __ballot_sync(kAll, lane < r.n_groups && before < r.topk_groups);
#pragma unroll
      for (int i = 0; i < EPL; ++i) {
        const int e = lane + 32 * i;
        if (e < E && !((kept >> (e / per)) & 1u)) c[i] = -CUDART_INF;
        else if (!bias && c[i] > -CUDART_INF) c[i] = (double)l[i];
      }
    }
    int my_id = -1;                 // slot `lane`
    float my_l = -CUDART_INF_F;
    for (int k = 0; k < K; ++k) {
      double v = -CUDART_INF;
      int idx = INT32_MAX;
      float lv = -CUDART_INF_F;
#pragma unroll
      for (int i = 0; i < EPL; ++i)
        if (c[i] > v) { v = c[i]; idx = lane + 32 * i; lv = l[i]; }
      const int mine = idx;
      warp_best(v, idx);
      if (!(v > -CUDART_INF)) break;  // nothing left (the same in every lane)
      const int owner = idx & 31;
      const float won = __shfl_sync(kAll, lv, owner);
      if (lane == owner && mine == idx) {
#pragma unroll
        for (int i = 0; i < EPL; ++i)
          if (lane + 32 * i == idx) c[i] = -CUDART_INF;
      }
      if (lane == k) { my_id = idx; my_l = won; }
    }
    {  // shared experts in slots K .. K + S - 1
      const float sl = __shfl_sync(kAll, ls, lane >= K ? lane - K : 0);
      if (lane >= K && lane < slots && sl > -CUDART_INF_F) {
        my_id = E + lane - K;
        my_l = sl;
      }
    }
    double wgt = my_id >= 0 ? score(my_l) : 0.0;
    if (r.renormalise) {
      // s / sum(s) from values scaled by exp(-m), m the largest chosen logit (sigmoid: where it is
      // negative), so that scores too small for a float keep their ratios
      float m = my_l;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(kAll, m, o));
      if (my_id >= 0) {
        if (r.scoring == DMEL_ROUTE_SOFTMAX) {
          wgt = exp((double)my_l - m);
        } else {
          const double shift = m < 0.0f ? (double)m : 0.0;
          wgt = (my_l > 0.0f ? 1.0 : exp((double)my_l - shift)) / (1.0 + exp(-fabs((double)my_l)));
        }
      }
      double sum = wgt;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(kAll, sum, o);
      wgt = sum > 0.0 ? wgt / sum : 0.0;
    }
    if (lane < slots) {
      ids[t * slots + lane] = my_id;
      weights[t * slots + lane] = (float)(wgt * (double)r.scale);
    }
  }
}

template <typename T>
cudaError_t launch_typed(const void *logits, int64_t n_tokens, const float *bias, const dmel_router &r, int32_t *ids,
                         float *weights, int num_sms, cudaStream_t stream) {
  const int64_t blocks = (n_tokens + kWarps - 1) / kWarps, cap = (int64_t)num_sms * 64;
  const unsigned grid = (unsigned)(blocks < cap ? blocks : cap);
  const size_t smem = r.n_groups > 1 ? (size_t)kWarps * r.n_experts * 8 : 0;
  const T *lt = static_cast<const T *>(logits);
#define DMEL_ROUTE(EPL) route_kernel<T, EPL><<<grid, 32 * kWarps, smem, stream>>>(lt, n_tokens, bias, r, ids, weights)
  const int epl = (r.n_experts + 31) / 32;
  if (epl <= 1) DMEL_ROUTE(1);
  else if (epl <= 2) DMEL_ROUTE(2);
  else if (epl <= 4) DMEL_ROUTE(4);
  else if (epl <= 8) DMEL_ROUTE(8);
  else if (epl <= 16) DMEL_ROUTE(16);
  else DMEL_ROUTE(32);
#undef DMEL_ROUTE
  return cudaGetLastError();
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
