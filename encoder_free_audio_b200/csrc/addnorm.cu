// Residual addition and RMSNorm, with outputs in fp32, bf16 or e4m3 with scales ("Inside Inkling:
// Audio Design", Part 3 · Inference: the decoder's residual stream, whose branch outputs pass
// through the ShortConv):  s = x + r,  y = w s / sqrt(mean(s^2) + eps).
//
// Each value is read once and written once (two inputs, the stream and the normed row out): HBM
// bound. A block owns a row at a time; each thread keeps its 8-value pieces of the row in
// registers between the sum of squares and the scaling, so nothing is read twice but the weights
// (which stay in L1 and L2). A piece is 16 bytes of bf16 or 32 of fp32.
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "common.cuh"
#include "internal.h"

namespace dmel {
namespace {

constexpr float kE4m3Max = 448.0f;
constexpr float kMinAmax = 1e-30f;  // a block of zeros gets this / 448 as its scale, never zero

// 8 consecutive values. The inputs may be the outputs' buffers, so these are plain (coherent)
// accesses; the rows are not read again, so they need no place in L1.
__device__ __forceinline__ void load8(const float *p, float (&v)[8]) {
#pragma unroll
  for (int h = 0; h < 2; ++h)
    asm volatile("ld.global.L1::no_allocate.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v[4 * h]), "=f"(v[4 * h + 1]), "=f"(v[4 * h + 2]), "=f"(v[4 * h + 3])
                 : "l"(p + 4 * h)
                 : "memory");
}
__device__ __forceinline__ void unpack8(const uint32_t (&u)[4], float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(u[i] << 16);
    v[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ void load8(const __nv_bfloat16 *p, float (&v)[8]) {
  uint32_t u[4];
  asm volatile("ld.global.L1::no_allocate.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3])
               : "l"(p)
               : "memory");
  unpack8(u, v);
}
// (Plain loads: what a launch reads may be written until wait_for_predecessors, above which the
// compiler may take loads of read-only memory.)
__device__ __forceinline__ void weight8(const float *p, float (&v)[8]) {
  const float4 a = *reinterpret_cast<const float4 *>(p), b = *(reinterpret_cast<const float4 *>(p) + 1);
  v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
  v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}
__device__ __forceinline__ void weight8(const __nv_bfloat16 *p, float (&v)[8]) {
  const uint4 q = *reinterpret_cast<const uint4 *>(p);
  const uint32_t u[4] = {q.x, q.y, q.z, q.w};
  unpack8(u, v);
}
__device__ __forceinline__ void store8(float *p, const float (&v)[8]) {
  reinterpret_cast<float4 *>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
  reinterpret_cast<float4 *>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}
__device__ __forceinline__ void store8(__nv_bfloat16 *p, const float (&v)[8]) {
  uint32_t u[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
    u[i] = *reinterpret_cast<const uint32_t *>(&h);
  }
  *reinterpret_cast<uint4 *>(p) = make_uint4(u[0], u[1], u[2], u[3]);
}
// e4m3, nearest even, clamped to +-448 (NaN stays NaN)
__device__ __forceinline__ void store8(__nv_fp8_e4m3 *p, const float (&v)[8]) {
  uint32_t w[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(v[4 * h], v[4 * h + 1]), __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(v[4 * h + 2], v[4 * h + 3]), __NV_SATFINITE, __NV_E4M3);
    w[h] = lo | (hi << 16);
  }
  *reinterpret_cast<uint2 *>(p) = make_uint2(w[0], w[1]);
}

__device__ __forceinline__ float scale_of(float amax) { return fmaxf(amax, kMinAmax) * (1.0f / kE4m3Max); }

struct Add {
  __device__ float operator()(float a, float b) const { return a + b; }
};
struct Max {
  __device__ float operator()(float a, float b) const { return fmaxf(a, b); }
};

// One value per block over its `warps` warps, the same in every thread; `slots` is this
// reduction's own 32 floats of shared memory.
template <typename Op>
__device__ __forceinline__ float block_reduce(float v, float *slots, int warps, Op op) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = op(v, __shfl_xor_sync(0xffffffffu, v, o));
  if (warps == 1) return v;
  const int lane = threadIdx.x & 31;
  if (lane == 0) slots[threadIdx.x >> 5] = v;
  __syncthreads();
  v = lane < warps ? slots[lane] : 0.0f;  // (0 is neutral: sums and magnitudes)
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = op(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

// The e4m3 output's scales: `shift` is log2 of the pieces per block (2, 3, 4), or -1 for one scale per
// row; n_blocks scales per row.
struct Scales {
  float *p;
  int shift, n_blocks;
};

// V pieces of 8 values per thread: piece j of thread x holds columns 8 (j blockDim.x + x) and on.
// With kWarpRows a row takes one warp and a block has blockDim.y of them, without barriers; else it
// takes the block (and its address is the same in every thread, which saves registers).
// Two pieces and 32 registers: what bounds the rate is how many threads an SM holds (2,048) and
// then, for e4m3, the instructions per value. 24,000 x 6144 bf16 with the stream in and out: 183 us,
// 6.4 TB/s (64 registers 198 us, one piece 230 us); 12,800 rows into e4m3 by 128 columns: 100 us (179
// and 92 with the grids of launch_typed, launches under one another's ends).
// With no more rows than SMs one piece is the shorter way (8 rows: 2.4 us against 3.0), and for fp32
// rows, which have twice the bytes per piece, it is the faster one (1,601 x 5992: 25 us against 29).
template <typename T, typename TO, int V, bool kWarpRows>
__global__ void __launch_bounds__(1024, 2) add_rmsnorm_kernel(const T *x, const T *res, int64_t n_rows, int dim,
                                                              const T *w, float eps, T *res_out, TO *out,
                                                              Scales sc) {
  __shared__ float red[2][2][32];
  wait_for_predecessors();
  launch_dependents();
  const int warps = kWarpRows ? 1 : blockDim.x >> 5, pieces = dim >> 3;
  const float inv_dim = 1.0f / (float)dim;
  const int64_t step = (int64_t)gridDim.x * (kWarpRows ? blockDim.y : 1);
  int turn = 0;  // two sets of slots: a row's second use of one is a barrier away from its first
  for (int64_t row = kWarpRows ? (int64_t)blockIdx.x * blockDim.y + threadIdx.y : blockIdx.x; row < n_rows;
       row += step, turn ^= 1) {
    const T *xr = x + row * dim;
    float s[V][8];
    float ss = 0.0f;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const uint32_t p = j * blockDim.x + threadIdx.x;
      if (p < (uint32_t)pieces) {
        load8(xr + 8u * p, s[j]);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) s[j][i] = 0.0f;
      }
    }
    if (res) {
      const T *rr = res + row * dim;
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const uint32_t p = j * blockDim.x + threadIdx.x;
        if (p < (uint32_t)pieces) {
          float r[8];
          load8(rr + 8u * p, r);
#pragma unroll
          for (int i = 0; i < 8; ++i) s[j][i] += r[i];
        }
      }
    }
#pragma unroll
    for (int j = 0; j < V; ++j) {
#pragma unroll
      for (int i = 0; i < 8; ++i) ss = fmaf(s[j][i], s[j][i], ss);
    }
    if (sizeof(T) == 2 && V == 2 && !kWarpRows && row + step < n_rows) {  // the block's next row into L2
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const uint32_t p = j * blockDim.x + threadIdx.x;
        if (p < (uint32_t)pieces && (p & 7u) == 0) {  // a line of 128 bytes
          asm volatile("prefetch.global.L2 [%0];" ::"l"(x + (row + step) * dim + 8u * p));
          if (res) asm volatile("prefetch.global.L2 [%0];" ::"l"(res + (row + step) * dim + 8u * p));
        }
      }
    }
    if (res_out) {
      T *ro = res_out + row * dim;
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const uint32_t p = j * blockDim.x + threadIdx.x;
        if (p < (uint32_t)pieces) store8(ro + 8u * p, s[j]);
      }
    }
    ss = block_reduce(ss, red[turn][0], warps, Add());
    float rstd = rsqrtf(fmaf(ss, inv_dim, eps));  // (within 2 ulps, on the special-function unit)
    if (sizeof(TO) == 1 && rstd > 1e4f) {  // rstd / scale would leave fp32's range: rstd first
#pragma unroll
      for (int j = 0; j < V; ++j) {
#pragma unroll
        for (int i = 0; i < 8; ++i) s[j][i] *= rstd;
      }
      rstd = 1.0f;
    }
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const uint32_t p = j * blockDim.x + threadIdx.x;
      if (p < (uint32_t)pieces) {
        float g[8];
        weight8(w + 8u * p, g);
#pragma unroll
        for (int i = 0; i < 8; ++i) s[j][i] *= g[i];
      }
    }
    float mult[V];  // what w s is multiplied by
#pragma unroll
    for (int j = 0; j < V; ++j) mult[j] = rstd;
    if (sizeof(TO) == 1) {
      // largest magnitude of each piece, then of its block: 4, 8 or 16 neighbouring threads (the
      // block's pieces, since blockDim.x is a multiple of 32), or the whole row. fmaxf drops NaN.
      // w s / sqrt(..) / scale is a product with an approximate reciprocal of the scale, which is far
      // from the ends of fp32's range: a few ulps before a rounding to 4 bits, and the block's
      // largest value, within those of 448, becomes 448.
      float top[V];
#pragma unroll
      for (int j = 0; j < V; ++j) {
        top[j] = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) top[j] = fmaxf(top[j], fabsf(s[j][i]));
      }
      if (sc.shift < 0) {
        float m = top[0];
#pragma unroll
        for (int j = 1; j < V; ++j) m = fmaxf(m, top[j]);
        const float scale = scale_of(rstd * block_reduce(m, red[turn][1], warps, Max()));
#pragma unroll
        for (int j = 0; j < V; ++j) mult[j] = rstd * __fdividef(1.0f, scale);
        if (threadIdx.x == 0) sc.p[row] = scale;
      } else {
        float *row_scales = sc.p + row * sc.n_blocks;
#pragma unroll
        for (int j = 0; j < V; ++j) {
          top[j] = fmaxf(top[j], __shfl_xor_sync(0xffffffffu, top[j], 1));
          top[j] = fmaxf(top[j], __shfl_xor_sync(0xffffffffu, top[j], 2));
          if (sc.shift > 2) top[j] = fmaxf(top[j], __shfl_xor_sync(0xffffffffu, top[j], 4));
          if (sc.shift > 3) top[j] = fmaxf(top[j], __shfl_xor_sync(0xffffffffu, top[j], 8));
          const uint32_t p = j * blockDim.x + threadIdx.x;
          const float scale = scale_of(rstd * top[j]);
          mult[j] = rstd * __fdividef(1.0f, scale);
          if (p < (uint32_t)pieces && (p & ((1u << sc.shift) - 1u)) == 0) row_scales[p >> sc.shift] = scale;
        }
      }
    }
    TO *orow = out + row * dim;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const uint32_t p = j * blockDim.x + threadIdx.x;
      if (p < (uint32_t)pieces) {
#pragma unroll
        for (int i = 0; i < 8; ++i) s[j][i] *= mult[j];
        store8(orow + 8u * p, s[j]);
      }
    }
  }
}

template <typename T, typename TO>
cudaError_t launch_typed(const void *x, const void *res, int64_t n_rows, int dim, const void *w, float eps,
                         void *res_out, void *out, Scales sc, int num_sms, cudaStream_t stream) {
  const int pieces = dim / 8;
  // (A row of 32 pieces or less has one per lane of its warp either way: 24,000 x 256 bf16 take 8.4 us,
  // with an empty second piece 10.6.)
  const bool two = pieces > 1024 || (sizeof(T) == 2 && n_rows > num_sms && pieces > 32);
  const int threads = ((two ? (pieces + 1) / 2 : pieces) + 31) / 32 * 32;
  const bool warp_rows = threads == 32;
  const dim3 block(threads, warp_rows ? 8 : 1);
  const int64_t blocks = (n_rows + block.y - 1) / block.y;
  // A grid as large as the SMs hold at a time, two or eight times: a block's rows follow one another,
  // and those of bf16 ask L2 for the next while they are at one. 12,800 x 6144 into e4m3: 93 us twice,
  // 94 eight times, 101 with 64 blocks per SM and no asking; 24,000 x 6144 bf16: 198, 181 and 185 us.
  // fp32 rows, which do not gain by asking (6,000 x 6144 into e4m3: 78, 82 with it): twice for e4m3 (84
  // us with 64), else 64 (97 us, twice 99).
  const int resident = 2048 / (threads * block.y), e4m3 = sizeof(TO) == 1;
  const int per_sm = warp_rows ? 64 : sizeof(T) == 2 ? (e4m3 ? 2 : 8) * resident : e4m3 && !two ? 2 * resident : 64;
  const int64_t cap = (int64_t)num_sms * per_sm;
  const unsigned grid = (unsigned)(blocks < cap ? blocks : cap);
  const T *xt = static_cast<const T *>(x), *rt = static_cast<const T *>(res), *wt = static_cast<const T *>(w);
  T *so = static_cast<T *>(res_out);
  TO *ot = static_cast<TO *>(out);
  cudaLaunchAttribute at;
  const cudaLaunchConfig_t cfg = programmatic_launch(grid, block, 0, stream, &at);
#define DMEL_NORM(V, ROWS) \
  return cudaLaunchKernelEx(&cfg, add_rmsnorm_kernel<T, TO, V, ROWS>, xt, rt, n_rows, dim, wt, eps, so, ot, sc)
  if constexpr (sizeof(T) == 2) {  // (fp32 rows of two pieces are wider than a warp)
    if (warp_rows && two) DMEL_NORM(2, true);
  }
  if (warp_rows) DMEL_NORM(1, true);
  else if (two) DMEL_NORM(2, false);
  else DMEL_NORM(1, false);
#undef DMEL_NORM
}

}  // namespace

cudaError_t launch_add_rmsnorm(const void *x, const void *residual, int64_t n_rows, int dim, dmel_dtype dtype,
                               const void *w, float eps, void *residual_out, void *out, dmel_dtype out_dtype,
                               float *scales, int scale_block, int num_sms, cudaStream_t stream, int *launches) {
  Scales sc;
  sc.p = scales;
  sc.shift = scale_block == 0 ? -1 : scale_block == 32 ? 2 : scale_block == 64 ? 3 : 4;
  sc.n_blocks = scale_block == 0 ? 1 : (dim + scale_block - 1) / scale_block;
#define DMEL_NORM(T, TO) launch_typed<T, TO>(x, residual, n_rows, dim, w, eps, residual_out, out, sc, num_sms, stream)
  cudaError_t e;
  if (dtype == DMEL_BF16)
    e = out_dtype == DMEL_E4M3   ? DMEL_NORM(__nv_bfloat16, __nv_fp8_e4m3)
        : out_dtype == DMEL_BF16 ? DMEL_NORM(__nv_bfloat16, __nv_bfloat16)
                                 : DMEL_NORM(__nv_bfloat16, float);
  else
    e = out_dtype == DMEL_E4M3   ? DMEL_NORM(float, __nv_fp8_e4m3)
        : out_dtype == DMEL_BF16 ? DMEL_NORM(float, __nv_bfloat16)
                                 : DMEL_NORM(float, float);
#undef DMEL_NORM
  if (e == cudaSuccess) ++*launches;
  return e;
}

}  // namespace dmel
