// The global norm over many gradient tensors, and clipping by it:
// norm = sqrt(sum over tensors of sum g^2), out = g min(1, max / (norm + 1e-6)).
//
// The tensors are cut into pieces of at most kPieceBytes; a piece is one
// record of the plan. One kernel sums squares and leaves a double for each
// CTA, the next adds those in one order and scales.
#include <cmath>

#include "common.cuh"
#include "kernels.h"

namespace dspark {

namespace {

constexpr int kThreads = 256;
constexpr int kCtasPerSm = 4;

__device__ __forceinline__ double block_sum(double x, double* parts) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  if ((threadIdx.x & 31) == 0) parts[threadIdx.x >> 5] = x;
  __syncthreads();
  double s = 0.0;
  for (int w = 0; w < kThreads / 32; ++w) s += parts[w];
  __syncthreads();
  return s;
}

template <typename T>
__device__ __forceinline__ double squares(const T* g, int64_t n) {
  double s = 0.0;
  for (int64_t i = threadIdx.x; i < n; i += kThreads) {
    const double x = (double)to_f32(g[i]);
    s += x * x;
  }
  return s;
}

__global__ void __launch_bounds__(kThreads) clip_norm_kernel(ClipArgs a) {
  __shared__ double parts[kThreads / 32];
  double s = 0.0;
  for (int64_t p = blockIdx.x; p < a.pieces; p += gridDim.x) {
    const dspark_markov_clip_piece q = a.plan[p];
    s += q.dtype == DSPARK_DTYPE_FP32 ? squares(static_cast<const float*>(q.grad), q.count)
                                      : squares(static_cast<const __nv_bfloat16*>(q.grad), q.count);
  }
  s = block_sum(s, parts);
  if (threadIdx.x == 0) a.partials[blockIdx.x] = s;
}

template <typename T>
__device__ __forceinline__ void scale_piece(const T* g, T* out, int64_t n, float c) {
  for (int64_t i = threadIdx.x; i < n; i += kThreads) out[i] = from_f32<T>(to_f32(g[i]) * c);
}

__global__ void __launch_bounds__(kThreads) clip_scale_kernel(ClipArgs a) {
  __shared__ double parts[kThreads / 32];
  double s = 0.0;
  for (int i = threadIdx.x; i < (int)gridDim.x; i += kThreads) s += a.partials[i];
  const double norm = sqrt(block_sum(s, parts));
  const double ratio = (double)a.max_norm / (norm + 1e-6);
  const float c = ratio > 1.0 ? 1.0f : (float)ratio;  // NaN stays NaN
  if (blockIdx.x == 0 && threadIdx.x == 0) *a.norm = (float)norm;
  for (int64_t p = blockIdx.x; p < a.pieces; p += gridDim.x) {
    const dspark_markov_clip_piece q = a.plan[p];
    if (c == 1.0f && q.out == q.grad) continue;
    if (q.dtype == DSPARK_DTYPE_FP32)
      scale_piece(static_cast<const float*>(q.grad), static_cast<float*>(q.out), q.count, c);
    else
      scale_piece(static_cast<const __nv_bfloat16*>(q.grad), static_cast<__nv_bfloat16*>(q.out), q.count, c);
  }
}

}  // namespace

cudaError_t launch_clip(const ClipArgs& a, int num_sms, cudaStream_t s) {
  int64_t grid = (int64_t)num_sms * kCtasPerSm;
  if (grid > DSPARK_CLIP_MAX_PARTIALS) grid = DSPARK_CLIP_MAX_PARTIALS;
  if (grid > a.pieces) grid = a.pieces > 0 ? a.pieces : 1;
  clip_norm_kernel<<<(unsigned)grid, kThreads, 0, s>>>(a);
  note_launch();
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  clip_scale_kernel<<<(unsigned)grid, kThreads, 0, s>>>(a);
  note_launch();
  return cudaGetLastError();
}

}  // namespace dspark
