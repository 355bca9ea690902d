// The teacher-forced training loss on corrected logits, with its gradient.
//
// Row i with target t, weight w_i and logits c: lse = log sum_v exp(c_v),
// nll_i = lse - c_t, loss = sum_i w_i nll_i / N with N = sum_i w_i (mean) or 1
// (sum), d loss / d c_v = w_i / N (exp(c_v - lse) - [v = t]).
#include <cmath>

#include "common.cuh"
#include "kernels.h"

namespace dspark {

namespace {

constexpr int kThreads = 512;

// The scratch of one call (DSPARK_LOSS_SCRATCH_BYTES).
struct LossScratch {
  double inv_n;  // 1 / N, 0 where N is 0
  uint32_t done;
};

// A row counts when its target is not the ignored one, lies in the vocabulary
// and its weight is not zero.
__device__ __forceinline__ bool live_row(const LossArgs& a, int64_t i, int64_t* target, float* weight) {
  const int64_t t = a.targets[i];
  const float w = a.weights ? a.weights[i] : 1.0f;
  *target = t;
  *weight = w;
  return t != a.ignore_index && t >= 0 && t < a.vocab && w != 0.0f;
}

__device__ __forceinline__ double block_sum(double x, double* parts) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  if ((threadIdx.x & 31) == 0) parts[threadIdx.x >> 5] = x;
  __syncthreads();
  double s = 0.0;
  for (int w = 0; w < (int)(blockDim.x >> 5); ++w) s += parts[w];
  __syncthreads();
  return s;
}

// N, the status of the targets and a cleared counter, before the rows.
__global__ void __launch_bounds__(kThreads) loss_total_kernel(LossArgs a) {
  __shared__ double parts[kThreads / 32];
  double s = 0.0;
  bool bad = false;
  for (int64_t i = threadIdx.x; i < a.rows; i += blockDim.x) {
    int64_t t;
    float w;
    if (live_row(a, i, &t, &w)) s += (double)w;
    if (t != a.ignore_index && (t < 0 || t >= a.vocab)) bad = true;
  }
  s = block_sum(s, parts);
  if (bad) report_status(a.status, DSPARK_STATUS_TOKEN_RANGE);
  if (threadIdx.x == 0) {
    LossScratch* sc = static_cast<LossScratch*>(a.scratch);
    sc->inv_n = a.mean ? (s != 0.0 ? 1.0 / s : 0.0) : 1.0;
    sc->done = 0u;
  }
}

// One CTA per row, two passes over it: the running maximum and sum, then the
// gradient.
template <typename T>
__global__ void __launch_bounds__(kThreads) loss_rows_kernel(LossArgs a) {
  __shared__ float part_m[kThreads / 32], part_s[kThreads / 32];
  const int64_t i = blockIdx.x;
  int64_t t;
  float w;
  const bool live = live_row(a, i, &t, &w);
  const T* c = static_cast<const T*>(a.logits) + i * a.vocab;
  T* g = a.grad ? static_cast<T*>(a.grad) + i * a.vocab : nullptr;
  if (!live) {
    if (threadIdx.x == 0) a.row_losses[i] = 0.0f;
    if (g)
      for (int64_t v = threadIdx.x; v < a.vocab; v += kThreads) g[v] = from_f32<T>(0.0f);
    return;
  }
  float m = -INFINITY, s = 0.0f;
  for (int64_t v = threadIdx.x; v < a.vocab; v += kThreads) {
    const float x = to_f32(c[v]);
    if (x > m) {
      s = s * __expf(m - x) + 1.0f;
      m = x;
    } else if (x != -INFINITY) {
      s += __expf(x - m);  // NaN passes into the sum
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const float om = __shfl_xor_sync(0xffffffffu, m, o), os = __shfl_xor_sync(0xffffffffu, s, o);
    const float nm = fmaxf(m, om);
    s = (m == nm ? s : s * __expf(m - nm)) + (om == nm ? os : os * __expf(om - nm));
    m = nm;
  }
  if ((threadIdx.x & 31) == 0) {
    part_m[threadIdx.x >> 5] = m;
    part_s[threadIdx.x >> 5] = s;
  }
  __syncthreads();
  m = part_m[0];
  for (int k = 1; k < kThreads / 32; ++k) m = fmaxf(m, part_m[k]);
  s = 0.0f;
  for (int k = 0; k < kThreads / 32; ++k) s += part_m[k] == m ? part_s[k] : part_s[k] * __expf(part_m[k] - m);
  if (isinf(m)) s = NAN;  // +inf somewhere, or -inf everywhere
  const LossScratch* sc = static_cast<const LossScratch*>(a.scratch);
  const float scale = (float)((double)w * sc->inv_n), inv = 1.0f / s;
  const float xt = to_f32(c[t]);
  __syncthreads();  // the target's logit is read before an in-place gradient overwrites it
  if (threadIdx.x == 0) a.row_losses[i] = logf(s) - (xt - m);
  if (!g) return;
  for (int64_t v = threadIdx.x; v < a.vocab; v += kThreads) {
    const float p = __expf(to_f32(c[v]) - m) * inv;
    g[v] = from_f32<T>((v == t ? p - 1.0f : p) * scale);
  }
}

// loss = sum_i w_i nll_i / N over the live rows, in row order per thread.
__global__ void __launch_bounds__(kThreads) loss_sum_kernel(LossArgs a) {
  __shared__ double parts[kThreads / 32];
  double s = 0.0;
  for (int64_t i = threadIdx.x; i < a.rows; i += blockDim.x) {
    int64_t t;
    float w;
    if (live_row(a, i, &t, &w)) s += (double)w * (double)a.row_losses[i];
  }
  s = block_sum(s, parts);
  if (threadIdx.x == 0) *a.loss = (float)(s * static_cast<const LossScratch*>(a.scratch)->inv_n);
}

}  // namespace

cudaError_t launch_loss(const LossArgs& a, int logits_dtype, int num_sms, cudaStream_t s) {
  (void)num_sms;
  static_assert(sizeof(LossScratch) <= DSPARK_LOSS_SCRATCH_BYTES, "the scratch holds the call's state");
  if (a.rows > 0x7fffffffll) return cudaErrorInvalidConfiguration;
  loss_total_kernel<<<1, kThreads, 0, s>>>(a);
  note_launch();
  if (a.rows > 0) {
    if (logits_dtype == DSPARK_DTYPE_FP32)
      loss_rows_kernel<float><<<(unsigned)a.rows, kThreads, 0, s>>>(a);
    else
      loss_rows_kernel<__nv_bfloat16><<<(unsigned)a.rows, kThreads, 0, s>>>(a);
    note_launch();
  }
  loss_sum_kernel<<<1, kThreads, 0, s>>>(a);
  note_launch();
  return cudaGetLastError();
}

}  // namespace dspark
