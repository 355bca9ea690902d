// The teacher-forced training loss on corrected logits, with its gradient.
//
// Row i with target t, weight w_i and logits c: lse = log sum_v exp(c_v),
// nll_i = lse - c_t, loss = sum_i w_i nll_i / N with N = sum_i w_i (mean) or 1
// (sum), d loss / d c_v = w_i / N (exp(c_v - lse) - [v = t]).
//
// The sum and the gradient both need the whole row, so a kernel that streams
// reads it twice. Here a cluster of CTAs holds a row in its registers (a
// 129280-id bf16 row is 252 KB, more than one SM's shared memory but an eighth
// of a four-SM register file): each logit is read once and each gradient
// written once, 4 bytes per bf16 logit, and that traffic is the bound.
//
// In units of log2: a warp's largest logit m_w gives its reference point
// r_w = m_w log2 e (rounded) and s_w = sum 2^(c log2 e - r_w) over its logits.
// The pairs (m_w, s_w) of all warps of the cluster meet in every CTA's shared
// memory behind one barrier; r = max r_w, S = sum s_w 2^(r_w - r),
// nll = ln 2 (log2 S - (c_t log2 e - r)), softmax_v = 2^(c_v log2 e - r) / S.
// The rounding of r is common to all of them and cancels.
#include <cmath>

#include "common.cuh"
#include "kernels.h"

namespace dspark {

namespace {

constexpr int kMaxThreads = 512;
constexpr int kMaxCluster = 16;
constexpr int kMaxWarps = kMaxThreads / 32;
constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.693147180559945309417f;

// 2^x by the hardware approximation (relative error 2^-22; 0 below 2^-126).
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// The factor from logits to the exponents' units for a row whose largest logit
// is m. Where m log2 e could overflow, two logits that differ at all do so by
// far more than any exponent, so a quarter of them serves as well (and stays
// finite): equal logits have equal exponents, all others vanish.
__device__ __forceinline__ float unit_for(float m) { return fabsf(m) > 0x1p126f ? 0.25f : kLog2e; }

// A row counts when its target is not the ignored one, lies in the vocabulary
// and its weight is not zero.
__device__ __forceinline__ bool live_row(const LossArgs& a, int64_t i, int64_t* target, float* weight) {
  const int64_t t = a.targets[i];
  const float w = a.weights ? a.weights[i] : 1.0f;
  *target = t;
  *weight = w;
  return t != a.ignore_index && t >= 0 && t < a.vocab && w != 0.0f;
}

// The sum over the block in one order; every thread gets it.
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

// 1 / N, 0 where N is 0. Every CTA forms it (12 bytes a row from L2, once per
// CTA), which costs less than a launch before the rows.
__device__ double inverse_total(const LossArgs& a, double* parts, bool report) {
  if (!a.mean && !report) return 1.0;
  double s = 0.0;
  bool bad = false;
  for (int64_t i = threadIdx.x; i < a.rows; i += blockDim.x) {
    int64_t t;
    float w;
    if (live_row(a, i, &t, &w)) s += (double)w;
    if (t != a.ignore_index && (t < 0 || t >= a.vocab)) bad = true;
  }
  if (bad && report) report_status(a.status, DSPARK_STATUS_TOKEN_RANGE);
  if (!a.mean) return 1.0;
  s = block_sum(s, parts);
  return s != 0.0 ? 1.0 / s : 0.0;
}

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
  uint32_t n;
  asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(n));
  return n;
}
__device__ __forceinline__ void cluster_barrier() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// Stores a pair at the same shared address of CTA `rank` of the cluster.
__device__ __forceinline__ void store_remote(float2* p, uint32_t rank, float2 v) {
  const uint32_t local = static_cast<uint32_t>(__cvta_generic_to_shared(p));
  uint32_t remote;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(local), "r"(rank));
  asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(remote), "f"(v.x), "f"(v.y) : "memory");
}

// 16 bytes of a row.
template <typename T>
struct Vectors;
template <>
struct Vectors<float> {
  static constexpr int kE = 4;
  static constexpr uint32_t kFill = 0xff800000u;  // -inf
  static __device__ __forceinline__ float get(const uint4& r, int e) {
    return __uint_as_float(e == 0 ? r.x : e == 1 ? r.y : e == 2 ? r.z : r.w);
  }
  static __device__ __forceinline__ float max_of(const uint4& r) {
    return fmaxf(fmaxf(get(r, 0), get(r, 1)), fmaxf(get(r, 2), get(r, 3)));
  }
  static __device__ __forceinline__ uint4 pack(const float* g) {
    return make_uint4(__float_as_uint(g[0]), __float_as_uint(g[1]), __float_as_uint(g[2]), __float_as_uint(g[3]));
  }
};
template <>
struct Vectors<__nv_bfloat16> {
  static constexpr int kE = 8;
  static constexpr uint32_t kFill = 0xff80ff80u;
  static __device__ __forceinline__ uint32_t word(const uint4& r, int i) {
    return i == 0 ? r.x : i == 1 ? r.y : i == 2 ? r.z : r.w;
  }
  static __device__ __forceinline__ float get(const uint4& r, int e) {
    const uint32_t w = word(r, e >> 1);
    return __uint_as_float((e & 1) ? (w & 0xffff0000u) : (w << 16));
  }
  static __device__ __forceinline__ __nv_bfloat162 pair(uint32_t w) {
    return *reinterpret_cast<const __nv_bfloat162*>(&w);
  }
  static __device__ __forceinline__ float max_of(const uint4& r) {
    const __nv_bfloat162 m = __hmax2(__hmax2(pair(r.x), pair(r.y)), __hmax2(pair(r.z), pair(r.w)));
    return fmaxf(__low2float(m), __high2float(m));
  }
  static __device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
  }
  static __device__ __forceinline__ uint4 pack(const float* g) {
    return make_uint4(pack2(g[0], g[1]), pack2(g[2], g[3]), pack2(g[4], g[5]), pack2(g[6], g[7]));
  }
};

// Where a row's 16-byte vectors lie: `head` elements before the first 16-byte
// address, `vecs` vectors, `tail` elements behind them. Every row of a
// vocabulary of whole vectors is all vectors; a row of odd length starts
// anywhere. The elements at the edges, fewer than two vectors', go to one
// thread each of the cluster's first CTA.
template <typename T>
struct RowShape {
  int head, vecs, edges;
  __device__ __forceinline__ RowShape(const T* row, int vocab) {
    constexpr int kE = Vectors<T>::kE;
    const int past = (int)((reinterpret_cast<uintptr_t>(row) / sizeof(T)) % kE);
    head = min(past ? kE - past : 0, vocab);
    vecs = (vocab - head) / kE;
    edges = vocab - vecs * kE;
  }
  // The id of edge element k.
  __device__ __forceinline__ int edge(int k) const { return k < head ? k : k + vecs * Vectors<T>::kE; }
};

__device__ __forceinline__ float edge_value(const float* p) { return __ldcs(p); }
__device__ __forceinline__ float edge_value(const __nv_bfloat16* p) { return __bfloat162float(*p); }

// Rows for one cluster each, a persistent grid walking them; NV vectors of the
// row in each thread's registers. While a row's gradient is written, each
// vector's registers already load the next row's.
// SAME: the gradient's rows start at the same offset from a 16-byte address as
// the logits' (in place, or any vocabulary of whole vectors), so that a vector
// read is a vector written; otherwise gradients are written one by one.
template <typename T, int NV, bool SAME>
__global__ void __launch_bounds__(kMaxThreads, 2) loss_rows_kernel(LossArgs a) {
  constexpr int kE = Vectors<T>::kE;
  __shared__ double sums[kMaxWarps];
  __shared__ float2 parts[2][kMaxCluster * kMaxWarps];
  const int warps = blockDim.x >> 5, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t ranks = cluster_size(), rank = cluster_rank();
  const int64_t step = gridDim.x / ranks;
  const int vocab = (int)a.vocab, threads = (int)blockDim.x;
  const int j0 = (int)rank * threads * NV + (int)threadIdx.x;  // this thread's vectors: j0 + n threads
  const T* logits = static_cast<const T*>(a.logits);
  T* grads = static_cast<T*>(a.grad);

  uint4 raw[NV];
  float edge = -INFINITY, xt = 0.0f;  // this thread's edge element; the target's logit (thread 0)
  auto load = [&](int64_t row, int n) {
    const T* c = logits + row * vocab;
    const RowShape<T> shape(c, vocab);
    const int j = j0 + n * threads;
    raw[n] = j < shape.vecs ? __ldcs(reinterpret_cast<const uint4*>(c + shape.head) + j)
                            : make_uint4(Vectors<T>::kFill, Vectors<T>::kFill, Vectors<T>::kFill, Vectors<T>::kFill);
  };
  auto load_singles = [&](int64_t row, int64_t t) {
    const T* c = logits + row * vocab;
    const RowShape<T> shape(c, vocab);
    edge = -INFINITY;
    if (rank == 0) {
      if ((int)threadIdx.x < shape.edges) edge = edge_value(c + shape.edge((int)threadIdx.x));
      if (threadIdx.x == 0) xt = edge_value(c + t);
    }
  };

  int64_t i = blockIdx.x / ranks;
  int64_t t = 0;
  float w = 0.0f;
  bool live = i < a.rows && live_row(a, i, &t, &w);
  if (live) {
#pragma unroll
    for (int n = 0; n < NV; ++n) load(i, n);
    load_singles(i, t);
  }
  const double inv_n = inverse_total(a, sums, false);
  if (ranks > 1) cluster_barrier();  // every CTA's shared memory is there

  int parity = 0;
  while (i < a.rows) {
    const int64_t next = i + step;
    int64_t next_t = 0;
    float next_w = 0.0f;
    const bool next_live = next < a.rows && live_row(a, next, &next_t, &next_w);
    const RowShape<T> shape(logits + i * vocab, vocab);
    T* g = grads + i * vocab;
    if (!live) {
      if (rank == 0 && threadIdx.x == 0) a.row_losses[i] = 0.0f;
      if (rank == 0 && grads && (int)threadIdx.x < shape.edges) g[shape.edge((int)threadIdx.x)] = from_f32<T>(0.0f);
#pragma unroll
      for (int n = 0; n < NV; ++n) {
        const int j = j0 + n * threads;
        if (grads && j < shape.vecs) {
          if (SAME)
            __stcs(reinterpret_cast<uint4*>(g + shape.head) + j, make_uint4(0u, 0u, 0u, 0u));
          else
            for (int e = 0; e < kE; ++e) g[shape.head + j * kE + e] = from_f32<T>(0.0f);
        }
        if (next_live) load(next, n);
      }
      if (next_live) load_singles(next, next_t);
    } else {
      float m = edge;
#pragma unroll
      for (int n = 0; n < NV; ++n) m = fmaxf(m, Vectors<T>::max_of(raw[n]));
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
      // A warp of -inf alone (or NaN) takes 0 as its reference and sums zeros (or NaN).
      float unit = m == -INFINITY ? kLog2e : unit_for(m);
      float ref = m == -INFINITY ? 0.0f : m * unit;
      float s = ex2(fmaf(edge, unit, -ref));
#pragma unroll
      for (int n = 0; n < NV; ++n)
#pragma unroll
        for (int e = 0; e < kE; ++e) s += ex2(fmaf(Vectors<T>::get(raw[n], e), unit, -ref));
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
      // The warp's pair into every CTA. The buffer written two rows ago was
      // read before the last barrier.
      if (lane < (int)ranks)
        store_remote(&parts[parity][rank * warps + warp], (uint32_t)lane, make_float2(m, s));
      if (ranks > 1)
        cluster_barrier();
      else
        __syncthreads();
      const int pairs = (int)ranks * warps;
      m = -INFINITY;
      for (int k = lane; k < pairs; k += 32) m = fmaxf(m, parts[parity][k].x);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
      unit = unit_for(m);
      ref = m * unit;
      float sum = 0.0f;
      for (int k = lane; k < pairs; k += 32) {
        const float2 q = parts[parity][k];
        // A warp in other units lies infinitely far below.
        if (q.x == -INFINITY)
          sum += q.y;
        else if (unit_for(q.x) == unit)
          sum += q.y * ex2(q.x * unit - ref);
        else
          sum += q.y * 0.0f;  // NaN stays
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      parity ^= 1;
      if (isinf(m)) sum = NAN;  // +inf somewhere, or -inf everywhere
      const float scale = (float)((double)w * inv_n);
      const float factor = scale / sum;
      if (rank == 0 && threadIdx.x == 0)  // in plain units where the exponents' would overflow
        a.row_losses[i] = unit == kLog2e && fabsf(xt) <= 0x1p126f ? kLn2 * (log2f(sum) - fmaf(xt, unit, -ref)) : logf(sum) + (m - xt);
      // The target's place among the vectors (negative or past them: an edge).
      const int at = (int)t - shape.head;
      const int tj = at >= 0 ? at / kE : -1, te = at % kE;
      if (grads && rank == 0 && (int)threadIdx.x < shape.edges) {
        const int v = shape.edge((int)threadIdx.x);
        const float p = ex2(fmaf(edge, unit, -ref)) * factor;
        g[v] = from_f32<T>(v == (int)t ? p - scale : p);
      }
#pragma unroll
      for (int n = 0; n < NV; ++n) {
        const int j = j0 + n * threads;
        if (grads && j < shape.vecs) {
          float p[kE];
#pragma unroll
          for (int e = 0; e < kE; ++e) p[e] = ex2(fmaf(Vectors<T>::get(raw[n], e), unit, -ref)) * factor;
          if (j == tj) {
#pragma unroll
            for (int e = 0; e < kE; ++e)
              if (e == te) p[e] -= scale;
          }
          if (SAME) {
            __stcs(reinterpret_cast<uint4*>(g + shape.head) + j, Vectors<T>::pack(p));
          } else {
#pragma unroll
            for (int e = 0; e < kE; ++e) g[shape.head + j * kE + e] = from_f32<T>(p[e]);
          }
        }
        if (next_live) load(next, n);
      }
      if (next_live) load_singles(next, next_t);
    }
    i = next;
    t = next_t;
    w = next_w;
    live = next_live;
  }
}

// Rows longer than a cluster's registers: one CTA per row reads it twice.
template <typename T>
__global__ void __launch_bounds__(kMaxThreads) loss_long_rows_kernel(LossArgs a) {
  __shared__ double sums[kMaxWarps];
  __shared__ float2 parts[kMaxWarps];
  const double inv_n = inverse_total(a, sums, false);
  for (int64_t i = blockIdx.x; i < a.rows; i += gridDim.x) {
    int64_t t;
    float w;
    const bool live = live_row(a, i, &t, &w);
    const T* c = static_cast<const T*>(a.logits) + i * a.vocab;
    T* g = a.grad ? static_cast<T*>(a.grad) + i * a.vocab : nullptr;
    if (!live) {
      if (threadIdx.x == 0) a.row_losses[i] = 0.0f;
      for (int64_t v = threadIdx.x; g && v < a.vocab; v += blockDim.x) g[v] = from_f32<T>(0.0f);
      continue;
    }
    float m = -INFINITY, s = 0.0f;
    for (int64_t v = threadIdx.x; v < a.vocab; v += blockDim.x) {
      const float x = to_f32(c[v]);
      if (x > m) {
        s = s * ex2((m - x) * kLog2e);
        m = x;
      }
      if (x != -INFINITY) s += ex2((x - m) * kLog2e);  // NaN passes into the sum
    }
    for (int o = 16; o > 0; o >>= 1) {
      const float m2 = __shfl_xor_sync(0xffffffffu, m, o), s2 = __shfl_xor_sync(0xffffffffu, s, o);
      const float top = fmaxf(m, m2);
      s = (m == top ? s : s * ex2((m - top) * kLog2e)) + (m2 == top ? s2 : s2 * ex2((m2 - top) * kLog2e));
      m = top;
    }
    __syncthreads();
    if ((threadIdx.x & 31) == 0) parts[threadIdx.x >> 5] = make_float2(m, s);
    __syncthreads();
    m = -INFINITY;
    for (int k = 0; k < (int)(blockDim.x >> 5); ++k) m = fmaxf(m, parts[k].x);
    s = 0.0f;
    for (int k = 0; k < (int)(blockDim.x >> 5); ++k)
      s += parts[k].x == m ? parts[k].y : parts[k].y * ex2((parts[k].x - m) * kLog2e);
    if (isinf(m)) s = NAN;
    const float scale = (float)((double)w * inv_n), factor = scale / s;
    const float xt = to_f32(c[t]);
    __syncthreads();  // the target's logit is read before an in-place gradient overwrites it
    if (threadIdx.x == 0) a.row_losses[i] = logf(s) + (m - xt);
    for (int64_t v = threadIdx.x; g && v < a.vocab; v += blockDim.x) {
      const float p = ex2((to_f32(c[v]) - m) * kLog2e) * factor;
      g[v] = from_f32<T>(v == t ? p - scale : p);
    }
  }
}

// loss = sum_i w_i nll_i / N over the live rows, and the status of the targets.
__global__ void __launch_bounds__(kMaxThreads) loss_sum_kernel(LossArgs a) {
  __shared__ double sums[kMaxWarps];
  const double inv_n = inverse_total(a, sums, true);
  double s = 0.0;
  for (int64_t i = threadIdx.x; i < a.rows; i += blockDim.x) {
    int64_t t;
    float w;
    if (live_row(a, i, &t, &w)) s += (double)w * (double)a.row_losses[i];
  }
  s = block_sum(s, sums);
  if (threadIdx.x == 0) *a.loss = (float)(s * inv_n);
}

struct LossPlan {
  int cluster, threads, vectors;  // vectors per thread
};

// The cluster that holds a row of `vecs` vectors, or cluster 0 where none does.
LossPlan plan_loss(int64_t rows, int64_t vecs, int num_sms) {
  LossPlan p{1, 0, 8};
  while (p.cluster <= kMaxCluster && (int64_t)p.cluster * kMaxThreads * 8 < vecs) p.cluster *= 2;
  if (p.cluster > kMaxCluster) return LossPlan{0, 0, 0};
  // Few rows: more, smaller CTAs per row.
  while (rows * p.cluster < num_sms && p.cluster < 8 && vecs >= (int64_t)p.cluster * 2 * 128 * 2) p.cluster *= 2;
  const int64_t per_cta = (vecs + p.cluster - 1) / p.cluster;
  while (p.vectors > 1 && per_cta < (int64_t)p.vectors * 128) p.vectors /= 2;
  const int64_t threads = (per_cta + p.vectors - 1) / p.vectors;
  p.threads = (int)(threads > 0 ? (threads + 31) / 32 * 32 : 32);
  return p;
}

template <typename T, int NV, bool SAME>
cudaError_t launch_rows(const LossArgs& a, const LossPlan& p, int num_sms, cudaStream_t s) {
  auto kernel = loss_rows_kernel<T, NV, SAME>;
  cudaLaunchConfig_t cfg{};
  cfg.blockDim = dim3((unsigned)p.threads);
  cfg.stream = s;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim = {(unsigned)p.cluster, 1, 1};
  cfg.attrs = &attr;
  cfg.numAttrs = p.cluster > 1 ? 1 : 0;
  if (p.cluster > 8) {
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
  }
  // As many clusters as run at once: a persistent grid larger than that would
  // leave its last clusters, and their rows, to a second wave.
  cfg.gridDim = dim3((unsigned)p.cluster);
  int clusters = 0;
  cudaError_t e;
  if (p.cluster > 1) {
    e = cudaOccupancyMaxActiveClusters(&clusters, kernel, &cfg);
  } else {
    e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&clusters, kernel, p.threads, 0);
    clusters *= num_sms;
  }
  if (e != cudaSuccess) return e;
  if (clusters < 1) clusters = 1;
  if (clusters > a.rows) clusters = (int)a.rows;
  cfg.gridDim = dim3((unsigned)(clusters * p.cluster));
  e = cudaLaunchKernelEx(&cfg, kernel, a);
  note_launch();
  return e;
}

template <typename T, bool SAME>
cudaError_t launch_vectors(const LossArgs& a, const LossPlan& p, int num_sms, cudaStream_t s) {
  switch (p.vectors) {
    case 1: return launch_rows<T, 1, SAME>(a, p, num_sms, s);
    case 2: return launch_rows<T, 2, SAME>(a, p, num_sms, s);
    case 4: return launch_rows<T, 4, SAME>(a, p, num_sms, s);
    default: return launch_rows<T, 8, SAME>(a, p, num_sms, s);
  }
}

template <typename T>
cudaError_t launch_typed(const LossArgs& a, int num_sms, cudaStream_t s) {
  constexpr int kE = Vectors<T>::kE;
  const LossPlan p = plan_loss(a.rows, a.vocab / kE, num_sms);
  if (p.cluster == 0) {
    const int64_t grid = a.rows < 2ll * num_sms ? a.rows : 2ll * num_sms;
    loss_long_rows_kernel<T><<<(unsigned)grid, kMaxThreads, 0, s>>>(a);
    note_launch();
    return cudaGetLastError();
  }
  const bool same = !a.grad || (reinterpret_cast<uintptr_t>(a.logits) - reinterpret_cast<uintptr_t>(a.grad)) % 16 == 0;
  return same ? launch_vectors<T, true>(a, p, num_sms, s) : launch_vectors<T, false>(a, p, num_sms, s);
}

}  // namespace

cudaError_t launch_loss(const LossArgs& a, int logits_dtype, int num_sms, cudaStream_t s) {
  if (a.rows > 0) {
    const cudaError_t e = logits_dtype == DSPARK_DTYPE_FP32 ? launch_typed<float>(a, num_sms, s)
                                                            : launch_typed<__nv_bfloat16>(a, num_sms, s);
    if (e != cudaSuccess) return e;
  }
  loss_sum_kernel<<<1, kMaxThreads, 0, s>>>(a);
  note_launch();
  return cudaGetLastError();
}

}  // namespace dspark
