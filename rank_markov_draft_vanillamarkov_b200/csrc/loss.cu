// The teacher-forced training loss on corrected logits, with its gradient.
//
// Row i with target t, weight w_i and logits c: lse = log sum_v exp(c_v),
// nll_i = lse - c_t, loss = sum_i w_i nll_i / N with N = sum_i w_i (mean) or 1
// (sum), d loss / d c_v = w_i / N (exp(c_v - lse) - [v = t]).
//
// The sum and the gradient both need the whole row, so a kernel that streams
// reads it twice. Here a cluster of CTAs keeps a row in its registers (a
// 129280-id bf16 row is 252 KB, a quarter of it in each of four CTAs): each
// logit is read once and each gradient written once, 4 bytes per bf16 logit,
// and that traffic is the bound.
//
// Pass 1: every thread takes its maximum m and sum s of 2^(c log2 e - r), where
// the reference r = m log2 e is rounded; the warps' pairs (m, s) meet in every
// CTA of the cluster. Pass 2 turns the registers into the gradient, and each
// vector's registers load the next row's as soon as it is written. All of a
// row goes by rounded references, so their rounding cancels. Two CTAs share an
// SM, so that one passes while the other meets. Plain loads and stores carry
// more here than bulk copies through shared memory, which held the same kernel
// to 4.3 TB/s whatever it computed.
//
// Measured: 2560 rows of 129280 bf16, a fifth of them ignored, 248 us (4.8 TB/s
// of 1.19 GB; a plain copy of as many bytes 190 us), 320 rows 46 us (3.6 TB/s;
// the copy 33 us), 320 fp32 rows 70.5 us (4.7 TB/s; 57 us). What keeps it from the
// copy: two exponentials a logit at 16 per clock and SM are 18 us for 320 rows
// (the pipe that makes them is busy for 24 of a launch's 43), and 71 clusters of
// four run at once, so that 320 rows go in five rounds of which the last is half
// empty. Without the gradient 320 rows take 32 us.
#include <algorithm>
#include <cmath>
#include <mutex>

#include "common.cuh"
#include "cluster.cuh"
#include "kernels.h"

namespace dspark {

namespace {

constexpr int kMaxThreads = 256;
constexpr int kMaxWarps = kMaxThreads / 32;
constexpr int kSumThreads = 512;  // of the kernels of one CTA per row or per call
constexpr int kMaxCluster = 16;
constexpr int kWholeCtas = 8;     // of a launch that is one cluster
constexpr int kMaxVectors = 16;   // of a row, in a thread's registers
constexpr int kNoFailure = 0x7fffffff;
constexpr uint64_t kDrainNs = 2000000000ull;  // the least limit of a wait for copies under way
constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.693147180559945309417f;

// 2^x by the hardware approximation (relative error 2^-22; 0 below 2^-126).
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Two fp32 operations in one instruction: a x + b and a x for a pair, and a sum.
__device__ __forceinline__ float2 fma2(float2 x, float a, float b) {
  float2 r;
  asm("{\n\t.reg .b64 p, q, r;\n\tmov.b64 p, {%2, %3};\n\tmov.b64 q, {%4, %4};\n\tmov.b64 r, {%5, %5};\n\t"
      "fma.rn.f32x2 p, p, q, r;\n\tmov.b64 {%0, %1}, p;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(x.x), "f"(x.y), "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float2 mul2(float2 x, float a) {
  float2 r;
  asm("{\n\t.reg .b64 p, q;\n\tmov.b64 p, {%2, %3};\n\tmov.b64 q, {%4, %4};\n\tmul.rn.f32x2 p, p, q;\n\t"
      "mov.b64 {%0, %1}, p;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(x.x), "f"(x.y), "f"(a));
  return r;
}
__device__ __forceinline__ float2 add2(float2 x, float2 y) {
  float2 r;
  asm("{\n\t.reg .b64 p, q;\n\tmov.b64 p, {%2, %3};\n\tmov.b64 q, {%4, %5};\n\tadd.rn.f32x2 p, p, q;\n\t"
      "mov.b64 {%0, %1}, p;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(x.x), "f"(x.y), "f"(y.x), "f"(y.y));
  return r;
}

// The factor from logits to the exponents' units for logits of which the
// largest is m. Where m log2 e could overflow, two logits that differ at all do
// so by far more than any exponent, so a quarter of them serves as well (and
// stays finite): equal logits have equal exponents, all others vanish.
__device__ __forceinline__ float unit_for(float m) { return fabsf(m) > 0x1p126f ? 0.25f : kLog2e; }
__device__ __forceinline__ float reference(float m) { return m == -INFINITY ? 0.0f : __fmul_rn(m, unit_for(m)); }
// A sum whose largest logit is m, brought to the reference of top >= m. One
// without a logit (m = -inf) is zero or NaN and stays; one in other units lies
// infinitely far below.
__device__ __forceinline__ float rescaled(float s, float m, float top) {
  if (m == top || m == -INFINITY) return s;
  return unit_for(m) == unit_for(top) ? s * ex2(reference(m) - reference(top)) : s * 0.0f;
}

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

// 16 bytes of a row.
template <typename T>
struct Vectors;
template <>
struct Vectors<float> {
  static constexpr int kE = 4;
  static constexpr uint32_t kFill = 0xff800000u;  // -inf
  static __device__ __forceinline__ float2 pair(const uint4& r, int i) {
    return i == 0 ? make_float2(__uint_as_float(r.x), __uint_as_float(r.y))
                  : make_float2(__uint_as_float(r.z), __uint_as_float(r.w));
  }
  static __device__ __forceinline__ float max_of(const uint4& r) {
    const float2 a = pair(r, 0), b = pair(r, 1);
    return fmaxf(fmaxf(a.x, a.y), fmaxf(b.x, b.y));
  }
  static __device__ __forceinline__ uint4 pack(const float2* g) {
    return make_uint4(__float_as_uint(g[0].x), __float_as_uint(g[0].y), __float_as_uint(g[1].x),
                      __float_as_uint(g[1].y));
  }
};
template <>
struct Vectors<__nv_bfloat16> {
  static constexpr int kE = 8;
  static constexpr uint32_t kFill = 0xff80ff80u;
  static __device__ __forceinline__ float2 pair(const uint4& r, int i) {
    const uint32_t w = i == 0 ? r.x : i == 1 ? r.y : i == 2 ? r.z : r.w;
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
  }
  static __device__ __forceinline__ __nv_bfloat162 both(uint32_t w) {
    return *reinterpret_cast<const __nv_bfloat162*>(&w);
  }
  static __device__ __forceinline__ float max_of(const uint4& r) {
    const __nv_bfloat162 m = __hmax2(__hmax2(both(r.x), both(r.y)), __hmax2(both(r.z), both(r.w)));
    return fmaxf(__low2float(m), __high2float(m));
  }
  static __device__ __forceinline__ uint32_t pack2(float2 x) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(x.x, x.y);
    return *reinterpret_cast<const uint32_t*>(&v);
  }
  static __device__ __forceinline__ uint4 pack(const float2* g) {
    return make_uint4(pack2(g[0]), pack2(g[1]), pack2(g[2]), pack2(g[3]));
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

// loss = sum_i w_i nll_i / N over the live rows, and the status of the targets,
// by one CTA.
__device__ void sum_loss(const LossArgs& a, double* sums) {
  const double inv_n = inverse_total(a, sums, true);
  double s = 0.0;
  for (int64_t i = threadIdx.x; i < a.rows; i += blockDim.x) {
    int64_t t;
    float w;
    if (live_row(a, i, &t, &w)) s += (double)w * (double)__ldcg(a.row_losses + i);
  }
  s = block_sum(s, sums);
  if (threadIdx.x == 0) *a.loss = (float)(s * inv_n);
}
__global__ void __launch_bounds__(kSumThreads) loss_sum_kernel(LossArgs a) {
  __shared__ double sums[kSumThreads / 32];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  sum_loss(a, sums);
}

struct LossPlan {
  int cluster;  // CTAs per row
  int threads;  // per CTA
  int slice;    // vectors of a row per CTA
  int vectors;  // of them per thread, at most
  int whole;    // the launch is one hardware cluster, a CTA per row, which also sums the loss
};

// The vectors of a row that lie in CTA `rank`'s slice.
__device__ __forceinline__ int slice_vectors(const LossPlan& p, int vecs, int rank) {
  return max(0, min(p.slice, vecs - rank * p.slice));
}

// A wait that expired ends its warp's rows. In all CTAs of the cluster the other
// warps' waits expire then too, at most one row later, since a row's wait needs
// the pairs of every warp. So each warp has sent its pair `failed`, counted from
// zero, and some have sent the next one. Those that have not send it now, so
// that both barriers complete and no CTA leaves before all stores to its shared
// memory have landed. The losses from the failed row on are NaN; gradients that
// are not written stay as they were.
__device__ void end_failed_rows(const LossArgs& a, int ranks, int failed, int sent, uint64_t* met_bar, float2* pairs) {
  const int tid = (int)threadIdx.x, warp = tid >> 5, lane = tid & 31, warps = (int)blockDim.x >> 5;
  const int rank = ranks > 1 ? (int)cluster_rank() : 0;
  if (ranks > 1) {
    const int next = failed + 1;
    if (sent == next) {
      float2* slots = pairs + (next & 1) * (kMaxCluster * kMaxWarps);
      if (tid == 0) mbar_arrive_expect_tx(&met_bar[next & 1], (uint32_t)(ranks * warps * sizeof(float2)));
      if (lane < ranks)
        store_async(remote_u32(&slots[rank * warps + warp], (uint32_t)lane), 0.0f, 0.0f,
                    remote_u32(&met_bar[next & 1], (uint32_t)lane));
    }
    if (tid == 0) {
      volatile int never = 0;
      const WaitCtl ctl{&never, a.status, a.wait_limit_ns > kDrainNs ? a.wait_limit_ns : kDrainNs};
      for (int k = failed; k <= next; ++k) mbar_wait_cluster(&met_bar[k & 1], (uint32_t)(k >> 1) & 1u, ctl);
    }
  }
  if (rank == 0 && tid == 0) {
    int before = 0;
    for (int64_t i = blockIdx.x / ranks; i < a.rows; i += gridDim.x / ranks) {
      int64_t t;
      float w;
      const bool live = live_row(a, i, &t, &w);
      if (before >= failed) a.row_losses[i] = live ? NAN : 0.0f;
      if (live) ++before;
    }
  }
}

// SAME: the gradient's rows start at the same offset from a 16-byte address as
// the logits' (in place, or any vocabulary of whole vectors), so that a vector
// read is a vector written; otherwise gradients are written one by one.
template <typename T, int NV, bool SAME>
__global__ void __launch_bounds__(kMaxThreads, 2) loss_rows_kernel(LossArgs a, LossPlan p) {
  constexpr int kE = Vectors<T>::kE;
  __shared__ uint64_t met_bar[2];  // a row's pairs are here
  __shared__ float2 pairs[2][kMaxCluster * kMaxWarps];
  __shared__ double sums[kMaxWarps];
  __shared__ int abort_flag, first_failed;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, tid = (int)threadIdx.x;
  const int threads = (int)blockDim.x, warps = threads >> 5;
  const int ranks = p.cluster, rank = ranks > 1 ? (int)cluster_rank() : 0;
  const int step = (int)gridDim.x / ranks, rows = (int)a.rows, vocab = (int)a.vocab;
  const T* logits = static_cast<const T*>(a.logits);
  T* grads = static_cast<T*>(a.grad);
  const WaitCtl ctl{&abort_flag, a.status, a.wait_limit_ns};
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (tid == 0) {
    abort_flag = 0;
    first_failed = kNoFailure;
    const uint32_t arrivals = ranks > 1 ? 1u : (uint32_t)warps;  // a cluster's pairs count as bytes
    mbar_init(&met_bar[0], arrivals);
    mbar_init(&met_bar[1], arrivals);
    fence_barrier_init();
  }

  int i = (int)blockIdx.x / ranks, t = 0;  // the row and its target
  float w = 0.0f;
  auto look_up = [&](int row, int* target, float* weight) {
    int64_t id = 0;
    const bool live = row < rows && live_row(a, row, &id, weight);
    *target = (int)id;
    return live;
  };
  // This thread's vectors: j0 + 32 n of the slice, each warp a run of 32 NV.
  const int j0 = warp * 32 * NV + lane;
  uint4 raw[NV];
  float edge = -INFINITY, xt = 0.0f;   // its edge element; the target's logit
  // Rows of whole vectors all begin alike.
  const bool ragged = vocab % kE != 0;
  const RowShape<T> first_shape(logits, vocab);
  auto shape_of = [&](int row) { return ragged ? RowShape<T>(logits + (int64_t)row * vocab, vocab) : first_shape; };
  auto load_singles = [&](int row, const RowShape<T>& shape, int target) {
    const T* c = logits + (int64_t)row * vocab;
    edge = rank == 0 && tid < shape.edges ? to_f32(c[shape.edge(tid)]) : -INFINITY;
    xt = to_f32(c[target]);
  };
  // Where a vector is not in the slice its registers hold -inf.
  auto load = [&](const uint4* from, int left, int n) {
    if (32 * n < left)
      raw[n] = __ldcs(from + 32 * n);
    else if (ragged)
      raw[n] = make_uint4(Vectors<T>::kFill, Vectors<T>::kFill, Vectors<T>::kFill, Vectors<T>::kFill);
  };
#pragma unroll
  for (int n = 0; n < NV; ++n)
    raw[n] = make_uint4(Vectors<T>::kFill, Vectors<T>::kFill, Vectors<T>::kFill, Vectors<T>::kFill);
  bool live = look_up(i, &t, &w);
  if (live) {
    const T* c = logits + (int64_t)i * vocab;
    const RowShape<T> shape = shape_of(i);
    const uint4* from = reinterpret_cast<const uint4*>(c + shape.head) + rank * p.slice + j0;
    const int left = slice_vectors(p, shape.vecs, rank) - j0;
#pragma unroll
    for (int n = 0; n < NV; ++n) load(from, left, n);
    load_singles(i, shape, t);
  }
  const double inv_n = inverse_total(a, sums, false);
  __syncthreads();
  if (ranks > 1) cluster_barrier();  // every CTA's barriers are there

  int sent = 0;  // pairs of this warp: live rows so far
  while (i < rows) {
    const int next = rows - i > step ? i + step : rows;
    int next_t = 0;
    float next_w = 0.0f;
    const bool next_live = look_up(next, &next_t, &next_w);
    const RowShape<T> shape = shape_of(i);
    const int count = slice_vectors(p, shape.vecs, rank);
    const int left = grads ? count - j0 : 0;
    T* g = grads ? grads + (int64_t)i * vocab : nullptr;
    T* to = g + shape.head + (rank * p.slice + j0) * kE;
    const T* cn = logits + (int64_t)next * vocab;
    const RowShape<T> next_shape = shape_of(next);
    const uint4* from = reinterpret_cast<const uint4*>(cn + next_shape.head) + rank * p.slice + j0;
    const int next_left = next_live ? slice_vectors(p, next_shape.vecs, rank) - j0 : 0;
    if (!live) {
      if (rank == 0 && tid == 0) a.row_losses[i] = 0.0f;
      if (g && rank == 0 && tid < shape.edges) g[shape.edge(tid)] = from_f32<T>(0.0f);
#pragma unroll
      for (int n = 0; n < NV; ++n) {
        if (32 * n < left) {
          if (SAME) {
            __stcs(reinterpret_cast<uint4*>(to) + 32 * n, make_uint4(0u, 0u, 0u, 0u));
          } else {
#pragma unroll
            for (int e = 0; e < kE; ++e) to[32 * n * kE + e] = from_f32<T>(0.0f);
          }
        }
        load(from, next_left, n);
      }
      if (next_live) load_singles(next, next_shape, next_t);
    } else {
      // Pass 1. A thread of -inf alone keeps m = -inf and sums zeros (or NaN).
      float m = edge;
#pragma unroll
      for (int n = 0; n < NV; ++n) m = fmaxf(m, Vectors<T>::max_of(raw[n]));
      float s;
      {
        const float unit = unit_for(m), ref = reference(m);
        float2 part[2] = {make_float2(ex2(fmaf(edge, unit, -ref)), 0.0f), make_float2(0.0f, 0.0f)};
#pragma unroll
        for (int n = 0; n < NV; ++n)
#pragma unroll
          for (int e = 0; e < kE / 2; ++e) {
            const float2 x = fma2(Vectors<T>::pair(raw[n], e), unit, -ref);
            part[e & 1] = add2(part[e & 1], make_float2(ex2(x.x), ex2(x.y)));
          }
        s = (part[0].x + part[0].y) + (part[1].x + part[1].y);
      }
      // The target's logit changes no maximum; with it here, it has been read
      // before the pair leaves, after which an in-place gradient may replace it.
      float top = fmaxf(m, xt);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
      s = rescaled(s, m, top);
      m = top;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
      // The warp's pair to every CTA. The other of the two buffers may still
      // be read; this one was left by all warps before they sent the pairs
      // that ended the last row's wait. Stores that the barrier counts, since an
      // arrival that releases one waits for the last row's gradients as well.
      const int parity = sent & 1;
      if (ranks > 1) {
        if (tid == 0) mbar_arrive_expect_tx(&met_bar[parity], (uint32_t)(ranks * warps * sizeof(float2)));
        if (lane < ranks)
          store_async(remote_u32(&pairs[parity][rank * warps + warp], (uint32_t)lane), m, s,
                      remote_u32(&met_bar[parity], (uint32_t)lane));
      } else if (lane == 0) {
        pairs[parity][warp] = make_float2(m, s);
        mbar_arrive(&met_bar[parity]);
      }
      ++sent;
      __syncwarp();
      const float row_xt = xt, row_edge = edge;
      if (next_live) load_singles(next, next_shape, next_t);
      // Whether the target is in one of this thread's vectors.
      const int at = t - shape.head, vec = at >= 0 ? at / kE - rank * p.slice : -1;
      const bool own_target = vec >= 0 && vec < count && vec / (32 * NV) == warp && vec % 32 == lane;
      const float scale = (float)((double)w * inv_n);
      if (!__all_sync(0xffffffffu, mbar_wait_cluster(&met_bar[parity], ((uint32_t)(sent - 1) >> 1) & 1u, ctl))) {
        if (ranks > 1) {
          if (lane < ranks) cluster_min(remote_u32(&first_failed, (uint32_t)lane), sent - 1);
        } else if (lane == 0) {
          atomicMin(&first_failed, sent - 1);
        }
        break;
      }
      // Each warp for itself. Without NaN, which is orderable above all: a
      // warp's maximum is NaN only where it has no number at all.
      const int met = ranks * warps;
      uint32_t high = 0u;
      for (int k = lane; k < met; k += 32) {
        const float x = pairs[parity][k].x;
        high = max(high, x == x ? orderable_bits(x) : 0u);
      }
      high = __reduce_max_sync(0xffffffffu, high);
      m = high == 0u ? -INFINITY : __uint_as_float((high & 0x80000000u) ? high & 0x7fffffffu : ~high);
      s = 0.0f;
      for (int k = lane; k < met; k += 32) {
        const float2 q = pairs[parity][k];
        s += rescaled(q.y, q.x, m);
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
      if (isinf(m)) s = NAN;  // +inf somewhere, or -inf everywhere
      const float factor = scale / s, unit = unit_for(m), ref = reference(m);
      if (rank == 0 && tid == 0) {
        // In plain units where the exponents' would overflow. Both terms lie
        // around a rounded reference: where they cancel, what their rounding
        // leaves below zero is zero (NaN stays).
        const float nll = unit == kLog2e && fabsf(row_xt) <= 0x1p126f ? kLn2 * (log2f(s) - fmaf(row_xt, unit, -ref))
                                                                      : logf(s) + (m - row_xt);
        a.row_losses[i] = nll <= 0.0f ? 0.0f : nll;
      }
      // The gradient at the target, which its owner writes over the rest.
      const float at_target = ex2(fmaf(row_xt, unit, -ref)) * factor - scale;
      if (g && rank == 0 && tid < shape.edges) {
        const int v = shape.edge(tid);
        g[v] = from_f32<T>(v == t ? at_target : ex2(fmaf(row_edge, unit, -ref)) * factor);
      }
      // Pass 2.
#pragma unroll
      for (int n = 0; n < NV; ++n) {
        if (32 * n < left) {
          float2 x[kE / 2];
#pragma unroll
          for (int e = 0; e < kE / 2; ++e) {
            x[e] = fma2(Vectors<T>::pair(raw[n], e), unit, -ref);
            x[e] = mul2(make_float2(ex2(x[e].x), ex2(x[e].y)), factor);
          }
          if (SAME) {
            __stcs(reinterpret_cast<uint4*>(to) + 32 * n, Vectors<T>::pack(x));
          } else {
#pragma unroll
            for (int e = 0; e < kE / 2; ++e) {
              to[32 * n * kE + 2 * e] = from_f32<T>(x[e].x);
              to[32 * n * kE + 2 * e + 1] = from_f32<T>(x[e].y);
            }
          }
        }
        load(from, next_left, n);
      }
      if (g && own_target) g[t] = from_f32<T>(at_target);  // after the vector that holds it, by the same thread
    }
    i = next;
    t = next_t;
    w = next_w;
    live = next_live;
  }
  __syncwarp();
  if (ranks > 1)
    cluster_barrier();  // no CTA leaves while others may still send to it
  else
    __syncthreads();
  if (first_failed != kNoFailure) end_failed_rows(a, ranks, first_failed, sent, met_bar, &pairs[0][0]);
  if (p.whole) {
    cluster_barrier();  // every row's loss is written
    if (blockIdx.x == 0) sum_loss(a, sums);
  }
}

// Rows longer than a cluster's registers (524288 bf16 or 262144 fp32 ids): one
// CTA per row reads it twice, an element at a time. 64 rows of 600001 bf16 ids
// take 863 us, 132 without the gradient; their traffic is worth 35.
template <typename T>
__global__ void __launch_bounds__(kSumThreads) loss_long_rows_kernel(LossArgs a) {
  __shared__ double sums[kSumThreads / 32];
  __shared__ float2 parts[kSumThreads / 32];
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

// The cluster for a row of `vecs` vectors, or cluster 0 where none holds it.
LossPlan plan_loss(int64_t rows, int64_t vecs, int num_sms) {
  constexpr int64_t kMaxSlice = (int64_t)kMaxThreads * kMaxVectors;
  int64_t cluster = 1;
  while (cluster <= kMaxCluster && cluster * kMaxSlice < vecs) cluster *= 2;
  LossPlan p{};
  if (cluster > kMaxCluster) return p;
  // Small calls: one launch, all rows in one cluster of CTAs with a row each at
  // a time, instead of a second kernel for the sum. As called from Python that
  // saves 1 us of about 14.4 while a CTA has two rows at most; from a graph
  // 8 x 16000 bf16 ids take 7.1 us against 7.4, 16 x 1024 take 6.9 against 6.0,
  // 32 x 1024 9.7 against 6.1 and 4 x 32000 8.6 against 7.0.
  p.whole = cluster == 1 && rows <= 2 * kWholeCtas && vecs <= 2048 ? 1 : 0;
  // Few rows: more CTAs for each.
  while (!p.whole && rows * cluster * 2 <= 2 * num_sms && cluster < 8 && vecs >= cluster * 2 * 512) cluster *= 2;
  const int64_t slice = std::max<int64_t>(1, (vecs + cluster - 1) / cluster);
  p.cluster = (int)cluster;
  p.slice = (int)slice;
  p.vectors = 1;
  while ((int64_t)p.vectors * kMaxThreads < slice) p.vectors *= 2;
  p.threads = (int)std::max<int64_t>(64, (slice + 32 * p.vectors - 1) / (32 * p.vectors) * 32);
  return p;
}

// How many clusters of a plan run at once on the current device, kept by the
// plan since asking takes longer than a launch.
template <typename T, int NV, bool SAME>
cudaError_t active_clusters(const LossPlan& p, cudaLaunchConfig_t cfg, int num_sms, int* out) {
  struct Known {
    int device, cluster, threads, clusters;
  };
  static std::mutex mu;
  static Known known[32];
  static int count = 0;
  int device = 0;
  cudaError_t e = cudaGetDevice(&device);
  if (e != cudaSuccess) return e;
  std::lock_guard<std::mutex> lock(mu);
  for (int i = 0; i < std::min(count, 32); ++i)
    if (known[i].device == device && known[i].cluster == p.cluster && known[i].threads == p.threads) {
      *out = known[i].clusters;
      return cudaSuccess;
    }
  auto kernel = loss_rows_kernel<T, NV, SAME>;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e != cudaSuccess) return e;
  int clusters = 0;
  if (p.cluster > 1) {
    cfg.gridDim = dim3((unsigned)p.cluster);
    e = cudaOccupancyMaxActiveClusters(&clusters, kernel, &cfg);
  } else {
    e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&clusters, kernel, p.threads, 0);
    clusters *= num_sms;
  }
  if (e != cudaSuccess) return e;
  *out = std::max(clusters, 1);
  known[count++ % 32] = Known{device, p.cluster, p.threads, *out};
  return cudaSuccess;
}

template <typename T, int NV, bool SAME>
cudaError_t launch_rows(const LossArgs& a, const LossPlan& p, int num_sms, cudaStream_t s) {
  cudaLaunchConfig_t cfg{};
  cfg.blockDim = dim3((unsigned)p.threads);
  cfg.stream = s;
  const int in_cluster = p.whole ? kWholeCtas : p.cluster;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim = {(unsigned)in_cluster, 1, 1};
  cfg.attrs = &attr;
  cfg.numAttrs = in_cluster > 1 ? 1 : 0;
  // As many clusters as run at once: a persistent grid larger than that would
  // leave its last clusters, and their rows, to a second wave.
  int clusters = 0;
  cudaError_t e = active_clusters<T, NV, SAME>(p, cfg, num_sms, &clusters);
  if (e != cudaSuccess) return e;
  cfg.gridDim = dim3((unsigned)(p.whole ? kWholeCtas : std::min<int64_t>(clusters, a.rows) * p.cluster));
  e = cudaLaunchKernelEx(&cfg, loss_rows_kernel<T, NV, SAME>, a, p);
  note_launch();
  return e;
}

template <typename T, bool SAME>
cudaError_t launch_vectors(const LossArgs& a, const LossPlan& p, int num_sms, cudaStream_t s) {
  switch (p.vectors) {
    case 1: return launch_rows<T, 1, SAME>(a, p, num_sms, s);
    case 2: return launch_rows<T, 2, SAME>(a, p, num_sms, s);
    case 4: return launch_rows<T, 4, SAME>(a, p, num_sms, s);
    case 8: return launch_rows<T, 8, SAME>(a, p, num_sms, s);
    default: return launch_rows<T, kMaxVectors, SAME>(a, p, num_sms, s);
  }
}

template <typename T>
cudaError_t launch_typed(const LossArgs& a, int num_sms, cudaStream_t s, bool* summed) {
  const LossPlan p = plan_loss(a.rows, a.vocab / Vectors<T>::kE, num_sms);
  *summed = p.whole != 0;
  if (p.cluster == 0) {
    const int64_t grid = a.rows < 2ll * num_sms ? a.rows : 2ll * num_sms;
    loss_long_rows_kernel<T><<<(unsigned)grid, kSumThreads, 0, s>>>(a);
    note_launch();
    return cudaGetLastError();
  }
  const bool same = !a.grad || (reinterpret_cast<uintptr_t>(a.logits) - reinterpret_cast<uintptr_t>(a.grad)) % 16 == 0;
  return same ? launch_vectors<T, true>(a, p, num_sms, s) : launch_vectors<T, false>(a, p, num_sms, s);
}

}  // namespace

cudaError_t launch_loss(const LossArgs& a, int logits_dtype, int num_sms, cudaStream_t s) {
  bool summed = false;
  if (a.rows > 0) {
    const cudaError_t e = logits_dtype == DSPARK_DTYPE_FP32 ? launch_typed<float>(a, num_sms, s, &summed)
                                                            : launch_typed<__nv_bfloat16>(a, num_sms, s, &summed);
    if (e != cudaSuccess || summed) return e;
  }
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(1);
  cfg.blockDim = dim3(kSumThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr{};  // its launch overlaps the rows; it waits for their end
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = a.rows > 0 ? 1 : 0;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, loss_sum_kernel, a);
  note_launch();
  return e;
}

}  // namespace dspark
