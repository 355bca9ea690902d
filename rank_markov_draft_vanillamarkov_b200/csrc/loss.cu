// The teacher-forced training loss on corrected logits, with its gradient.
//
// Row i with target t, weight w_i and logits c: lse = log sum_v exp(c_v),
// nll_i = lse - c_t, loss = sum_i w_i nll_i / N with N = sum_i w_i (mean) or 1
// (sum), d loss / d c_v = w_i / N (exp(c_v - lse) - [v = t]).
//
// The sum and the gradient both need the whole row, so a kernel that streams
// reads it twice. Here a cluster of CTAs keeps a row in its shared memory (a
// 129280-id bf16 row is 252 KB, more than one SM's): each logit is read once
// and each gradient written once, 4 bytes per bf16 logit, and that traffic is
// the bound.
//
// A CTA's slice of a row lies in a ring of chunks, filled and emptied by bulk
// copies that one thread issues. Pass 1 walks the chunks as they land, every
// thread with its own running maximum m and sum s of 2^(c log2 e - r), where
// the reference r = m log2 e is rounded; the warps' pairs (m, s) meet in every
// CTA of the cluster. Pass 2 overwrites the chunks by the gradient, each copied
// out as it is done and its place filled with the next row's chunk. All of a
// row goes by rounded references, so their rounding cancels.
#include <algorithm>
#include <cmath>
#include <mutex>

#include "common.cuh"
#include "kernels.h"
#include "ptx.cuh"

namespace dspark {

namespace {

constexpr int kMaxThreads = 256;  // that compute; one warp more issues the copies
constexpr int kMaxWarps = kMaxThreads / 32;
constexpr int kSumThreads = 512;  // of the kernels of one CTA per row or per call
constexpr int kMaxCluster = 16;
constexpr int kWholeCtas = 8;   // of a launch that is one cluster
constexpr int kMaxSlots = 8;
constexpr int kRing = 108 * 1024;  // bytes, at most: two CTAs per SM, one passing while the other meets
constexpr int kPerThread = 4;  // vectors of a chunk for each thread: 4, in small chunks 2 or 1
constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.693147180559945309417f;

// 2^x by the hardware approximation (relative error 2^-22; 0 below 2^-126).
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
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
  static __device__ __forceinline__ float get(const uint4& r, int e) {
    const uint32_t w = e < 2 ? r.x : e < 4 ? r.y : e < 6 ? r.z : r.w;
    return __uint_as_float((e & 1) ? (w & 0xffff0000u) : (w << 16));
  }
  static __device__ __forceinline__ __nv_bfloat162 both(uint32_t w) {
    return *reinterpret_cast<const __nv_bfloat162*>(&w);
  }
  static __device__ __forceinline__ float max_of(const uint4& r) {
    const __nv_bfloat162 m = __hmax2(__hmax2(both(r.x), both(r.y)), __hmax2(both(r.z), both(r.w)));
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
  int warps;    // that compute, per CTA
  int slice;    // vectors of a row per CTA
  int chunk;    // vectors per chunk, at most 32 per_thread warps
  int per_thread;
  int chunks;   // chunks per slice
  int slots;    // chunks in the ring, at least `chunks`
  int whole;    // the launch is one hardware cluster, a CTA per row, which also sums the loss
};

struct RowBarriers {
  uint64_t full[kMaxSlots];  // a chunk has landed
  uint64_t done[kMaxSlots];  // every warp has left a chunk
  uint64_t met[2];           // a row's pairs are here
};

// Chunk c of a slice of `count` vectors: the vectors in it.
__device__ __forceinline__ int chunk_vectors(const LossPlan& p, int count, int c) {
  return max(0, min(p.chunk, count - c * p.chunk));
}
// The vectors of a row that lie in CTA `rank`'s slice.
__device__ __forceinline__ int slice_vectors(const LossPlan& p, int vecs, int rank) {
  return max(0, min(p.slice, vecs - rank * p.slice));
}

// SAME: the gradient's rows start at the same offset from a 16-byte address as
// the logits' (in place, or any vocabulary of whole vectors), so that a chunk
// is copied out as it was copied in; otherwise gradients are written one by one.
// PT: vectors of a chunk per thread; all but the last exist in every chunk.
template <typename T, int PT, bool SAME>
__global__ void __launch_bounds__(kMaxThreads + 32, 2) loss_rows_kernel(LossArgs a, LossPlan p) {
  constexpr int kE = Vectors<T>::kE;
  extern __shared__ __align__(128) uint4 ring[];
  __shared__ RowBarriers bars;
  __shared__ float2 pairs[2][kMaxCluster * kMaxWarps];
  __shared__ double sums[kMaxWarps + 1];
  __shared__ int abort_flag;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, tid = (int)threadIdx.x;
  const int ranks = p.cluster, rank = ranks > 1 ? (int)cluster_rank() : 0, warps = p.warps, threads = warps * 32;
  const int64_t step = gridDim.x / ranks, first = blockIdx.x / ranks;
  const int vocab = (int)a.vocab;
  const T* logits = static_cast<const T*>(a.logits);
  T* grads = static_cast<T*>(a.grad);
  const WaitCtl ctl{&abort_flag, a.status, a.wait_limit_ns};
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  // The next live row at or after i.
  auto seek = [&](int64_t i, int64_t* t, float* w) {
    while (i < a.rows && !live_row(a, i, t, w)) i += step;
    return i;
  };

  if (tid == 0) {
    abort_flag = 0;
    for (int k = 0; k < p.slots; ++k) {
      mbar_init(&bars.full[k], 1);
      mbar_init(&bars.done[k], (uint32_t)warps);
    }
    mbar_init(&bars.met[0], (uint32_t)(ranks * warps));
    mbar_init(&bars.met[1], (uint32_t)(ranks * warps));
    fence_barrier_init();
  }
  const double inv_n = inverse_total(a, sums, false);
  __syncthreads();
  if (ranks > 1) cluster_barrier();  // every CTA's barriers are there

  if (warp == warps) {
    if (lane == 0) {
      // The copies: chunk q goes to slot q % slots once the chunk that was
      // there has been copied out.
      int64_t t;
      float w;
      int64_t out_row = first, in_row = first;
      int out_c = 0, slot = 0, out_slot = 0;
      uint32_t out_phase = 0;
      int64_t in_flight = 0;  // chunks loaded and not yet copied out
      out_row = seek(out_row, &t, &w);
      auto copy_out = [&]() {
        if (!mbar_wait(&bars.done[out_slot], out_phase, ctl)) return false;
        if (SAME && grads) {
          const RowShape<T> shape(logits + out_row * vocab, vocab);
          const int n = chunk_vectors(p, slice_vectors(p, shape.vecs, rank), out_c);
          if (n > 0) {
            T* to = grads + out_row * vocab + shape.head + ((int64_t)rank * p.slice + out_c * p.chunk) * kE;
            bulk_store(to, ring + (size_t)out_slot * p.chunk, (uint32_t)n * 16u);
            bulk_commit_group();
            bulk_wait_group_read<0>();
          }
        }
        if (++out_slot == p.slots) {
          out_slot = 0;
          out_phase ^= 1u;
        }
        if (++out_c == p.chunks) {
          out_c = 0;
          out_row = seek(out_row + step, &t, &w);
        }
        --in_flight;
        return true;
      };
      bool ok = true;
      for (in_row = seek(in_row, &t, &w); ok && in_row < a.rows; in_row = seek(in_row + step, &t, &w)) {
        const RowShape<T> shape(logits + in_row * vocab, vocab);
        const int count = slice_vectors(p, shape.vecs, rank);
        const T* from = logits + in_row * vocab + shape.head + (int64_t)rank * p.slice * kE;
        for (int c = 0; c < p.chunks; ++c) {
          if (in_flight == p.slots && !(ok = copy_out())) break;
          const int n = chunk_vectors(p, count, c);
          if (n > 0) {
            mbar_arrive_expect_tx(&bars.full[slot], (uint32_t)n * 16u);
            bulk_load(ring + (size_t)slot * p.chunk, from + (int64_t)c * p.chunk * kE, (uint32_t)n * 16u,
                      &bars.full[slot]);
          } else {
            mbar_arrive(&bars.full[slot]);
          }
          ++in_flight;
          if (++slot == p.slots) slot = 0;
        }
      }
      while (ok && in_flight > 0) ok = copy_out();
      bulk_wait_group<0>();
      // After a wait that ran out, copies still under way end before the CTA does.
      if (!ok) {
        const uint64_t t0 = globaltimer_ns();
        for (int k = 0; k < p.slots && in_flight > 0; ++k)
          for (uint32_t phase = 0; phase < 2; ++phase)
            while (!mbar_try_wait(&bars.full[k], phase) && globaltimer_ns() - t0 < a.wait_limit_ns) {
            }
      }
    }
    __syncwarp();
  } else {
    int slot1 = 0, slot2 = 0, parity = 0;  // of pass 1 and pass 2 in the ring; of the pairs' buffer
    uint32_t phase1 = 0, met_phase = 0;
    int64_t i = first;
    int64_t t = 0;
    float w = 0.0f;
    float edge = -INFINITY, xt = 0.0f;  // this thread's edge element; the target's logit
    auto load_singles = [&](int64_t row, int64_t target) {
      const T* c = logits + row * vocab;
      const RowShape<T> shape(c, vocab);
      edge = rank == 0 && tid < shape.edges ? to_f32(c[shape.edge(tid)]) : -INFINITY;
      xt = to_f32(c[target]);
    };
    bool live = i < a.rows && live_row(a, i, &t, &w);
    if (live) load_singles(i, t);
    while (i < a.rows) {
      const int64_t next = i + step;
      int64_t next_t = 0;
      float next_w = 0.0f;
      const bool next_live = next < a.rows && live_row(a, next, &next_t, &next_w);
      const RowShape<T> shape(logits + i * vocab, vocab);
      const int count = slice_vectors(p, shape.vecs, rank);
      T* g = grads ? grads + i * vocab : nullptr;
      if (!live) {
        if (rank == 0 && tid == 0) a.row_losses[i] = 0.0f;
        if (g) {
          if (rank == 0 && tid < shape.edges) g[shape.edge(tid)] = from_f32<T>(0.0f);
          T* to = g + shape.head + (int64_t)rank * p.slice * kE;
          if (SAME) {
            for (int j = tid; j < count; j += threads)
              __stcs(reinterpret_cast<uint4*>(to) + j, make_uint4(0u, 0u, 0u, 0u));
          } else {
            for (int j = tid; j < count * kE; j += threads) to[j] = from_f32<T>(0.0f);
          }
        }
        if (next_live) load_singles(next, next_t);
      } else {
        // Pass 1. A thread of -inf alone keeps m = -inf and sums zeros (or NaN).
        float m = edge;
        float s = edge == -INFINITY ? 0.0f : ex2(fmaf(edge, unit_for(edge), -reference(edge)));
        for (int c = 0; c < p.chunks; ++c) {
          mbar_wait(&bars.full[slot1], phase1, ctl);
          const int n = chunk_vectors(p, count, c);
          const uint4* from = ring + (size_t)slot1 * p.chunk + tid;
          uint4 raw[PT];
#pragma unroll
          for (int k = 0; k < PT - 1; ++k) raw[k] = from[k * threads];
          raw[PT - 1] = make_uint4(Vectors<T>::kFill, Vectors<T>::kFill, Vectors<T>::kFill, Vectors<T>::kFill);
          if (tid + (PT - 1) * threads < n) raw[PT - 1] = from[(PT - 1) * threads];
          float top = m;
#pragma unroll
          for (int k = 0; k < PT; ++k) top = fmaxf(top, Vectors<T>::max_of(raw[k]));
          s = rescaled(s, m, top);
          m = top;
          const float unit = unit_for(top), ref = reference(top);
          float part[2] = {0.0f, 0.0f};
#pragma unroll
          for (int k = 0; k < PT; ++k)
#pragma unroll
            for (int e = 0; e < kE; ++e) part[e & 1] += ex2(fmaf(Vectors<T>::get(raw[k], e), unit, -ref));
          s += part[0] + part[1];
          if (++slot1 == p.slots) {
            slot1 = 0;
            phase1 ^= 1u;
          }
        }
        float top = m;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        s = rescaled(s, m, top);
        m = top;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        // The warp's pair to every CTA. The other of the two buffers may still
        // be read; this one was left by all warps before they sent the pairs
        // that ended the last row's wait.
        if (ranks > 1) {
          if (lane < ranks) {
            store_remote(remote_u32(&pairs[parity][rank * warps + warp], (uint32_t)lane), m, s);
            mbar_arrive_remote(remote_u32(&bars.met[parity], (uint32_t)lane));
          }
        } else if (lane == 0) {
          pairs[parity][warp] = make_float2(m, s);
          mbar_arrive(&bars.met[parity]);
        }
        __syncwarp();
        const float row_xt = xt, row_edge = edge;
        if (next_live) load_singles(next, next_t);
        // The target's place in this slice, as chunk and vector, if any.
        const int at = (int)t - shape.head, vec = at >= 0 ? at / kE - rank * p.slice : -1, te = at % kE;
        const int tc = vec >= 0 && vec < count ? vec / p.chunk : -1, tj = vec - tc * p.chunk;
        const bool own_target = tc >= 0 && tj % threads == tid;
        const float scale = (float)((double)w * inv_n);
        mbar_wait_cluster(&bars.met[parity], met_phase, ctl);
        // Each warp for itself, a lane for up to four pairs.
        float2 met[kMaxCluster * kMaxWarps / 32];
        uint32_t high = 0u;
#pragma unroll
        for (int k = 0; k < kMaxCluster * kMaxWarps / 32; ++k) {
          met[k] = lane + 32 * k < ranks * warps ? pairs[parity][lane + 32 * k] : make_float2(-INFINITY, 0.0f);
          // Without NaN (orderable above all): a warp's maximum is NaN only where it has no number at all.
          high = max(high, met[k].x == met[k].x ? orderable_bits(met[k].x) : 0u);
        }
        high = __reduce_max_sync(0xffffffffu, high);
        m = __uint_as_float((high & 0x80000000u) ? high & 0x7fffffffu : ~high);
        s = 0.0f;
#pragma unroll
        for (int k = 0; k < kMaxCluster * kMaxWarps / 32; ++k) s += rescaled(met[k].y, met[k].x, m);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        parity ^= 1;
        if (parity == 0) met_phase ^= 1u;
        if (isinf(m)) s = NAN;  // +inf somewhere, or -inf everywhere
        const float factor = scale / s, unit = unit_for(m), ref = reference(m);
        if (rank == 0 && tid == 0)  // in plain units where the exponents' would overflow
          a.row_losses[i] = unit == kLog2e && fabsf(row_xt) <= 0x1p126f
                                ? kLn2 * (log2f(s) - fmaf(row_xt, unit, -ref))
                                : logf(s) + (m - row_xt);
        // The gradient at the target, which its owner writes over the rest.
        const float at_target = ex2(fmaf(row_xt, unit, -ref)) * factor - scale;
        if (g && rank == 0 && tid < shape.edges) {
          const int v = shape.edge(tid);
          g[v] = from_f32<T>(v == (int)t ? at_target : ex2(fmaf(row_edge, unit, -ref)) * factor);
        }
        // Pass 2.
        T* to = g + shape.head + (int64_t)rank * p.slice * kE;
        for (int c = 0; c < p.chunks; ++c) {
          const int n = chunk_vectors(p, count, c);
          uint4* place = ring + (size_t)slot2 * p.chunk + tid;
          if (g) {
#pragma unroll
            for (int k = 0; k < PT; ++k) {
              const int j = tid + k * threads;
              if (k == PT - 1 && j >= n) break;
              const uint4 raw = place[k * threads];
              float x[kE];
#pragma unroll
              for (int e = 0; e < kE; ++e) x[e] = ex2(fmaf(Vectors<T>::get(raw, e), unit, -ref)) * factor;
              if (SAME) {
                place[k * threads] = Vectors<T>::pack(x);
              } else {
#pragma unroll
                for (int e = 0; e < kE; ++e) to[((int64_t)c * p.chunk + j) * kE + e] = from_f32<T>(x[e]);
              }
            }
            if (own_target && c == tc) {
              if (SAME)
                reinterpret_cast<T*>(ring + (size_t)slot2 * p.chunk + tj)[te] = from_f32<T>(at_target);
              else
                g[t] = from_f32<T>(at_target);
            }
          }
          if (SAME) fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(&bars.done[slot2]);
          if (++slot2 == p.slots) slot2 = 0;
        }
      }
      i = next;
      t = next_t;
      w = next_w;
      live = next_live;
    }
    __syncwarp();
  }
  if (ranks > 1) cluster_barrier();  // no CTA leaves while others may still send to it
  if (p.whole) {
    cluster_barrier();  // every row's loss is written
    if (blockIdx.x == 0) sum_loss(a, sums);
  }
}

// Rows longer than a cluster's shared memory: one CTA per row reads it twice.
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

// The cluster and ring for a row of `vecs` vectors, or cluster 0 where none
// holds it.
LossPlan plan_loss(int64_t rows, int64_t vecs, int num_sms) {
  constexpr int64_t kMaxSlice = 4864;  // vectors; 76 KB, so that the ring has room beyond a slice
  constexpr int64_t kRingBytes = kRing;
  int64_t cluster = 1;
  while (cluster <= kMaxCluster && cluster * kMaxSlice < vecs) cluster *= 2;
  LossPlan p{};
  if (cluster > kMaxCluster) return p;
  // Small calls: one launch, all rows in one cluster of CTAs with a row each at
  // a time, instead of a second kernel for the sum.
  p.whole = cluster == 1 && rows <= 64 && rows * vecs <= 16384 ? 1 : 0;
  // Few rows: more CTAs for each.
  while (!p.whole && rows * cluster * 2 <= num_sms && cluster < 8 && vecs >= cluster * 2 * 512) cluster *= 2;
  const int64_t slice = std::max<int64_t>(1, (vecs + cluster - 1) / cluster);
  p.cluster = (int)cluster;
  p.slice = (int)slice;
  // Chunks of at most four vectors a thread. All but the last of them exist in
  // every chunk of every slice: those differ by fewer than 26 vectors.
  constexpr int64_t kMost = (int64_t)kMaxThreads * kPerThread;
  p.chunks = (int)((slice + kMost - 1) / kMost);
  p.chunk = (int)((slice + p.chunks - 1) / p.chunks);
  p.per_thread = p.chunk > 2 * kMaxThreads ? kPerThread : p.chunk > kMaxThreads ? 2 : 1;
  p.warps = (int)std::max<int64_t>(2, (p.chunk + 32 * p.per_thread - 1) / (32 * p.per_thread));
  int64_t slots = std::min<int64_t>(kMaxSlots, kRingBytes / ((int64_t)p.chunk * 16));
  if (slots > p.chunks + 3) slots = p.chunks + 3;
  p.slots = (int)slots;
  return p;
}

// How many clusters of a plan run at once on the current device, kept by the
// plan since asking takes longer than a launch.
template <typename T, int PT, bool SAME>
cudaError_t active_clusters(const LossPlan& p, cudaLaunchConfig_t cfg, int num_sms, int* out) {
  struct Known {
    int device, cluster, warps;
    size_t bytes;
    int clusters;
  };
  static std::mutex mu;
  static Known known[16];
  static int count = 0;
  int device = 0;
  cudaError_t e = cudaGetDevice(&device);
  if (e != cudaSuccess) return e;
  std::lock_guard<std::mutex> lock(mu);
  for (int i = 0; i < std::min(count, 16); ++i)
    if (known[i].device == device && known[i].cluster == p.cluster && known[i].warps == p.warps &&
        known[i].bytes == cfg.dynamicSmemBytes) {
      *out = known[i].clusters;
      return cudaSuccess;
    }
  auto kernel = loss_rows_kernel<T, PT, SAME>;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kRing);
  if (e == cudaSuccess) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e != cudaSuccess) return e;
  int clusters = 0;
  if (p.cluster > 1) {
    cfg.gridDim = dim3((unsigned)p.cluster);
    e = cudaOccupancyMaxActiveClusters(&clusters, kernel, &cfg);
  } else {
    e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&clusters, kernel, (int)cfg.blockDim.x, cfg.dynamicSmemBytes);
    clusters *= num_sms;
  }
  if (e != cudaSuccess) return e;
  *out = std::max(clusters, 1);
  known[count++ % 16] = Known{device, p.cluster, p.warps, cfg.dynamicSmemBytes, *out};
  return cudaSuccess;
}

template <typename T, int PT, bool SAME>
cudaError_t launch_rows(const LossArgs& a, const LossPlan& p, int num_sms, cudaStream_t s) {
  cudaLaunchConfig_t cfg{};
  cfg.blockDim = dim3((unsigned)(p.warps * 32 + 32));
  cfg.dynamicSmemBytes = (size_t)p.slots * p.chunk * 16;
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
  cudaError_t e = active_clusters<T, PT, SAME>(p, cfg, num_sms, &clusters);
  if (e != cudaSuccess) return e;
  cfg.gridDim = dim3((unsigned)(p.whole ? kWholeCtas : std::min<int64_t>(clusters, a.rows) * p.cluster));
  e = cudaLaunchKernelEx(&cfg, loss_rows_kernel<T, PT, SAME>, a, p);
  note_launch();
  return e;
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
  if (p.per_thread == 2)
    return same ? launch_rows<T, 2, true>(a, p, num_sms, s) : launch_rows<T, 2, false>(a, p, num_sms, s);
  if (p.per_thread == 1)
    return same ? launch_rows<T, 1, true>(a, p, num_sms, s) : launch_rows<T, 1, false>(a, p, num_sms, s);
  return same ? launch_rows<T, kPerThread, true>(a, p, num_sms, s)
              : launch_rows<T, kPerThread, false>(a, p, num_sms, s);
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
