// Token constraints on corrected logits: penalties for repeated tokens,
// additive biases and grammar masks, with the choice of every row.
//
// For row (b, k) with corrected logit c_v, n_v generated occurrences of v (in
// sequence b's history past its prompt and among the drafted tokens before
// position k) and s_v = n_v > 0 or v in the prompt:
//
//   x = c_v;  if s_v: x = x > 0 ? x / rho : x * rho;  x -= f n_v;
//   if n_v > 0: x -= p;  x += beta_v;  if v is not allowed: x = -inf
//
// each operation in fp32, one rounding to the logits dtype at the end.
//
// Almost every logit only passes through, so the bound is the copy: 4 bytes
// per bf16 logit and an eighth of a byte of mask. A CTA takes one stretch of
// the vocabulary of one sequence and walks that sequence's rows over it. It
// first builds the stretch's state in shared memory: a word per id (prompt
// bit and count), the last bias entry of each id, and one bit per id that has
// either. Rows then go by 16-byte vectors: a mask byte and a byte of those
// bits decide for eight logits at once. The history is read once per cluster:
// its CTAs share the reading and send each id to the CTA that owns it.
#include <algorithm>
#include <cmath>

#include "common.cuh"
#include "kernels.h"
#include "ptx.cuh"

namespace dspark {

namespace {

constexpr int kThreads = 256;
constexpr int kBatch = 4;                     // vectors in flight per thread
constexpr int kAhead = 4;                     // history ids in flight per thread
constexpr int kMinStretch = 1024;             // ids
constexpr int kMaxStretch = 8192;
constexpr uint32_t kPromptBit = 0x80000000u;  // count word: seen in the prompt; low bits: generated occurrences

struct ConstrainPlan {
  int stretch;    // ids per CTA, a power of two from kMinStretch
  int shift;      // its logarithm
  int stretches;  // per sequence, rounded up to whole clusters
  int cluster;    // CTAs that share the reading of a history
  int has_bias;
};

// The bits of a bit string from bit `at` on. Where `at` is a multiple of 8 the
// first eight lie in one word.
template <bool ALIGNED>
__device__ __forceinline__ uint32_t bits_at(const uint32_t* words, int at, int last_word) {
  const int w = at >> 5;
  if (ALIGNED) return words[w] >> (at & 31);
  const uint32_t lo = words[w], hi = w < last_word ? words[w + 1] : 0u;
  return __funnelshift_r(lo, hi, at & 31);
}

// Bits 0..3 of n as all-ones or zero halves of two words: element 2i in the
// low half of word i. The product spreads the bits to the signs of four bytes
// (no two partial products share a position), which are then replicated.
__device__ __forceinline__ void half_masks(uint32_t n, uint32_t* m0, uint32_t* m1) {
  const uint32_t signs = (n & 15u) * 0x10204080u;
  asm("prmt.b32 %0, %1, 0, 0x9988;" : "=r"(*m0) : "r"(signs));
  asm("prmt.b32 %0, %1, 0, 0xbbaa;" : "=r"(*m1) : "r"(signs));
}

template <typename T>
struct Vec;
template <>
struct Vec<float> {
  static constexpr int kE = 4;
  static __device__ __forceinline__ uint4 masked(const uint4& r, uint32_t allowed) {
    return make_uint4((allowed & 1u) ? r.x : 0xff800000u, (allowed & 2u) ? r.y : 0xff800000u,
                      (allowed & 4u) ? r.z : 0xff800000u, (allowed & 8u) ? r.w : 0xff800000u);
  }
  static __device__ __forceinline__ float get(const uint4& r, int e) {
    return __uint_as_float(e == 0 ? r.x : e == 1 ? r.y : e == 2 ? r.z : r.w);
  }
  static __device__ __forceinline__ void set(uint4& r, int e, float x) {
    const uint32_t b = __float_as_uint(x);
    if (e == 0) r.x = b;
    if (e == 1) r.y = b;
    if (e == 2) r.z = b;
    if (e == 3) r.w = b;
  }
  // The largest element; NaN if there is one.
  static __device__ __forceinline__ float max_of(const uint4& r) {
    float m = get(r, 0);
#pragma unroll
    for (int e = 1; e < 4; ++e) {
      const float x = get(r, e);
      m = (x > m || x != x) ? x : m;  // a NaN in m compares false and stays
    }
    return m;
  }
};
template <>
struct Vec<__nv_bfloat16> {
  static constexpr int kE = 8;
  static __device__ __forceinline__ uint4 masked(const uint4& r, uint32_t allowed) {
    uint32_t m0, m1, m2, m3;
    half_masks(allowed, &m0, &m1);
    half_masks(allowed >> 4, &m2, &m3);
    constexpr uint32_t kInf = 0xff80ff80u;
    return make_uint4((r.x & m0) | (kInf & ~m0), (r.y & m1) | (kInf & ~m1), (r.z & m2) | (kInf & ~m2),
                      (r.w & m3) | (kInf & ~m3));
  }
  static __device__ __forceinline__ float get(const uint4& r, int e) {
    const uint32_t w = (e >> 1) == 0 ? r.x : (e >> 1) == 1 ? r.y : (e >> 1) == 2 ? r.z : r.w;
    return __uint_as_float((e & 1) ? (w & 0xffff0000u) : (w << 16));
  }
  static __device__ __forceinline__ void set(uint4& r, int e, float x) {
    const uint32_t b = __bfloat16_as_ushort(__float2bfloat16_rn(x));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t& w = i == 0 ? r.x : i == 1 ? r.y : i == 2 ? r.z : r.w;
      if ((e >> 1) == i) w = (e & 1) ? (w & 0xffffu) | (b << 16) : (w & 0xffff0000u) | b;
    }
  }
  static __device__ __forceinline__ float max_of(const uint4& r) {
    const auto p = [](uint32_t w) { return *reinterpret_cast<const __nv_bfloat162*>(&w); };
    const __nv_bfloat162 m = __hmax2_nan(__hmax2_nan(p(r.x), p(r.y)), __hmax2_nan(p(r.z), p(r.w)));
    const float a = __low2float(m), b = __high2float(m);
    return (b > a || b != b) ? b : a;
  }
};

// One logit with its state.
struct Penalty {
  float repetition, frequency, presence;
  __device__ __forceinline__ float apply(float x, uint32_t count) const {
    const uint32_t times = count & ~kPromptBit;
    if (count) x = x > 0.0f ? __fdiv_rn(x, repetition) : __fmul_rn(x, repetition);
    if (times) x = __fsub_rn(__fsub_rn(x, __fmul_rn(frequency, (float)times)), presence);
    return x;
  }
};

__device__ __forceinline__ unsigned long long max_key(unsigned long long a, unsigned long long b) {
  return a > b ? a : b;
}

template <typename T, bool ALIGNED>
__global__ void __launch_bounds__(kThreads, 3) constrain_kernel(ConstrainArgs a, ConstrainPlan p) {
  constexpr int kE = Vec<T>::kE;
  extern __shared__ __align__(16) uint32_t smem[];
  __shared__ unsigned long long warp_best[2][kThreads / 32];
  const int tid = (int)threadIdx.x, lane = tid & 31;
  const int64_t b = blockIdx.x / p.stretches;
  const int stretch = (int)(blockIdx.x % p.stretches);
  const int64_t c0 = (int64_t)stretch * p.stretch;
  const int n = (int)max((int64_t)0, min((int64_t)p.stretch, a.vocab - c0));  // none in a cluster's last CTAs, perhaps
  const int rank = p.cluster > 1 ? (int)cluster_rank() : 0;
  uint32_t* touched = smem;                     // stretch / 32 words
  uint32_t* count = touched + p.stretch / 32;   // stretch words
  uint32_t* slot = count + p.stretch;           // stretch words where there are biases

  const int64_t rows = a.block;

  // A row's place: elements before the first 16-byte address, vectors, and
  // what is left. Loads run one batch of vectors ahead, so that the first is
  // under way while the state is built.
  struct Row {
    const T* in;
    T* out;
    const uint32_t* mask;
    int head, vecs;
  };
  const int mask_last = (n + 31) / 32 - 1;
  auto row_at = [&](int64_t k) {
    Row r;
    r.in = static_cast<const T*>(a.in) + b * a.in_batch + k * a.in_row + c0;
    r.out = static_cast<T*>(a.out) + b * a.out_batch + k * a.out_row + c0;
    r.mask = a.allowed ? a.allowed + b * a.allowed_batch + k * a.allowed_row + (c0 >> 5) : nullptr;
    r.head = 0;
    if (!ALIGNED) {
      const int past = (int)((reinterpret_cast<uintptr_t>(r.in) / sizeof(T)) % kE);
      const bool same = (reinterpret_cast<uintptr_t>(r.in) - reinterpret_cast<uintptr_t>(r.out)) % 16 == 0;
      r.head = same ? min(past ? kE - past : 0, n) : n;  // all single where the output's vectors lie elsewhere
    }
    r.vecs = (n - r.head) / kE;
    return r;
  };
  uint4 ahead[kBatch];
  uint32_t ahead_allowed[kBatch];
  auto load = [&](const Row& r, int j0) {
#pragma unroll
    for (int q = 0; q < kBatch; ++q) {
      const int j = j0 + tid + q * kThreads;
      if (j < r.vecs) {
        ahead[q] = __ldcs(reinterpret_cast<const uint4*>(r.in + r.head) + j);
        ahead_allowed[q] = r.mask ? bits_at<ALIGNED>(r.mask, r.head + j * kE, mask_last) : ~0u;
      }
    }
  };
  Row row = row_at(0);
  load(row, 0);

  for (int i = tid * 4; i < p.stretch; i += kThreads * 4) {
    *reinterpret_cast<uint4*>(count + i) = make_uint4(0u, 0u, 0u, 0u);
    if (p.has_bias) *reinterpret_cast<uint4*>(slot + i) = make_uint4(0u, 0u, 0u, 0u);
  }
  if (p.cluster > 1)
    cluster_barrier();
  else
    __syncthreads();

  bool bad = false;
  const int64_t cap = a.history ? a.history_cap : 0;
  int64_t len = cap;
  if (a.history && a.history_lens) len = min(max(a.history_lens[b], (int64_t)0), cap);
  const int64_t prompt = a.prompt_lens ? min(max(a.prompt_lens[b], (int64_t)0), len) : 0;
  const int64_t first = c0 - (int64_t)rank * p.stretch;  // the cluster's first id
  auto note = [&](int64_t id, bool generated) {
    const int64_t l = id - first;
    if (l < 0 || l >= (int64_t)p.stretch * p.cluster || id >= a.vocab) return;
    const int owner = (int)l >> p.shift, at = (int)l & (p.stretch - 1);
    if (p.cluster == 1) {
      if (generated)
        atomicAdd(&count[at], 1u);
      else
        atomicOr(&count[at], kPromptBit);
    } else {
      const uint32_t where = remote_u32(&count[at], (uint32_t)owner);
      if (generated)
        asm volatile("red.relaxed.cluster.shared::cluster.add.u32 [%0], %1;" ::"r"(where), "r"(1u) : "memory");
      else
        asm volatile("red.relaxed.cluster.shared::cluster.or.b32 [%0], %1;" ::"r"(where), "r"(kPromptBit) : "memory");
    }
  };
  const int64_t* history = a.history + b * a.history_stride;
  const int64_t readers = (int64_t)kThreads * p.cluster;
  for (int64_t i = (int64_t)rank * kThreads + tid; i < len; i += readers * kAhead) {
    int64_t ids[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) ids[u] = i + u * readers < len ? history[i + u * readers] : 0;
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      if (i + u * readers >= len) break;
      if (ids[u] < 0 || ids[u] >= a.vocab) bad = true;
      note(ids[u], i + u * readers >= prompt);
    }
  }
  const int64_t* draft = a.draft ? a.draft + b * a.draft_stride : nullptr;
  for (int64_t i = (int64_t)rank * kThreads + tid; draft && i < a.draft_first; i += (int64_t)kThreads * p.cluster) {
    const int64_t id = draft[i];
    if (id >= a.vocab) bad = true;
    if (id >= 0) note(id, true);
  }
  for (int64_t i = tid; i < a.bias_count; i += kThreads) {
    const int64_t id = a.bias_ids[b * a.bias_stride + i];
    if (id >= a.vocab) bad = true;
    const int64_t l = id - c0;
    if (l >= 0 && l < n) atomicMax(&slot[l], (uint32_t)i + 1u);
  }
  if (p.cluster > 1)
    cluster_barrier();
  else
    __syncthreads();
  for (int i = tid; i < p.stretch; i += kThreads) {  // whole warps: the stretch is a multiple of 32
    const bool any = count[i] != 0u || (p.has_bias && slot[i] != 0u);
    const uint32_t word = __ballot_sync(0xffffffffu, any);
    if (lane == 0) touched[i >> 5] = word;
  }
  const Penalty penalty{a.repetition ? a.repetition[b] : a.repetition_value,
                        a.frequency ? a.frequency[b] : a.frequency_value,
                        a.presence ? a.presence[b] : a.presence_value};
  const float* bias = a.bias_values + b * a.bias_stride;
  auto one = [&](float x, int l) {  // the state of local id l applied to a logit
    x = penalty.apply(x, count[l]);
    if (p.has_bias) {
      const uint32_t entry = slot[l];
      if (entry) x = __fadd_rn(x, bias[entry - 1u]);
    }
    return x;
  };
  __syncthreads();

  for (int64_t k = 0; k < rows; ++k) {
    if (k > 0 && draft) {  // the token drafted before this row joins the history
      if (tid == 0) {
        const int64_t id = draft[a.draft_first + k - 1];
        if (id >= a.vocab) bad = true;
        const int64_t l = id - c0;
        if (l >= 0 && l < n) {
          count[l] += 1u;
          touched[l >> 5] |= 1u << (l & 31);
        }
      }
      __syncthreads();
    }
    // Greedy: the largest so far and its local id. A row of -inf alone keeps
    // the first threads' own ids, of which the lowest wins.
    float best = -INFINITY;
    int best_at = tid < n ? tid : -1;
    unsigned long long key = 0ull;
    auto consider = [&](float y, int l) {
      if (a.greedy) {
        // Strictly larger, or a first NaN: ids rise, so equal values keep the lower one.
        if (y > best || (y != y && best == best)) {
          best = y;
          best_at = l;
        }
      } else {
        const uint32_t v = (uint32_t)(c0 + l);
        key = max_key(key, pack_key(y / a.temperature + noise_for(a.seed, (uint32_t)b, (uint32_t)(a.draft_first + k), v), v));
      }
    };
    auto scalar = [&](int l) {
      float x = one(to_f32(row.in[l]), l);
      if (row.mask && !((row.mask[l >> 5] >> (l & 31)) & 1u)) x = -INFINITY;
      const T y = from_f32<T>(x);
      row.out[l] = y;
      if (a.keys) consider(to_f32(y), l);
    };
    if (!ALIGNED)
      for (int l = tid; l < row.head; l += kThreads) scalar(l);
    uint4* to = reinterpret_cast<uint4*>(row.out + row.head);
    const Row next = row_at(k + 1 < rows ? k + 1 : k);
    int j0 = 0;
    do {
      uint4 raw[kBatch];
      uint32_t allowed[kBatch];
#pragma unroll
      for (int q = 0; q < kBatch; ++q) {
        raw[q] = ahead[q];
        allowed[q] = ahead_allowed[q];
      }
      const int j1 = j0 + kThreads * kBatch;
      if (j1 < row.vecs)
        load(row, j1);
      else if (k + 1 < rows)
        load(next, 0);
#pragma unroll
      for (int q = 0; q < kBatch; ++q) {
        const int j = j0 + tid + q * kThreads;
        if (j >= row.vecs) break;
        const int l = row.head + j * kE;
        uint32_t t = bits_at<ALIGNED>(touched, l, p.stretch / 32 - 1) & ((1u << kE) - 1u) & allowed[q];
        for (; t; t &= t - 1u) {
          const int e = __ffs((int)t) - 1;
          Vec<T>::set(raw[q], e, one(Vec<T>::get(raw[q], e), l + e));
        }
        if (row.mask) raw[q] = Vec<T>::masked(raw[q], allowed[q]);
        __stcs(to + j, raw[q]);
        // Most vectors hold nothing larger than the thread's best.
        if (a.keys && !(a.greedy && Vec<T>::max_of(raw[q]) <= best)) {
#pragma unroll
          for (int e = 0; e < kE; ++e) consider(Vec<T>::get(raw[q], e), l + e);
        }
      }
      j0 = j1;
    } while (j0 < row.vecs);
    for (int l = row.head + row.vecs * kE + tid; l < n; l += kThreads) scalar(l);
    row = next;
    if (a.keys) {
      if (a.greedy && best_at >= 0) key = pack_key(best, (uint32_t)(c0 + best_at));
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) key = max_key(key, __shfl_xor_sync(0xffffffffu, key, o));
      // Two buffers: the row before last was read before the barrier of the last.
      if (lane == 0) warp_best[k & 1][tid >> 5] = key;
      __syncthreads();
      if (tid == 0) {
        for (int w = 1; w < kThreads / 32; ++w) key = max_key(key, warp_best[k & 1][w]);
        a.keys[(b * rows + k) * p.stretches + stretch] = key;
      }
    } else {
      __syncthreads();  // the next draft token's count comes after this row's reads
    }
  }
  if (bad) report_status(a.status, DSPARK_STATUS_TOKEN_RANGE);
}

// The token of each row: the id in the largest of its stretches' keys.
__global__ void __launch_bounds__(32) choose_kernel(ConstrainArgs a, int stretches) {
  const int64_t row = blockIdx.x;
  unsigned long long best = 0ull;
  for (int i = threadIdx.x; i < stretches; i += 32) best = max_key(best, a.keys[row * stretches + i]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) best = max_key(best, __shfl_xor_sync(0xffffffffu, best, o));
  if (threadIdx.x == 0) a.tokens[row / a.block * a.tokens_batch + row % a.block] = (int64_t)key_token(best);
}

ConstrainPlan plan_constrain(const ConstrainArgs& a, int num_sms) {
  ConstrainPlan p{};
  p.has_bias = a.bias_count > 0 ? 1 : 0;
  // Stretches small enough for two CTAs per SM's worth of them.
  p.stretch = kMaxStretch;
  p.shift = 13;
  static_assert(kMaxStretch == 1 << 13, "the logarithm above");
  while (p.stretch > kMinStretch && a.batch * ((a.vocab + p.stretch - 1) / p.stretch) < 2ll * num_sms) {
    p.stretch /= 2;
    --p.shift;
  }
  const int64_t stretches = (a.vocab + p.stretch - 1) / p.stretch;
  p.cluster = 1;
  while (p.cluster < 8 && a.history && a.history_cap > 512ll * p.cluster && stretches >= p.cluster * 2) p.cluster *= 2;
  p.stretches = (int)((stretches + p.cluster - 1) / p.cluster * p.cluster);
  return p;
}

template <typename T>
cudaError_t launch_typed(const ConstrainArgs& a, const ConstrainPlan& p, cudaStream_t s) {
  const auto whole = [](const void* base, int64_t batch, int64_t row, const ConstrainArgs& c) {
    constexpr int64_t kE = Vec<T>::kE;
    return reinterpret_cast<uintptr_t>(base) % 16 == 0 && (c.batch == 1 || batch % kE == 0) &&
           (c.block == 1 || row % kE == 0);
  };
  const bool aligned = whole(a.in, a.in_batch, a.in_row, a) && whole(a.out, a.out_batch, a.out_row, a);
  auto kernel = aligned ? constrain_kernel<T, true> : constrain_kernel<T, false>;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(a.batch * p.stretches));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = (size_t)p.stretch / 8 + (size_t)p.stretch * 4 * (p.has_bias ? 2 : 1);
  cfg.stream = s;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim = {(unsigned)p.cluster, 1, 1};
  cfg.attrs = &attr;
  cfg.numAttrs = p.cluster > 1 ? 1 : 0;
  if (cfg.dynamicSmemBytes > 48 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 68 * 1024);
    if (e != cudaSuccess) return e;
  }
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, a, p);
  note_launch();
  return e;
}

}  // namespace

int64_t constrain_key_count(int64_t batch, int64_t block, int64_t vocab) {
  return batch * block * ((vocab + kMinStretch - 1) / kMinStretch + 8);
}

cudaError_t launch_constrain(const ConstrainArgs& a, int logits_dtype, int num_sms, cudaStream_t s) {
  const ConstrainPlan p = plan_constrain(a, num_sms);
  if (a.batch * p.stretches > 0x7fffffffll || a.batch * a.block > 0x7fffffffll) return cudaErrorInvalidConfiguration;
  cudaError_t e = logits_dtype == DSPARK_DTYPE_FP32 ? launch_typed<float>(a, p, s) : launch_typed<__nv_bfloat16>(a, p, s);
  if (e != cudaSuccess || !a.keys) return e;
  choose_kernel<<<(unsigned)(a.batch * a.block), 32, 0, s>>>(a, p.stretches);
  note_launch();
  return cudaGetLastError();
}

}  // namespace dspark
