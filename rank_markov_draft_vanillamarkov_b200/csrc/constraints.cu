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
// first builds the stretch's state in shared memory from the whole history
// (which comes from L2 for all but the first): a count and a prompt bit per
// id, the last bias entry of each id, and a list of the ids that have any of
// these or are drafted. Rows then go by 16-byte vectors, masked and copied,
// eight rows at a time, and the few listed logits of all eight are worked out
// afterwards, one thread for each; within the copy they would cost every warp
// the whole arithmetic for a lane or two.
#include <algorithm>
#include <cmath>

#include "common.cuh"
#include "kernels.h"
#include "ptx.cuh"

namespace dspark {

namespace {

constexpr int kMaxThreads = 512;
constexpr int kInFlight = 4;       // vectors under way per thread
constexpr int kRows = 8;           // rows copied before their listed logits are worked out
constexpr int kListed = 4;         // listed logits in flight per thread
constexpr int kAhead = 8;          // history ids in flight per thread
constexpr int kMinStretch = 512;   // ids
constexpr int kMaxStretch = 32256;
constexpr int kSmem = 222 * 1024;  // dynamic shared memory of a CTA, at most

struct ConstrainPlan {
  int stretch;    // ids per CTA, a multiple of kMinStretch
  int stretches;  // per sequence
  int threads;    // per CTA
  int has_bias;
};

// Bytes of state per kMinStretch ids: counts and bias entries of W bytes each,
// the list, prompt and touched bits.
constexpr int64_t state_bytes(int64_t stretch, int width, bool has_bias) {
  return stretch * (width * (has_bias ? 2 : 1) + 2) + stretch / 8 * 2;
}

// An array of counts, or of the last entry of each id, in shared memory.
// 16-bit elements share the atomics of their 32-bit word.
template <typename C>
struct Cells;
template <>
struct Cells<uint32_t> {
  static __device__ __forceinline__ void add(uint32_t* a, int l) { atomicAdd(&a[l], 1u); }
  static __device__ __forceinline__ void keep_max(uint32_t* a, int l, uint32_t x) { atomicMax(&a[l], x); }
};
template <>
struct Cells<uint16_t> {
  static __device__ __forceinline__ void add(uint16_t* a, int l) {
    atomicAdd(reinterpret_cast<uint32_t*>(a) + (l >> 1), (l & 1) ? 0x10000u : 1u);
  }
  static __device__ __forceinline__ void keep_max(uint16_t* a, int l, uint32_t x) {
    uint32_t* word = reinterpret_cast<uint32_t*>(a) + (l >> 1);
    const int shift = (l & 1) * 16;
    uint32_t seen = *reinterpret_cast<volatile uint32_t*>(word);
    while (((seen >> shift) & 0xffffu) < x) {  // ends: the half only grows, and by whoever wins
      const uint32_t was = atomicCAS(word, seen, (seen & ~(0xffffu << shift)) | (x << shift));
      if (was == seen) break;
      seen = was;
    }
  }
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
__device__ __forceinline__ bool bit(const uint32_t* words, int at) { return (words[at >> 5] >> (at & 31)) & 1u; }

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

__device__ __forceinline__ unsigned long long max_key(unsigned long long a, unsigned long long b) {
  return a > b ? a : b;
}

// C: uint16_t where no count nor bias entry passes 65535, else uint32_t.
// ALIGNED: every row starts at a 16-byte address, in and out.
template <typename T, typename C, bool ALIGNED>
__global__ void __launch_bounds__(kMaxThreads, 2) constrain_kernel(ConstrainArgs a, ConstrainPlan p) {
  constexpr int kE = Vec<T>::kE;
  extern __shared__ __align__(16) uint32_t smem[];
  __shared__ int drafted[kRows];  // local ids (-1: elsewhere) of the tokens drafted after each of the rows
  __shared__ unsigned long long warp_key[kRows][kMaxThreads / 32], listed_key[kRows];
  __shared__ int listed_count;
  const int tid = (int)threadIdx.x, lane = tid & 31, threads = (int)blockDim.x;
  const int64_t b = blockIdx.x / p.stretches;
  const int stretch = (int)(blockIdx.x % p.stretches);
  const int64_t c0 = (int64_t)stretch * p.stretch, rows = a.block;
  const int n = (int)min((int64_t)p.stretch, a.vocab - c0);
  const int words = p.stretch / 32, mask_last = (n + 31) / 32 - 1;
  uint32_t* touched = smem;
  uint32_t* in_prompt = touched + words;
  C* count = reinterpret_cast<C*>(in_prompt + words);
  C* slot = count + p.stretch;  // where there are biases
  uint16_t* list = reinterpret_cast<uint16_t*>(slot + (p.has_bias ? p.stretch : 0));
  auto score = [&](float y, int64_t k, int l) {
    const uint32_t v = (uint32_t)(c0 + l);
    return pack_key(y / a.temperature + noise_for(a.seed, (uint32_t)b, (uint32_t)(a.draft_first + k), v), v);
  };

  // Rows are walked by pointers. A row's stretch is `head` elements before the
  // first 16-byte address, `vecs` vectors, and what is left.
    const T* const in0 = static_cast<const T*>(a.in) + b * a.in_batch + c0;
  T* const out0 = static_cast<T*>(a.out) + b * a.out_batch + c0;
  const uint32_t* const mask0 = a.allowed ? a.allowed + b * a.allowed_batch + (c0 >> 5) : nullptr;
  auto head_of = [&](const T* in, const T* out) {
    if (ALIGNED) return 0;
    const int past = (int)((reinterpret_cast<uintptr_t>(in) / sizeof(T)) % kE);
    const bool same = (reinterpret_cast<uintptr_t>(in) - reinterpret_cast<uintptr_t>(out)) % 16 == 0;
    return same ? min(past ? kE - past : 0, n) : n;  // all single where the output's vectors lie elsewhere
  };
  // The thread's vectors of all rows in one stream: vector tid + q threads of
  // a row, then the next q below `per_row`, then the next row. kInFlight of
  // them are loaded ahead, the first while the state is built. A vector's mask
  // words are shifted when used: a use here would wait for the load.
  const int per_row = max(1, (n / kE + threads - 1) / threads);
  struct Loaded {
    uint4 raw;
    uint32_t lo, hi;
  };
  Loaded ahead[kInFlight];
  const T* load_in = in0;
  const T* load_out = out0;
  const uint32_t* load_mask = mask0;
  int64_t load_left = rows;
  int load_q = per_row, load_j = tid, load_head = head_of(in0, out0);  // load_q counts down
  auto load = [&](Loaded& to) {
    if (load_left <= 0) return;
    if (load_j < (n - load_head) / kE) {
      to.raw = __ldcs(reinterpret_cast<const uint4*>(load_in + load_head) + load_j);
      if (load_mask) {
        const int w = (load_head + load_j * kE) >> 5;
        to.lo = load_mask[w];
        if (!ALIGNED) to.hi = w < mask_last ? load_mask[w + 1] : 0u;
      }
    }
    load_j += threads;
    if (--load_q == 0) {
      load_q = per_row;
      load_j = tid;
      --load_left;
      load_in += a.in_row;
      load_out += a.out_row;
      load_head = head_of(load_in, load_out);
      if (load_mask) load_mask += a.allowed_row;
    }
  };
#pragma unroll
  for (int u = 0; u < kInFlight; ++u) load(ahead[u]);

  // The state. The first ids of the history and of the biases are read while
  // the cells are cleared; the history's before its length is known, which its
  // buffer covers.
  const int64_t cap = a.history ? a.history_cap : 0;
  const int64_t* history = a.history + b * a.history_stride;
  const int64_t* bias_ids = a.bias_ids + b * a.bias_stride;
  const int64_t* draft = a.draft ? a.draft + b * a.draft_stride : nullptr;
  int64_t first_ids[kAhead / 2], first_bias = -1;
#pragma unroll
  for (int u = 0; u < kAhead / 2; ++u) first_ids[u] = tid + u * threads < cap ? history[tid + u * threads] : 0;
  if (tid < a.bias_count) first_bias = bias_ids[tid];
  int64_t len = a.history && a.history_lens ? a.history_lens[b] : cap;
  int64_t prompt = a.prompt_lens ? a.prompt_lens[b] : 0;
  if (tid == 0) listed_count = 0;
  {
    uint4* cells = reinterpret_cast<uint4*>(in_prompt);
    const int vecs = (words * 4 + p.stretch * (int)sizeof(C) * (p.has_bias ? 2 : 1)) / 16;
    for (int i = tid; i < vecs; i += threads) cells[i] = make_uint4(0u, 0u, 0u, 0u);
  }
  len = min(max(len, (int64_t)0), cap);
  prompt = min(max(prompt, (int64_t)0), len);
  __syncthreads();
  bool bad = false;
  auto note_token = [&](int64_t id, int64_t i) {
    const uint64_t l = (uint64_t)(id - c0);
    if (l < (uint64_t)n) {
      if (i < prompt)
        atomicOr(&in_prompt[l >> 5], 1u << (l & 31));
      else
        Cells<C>::add(count, (int)l);
    }
    if ((uint64_t)id >= (uint64_t)a.vocab) bad = true;
  };
  auto note_bias = [&](int64_t id, int64_t i) {
    const uint64_t l = (uint64_t)(id - c0);
    if (l < (uint64_t)n) Cells<C>::keep_max(slot, (int)l, (uint32_t)i + 1u);
    if (id >= a.vocab) bad = true;
  };
#pragma unroll
  for (int u = 0; u < kAhead / 2; ++u)
    if (tid + u * threads < len) note_token(first_ids[u], tid + u * threads);
  for (int64_t i = tid + threads * (kAhead / 2); i < len; i += (int64_t)threads * kAhead) {
    int64_t id[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) id[u] = i + u * threads < len ? history[i + u * threads] : 0;
#pragma unroll
    for (int u = 0; u < kAhead; ++u)
      if (i + u * threads < len) note_token(id[u], i + u * threads);
  }
  if (draft) {
    for (int64_t i = tid; i < a.draft_first; i += threads) {
      const int64_t id = draft[i];
      const uint64_t l = (uint64_t)(id - c0);
      if (l < (uint64_t)n) Cells<C>::add(count, (int)l);
      if (id >= a.vocab) bad = true;
    }
  }
  if (tid < a.bias_count) note_bias(first_bias, tid);
  for (int64_t i = tid + threads; i < a.bias_count; i += threads) note_bias(bias_ids[i], i);
  __syncthreads();
  // A thread looks at 32 ids and keeps their bits; the warp then takes its
  // places in the list at once.
  for (int w0 = (tid >> 5) * 32; w0 < words; w0 += threads) {
    const int w = w0 + lane;
    uint32_t word = 0u;
    if (w < words) {
      word = in_prompt[w];
      constexpr int kPer = 16 / sizeof(C);  // cells of 16 bytes
      auto look = [&](const C* cells) {
#pragma unroll
        for (int i = 0; i < 32 / kPer; ++i) {
          const uint4 x = *reinterpret_cast<const uint4*>(cells + w * 32 + i * kPer);
          if (x.x | x.y | x.z | x.w) {
#pragma unroll
            for (int e = 0; e < kPer; ++e) {
              const uint32_t v = sizeof(C) == 4 ? (e == 0 ? x.x : e == 1 ? x.y : e == 2 ? x.z : x.w)
                                                : ((e < 2 ? x.x : e < 4 ? x.y : e < 6 ? x.z : x.w) >> (16 * (e & 1))) & 0xffffu;
              if (v) word |= 1u << (i * kPer + e);
            }
          }
        }
      };
      look(count);
      if (p.has_bias) look(slot);
      touched[w] = word;
    }
    const int mine = __popc(word);
    int sum = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int before = __shfl_up_sync(0xffffffffu, sum, o);
      if (lane >= o) sum += before;
    }
    int base = 0;
    if (lane == 31 && sum) base = atomicAdd(&listed_count, sum);
    base = __shfl_sync(0xffffffffu, base, 31) + sum - mine;
    for (; word; word &= word - 1u) list[base++] = (uint16_t)(w * 32 + __ffs((int)word) - 1);
  }
  const float rho = a.repetition ? a.repetition[b] : a.repetition_value;
  const float freq = a.frequency ? a.frequency[b] : a.frequency_value;
  const float pres = a.presence ? a.presence[b] : a.presence_value;
  const float* bias = a.bias_values + b * a.bias_stride;
  __syncthreads();

  for (int64_t k0 = 0; k0 < rows; k0 += kRows) {
    const int group = (int)min((int64_t)kRows, rows - k0);
    // The last rows' drafted tokens join the counts. Those of these rows are
    // laid out and listed, which changes nothing for rows before them.
    if (draft && tid == 0) {
      for (int q = 0; k0 > 0 && q < kRows; ++q)
        if (drafted[q] >= 0) count[drafted[q]] += 1;
      for (int q = 0; q < kRows; ++q) {
        const int64_t id = k0 + q < rows - 1 ? draft[a.draft_first + k0 + q] : -1;
        if (id >= a.vocab) bad = true;
        const int64_t l = id - c0;
        const bool here = id >= 0 && l >= 0 && l < n;
        drafted[q] = here ? (int)l : -1;
        if (here && !bit(touched, (int)l)) {
          touched[l >> 5] |= 1u << (l & 31);
          list[listed_count++] = (uint16_t)l;
        }
      }
    }
    if (tid < kRows) listed_key[tid] = 0ull;
    __syncthreads();

    const T* in = in0 + k0 * a.in_row;
    T* out = out0 + k0 * a.out_row;
    const uint32_t* mask = mask0 ? mask0 + k0 * a.allowed_row : nullptr;

    // The copy. Greedy keys: the largest value so far, the vector (and its
    // first id) that holds it; a single element is a vector of its own. A row
    // of -inf alone keeps the first threads' own ids, of which the lowest
    // wins. Listed logits stand aside as -inf.
    float best = -INFINITY;
    int best_at = tid < n ? tid : -1;
    uint4 best_vec = make_uint4(0u, 0u, 0u, 0u);
    bool best_single = true;
    unsigned long long key = 0ull;
    // Strictly larger, or the first NaN: ids rise, so equal values keep the lower one.
    auto better = [&](float y) { return y > best || (y != y && best == best); };
    auto single = [&](int64_t k, int l) {
      const T y = !mask || bit(mask, l) ? in[l] : from_f32<T>(-INFINITY);
      out[l] = y;
      if (!a.keys || bit(touched, l)) return;
      if (!a.greedy) {
        key = max_key(key, score(to_f32(y), k, l));
      } else if (better(to_f32(y))) {
        best = to_f32(y);
        best_at = l;
        best_single = true;
      }
    };
    int r = 0, q = per_row, j = tid, head = head_of(in, out);  // q counts down
    while (r < group) {
#pragma unroll
      for (int u = 0; u < kInFlight; ++u) {
        if (r >= group) break;
        if (!ALIGNED && q == per_row)
          for (int l = tid; l < head; l += threads) single(k0 + r, l);
        const int l = head + j * kE;
        if (j < (n - head) / kE) {
          uint4 raw = ahead[u].raw;
          if (mask)
            raw = Vec<T>::masked(raw, ALIGNED ? ahead[u].lo >> (l & 31)
                                              : __funnelshift_r(ahead[u].lo, ahead[u].hi, l & 31));
          __stcs(reinterpret_cast<uint4*>(out + head) + j, raw);
          if (a.keys) {
            raw = Vec<T>::masked(raw, ~bits_at<ALIGNED>(touched, l, words - 1));
            if (a.greedy) {
              const float top = Vec<T>::max_of(raw);
              if (better(top)) {
                best = top;
                best_at = l;
                best_vec = raw;
                best_single = false;
              }
            } else {
#pragma unroll
              for (int e = 0; e < kE; ++e) key = max_key(key, score(Vec<T>::get(raw, e), k0 + r, l + e));
            }
          }
        }
        load(ahead[u]);
        j += threads;
        if (--q == 0) {
          for (int t = head + (n - head) / kE * kE + tid; t < n; t += threads) single(k0 + r, t);
          if (a.keys) {
            if (a.greedy && best_at >= 0) {
              if (!best_single) {
                int first = kE;
#pragma unroll
                for (int e = kE - 1; e >= 0; --e) {
                  const float y = Vec<T>::get(best_vec, e);
                  if (y == best || (y != y && best != best)) first = e;
                }
                best_at += first;
              }
              key = pack_key(best, (uint32_t)(c0 + best_at));
            }
            // The warp's largest key: the larger high word, then the larger low one.
            const uint32_t high = __reduce_max_sync(0xffffffffu, (uint32_t)(key >> 32));
            const uint32_t low = __reduce_max_sync(0xffffffffu, (uint32_t)(key >> 32) == high ? (uint32_t)key : 0u);
            if (lane == 0) warp_key[r][tid >> 5] = ((unsigned long long)high << 32) | low;
            best = -INFINITY;
            best_at = tid < n ? tid : -1;
            best_single = true;
            key = 0ull;
          }
          q = per_row;
          j = tid;
          ++r;
          in += a.in_row;
          out += a.out_row;
          if (mask) mask += a.allowed_row;
          head = head_of(in, out);
        }
      }
    }
    __syncthreads();

    // The listed logits of these rows, after the copies of them. What the copy
    // left in place of a masked one stays; in place, an allowed one's input is
    // what the copy wrote.
    const int listed = listed_count, items = listed * group;
    for (int i0 = tid; i0 < items; i0 += threads * kListed) {
      T x[kListed];
      uint32_t word[kListed];
#pragma unroll
      for (int u = 0; u < kListed; ++u) {
        const int item = min(i0 + u * threads, items - 1), g = item / listed;
        const int64_t k = k0 + g;
        const int l = (int)list[item - g * listed];
        x[u] = in0[k * a.in_row + l];
        word[u] = mask0 ? mask0[k * a.allowed_row + (l >> 5)] : ~0u;
      }
#pragma unroll
      for (int u = 0; u < kListed; ++u) {
        const int item = i0 + u * threads;
        if (item >= items) break;
        const int g = item / listed;
        const int64_t k = k0 + g;
        const int l = (int)list[item - g * listed];
        if (!((word[u] >> (l & 31)) & 1u)) continue;
        uint32_t times = (uint32_t)count[l];
        if (draft) {
#pragma unroll
          for (int d = 0; d < kRows - 1; ++d) times += d < g && drafted[d] == l ? 1u : 0u;
        }
        float f = to_f32(x[u]);
        if (times || bit(in_prompt, l)) f = f > 0.0f ? __fdiv_rn(f, rho) : __fmul_rn(f, rho);
        if (times) f = __fsub_rn(__fsub_rn(f, __fmul_rn(freq, (float)times)), pres);
        if (p.has_bias && slot[l]) f = __fadd_rn(f, bias[(uint32_t)slot[l] - 1u]);
        const T y = from_f32<T>(f);
        out0[k * a.out_row + l] = y;
        if (a.keys) {
          const unsigned long long mine = a.greedy ? pack_key(to_f32(y), (uint32_t)(c0 + l)) : score(to_f32(y), k, l);
          if (mine > *reinterpret_cast<volatile unsigned long long*>(&listed_key[g])) atomicMax(&listed_key[g], mine);
        }
      }
    }
    __syncthreads();
    if (a.keys && tid < group) {
      unsigned long long top = listed_key[tid];
      for (int w = 0; w < threads / 32; ++w) top = max_key(top, warp_key[tid][w]);
      a.keys[(b * rows + k0 + tid) * p.stretches + stretch] = top;
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

// The stretches for which the waves of CTAs take least. A CTA's cost, in ids:
// its own ids for each row and once for the state, and a fixed part for its
// start and the history, which all CTAs of a sequence read whole. CTAs that
// share an SM share its rate.
ConstrainPlan plan_constrain(const ConstrainArgs& a, int width, int num_sms) {
  ConstrainPlan best{};
  best.has_bias = a.bias_count > 0 ? 1 : 0;
  int64_t best_cost = INT64_MAX;
  const int64_t fixed = 4096 + (a.history ? a.history_cap / 4 : 0), passes = std::min<int64_t>(a.block, 1024) + 1;
  const auto consider = [&](int64_t stretches) {
    const int64_t least = (a.vocab + kMaxStretch - 1) / kMaxStretch;
    stretches = std::max<int64_t>(least, std::min<int64_t>(stretches, (a.vocab + kMinStretch - 1) / kMinStretch));
    const int64_t stretch = ((a.vocab + stretches - 1) / stretches + kMinStretch - 1) / kMinStretch * kMinStretch;
    const int64_t real = (a.vocab + stretch - 1) / stretch;
    const int64_t bytes = state_bytes(stretch, width, best.has_bias != 0);
    if (bytes > kSmem) return;
    const int64_t threads = std::min<int64_t>(kMaxThreads, std::max<int64_t>(64, stretch / 16)) / 32 * 32;
    const int64_t per_sm = std::min<int64_t>(1024 / threads, (227 * 1024) / (bytes + 2304));
    const int64_t waves = (a.batch * real + per_sm * num_sms - 1) / (per_sm * num_sms);
    const int64_t shared = std::min(per_sm, (a.batch * real + num_sms - 1) / num_sms);
    const int64_t cost = waves * shared * (fixed + stretch * passes);
    if (cost < best_cost) {
      best_cost = cost;
      best.stretch = (int)stretch;
      best.stretches = (int)real;
      best.threads = (int)threads;
    }
  };
  for (int64_t ctas = 1; ctas <= 8; ++ctas) consider(ctas * num_sms / a.batch);  // per SM, in all
  consider((a.vocab + kMaxStretch / 4 - 1) / (kMaxStretch / 4));
  return best;
}

template <typename T, typename C>
cudaError_t launch_typed(const ConstrainArgs& a, int num_sms, cudaStream_t s, ConstrainPlan* plan) {
  const auto whole = [&a](const void* base, int64_t batch, int64_t row) {
    constexpr int64_t kE = Vec<T>::kE;
    return reinterpret_cast<uintptr_t>(base) % 16 == 0 && (a.batch == 1 || batch % kE == 0) &&
           (a.block == 1 || row % kE == 0);
  };
  const bool aligned = whole(a.in, a.in_batch, a.in_row) && whole(a.out, a.out_batch, a.out_row);
  auto kernel = aligned ? constrain_kernel<T, C, true> : constrain_kernel<T, C, false>;
  const ConstrainPlan p = plan_constrain(a, (int)sizeof(C), num_sms);
  *plan = p;
  if (a.batch * p.stretches > 0x7fffffffll) return cudaErrorInvalidConfiguration;
  const size_t bytes = (size_t)state_bytes(p.stretch, (int)sizeof(C), p.has_bias != 0);
  if (bytes > 40 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e != cudaSuccess) return e;
  }
  kernel<<<(unsigned)(a.batch * p.stretches), p.threads, bytes, s>>>(a, p);
  note_launch();
  return cudaGetLastError();
}

}  // namespace

int64_t constrain_key_count(int64_t batch, int64_t block, int64_t vocab) {
  return batch * block * ((vocab + kMinStretch - 1) / kMinStretch);
}

cudaError_t launch_constrain(const ConstrainArgs& a, int logits_dtype, int num_sms, cudaStream_t s) {
  if (a.batch * a.block > 0x7fffffffll) return cudaErrorInvalidConfiguration;
  // The most that one id can count, and the largest bias entry.
  const int64_t most = (a.history ? a.history_cap : 0) + a.draft_first + a.block;
  const bool narrow = most <= 0xffff && a.bias_count <= 0xfffe;
  ConstrainPlan p{};
  cudaError_t e;
  if (logits_dtype == DSPARK_DTYPE_FP32)
    e = narrow ? launch_typed<float, uint16_t>(a, num_sms, s, &p) : launch_typed<float, uint32_t>(a, num_sms, s, &p);
  else
    e = narrow ? launch_typed<__nv_bfloat16, uint16_t>(a, num_sms, s, &p)
               : launch_typed<__nv_bfloat16, uint32_t>(a, num_sms, s, &p);
  if (e != cudaSuccess || !a.keys) return e;
  choose_kernel<<<(unsigned)(a.batch * a.block), 32, 0, s>>>(a, p.stretches);
  note_launch();
  return cudaGetLastError();
}

}  // namespace dspark
