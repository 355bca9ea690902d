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
// per bf16 logit and an eighth of a byte of mask. Two kernels:
//
//   list_kernel  finds the ids of each sequence that have a state at all (in
//                the history, biased, drafted) and writes them with it, in
//                order of the ids. A CTA takes a part of the vocabulary, as
//                much as its shared memory can count, and reads the history.
//   copy_kernel  masks and copies the rows by 16-byte vectors, a stretch of
//                the vocabulary of one sequence per CTA and up to eight rows
//                at a time, then works out the listed logits of those rows,
//                one thread for each.
//
// Measured, 32 x 8 rows of 151936 bf16 logits behind 2048 tokens, masks, greedy:
// 66 us (2.4 TB/s of 160 MB), of which the lists are about 11, the copy 26 to 33
// and the listed logits the rest. Their traffic, a 32-byte sector each way for
// about 200 thousand of them, is worth 2 us; what they cost is the time after
// the copies, when the CTA of a sequence's frequent ids has 8 times the mean of
// listed ids to settle and few warps run. The same calls with ids spread evenly
// over the vocabulary take 62 us, and 64 long histories of 129280 fp32 logits
// 49.5 instead of 57.3. Other divisions cost more: listed
// logits within the copy 113 us (every warp runs the whole arithmetic for a lane
// or two), a history counted by a cluster through each other's shared memory 91,
// the listed logits in a third kernel 72, the state counted by every CTA of the
// copy 67 (but 70 us rather than 57 for 64 rows behind 32768 tokens).
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "common.cuh"
#include "kernels.h"

namespace dspark {

namespace {

constexpr int kBlock = 512;        // ids; the unit of parts and stretches, with a place of its own in the lists
constexpr int kListThreads = 1024;
constexpr int kRounds = 2;         // words of 32 ids per thread of list_kernel, at most
constexpr int kMaxPart = kListThreads * kRounds * 32;  // 16-bit places in its list
constexpr int kListSmem = 222 * 1024;
constexpr int kAhead = 8;          // history ids in flight per thread
constexpr int kCopyThreads = 256;
// Per SM: a copy of 32 x 8 x 151936 takes 66 us with three, of 80 registers a
// thread, 71 with four, which leave it 64, and as much with two of 512 threads.
constexpr int kCopyCtas = 3;
constexpr int kMaxStretch = 16384;
constexpr int kInFlight = 4;       // vectors, or listed logits, under way per thread
constexpr int kRows = 8;           // rows copied before their listed logits are worked out
template <int N>
using Int = std::integral_constant<int, N>;

constexpr uint32_t kFlag = 0x80000000u;  // of an entry's id: biased; of its count: in the prompt

// The sizes of both kernels and the places in the scratch, for one call.
struct ConstrainPlan {
  int has_bias, narrow;
  int part, parts, list_threads;  // ids per CTA of list_kernel, per sequence; parts 0: nothing is listed
  int stretch, stretches, copy_threads;  // ids per CTA of copy_kernel, per sequence and rows
  int rows, groups;                      // rows per CTA of it
  int64_t entries;                // places for entries per part
  // Byte offsets in the scratch: [rows] keys and [batch] counters, both cleared
  // by list_kernel; per part, the number of entries before each block and in
  // all; entries as planes of ids, counts and biases.
  int64_t counters, before, ids, counts, biases, bytes;
};

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

template <typename P>
__device__ __forceinline__ P* plane(const ConstrainArgs& a, int64_t offset) {
  return reinterpret_cast<P*>(static_cast<unsigned char*>(a.scratch) + offset);
}

// C: uint16_t where no count nor bias entry passes 65535, else uint32_t.
template <typename C>
__global__ void __launch_bounds__(kListThreads, 1) list_kernel(ConstrainArgs a, ConstrainPlan p) {
  extern __shared__ __align__(16) uint32_t smem[];
  __shared__ int totals[kRounds * kListThreads / 32 + 1];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int tid = (int)threadIdx.x, lane = tid & 31, warp = tid >> 5, threads = (int)blockDim.x, warps = threads >> 5;
  const int64_t b = blockIdx.x / p.parts;
  const int part = (int)(blockIdx.x % p.parts);
  const int64_t c0 = (int64_t)part * p.part;
  const int n = (int)min((int64_t)p.part, a.vocab - c0), words = p.part / 32;
  uint32_t* in_prompt = smem;            // one bit per id
  uint32_t* in_block = smem + words;     // drafted in this block
  C* count = reinterpret_cast<C*>(smem + 2 * words);
  C* slot = count + p.part;              // last bias entry + 1, where there are biases
  uint16_t* list = reinterpret_cast<uint16_t*>(slot + (p.has_bias ? p.part : 0));  // what there is, in order
  // The first ids of the history are read while the cells are cleared, before
  // its length is known: its buffer covers them.
  const int cap = a.history ? (int)a.history_cap : 0;
  const int64_t* history = a.history + b * a.history_stride;
  const int64_t* bias_ids = a.bias_ids + b * a.bias_stride;
  const int64_t* draft = a.draft ? a.draft + b * a.draft_stride : nullptr;
  int64_t first_ids[kAhead], first_bias = -1;
#pragma unroll
  for (int u = 0; u < kAhead; ++u) first_ids[u] = tid + u * threads < cap ? history[tid + u * threads] : 0;
  if (tid < a.bias_count) first_bias = bias_ids[tid];
  int64_t length = a.history && a.history_lens ? a.history_lens[b] : cap;
  int64_t prompted = a.prompt_lens ? a.prompt_lens[b] : 0;
  {
    uint4* cells = reinterpret_cast<uint4*>(smem);
    const int vecs = (words * 8 + p.part * (int)sizeof(C) * (p.has_bias ? 2 : 1)) / 16;
    for (int i = tid; i < vecs; i += threads) cells[i] = make_uint4(0u, 0u, 0u, 0u);
  }
  if (part == 0 && a.tokens) {
    if (tid == 0) plane<uint32_t>(a, p.counters)[b] = 0u;
    for (int64_t k = tid; k < a.block; k += threads) plane<unsigned long long>(a, 0)[b * a.block + k] = 0ull;
  }
  const int len = (int)min(max(length, (int64_t)0), (int64_t)cap);
  const int prompt = (int)min(max(prompted, (int64_t)0), (int64_t)len);
  __syncthreads();
  bool bad = false;
  auto note_token = [&](int64_t id, int i) {
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
  for (int u = 0; u < kAhead; ++u)
    if (tid + u * threads < len) note_token(first_ids[u], tid + u * threads);
  for (int i = tid + threads * kAhead; i < len; i += threads * kAhead) {
    int64_t id[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) id[u] = i + u * threads < len ? history[i + u * threads] : 0;
#pragma unroll
    for (int u = 0; u < kAhead; ++u)
      if (i + u * threads < len) note_token(id[u], i + u * threads);
  }
  if (tid < a.bias_count) note_bias(first_bias, tid);
  for (int64_t i = tid + threads; i < a.bias_count; i += threads) note_bias(bias_ids[i], i);
  if (draft) {
    // Those before the block count; those of the block are listed, and counted
    // row by row later. The last row's own token precedes no row.
    for (int64_t i = tid; i < a.draft_first + a.block - 1; i += threads) {
      const int64_t id = draft[i];
      const uint64_t l = (uint64_t)(id - c0);
      if (id >= a.vocab) bad = true;
      if (l >= (uint64_t)n) continue;
      if (i < a.draft_first)
        Cells<C>::add(count, (int)l);
      else
        atomicOr(&in_block[l >> 5], 1u << (l & 31));
    }
  }
  __syncthreads();

  // A word of 32 ids per lane and round, in order of the ids over rounds, warps
  // and lanes.
  uint32_t word[kRounds];
  int mine[kRounds];  // entries before the lane's within the warp's words
#pragma unroll
  for (int r = 0; r < kRounds; ++r) {
    const int w = (r * warps + warp) * 32 + lane;
    word[r] = 0u;
    if (w < words) {
      word[r] = in_prompt[w] | in_block[w];
      constexpr int kPer = 16 / sizeof(C);  // cells of 16 bytes
      // Neighbouring lanes begin at different places of their 32 cells, which
      // lie a multiple of the banks apart.
      auto look = [&](const C* cells) {
#pragma unroll
        for (int i = 0; i < 32 / kPer; ++i) {
          const int at = (i + lane / (8 / (32 / kPer > 8 ? 8 : 32 / kPer))) % (32 / kPer) * kPer;
          const uint4 x = *reinterpret_cast<const uint4*>(cells + w * 32 + at);
          if (x.x | x.y | x.z | x.w) {
            uint32_t some = 0u;
#pragma unroll
            for (int e = 0; e < kPer; ++e) {
              const uint32_t v = sizeof(C) == 4 ? (e == 0 ? x.x : e == 1 ? x.y : e == 2 ? x.z : x.w)
                                                : ((e < 2 ? x.x : e < 4 ? x.y : e < 6 ? x.z : x.w) >> (16 * (e & 1))) & 0xffffu;
              if (v) some |= 1u << e;
            }
            word[r] |= some << at;
          }
        }
      };
      look(count);
      if (p.has_bias) look(slot);
    }
    int sum = __popc(word[r]);
    mine[r] = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int before = __shfl_up_sync(0xffffffffu, sum, o);
      if (lane >= o) sum += before;
    }
    mine[r] = sum - mine[r];
    if (lane == 31) totals[r * warps + warp] = sum;
  }
  __syncthreads();
  if (warp == 0) {  // totals of warps before each, and of all
    int carry = 0;
    for (int i0 = 0; i0 < kRounds * warps; i0 += 32) {
      const int own = i0 + lane < kRounds * warps ? totals[i0 + lane] : 0;
      int sum = own;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int before = __shfl_up_sync(0xffffffffu, sum, o);
        if (lane >= o) sum += before;
      }
      if (i0 + lane < kRounds * warps) totals[i0 + lane] = carry + sum - own;
      carry += __shfl_sync(0xffffffffu, sum, 31);
    }
    if (lane == 0) totals[kRounds * warps] = carry;
  }
  __syncthreads();

  const int blocks = p.part / kBlock, total = totals[kRounds * warps];
  const int64_t which = b * p.parts + part;
  uint32_t* before = plane<uint32_t>(a, p.before) + which * (blocks + 1);
#pragma unroll
  for (int r = 0; r < kRounds; ++r) {
    const int w = (r * warps + warp) * 32 + lane;
    int at = totals[r * warps + warp] + mine[r];
    if (w < words && w % (kBlock / 32) == 0) before[w / (kBlock / 32)] = (uint32_t)at;
    for (uint32_t bits = word[r]; bits; bits &= bits - 1u) list[at++] = (uint16_t)(w * 32 + __ffs((int)bits) - 1);
  }
  if (tid == 0) before[blocks] = (uint32_t)total;
  __syncthreads();
  uint32_t* ids = plane<uint32_t>(a, p.ids) + which * p.entries;
  uint32_t* counts = plane<uint32_t>(a, p.counts) + which * p.entries;
  float* biases = plane<float>(a, p.biases) + which * p.entries;
  const float* bias = a.bias_values + b * a.bias_stride;
  for (int e = tid; e < total; e += threads) {
    const int l = (int)list[e];
    const uint32_t entry = p.has_bias ? (uint32_t)slot[l] : 0u;
    ids[e] = (uint32_t)(c0 + l) | (entry ? kFlag : 0u);
    counts[e] = (uint32_t)count[l] | (bit(in_prompt, l) ? kFlag : 0u);
    if (entry) biases[e] = bias[entry - 1u];
  }
  if (bad) report_status(a.status, DSPARK_STATUS_TOKEN_RANGE);
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

// ALIGNED: every row starts at a 16-byte address, in and out.
template <typename T, bool ALIGNED>
__global__ void __launch_bounds__(kCopyThreads, kCopyCtas) copy_kernel(ConstrainArgs a, ConstrainPlan p) {
  constexpr int kE = Vec<T>::kE;
  extern __shared__ __align__(16) uint32_t touched[];  // one bit per id of the stretch: listed
  __shared__ int drafted[kRows];  // the tokens drafted after each of the rows (-1: none)
  __shared__ unsigned long long warp_key[kRows][kCopyThreads / 32], listed_key[kRows];
  __shared__ float warp_best[kRows][kCopyThreads / 32];  // greedy: the warp's largest value
  __shared__ int warp_at[kRows][kCopyThreads / 32];      // and the first id of its vector, or ~ the id of a single
  __shared__ bool last;
  const int tid = (int)threadIdx.x, lane = tid & 31, warp = tid >> 5, threads = (int)blockDim.x;
  const int64_t b = blockIdx.x / p.stretches;
  const int stretch = (int)(blockIdx.x % p.stretches);
  const int64_t c0 = (int64_t)stretch * p.stretch;
  const int rows = (int)a.block, k_begin = (int)blockIdx.y * p.rows, k_end = rows - k_begin > p.rows ? k_begin + p.rows : rows;
  const int n = (int)min((int64_t)p.stretch, a.vocab - c0);
  const int words = p.stretch / 32, mask_last = (n + 31) / 32 - 1;
  const bool keyed = a.tokens != nullptr;
  constexpr int kNone = 0x7fffffff;
  // The key of a draw. A quotient from 2^127 on, in whose place 2^127 + |y| / 4
  // stands, keeps the order of the logits and is finite where the logit is: a
  // logit near the lowest value ranks above -inf (not allowed) at any
  // temperature. No noise reaches that far.
  auto score = [&](float y, int64_t k, int l) {
    const uint32_t v = (uint32_t)(c0 + l);
    float q = y / a.temperature;
    if (fabsf(q) >= 0x1p127f) q = fmaf(0.25f, y, copysignf(0x1p127f, y));
    return pack_key(q + noise_for(a.seed, (uint32_t)b, (uint32_t)(a.draft_first + k), v), v);
  };
  const T* const in0 = static_cast<const T*>(a.in) + b * a.in_batch + c0;
  T* const out0 = static_cast<T*>(a.out) + b * a.out_batch + c0;
  const uint32_t* const mask0 = a.allowed ? a.allowed + b * a.allowed_batch + (c0 >> 5) : nullptr;
  // The first rows come into L2 while the lists are made.
  for (int k = k_begin; k < min(k_end, k_begin + kRows); ++k) {
    const char* row = reinterpret_cast<const char*>(in0 + (int64_t)k * a.in_row);
    for (int at = tid * 128; at < n * (int)sizeof(T); at += threads * 128)
      asm volatile("prefetch.global.L2 [%0];" ::"l"(row + at));
  }

  // What is listed in the stretch: a run of entries in each of the one or two
  // parts that it meets (a part is no smaller than a stretch).
  for (int i = tid; i < words; i += threads) touched[i] = 0u;
  const float rho = a.repetition ? a.repetition[b] : a.repetition_value;
  const float freq = a.frequency ? a.frequency[b] : a.frequency_value;
  const float pres = a.presence ? a.presence[b] : a.presence_value;
  const int64_t* draft = a.draft ? a.draft + b * a.draft_stride + a.draft_first : nullptr;
  const int blocks = p.parts ? p.part / kBlock : 1, block0 = (int)(c0 / kBlock), block1 = (int)((c0 + n + kBlock - 1) / kBlock);
  const int part0 = block0 / blocks, part1 = p.parts ? (block1 - 1) / blocks + 1 : part0;
  const uint32_t* ids = plane<uint32_t>(a, p.ids);
  const uint32_t* counts = plane<uint32_t>(a, p.counts);
  const float* biases = plane<float>(a, p.biases);
  __syncthreads();
  asm volatile("griddepcontrol.wait;" ::: "memory");  // the lists are there
  int64_t run_from[2] = {0, 0};
  int run_length[2] = {0, 0};
#pragma unroll
  for (int i = 0; i < 2; ++i)
    if (part0 + i < part1) {
      const int part = part0 + i;
      const int64_t which = b * p.parts + part;
      const uint32_t* before = plane<uint32_t>(a, p.before) + which * (blocks + 1);
      const uint32_t from = before[max(block0 - part * blocks, 0)];
      run_from[i] = which * p.entries + from;
      run_length[i] = (int)(before[min(block1 - part * blocks, blocks)] - from);
    }
  if (keyed) {
#pragma unroll
    for (int i = 0; i < 2; ++i)
      for (int e0 = tid; e0 < run_length[i]; e0 += threads * kInFlight) {
        uint32_t id[kInFlight];
#pragma unroll
        for (int u = 0; u < kInFlight; ++u) id[u] = ids[run_from[i] + min(e0 + u * threads, run_length[i] - 1)];
#pragma unroll
        for (int u = 0; u < kInFlight; ++u) {
          const int l = (int)((id[u] & ~kFlag) - (uint32_t)c0);
          atomicOr(&touched[l >> 5], 1u << (l & 31));
        }
      }
    __syncthreads();
  }

  for (int k0 = k_begin; k0 < k_end; k0 += kRows) {
    const int group = min(kRows, k_end - k0);
    if (k0 > k_begin) __syncthreads();  // the last rows' keys have been read
    if (tid < kRows) {
      listed_key[tid] = 0ull;
      const int64_t id = draft && k0 + tid < rows - 1 ? draft[k0 + tid] : -1;
      drafted[tid] = id >= 0 && id < a.vocab ? (int)id : -1;
    }

    // The copy. Greedy keys: the largest value so far and the first id of its
    // vector; a single element has the complement of its id. Keys of both kinds
    // begin with -inf at the first threads' own ids, so that a row of -inf alone
    // takes the lowest, id 0, whichever of its logits are listed. Listed logits
    // stand aside as -inf.
    const T* in = in0 + (int64_t)k0 * a.in_row;
    T* out = out0 + (int64_t)k0 * a.out_row;
    const uint32_t* mask = mask0 ? mask0 + (int64_t)k0 * a.allowed_row : nullptr;
    for (int r = 0; r < group; ++r) {
      float best = -INFINITY;
      int best_at = tid < n ? ~tid : kNone;
      unsigned long long key = tid < n ? pack_key(-INFINITY, (uint32_t)(c0 + tid)) : 0ull;
      // Strictly larger, or the first NaN: ids rise, so equal values keep the lower one.
      auto better = [&](float y) { return y > best || (y != y && best == best); };
      auto single = [&](int l) {
        const T y = !mask || bit(mask, l) ? in[l] : from_f32<T>(-INFINITY);
        out[l] = y;
        if (!keyed || bit(touched, l)) return;
        if (!a.greedy) {
          key = max_key(key, score(to_f32(y), k0 + r, l));
        } else if (better(to_f32(y))) {
          best = to_f32(y);
          best_at = ~l;
        }
      };
      // Elements before the first 16-byte address, vectors, and what is left;
      // all single where the output's vectors lie elsewhere.
      int head = 0;
      if (!ALIGNED) {
        const int past = (int)((reinterpret_cast<uintptr_t>(in) / sizeof(T)) % kE);
        const bool same = (reinterpret_cast<uintptr_t>(in) - reinterpret_cast<uintptr_t>(out)) % 16 == 0;
        head = same ? min(past ? kE - past : 0, n) : n;
        for (int l = tid; l < head; l += threads) single(l);
      }
      const int vecs = (n - head) / kE;
      const uint4* from = reinterpret_cast<const uint4*>(in + head);
      uint4* to = reinterpret_cast<uint4*>(out + head);
      for (int j0 = tid; j0 < vecs; j0 += threads * kInFlight) {
        uint4 raw[kInFlight];
        uint32_t lo[kInFlight], hi[kInFlight];
#pragma unroll
        for (int u = 0; u < kInFlight; ++u) {
          const int j = j0 + u * threads;
          if (j < vecs) {
            raw[u] = __ldcs(from + j);
            if (mask) {
              const int w = (head + j * kE) >> 5;
              lo[u] = mask[w];
              if (!ALIGNED) hi[u] = w < mask_last ? mask[w + 1] : 0u;
            }
          }
        }
#pragma unroll
        for (int u = 0; u < kInFlight; ++u) {
          const int j = j0 + u * threads, l = head + j * kE;
          if (j < vecs) {
            if (mask) raw[u] = Vec<T>::masked(raw[u], ALIGNED ? lo[u] >> (l & 31) : __funnelshift_r(lo[u], hi[u], l & 31));
            __stcs(to + j, raw[u]);
            if (keyed) {
              const uint32_t aside = bits_at<ALIGNED>(touched, l, words - 1) & ((1u << kE) - 1u);
              if (aside) raw[u] = Vec<T>::masked(raw[u], ~aside);
              if (a.greedy) {
                const float top = Vec<T>::max_of(raw[u]);
                if (better(top)) {
                  best = top;
                  best_at = l;
                }
              } else {
#pragma unroll
                for (int e = 0; e < kE; ++e) key = max_key(key, score(Vec<T>::get(raw[u], e), k0 + r, l + e));
              }
            }
          }
        }
      }
      for (int l = head + vecs * kE + tid; l < n; l += threads) single(l);
      if (keyed && a.greedy) {
        // The warp's largest value, of equal ones the first; which element of
        // its vector is found for all rows together.
        const uint32_t order = best_at != kNone ? orderable_bits(best) : 0u, top = __reduce_max_sync(0xffffffffu, order);
        const int id = best_at < 0 ? ~best_at : best_at;
        const int first = __reduce_min_sync(0xffffffffu, order == top ? id : kNone);
        if (order == top && id == first) {
          warp_best[r][warp] = best;
          warp_at[r][warp] = best_at;
        }
      } else if (keyed) {
        // The warp's largest key: the larger high word, then the larger low one.
        const uint32_t high = __reduce_max_sync(0xffffffffu, (uint32_t)(key >> 32));
        const uint32_t low = __reduce_max_sync(0xffffffffu, (uint32_t)(key >> 32) == high ? (uint32_t)key : 0u);
        if (lane == 0) warp_key[r][warp] = ((unsigned long long)high << 32) | low;
      }
      in += a.in_row;
      out += a.out_row;
      if (mask) mask += a.allowed_row;
    }
    __syncthreads();
    if (keyed && a.greedy && tid < group * (threads >> 5)) {
      const int row = tid / (threads >> 5), w = tid % (threads >> 5), at = warp_at[row][w];
      unsigned long long own = 0ull;
      if (at != kNone) {
        const float top = warp_best[row][w];
        int id = ~at;
        if (at >= 0) {
          const uint4 vec = *reinterpret_cast<const uint4*>(out0 + (int64_t)(k0 + row) * a.out_row + at);
          const uint32_t aside = bits_at<ALIGNED>(touched, at, words - 1);
          int first = 0;
#pragma unroll
          for (int e = kE - 1; e >= 0; --e) {
            const float y = Vec<T>::get(vec, e);
            if ((y == top || (y != y && top != top)) && !((aside >> e) & 1u)) first = e;
          }
          id = at + first;
        }
        own = pack_key(top, (uint32_t)(c0 + id));
      }
      warp_key[row][w] = own;
    }
    if (keyed) __syncthreads();  // before listed logits change the vectors just looked at

    // The listed logits of these rows, after the copies of them: EN entries in
    // flight per thread, RN of their rows. What the copy left in place of a
    // masked one stays; in place, an allowed one's input is what the copy wrote.
    auto settle = [&](auto entries_in_flight, auto rows_in_flight) {
      constexpr int EN = decltype(entries_in_flight)::value, RN = decltype(rows_in_flight)::value;
#pragma unroll 1
      for (int i = 0; i < 2; ++i) {
        const int length = i == 0 ? run_length[0] : run_length[1];
        const int64_t from = i == 0 ? run_from[0] : run_from[1];
        for (int e0 = tid; e0 < length; e0 += threads * EN) {
          uint32_t id[EN], counted[EN], allowed[EN];
          float beta[EN];
          T x[EN][RN];
#pragma unroll
          for (int u = 0; u < EN; ++u) {
            const int64_t e = from + min(e0 + u * threads, length - 1);
            id[u] = ids[e];
            counted[u] = counts[e];
            beta[u] = p.has_bias ? biases[e] : 0.0f;  // of no meaning where the id has no flag
          }
          for (int g0 = 0; g0 < group; g0 += RN) {
#pragma unroll
            for (int u = 0; u < EN; ++u) {
              const int l = (int)((id[u] & ~kFlag) - (uint32_t)c0);
              const T* rin = in0 + (int64_t)(k0 + g0) * a.in_row + l;
              const uint32_t* rmask = mask0 + (int64_t)(k0 + g0) * a.allowed_row + (l >> 5);
              uint32_t word[RN];
#pragma unroll
              for (int g = 0; g < RN; ++g) {
                x[u][g] = from_f32<T>(0.0f);
                word[g] = ~0u;
                if (g0 + g < group) {
                  x[u][g] = rin[g * a.in_row];
                  if (mask0) word[g] = rmask[g * a.allowed_row];
                }
              }
              allowed[u] = 0u;
#pragma unroll
              for (int g = 0; g < RN; ++g) allowed[u] |= ((word[g] >> (l & 31)) & 1u) << g;
            }
            if (draft && g0 == 0)  // drafted before these rows
              for (int d = 0; d < k0; ++d) {
                const int64_t t = draft[d];
#pragma unroll
                for (int u = 0; u < EN; ++u) counted[u] += t == (int64_t)(id[u] & ~kFlag) ? 1u : 0u;
              }
#pragma unroll
            for (int u = 0; u < EN; ++u) {
              if (e0 + u * threads >= length) break;
              const int token = (int)(id[u] & ~kFlag), l = (int)((uint32_t)token - (uint32_t)c0);
              T* rout = out0 + (int64_t)(k0 + g0) * a.out_row + l;
#pragma unroll
              for (int g = 0; g < RN; ++g) {
                if (g0 + g >= group) break;
                const uint32_t times = counted[u] & ~kFlag;
                if (drafted[g0 + g] == token) counted[u] += 1u;  // from the next row on
                if (!((allowed[u] >> g) & 1u)) continue;
                float f = to_f32(x[u][g]);
                if ((counted[u] & kFlag) || times) f = f > 0.0f ? __fdiv_rn(f, rho) : __fmul_rn(f, rho);
                if (times) f = __fsub_rn(__fsub_rn(f, __fmul_rn(freq, (float)times)), pres);
                if (id[u] & kFlag) f = __fadd_rn(f, beta[u]);
                const T y = from_f32<T>(f);
                rout[g * a.out_row] = y;
                if (keyed) {
                  const unsigned long long own =
                      a.greedy ? pack_key(to_f32(y), (uint32_t)token) : score(to_f32(y), k0 + g0 + g, l);
                  if (own > *reinterpret_cast<volatile unsigned long long*>(&listed_key[g0 + g]))
                    atomicMax(&listed_key[g0 + g], own);
                }
              }
            }
          }
        }
      }
    };
    if (group > 2)
      settle(Int<1>{}, Int<kRows>{});
    else
      settle(Int<kInFlight>{}, Int<1>{});
    __syncthreads();
    if (keyed && tid < group) {
      unsigned long long top = listed_key[tid];
      for (int w = 0; w < threads / 32; ++w) top = max_key(top, warp_key[tid][w]);
      atomicMax(plane<unsigned long long>(a, 0) + b * rows + k0 + tid, top);
      __threadfence();
    }
  }
  // The last CTA of a sequence has all its keys; their ids are the tokens.
  if (keyed) {
    __syncthreads();
    if (tid == 0) {
      __threadfence();
      last = atomicAdd(plane<uint32_t>(a, p.counters) + b, 1u) == (uint32_t)(p.stretches * p.groups) - 1u;
      __threadfence();
    }
    __syncthreads();
    if (last)
      for (int k = tid; k < rows; k += threads)
        a.tokens[b * a.tokens_batch + k] = (int64_t)key_token(__ldcg(plane<unsigned long long>(a, 0) + b * rows + k));
  }
}

int64_t round_up(int64_t x, int64_t to) { return (x + to - 1) / to * to; }

// Shared memory of list_kernel: two bits per id, counts, bias entries, the list.
int64_t list_bytes(int64_t part, int64_t entries, bool narrow, bool has_bias) {
  return part / 4 + part * (narrow ? 2 : 4) * (has_bias ? 2 : 1) + round_up(std::min(part, entries) * 2, 16);
}

// The plan goes by sizes alone, so that a caller can make the scratch anywhere.
ConstrainPlan plan_constrain(const ConstrainArgs& a) {
  constexpr int64_t num_sms = 148;
  ConstrainPlan p{};
  p.has_bias = a.bias_count > 0 ? 1 : 0;
  const int64_t tokens = (a.history ? a.history_cap : 0) + a.draft_most;
  p.narrow = tokens <= 0xffff && a.bias_count <= 0xfffe ? 1 : 0;
  const int64_t vocab = round_up(a.vocab, kBlock);
  // Stretches: as many CTAs as run at once, and as few waves of them as the
  // largest stretch allows. Where there are few, rows go to different CTAs
  // rather than one after another, each of which then reads the lists, until
  // stretches of 8192 ids fill the device. Kernels behind 1000 tokens with rows
  // divided until stretches of 2048, 8192 and 32768 ids do: 16 x 8 rows of 32003
  // ids 32.7, 17.0 and 16.9 us, 8 x 8 of 129280 46.7, 18.6 and 23.2, 32 x 8 of
  // 129280 46.2, 46.2 and 50.9.
  const int64_t slots = kCopyCtas * num_sms;
  int64_t rows = a.block;
  while (rows > 1 && a.batch * ((a.block + rows - 1) / rows) * (vocab / 8192 + 1) <= slots) rows = (rows + 1) / 2;
  p.rows = (int)std::min<int64_t>(rows, 0x7fffffff);
  p.groups = (int)((a.block + rows - 1) / rows);
  int64_t stretch = vocab;
  for (int64_t waves = 1; waves <= 64; ++waves) {
    const int64_t each = std::max<int64_t>(1, waves * slots / (a.batch * p.groups));  // stretches of a sequence's rows
    stretch = round_up((vocab + each - 1) / each, kBlock);
    if (stretch <= kMaxStretch) break;
  }
  stretch = std::min<int64_t>(stretch, kMaxStretch);
  p.stretch = (int)stretch;
  p.stretches = (int)((a.vocab + stretch - 1) / stretch);
  p.copy_threads = (int)std::min<int64_t>(kCopyThreads, std::max<int64_t>(64, stretch / 32 / 32 * 32));

  if (tokens + a.bias_count > 0 || a.tokens) {
    // Parts: as few as shared memory allows, since each reads all of a history,
    // but as many CTAs as there are SMs. Four times as many were no faster even
    // where the history is one read of each thread: 64 rows of 129280 ids behind
    // 600 tokens 28.7 us instead of 24.9, 1 row 10.4 instead of 10.2.
    const int64_t entries = tokens + a.bias_count;
    const auto bytes = [&](int64_t part) { return list_bytes(part, entries, p.narrow, p.has_bias); };
    int64_t most = kMaxPart;
    while (bytes(most) > kListSmem) most -= kBlock;
    const int64_t parts = std::max((vocab + most - 1) / most, std::min(num_sms / a.batch, vocab / (2 * kBlock)));
    p.part = (int)std::max(round_up((vocab + parts - 1) / parts, kBlock), stretch);  // a stretch meets two parts at most
    p.parts = (int)((vocab + p.part - 1) / p.part);
    p.list_threads = (int)std::min<int64_t>(kListThreads, std::max<int64_t>(256, round_up(p.part / 32, 32)));
  }
  p.entries = std::min<int64_t>(p.part, tokens + a.bias_count);
  const int64_t lists = a.batch * p.parts;
  int64_t at = round_up(a.tokens ? a.batch * a.block * 8 : 0, 16);
  const auto take = [&at](int64_t bytes) {
    const int64_t from = at;
    at = round_up(at + bytes, 16);
    return from;
  };
  p.counters = take(a.tokens ? a.batch * 4 : 0);
  p.before = take(p.parts ? lists * (p.part / kBlock + 1) * 4 : 0);
  p.ids = take(lists * p.entries * 4);
  p.counts = take(lists * p.entries * 4);
  p.biases = take(p.has_bias ? lists * p.entries * 4 : 0);
  p.bytes = at;
  return p;
}

template <typename C>
cudaError_t launch_list(const ConstrainArgs& a, const ConstrainPlan& p, cudaStream_t s) {
  const size_t bytes = (size_t)list_bytes(p.part, p.entries, p.narrow, p.has_bias);
  if (bytes > 40 * 1024) {
    const cudaError_t e =
        cudaFuncSetAttribute(list_kernel<C>, cudaFuncAttributeMaxDynamicSharedMemorySize, kListSmem);
    if (e != cudaSuccess) return e;
  }
  list_kernel<C><<<(unsigned)(a.batch * p.parts), p.list_threads, bytes, s>>>(a, p);
  note_launch();
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_copy(const ConstrainArgs& a, const ConstrainPlan& p, cudaStream_t s) {
  const auto whole = [&a](const void* base, int64_t batch, int64_t row) {
    constexpr int64_t kE = Vec<T>::kE;
    return reinterpret_cast<uintptr_t>(base) % 16 == 0 && (a.batch == 1 || batch % kE == 0) &&
           (a.block == 1 || row % kE == 0);
  };
  const bool aligned = whole(a.in, a.in_batch, a.in_row) && whole(a.out, a.out_batch, a.out_row);
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(a.batch * p.stretches), (unsigned)p.groups);
  cfg.blockDim = dim3((unsigned)p.copy_threads);
  cfg.dynamicSmemBytes = (size_t)p.stretch / 8;
  cfg.stream = s;
  // Starts while the lists are made; its first loads do not need them.
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = p.parts ? 1 : 0;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, aligned ? copy_kernel<T, true> : copy_kernel<T, false>, a, p);
  note_launch();
  return e;
}

}  // namespace

int64_t constrain_scratch_bytes(const ConstrainArgs& a) { return plan_constrain(a).bytes; }

cudaError_t launch_constrain(const ConstrainArgs& a, int logits_dtype, cudaStream_t s) {
  const ConstrainPlan p = plan_constrain(a);
  if (a.batch * std::max(p.parts, p.stretches) > 0x7fffffffll) return cudaErrorInvalidConfiguration;
  if (p.parts) {
    const cudaError_t e = p.narrow ? launch_list<uint16_t>(a, p, s) : launch_list<uint32_t>(a, p, s);
    if (e != cudaSuccess) return e;
  }
  return logits_dtype == DSPARK_DTYPE_FP32 ? launch_copy<float>(a, p, s) : launch_copy<__nv_bfloat16>(a, p, s);
}

}  // namespace dspark
