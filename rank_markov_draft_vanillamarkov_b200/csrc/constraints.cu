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
#include <cmath>

#include "common.cuh"
#include "kernels.h"

namespace dspark {

namespace {

constexpr int kThreads = 256;
constexpr int kChunk = 4096;                  // vocabulary ids per CTA
constexpr uint32_t kPromptBit = 0x80000000u;  // count word: seen in the prompt; low bits: generated occurrences

template <typename T>
__global__ void __launch_bounds__(kThreads) constrain_kernel(ConstrainArgs a, int chunks) {
  __shared__ uint32_t count[kChunk];
  __shared__ uint32_t slot[kChunk];  // 1 + the last bias entry naming this id, 0 for none
  __shared__ unsigned long long warp_best[kThreads / 32];
  const int64_t b = blockIdx.x / chunks;
  const int chunk = (int)(blockIdx.x % chunks);
  const int64_t c0 = (int64_t)chunk * kChunk;
  const int n = (int)(a.vocab - c0 < kChunk ? a.vocab - c0 : kChunk);
  for (int i = threadIdx.x; i < n; i += kThreads) count[i] = slot[i] = 0u;
  __syncthreads();

  bool bad = false;
  int64_t len = a.history ? a.history_cap : 0;
  if (a.history && a.history_lens) len = min(max(a.history_lens[b], (int64_t)0), len);
  const int64_t prompt = a.prompt_lens ? min(max(a.prompt_lens[b], (int64_t)0), len) : 0;
  for (int64_t i = threadIdx.x; i < len; i += kThreads) {
    const int64_t id = a.history[b * a.history_stride + i];
    if (id < 0 || id >= a.vocab) bad = true;
    const int64_t l = id - c0;
    if (l < 0 || l >= n) continue;
    if (i < prompt)
      atomicOr(&count[l], kPromptBit);
    else
      atomicAdd(&count[l], 1u);
  }
  for (int64_t i = threadIdx.x; i < a.bias_count; i += kThreads) {
    const int64_t id = a.bias_ids[b * a.bias_stride + i];
    if (id >= a.vocab) bad = true;
    const int64_t l = id - c0;
    if (l >= 0 && l < n) atomicMax(&slot[l], (uint32_t)i + 1u);
  }
  const int64_t* draft = a.draft ? a.draft + b * a.draft_stride : nullptr;
  for (int64_t i = threadIdx.x; draft && i < a.draft_first; i += kThreads) {
    const int64_t id = draft[i];
    if (id >= a.vocab) bad = true;
    const int64_t l = id - c0;
    if (l >= 0 && l < n) atomicAdd(&count[l], 1u);
  }
  const float rho = a.repetition ? a.repetition[b] : a.repetition_value;
  const float freq = a.frequency ? a.frequency[b] : a.frequency_value;
  const float pres = a.presence ? a.presence[b] : a.presence_value;

  for (int64_t k = 0; k < a.block; ++k) {
    __syncthreads();
    if (k > 0 && draft) {
      if (threadIdx.x == 0) {
        const int64_t id = draft[a.draft_first + k - 1];
        if (id >= a.vocab) bad = true;
        const int64_t l = id - c0;
        if (l >= 0 && l < n) count[l] += 1u;
      }
      __syncthreads();
    }
    const T* in = static_cast<const T*>(a.in) + b * a.in_batch + k * a.in_row + c0;
    T* out = static_cast<T*>(a.out) + b * a.out_batch + k * a.out_row + c0;
    const uint32_t* mask = a.allowed ? a.allowed + b * a.allowed_batch + k * a.allowed_row : nullptr;
    unsigned long long best = 0ull;
    for (int i = threadIdx.x; i < n; i += kThreads) {
      float x = to_f32(in[i]);
      const uint32_t c = count[i];
      const uint32_t times = c & ~kPromptBit;
      if (c) x = x > 0.0f ? __fdiv_rn(x, rho) : __fmul_rn(x, rho);
      if (times) x = __fsub_rn(__fsub_rn(x, __fmul_rn(freq, (float)times)), pres);
      if (slot[i]) x = __fadd_rn(x, a.bias_values[b * a.bias_stride + slot[i] - 1]);
      const int64_t v = c0 + i;
      if (mask && !((mask[v >> 5] >> (v & 31)) & 1u)) x = -INFINITY;
      const T y = from_f32<T>(x);
      out[i] = y;
      if (a.keys) {
        float s = to_f32(y);
        if (!a.greedy) s = s / a.temperature + noise_for(a.seed, (uint32_t)b, (uint32_t)(a.draft_first + k), (uint32_t)v);
        const unsigned long long key = pack_key(s, (uint32_t)v);
        best = best > key ? best : key;
      }
    }
    if (a.keys) {
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        const unsigned long long other = __shfl_xor_sync(0xffffffffu, best, o);
        best = best > other ? best : other;
      }
      if ((threadIdx.x & 31) == 0) warp_best[threadIdx.x >> 5] = best;
      __syncthreads();
      if (threadIdx.x == 0) {
        for (int w = 1; w < kThreads / 32; ++w) best = best > warp_best[w] ? best : warp_best[w];
        a.keys[(b * a.block + k) * chunks + chunk] = best;
      }
    }
  }
  if (bad) report_status(a.status, DSPARK_STATUS_TOKEN_RANGE);
}

// The token of each row: the id in the largest of its chunks' keys.
__global__ void __launch_bounds__(32) choose_kernel(ConstrainArgs a, int chunks) {
  const int64_t row = blockIdx.x;
  unsigned long long best = 0ull;
  for (int i = threadIdx.x; i < chunks; i += 32) {
    const unsigned long long key = a.keys[row * chunks + i];
    best = best > key ? best : key;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const unsigned long long other = __shfl_xor_sync(0xffffffffu, best, o);
    best = best > other ? best : other;
  }
  if (threadIdx.x == 0) a.tokens[row / a.block * a.tokens_batch + row % a.block] = (int64_t)key_token(best);
}

}  // namespace

int64_t constrain_key_count(int64_t batch, int64_t block, int64_t vocab) {
  return batch * block * ((vocab + kChunk - 1) / kChunk);
}

cudaError_t launch_constrain(const ConstrainArgs& a, int logits_dtype, int num_sms, cudaStream_t s) {
  (void)num_sms;
  const int64_t chunks = (a.vocab + kChunk - 1) / kChunk;
  if (a.batch * chunks > 0x7fffffffll || a.batch * a.block > 0x7fffffffll) return cudaErrorInvalidConfiguration;
  if (logits_dtype == DSPARK_DTYPE_FP32)
    constrain_kernel<float><<<(unsigned)(a.batch * chunks), kThreads, 0, s>>>(a, (int)chunks);
  else
    constrain_kernel<__nv_bfloat16><<<(unsigned)(a.batch * chunks), kThreads, 0, s>>>(a, (int)chunks);
  note_launch();
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || !a.keys) return e;
  choose_kernel<<<(unsigned)(a.batch * a.block), 32, 0, s>>>(a, (int)chunks);
  note_launch();
  return cudaGetLastError();
}

}  // namespace dspark
