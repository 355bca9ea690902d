// The global norm over many gradient tensors, and clipping by it:
// norm = sqrt(sum over tensors of sum g^2), out = g min(1, max / (norm + 1e-6)).
//
// The scale needs the whole norm, so the gradients are read twice and written
// once; what the second reading still finds in L2 costs no DRAM traffic. The
// plan cuts the tensors into pieces of at most kClipPieceBytes. One kernel sums
// squares, a double for each CTA; the next adds those in one order and scales,
// each CTA its own pieces again, the last first, since they were read last.
// Small plans run both passes in one cluster, with its barrier between them.
//
// Two readings and a writing of 132 MB (two fp32 [129280, 128]) take 68 us, 5.8
// TB/s counted so and bound by memory: of the second reading 79 MB come from
// DRAM, the rest is still in L2 (126 MB). 55 MB in 182 tensors of both types
// take 34.5 us: the second reading finds all of it in L2, but pieces in turn
// give the fullest CTA 1.58 times the mean bytes (1.10 in the larger case). A
// plan of one to eight pieces takes 8 us, of which most is the launch.
//
// Squares of four elements are summed in 32 bits and then in 64. A group whose
// sum leaves the range in which that is exact to a few roundings (it overflows,
// or an element that is not zero vanishes) is summed again in 64 bits.
#include <cmath>

#include "common.cuh"
#include "cluster.cuh"
#include "kernels.h"

namespace dspark {

namespace {

constexpr int kThreads = 256;
constexpr int kCtasPerSm = 3;
constexpr int kInFlight = 8;  // 16-byte vectors per thread
constexpr int kSmallCtas = 8;
// Plans of one cluster: a piece for each of its CTAs, 512 KB in all. Eight pieces
// take 5.7 us from a graph and 7.8 as called from Python, 5.9 and 10.5 in two
// launches; sixteen would take 8.8 and 10.3, in two launches 6.0 and 10.6.
constexpr int64_t kSmallPieces = kSmallCtas;

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

// Four squares whose 32-bit sum holds, or in 64 bits.
__device__ __forceinline__ double squares4(float a, float b, float c, float d) {
  const float s = fmaf(a, a, b * b) + fmaf(c, c, d * d);
  // Below 2^-100 an element that vanished could count; zeros are common.
  if (s >= 0x1p-100f && s < INFINITY) return (double)s;
  if (s == 0.0f && a == 0.0f && b == 0.0f && c == 0.0f && d == 0.0f) return 0.0;
  return (double)a * a + (double)b * b + ((double)c * c + (double)d * d);
}

template <typename T>
struct Piece;
template <>
struct Piece<float> {
  static constexpr int kE = 4;
  static __device__ __forceinline__ double squares(const uint4& r) {
    return squares4(__uint_as_float(r.x), __uint_as_float(r.y), __uint_as_float(r.z), __uint_as_float(r.w));
  }
  static __device__ __forceinline__ uint4 scaled(const uint4& r, float c) {
    return make_uint4(__float_as_uint(__uint_as_float(r.x) * c), __float_as_uint(__uint_as_float(r.y) * c),
                      __float_as_uint(__uint_as_float(r.z) * c), __float_as_uint(__uint_as_float(r.w) * c));
  }
};
template <>
struct Piece<__nv_bfloat16> {
  static constexpr int kE = 8;
  static __device__ __forceinline__ float lo(uint32_t w) { return __uint_as_float(w << 16); }
  static __device__ __forceinline__ float hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
  static __device__ __forceinline__ double squares(const uint4& r) {
    return squares4(lo(r.x), hi(r.x), lo(r.y), hi(r.y)) + squares4(lo(r.z), hi(r.z), lo(r.w), hi(r.w));
  }
  static __device__ __forceinline__ uint32_t scaled2(uint32_t w, float c) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo(w) * c, hi(w) * c);
    return *reinterpret_cast<const uint32_t*>(&v);
  }
  static __device__ __forceinline__ uint4 scaled(const uint4& r, float c) {
    return make_uint4(scaled2(r.x, c), scaled2(r.y, c), scaled2(r.z, c), scaled2(r.w, c));
  }
};

// Elements of a piece before its first 16-byte address.
template <typename T>
__device__ __forceinline__ int head_of(const T* g, int n) {
  const int past = (int)((reinterpret_cast<uintptr_t>(g) / sizeof(T)) % Piece<T>::kE);
  return min(past ? Piece<T>::kE - past : 0, n);
}

template <typename T>
__device__ __forceinline__ double piece_squares(const T* g, int n) {
  constexpr int kE = Piece<T>::kE;
  const int head = head_of(g, n), vecs = (n - head) / kE, tid = (int)threadIdx.x;
  const uint4* from = reinterpret_cast<const uint4*>(g + head);
  double s = 0.0;
  for (int j = tid; j < vecs; j += kThreads * kInFlight) {
    uint4 raw[kInFlight];
#pragma unroll
    for (int u = 0; u < kInFlight; ++u)
      raw[u] = j + u * kThreads < vecs ? from[j + u * kThreads] : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
    for (int u = 0; u < kInFlight; ++u) s += Piece<T>::squares(raw[u]);
  }
  for (int i = tid; i < n - vecs * kE; i += kThreads) {  // fewer than two vectors' elements at the edges
    const double x = (double)to_f32(g[i < head ? i : i + vecs * kE]);
    s += x * x;
  }
  return s;
}

template <typename T>
__device__ __forceinline__ void scale_piece(const T* g, T* out, int n, float c) {
  constexpr int kE = Piece<T>::kE;
  const int tid = (int)threadIdx.x;
  if ((reinterpret_cast<uintptr_t>(g) - reinterpret_cast<uintptr_t>(out)) % 16 != 0) {
    for (int i = tid; i < n; i += kThreads) out[i] = from_f32<T>(to_f32(g[i]) * c);
    return;
  }
  const int head = head_of(g, n), vecs = (n - head) / kE;
  const uint4* from = reinterpret_cast<const uint4*>(g + head);
  uint4* to = reinterpret_cast<uint4*>(out + head);
  for (int j = tid; j < vecs; j += kThreads * kInFlight) {
    uint4 raw[kInFlight];
#pragma unroll
    for (int u = 0; u < kInFlight; ++u)
      if (j + u * kThreads < vecs) raw[u] = from[j + u * kThreads];
    // Written past the caches' keeping: what is still to be read stays in L2.
#pragma unroll
    for (int u = 0; u < kInFlight; ++u)
      if (j + u * kThreads < vecs) __stcs(to + j + u * kThreads, Piece<T>::scaled(raw[u], c));
  }
  for (int i = tid; i < n - vecs * kE; i += kThreads) {
    const int at = i < head ? i : i + vecs * kE;
    out[at] = from_f32<T>(to_f32(g[at]) * c);
  }
}

// This CTA's pieces are blockIdx.x, blockIdx.x + gridDim.x, ...; the next
// record is read while a piece is worked on.
__device__ __forceinline__ double sum_pieces(const ClipArgs& a) {
  double s = 0.0;
  dspark_markov_clip_piece next{};
  if (blockIdx.x < a.pieces) next = a.plan[blockIdx.x];
  for (int64_t p = blockIdx.x; p < a.pieces; p += gridDim.x) {
    const dspark_markov_clip_piece q = next;
    if (p + gridDim.x < a.pieces) next = a.plan[p + gridDim.x];
    s += q.dtype == DSPARK_DTYPE_FP32 ? piece_squares(static_cast<const float*>(q.grad), q.count)
                                      : piece_squares(static_cast<const __nv_bfloat16*>(q.grad), q.count);
  }
  return s;
}

__device__ __forceinline__ float factor_of(double norm, double max_norm) {
  if (isinf(max_norm)) return 1.0f;  // measured only, whatever the norm
  const double ratio = max_norm / (norm + 1e-6);
  return ratio > 1.0 ? 1.0f : (float)ratio;  // NaN stays NaN
}

// The same pieces, the last first.
__device__ __forceinline__ void scale_pieces(const ClipArgs& a, float c) {
  const int64_t mine = a.pieces > blockIdx.x ? (a.pieces - 1 - blockIdx.x) / gridDim.x : -1;
  dspark_markov_clip_piece next{};
  if (mine >= 0) next = a.plan[mine * gridDim.x + blockIdx.x];
  for (int64_t k = mine; k >= 0; --k) {
    const dspark_markov_clip_piece q = next;
    if (k > 0) next = a.plan[(k - 1) * gridDim.x + blockIdx.x];
    if (c == 1.0f && q.out == q.grad) continue;
    if (q.dtype == DSPARK_DTYPE_FP32)
      scale_piece(static_cast<const float*>(q.grad), static_cast<float*>(q.out), q.count, c);
    else
      scale_piece(static_cast<const __nv_bfloat16*>(q.grad), static_cast<__nv_bfloat16*>(q.out), q.count, c);
  }
}

__global__ void __launch_bounds__(kThreads, kCtasPerSm) clip_norm_kernel(ClipArgs a) {
  __shared__ double parts[kThreads / 32];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const double s = block_sum(sum_pieces(a), parts);
  if (threadIdx.x == 0) a.partials[blockIdx.x] = s;
}

__global__ void __launch_bounds__(kThreads, kCtasPerSm) clip_scale_kernel(ClipArgs a) {
  __shared__ double parts[kThreads / 32];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  double s = 0.0;
  for (int i = threadIdx.x; i < (int)gridDim.x; i += kThreads) s += a.partials[i];
  const double norm = sqrt(block_sum(s, parts));
  if (blockIdx.x == 0 && threadIdx.x == 0) *a.norm = (float)norm;
  scale_pieces(a, factor_of(norm, a.max_norm));
}

// Both passes in one cluster.
__global__ void __launch_bounds__(kThreads, kCtasPerSm) clip_small_kernel(ClipArgs a) {
  __shared__ double parts[kThreads / 32], sums[kSmallCtas];
  const double s = block_sum(sum_pieces(a), parts);
  cluster_barrier();  // every CTA's shared memory is there
  if (threadIdx.x < kSmallCtas) {
    const uint32_t to = remote_u32(&sums[blockIdx.x], threadIdx.x);
    asm volatile("st.shared::cluster.f64 [%0], %1;" ::"r"(to), "d"(s) : "memory");
  }
  __syncwarp();
  cluster_barrier();
  double total = 0.0;
  for (int k = 0; k < kSmallCtas; ++k) total += sums[k];
  const double norm = sqrt(total);
  if (blockIdx.x == 0 && threadIdx.x == 0) *a.norm = (float)norm;
  scale_pieces(a, factor_of(norm, a.max_norm));
}

}  // namespace

cudaError_t launch_clip(const ClipArgs& a, int num_sms, cudaStream_t s) {
  cudaLaunchConfig_t cfg{};
  cfg.blockDim = dim3(kThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr{};
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  cudaError_t e;
  if (a.pieces <= kSmallPieces) {
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim = {kSmallCtas, 1, 1};
    cfg.gridDim = dim3(kSmallCtas);
    e = cudaLaunchKernelEx(&cfg, clip_small_kernel, a);
    note_launch();
    return e;
  }
  int64_t grid = (int64_t)num_sms * kCtasPerSm;
  if (grid > DSPARK_CLIP_MAX_PARTIALS) grid = DSPARK_CLIP_MAX_PARTIALS;
  if (grid > a.pieces) grid = a.pieces;
  clip_norm_kernel<<<(unsigned)grid, kThreads, 0, s>>>(a);
  note_launch();
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3((unsigned)grid);
  e = cudaLaunchKernelEx(&cfg, clip_scale_kernel, a);
  note_launch();
  return e;
}

}  // namespace dspark
