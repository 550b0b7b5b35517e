// Clipping of a step's gradients by their global norm: n = sqrt(sum g^2),
// out = g * min(1, max_norm / (n + eps)).
//
// Two launches over the same chunks of all tensors: squares into one partial
// sum a block, then every block adds the partial sums in the same order (so
// that all agree on n without an atomic or a third launch) and scales.  The
// tensors' addresses travel as kernel arguments; more than kMost tensors take
// further launches of each kind.

#include "ssm.cuh"

namespace falcon {
namespace {

constexpr int kMost = 512;        // tensors of one launch
constexpr int kThreads = 256;
constexpr int kChunk = 16384;     // elements a block takes at a time
constexpr int kBlocks = 152 * 4;  // of one launch

struct Batch {
  const void* grad[kMost];
  void* out[kMost];
  int64_t count[kMost];
  int64_t first[kMost];  // chunks before this tensor's
  unsigned char dtype[kMost];
  int tensors;
  int64_t chunks;
};

__device__ __forceinline__ int tensor_of(const Batch& p, int64_t chunk) {
  int lo = 0, hi = p.tensors - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (p.first[mid] <= chunk)
      lo = mid;
    else
      hi = mid - 1;
  }
  return lo;
}

__device__ __forceinline__ float block_sum_f64(double v, double* sh, double* total) {
  for (int k = 16; k > 0; k >>= 1) v += __shfl_xor_sync(0xffffffffu, v, k);
  if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = v;
  __syncthreads();
  double s = 0.0;
  for (int w = 0; w < kThreads / 32; ++w) s += sh[w];
  *total = s;
  return (float)s;
}

template <typename E>
__device__ __forceinline__ float chunk_squares(const E* g, int64_t n) {
  constexpr int V = 16 / (int)sizeof(E);
  // elements before the first 16-byte boundary, whole vectors, the rest
  int64_t head = (int64_t)((16 - (reinterpret_cast<uintptr_t>(g) & 15)) & 15) / (int)sizeof(E);
  if (head > n) head = n;
  const int64_t vecs = (n - head) / V, tail = head + vecs * V;
  float s0 = 0.f, s1 = 0.f;
  if (threadIdx.x < head) {
    const float x = load_vec<E, 1>(g + threadIdx.x).v[0];
    s0 = fmaf(x, x, s0);
  }
  if (threadIdx.x < n - tail) {
    const float x = load_vec<E, 1>(g + tail + threadIdx.x).v[0];
    s0 = fmaf(x, x, s0);
  }
#pragma unroll 4
  for (int64_t i = threadIdx.x; i < vecs; i += kThreads) {
    const FloatV<V> x = load_vec<E, V>(g + head + i * V);
#pragma unroll
    for (int k = 0; k < V; k += 2) {
      s0 = fmaf(x.v[k], x.v[k], s0);
      s1 = fmaf(x.v[k + 1], x.v[k + 1], s1);
    }
  }
  return s0 + s1;
}

__global__ void __launch_bounds__(kThreads) clip_squares_kernel(const __grid_constant__ Batch p,
                                                                double* partial) {
  __shared__ double sh[kThreads / 32];
  double acc = 0.0;
  for (int64_t c = blockIdx.x; c < p.chunks; c += gridDim.x) {
    const int k = tensor_of(p, c);
    const int64_t at = (c - p.first[k]) * kChunk;
    const int64_t n = p.count[k] - at < kChunk ? p.count[k] - at : kChunk;
    acc += p.dtype[k] == FALCON_BF16
               ? chunk_squares(static_cast<const __nv_bfloat16*>(p.grad[k]) + at, n)
               : chunk_squares(static_cast<const float*>(p.grad[k]) + at, n);
  }
  double total;
  block_sum_f64(acc, sh, &total);
  if (threadIdx.x == 0) partial[blockIdx.x] = total;
}

template <typename E>
__device__ __forceinline__ void chunk_scale(const E* g, E* o, int64_t n, float c) {
  constexpr int V = 16 / (int)sizeof(E);
  const bool same = (reinterpret_cast<uintptr_t>(g) & 15) == (reinterpret_cast<uintptr_t>(o) & 15);
  int64_t head = (int64_t)((16 - (reinterpret_cast<uintptr_t>(g) & 15)) & 15) / (int)sizeof(E);
  if (head > n || !same) head = n;  // alignments that differ: one element at a time
  const int64_t vecs = (n - head) / V, tail = head + vecs * V;
  for (int64_t i = threadIdx.x; i < head; i += kThreads)
    store_vec<E, 1>(o + i, FloatV<1>{{load_vec<E, 1>(g + i).v[0] * c}});
  for (int64_t i = tail + threadIdx.x; i < n; i += kThreads)
    store_vec<E, 1>(o + i, FloatV<1>{{load_vec<E, 1>(g + i).v[0] * c}});
#pragma unroll 4
  for (int64_t i = threadIdx.x; i < vecs; i += kThreads) {
    FloatV<V> x = load_vec<E, V>(g + head + i * V);
#pragma unroll
    for (int k = 0; k < V; ++k) x.v[k] *= c;
    store_vec<E, V>(o + head + i * V, x);
  }
}

__global__ void __launch_bounds__(kThreads) clip_scale_kernel(const __grid_constant__ Batch p,
                                                              const double* partial, int parts,
                                                              float max_norm, float eps,
                                                              float* norm) {
  __shared__ double sh[kThreads / 32];
  double acc = 0.0;
  for (int i = threadIdx.x; i < parts; i += kThreads) acc += partial[i];
  double total;
  block_sum_f64(acc, sh, &total);
  const float n = (float)sqrt(total);
  if (norm && blockIdx.x == 0 && threadIdx.x == 0) *norm = n;
  const float ratio = max_norm / (n + eps);
  const float c = ratio > 1.f ? 1.f : ratio;  // a NaN stays
  for (int64_t i = blockIdx.x; i < p.chunks; i += gridDim.x) {
    const int k = tensor_of(p, i);
    if (c == 1.f && p.grad[k] == p.out[k]) continue;
    const int64_t at = (i - p.first[k]) * kChunk;
    const int64_t m = p.count[k] - at < kChunk ? p.count[k] - at : kChunk;
    if (p.dtype[k] == FALCON_BF16)
      chunk_scale(static_cast<const __nv_bfloat16*>(p.grad[k]) + at,
                  static_cast<__nv_bfloat16*>(p.out[k]) + at, m, c);
    else
      chunk_scale(static_cast<const float*>(p.grad[k]) + at, static_cast<float*>(p.out[k]) + at, m,
                  c);
  }
}

// Fills p with the next tensors from `at` on; returns the index after them.
int64_t fill(Batch* p, const falcon_grad* grads, int64_t tensors, int64_t at) {
  p->tensors = 0;
  p->chunks = 0;
  for (; at < tensors && p->tensors < kMost; ++at) {
    if (grads[at].count == 0) continue;
    const int k = p->tensors++;
    p->grad[k] = grads[at].grad;
    p->out[k] = grads[at].out;
    p->count[k] = grads[at].count;
    p->dtype[k] = (unsigned char)grads[at].dtype;
    p->first[k] = p->chunks;
    p->chunks += (grads[at].count + kChunk - 1) / kChunk;
  }
  return at;
}

unsigned blocks_of(const Batch& p) {
  return (unsigned)(p.chunks < kBlocks ? (p.chunks > 0 ? p.chunks : 1) : kBlocks);
}

}  // namespace

size_t clip_workspace_bytes(const falcon_grad*, int64_t tensors) {
  return sizeof(double) * kBlocks * (size_t)((tensors + kMost - 1) / kMost + 1);
}

cudaError_t launch_clip(const falcon_grad* grads, int64_t tensors, float max_norm, float eps,
                        float* norm, void* ws, cudaStream_t stream) {
  static thread_local Batch p;
  double* partial = static_cast<double*>(ws);
  int parts = 0;
  int64_t at = 0;
  do {
    at = fill(&p, grads, tensors, at);
    const unsigned blocks = blocks_of(p);
    clip_squares_kernel<<<blocks, kThreads, 0, stream>>>(p, partial + parts);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    parts += (int)blocks;
  } while (at < tensors);
  at = 0;
  bool first = true;
  do {
    at = fill(&p, grads, tensors, at);
    clip_scale_kernel<<<blocks_of(p), kThreads, 0, stream>>>(p, partial, parts, max_norm, eps,
                                                            first ? norm : nullptr);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    first = false;
  } while (at < tensors);
  return cudaSuccess;
}

}  // namespace falcon
