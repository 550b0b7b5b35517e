// Clipping of a step's gradients by their global norm: n = sqrt(sum g^2),
// out = g * min(1, max_norm / (n + eps)).
//
// Two launches over the same chunks of all tensors: squares into one partial
// sum a block, then every block adds the partial sums in the same order (so
// that all agree on n without an atomic or a third launch) and scales, from the
// back, where L2 still holds what the first launch read last.  The
// tensors' addresses travel as kernel arguments; more than kMost tensors take
// further launches of each kind (arguments for 64 instead of 512 tensors save nothing:
// 1 to 61 small tensors take 4.8 to 5.7 us in a graph, and 12 to 36 us a call, with either).
//
// Bound by memory: 88 M bf16 gradients (177 MB) 84 us a call in a graph, 32 and 54 us each
// launch alone; reading them twice and writing them once at a copy's rate takes 78.  The
// order and the marks save 1.5 to 2.5 us of a call's 90: scaling from the front takes 91.2,
// all loads of the first pass marked as passing 92.2, none 91.1.  Measured and not
// kept: finding the next chunk's tensor while a chunk's loads are under way (98 us: the
// registers cost more blocks than the search costs time), four vectors a batch with
// more blocks (94).

#include "ssm.cuh"

namespace falcon {
namespace {

constexpr int kMost = 512;        // tensors of one launch
constexpr int kThreads = 256;
// Elements a block takes at a time: many of a large set, where finding a chunk's
// tensor should cost little beside it, few of a small one, where all blocks
// should have some.
constexpr int kChunkMost = 16384, kChunkLeast = 4096;
constexpr int64_t kLarge = 152LL * 4 * kChunkMost;
// Bytes read last in the first pass that the second finds in L2 (of 126 MB, each
// half of which may hold its own copy); what comes before is marked as passing.
constexpr int64_t kStays = 40LL << 20;
// Blocks of a launch: what the SMs hold at once.
constexpr int kSquareBlocks = 152 * 4, kScaleBlocks = 152 * 3;

struct Batch {
  const void* grad[kMost];
  void* out[kMost];
  int64_t count[kMost];
  int64_t first[kMost];  // chunks before this tensor's
  unsigned char dtype[kMost];
  int tensors, chunk;
  int64_t chunks, passing;  // chunks of the batch, those not to be kept in L2
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

// Sum over the block, for thread 0.
__device__ __forceinline__ double block_sum_f64(double v, double* sh) {
  for (int k = 16; k > 0; k >>= 1) v += __shfl_xor_sync(0xffffffffu, v, k);
  if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = v;
  __syncthreads();
  double s = 0.0;
  if (threadIdx.x == 0)
    for (int w = 0; w < kThreads / 32; ++w) s += sh[w];
  return s;
}

// A block's part of a tensor as 16-byte vectors between the elements before the
// first 16-byte boundary and those after the last.
struct Span {
  int head, vecs, tail;  // elements, vectors, first element of the rest
  __device__ __forceinline__ Span(const void* p, int n, int esz, bool vectors) {
    head = (int)((16 - (reinterpret_cast<uintptr_t>(p) & 15)) & 15) / esz;
    if (!vectors || head > n) head = n;
    vecs = (n - head) / (16 / esz);
    tail = head + vecs * (16 / esz);
  }
};
constexpr int kBatch = 8;  // vectors of a thread under way at a time

// A thread's squares of a chunk are summed in float32, which holds them to 2^-19 while
// the sum is neither infinite nor so small that squares may have vanished below
// float32's range; where it is, or where a value is no number, the thread takes its
// elements again in float64.
constexpr float kLeastSum = 7.9e-31f;  // about 2^-100: what vanishes is below 2^-40 of it

template <typename E>
__device__ __noinline__ double chunk_squares_f64(const E* g, int n, Span s) {
  constexpr int V = 16 / (int)sizeof(E);
  double sum = 0.0;
  auto add = [&](int i) {
    const double x = load_vec<E, 1>(g + i).v[0];
    sum = fma(x, x, sum);
  };
  if ((int)threadIdx.x < s.head) add(threadIdx.x);
  if ((int)threadIdx.x < n - s.tail) add(s.tail + threadIdx.x);
  for (int i = threadIdx.x; i < s.vecs; i += kThreads)
    for (int k = 0; k < V; ++k) add(s.head + i * V + k);
  return sum;
}

template <typename E>
__device__ __forceinline__ double chunk_squares(const E* g, int n, bool passing) {
  constexpr int V = 16 / (int)sizeof(E);
  const Span s(g, n, (int)sizeof(E), true);
  float s0 = 0.f, s1 = 0.f;
  uint32_t bits = 0;  // of all elements: zero where every one is zero
  auto edge = [&](int i) {
    const float x = load_vec<E, 1>(g + i).v[0];
    s0 = fmaf(x, x, s0);
    bits |= __float_as_uint(x);
  };
  if ((int)threadIdx.x < s.head) edge(threadIdx.x);
  if ((int)threadIdx.x < n - s.tail) edge(s.tail + threadIdx.x);
  for (int i0 = threadIdx.x; i0 < s.vecs; i0 += kThreads * kBatch) {
    uint4 q[kBatch];
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      const int i = i0 + j * kThreads;
      const uint4* from = reinterpret_cast<const uint4*>(g + s.head) + i;
      q[j] = make_uint4(0, 0, 0, 0);
      if (i < s.vecs) q[j] = passing ? __ldcs(from) : *from;
    }
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      const FloatV<V> x = load_vec<E, V>(reinterpret_cast<const E*>(&q[j]));
#pragma unroll
      for (int k = 0; k < V; k += 2) {
        s0 = fmaf(x.v[k], x.v[k], s0);
        s1 = fmaf(x.v[k + 1], x.v[k + 1], s1);
      }
      bits |= q[j].x | q[j].y | q[j].z | q[j].w;
    }
  }
  const float sum = s0 + s1;
  if (!(sum <= kLargest) || (sum < kLeastSum && bits != 0)) return chunk_squares_f64(g, n, s);
  return sum;
}

__global__ void __launch_bounds__(kThreads)
    clip_squares_kernel(const __grid_constant__ Batch p, double* partial) {
  __shared__ double sh[kThreads / 32];
  double acc = 0.0;
  for (int64_t c = blockIdx.x; c < p.chunks; c += gridDim.x) {
    const int k = tensor_of(p, c);
    const int64_t at = (c - p.first[k]) * p.chunk;
    const int n = (int)(p.count[k] - at < p.chunk ? p.count[k] - at : p.chunk);
    acc += p.dtype[k] == FALCON_BF16
               ? chunk_squares(static_cast<const __nv_bfloat16*>(p.grad[k]) + at, n, c < p.passing)
               : chunk_squares(static_cast<const float*>(p.grad[k]) + at, n, c < p.passing);
  }
  const double total = block_sum_f64(acc, sh);
  if (threadIdx.x == 0) partial[blockIdx.x] = total;
}

template <typename E>
__device__ __forceinline__ void chunk_scale(const E* g, E* o, int n, float c) {
  constexpr int V = 16 / (int)sizeof(E);
  // alignments that differ: one element at a time
  const bool same = (reinterpret_cast<uintptr_t>(g) & 15) == (reinterpret_cast<uintptr_t>(o) & 15);
  const Span s(g, n, (int)sizeof(E), same);
  for (int i = threadIdx.x; i < s.head; i += kThreads)
    store_vec<E, 1>(o + i, FloatV<1>{{load_vec<E, 1>(g + i).v[0] * c}});
  for (int i = s.tail + threadIdx.x; i < n; i += kThreads)
    store_vec<E, 1>(o + i, FloatV<1>{{load_vec<E, 1>(g + i).v[0] * c}});
  for (int i0 = threadIdx.x; i0 < s.vecs; i0 += kThreads * kBatch) {
    uint4 q[kBatch];
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      const int i = i0 + j * kThreads;
      if (i < s.vecs) q[j] = __ldcs(reinterpret_cast<const uint4*>(g + s.head) + i);
    }
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      const int i = i0 + j * kThreads;
      if (i < s.vecs) {
        FloatV<V> x = load_vec<E, V>(reinterpret_cast<const E*>(&q[j]));
#pragma unroll
        for (int k = 0; k < V; ++k) x.v[k] *= c;
        uint4 r;
        store_vec<E, V>(reinterpret_cast<E*>(&r), x);
        __stcs(reinterpret_cast<uint4*>(o + s.head) + i, r);  // not read again here
      }
    }
  }
}

__global__ void __launch_bounds__(kThreads)
    clip_scale_kernel(const __grid_constant__ Batch p, const double* partial, int parts,
                      float max_norm, float eps, float* norm) {
  __shared__ double sh[kThreads / 32];
  __shared__ float factor;
  cudaGridDependencySynchronize();
  double acc = 0.0;
  for (int i = threadIdx.x; i < parts; i += kThreads) acc += partial[i];
  acc = block_sum_f64(acc, sh);
  if (threadIdx.x == 0) {
    // in float64: gradients that float32 holds can have a norm that it does not
    const double n = sqrt(acc);
    if (norm && blockIdx.x == 0) *norm = (float)n;
    const double ratio = (double)max_norm / (n + (double)eps);
    factor = ratio > 1.0 ? 1.f : (float)ratio;  // a NaN stays
  }
  __syncthreads();
  const float c = factor;
  // from the back: the first pass has left the last chunks in L2
  for (int64_t i = p.chunks - 1 - blockIdx.x; i >= 0; i -= gridDim.x) {
    const int k = tensor_of(p, i);
    if (c == 1.f && p.grad[k] == p.out[k]) continue;
    const int64_t at = (i - p.first[k]) * p.chunk;
    const int m = (int)(p.count[k] - at < p.chunk ? p.count[k] - at : p.chunk);
    if (p.dtype[k] == FALCON_BF16)
      chunk_scale(static_cast<const __nv_bfloat16*>(p.grad[k]) + at,
                  static_cast<__nv_bfloat16*>(p.out[k]) + at, m, c);
    else
      chunk_scale(static_cast<const float*>(p.grad[k]) + at, static_cast<float*>(p.out[k]) + at, m,
                  c);
  }
}

// Fills p with the next tensors from `at` on; returns the index after them.
int64_t fill(Batch* p, const falcon_grad* grads, int64_t tensors, int64_t at, int chunk) {
  p->tensors = 0;
  p->chunk = chunk;
  p->chunks = 0;
  int64_t bytes = 0;
  for (; at < tensors && p->tensors < kMost; ++at) {
    if (grads[at].count == 0) continue;
    const int k = p->tensors++;
    p->grad[k] = grads[at].grad;
    p->out[k] = grads[at].out;
    p->count[k] = grads[at].count;
    p->dtype[k] = (unsigned char)grads[at].dtype;
    p->first[k] = p->chunks;
    p->chunks += (grads[at].count + chunk - 1) / chunk;
    bytes += grads[at].count * (grads[at].dtype == FALCON_BF16 ? 2 : 4);
  }
  p->passing = bytes > kStays ? (int64_t)((double)(bytes - kStays) / bytes * p->chunks) : 0;
  return at;
}

}  // namespace

size_t clip_workspace_bytes(const falcon_grad*, int64_t tensors) {
  return sizeof(double) * kSquareBlocks * (size_t)((tensors + kMost - 1) / kMost + 1);
}

cudaError_t launch_clip(const falcon_grad* grads, int64_t tensors, float max_norm, float eps,
                        float* norm, void* ws, cudaStream_t stream) {
  double* partial = static_cast<double*>(ws);
  static thread_local Batch p;
  auto blocks_of = [](int most) {
    return (unsigned)(p.chunks < 1 ? 1 : p.chunks < most ? p.chunks : most);
  };
  int64_t all = 0;
  for (int64_t i = 0; i < tensors; ++i) all += grads[i].count;
  const int chunk = all >= kLarge ? kChunkMost : kChunkLeast;
  int parts = 0;
  int64_t at = 0;
  do {
    at = fill(&p, grads, tensors, at, chunk);
    const unsigned blocks = blocks_of(kSquareBlocks);
    clip_squares_kernel<<<blocks, kThreads, 0, stream>>>(p, partial + parts);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    parts += (int)blocks;
  } while (at < tensors);
  const bool again = tensors > kMost;  // otherwise p still holds all of them
  at = again ? 0 : tensors;
  do {
    if (again) at = fill(&p, grads, tensors, at, chunk);
    // set up while the launch before it ends; it waits for that launch's results
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(blocks_of(kScaleBlocks));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = stream;
    cudaLaunchAttribute early[1];
    early[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    early[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = early;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, clip_scale_kernel, p, (const double*)partial,
                                             parts, max_norm, eps, norm);
    norm = nullptr;
    if (e != cudaSuccess) return e;
  } while (at < tensors);
  return cudaSuccess;
}

}  // namespace falcon
