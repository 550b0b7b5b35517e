// Shared by the kernels of the gated norm (gated_norm.cu, gated_norm_bwd.cu): a row's
// layout over threads, its sums, and the choice of a launch shape.
#pragma once

#include "linear.cuh"

namespace falcon {
namespace {

// How a head's sum is formed.
enum { kWhole = 0,   // one head: the threads of a row
       kLanes = 1,   // m / V threads, a power of two up to 32, side by side in a warp
       kStaged = 2   // any: products in shared memory, a warp a head
};

// V neighbouring elements as they lie in memory: a row's inputs wait in registers in half
// the space that bf16 takes as fp32.
template <typename E, int V>
struct Held {
  static constexpr bool kPairs = sizeof(E) == 2 && V > 1;
  static constexpr int kWords = kPairs ? V / 2 : V;
  uint32_t w[kWords];
  __device__ __forceinline__ float get(int i) const {
    if constexpr (kPairs) return i & 1 ? bf16_hi(w[i / 2]) : bf16_lo(w[i / 2]);
    return __uint_as_float(w[i]);
  }
};
// As fp32.
template <typename E, int V>
__device__ __forceinline__ FloatV<V> wide(const Held<E, V>& h) {
  FloatV<V> r;
#pragma unroll
  for (int i = 0; i < V; ++i) r.v[i] = h.get(i);
  return r;
}
template <int V>
__device__ __forceinline__ FloatV<V> times(const FloatV<V>& x, float s) {
  FloatV<V> t;
#pragma unroll
  for (int i = 0; i < V; ++i) t.v[i] = s;
  return mul_vec<V>(x, t);
}
template <int V>
__device__ __forceinline__ FloatV<V> mul_of(const FloatV<V>& x, const FloatV<V>& y) {
  return mul_vec<V>(x, y);
}
template <int V>
__device__ __forceinline__ FloatV<V> fma_of(const FloatV<V>& x, const FloatV<V>& y,
                                            const FloatV<V>& z) {
  return fma_vec<V>(x, y, z);
}
// x s + z
template <int V>
__device__ __forceinline__ FloatV<V> fma_of(const FloatV<V>& x, float s, const FloatV<V>& z) {
  FloatV<V> t;
#pragma unroll
  for (int i = 0; i < V; ++i) t.v[i] = s;
  return fma_vec<V>(x, t, z);
}
// acc + sum of a b, in two partial sums.
template <int V>
struct Dot {
  FloatV<2> two = {{0.f, 0.f}};
  __device__ __forceinline__ void add(const FloatV<V>& a, const FloatV<V>& b) {
    if constexpr (V == 1) {
      two.v[0] = fmaf(a.v[0], b.v[0], two.v[0]);
    } else {
#pragma unroll
      for (int i = 0; i < V; i += 2)
        two = fma_vec<2>({{a.v[i], a.v[i + 1]}}, {{b.v[i], b.v[i + 1]}}, two);
    }
  }
  __device__ __forceinline__ float sum() const { return two.v[0] + two.v[1]; }
};
// V elements stored where `live`, zeros for a row that holds no token.
template <typename E, int V>
__device__ __forceinline__ void put_vec(E* p, const FloatV<V>& x, bool live, bool held) {
  if (!live) return;
  if constexpr (Held<E, V>::kPairs) {
    uint32_t w[V / 2];
#pragma unroll
    for (int i = 0; i < V / 2; ++i) w[i] = held ? pack_bf16(x.v[2 * i], x.v[2 * i + 1]) : 0u;
    *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
  } else {
    FloatV<V> y;
#pragma unroll
    for (int i = 0; i < V; ++i) y.v[i] = held ? x.v[i] : 0.f;
    store_vec<E, V>(p, y);
  }
}

// Inputs of the rows ahead wait in shared memory: a thread copies what it will read
// itself (cp.async, 16 bytes), so that nobody waits for another's copies, and registers
// hold one row only.  Rows on no such boundary are loaded into registers, one row ahead.
template <typename E, int V>
struct Slot {
  static constexpr int kBytes = V * sizeof(E);
  static constexpr bool kAhead = kBytes == 16;
};
template <typename E>
__device__ __forceinline__ void copy_ahead(unsigned char* to, const E* from, bool live) {
  const uint32_t dst = static_cast<uint32_t>(__cvta_generic_to_shared(to));
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(from),
               "r"(live ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void ahead_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
// All but the newest `n` groups (0 .. 3) have arrived.
__device__ __forceinline__ void ahead_wait(int n) {
  if (n >= 3)
    asm volatile("cp.async.wait_group 3;" ::: "memory");
  else if (n == 2)
    asm volatile("cp.async.wait_group 2;" ::: "memory");
  else if (n == 1)
    asm volatile("cp.async.wait_group 1;" ::: "memory");
  else
    asm volatile("cp.async.wait_group 0;" ::: "memory");
}
// An input's vector out of its slot.
template <typename E, int V>
__device__ __forceinline__ Held<E, V> slot_vec(const unsigned char* slot) {
  const uint4 q = *reinterpret_cast<const uint4*>(slot);
  return {{q.x, q.y, q.z, q.w}};
}
// An input's element out of memory, without a branch: all loads are under way at once.
template <typename E>
__device__ __forceinline__ Held<E, 1> load_own(const E* from, bool live) {
  const float x = load_vec<E, 1>(from).v[0];
  return {{live ? __float_as_uint(x) : 0u}};
}

template <typename E, int V>
__device__ __forceinline__ FloatV<V> zeros() {
  FloatV<V> r;
#pragma unroll
  for (int i = 0; i < V; ++i) r.v[i] = 0.f;
  return r;
}

// The channels' parameters in shared memory, read for every row: weight times scale, and
// next_weight (ones where there are none).
__device__ __forceinline__ void stage_params(const NormArgs& a, float* to) {
  const int threads = blockDim.x * blockDim.y;
  for (int c = threadIdx.y * blockDim.x + threadIdx.x; c < a.D; c += threads) {
    const float w = a.weight ? a.weight[c] : 1.f;
    to[c] = a.scale ? w * a.scale[c] : w;
    if (a.next_weight) to[a.D + c] = a.next_weight[c];
  }
  __syncthreads();
}
template <int V>
__device__ __forceinline__ FloatV<V> param_vec(const float* p) {
  FloatV<V> r;
  constexpr int Q = V < 4 ? V : 4;
#pragma unroll
  for (int i = 0; i < V; i += Q) {
    const FloatV<Q> q = load_vec<float, Q>(p + i);
#pragma unroll
    for (int j = 0; j < Q; ++j) r.v[i + j] = q.v[j];
  }
  return r;
}

// The threads of one row of a block (rows of whole warps).
__device__ __forceinline__ void row_sync(int nt) {
  asm volatile("bar.sync %0, %1;" ::"r"((int)threadIdx.y + 1), "r"(nt) : "memory");
}

// Sums of N values over the nt threads of a row (a power of two up to 32, or whole
// warps); `red` holds 2 x 32 pairs a row, `turn` says which were used last.
template <int N>
struct Sums {
  float v[N];
};
template <int N>
__device__ __forceinline__ Sums<N> row_sum(Sums<N> x, int nt, float2* red, int& turn) {
  if (nt >= 32) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
#pragma unroll
      for (int i = 0; i < N; ++i) x.v[i] += __shfl_xor_sync(0xffffffffu, x.v[i], o);
  } else {
    for (int o = nt / 2; o > 0; o >>= 1)
#pragma unroll
      for (int i = 0; i < N; ++i) x.v[i] += __shfl_xor_sync(0xffffffffu, x.v[i], o);
  }
  if (nt <= 32) return x;
  turn ^= 32;
  red += turn;
  if (threadIdx.x % 32 == 0) red[threadIdx.x / 32] = make_float2(x.v[0], x.v[N - 1]);
  row_sync(nt);
  float2 s = red[0];
  for (int w = 1; w < nt / 32; ++w) s.x += red[w].x, s.y += red[w].y;
  x.v[0] = s.x;
  if (N > 1) x.v[N - 1] = s.y;
  return x;
}

// act(z), and act'(z)
template <typename E, int V>
__device__ __forceinline__ FloatV<V> gates(const Held<E, V>& z, int gate) {
  FloatV<V> g;
#pragma unroll
  for (int i = 0; i < V; ++i) g.v[i] = z.get(i);
  if (gate == FALCON_ACT_IDENTITY) return g;
  if (gate == FALCON_ACT_SIGMOID) {
#pragma unroll
    for (int i = 0; i < V; ++i) g.v[i] = sigmoid(g.v[i]);
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) g.v[i] *= sigmoid(g.v[i]);
  }
  return g;
}
template <typename E, int V>
__device__ __forceinline__ FloatV<V> slopes(const Held<E, V>& z, int gate) {
  FloatV<V> s;
#pragma unroll
  for (int i = 0; i < V; ++i) s.v[i] = 1.f;
  if (gate == FALCON_ACT_IDENTITY) return s;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    // 1 - p is e^{-x} p where x > 0: the difference would be p's rounding there
    const float x = z.get(i), p = sigmoid(x);
    const float q = x > 0.f ? exp2_approx(-x * kLog2e) * p : 1.f - p;
    s.v[i] = gate == FALCON_ACT_SIGMOID ? p * q : p * fmaf(x, q, 1.f);
  }
  return s;
}

// (b, t) of the row that lies step_b batches and step_t < T tokens further on; no sum passes
// 2^31 on the way, however long a row.
__host__ __device__ __forceinline__ void advance_row(unsigned& b, int& t, int step_b, int step_t,
                                                     int T) {
  b += step_b;
  if (t >= T - step_t)
    t -= T - step_t, ++b;
  else
    t += step_t;
}

// A row of the problem, and the way to the row `step` further on (no division in a loop).
struct RowAt {
  unsigned b;  // runs past 2^31 behind the last row of the largest problem
  int t;
  bool in, held;  // inside the problem; a token of its row
  int step_b, step_t;
  __device__ __forceinline__ RowAt(const NormArgs& a, int64_t row, int64_t step) {
    const unsigned T = (unsigned)a.T;
    b = (unsigned)((uint64_t)row / T), t = (int)(row - (int64_t)b * T);
    step_b = (int)((uint64_t)step / T), step_t = (int)(step - (int64_t)step_b * T);
    look(a);
  }
  __device__ __forceinline__ void look(const NormArgs& a) {
    in = b < (unsigned)a.B;
    held = in && t < row_length(a.lengths, in ? b : 0, a.T);
  }
  __device__ __forceinline__ void advance(const NormArgs& a) {
    advance_row(b, t, step_b, step_t, (int)a.T);
    look(a);
  }
};

// Channel and head of vector k of a thread (the row's first where it has none).
struct Place {
  int c, head;
  bool live;
};
template <int V, int MODE>
__device__ __forceinline__ Place place_of(const NormArgs& a, int k) {
  Place p;
  p.c = (k * (int)blockDim.x + (int)threadIdx.x) * V;
  p.live = p.c < a.D;
  if (!p.live) p.c = 0;
  p.head = MODE == kWhole ? 0 : p.c / a.m;
  return p;
}

// Where the row's tensors begin (the first row's where none is to be read), and vector
// `at` of a head-major one in it.
template <typename E>
__device__ __forceinline__ const E* row_in(const void* p, const falcon_strides& s,
                                           const RowAt& r) {
  return static_cast<const E*>(p) + (r.held ? r.b * s.batch + r.t * s.time : 0);
}
template <typename E>
__device__ __forceinline__ E* row_of(const void* p, const falcon_strides& s, const RowAt& r) {
  return static_cast<E*>(const_cast<void*>(p)) + (r.in ? r.b * s.batch + r.t * s.time : 0);
}
template <int MODE>
__device__ __forceinline__ int64_t in_heads(const NormArgs& a, const falcon_strides& s,
                                            const Place& at) {
  return MODE == kWhole ? at.c : at.head * s.head + (at.c - at.head * a.m);
}

// Sums over each vector's head of N values a vector, in place.
template <int K, int MODE, int N>
__device__ __forceinline__ void head_sums(const NormArgs& a, const Place (&at)[K],
                                          Sums<N> (&x)[K], int V, float2* red, int& turn,
                                          float2* staged) {
  if constexpr (MODE == kWhole) {
    Sums<N> s = x[0];
#pragma unroll
    for (int k = 1; k < K; ++k)
#pragma unroll
      for (int i = 0; i < N; ++i) s.v[i] += x[k].v[i];
    s = row_sum<N>(s, blockDim.x, red, turn);
#pragma unroll
    for (int k = 0; k < K; ++k) x[k] = s;
  } else if constexpr (MODE == kLanes) {
    const int lanes = a.m / V;
    for (int o = lanes / 2; o > 0; o >>= 1)
#pragma unroll
      for (int k = 0; k < K; ++k)
#pragma unroll
        for (int i = 0; i < N; ++i) x[k].v[i] += __shfl_xor_sync(0xffffffffu, x[k].v[i], o);
  } else {
    // a vector lies inside one head (V divides m)
    const int vecs = a.D / V, each = a.m / V;
    float2* mine = staged + (int)threadIdx.y * (vecs + a.H);
    float2* sums = mine + vecs;
    row_sync(blockDim.x);
#pragma unroll
    for (int k = 0; k < K; ++k)
      if (at[k].live) mine[at[k].c / V] = make_float2(x[k].v[0], x[k].v[N - 1]);
    row_sync(blockDim.x);
    const int warps = blockDim.x / 32, lane = threadIdx.x % 32;
    for (int h = threadIdx.x / 32; h < a.H; h += warps) {
      float2 s = make_float2(0.f, 0.f);
      for (int i = lane; i < each; i += 32) {
        const float2 q = mine[h * each + i];
        s.x += q.x, s.y += q.y;
      }
      s.x = warp_sum(s.x);
      if (N > 1) s.y = warp_sum(s.y);
      if (lane == 0) sums[h] = s;
    }
    row_sync(blockDim.x);
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const float2 s = sums[at[k].head];
      x[k].v[0] = s.x;
      if (N > 1) x[k].v[N - 1] = s.y;
    }
  }
}

// Launch shape: V channels a vector, K vectors a thread, nt threads a row, `rows` rows a
// block.
struct NormPlan {
  int V, K, nt, rows, mode;
  int blocks;  // at most
  int ring;    // rows whose inputs are in shared memory at once, one of them being read (V > 1)
  // bytes: of a block's parameters, with its products (kStaged), and in all
  size_t params, staged, shared;
};

bool fits(const void* p, const falcon_strides& s, int V, int esize, bool head) {
  if (!p) return true;
  return reinterpret_cast<uintptr_t>(p) % (uintptr_t)(V * esize) == 0 && s.batch % V == 0 &&
         s.time % V == 0 && (!head || s.head % V == 0);
}

// How many vectors a thread may hold, the threads of a row (and block) at most, and the
// threads of an SM that their registers leave room for.
struct Width {
  int K, threads, resident;
};
// Threads a block aims at.
constexpr int kRowThreads = 128, kNarrowThreads = 256;
// Dynamic shared memory of each of `per` blocks of an SM, beside 5 KB of its own.
constexpr size_t shared_for(int per) { return 228 * 1024 / per - 5 * 1024 - 256; }

// Those of single elements; the last is for the widest rows (2048 fp32 rows of 8190 channels:
// gradient 296 us, 618 with 32 elements in each of 256 threads).  A row ahead in registers
// and loads without branches: 7312 bf16 rows of 1051 channels 38 us, 51 without the row ahead,
// 158 with branches.  Copies of 4 bytes into shared memory were slower still.
constexpr Width kNarrow[] = {{1, 256, 512}, {4, 512, 512}, {8, 512, 512}, {16, 512, 512}};

// widths: rising; the last one has to do for the widest row.  Of those that leave `enough`
// warps in all, the one whose row takes the fewest instructions: about as many for a warp's
// sums and addresses as for 24 values a thread (2048 channels in 128 threads: 107 us, in
// 32: 53 us).  With few rows the narrowest, which spreads a row over the most threads.
// More than `prefer` (single elements: two more) only where that makes a row one warp's, up
// to four (eight), or nothing less will do: a thread's registers.
template <int COUNTS>
NormPlan plan_norm(const NormArgs& a, const Width (&widths)[COUNTS], int prefer, int64_t enough,
                   int inputs, bool narrow) {
  NormPlan p = {};
  const int es = a.dtype == FALCON_BF16 ? 2 : 4;
  p.V = 16 / es;
  auto all = [&](int V) {
    const bool heads = a.H > 1;
    return a.m % V == 0 && fits(a.h, a.hs, V, es, heads) && fits(a.dh, a.dhs, V, es, heads) &&
           fits(a.z, a.zs, V, es, false) && fits(a.x, a.xs, V, es, false) &&
           fits(a.out, a.os, V, es, false) && fits(a.next, a.ns, V, es, false) &&
           fits(a.y, a.os, V, es, false) && fits(a.dout, a.dos, V, es, false) &&
           fits(a.dnext, a.dns, V, es, false) && fits(a.dx, a.dxs, V, es, false) &&
           fits(a.dz, a.dzs, V, es, false);
  };
  if (narrow || !all(p.V)) p.V = 1;
  const int vecs = a.D / p.V, each = a.m / p.V;
  const bool lanes = each <= 32 && (each & (each - 1)) == 0;
  p.mode = lanes ? kLanes : a.H == 1 ? kWhole : kStaged;
  const int64_t rows = a.B * a.T;
  int resident = 0, least = 0;
  const int counts = p.V > 1 ? COUNTS : 4;
  for (int i = 0; i < counts; ++i) {
    const Width& w = p.V > 1 ? widths[i] : kNarrow[i];
    const int K = w.K;
    int nt = (vecs + K - 1) / K;
    if (nt <= 16 && p.mode != kStaged) {
      int up = 1;
      while (up < nt) up *= 2;
      nt = up;
    } else {
      nt = (nt + 31) / 32 * 32;
    }
    if (nt > w.threads) continue;
    // a head's lanes lie in one row, side by side
    if (p.mode == kLanes && nt < each) continue;
    const int cost = (nt < 32 ? 1 : nt / 32) * (24 + K * p.V);
    if (p.K && (cost >= least || (rows * nt + 31) / 32 < enough ||
                (p.V > 1 ? K > prefer && (nt > 32 || K > 4)
                         : K > prefer + 2 && (nt > 32 || K > 8))))
      continue;
    p.K = K, p.nt = nt, least = cost, resident = w.resident;
  }
  p.rows = (p.V == 1 ? kNarrowThreads : kRowThreads) / p.nt;
  if (p.rows < 1) p.rows = 1;
  if (p.rows > 8 && p.nt >= 32) p.rows = 8;
  p.params = (size_t)(a.next_weight ? 2 : 1) * a.D * 4;
  p.params = (p.params + 15) / 16 * 16;
  p.staged = p.params;
  if (p.mode == kStaged) {
    const size_t one = (size_t)(vecs + a.H) * 8;
    while (p.rows > 1 && p.rows * one > 40 * 1024) p.rows /= 2;
    p.staged += (p.rows * one + 15) / 16 * 16;
  }
  // blocks that fit an SM with a row each at least; what is left of
  // shared memory takes more rows ahead
  const size_t row = (size_t)p.nt * p.rows * p.K * inputs * (p.V * es);
  const bool ahead = p.V > 1;
  int per = resident / (p.nt * p.rows);
  if (per < 1) per = 1;
  if (per > 4) per = 4;  // a block takes all sixteen barriers
  while (per > 1 && p.staged + (ahead ? row : 0) > shared_for(per)) --per;
  if (ahead && shared_for(per) > p.staged) {
    const size_t fit = (shared_for(per) - p.staged) / (row ? row : 1);
    p.ring = fit > 4 ? 4 : (int)fit;
  }
  // no room for a single row: single elements, whose row ahead is in registers (2048 fp32 rows
  // of 8192 channels with all inputs: gradient 297 us)
  if (ahead && p.ring == 0) return plan_norm(a, widths, prefer, enough, inputs, true);
  p.shared = p.staged + p.ring * row;
  p.blocks = 152 * per;
  return p;
}

template <typename F>
cudaError_t start_norm(F kernel, const NormArgs& a, const NormPlan& p, unsigned grid,
                       std::atomic<uint64_t>* allowed, cudaStream_t stream) {
  // asked for with the most that any shape needs
  if (p.shared > 40 * 1024) {
    cudaError_t e = allow_shared(kernel, (int)shared_for(1), allowed);
    if (e != cudaSuccess) return e;
  }
  kernel<<<grid, dim3(p.nt, p.rows), p.shared, stream>>>(a, p.ring, (int)p.params,
                                                                (int)p.staged);
  return cudaGetLastError();
}

}  // namespace
}  // namespace falcon
