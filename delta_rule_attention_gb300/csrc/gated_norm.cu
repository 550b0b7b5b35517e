// The norm behind a block, its gate, scale and residual, and the norm before the next
// block, in one pass over the rows; and its gradient.  Bound by the rows' traffic.
//
//   y = x + scale act(z) n w,  n = h r,  r = 1 / sqrt(mean_head h^2 + eps)
//   u = y s w',                s = 1 / sqrt(mean y^2 + eps)
// A row stays in registers between its loads and its stores: a thread holds K vectors of
// V neighbouring channels, all loads under way before the first sum.  The gradient, with
// d the gradient of y:
//   d  = dy + s (e - y s^2 mean(e y)),  e = du w'
//   dz = d scale w n act'(z);   f = d act(z) scale w
//   dh = r (f - h r^2 mean_head(f h))
//   dw = scale sum(d act(z) n),  dscale = w sum(d act(z) n),  dw' = sum(du y s)
// whose sums over rows a thread keeps for its channels over the rows of its block; a
// second kernel adds the blocks' sums in a fixed order.
#include "linear.cuh"

namespace falcon {
namespace {

// How a head's sum is formed.
enum { kWhole = 0,   // one head: the threads of a row
       kLanes = 1,   // m / V threads, a power of two up to 32, side by side in a warp
       kStaged = 2   // any: products in shared memory, a warp a head
};

template <typename E, int V>
__device__ __forceinline__ FloatV<V> zeros() {
  FloatV<V> r;
#pragma unroll
  for (int i = 0; i < V; ++i) r.v[i] = 0.f;
  return r;
}

// V fp32 parameters of neighbouring channels (1 where there are none).
template <int V>
__device__ __forceinline__ FloatV<V> params(const float* p, int c, bool live, bool vec) {
  FloatV<V> r;
#pragma unroll
  for (int i = 0; i < V; ++i) r.v[i] = 1.f;
  if (!p || !live) return r;
  if (vec) {
#pragma unroll
    for (int i = 0; i < V; i += V < 4 ? V : 4) {
      const FloatV<V < 4 ? V : 4> q = load_vec<float, V < 4 ? V : 4>(p + c + i);
#pragma unroll
      for (int j = 0; j < (V < 4 ? V : 4); ++j) r.v[i + j] = q.v[j];
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) r.v[i] = p[c + i];
  }
  return r;
}

// Sums of two values over the nt threads of a row (a power of two up to 32, or whole
// warps); `red` holds 32 pairs a row.
__device__ __forceinline__ float2 row_sum(float2 x, int nt, float2* red) {
  for (int o = nt < 32 ? nt / 2 : 16; o > 0; o >>= 1) {
    x.x += __shfl_xor_sync(0xffffffffu, x.x, o);
    x.y += __shfl_xor_sync(0xffffffffu, x.y, o);
  }
  if (nt <= 32) return x;
  __syncthreads();  // the last sum has been read
  if (threadIdx.x % 32 == 0) red[threadIdx.x / 32] = x;
  __syncthreads();
  float2 s = make_float2(0.f, 0.f);
  for (int w = 0; w < nt / 32; ++w) s.x += red[w].x, s.y += red[w].y;
  return s;
}

struct Gate {
  float act, slope;
};
__device__ __forceinline__ Gate gate_of(float z, int gate) {
  if (gate == FALCON_ACT_IDENTITY) return {z, 1.f};
  const float p = sigmoid(z);
  if (gate == FALCON_ACT_SIGMOID) return {p, p * (1.f - p)};
  return {z * p, p * fmaf(z, 1.f - p, 1.f)};
}

struct RowAt {
  int64_t b, t;
  bool in, held;  // inside the problem; a token of its row
};
__device__ __forceinline__ RowAt row_at(const NormArgs& a, int64_t row) {
  RowAt r;
  r.in = row < a.B * a.T;
  if (!r.in) row = 0;
  r.b = row / a.T, r.t = row - r.b * a.T;
  r.held = r.in && r.t < row_length(a.lengths, r.b, a.T);
  return r;
}

// Channel and head of vector k of a thread.
struct Place {
  int c, head;
  bool live;
};
template <int V, int MODE>
__device__ __forceinline__ Place place_of(const NormArgs& a, int k) {
  Place p;
  p.c = (k * (int)blockDim.x + (int)threadIdx.x) * V;
  p.live = p.c < a.D;
  p.head = MODE == kWhole || !p.live ? 0 : p.c / a.m;
  return p;
}

template <typename E, int V>
__device__ __forceinline__ FloatV<V> row_vec(const void* p, int64_t at, bool live) {
  return live ? load_vec<E, V>(static_cast<const E*>(p) + at) : zeros<E, V>();
}

// Sums over each vector's head of one or two values a vector, in place.
template <int K, int MODE>
__device__ __forceinline__ void head_sums(const NormArgs& a, const Place (&at)[K],
                                          float2 (&x)[K], int V, float2* red) {
  if constexpr (MODE == kWhole) {
    float2 s = make_float2(0.f, 0.f);
#pragma unroll
    for (int k = 0; k < K; ++k) s.x += x[k].x, s.y += x[k].y;
    s = row_sum(s, blockDim.x, red);
#pragma unroll
    for (int k = 0; k < K; ++k) x[k] = s;
  } else if constexpr (MODE == kLanes) {
    const int lanes = a.m / V;
#pragma unroll
    for (int k = 0; k < K; ++k)
      for (int o = lanes / 2; o > 0; o >>= 1) {
        x[k].x += __shfl_xor_sync(0xffffffffu, x[k].x, o);
        x[k].y += __shfl_xor_sync(0xffffffffu, x[k].y, o);
      }
  } else {
    // a vector lies inside one head (V divides m)
    extern __shared__ float2 staged[];
    const int vecs = a.D / V, each = a.m / V;
    float2* mine = staged + (int)threadIdx.y * (vecs + a.H);
    float2* sums = mine + vecs;
    __syncthreads();
#pragma unroll
    for (int k = 0; k < K; ++k)
      if (at[k].live) mine[at[k].c / V] = x[k];
    __syncthreads();
    const int warps = blockDim.x / 32, lane = threadIdx.x % 32;
    for (int h = threadIdx.x / 32; h < a.H; h += warps) {
      float2 s = make_float2(0.f, 0.f);
      for (int i = lane; i < each; i += 32) {
        const float2 q = mine[h * each + i];
        s.x += q.x, s.y += q.y;
      }
      s.x = warp_sum(s.x), s.y = warp_sum(s.y);
      if (lane == 0) sums[h] = s;
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < K; ++k) x[k] = sums[at[k].head];
  }
}

template <typename E, int V, int K, int MODE>
__global__ void __launch_bounds__(K > 4 ? 1024 : 512)
    norm_fwd_kernel(const __grid_constant__ NormArgs a, bool vec_p) {
  __shared__ float2 reds[8][32];
  float2* red = reds[threadIdx.y];
  const RowAt r = row_at(a, (int64_t)blockIdx.x * blockDim.y + threadIdx.y);
  Place at[K];
  FloatV<V> h[K], z[K], x[K];
#pragma unroll
  for (int k = 0; k < K; ++k) {
    at[k] = place_of<V, MODE>(a, k);
    const bool on = at[k].live && r.held;
    h[k] = row_vec<E, V>(a.h, r.b * a.hs.batch + r.t * a.hs.time + at[k].head * a.hs.head +
                                  (at[k].c - at[k].head * (MODE == kWhole ? 0 : a.m)),
                         on && a.h);
    z[k] = row_vec<E, V>(a.z, r.b * a.zs.batch + r.t * a.zs.time + at[k].c, on && a.z);
    x[k] = row_vec<E, V>(a.x, r.b * a.xs.batch + r.t * a.xs.time + at[k].c, on && a.x);
  }
  if (a.h) {
    float2 ss[K];
#pragma unroll
    for (int k = 0; k < K; ++k) {
      ss[k] = make_float2(0.f, 0.f);
#pragma unroll
      for (int i = 0; i < V; ++i) ss[k].x = fmaf(h[k].v[i], h[k].v[i], ss[k].x);
    }
    head_sums<K, MODE>(a, at, ss, V, red);
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const float rn = rsqrtf(ss[k].x / (float)a.m + a.eps);
      const FloatV<V> w = params<V>(a.weight, at[k].c, at[k].live, vec_p);
      const FloatV<V> sc = params<V>(a.scale, at[k].c, at[k].live, vec_p);
      const bool on = at[k].live && r.held;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        float y = h[k].v[i] * rn * w.v[i];
        if (a.z) y *= gate_of(z[k].v[i], a.gate).act;
        x[k].v[i] = on ? fmaf(y, sc.v[i], x[k].v[i]) : 0.f;
      }
      if (at[k].live && r.in)
        store_vec<E, V>(static_cast<E*>(a.out) + r.b * a.os.batch + r.t * a.os.time + at[k].c,
                        x[k]);
    }
  }
  if (a.next) {
    float2 s = make_float2(0.f, 0.f);
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int i = 0; i < V; ++i) s.x = fmaf(x[k].v[i], x[k].v[i], s.x);
    s = row_sum(s, blockDim.x, red);
    const float rn = rsqrtf(s.x / (float)a.D + a.eps);
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const FloatV<V> w = params<V>(a.next_weight, at[k].c, at[k].live, vec_p);
      FloatV<V> u;
#pragma unroll
      for (int i = 0; i < V; ++i) u.v[i] = x[k].v[i] * rn * w.v[i];
      if (at[k].live && r.in)
        store_vec<E, V>(static_cast<E*>(a.next) + r.b * a.ns.batch + r.t * a.ns.time + at[k].c,
                        u);
    }
  }
}

template <typename E, int V, int K, int MODE>
__global__ void __launch_bounds__(K > 4 ? 1024 : 512)
    norm_bwd_kernel(const __grid_constant__ NormArgs a, bool vec_p) {
  __shared__ float2 reds[8][32];
  float2* red = reds[threadIdx.y];
  const int64_t rows = a.B * a.T, step = (int64_t)gridDim.x * blockDim.y;
  FloatV<V> each[K], nextw[K];  // sums for dweight and dscale, and for dnext_weight
#pragma unroll
  for (int k = 0; k < K; ++k) each[k] = zeros<E, V>(), nextw[k] = zeros<E, V>();
  // every thread takes part in every turn's barriers
  for (int64_t r0 = (int64_t)blockIdx.x * blockDim.y; r0 < rows; r0 += step) {
    const RowAt r = row_at(a, r0 + threadIdx.y);
    Place at[K];
    FloatV<V> h[K], z[K], d[K], y[K], e[K];
#pragma unroll
    for (int k = 0; k < K; ++k) {
      at[k] = place_of<V, MODE>(a, k);
      const bool on = at[k].live && r.held;
      h[k] = row_vec<E, V>(a.h, r.b * a.hs.batch + r.t * a.hs.time + at[k].head * a.hs.head +
                                    (at[k].c - at[k].head * (MODE == kWhole ? 0 : a.m)),
                           on && a.h);
      z[k] = row_vec<E, V>(a.z, r.b * a.zs.batch + r.t * a.zs.time + at[k].c, on && a.z);
      d[k] = row_vec<E, V>(a.dout, r.b * a.dos.batch + r.t * a.dos.time + at[k].c,
                           on && a.dout);
      y[k] = row_vec<E, V>(a.y, r.b * a.os.batch + r.t * a.os.time + at[k].c,
                           on && a.next_weight);
      e[k] = row_vec<E, V>(a.dnext, r.b * a.dns.batch + r.t * a.dns.time + at[k].c,
                           on && a.next_weight);
    }
    if (a.next_weight) {
      float2 s = make_float2(0.f, 0.f);
      FloatV<V> w[K];
#pragma unroll
      for (int k = 0; k < K; ++k) {
        w[k] = params<V>(a.next_weight, at[k].c, at[k].live, vec_p);
#pragma unroll
        for (int i = 0; i < V; ++i) {
          s.x = fmaf(y[k].v[i], y[k].v[i], s.x);
          s.y = fmaf(e[k].v[i] * w[k].v[i], y[k].v[i], s.y);
        }
      }
      s = row_sum(s, blockDim.x, red);
      const float rn = rsqrtf(s.x / (float)a.D + a.eps);
      const float back = rn * rn * s.y / (float)a.D;
#pragma unroll
      for (int k = 0; k < K; ++k)
#pragma unroll
        for (int i = 0; i < V; ++i) {
          nextw[k].v[i] = fmaf(e[k].v[i] * rn, y[k].v[i], nextw[k].v[i]);
          d[k].v[i] = fmaf(rn, fmaf(-back, y[k].v[i], e[k].v[i] * w[k].v[i]), d[k].v[i]);
        }
    }
    if (a.dx) {
#pragma unroll
      for (int k = 0; k < K; ++k)
        if (at[k].live && r.in)
          store_vec<E, V>(static_cast<E*>(a.dx) + r.b * a.dxs.batch + r.t * a.dxs.time + at[k].c,
                          d[k]);
    }
    if (a.h) {
      float2 s[K];
      FloatV<V> f[K];
#pragma unroll
      for (int k = 0; k < K; ++k) {
        const FloatV<V> w = params<V>(a.weight, at[k].c, at[k].live, vec_p);
        const FloatV<V> sc = params<V>(a.scale, at[k].c, at[k].live, vec_p);
        s[k] = make_float2(0.f, 0.f);
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const Gate g = a.z ? gate_of(z[k].v[i], a.gate) : Gate{1.f, 0.f};
          const float dg = d[k].v[i] * w.v[i] * sc.v[i];
          z[k].v[i] = dg * g.slope;        // times n: dz
          d[k].v[i] *= g.act;              // times n: a row's part of the sums
          f[k].v[i] = dg * g.act;
          s[k].x = fmaf(h[k].v[i], h[k].v[i], s[k].x);
          s[k].y = fmaf(f[k].v[i], h[k].v[i], s[k].y);
        }
      }
      head_sums<K, MODE>(a, at, s, V, red);
#pragma unroll
      for (int k = 0; k < K; ++k) {
        const float rn = rsqrtf(s[k].x / (float)a.m + a.eps);
        const float back = rn * rn * s[k].y / (float)a.m;
        FloatV<V> dh;
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const float n = h[k].v[i] * rn;
          each[k].v[i] = fmaf(d[k].v[i], n, each[k].v[i]);
          z[k].v[i] *= n;
          dh.v[i] = rn * fmaf(-back, h[k].v[i], f[k].v[i]);
        }
        if (at[k].live && r.in) {
          store_vec<E, V>(static_cast<E*>(a.dh) + r.b * a.dhs.batch + r.t * a.dhs.time +
                              at[k].head * a.dhs.head +
                              (at[k].c - at[k].head * (MODE == kWhole ? 0 : a.m)),
                          dh);
          if (a.z)
            store_vec<E, V>(static_cast<E*>(a.dz) + r.b * a.dzs.batch + r.t * a.dzs.time +
                                at[k].c,
                            z[k]);
        }
      }
    }
  }
  float* ws = a.ws + ((int64_t)blockIdx.x * blockDim.y + threadIdx.y) * 2 * a.D;
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const int c = (k * (int)blockDim.x + (int)threadIdx.x) * V;
    if (c < a.D) {
#pragma unroll
      for (int i = 0; i < V; ++i) ws[c + i] = each[k].v[i], ws[a.D + c + i] = nextw[k].v[i];
    }
  }
}

// Adds the blocks' sums: 32 channels a block, 8 threads a channel, in a fixed order.
__global__ void __launch_bounds__(256) norm_params_kernel(const __grid_constant__ NormArgs a) {
  __shared__ float red[2][8][33];
  const int c = blockIdx.x * 32 + threadIdx.x;
  float s0 = 0.f, s1 = 0.f;
  if (c < a.D)
    for (int p = threadIdx.y; p < a.parts; p += 8) {
      s0 += a.ws[(int64_t)p * 2 * a.D + c];
      s1 += a.ws[(int64_t)p * 2 * a.D + a.D + c];
    }
  red[0][threadIdx.y][threadIdx.x] = s0;
  red[1][threadIdx.y][threadIdx.x] = s1;
  __syncthreads();
  if (threadIdx.y == 0 && c < a.D) {
    for (int p = 1; p < 8; ++p) s0 += red[0][p][threadIdx.x], s1 += red[1][p][threadIdx.x];
    if (a.dweight) a.dweight[c] = a.scale ? s0 * a.scale[c] : s0;
    if (a.dscale) a.dscale[c] = a.weight ? s0 * a.weight[c] : s0;
    if (a.dnext_weight) a.dnext_weight[c] = s1;
  }
}

// Launch shape: V channels a vector, K vectors a thread, nt threads a row, `rows` rows a
// block.
struct NormPlan {
  int V, K, nt, rows, mode;
  size_t shared;
  bool vec_p;
};

bool fits(const void* p, const falcon_strides& s, int V, int esize, bool head) {
  if (!p) return true;
  return reinterpret_cast<uintptr_t>(p) % (uintptr_t)(V * esize) == 0 && s.batch % V == 0 &&
         s.time % V == 0 && (!head || s.head % V == 0);
}

constexpr int kRowThreads = 256;  // threads a block aims at

NormPlan plan_norm(const NormArgs& a, bool narrow = false) {
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
  p.K = vecs <= 512 ? 1 : vecs <= 1024 ? 2 : vecs <= 2048 ? 4 : 8;
  p.nt = (vecs + p.K - 1) / p.K;
  const bool lanes = each <= 32 && (each & (each - 1)) == 0;
  p.mode = lanes ? kLanes : a.H == 1 ? kWhole : kStaged;
  if (p.nt <= 16 && p.mode != kStaged) {
    int up = 1;
    while (up < p.nt) up *= 2;
    p.nt = up;
  } else {
    p.nt = (p.nt + 31) / 32 * 32;
  }
  p.rows = kRowThreads / p.nt;
  if (p.rows < 1) p.rows = 1;
  if (p.rows > 8 && p.nt > 32) p.rows = 8;
  if (p.mode == kStaged) {
    const size_t one = (size_t)(vecs + a.H) * 8;
    while (p.rows > 1 && p.rows * one > 40 * 1024) p.rows /= 2;
    p.shared = p.rows * one;
  }
  auto aligned = [](const float* q) { return reinterpret_cast<uintptr_t>(q) % 16 == 0; };
  p.vec_p = aligned(a.weight) && aligned(a.scale) && aligned(a.next_weight);
  return p;
}

template <typename E, int V, int K, int MODE>
cudaError_t start(const NormArgs& a, const NormPlan& p, bool back, unsigned grid,
                  cudaStream_t stream) {
  static std::atomic<uint64_t> allowed[2];
  const dim3 block(p.nt, p.rows);
  auto kernel = back ? norm_bwd_kernel<E, V, K, MODE> : norm_fwd_kernel<E, V, K, MODE>;
  // asked for with the most that any shape needs
  if (MODE == kStaged && p.shared > 40 * 1024) {
    cudaError_t e = allow_shared(kernel, 144 * 1024, &allowed[back]);
    if (e != cudaSuccess) return e;
  }
  kernel<<<grid, block, p.shared, stream>>>(a, p.vec_p);
  return cudaGetLastError();
}

template <typename E, int V, int K>
cudaError_t start_mode(const NormArgs& a, const NormPlan& p, bool back, unsigned grid,
                       cudaStream_t stream) {
  if (p.mode == kWhole) return start<E, V, K, kWhole>(a, p, back, grid, stream);
  if (p.mode == kLanes) return start<E, V, K, kLanes>(a, p, back, grid, stream);
  return start<E, V, K, kStaged>(a, p, back, grid, stream);
}

template <typename E, int V>
cudaError_t start_count(const NormArgs& a, const NormPlan& p, bool back, unsigned grid,
                        cudaStream_t stream) {
  if (p.K == 1) return start_mode<E, V, 1>(a, p, back, grid, stream);
  if (p.K == 2) return start_mode<E, V, 2>(a, p, back, grid, stream);
  if (p.K == 4) return start_mode<E, V, 4>(a, p, back, grid, stream);
  return start_mode<E, V, 8>(a, p, back, grid, stream);
}

cudaError_t start_norm(const NormArgs& a, const NormPlan& p, bool back, unsigned grid,
                       cudaStream_t stream) {
  if (a.dtype == FALCON_BF16)
    return p.V == 8 ? start_count<__nv_bfloat16, 8>(a, p, back, grid, stream)
                    : start_count<__nv_bfloat16, 1>(a, p, back, grid, stream);
  return p.V == 4 ? start_count<float, 4>(a, p, back, grid, stream)
                  : start_count<float, 1>(a, p, back, grid, stream);
}

constexpr int kBwdBlocks = 608;  // four blocks for each of 152 SMs

unsigned bwd_blocks(const NormArgs& a, const NormPlan& p) {
  const int64_t blocks = (a.B * a.T + p.rows - 1) / p.rows;
  return (unsigned)(blocks < kBwdBlocks ? blocks : kBwdBlocks);
}

}  // namespace

// Room for either width of access: which one a call takes goes by its pointers.
size_t norm_bwd_workspace_bytes(const falcon_norm_shape& s) {
  NormArgs a = {};
  a.B = s.B, a.T = s.T, a.H = (int)s.H, a.m = s.m, a.D = (int)(s.H * s.m), a.dtype = s.dtype;
  const NormPlan wide = plan_norm(a, false), narrow = plan_norm(a, true);
  const int64_t x = (int64_t)bwd_blocks(a, wide) * wide.rows,
                y = (int64_t)bwd_blocks(a, narrow) * narrow.rows;
  return (size_t)(x > y ? x : y) * 2 * a.D * 4;
}

cudaError_t launch_norm_fwd(const NormArgs& a, cudaStream_t stream) {
  const NormPlan p = plan_norm(a);
  const int64_t rows = a.B * a.T;
  return start_norm(a, p, false, (unsigned)((rows + p.rows - 1) / p.rows), stream);
}

cudaError_t launch_norm_bwd(const NormArgs& args, cudaStream_t stream) {
  NormArgs a = args;
  const NormPlan p = plan_norm(a);
  const unsigned grid = bwd_blocks(a, p);
  a.parts = (int)grid * p.rows;
  if (grid > 0) {
    const cudaError_t e = start_norm(a, p, true, grid, stream);
    if (e != cudaSuccess) return e;
  }
  if (a.dweight || a.dscale || a.dnext_weight)
    norm_params_kernel<<<(unsigned)((a.D + 31) / 32), dim3(32, 8), 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace falcon
