// Short causal convolution: forward, gradient, and one token of many sequences.
//
//   p_t = bias + sum_{j<W} w_j x_{t-W+1+j},  y_t = act(p_t)
//   dp_t = dy_t act'(p_t),  dx_t = sum_j w_j dp_{t+W-1-j},
//   dw_j = sum_t dp_t x_{t-W+1+j},  dbias = sum_t dp_t
//
// Bound by memory traffic.  A thread owns V neighbouring channels (one access of
// up to 16 bytes) and a run of tokens; all rows of the run, with the W - 1 before
// it (and after it, for the gradient), are loaded before the first is used, so
// that the traffic does not wait for the arithmetic.  A run's edge rows are read
// twice, the second time from cache.
//
// B8 H12 T2048 m64 W4 bf16, silu, from strided heads: 13.3 us in a graph of calls (3.8 TB/s
// of the 50 MB it must move; 16.2 us from cold caches, issue slots 60% busy).  The
// gradient for B8 T2048 C2048: 53 us with its sums (3.8 TB/s of 202 MB; 50 and 6.6 from
// cold caches): bound by the latency of its loads at 14 warps an SM.
// Eight tokens a forward run and four channels a thread.  Runs of 16 take 3% less where
// there are rows enough (B32: 48.9 us a call, 50.8 with 8) but halve the threads of a
// small call (B1: 19 to 22 us, 17 to 18 with 8); runs of 4 took 25% more, and eight
// channels a thread 14% more.

#include <type_traits>

#include "ssm.cuh"

namespace falcon {
namespace {

constexpr int kThreads = 128;

// a / b; a 64-bit division costs many times a 32-bit one.
__device__ __forceinline__ int64_t quotient(int64_t a, int64_t b) {
  if (((uint64_t)(a | b) >> 32) == 0) return (uint32_t)a / (uint32_t)b;
  return a / b;
}

// Offset of channel c of row (b, t): channels are grouped in heads of m.
__device__ __forceinline__ int64_t row_offset(const falcon_strides& s, int64_t b, int64_t c,
                                              int m) {
  const int64_t h = quotient(c, m);
  return b * s.batch + h * s.head + (c - h * m);
}

template <int V>
__device__ __forceinline__ FloatV<V> zeros() {
  FloatV<V> r;
#pragma unroll
  for (int i = 0; i < V; ++i) r.v[i] = 0.f;
  return r;
}

template <int V>
__device__ __forceinline__ FloatV<V> ones() {
  FloatV<V> r;
#pragma unroll
  for (int i = 0; i < V; ++i) r.v[i] = 1.f;
  return r;
}
template <int V>
__device__ __forceinline__ FloatV<V> sigmoid_vec(const FloatV<V>& x) {
  FloatV<V> r;
#pragma unroll
  for (int i = 0; i < V; ++i) r.v[i] = sigmoid(x.v[i]);
  return r;
}

// Input at time t of row b, which may be a carried one (t < 0) or none (t >= n).
template <typename E, int V, int W>
__device__ __forceinline__ FloatV<V> input_at(const E* xrow, int64_t tstride, const E* state,
                                              int64_t b, int64_t C, int64_t c, int64_t t,
                                              int64_t n) {
  if (t >= n) return zeros<V>();
  if (t >= 0) return load_vec<E, V>(xrow + t * tstride);
  if (state) return load_vec<E, V>(state + (b * (W - 1) + (t + W - 1)) * C + c);
  return zeros<V>();
}

template <int V, int W>
struct Filter {
  FloatV<V> w[W];
  FloatV<V> bias;
};

// vec: the weights lie on a 16-byte boundary, and so does every V-th filter where
// V * W is a multiple of four.
template <int V, int W>
__device__ __forceinline__ Filter<V, W> load_filter(const float* weight, const float* bias,
                                                    int64_t c, bool vec) {
  Filter<V, W> f;
  if (vec && V * W % 4 == 0) {
    float4 v[V * W / 4 > 0 ? V * W / 4 : 1];
#pragma unroll
    for (int i = 0; i < V * W / 4; ++i) v[i] = reinterpret_cast<const float4*>(weight + c * W)[i];
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
      for (int j = 0; j < W; ++j) {
        const float4 q = v[(i * W + j) / 4];
        const int k = (i * W + j) % 4;
        f.w[j].v[i] = k == 0 ? q.x : k == 1 ? q.y : k == 2 ? q.z : q.w;
      }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
      for (int j = 0; j < W; ++j) f.w[j].v[i] = weight[(c + i) * W + j];
  }
#pragma unroll
  for (int i = 0; i < V; ++i) f.bias.v[i] = bias ? bias[c + i] : 0.f;
  return f;
}

// V elements as they lie in memory.
template <typename E, int V>
struct alignas(V * sizeof(E)) Row {
  E e[V];
};
template <typename E, int V>
__device__ __forceinline__ FloatV<V> open_row(const Row<E, V>& r) {
  return load_vec<E, V>(r.e);
}

constexpr int kFwdRun = 8;

// One thread for V channels and a run; a row's last run + 1 writes state_out.
template <typename E, int V, int W, bool SILU>
__global__ void __launch_bounds__(kThreads)
    conv_fwd_kernel(const __grid_constant__ ConvArgs a, int64_t nruns) {
  typedef Row<E, V> R;
  const int64_t nvec = a.C / V, id = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  if (id >= nvec * a.B * (nruns + 1)) return;
  const int64_t job = quotient(id, nvec), c = (id - job * nvec) * V;
  const int64_t b = quotient(job, nruns + 1), r = job - b * (nruns + 1);
  const int64_t n = row_length(a.lengths, b, a.T);
  const E* x = static_cast<const E*>(a.x) + row_offset(a.xs, b, c, a.m);
  const E* state = static_cast<const E*>(a.state);
  if (r == nruns) {  // the row's last W - 1 inputs
    if (!a.state_out) return;
#pragma unroll
    for (int j = 0; j < W - 1; ++j)
      store_vec<E, V>(static_cast<E*>(a.state_out) + (b * (W - 1) + j) * a.C + c,
                      input_at<E, V, W>(x, a.xs.time, state, b, a.C, c, n - (W - 1) + j, n));
    return;
  }
  const int64_t t0 = r * kFwdRun;
  E* y = static_cast<E*>(a.y) + row_offset(a.ys, b, c, a.m);
  if (t0 >= n) {
    for (int64_t t = t0; t < t0 + kFwdRun && t < a.T; ++t)
      store_vec<E, V>(y + t * a.ys.time, zeros<V>());
    return;
  }
  R rows[kFwdRun + W - 1];
  const bool whole = t0 > 0 && t0 + kFwdRun <= n;  // no carried input, no missing token
  const E* px = x + (t0 - (W - 1)) * a.xs.time;
  if (whole) {
#pragma unroll
    for (int k = 0; k < kFwdRun + W - 1; ++k) {
      rows[k] = *reinterpret_cast<const R*>(px);
      px += a.xs.time;
    }
  } else {
#pragma unroll
    for (int k = 0; k < kFwdRun + W - 1; ++k) {
      const int64_t t = t0 + k - (W - 1);
      rows[k] = R();
      if (t >= 0) {
        if (t < n) rows[k] = *reinterpret_cast<const R*>(px);
      } else if (state) {
        rows[k] = *reinterpret_cast<const R*>(state + (b * (W - 1) + (t + W - 1)) * a.C + c);
      }
      px += a.xs.time;
    }
  }
  const Filter<V, W> f = load_filter<V, W>(a.weight, a.bias, c, a.vec_w);
  FloatV<V> win[W];
#pragma unroll
  for (int j = 0; j < W - 1; ++j) win[j] = open_row<E, V>(rows[j]);
  E* py = y + t0 * a.ys.time;
#pragma unroll
  for (int k = 0; k < kFwdRun; ++k) {
    win[W - 1] = open_row<E, V>(rows[k + W - 1]);
    FloatV<V> o = f.bias;
#pragma unroll
    for (int j = 0; j < W; ++j) o = fma_vec(f.w[j], win[j], o);
    if (SILU) o = mul_vec(o, sigmoid_vec(o));
    if (whole)
      store_vec<E, V>(py, o);
    else if (t0 + k < a.T)
      store_vec<E, V>(py, t0 + k < n ? o : zeros<V>());
    py += a.ys.time;
#pragma unroll
    for (int j = 0; j < W - 1; ++j) win[j] = win[j + 1];
  }
}

constexpr int kBwdBlock = 8;  // tokens whose rows are under way together

// Gradient: a thread walks a run of `run` tokens and the W - 1 after it, whose dp
// it recomputes from x; each dp_t adds w_j dp_t to dx_{t-W+1+j}.  A thread takes
// every `parts`-th run of its channels with its sums of dw and dbias in registers and
// writes them once; conv_sum_kernel adds the parts in their order.
template <typename E, int V, int W, bool SILU>
__global__ void __launch_bounds__(kThreads)
    conv_bwd_kernel(const __grid_constant__ ConvArgs a, int run, int64_t nruns, int parts) {
  typedef Row<E, V> R;
  const int64_t nvec = a.C / V, id = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  if (id >= nvec * parts) return;
  const int64_t part = quotient(id, nvec), c = (id - part * nvec) * V;
  const Filter<V, W> f = load_filter<V, W>(a.weight, a.bias, c, a.vec_w);
  FloatV<V> dw[W], db = zeros<V>();
#pragma unroll
  for (int j = 0; j < W; ++j) dw[j] = zeros<V>();
  for (int64_t job = part; job < a.B * nruns; job += parts) {
    const int64_t b = quotient(job, nruns), r = job - b * nruns;
    const int64_t n = row_length(a.lengths, b, a.T);
    const E* x = static_cast<const E*>(a.x) + row_offset(a.xs, b, c, a.m);
    const E* dy = static_cast<const E*>(a.dy) + row_offset(a.dys, b, c, a.m);
    E* dx = static_cast<E*>(a.dx) + row_offset(a.dxs, b, c, a.m);
    const E* state = static_cast<const E*>(a.state);
    const E* dso = static_cast<const E*>(a.dstate_out);
    const int64_t t0 = r * run, t1 = t0 + run < a.T ? t0 + run : a.T, te = t1 + W - 1;
    R xr[kBwdBlock], gr[kBwdBlock];
    // pointers walk with the tokens: a product for every row would fill the registers
    const E *px = x + t0 * a.xs.time, *pg = dy + t0 * a.dys.time;
    E* po = dx + (t0 - (W - 1)) * a.dxs.time;
    const int readable = (int)((n < te ? n : te) - t0), total = (int)(te - t0),
              own = (int)(t1 - t0);
    auto fetch = [&](int k0) {
      if (k0 + kBwdBlock <= readable) {
#pragma unroll
        for (int k = 0; k < kBwdBlock; ++k) {
          xr[k] = *reinterpret_cast<const R*>(px);
          gr[k] = *reinterpret_cast<const R*>(pg);
          px += a.xs.time;
          pg += a.dys.time;
        }
      } else {
#pragma unroll
        for (int k = 0; k < kBwdBlock; ++k) {
          xr[k] = gr[k] = R();
          if (k0 + k < readable) {
            xr[k] = *reinterpret_cast<const R*>(px);
            gr[k] = *reinterpret_cast<const R*>(pg);
          }
          px += a.xs.time;
          pg += a.dys.time;
        }
      }
    };
    fetch(0);
    // acc[j] gathers the gradient of input t - W + 1 + j
    FloatV<V> win[W], acc[W];
#pragma unroll
    for (int j = 0; j < W - 1; ++j) {
      win[j] = input_at<E, V, W>(x, a.xs.time, state, b, a.C, c, t0 - (W - 1) + j, n);
      acc[j] = zeros<V>();
    }
    // places in state_out begin at token n - (W - 1); the row's last inputs only
    const int tail = dso && n - (W - 1) < te ? (int)(n - t0) - (W - 1) : total;
    // one block of tokens; WHOLE: all are the run's own tokens, and all inputs that
    // they complete are the run's own and not among the row's last
    auto block = [&](int k0, const R(&xc)[kBwdBlock], const R(&gc)[kBwdBlock], auto whole) {
      constexpr bool WHOLE = decltype(whole)::value;
#pragma unroll
      for (int k = 0; k < kBwdBlock; ++k) {
        const int kt = k0 + k;  // token, counted from the run's first
        acc[W - 1] = zeros<V>();
        win[W - 1] = open_row<E, V>(xc[k]);
        FloatV<V> d = open_row<E, V>(gc[k]);  // zero where there is no token
        if (SILU && (WHOLE || kt < readable)) {
          // silu'(p) = s (1 + p (1 - s)), s = sigmoid(p)
          FloatV<V> p = f.bias;
#pragma unroll
          for (int j = 0; j < W; ++j) p = fma_vec(f.w[j], win[j], p);
          const FloatV<V> s = sigmoid_vec(p), one = ones<V>();
          FloatV<V> m;
#pragma unroll
          for (int i = 0; i < V; ++i) m.v[i] = -s.v[i];
          d = mul_vec(d, mul_vec(s, fma_vec(p, add_vec(one, m), one)));
        }
#pragma unroll
        for (int j = 0; j < W; ++j) acc[j] = fma_vec(f.w[j], d, acc[j]);
        if (WHOLE || kt < own) {
          db = add_vec(db, d);
#pragma unroll
          for (int j = 0; j < W; ++j) dw[j] = fma_vec(d, win[j], dw[j]);
        }
        // input ks has met its last token: stored where it is this run's own; the
        // first run also stores the carried inputs' gradients
        const int ks = kt - (W - 1);
        if (WHOLE) {
          store_vec<E, V>(po, acc[0]);
        } else if (kt < total && (ks >= 0 || t0 == 0)) {
          FloatV<V> o = acc[0];
          if (ks >= tail && t0 + ks < n)
            o = add_vec(o, load_vec<E, V>(dso + (b * (W - 1) + (ks - tail)) * a.C + c));
          if (ks >= 0)
            store_vec<E, V>(po, o);
          else if (a.dstate)
            store_vec<E, V>(static_cast<E*>(a.dstate) + (b * (W - 1) + kt) * a.C + c, o);
        }
        po += a.dxs.time;
#pragma unroll
        for (int j = 0; j < W - 1; ++j) {
          win[j] = win[j + 1];
          acc[j] = acc[j + 1];
        }
      }
    };
    const int plain = (own < readable ? own : readable) < tail + W - 1
                          ? (own < readable ? own : readable) : tail + W - 1;
#pragma unroll 1
    for (int k0 = 0; k0 < total; k0 += kBwdBlock) {
      R xc[kBwdBlock], gc[kBwdBlock];
#pragma unroll
      for (int k = 0; k < kBwdBlock; ++k) xc[k] = xr[k], gc[k] = gr[k];
      if (k0 + kBwdBlock < total) fetch(k0 + kBwdBlock);
      if (k0 >= kBwdBlock && k0 + kBwdBlock <= plain)
        block(k0, xc, gc, std::true_type());
      else
        block(k0, xc, gc, std::false_type());
    }
  }
  float* ws = a.ws + part * (W + 1) * a.C;
#pragma unroll
  for (int j = 0; j <= W; ++j)
#pragma unroll
    for (int i = 0; i < V; ++i) ws[j * a.C + c + i] = j < W ? dw[j < W ? j : 0].v[i] : db.v[i];
}

// Sums of the parts: a warp's lanes hold neighbouring channels, a block's eight
// warps an eighth of the parts each.
__global__ void __launch_bounds__(256)
    conv_sum_kernel(const float* ws, int parts, int64_t C, int W, float* dweight, float* dbias) {
  __shared__ float sh[8][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, j = blockIdx.y;
  const int64_t c = (int64_t)blockIdx.x * 32 + lane;
  float s = 0.f;
  if (c < C) {
#pragma unroll 8
    for (int p = warp; p < parts; p += 8) s += ws[((int64_t)p * (W + 1) + j) * C + c];
  }
  sh[warp][lane] = s;
  __syncthreads();
  if (warp != 0 || c >= C) return;
  s = 0.f;
#pragma unroll
  for (int w = 0; w < 8; ++w) s += sh[w][lane];
  if (j < W)
    dweight[c * W + j] = s;
  else if (dbias)
    dbias[c] = s;
}

template <typename E, int V, int W, bool SILU>
__global__ void __launch_bounds__(kThreads)
    conv_step_kernel(const __grid_constant__ ConvStepArgs a) {
  const int64_t per_row = (a.C + V - 1) / V;
  const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  if (i >= a.N * per_row) return;
  const int64_t row = quotient(i, per_row), c = (i - row * per_row) * V;
  const int64_t slot = a.slots ? a.slots[row] : row;
  E* y = static_cast<E*>(a.y) + row * a.C + c;
  if (slot < 0 || slot >= a.pool) {
    store_vec<E, V>(y, zeros<V>());
    return;
  }
  const bool fresh = a.fresh && a.fresh[row];
  E* st = static_cast<E*>(a.state) + slot * (W - 1) * a.C + c;
  const Filter<V, W> f = load_filter<V, W>(a.weight, a.bias, c, a.vec_w);
  FloatV<V> win[W], o = f.bias;
#pragma unroll
  for (int j = 0; j < W - 1; ++j) win[j] = fresh ? zeros<V>() : load_vec<E, V>(st + j * a.C);
  win[W - 1] = load_vec<E, V>(static_cast<const E*>(a.x) + row * a.x_stride + c);
#pragma unroll
  for (int j = 0; j < W; ++j) o = fma_vec(f.w[j], win[j], o);
  if (SILU) o = mul_vec(o, sigmoid_vec(o));
  store_vec<E, V>(y, o);
#pragma unroll
  for (int j = 0; j < W - 1; ++j) store_vec<E, V>(st + j * a.C, win[j + 1]);
}

bool fits(const void* p, int bytes) { return reinterpret_cast<uintptr_t>(p) % bytes == 0; }
bool fits(const falcon_strides& s, int64_t H, int v) {
  return s.batch % v == 0 && s.time % v == 0 && (H == 1 || s.head % v == 0);
}

template <typename F>
cudaError_t with_width(int width, int act, F&& f) {
#define FALCON_CONV_CASE(W)                                                          \
  case W:                                                                            \
    return act == FALCON_ACT_SILU ? f(std::integral_constant<int, W>(), std::true_type()) \
                                  : f(std::integral_constant<int, W>(), std::false_type());
  switch (width) {
    FALCON_CONV_CASE(2)
    FALCON_CONV_CASE(3)
    FALCON_CONV_CASE(4)
  }
#undef FALCON_CONV_CASE
  return cudaErrorInvalidValue;
}

template <typename E, int V>
cudaError_t fwd_typed(const ConvArgs& a, cudaStream_t stream) {
  const int64_t nruns = (a.T + kFwdRun - 1) / kFwdRun;
  const int64_t blocks = (a.C / V * a.B * (nruns + 1) + kThreads - 1) / kThreads;
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
  return with_width(a.width, a.act, [&](auto w, auto silu) {
    conv_fwd_kernel<E, V, decltype(w)::value, decltype(silu)::value>
        <<<(unsigned)blocks, kThreads, 0, stream>>>(a, nruns);
    return cudaGetLastError();
  });
}

// How the gradient's tokens are cut: runs (whole blocks of tokens) and parts of the
// sums, one a run while they are few.  Of the runs up to 128 tokens, the one with the
// least estimated time, in tokens of a thread: waves of resident blocks (four an SM)
// times a run with its edge, and 0.06 for each part that the sums add up (measured: a
// token 0.19 us, 64 parts 0.7 us).  It counts the bf16 kernel of two channels a thread
// (112 tokens for B8 T2048 C2048); the others take the same cut, so that the workspace
// goes by the sizes alone, and their last wave may be partly full: one channel a thread
// makes twice the blocks, and in fp32 with silu and four taps three fit an SM
// (155 registers).
struct Cut {
  int run, parts;
};
constexpr int kMostParts = 1024;
Cut bwd_cut(int64_t B, int64_t T, int64_t C) {
  Cut best = {kBwdBlock, 1};
  double least = -1.0;
  for (int run = kBwdBlock; run <= 128; run += kBwdBlock) {
    const int64_t jobs = B * ((T + run - 1) / run);
    const int64_t parts = jobs < kMostParts ? jobs : kMostParts;
    const int64_t blocks = ((C + 1) / 2 * parts + kThreads - 1) / kThreads;
    const int64_t waves = (blocks + 152 * 4 - 1) / (152 * 4), turns = (jobs + parts - 1) / parts;
    const double cost = (double)(waves * turns) * (run + 8) + 0.06 * (double)parts;
    if (least < 0.0 || cost <= least) least = cost, best = {run, (int)parts};
    if (run >= T) break;
  }
  return best;
}

template <typename E, int V>
cudaError_t bwd_typed(const ConvArgs& a, cudaStream_t stream) {
  const Cut cut = bwd_cut(a.B, a.T, a.C);
  const int run = cut.run, parts = cut.parts;
  const int64_t nruns = (a.T + run - 1) / run;
  const int64_t blocks = (a.C / V * parts + kThreads - 1) / kThreads;
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
  return with_width(a.width, a.act, [&](auto w, auto silu) {
    constexpr int W = decltype(w)::value;
    conv_bwd_kernel<E, V, W, decltype(silu)::value>
        <<<(unsigned)blocks, kThreads, 0, stream>>>(a, run, nruns, parts);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    conv_sum_kernel<<<dim3((unsigned)((a.C + 31) / 32), W + 1), 256, 0, stream>>>(
        a.ws, parts, a.C, W, a.dweight, a.dbias);
    return cudaGetLastError();
  });
}

template <typename E, int V>
cudaError_t step_typed(const ConvStepArgs& a, cudaStream_t stream) {
  const int64_t count = a.N * ((a.C + V - 1) / V);
  return with_width(a.width, a.act, [&](auto w, auto silu) {
    conv_step_kernel<E, V, decltype(w)::value, decltype(silu)::value>
        <<<(unsigned)((count + kThreads - 1) / kThreads), kThreads, 0, stream>>>(a);
    return cudaGetLastError();
  });
}

}  // namespace

size_t conv_bwd_workspace_bytes(int64_t B, int64_t T, int64_t C, int width) {
  if (B == 0 || T == 0 || C == 0) return 0;
  return sizeof(float) * (size_t)bwd_cut(B, T, C).parts * (size_t)(width + 1) * (size_t)C;
}

cudaError_t launch_conv_fwd(const ConvArgs& in, cudaStream_t stream) {
  ConvArgs a = in;
  a.vec_w = fits(a.weight, 16);
  const int bytes = a.dtype == FALCON_BF16 ? 8 : 16;
  const bool vec = a.m % 4 == 0 && fits(a.x, bytes) && fits(a.y, bytes) && fits(a.state, bytes) &&
                   fits(a.state_out, bytes) && fits(a.xs, a.H, 4) && fits(a.ys, a.H, 4);
  if (a.dtype == FALCON_BF16)
    return vec ? fwd_typed<__nv_bfloat16, 4>(a, stream) : fwd_typed<__nv_bfloat16, 1>(a, stream);
  return vec ? fwd_typed<float, 4>(a, stream) : fwd_typed<float, 1>(a, stream);
}

cudaError_t launch_conv_bwd(const ConvArgs& in, cudaStream_t stream) {
  ConvArgs a = in;
  a.vec_w = fits(a.weight, 16);
  const int esz = a.dtype == FALCON_BF16 ? 2 : 4;
  const int64_t tail = a.B * (a.width - 1) * a.C;
  if (a.T == 0 || a.B == 0) {  // no token: dweight = dbias = 0, dstate = dstate_out
    cudaError_t e = cudaMemsetAsync(a.dweight, 0, sizeof(float) * a.C * a.width, stream);
    if (e == cudaSuccess && a.dbias)
      e = cudaMemsetAsync(a.dbias, 0, sizeof(float) * a.C, stream);
    if (e != cudaSuccess || !a.dstate || tail == 0) return e;
    if (!a.dstate_out) return cudaMemsetAsync(a.dstate, 0, (size_t)tail * esz, stream);
    return cudaMemcpyAsync(a.dstate, a.dstate_out, (size_t)tail * esz, cudaMemcpyDeviceToDevice,
                           stream);
  }
  // two channels a thread: four need over 150 registers (97 us for 8 x 2048 x 2048
  // bf16 elements when runs were 8 tokens long, against 68 with two)
  const int bytes = 2 * esz;
  const bool vec = a.m % 2 == 0 && fits(a.x, bytes) && fits(a.dy, bytes) && fits(a.dx, bytes) &&
                   fits(a.state, bytes) && fits(a.dstate_out, bytes) && fits(a.dstate, bytes) &&
                   fits(a.xs, a.H, 2) && fits(a.dys, a.H, 2) && fits(a.dxs, a.H, 2);
  if (a.dtype == FALCON_BF16)
    return vec ? bwd_typed<__nv_bfloat16, 2>(a, stream) : bwd_typed<__nv_bfloat16, 1>(a, stream);
  return vec ? bwd_typed<float, 2>(a, stream) : bwd_typed<float, 1>(a, stream);
}

cudaError_t launch_conv_step(const ConvStepArgs& in, cudaStream_t stream) {
  // four channels a thread for either type: the call is short, and more threads
  // with fewer loads each end sooner (256 sequences of 2048 channels, bf16: 5.3 us,
  // 12.6 with eight channels and filters read one weight at a time)
  ConvStepArgs a = in;
  a.vec_w = fits(a.weight, 16);
  const int bytes = a.dtype == FALCON_BF16 ? 8 : 16;
  const bool vec = a.C % 4 == 0 && a.x_stride % 4 == 0 && fits(a.x, bytes) &&
                   fits(a.state, bytes) && fits(a.y, bytes);
  if (a.dtype == FALCON_BF16)
    return vec ? step_typed<__nv_bfloat16, 4>(a, stream) : step_typed<__nv_bfloat16, 1>(a, stream);
  return vec ? step_typed<float, 4>(a, stream) : step_typed<float, 1>(a, stream);
}

}  // namespace falcon
