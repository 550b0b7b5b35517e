// Short causal convolution: forward, gradient, and one token of many sequences.
//
//   p_t = bias + sum_{j<W} w_j x_{t-W+1+j},  y_t = act(p_t)
//   dp_t = dy_t act'(p_t),  dx_t = sum_j w_j dp_{t+W-1-j},
//   dw_j = sum_t dp_t x_{t-W+1+j},  dbias = sum_t dp_t
//
// A thread owns V neighbouring channels (one access of up to 16 bytes) and
// walks a run of tokens with the last W inputs in registers, so each input is
// read from memory once and W - 1 times more at a run's edge, from cache.

#include <type_traits>

#include "ssm.cuh"

namespace falcon {
namespace {

constexpr int kThreads = 128;

// Offset of channel c of row (b, t): channels are grouped in heads of m.
__device__ __forceinline__ int64_t row_offset(const falcon_strides& s, int64_t b, int64_t c,
                                              int m) {
  const int64_t h = c / m;
  return b * s.batch + h * s.head + (c - h * m);
}

template <int V>
__device__ __forceinline__ FloatV<V> zeros() {
  FloatV<V> r;
#pragma unroll
  for (int i = 0; i < V; ++i) r.v[i] = 0.f;
  return r;
}

// Input at time t of row b, which may be a carried one (t < 0).
template <typename E, int V, int W>
__device__ __forceinline__ FloatV<V> input_at(const E* xrow, int64_t tstride, const E* state,
                                              int64_t b, int64_t C, int64_t c, int64_t t) {
  if (t >= 0) return load_vec<E, V>(xrow + t * tstride);
  if (state) return load_vec<E, V>(state + (b * (W - 1) + (t + W - 1)) * C + c);
  return zeros<V>();
}

template <int V, int W>
struct Filter {
  float w[W][V];
  float bias[V];
};

template <int V, int W>
__device__ __forceinline__ Filter<V, W> load_filter(const float* weight, const float* bias,
                                                    int64_t c) {
  Filter<V, W> f;
#pragma unroll
  for (int i = 0; i < V; ++i) {
#pragma unroll
    for (int j = 0; j < W; ++j) f.w[j][i] = weight[(c + i) * W + j];
    f.bias[i] = bias ? bias[c + i] : 0.f;
  }
  return f;
}

template <typename E, int V, int W, bool SILU>
__global__ void __launch_bounds__(kThreads) conv_fwd_kernel(ConvArgs a, int run, int64_t nruns) {
  const int64_t c = ((int64_t)blockIdx.x * kThreads + threadIdx.x) * V;
  if (c >= a.C) return;
  for (int64_t job = blockIdx.y; job < a.B * (nruns + 1); job += gridDim.y) {
    const int64_t b = job / (nruns + 1), r = job - b * (nruns + 1);
    const int64_t n = row_length(a.lengths, b, a.T);
    const E* x = static_cast<const E*>(a.x) + row_offset(a.xs, b, c, a.m);
    const E* state = static_cast<const E*>(a.state);
    if (r == nruns) {  // the row's last W - 1 inputs
      if (!a.state_out) continue;
#pragma unroll
      for (int j = 0; j < W - 1; ++j)
        store_vec<E, V>(static_cast<E*>(a.state_out) + (b * (W - 1) + j) * a.C + c,
                        input_at<E, V, W>(x, a.xs.time, state, b, a.C, c, n - (W - 1) + j));
      continue;
    }
    const int64_t t0 = r * run, t1 = t0 + run < a.T ? t0 + run : a.T;
    const int64_t te = t1 < n ? t1 : n;
    E* y = static_cast<E*>(a.y) + row_offset(a.ys, b, c, a.m);
    if (t0 < te) {
      const Filter<V, W> f = load_filter<V, W>(a.weight, a.bias, c);
      FloatV<V> win[W];
#pragma unroll
      for (int j = 0; j < W - 1; ++j)
        win[j] = input_at<E, V, W>(x, a.xs.time, state, b, a.C, c, t0 - (W - 1) + j);
#pragma unroll 4
      for (int64_t t = t0; t < te; ++t) {
        win[W - 1] = load_vec<E, V>(x + t * a.xs.time);
        FloatV<V> o;
#pragma unroll
        for (int i = 0; i < V; ++i) {
          float p = f.bias[i];
#pragma unroll
          for (int j = 0; j < W; ++j) p = fmaf(f.w[j][i], win[j].v[i], p);
          o.v[i] = SILU ? p * sigmoid(p) : p;
        }
        store_vec<E, V>(y + t * a.ys.time, o);
#pragma unroll
        for (int j = 0; j < W - 1; ++j) win[j] = win[j + 1];
      }
    }
    for (int64_t t = te > t0 ? te : t0; t < t1; ++t) store_vec<E, V>(y + t * a.ys.time, zeros<V>());
  }
}

// Gradient: dp of the run's tokens and of the W - 1 after it (recomputed from
// x), each dp_t adding w_j dp_t to dx_{t-W+1+j}.  A block walks every
// gridDim.y-th run with its sums of dw and dbias in registers and writes them
// once; conv_sum_kernel adds the blocks' sums in their order.
template <typename E, int V, int W, bool SILU>
__global__ void __launch_bounds__(kThreads) conv_bwd_kernel(ConvArgs a, int run, int64_t nruns) {
  const int64_t c = ((int64_t)blockIdx.x * kThreads + threadIdx.x) * V;
  if (c >= a.C) return;
  const Filter<V, W> f = load_filter<V, W>(a.weight, a.bias, c);
  float dw[W][V] = {}, db[V] = {};
  for (int64_t job = blockIdx.y; job < a.B * nruns; job += gridDim.y) {
    const int64_t b = job / nruns, r = job - b * nruns;
    const int64_t n = row_length(a.lengths, b, a.T);
    const E* x = static_cast<const E*>(a.x) + row_offset(a.xs, b, c, a.m);
    const E* dy = static_cast<const E*>(a.dy) + row_offset(a.dys, b, c, a.m);
    E* dx = static_cast<E*>(a.dx) + row_offset(a.dxs, b, c, a.m);
    const E* state = static_cast<const E*>(a.state);
    const E* dso = static_cast<const E*>(a.dstate_out);
    const int64_t t0 = r * run, t1 = t0 + run < a.T ? t0 + run : a.T;
    // acc[j] gathers the gradient of input t - W + 1 + j
    FloatV<V> win[W], acc[W];
#pragma unroll
    for (int j = 0; j < W - 1; ++j) {
      win[j] = input_at<E, V, W>(x, a.xs.time, state, b, a.C, c, t0 - (W - 1) + j);
      acc[j] = zeros<V>();
    }
    // gradient of an input: stored where the input is this run's own; the
    // first run also stores those of the carried inputs
    auto finish = [&](int64_t s, FloatV<V> g) {
      if (s >= t1 || (s < t0 && s >= 0) || (s < 0 && t0 > 0)) return;
      const int64_t k = s - (n - (W - 1));  // its place in state_out
      if (dso && k >= 0 && s < n) {
        const FloatV<V> d = load_vec<E, V>(dso + (b * (W - 1) + k) * a.C + c);
#pragma unroll
        for (int i = 0; i < V; ++i) g.v[i] += d.v[i];
      }
      if (s >= 0)
        store_vec<E, V>(dx + s * a.dxs.time, g);
      else if (a.dstate)
        store_vec<E, V>(static_cast<E*>(a.dstate) + (b * (W - 1) + s + W - 1) * a.C + c, g);
    };
    const int64_t last = t1 + W - 1;
#pragma unroll 2
    for (int64_t t = t0; t < last; ++t) {
      acc[W - 1] = zeros<V>();
      win[W - 1] = zeros<V>();
      if (t < n) {
        win[W - 1] = load_vec<E, V>(x + t * a.xs.time);
        FloatV<V> d = load_vec<E, V>(dy + t * a.dys.time);
#pragma unroll
        for (int i = 0; i < V; ++i) {
          if (SILU) {
            float p = f.bias[i];
#pragma unroll
            for (int j = 0; j < W; ++j) p = fmaf(f.w[j][i], win[j].v[i], p);
            const float s = sigmoid(p);
            d.v[i] *= s * fmaf(p, 1.f - s, 1.f);
          }
#pragma unroll
          for (int j = 0; j < W; ++j) acc[j].v[i] = fmaf(f.w[j][i], d.v[i], acc[j].v[i]);
          if (t < t1) {
            db[i] += d.v[i];
#pragma unroll
            for (int j = 0; j < W; ++j) dw[j][i] = fmaf(d.v[i], win[j].v[i], dw[j][i]);
          }
        }
      }
      finish(t - (W - 1), acc[0]);
#pragma unroll
      for (int j = 0; j < W - 1; ++j) {
        win[j] = win[j + 1];
        acc[j] = acc[j + 1];
      }
    }
  }
  float* ws = a.ws + (int64_t)blockIdx.y * (W + 1) * a.C;
#pragma unroll
  for (int i = 0; i < V; ++i) {
#pragma unroll
    for (int j = 0; j < W; ++j) ws[j * a.C + c + i] = dw[j][i];
    ws[W * a.C + c + i] = db[i];
  }
}

__global__ void conv_sum_kernel(const float* ws, int parts, int64_t C, int W, float* dweight,
                                float* dbias) {
  const int64_t c = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  const int j = blockIdx.y;
  if (c >= C) return;
  float s = 0.f;
  for (int p = 0; p < parts; ++p) s += ws[((int64_t)p * (W + 1) + j) * C + c];
  if (j < W)
    dweight[c * W + j] = s;
  else if (dbias)
    dbias[c] = s;
}

template <typename E, int V, int W, bool SILU>
__global__ void __launch_bounds__(kThreads) conv_step_kernel(ConvStepArgs a) {
  const int64_t per_row = (a.C + V - 1) / V;
  const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  if (i >= a.N * per_row) return;
  const int64_t row = i / per_row, c = (i - row * per_row) * V;
  const int64_t slot = a.slots ? a.slots[row] : row;
  E* y = static_cast<E*>(a.y) + row * a.C + c;
  if (slot < 0 || slot >= a.pool) {
    store_vec<E, V>(y, zeros<V>());
    return;
  }
  const bool fresh = a.fresh && a.fresh[row];
  E* st = static_cast<E*>(a.state) + slot * (W - 1) * a.C + c;
  const Filter<V, W> f = load_filter<V, W>(a.weight, a.bias, c);
  FloatV<V> win[W], o;
#pragma unroll
  for (int j = 0; j < W - 1; ++j) win[j] = fresh ? zeros<V>() : load_vec<E, V>(st + j * a.C);
  win[W - 1] = load_vec<E, V>(static_cast<const E*>(a.x) + row * a.x_stride + c);
#pragma unroll
  for (int k = 0; k < V; ++k) {
    float p = f.bias[k];
#pragma unroll
    for (int j = 0; j < W; ++j) p = fmaf(f.w[j][k], win[j].v[k], p);
    o.v[k] = SILU ? p * sigmoid(p) : p;
  }
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
  const int run = 16;
  const int64_t nruns = (a.T + run - 1) / run;
  const int64_t cblocks = (a.C + (int64_t)kThreads * V - 1) / ((int64_t)kThreads * V);
  const int64_t jobs = a.B * (nruns + 1);
  const dim3 grid((unsigned)cblocks, (unsigned)(jobs < 65535 ? jobs : 65535));
  return with_width(a.width, a.act, [&](auto w, auto silu) {
    conv_fwd_kernel<E, V, decltype(w)::value, decltype(silu)::value>
        <<<grid, kThreads, 0, stream>>>(a, run, nruns);
    return cudaGetLastError();
  });
}

constexpr int kBwdRun = 32;
// Blocks along (row, run): each leaves one set of sums.
int bwd_parts(int64_t B, int64_t T) {
  const int64_t jobs = B * ((T + kBwdRun - 1) / kBwdRun);
  return (int)(jobs < 256 ? jobs : 256);
}

template <typename E, int V>
cudaError_t bwd_typed(const ConvArgs& a, cudaStream_t stream) {
  const int64_t nruns = (a.T + kBwdRun - 1) / kBwdRun;
  const int64_t cblocks = (a.C + (int64_t)kThreads * V - 1) / ((int64_t)kThreads * V);
  const int parts = bwd_parts(a.B, a.T);
  const dim3 grid((unsigned)cblocks, (unsigned)parts);
  return with_width(a.width, a.act, [&](auto w, auto silu) {
    constexpr int W = decltype(w)::value;
    conv_bwd_kernel<E, V, W, decltype(silu)::value><<<grid, kThreads, 0, stream>>>(a, kBwdRun,
                                                                                nruns);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    conv_sum_kernel<<<dim3((unsigned)((a.C + 127) / 128), W + 1), 128, 0, stream>>>(
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
  return sizeof(float) * (size_t)bwd_parts(B, T) * (size_t)(width + 1) * (size_t)C;
}

cudaError_t launch_conv_fwd(const ConvArgs& a, cudaStream_t stream) {
  const int esz = a.dtype == FALCON_BF16 ? 2 : 4;
  const int v = 16 / esz;
  const bool vec = a.m % v == 0 && fits(a.x, 16) && fits(a.y, 16) && fits(a.state, 16) &&
                   fits(a.state_out, 16) && fits(a.xs, a.H, v) && fits(a.ys, a.H, v);
  if (a.dtype == FALCON_BF16)
    return vec ? fwd_typed<__nv_bfloat16, 8>(a, stream) : fwd_typed<__nv_bfloat16, 1>(a, stream);
  return vec ? fwd_typed<float, 4>(a, stream) : fwd_typed<float, 1>(a, stream);
}

cudaError_t launch_conv_bwd(const ConvArgs& a, cudaStream_t stream) {
  const int esz = a.dtype == FALCON_BF16 ? 2 : 4;
  const int64_t tail = a.B * (a.width - 1) * a.C;
  if (a.T == 0) {  // no token: dweight = dbias = 0, dstate = dstate_out
    cudaError_t e = cudaMemsetAsync(a.dweight, 0, sizeof(float) * a.C * a.width, stream);
    if (e == cudaSuccess && a.dbias)
      e = cudaMemsetAsync(a.dbias, 0, sizeof(float) * a.C, stream);
    if (e != cudaSuccess || !a.dstate) return e;
    if (!a.dstate_out) return cudaMemsetAsync(a.dstate, 0, (size_t)tail * esz, stream);
    return cudaMemcpyAsync(a.dstate, a.dstate_out, (size_t)tail * esz, cudaMemcpyDeviceToDevice,
                           stream);
  }
  const int bytes = 4 * esz;
  const bool vec = a.m % 4 == 0 && fits(a.x, bytes) && fits(a.dy, bytes) && fits(a.dx, bytes) &&
                   fits(a.state, bytes) && fits(a.dstate_out, bytes) && fits(a.dstate, bytes) &&
                   fits(a.xs, a.H, 4) && fits(a.dys, a.H, 4) && fits(a.dxs, a.H, 4);
  if (a.dtype == FALCON_BF16)
    return vec ? bwd_typed<__nv_bfloat16, 4>(a, stream) : bwd_typed<__nv_bfloat16, 1>(a, stream);
  return vec ? bwd_typed<float, 4>(a, stream) : bwd_typed<float, 1>(a, stream);
}

cudaError_t launch_conv_step(const ConvStepArgs& a, cudaStream_t stream) {
  const int v = a.dtype == FALCON_BF16 ? 8 : 4;
  const bool vec = a.C % v == 0 && a.x_stride % v == 0 && fits(a.x, 16) && fits(a.state, 16) &&
                   fits(a.y, 16);
  if (a.dtype == FALCON_BF16)
    return vec ? step_typed<__nv_bfloat16, 8>(a, stream) : step_typed<__nv_bfloat16, 1>(a, stream);
  return vec ? step_typed<float, 4>(a, stream) : step_typed<float, 1>(a, stream);
}

}  // namespace falcon
