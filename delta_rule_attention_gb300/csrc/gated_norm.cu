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
// whose kernel is in gated_norm_bwd.cu.
//
// Measured: 16384 rows of 2048 channels with gate, residual and next norm (bf16, 268 MB)
// 52.7 us, 5.1 TB/s; 16384 rows of 12 heads of 64 (75 MB) 23 us.  With many rows a row is one
// warp's: a row costs a warp about 450 instructions for sums and addresses whatever its
// width, so 2048 channels in four warps took 107 us.  What is left there is issue slots (49%)
// and the shared-memory pipe (62%), through which the inputs and parameters pass; with
// heads, 15 warps an SM (101 registers) that issue once in 6.7 cycles each: 59% of the slots.
#include "gated_norm.cuh"

namespace falcon {
namespace {

// Inputs: h, z and x, those that there are.
template <typename E, int V, int K, int MODE>
__global__ void __launch_bounds__(V == 1 && K > 1 ? 512 : 256, V == 1 && K > 1 ? 1 : 2)
    norm_fwd_kernel(const __grid_constant__ NormArgs a, int ring, int params_bytes,
                    int staged_bytes) {
  extern __shared__ __align__(16) unsigned char shared[];
  float* par = reinterpret_cast<float*>(shared);
  float2* staged = reinterpret_cast<float2*>(shared + params_bytes);
  __shared__ float2 reds[8][64];
  float2* red = reds[threadIdx.y & 7];
  int turn = 0;
  const int64_t rows = a.B * a.T, step = (int64_t)gridDim.x * blockDim.y;
  constexpr int kBytes = Slot<E, V>::kBytes;
  const int threads = blockDim.x * blockDim.y, vec = threads * kBytes;  // a vector of all threads
  const int at_z = a.h ? K * vec : 0, at_x = at_z + (a.z ? K * vec : 0);
  const int row_bytes = at_x + (a.x ? K * vec : 0);
  unsigned char* mine =
      shared + staged_bytes + (threadIdx.y * blockDim.x + threadIdx.x) * kBytes;
  Place at[K];
#pragma unroll
  for (int k = 0; k < K; ++k) at[k] = place_of<V, MODE>(a, k);
  constexpr bool ahead = Slot<E, V>::kAhead;
  Held<E, V> own[3][ahead ? 1 : K];  // without slots: the next row's h, z and x
  auto copy_row = [&](const RowAt& r, int slot) {
    unsigned char* to = mine + slot * row_bytes;
    const E *hp = row_in<E>(a.h, a.hs, r), *zp = row_in<E>(a.z, a.zs, r),
            *xp = row_in<E>(a.x, a.xs, r);
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const bool on = at[k].live && r.held;
      auto copy = [&](int which, int off, const E* p) {
        if constexpr (ahead)
          copy_ahead<E>(to + off + k * vec, p, on);
        else
          own[which][k] = load_own<E>(p, on);
      };
      if (a.h) copy(0, 0, hp + in_heads<MODE>(a, a.hs, at[k]));
      if (a.z) copy(1, at_z, zp + at[k].c);
      if (a.x) copy(2, at_x, xp + at[k].c);
    }
    if (ahead) ahead_commit();
  };
  const int64_t row0 = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
  RowAt r(a, row0, step), next = r;
  for (int i = 0; i < (ahead ? ring : 1); ++i) {
    copy_row(next, i);
    next.advance(a);
  }
  stage_params(a, par);
  int slot = 0;
  // every thread takes part in every turn's barriers
  for (int64_t row = row0; row - threadIdx.y < rows; row += step, r.advance(a)) {
    if (ahead) ahead_wait(ring - 1);
    const unsigned char* from = mine + slot * row_bytes;
    auto input = [&](bool given, int which, int off, int k) {
      Held<E, V> v = {};
      if constexpr (ahead) {
        if (given) v = slot_vec<E, V>(from + off + k * vec);
      } else {
        if (given) v = own[which][k];
      }
      return v;
    };
    auto in_h = [&](int k) { return wide(input(true, 0, 0, k)); };
    FloatV<V> y[K];
    if (a.h) {
      Sums<1> ss[K];
#pragma unroll
      for (int k = 0; k < K; ++k) {
        const FloatV<V> hk = in_h(k);
        Dot<V> dot;
        dot.add(hk, hk);
        ss[k].v[0] = dot.sum();
      }
      head_sums<K, MODE, 1>(a, at, ss, V, red, turn, staged);
      E* op = row_of<E>(a.out, a.os, r);
#pragma unroll
      for (int k = 0; k < K; ++k) {
        FloatV<V> n = times<V>(in_h(k), rsqrtf(ss[k].v[0] / (float)a.m + a.eps));
        if (a.z) {
          n = mul_of<V>(n, gates(input(true, 1, at_z, k), a.gate));
        }
        const FloatV<V> x = wide(input(a.x, 2, at_x, k));
        n = fma_of<V>(n, param_vec<V>(par + at[k].c), x);
        y[k] = n;
        put_vec<E, V>(op + at[k].c, n, at[k].live && r.in, r.held);
      }
    } else {
#pragma unroll
      for (int k = 0; k < K; ++k) y[k] = wide(input(true, 2, at_x, k));
    }
    // this row's inputs are read
    copy_row(next, slot);
    next.advance(a);
    slot = slot + 1 < ring ? slot + 1 : 0;
    if (a.next) {
      Dot<V> dot;
#pragma unroll
      for (int k = 0; k < K; ++k) dot.add(y[k], y[k]);
      const Sums<1> s = row_sum<1>({dot.sum()}, blockDim.x, red, turn);
      const float rn = rsqrtf(s.v[0] / (float)a.D + a.eps);
      E* np = row_of<E>(a.next, a.ns, r);
#pragma unroll
      for (int k = 0; k < K; ++k)
        put_vec<E, V>(np + at[k].c,
                      mul_of<V>(times<V>(y[k], rn), param_vec<V>(par + a.D + at[k].c)),
                      at[k].live && r.in, r.held);
    }
  }
  if (ahead) ahead_wait(0);  // the last turns' copies, zeros for rows that there are not
}

template <typename E, int V, int K>
cudaError_t start_mode(const NormArgs& a, const NormPlan& p, unsigned grid, cudaStream_t stream) {
  static std::atomic<uint64_t> allowed[3];  // one a kernel
  if (p.mode == kWhole)
    return start_norm(norm_fwd_kernel<E, V, K, kWhole>, a, p, grid, &allowed[0], stream);
  if (p.mode == kLanes)
    return start_norm(norm_fwd_kernel<E, V, K, kLanes>, a, p, grid, &allowed[1], stream);
  return start_norm(norm_fwd_kernel<E, V, K, kStaged>, a, p, grid, &allowed[2], stream);
}

template <typename E, int V>
cudaError_t start_count(const NormArgs& a, const NormPlan& p, unsigned grid,
                        cudaStream_t stream) {
  if (p.K == 1) return start_mode<E, V, 1>(a, p, grid, stream);
  if constexpr (V > 1) {
    if (p.K == 2) return start_mode<E, V, 2>(a, p, grid, stream);
    if (p.K == 3) return start_mode<E, V, 3>(a, p, grid, stream);
  } else {
    if (p.K == 16) return start_mode<E, V, 16>(a, p, grid, stream);
  }
  if (p.K == 4) return start_mode<E, V, 4>(a, p, grid, stream);
  return start_mode<E, V, 8>(a, p, grid, stream);
}

}  // namespace

cudaError_t launch_norm_fwd(const NormArgs& a, cudaStream_t stream) {
  const Width widths[] = {{1, 256, 512}, {2, 256, 512}, {3, 256, 512}, {4, 256, 512},
                          {8, 256, 512}};
  const int inputs = (a.h ? 1 : 0) + (a.z ? 1 : 0) + (a.x ? 1 : 0);
  const NormPlan p = plan_norm(a, widths, 8, 152 * 16, inputs, false);
  const int64_t blocks = (a.B * a.T + p.rows - 1) / p.rows;
  const unsigned grid = (unsigned)(blocks < p.blocks ? blocks : p.blocks);
  if (a.dtype == FALCON_BF16)
    return p.V == 8 ? start_count<__nv_bfloat16, 8>(a, p, grid, stream)
                    : start_count<__nv_bfloat16, 1>(a, p, grid, stream);
  return p.V == 4 ? start_count<float, 4>(a, p, grid, stream)
                  : start_count<float, 1>(a, p, grid, stream);
}

}  // namespace falcon
