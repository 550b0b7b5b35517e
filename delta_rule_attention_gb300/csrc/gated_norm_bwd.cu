// The gradient of the gated norm (formulas: gated_norm.cu).  A block takes rows in turn:
// the next row's inputs are loaded while this row's sums are formed, and a thread keeps
// the sums over rows of its channels for the parameters; a second kernel adds the blocks'
// sums in a fixed order.
//
// Bound by latency: 16384 rows of 2048 channels (bf16, 403 MB) 110 us, 3.7 TB/s, of which the
// blocks' sums take 6 (8 with a block for every 32 channels).  63 instructions a value go
// through half of the issue slots (54%): 125 registers leave 15 warps an SM, and a warp issues
// once in 6.9 cycles, waiting for fixed latencies (1.6) and shared memory (1.7) most.  12
// heads of 64 with a gate (16384 rows): 61 us, 168 registers, 11 warps, 49%.  The plan's limit
// of two vectors a thread: with four, 384 threads an SM hold the registers and the same rows
// take 118 us; one instruction for two values (112 us before: 114).
#include "gated_norm.cuh"

namespace falcon {
namespace {

// Inputs: h, z, dout, out and dnext, those that there are.
template <typename E, int V, int K, int MODE>
__global__ void __launch_bounds__(V == 1 ? (K > 1 ? 512 : 256) : K == 3 || K == 4 ? 128 : 256,
                                  V == 1 ? (K > 1 ? 1 : 2)
                                  : K == 3 || K == 4 ? 3
                                  : K == 8           ? 1
                                                     : 2)
    norm_bwd_kernel(const __grid_constant__ NormArgs a, int ring, int params_bytes,
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
  const int at_z = a.h ? K * vec : 0, at_d = at_z + (a.z ? K * vec : 0),
            at_y = at_d + (a.dout ? K * vec : 0), at_e = at_y + (a.next_weight ? K * vec : 0),
            row_bytes = at_e + (a.next_weight ? K * vec : 0);
  unsigned char* mine =
      shared + staged_bytes + (threadIdx.y * blockDim.x + threadIdx.x) * kBytes;
  FloatV<V> each[K], nextw[K];  // sums for dweight and dscale, and for dnext_weight
  Place at[K];
#pragma unroll
  for (int k = 0; k < K; ++k) {
    each[k] = zeros<E, V>(), nextw[k] = zeros<E, V>();
    at[k] = place_of<V, MODE>(a, k);
  }
  constexpr bool ahead = Slot<E, V>::kAhead;
  Held<E, V> own[5][ahead ? 1 : K];  // without slots: the next row's h, z, dout, out and dnext
  auto copy_row = [&](const RowAt& r, int slot) {
    unsigned char* to = mine + slot * row_bytes;
    const E *hp = row_in<E>(a.h, a.hs, r), *zp = row_in<E>(a.z, a.zs, r),
            *dp = row_in<E>(a.dout, a.dos, r), *yp = row_in<E>(a.y, a.os, r),
            *ep = row_in<E>(a.dnext, a.dns, r);
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
      if (a.dout) copy(2, at_d, dp + at[k].c);
      if (a.next_weight) copy(3, at_y, yp + at[k].c), copy(4, at_e, ep + at[k].c);
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
    auto in_z = [&](int k) { return input(true, 1, at_z, k); };
    auto in_y = [&](int k) { return wide(input(true, 3, at_y, k)); };
    auto in_e = [&](int k) { return wide(input(true, 4, at_e, k)); };
    auto ws = [&](int k) { return param_vec<V>(par + at[k].c); };
    auto wn = [&](int k) { return param_vec<V>(par + a.D + at[k].c); };
    FloatV<V> d[K];
#pragma unroll
    for (int k = 0; k < K; ++k) d[k] = wide(input(a.dout, 2, at_d, k));
    if (a.next_weight) {
      Dot<V> yy, ey;
#pragma unroll
      for (int k = 0; k < K; ++k) {
        const FloatV<V> y = in_y(k);
        yy.add(y, y);
        ey.add(mul_of<V>(in_e(k), wn(k)), y);
      }
      const Sums<2> s = row_sum<2>({yy.sum(), ey.sum()}, blockDim.x, red, turn);
      const float rn = rsqrtf(s.v[0] / (float)a.D + a.eps);
      // zero where rn is, whatever the other sum has come to
      const float back = rn > 0.f ? -rn * (rn * s.v[1] / (float)a.D) : 0.f;
#pragma unroll
      for (int k = 0; k < K; ++k) {
        const FloatV<V> y = in_y(k), er = times<V>(in_e(k), rn);
        nextw[k] = fma_of<V>(er, y, nextw[k]);
        d[k] = fma_of<V>(er, wn(k), d[k]);
        d[k] = fma_of<V>(y, rn * back, d[k]);
      }
    }
    if (a.dx) {
      E* p = row_of<E>(a.dx, a.dxs, r);
#pragma unroll
      for (int k = 0; k < K; ++k) put_vec<E, V>(p + at[k].c, d[k], at[k].live && r.in, r.held);
    }
    if (a.h) {
      Sums<2> s[K];
#pragma unroll
      for (int k = 0; k < K; ++k) {
        FloatV<V> f = mul_of<V>(d[k], ws(k));  // of n times the parameters
        const FloatV<V> h = in_h(k);
        Dot<V> hh, fh;
        hh.add(h, h);
        if (a.z) {
          f = mul_of<V>(f, gates(in_z(k), a.gate));
        }
        fh.add(f, h);
        s[k].v[0] = hh.sum(), s[k].v[1] = fh.sum();
      }
      head_sums<K, MODE, 2>(a, at, s, V, red, turn, staged);
      E *hp = row_of<E>(a.dh, a.dhs, r), *zp = row_of<E>(a.dz, a.dzs, r);
#pragma unroll
      for (int k = 0; k < K; ++k) {
        const float rn = rsqrtf(s[k].v[0] / (float)a.m + a.eps);
        const float back = rn > 0.f ? -rn * (rn * s[k].v[1] / (float)a.m) : 0.f;
        const FloatV<V> h = in_h(k), n = times<V>(h, rn);
        FloatV<V> f = mul_of<V>(d[k], ws(k));
        if (a.z) {
          const FloatV<V> g = gates(in_z(k), a.gate);
          const FloatV<V> dz = mul_of<V>(mul_of<V>(f, n), slopes(in_z(k), a.gate));
          f = mul_of<V>(f, g);
          d[k] = mul_of<V>(d[k], g);
          put_vec<E, V>(zp + at[k].c, dz, at[k].live && r.in, r.held);
        }
        each[k] = fma_of<V>(d[k], n, each[k]);
        put_vec<E, V>(hp + in_heads<MODE>(a, a.dhs, at[k]),
                      times<V>(fma_of<V>(h, back, f), rn), at[k].live && r.in,
                      r.held);
      }
    }
    // this row's inputs are read
    copy_row(next, slot);
    next.advance(a);
    slot = slot + 1 < ring ? slot + 1 : 0;
  }
  if (ahead) ahead_wait(0);  // the last turns' copies, zeros for rows that there are not
  float* part = a.ws + ((int64_t)blockIdx.x * blockDim.y + threadIdx.y) * 2 * a.D;
#pragma unroll
  for (int k = 0; k < K; ++k) {
    if (at[k].live) {
#pragma unroll
      for (int i = 0; i < V; ++i)
        part[at[k].c + i] = each[k].v[i], part[a.D + at[k].c + i] = nextw[k].v[i];
    }
  }
}

// Adds the blocks' sums: 8 channels a block, 128 threads a channel, in a fixed order.
constexpr int kPartThreads = 128, kPartChannels = 8;
__global__ void __launch_bounds__(kPartChannels* kPartThreads)
    norm_params_kernel(const __grid_constant__ NormArgs a) {
  constexpr int kWarps = kPartChannels * kPartThreads / 32;
  __shared__ float red[2][kWarps][kPartChannels];
  const int c = blockIdx.x * kPartChannels + threadIdx.x;
  float s0 = 0.f, s1 = 0.f;
  if (c < a.D) {
    for (int p = threadIdx.y; p < a.parts; p += kPartThreads) {
      s0 += a.ws[(int64_t)p * 2 * a.D + c];
      if (a.dnext_weight) s1 += a.ws[(int64_t)p * 2 * a.D + a.D + c];
    }
  }
#pragma unroll
  for (int o = kPartChannels; o < 32; o *= 2) {
    s0 += __shfl_xor_sync(0xffffffffu, s0, o);
    s1 += __shfl_xor_sync(0xffffffffu, s1, o);
  }
  const int lane = (threadIdx.y * kPartChannels + threadIdx.x) % 32,
            warp = (threadIdx.y * kPartChannels + threadIdx.x) / 32;
  if (lane < kPartChannels) red[0][warp][lane] = s0, red[1][warp][lane] = s1;
  __syncthreads();
  if (threadIdx.y == 0 && c < a.D) {
    s0 = s1 = 0.f;
    for (int w = 0; w < kWarps; ++w) s0 += red[0][w][threadIdx.x], s1 += red[1][w][threadIdx.x];
    if (a.dweight) a.dweight[c] = a.scale ? s0 * a.scale[c] : s0;
    if (a.dscale) a.dscale[c] = a.weight ? s0 * a.weight[c] : s0;
    if (a.dnext_weight) a.dnext_weight[c] = s1;
  }
}

unsigned bwd_blocks(const NormArgs& a, const NormPlan& p) {
  const int64_t blocks = (a.B * a.T + p.rows - 1) / p.rows;
  return (unsigned)(blocks < p.blocks ? blocks : p.blocks);
}

NormPlan plan_bwd(const NormArgs& a, int inputs, bool narrow) {
  const Width widths[] = {{1, 256, 512}, {2, 256, 512}, {3, 128, 384}, {4, 128, 384},
                          {8, 256, 256}};
  return plan_norm(a, widths, 2, 152 * 16, inputs, narrow);
}

template <typename E, int V, int K>
cudaError_t start_mode(const NormArgs& a, const NormPlan& p, unsigned grid, cudaStream_t stream) {
  static std::atomic<uint64_t> allowed[3];  // one a kernel
  if (p.mode == kWhole)
    return start_norm(norm_bwd_kernel<E, V, K, kWhole>, a, p, grid, &allowed[0], stream);
  if (p.mode == kLanes)
    return start_norm(norm_bwd_kernel<E, V, K, kLanes>, a, p, grid, &allowed[1], stream);
  return start_norm(norm_bwd_kernel<E, V, K, kStaged>, a, p, grid, &allowed[2], stream);
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

// Room for every launch that a call of this shape may make: it goes by its pointers.
size_t norm_bwd_workspace_bytes(const falcon_norm_shape& s) {
  NormArgs a = {};
  a.B = s.B, a.T = s.T, a.H = (int)s.H, a.m = s.m, a.D = (int)(s.H * s.m), a.dtype = s.dtype;
  int64_t most = 0;
  for (int inputs = 1; inputs <= 5; ++inputs)
    for (int narrow = 0; narrow < 2; ++narrow) {
      const NormPlan p = plan_bwd(a, inputs, narrow != 0);
      const int64_t parts = (int64_t)bwd_blocks(a, p) * p.rows;
      most = parts > most ? parts : most;
    }
  return (size_t)most * 2 * a.D * 4;
}

cudaError_t launch_norm_bwd(const NormArgs& args, cudaStream_t stream) {
  NormArgs a = args;
  const int inputs =
      (a.h ? 1 : 0) + (a.z ? 1 : 0) + (a.dout ? 1 : 0) + (a.next_weight ? 2 : 0);
  const NormPlan p = plan_bwd(a, inputs, false);
  const unsigned grid = bwd_blocks(a, p);
  a.parts = (int)grid * p.rows;
  if (grid > 0) {
    cudaError_t e;
    if (a.dtype == FALCON_BF16)
      e = p.V == 8 ? start_count<__nv_bfloat16, 8>(a, p, grid, stream)
                   : start_count<__nv_bfloat16, 1>(a, p, grid, stream);
    else
      e = p.V == 4 ? start_count<float, 4>(a, p, grid, stream)
                   : start_count<float, 1>(a, p, grid, stream);
    if (e != cudaSuccess) return e;
  }
  if (a.dweight || a.dscale || a.dnext_weight)
    norm_params_kernel<<<(unsigned)((a.D + kPartChannels - 1) / kPartChannels),
                         dim3(kPartChannels, kPartThreads), 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace falcon
