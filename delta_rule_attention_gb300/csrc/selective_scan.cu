// Selective scan over prompts:
//   s_t = softplus(delta_t + bias),  h_t = exp(s_t A) h_{t-1} + s_t u_t B_t,
//   y_t = (<C_t, h_t> + Dskip u_t) silu(z_t)
// for every channel with its N states.  A group of LN lanes owns a channel, four
// states a lane, and walks the tokens in order with the states in registers.

#include <type_traits>

#include "ssm.cuh"

namespace falcon {
namespace {

constexpr int kWarps = 4;

template <typename E, int LN>
__global__ void __launch_bounds__(kWarps * 32) scan_fwd_kernel(ScanArgs a) {
  constexpr int kCh = 32 / LN;  // channels of a warp
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int q = lane % LN, n0 = q * 4;
  const int R = a.D / a.G;
  const int blocks = (R + kCh * kWarps - 1) / (kCh * kWarps);  // per group
  const int g = blockIdx.x / blocks;
  const int r = ((blockIdx.x - g * blocks) * kWarps + warp) * kCh + lane / LN;
  const bool live = r < R;
  const int d = g * R + (live ? r : 0);
  const int64_t b = blockIdx.y;
  const int64_t n = row_length(a.lengths, b, a.T);

  float A2[4], h[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const bool in = n0 + i < a.N;
    A2[i] = in ? a.A[(int64_t)d * a.N + n0 + i] * kLog2e : 0.f;
    h[i] = in && a.h0 ? a.h0[(b * a.D + d) * a.N + n0 + i] : 0.f;
  }
  const float bias = a.delta_bias ? a.delta_bias[d] : 0.f;
  const float skip = a.Dskip ? a.Dskip[d] : 0.f;
  const E* u = static_cast<const E*>(a.u) + b * a.us.batch + d;
  const E* dl = static_cast<const E*>(a.delta) + b * a.ds.batch + d;
  const E* z = a.z ? static_cast<const E*>(a.z) + b * a.zs.batch + d : nullptr;
  const E* Bm = static_cast<const E*>(a.Bm) + b * a.bs.batch + g * a.bs.head + n0;
  const E* Cm = static_cast<const E*>(a.Cm) + b * a.cs.batch + g * a.cs.head + n0;
  E* y = static_cast<E*>(a.y) + b * a.ys.batch + d;

  for (int64_t t = 0; t < n; ++t) {
    const float ut = load_vec<E, 1>(u + t * a.us.time).v[0];
    float s = load_vec<E, 1>(dl + t * a.ds.time).v[0] + bias;
    if (a.softplus) s = softplus(s);
    float o = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const bool in = n0 + i < a.N;
      const float Bt = in ? load_vec<E, 1>(Bm + t * a.bs.time + i).v[0] : 0.f;
      const float Ct = in ? load_vec<E, 1>(Cm + t * a.cs.time + i).v[0] : 0.f;
      h[i] = fmaf(decay(s, A2[i]), h[i], s * ut * Bt);
      o = fmaf(Ct, h[i], o);
    }
#pragma unroll
    for (int k = LN / 2; k > 0; k >>= 1) o += __shfl_xor_sync(0xffffffffu, o, k);
    if (live && q == 0) {
      o = fmaf(skip, ut, o);
      if (z) {
        const float zt = load_vec<E, 1>(z + t * a.zs.time).v[0];
        o *= zt * sigmoid(zt);
      }
      store_vec<E, 1>(y + t * a.ys.time, FloatV<1>{{o}});
    }
  }
  if (!live) return;
  for (int64_t t = n + q; t < a.T; t += LN) store_vec<E, 1>(y + t * a.ys.time, FloatV<1>{{0.f}});
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (n0 + i < a.N) a.h_out[(b * a.D + d) * a.N + n0 + i] = h[i];
}

template <typename E, int LN>
cudaError_t fwd_lanes(const ScanArgs& a, cudaStream_t stream) {
  const int R = a.D / a.G, per = 32 / LN * kWarps;
  const dim3 grid((unsigned)(a.G * ((R + per - 1) / per)), (unsigned)a.B);
  scan_fwd_kernel<E, LN><<<grid, kWarps * 32, 0, stream>>>(a);
  return cudaGetLastError();
}

template <typename E>
cudaError_t fwd_typed(const ScanArgs& a, cudaStream_t stream) {
  if (a.N <= 4) return fwd_lanes<E, 1>(a, stream);
  if (a.N <= 8) return fwd_lanes<E, 2>(a, stream);
  if (a.N <= 16) return fwd_lanes<E, 4>(a, stream);
  if (a.N <= 32) return fwd_lanes<E, 8>(a, stream);
  if (a.N <= 64) return fwd_lanes<E, 16>(a, stream);
  return fwd_lanes<E, 32>(a, stream);
}

}  // namespace

cudaError_t launch_scan_fwd(const ScanArgs& a, cudaStream_t stream) {
  return a.dtype == FALCON_BF16 ? fwd_typed<__nv_bfloat16>(a, stream)
                                : fwd_typed<float>(a, stream);
}

}  // namespace falcon
