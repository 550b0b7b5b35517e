// One token of the selective scan for N sequences: the scan's formulas with the
// state read from and written to a pool.  A group of lanes owns a channel's
// state, four states (16 bytes) a lane: the step is bound by the state's traffic.

#include "ssm.cuh"

namespace falcon {
namespace {

constexpr int kThreads = 256;

// LN lanes of a channel (a power of two); VEC: S is a multiple of four and the
// state rows are 16-byte aligned.
template <typename E, int LN, bool VEC>
__global__ void __launch_bounds__(kThreads) scan_step_kernel(ScanStepArgs a) {
  const int64_t at = ((int64_t)blockIdx.x * kThreads + threadIdx.x) / LN;
  const int q = threadIdx.x % LN, n0 = q * 4;
  const bool live = at < a.N * a.D;
  const int64_t row = live ? at / a.D : 0;
  const int d = live ? (int)(at - row * a.D) : 0;
  const int64_t slot = a.slots ? a.slots[row] : row;
  const bool has = live && slot >= 0 && slot < a.pool;
  const bool fresh = a.fresh && a.fresh[row];
  const int g = d / (a.D / a.G);
  float* hp = a.h + ((has ? slot : 0) * a.D + d) * a.S + n0;
  float h[4] = {0.f, 0.f, 0.f, 0.f};
  if (has && !fresh) {
    if (VEC) {
      if (n0 < a.S) {
        const float4 v = *reinterpret_cast<const float4*>(hp);
        h[0] = v.x, h[1] = v.y, h[2] = v.z, h[3] = v.w;
      }
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (n0 + i < a.S) h[i] = hp[i];
    }
  }
  const float ut = load_vec<E, 1>(static_cast<const E*>(a.u) + row * a.u_stride + d).v[0];
  float s = load_vec<E, 1>(static_cast<const E*>(a.delta) + row * a.delta_stride + d).v[0];
  if (a.delta_bias) s += a.delta_bias[d];
  if (a.softplus) s = softplus(s);
  const E* Bm = static_cast<const E*>(a.Bm) + row * a.bs.batch + g * a.bs.head + n0;
  const E* Cm = static_cast<const E*>(a.Cm) + row * a.cs.batch + g * a.cs.head + n0;
  float o = 0.f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (n0 + i < a.S) {
      const float A2 = a.A[(int64_t)d * a.S + n0 + i] * kLog2e;
      h[i] = fmaf(decay(s, A2), h[i], s * ut * load_vec<E, 1>(Bm + i).v[0]);
      o = fmaf(load_vec<E, 1>(Cm + i).v[0], h[i], o);
    }
  }
  if (has) {
    if (VEC) {
      if (n0 < a.S) *reinterpret_cast<float4*>(hp) = make_float4(h[0], h[1], h[2], h[3]);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (n0 + i < a.S) hp[i] = h[i];
    }
  }
#pragma unroll
  for (int k = LN / 2; k > 0; k >>= 1) o += __shfl_xor_sync(0xffffffffu, o, k);
  if (live && q == 0) {
    if (a.Dskip) o = fmaf(a.Dskip[d], ut, o);
    if (a.z) {
      const float zt = load_vec<E, 1>(static_cast<const E*>(a.z) + row * a.z_stride + d).v[0];
      o *= zt * sigmoid(zt);
    }
    store_vec<E, 1>(static_cast<E*>(a.y) + row * a.D + d, FloatV<1>{{has ? o : 0.f}});
  }
}

template <typename E, int LN>
cudaError_t step_lanes(const ScanStepArgs& a, cudaStream_t stream) {
  const int64_t blocks = (a.N * a.D * LN + kThreads - 1) / kThreads;
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
  const bool vec = a.S % 4 == 0 && reinterpret_cast<uintptr_t>(a.h) % 16 == 0;
  if (vec)
    scan_step_kernel<E, LN, true><<<(unsigned)blocks, kThreads, 0, stream>>>(a);
  else
    scan_step_kernel<E, LN, false><<<(unsigned)blocks, kThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

template <typename E>
cudaError_t step_typed(const ScanStepArgs& a, cudaStream_t stream) {
  if (a.S <= 4) return step_lanes<E, 1>(a, stream);
  if (a.S <= 8) return step_lanes<E, 2>(a, stream);
  if (a.S <= 16) return step_lanes<E, 4>(a, stream);
  if (a.S <= 32) return step_lanes<E, 8>(a, stream);
  if (a.S <= 64) return step_lanes<E, 16>(a, stream);
  return step_lanes<E, 32>(a, stream);
}

}  // namespace

cudaError_t launch_scan_step(const ScanStepArgs& a, cudaStream_t stream) {
  return a.dtype == FALCON_BF16 ? step_typed<__nv_bfloat16>(a, stream)
                                : step_typed<float>(a, stream);
}

}  // namespace falcon
