// One token of the selective scan for N sequences: the scan's formulas with the
// state read from and written to a pool.  Bound by the state's traffic: 1024
// sequences of D 2048, S 16, bf16: 52 us, 5.5 TB/s (81% of a copy's rate).

#include "ssm.cuh"

namespace falcon {
namespace {

constexpr int kThreads = 128;

// LN lanes share two neighbouring channels.  vec_h: S is a multiple of four and
// the states lie on 16-byte boundaries; vec_ch, vec_bc: channel pairs and quads of B
// and C are one access.  A lane's loads do not depend on one another (but for the
// slot), so that its 32 bytes of state and 32 of A are under way together.
// WHOLE: all of these hold, S = 4 LN and no pair spans two groups.
template <typename E, int LN, bool WHOLE>
__global__ void __launch_bounds__(kThreads)
    scan_step_kernel(const __grid_constant__ ScanStepArgs a) {
  const bool vec_h = WHOLE || a.vec_h, vec_A = WHOLE || a.vec_A, vec_ch = WHOLE || a.vec_ch,
             vec_bc = WHOLE || a.vec_bc;
  // a block stays within one row, whose addresses are then the same for all its lanes
  const int row = blockIdx.x, pairs = (a.D + 1) / 2;
  const int at = ((int)blockIdx.y * kThreads + (int)threadIdx.x) / LN;
  const int q = threadIdx.x % LN, n0 = q * 4;
  const bool live = at < pairs;
  const int d = live ? at * 2 : 0;
  // surplus lanes of a whole launch read channel 0 and store nothing
  const int have = WHOLE ? 2 : !live ? 0 : d + 1 < a.D ? 2 : 1;
  const int64_t slot = a.slots ? a.slots[row] : row;
  const bool has = live && slot >= 0 && slot < a.pool;
  const bool fresh = a.fresh && a.fresh[row];
  const int R = a.G == 1 ? a.D : a.D / a.G, g0 = a.G == 1 ? 0 : d / R;
  const int g1 = !WHOLE && have == 2 && a.G > 1 ? (d + 1) / R : g0;
  float* hp = a.h + ((has ? slot : 0) * a.D + d) * a.S + n0;
  // states of this lane
  const int own = WHOLE ? 4 : n0 < a.S ? (a.S - n0 < 4 ? a.S - n0 : 4) : 0;
  float4 h[2], A[2];
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    const int k = c < have ? own : 0;
    h[c] = load_quad<float>(hp + c * a.S, vec_h, has && !fresh ? k : 0);
    A[c] = load_quad<float>(a.A + (int64_t)(d + c) * a.S + n0, vec_A, k);
  }
  const E* Bm = static_cast<const E*>(a.Bm) + row * a.bs.batch + n0;
  const E* Cm = static_cast<const E*>(a.Cm) + row * a.cs.batch + n0;
  const int kb = WHOLE || live ? own : 0;
  const float4 B0 = widen(load_quad<E>(Bm + g0 * a.bs.head, vec_bc, kb));
  const float4 C0 = widen(load_quad<E>(Cm + g0 * a.cs.head, vec_bc, kb));
  const float4 B1 = g1 == g0 ? B0 : widen(load_quad<E>(Bm + g1 * a.bs.head, vec_bc, kb));
  const float4 C1 = g1 == g0 ? C0 : widen(load_quad<E>(Cm + g1 * a.cs.head, vec_bc, kb));
  auto pair_of = [&](const void* p, int64_t stride) {
    return widen(load_pair<E>(static_cast<const E*>(p) + row * stride + d, vec_ch, have));
  };
  const float2 u = pair_of(a.u, a.u_stride);
  float2 s = pair_of(a.delta, a.delta_stride), z = make_float2(0.f, 0.f);
  if (a.z) z = pair_of(a.z, a.z_stride);
  if (a.delta_bias) {
    if (have > 0) s.x += a.delta_bias[d];
    if (have > 1) s.y += a.delta_bias[d + 1];
  }
  if (a.softplus) s = softplus2(s);
  float o[2];
  const f32x2 lift = pack2(kDecayLift, kDecayLift);
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    const float sc = c ? s.y : s.x, v = sc * (c ? u.y : u.x), s2 = sc * kLog2e;
    const float4 B = c ? B1 : B0, Ct = c ? C1 : C0;
    // one test for four rates, behind the loads (a call at the size above: 54 us, 60 with
    // each rate held finite by itself, 58 with no test at all)
    if (fmaxf(fmaxf(fabsf(A[c].x), fabsf(A[c].y)), fmaxf(fabsf(A[c].z), fabsf(A[c].w))) > kLargest)
      A[c] = make_float4(finite_rate(A[c].x), finite_rate(A[c].y), finite_rate(A[c].z),
                         finite_rate(A[c].w));
    const float2 d0 = decay2(pack2(s2, s2), pack2(A[c].x, A[c].y), lift);
    const float2 d1 = decay2(pack2(s2, s2), pack2(A[c].z, A[c].w), lift);
    h[c].x = fmaf(d0.x, h[c].x, v * B.x);
    h[c].y = fmaf(d0.y, h[c].y, v * B.y);
    h[c].z = fmaf(d1.x, h[c].z, v * B.z);
    h[c].w = fmaf(d1.y, h[c].w, v * B.w);
    o[c] = fmaf(Ct.w, h[c].w, fmaf(Ct.z, h[c].z, fmaf(Ct.y, h[c].y, Ct.x * h[c].x)));
    if (has && c < have) {
      float* to = hp + c * a.S;
      if (vec_h) {
        if (own > 0) *reinterpret_cast<float4*>(to) = h[c];
      } else {
        const float f[4] = {h[c].x, h[c].y, h[c].z, h[c].w};
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (i < own) to[i] = f[i];
      }
    }
  }
#pragma unroll
  for (int k = LN / 2; k > 0; k >>= 1) {
    o[0] += __shfl_xor_sync(0xffffffffu, o[0], k);
    o[1] += __shfl_xor_sync(0xffffffffu, o[1], k);
  }
  if (q == 0 && live) {
    if (a.Dskip) {
      if (have > 0) o[0] = fmaf(a.Dskip[d], u.x, o[0]);
      if (have > 1) o[1] = fmaf(a.Dskip[d + 1], u.y, o[1]);
    }
    if (a.z) o[0] *= z.x * sigmoid(z.x), o[1] *= z.y * sigmoid(z.y);
    store_pair<E>(static_cast<E*>(a.y) + (int64_t)row * a.D + d, vec_ch, have,
                  has ? make_float2(o[0], o[1]) : make_float2(0.f, 0.f));
  }
}

template <typename E, int LN>
cudaError_t step_lanes(const ScanStepArgs& a, cudaStream_t stream) {
  const int64_t blocks = ((int64_t)((a.D + 1) / 2) * LN + kThreads - 1) / kThreads;
  if (blocks > 65535) return cudaErrorInvalidValue;
  const dim3 grid((unsigned)a.N, (unsigned)blocks);
  const bool whole = a.vec_h && a.vec_A && a.vec_ch && a.vec_bc && a.S == 4 * LN &&
                     a.D / a.G % 2 == 0;
  if (whole)
    scan_step_kernel<E, LN, true><<<grid, kThreads, 0, stream>>>(a);
  else
    scan_step_kernel<E, LN, false><<<grid, kThreads, 0, stream>>>(a);
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

cudaError_t launch_scan_step(const ScanStepArgs& in, cudaStream_t stream) {
  ScanStepArgs a = in;
  const int esz = a.dtype == FALCON_BF16 ? 2 : 4;
  auto on = [](const void* p, int bytes) { return reinterpret_cast<uintptr_t>(p) % bytes == 0; };
  a.vec_h = a.S % 4 == 0 && on(a.h, 16);
  a.vec_A = a.S % 4 == 0 && on(a.A, 16);
  a.vec_ch = a.D % 2 == 0 && a.u_stride % 2 == 0 && a.delta_stride % 2 == 0 &&
             (!a.z || a.z_stride % 2 == 0) && on(a.u, 2 * esz) && on(a.delta, 2 * esz) &&
             on(a.z, 2 * esz) && on(a.y, 2 * esz);
  a.vec_bc = a.S % 4 == 0 && on(a.Bm, 4 * esz) && on(a.Cm, 4 * esz) && a.bs.batch % 4 == 0 &&
             a.cs.batch % 4 == 0 && a.bs.head % 4 == 0 && a.cs.head % 4 == 0;
  return a.dtype == FALCON_BF16 ? step_typed<__nv_bfloat16>(a, stream)
                                : step_typed<float>(a, stream);
}

}  // namespace falcon
