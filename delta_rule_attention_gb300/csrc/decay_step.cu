// One token of the attention with a decay for N sequences: S <- gamma S + k v^T,
// o = scale S^T q, the states in a pool.  Bound by the states' traffic, each read and
// written once in fp32.
//
// A block takes one (sequence, head) state.  A thread holds four neighbouring values of
// several rows: all its loads are under way before the first is used, the rank-one update
// and the read's partial sums run in registers, and the sums over the rows are joined
// through shared memory.  8192 states of 128 x 128: 161 us, 6.7 TB/s, 99% of a copy's rate;
// few states are bound by the launch (24 states of 64 x 64: 4.2 us in a graph).
#include "linear.cuh"

namespace falcon {
namespace {

constexpr int kMostThreads = 256;

template <typename E>
__global__ void __launch_bounds__(kMostThreads)
    decay_step_kernel(const __grid_constant__ DecayStepArgs a, int lanes, bool vec) {
  // lanes: threads along a row of the state, four values each
  __shared__ float q[128], k[128];
  __shared__ float4 part[kMostThreads];
  const int64_t row = blockIdx.x / a.H;
  const int h = blockIdx.x % a.H, tid = threadIdx.x, groups = blockDim.x / lanes;
  const int grp = tid / lanes, c = tid % lanes * 4;
  const int64_t slot = a.slots ? a.slots[row] : row;
  const bool has = slot >= 0 && slot < a.pool;
  const bool fresh = a.fresh && a.fresh[row];
  const int have = grp < groups ? a.dv - c : 0;
  float* S = a.S + ((has ? slot : 0) * a.H + h) * a.m * a.dv + c;
  const E* vp = static_cast<const E*>(a.v) + row * a.vs.batch + h * a.vs.head + c;
  float4 s[16];
#pragma unroll
  for (int r = 0; r < 16; ++r) {
    const int i = grp + r * groups;
    s[r] = load_quad<float>(S + (int64_t)i * a.dv, vec,
                            has && !fresh && i < a.m ? (have < 4 ? have : 4) : 0);
  }
  const E* qp = static_cast<const E*>(a.q) + row * a.qs.batch + h * a.qs.head;
  const E* kp = static_cast<const E*>(a.k) + row * a.ks.batch + h * a.ks.head;
  for (int i = tid; i < a.m; i += blockDim.x) {
    q[i] = load_vec<E, 1>(qp + i).v[0];
    k[i] = load_vec<E, 1>(kp + i).v[0];
  }
  const float4 v = widen(load_quad<E>(vp, false, have < 4 ? have : 4));
  // what a token loses is subtracted: gamma's own rounding would repeat itself token after
  // token (off by 2^-25 a step, 1e-4 of a slow head's state after 4096)
  const Carry carry(decay_rate(a.log_decay, h), 1.f);
  __syncthreads();
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
  for (int r = 0; r < 16; ++r) {
    const int i = grp + r * groups;
    if (i < a.m) {
      const float ki = k[i], qi = q[i];
      s[r].x = fmaf(ki, v.x, carry.of(s[r].x)), s[r].y = fmaf(ki, v.y, carry.of(s[r].y));
      s[r].z = fmaf(ki, v.z, carry.of(s[r].z)), s[r].w = fmaf(ki, v.w, carry.of(s[r].w));
      o.x = fmaf(qi, s[r].x, o.x), o.y = fmaf(qi, s[r].y, o.y);
      o.z = fmaf(qi, s[r].z, o.z), o.w = fmaf(qi, s[r].w, o.w);
      if (has) {
        float* to = S + (int64_t)i * a.dv;
        if (vec && have > 0) {
          *reinterpret_cast<float4*>(to) = s[r];
        } else {
          if (have > 0) to[0] = s[r].x;
          if (have > 1) to[1] = s[r].y;
          if (have > 2) to[2] = s[r].z;
          if (have > 3) to[3] = s[r].w;
        }
      }
    }
  }
  part[tid] = o;
  __syncthreads();
  if (grp == 0) {
    for (int p = 1; p < groups; ++p) {
      const float4 x = part[p * lanes + tid];
      o.x += x.x, o.y += x.y, o.z += x.z, o.w += x.w;
    }
    const float f = has ? a.scale : 0.f;
    E* to = static_cast<E*>(a.o) + (row * a.H + h) * a.dv + c;
    const float out[4] = {o.x, o.y, o.z, o.w};
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (j < have) store_vec<E, 1>(to + j, FloatV<1>{{has ? f * out[j] : 0.f}});
  }
}

}  // namespace

cudaError_t launch_decay_step(const DecayStepArgs& a, cudaStream_t stream) {
  const int lanes = (a.dv + 3) / 4;
  // a thread holds at most 16 rows
  int groups = (a.m + 15) / 16;
  while (groups * 2 * lanes <= kMostThreads && groups * 2 <= a.m) groups *= 2;
  const bool vec = a.dv % 4 == 0 && reinterpret_cast<uintptr_t>(a.S) % 16 == 0;
  const unsigned grid = (unsigned)(a.N * a.H);
  if (a.dtype == FALCON_BF16)
    decay_step_kernel<__nv_bfloat16><<<grid, lanes * groups, 0, stream>>>(a, lanes, vec);
  else
    decay_step_kernel<float><<<grid, lanes * groups, 0, stream>>>(a, lanes, vec);
  return cudaGetLastError();
}

}  // namespace falcon
