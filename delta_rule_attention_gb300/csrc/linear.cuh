// Shared by the kernels of the linear attention block: argument blocks of the attention
// with a decay and of the gated norm.
#pragma once

#include "ssm.cuh"

namespace falcon {

// One pass of the attention with a decay, over rows of T tokens with keys of m and
// values of dv channels.  Forward in time (rev = 0):
//   S_t = gamma S_{t-1} + w k_t v_t^T,  o_t = inter S_t^T q_t,  S_{-1} = S_init,
// S_out the state after the last token.  Backward in time (rev = 1):
//   S_t = gamma S_{t+1} + w k_t v_t^T,  o_t = inter S_t^T q_t,
// S_init added to S at the row's last token, S_out = gamma S_0.
// The gradient is three such passes: dq reads (dO, v, k) forward with the transposed
// state, dk (v, dO, q) and dv (k, q, dO) backward.
struct DecayPass {
  int64_t B, H, T;
  int m, dv, dtype, rev;
  falcon_strides qs, ks, vs, os;
  const void *q, *k, *v;
  void* o;
  const float* log_decay;
  const int32_t* lengths;
  const float* S_init;  // element (i, j) at i * si + j * sj (the other order: transposed)
  float* S_out;         // laid out the same; nullable
  int si, sj;
  float inter, w;
  // runs of tokens that are worked on by themselves: run_len tokens each (a multiple of
  // the chunk), and a state [m, dv] for each, [B*H, runs, m, dv]: what it adds, then the
  // state that enters it
  int64_t run_len;
  int runs;
  bool whole;  // CUDA cores: one run a row, from S_init to S_out in one launch
  float* states;
  // tensor-core passes: whether the states are formed (or taken as they are, key i and
  // value j of one at i * xi + j * xj), and whether the kernels that form and read them
  // may be set up while the kernel before them runs
  bool sums, behind_states, behind_reads;
  int xi, xj;
  bool vec_q, vec_k, vec_v, vec_o;  // quads of channels are one aligned access
};

// gamma^n; log_decay held at most 0 and finite.
__device__ __forceinline__ float decay_rate(const float* log_decay, int h) {
  const float g = log_decay[h];
  return g > 0.f ? 0.f : (g < -kLargest ? -kLargest : g);
}
__device__ __forceinline__ float decay_power(float g, float n) { return expf(g * n); }

// A state n tokens later.  Where gamma^n is near 1 its rounding would repeat itself run
// after run, so what is lost is subtracted (expm1); where it is small, that difference
// would cancel: off by 2^-25 of X where gamma^n X is left (exactly zero for gamma^n < 2^-25).
struct Carry {
  float f;
  bool near;
  __device__ __forceinline__ Carry(float g, float n) {
    const float x = g * n;
    near = !(x < -0.69314718f);
    f = near ? expm1f(x) : expf(x);
  }
  __device__ __forceinline__ float of(float X) const { return fmaf(f, X, near ? X : 0.f); }
};
// Those of a row's steps of `step` tokens each: n of them whole, then one of what is left.
struct Carries {
  Carry whole, rest;
  __device__ __forceinline__ Carries(float g, unsigned step, unsigned n)
      : whole(g, (float)step), rest(g, (float)(n % step)) {}
  __device__ __forceinline__ Carry after(int64_t tokens, int64_t step) const {
    return tokens == step ? whole : rest;
  }
};

// Tokens of run r of a row of n.
__device__ __forceinline__ int64_t run_tokens(int64_t n, int64_t r, int64_t run_len) {
  const int64_t left = n - r * run_len;
  return left < 0 ? 0 : (left < run_len ? left : run_len);
}

struct DecayCall {
  falcon_decay_shape s;
  falcon_strides qs, ks, vs, os, dqs, dks, dvs, dos;
  const void *q, *k, *v, *dO;
  const float *log_decay, *S0, *dS_T;
  const int32_t* lengths;
  void *o, *dq, *dk, *dv;
  float *S_out, *dS0;
  void* ws;
};
size_t decay_workspace_bytes(const falcon_decay_shape& s);
cudaError_t launch_decay_fwd(const DecayCall& c, cudaStream_t stream);
cudaError_t launch_decay_bwd(const DecayCall& c, cudaStream_t stream);

struct DecayStepArgs {
  int64_t N, pool;
  int H, m, dv, dtype;
  float scale;
  falcon_strides qs, ks, vs;
  const void *q, *k, *v;
  const float* log_decay;
  float* S;
  const int32_t* slots;
  const uint8_t* fresh;
  void* o;
};
cudaError_t launch_decay_step(const DecayStepArgs& a, cudaStream_t stream);

struct NormArgs {
  int64_t B, T;
  int H, m, D, dtype, gate;
  float eps;
  falcon_strides hs, zs, xs, os, ns;  // os: out, ns: next
  const void *h, *z, *x;
  const float *weight, *scale, *next_weight;
  const int32_t* lengths;
  void *out, *next;
  // the gradient
  falcon_strides dos, dns, dxs, dhs, dzs;
  const void *y, *dout, *dnext;  // y: the stored out
  void *dx, *dh, *dz;
  float *dweight, *dscale, *dnext_weight;
  float* ws;
  int parts;  // rows of per-channel sums in ws
};
size_t norm_bwd_workspace_bytes(const falcon_norm_shape& s);
cudaError_t launch_norm_fwd(const NormArgs& a, cudaStream_t stream);
cudaError_t launch_norm_bwd(const NormArgs& a, cudaStream_t stream);

}  // namespace falcon
