// Shared by the kernels of the selective state space block: argument blocks,
// vector loads of bf16 or fp32 rows, softplus and silu in fp32.
#pragma once

#include <atomic>

#include "common.cuh"

namespace falcon {

int check_sm103_device();  // FALCON_OK on an sm_103 device (api.cu)

template <int V>
struct FloatV {
  float v[V];
};

// V consecutive elements (V * sizeof(element) bytes, aligned to that size).
template <typename E, int V>
__device__ __forceinline__ FloatV<V> load_vec(const E* p) {
  FloatV<V> r;
  if constexpr (sizeof(E) == 4) {
    if constexpr (V == 1) {
      r.v[0] = *p;
    } else if constexpr (V == 2) {
      const float2 q = *reinterpret_cast<const float2*>(p);
      r.v[0] = q.x, r.v[1] = q.y;
    } else {
      static_assert(V == 4, "fp32 rows move 1, 2 or 4 channels");
      const float4 q = *reinterpret_cast<const float4*>(p);
      r.v[0] = q.x, r.v[1] = q.y, r.v[2] = q.z, r.v[3] = q.w;
    }
  } else {
    if constexpr (V == 1) {
      r.v[0] = __bfloat162float(*p);
    } else {
      uint32_t w[V / 2];
      if constexpr (V == 2) {
        w[0] = *reinterpret_cast<const uint32_t*>(p);
      } else if constexpr (V == 4) {
        const uint2 q = *reinterpret_cast<const uint2*>(p);
        w[0] = q.x, w[1] = q.y;
      } else {
        static_assert(V == 8, "bf16 rows move 1, 2, 4 or 8 channels");
        const uint4 q = *reinterpret_cast<const uint4*>(p);
        w[0] = q.x, w[1] = q.y, w[2] = q.z, w[3] = q.w;
      }
#pragma unroll
      for (int i = 0; i < V / 2; ++i) {
        r.v[2 * i] = __uint_as_float(w[i] << 16);
        r.v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
      }
    }
  }
  return r;
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 q = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&q);
}

template <typename E, int V>
__device__ __forceinline__ void store_vec(E* p, const FloatV<V>& x) {
  if constexpr (sizeof(E) == 4) {
    if constexpr (V == 1)
      *p = x.v[0];
    else if constexpr (V == 2)
      *reinterpret_cast<float2*>(p) = make_float2(x.v[0], x.v[1]);
    else
      *reinterpret_cast<float4*>(p) = make_float4(x.v[0], x.v[1], x.v[2], x.v[3]);
  } else {
    if constexpr (V == 1)
      *p = __float2bfloat16_rn(x.v[0]);
    else if constexpr (V == 2)
      *reinterpret_cast<uint32_t*>(p) = pack_bf16(x.v[0], x.v[1]);
    else if constexpr (V == 4)
      *reinterpret_cast<uint2*>(p) =
          make_uint2(pack_bf16(x.v[0], x.v[1]), pack_bf16(x.v[2], x.v[3]));
    else
      *reinterpret_cast<uint4*>(p) =
          make_uint4(pack_bf16(x.v[0], x.v[1]), pack_bf16(x.v[2], x.v[3]),
                     pack_bf16(x.v[4], x.v[5]), pack_bf16(x.v[6], x.v[7]));
  }
}

__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// A held finite (an infinite one as the largest number, a NaN as it is), so that a step
// of zero leaves the state: exp(0 A) = 1.
constexpr float kLargest = 3.402823466e38f;
__device__ __forceinline__ float finite_rate(float A) {
  return fabsf(A) > kLargest ? copysignf(kLargest, A) : A;
}
// In units of log2(e), where a rate above 2.36e38 would overflow.
__device__ __forceinline__ float rate_log2(float A) { return finite_rate(A * kLog2e); }

// exp(s A), A2 = rate_log2(A).  ex2.approx comes out low by 2e-8 to 5e-8 of its
// value on average, which a state with a long memory adds up; the constant in
// the exponent's fma cancels the mean at no cost (relative error of a state
// after 2048 tokens with steps of 0.001 .. 0.1 and A of -1 .. -16: 2.3e-7, against
// 4.9e-7 without it and 3.2e-7 with expf).
constexpr float kDecayLift = 2.2e-8f;
__device__ __forceinline__ float decay(float s, float A2) {
  return exp2_approx(fmaf(s, A2, kDecayLift));
}

// 1 / (1 + e^{-x}).  Where the denominator is above 2^126, or infinite, the reciprocal
// is flushed to zero: x sigmoid(x) is then zero for every finite x, where a value held
// above zero would grow with x (-4 for the lowest float32).
__device__ __forceinline__ float sigmoid(float x) {
  return rcp_approx(1.f + exp2_approx(-x * kLog2e));
}

// softplus(x) = max(x, 0) + log1p(e), e = e^{-|x|} in (0, 1].
// log1p(e) = 2 atanh(w), w = e / (2 + e) in (0, 1/3]: w times a polynomial of
// degree 4 in w^2, fitted to 2 atanh(w) / w at Chebyshev nodes of [0, 1/9] (off by
// less than 8e-9 of it there).  The result keeps its relative precision where it is
// small, which a logarithm of 1 + e would not.
constexpr float kAtanh0 = 2.0000000078777487f, kAtanh1 = 0.6666631593508076f,
                kAtanh2 = 0.40024853723465403f, kAtanh3 = 0.2796141883493225f,
                kAtanh4 = 0.28174657262265285f;
__device__ __forceinline__ float softplus(float x) {
  const float e = exp2_approx(-fabsf(x) * kLog2e);
  const float w = e * rcp_approx(2.f + e);
  const float q = w * w;
  const float p =
      fmaf(fmaf(fmaf(fmaf(kAtanh4, q, kAtanh3), q, kAtanh2), q, kAtanh1), q, kAtanh0);
  return fmaf(w, p, fmaxf(x, 0.f));
}

// Two floats in one 64-bit register pair: one instruction for two lanes' worth.
typedef unsigned long long f32x2;
__device__ __forceinline__ f32x2 pack2(float lo, float hi) {
  f32x2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ float2 unpack2(f32x2 v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b) {
  f32x2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
  f32x2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ f32x2 add2(f32x2 a, f32x2 b) {
  f32x2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f32x2 pair2(float2 v) { return pack2(v.x, v.y); }
// The same pair, its halves unknown to the compiler: a doubled value stays in its
// two registers instead of being copied together before every use.
__device__ __forceinline__ f32x2 opaque2(f32x2 v) {
  asm volatile("" : "+l"(v));
  return v;
}
// decay() twice: two steps of one state, or one step of two.
__device__ __forceinline__ float2 decay2(f32x2 s, f32x2 A2, f32x2 lift) {
  const float2 x = unpack2(fma2(s, A2, lift));
  return make_float2(exp2_approx(x.x), exp2_approx(x.y));
}
// softplus() twice.
__device__ __forceinline__ float2 softplus2(float2 x) {
  const float2 e =
      make_float2(exp2_approx(-fabsf(x.x) * kLog2e), exp2_approx(-fabsf(x.y) * kLog2e));
  const float2 den = unpack2(add2(pair2(e), pack2(2.f, 2.f)));
  const f32x2 w = mul2(pair2(e), pack2(rcp_approx(den.x), rcp_approx(den.y)));
  const f32x2 q = mul2(w, w);
  f32x2 p = fma2(pack2(kAtanh4, kAtanh4), q, pack2(kAtanh3, kAtanh3));
  p = fma2(p, q, pack2(kAtanh2, kAtanh2));
  p = fma2(p, q, pack2(kAtanh1, kAtanh1));
  p = fma2(p, q, pack2(kAtanh0, kAtanh0));
  return unpack2(fma2(w, p, pack2(fmaxf(x.x, 0.f), fmaxf(x.y, 0.f))));
}

// 1, 2 or 4 neighbouring elements as they lie in memory.
template <typename E>
struct Raw;
template <>
struct Raw<__nv_bfloat16> {
  typedef uint32_t Pair;
  typedef uint2 Quad;
};
template <>
struct Raw<float> {
  typedef float2 Pair;
  typedef float4 Quad;
};
__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
__device__ __forceinline__ float2 widen(uint32_t w) { return make_float2(bf16_lo(w), bf16_hi(w)); }
__device__ __forceinline__ float2 widen(float2 w) { return w; }
__device__ __forceinline__ float4 widen(uint2 w) {
  return make_float4(bf16_lo(w.x), bf16_hi(w.x), bf16_lo(w.y), bf16_hi(w.y));
}
__device__ __forceinline__ float4 widen(float4 w) { return w; }
__device__ __forceinline__ uint32_t narrow(float2 v, uint32_t) { return pack_bf16(v.x, v.y); }
__device__ __forceinline__ float2 narrow(float2 v, float2) { return v; }
__device__ __forceinline__ uint2 narrow(float4 v, uint2) {
  return make_uint2(pack_bf16(v.x, v.y), pack_bf16(v.z, v.w));
}
__device__ __forceinline__ float4 narrow(float4 v, float4) { return v; }

// Elements `have` of a pair or quad at p (vec: in one access); the others are zero.
template <typename E>
__device__ __forceinline__ typename Raw<E>::Pair load_pair(const E* p, bool vec, int have) {
  typedef typename Raw<E>::Pair P;
  if (vec && have > 0) return *reinterpret_cast<const P*>(p);
  return narrow(make_float2(have > 0 ? load_vec<E, 1>(p).v[0] : 0.f,
                            have > 1 ? load_vec<E, 1>(p + 1).v[0] : 0.f),
                P());
}
template <typename E>
__device__ __forceinline__ typename Raw<E>::Quad load_quad(const E* p, bool vec, int have) {
  typedef typename Raw<E>::Quad Q;
  if (vec && have > 0) return *reinterpret_cast<const Q*>(p);
  float v[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = have > i ? load_vec<E, 1>(p + i).v[0] : 0.f;
  return narrow(make_float4(v[0], v[1], v[2], v[3]), Q());
}
template <typename E>
__device__ __forceinline__ void store_pair(E* p, bool vec, int have, float2 v) {
  typedef typename Raw<E>::Pair P;
  if (vec && have > 0) {
    *reinterpret_cast<P*>(p) = narrow(v, P());
    return;
  }
  if (have > 0) store_vec<E, 1>(p, FloatV<1>{{v.x}});
  if (have > 1) store_vec<E, 1>(p + 1, FloatV<1>{{v.y}});
}

// acc + a * b and a * b of V values, two to an instruction.
template <int V>
__device__ __forceinline__ FloatV<V> fma_vec(const FloatV<V>& a, const FloatV<V>& b,
                                             const FloatV<V>& acc) {
  FloatV<V> r;
  if constexpr (V % 2 == 0) {
#pragma unroll
    for (int i = 0; i < V; i += 2) {
      const float2 v = unpack2(fma2(pack2(a.v[i], a.v[i + 1]), pack2(b.v[i], b.v[i + 1]),
                                    pack2(acc.v[i], acc.v[i + 1])));
      r.v[i] = v.x, r.v[i + 1] = v.y;
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) r.v[i] = fmaf(a.v[i], b.v[i], acc.v[i]);
  }
  return r;
}
template <int V>
__device__ __forceinline__ FloatV<V> mul_vec(const FloatV<V>& a, const FloatV<V>& b) {
  FloatV<V> r;
  if constexpr (V % 2 == 0) {
#pragma unroll
    for (int i = 0; i < V; i += 2) {
      const float2 v = unpack2(mul2(pack2(a.v[i], a.v[i + 1]), pack2(b.v[i], b.v[i + 1])));
      r.v[i] = v.x, r.v[i + 1] = v.y;
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) r.v[i] = a.v[i] * b.v[i];
  }
  return r;
}
template <int V>
__device__ __forceinline__ FloatV<V> add_vec(const FloatV<V>& a, const FloatV<V>& b) {
  FloatV<V> r;
  if constexpr (V % 2 == 0) {
#pragma unroll
    for (int i = 0; i < V; i += 2) {
      const float2 v = unpack2(add2(pack2(a.v[i], a.v[i + 1]), pack2(b.v[i], b.v[i + 1])));
      r.v[i] = v.x, r.v[i + 1] = v.y;
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) r.v[i] = a.v[i] + b.v[i];
  }
  return r;
}

struct ConvArgs {
  int64_t B, H, T;
  int m, width, dtype, act;
  int64_t C;  // H * m
  falcon_strides xs, ys, dys, dxs;
  const void *x, *state, *dy, *dstate_out;
  const float *weight, *bias;
  const int32_t* lengths;
  void *y, *state_out, *dx, *dstate;
  float *dweight, *dbias;
  float* ws;
  bool vec_w;  // weight is 16-byte aligned
};
cudaError_t launch_conv_fwd(const ConvArgs& a, cudaStream_t stream);
size_t conv_bwd_workspace_bytes(int64_t B, int64_t T, int64_t C, int width);
cudaError_t launch_conv_bwd(const ConvArgs& a, cudaStream_t stream);

struct ConvStepArgs {
  int64_t N, pool, x_stride;
  int C, width, dtype, act;
  const void* x;
  const float *weight, *bias;
  void* state;
  const int32_t* slots;
  const uint8_t* fresh;
  void* y;
  bool vec_w;
};
cudaError_t launch_conv_step(const ConvStepArgs& a, cudaStream_t stream);

struct ScanArgs {
  int64_t B, T;
  int D, G, N, dtype, softplus;
  falcon_strides us, ds, bs, cs, zs, ys, dys;
  const void *u, *delta, *Bm, *Cm, *z, *dy;
  const float *A, *Dskip, *delta_bias, *h0, *dh_T;
  const int32_t* lengths;
  void *y, *du, *ddelta, *dB, *dC, *dz;
  float *h_out, *dA, *dDskip, *ddelta_bias, *dh0;
  void* ws;
  // every channel pair of u, delta, z (dy) and the outputs, and every quad of
  // states of Bm and Cm, is one aligned access
  bool vec_ch, vec_bc;
  // both, and the offsets inside a tile of 32 tokens fit 31 bits
  bool fast;
};
// Fills vec_ch, vec_bc and fast (outputs besides y are dense).
void scan_access(ScanArgs* a);
cudaError_t launch_scan_fwd(const ScanArgs& a, cudaStream_t stream);
size_t scan_bwd_workspace_bytes(const falcon_scan_shape& s);
cudaError_t launch_scan_bwd(const ScanArgs& a, cudaStream_t stream);

struct ScanStepArgs {
  int64_t N, pool, u_stride, delta_stride, z_stride;
  int D, G, S, dtype, softplus;
  falcon_strides bs, cs;
  const void *u, *delta, *Bm, *Cm, *z;
  const float *A, *Dskip, *delta_bias;
  float* h;
  const int32_t* slots;
  const uint8_t* fresh;
  void* y;
  bool vec_h, vec_A, vec_ch, vec_bc;  // aligned quads and pairs
};
cudaError_t launch_scan_step(const ScanStepArgs& a, cudaStream_t stream);

size_t clip_workspace_bytes(const falcon_grad* grads, int64_t tensors);
cudaError_t launch_clip(const falcon_grad* grads, int64_t tensors, float max_norm, float eps,
                        float* norm, void* ws, cudaStream_t stream);

// Lets `kernel` use `bytes` of dynamic shared memory on the current device; asked
// once for each kernel (one `done` each) and device.
template <typename K>
inline cudaError_t allow_shared(K kernel, int bytes, std::atomic<uint64_t>* done) {
  if (bytes <= 48 * 1024) return cudaSuccess;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev >= 0 && dev < 64 ? 1ull << dev : 0;
  if (bit && (done->load(std::memory_order_relaxed) & bit)) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) done->fetch_or(bit, std::memory_order_relaxed);
  return e;
}

// Row length of batch entry b.
__device__ __forceinline__ int64_t row_length(const int32_t* lengths, int64_t b, int64_t T) {
  if (!lengths) return T;
  const int64_t n = lengths[b];
  return n < 0 ? 0 : (n < T ? n : T);
}

}  // namespace falcon
