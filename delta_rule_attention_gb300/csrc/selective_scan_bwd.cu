// Gradient of the selective scan.  With a_t = exp(s_t A), g_t the adjoint of h_t:
//   g_t = C_t dy_t + a_{t+1} g_{t+1},   w_t = g_t a_t h_{t-1}
//   dC_t = sum_d dy_t h_t,  dB_t = sum_d g_t s_t u_t,  dA = sum_t w_t s_t,
//   du_t = s_t <g_t, B_t> + Dskip dy_t,  ds_t = <w_t, A> + <g_t, B_t> u_t.
// A forward sweep keeps the state entering every tile of kTile tokens; the
// reverse sweep recomputes a tile's states in registers and walks it back.
// dB and dC sum over the channels of a block in shared memory, and over blocks
// (and rows, for dA, dDskip and ddelta_bias) in a second launch, in a fixed order.

#include <type_traits>

#include "ssm.cuh"

namespace falcon {
namespace {

constexpr int kWarps = 4;
constexpr int kTile = 8;

int lanes_of(int N) {
  int ln = 1;
  while (ln * 4 < N) ln *= 2;
  return ln;
}

// Parts of the workspace, in floats.
struct Layout {
  int64_t tiles, parts, N4;
  size_t ckpt, dbc, dA, dD, dbias, total;
  Layout(int64_t B, int64_t T, int D, int G, int N) {
    const int ln = lanes_of(N), per = 32 / ln * kWarps;
    N4 = 4 * ln;
    tiles = (T + kTile - 1) / kTile;
    parts = (D / G + per - 1) / per;
    ckpt = 0;
    dbc = ckpt + (size_t)(B * tiles * D * N4);
    dA = dbc + (size_t)(parts * B * T * G * 2 * N4);
    dD = dA + (size_t)(B * D * N4);
    dbias = dD + (size_t)(B * D);
    total = dbias + (size_t)(B * D);
  }
};

template <typename E, int LN>
__global__ void __launch_bounds__(kWarps * 32) scan_bwd_kernel(ScanArgs a, float* ws, Layout l) {
  constexpr int kCh = 32 / LN, N4 = 4 * LN;
  __shared__ float bc[kWarps][kTile][2][N4];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int q = lane % LN, n0 = q * 4;
  const int R = a.D / a.G;
  const int g = blockIdx.x / (int)l.parts, part = blockIdx.x - g * (int)l.parts;
  const int r = (part * kWarps + warp) * kCh + lane / LN;
  const bool live = r < R;
  const int d = g * R + (live ? r : 0);
  const int64_t b = blockIdx.y;
  const int64_t n = row_length(a.lengths, b, a.T);

  float A2[4], h[4], dA[4] = {0.f, 0.f, 0.f, 0.f}, gc[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const bool in = n0 + i < a.N;
    const int64_t k = (b * a.D + d) * a.N + n0 + i;
    A2[i] = in ? a.A[(int64_t)d * a.N + n0 + i] * kLog2e : 0.f;
    h[i] = in && a.h0 ? a.h0[k] : 0.f;
    gc[i] = in && a.dh_T ? a.dh_T[k] : 0.f;
  }
  const float bias = a.delta_bias ? a.delta_bias[d] : 0.f;
  const float skip = a.Dskip ? a.Dskip[d] : 0.f;
  const E* u = static_cast<const E*>(a.u) + b * a.us.batch + d;
  const E* dl = static_cast<const E*>(a.delta) + b * a.ds.batch + d;
  const E* z = a.z ? static_cast<const E*>(a.z) + b * a.zs.batch + d : nullptr;
  const E* dy = static_cast<const E*>(a.dy) + b * a.dys.batch + d;
  const E* Bm = static_cast<const E*>(a.Bm) + b * a.bs.batch + g * a.bs.head + n0;
  const E* Cm = static_cast<const E*>(a.Cm) + b * a.cs.batch + g * a.cs.head + n0;
  E* du = static_cast<E*>(a.du) + b * a.T * a.D + d;
  E* dd = static_cast<E*>(a.ddelta) + b * a.T * a.D + d;
  E* dz = a.z ? static_cast<E*>(a.dz) + b * a.T * a.D + d : nullptr;
  auto bc_at = [&](const E* p, int64_t stride, int64_t t, int i) {
    return n0 + i < a.N ? load_vec<E, 1>(p + t * stride + i).v[0] : 0.f;
  };
  float* ck = ws + l.ckpt + (b * l.tiles * a.D + d) * N4 + n0;

  for (int64_t t = 0; t < n; ++t) {
    if (t % kTile == 0 && live)
      *reinterpret_cast<float4*>(ck + t / kTile * a.D * N4) = make_float4(h[0], h[1], h[2], h[3]);
    const float ut = load_vec<E, 1>(u + t * a.us.time).v[0];
    float s = load_vec<E, 1>(dl + t * a.ds.time).v[0] + bias;
    if (a.softplus) s = softplus(s);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      h[i] = fmaf(decay(s, A2[i]), h[i], s * ut * bc_at(Bm, a.bs.time, t, i));
  }

  float dD = 0.f, dbias = 0.f;
  for (int64_t tile = l.tiles - 1; tile >= 0; --tile) {
    const int64_t t0 = tile * kTile;
    const float4 c0 = live && t0 < n ? *reinterpret_cast<const float4*>(ck + tile * a.D * N4)
                                     : make_float4(0.f, 0.f, 0.f, 0.f);
    float hs[kTile + 1][4] = {{c0.x, c0.y, c0.z, c0.w}};
    float s[kTile], raw[kTile], ut[kTile];
#pragma unroll
    for (int k = 0; k < kTile; ++k) {
      const int64_t t = t0 + k;
      s[k] = ut[k] = raw[k] = 0.f;
      if (t < n) {
        ut[k] = load_vec<E, 1>(u + t * a.us.time).v[0];
        raw[k] = load_vec<E, 1>(dl + t * a.ds.time).v[0] + bias;
        s[k] = a.softplus ? softplus(raw[k]) : raw[k];
      }
#pragma unroll
      for (int i = 0; i < 4; ++i)
        hs[k + 1][i] = fmaf(decay(s[k], A2[i]), hs[k][i],
                            t < n ? s[k] * ut[k] * bc_at(Bm, a.bs.time, t, i) : 0.f);
    }
#pragma unroll
    for (int k = kTile - 1; k >= 0; --k) {
      const int64_t t = t0 + k;
      float s1 = 0.f, s2 = 0.f, yo = 0.f, vB[4], vC[4];
      float dyt = 0.f, zt = 0.f;
      if (t < n) {
        dyt = load_vec<E, 1>(dy + t * a.dys.time).v[0];
        zt = z ? load_vec<E, 1>(z + t * a.zs.time).v[0] : 0.f;
      }
      const float sg = sigmoid(zt), dyg = z ? dyt * zt * sg : dyt;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float Bt = t < n ? bc_at(Bm, a.bs.time, t, i) : 0.f;
        const float Ct = t < n ? bc_at(Cm, a.cs.time, t, i) : 0.f;
        yo = fmaf(Ct, hs[k + 1][i], yo);
        vC[i] = live ? dyg * hs[k + 1][i] : 0.f;
        const float gt = fmaf(dyg, Ct, gc[i]);
        s1 = fmaf(gt, Bt, s1);
        vB[i] = live ? gt * s[k] * ut[k] : 0.f;
        gc[i] = gt * decay(s[k], A2[i]);
        const float w = gc[i] * hs[k][i];
        dA[i] = fmaf(w, s[k], dA[i]);
        s2 = fmaf(w, A2[i], s2);
      }
#pragma unroll
      for (int x = LN / 2; x > 0; x >>= 1) {
        s1 += __shfl_xor_sync(0xffffffffu, s1, x);
        s2 += __shfl_xor_sync(0xffffffffu, s2, x);
        yo += __shfl_xor_sync(0xffffffffu, yo, x);
      }
#pragma unroll
      for (int x = 16; x >= LN; x >>= 1)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          vB[i] += __shfl_xor_sync(0xffffffffu, vB[i], x);
          vC[i] += __shfl_xor_sync(0xffffffffu, vC[i], x);
        }
      if (lane < LN)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          bc[warp][k][0][n0 + i] = vB[i];
          bc[warp][k][1][n0 + i] = vC[i];
        }
      if (live && q == 0 && t < a.T) {
        const float ds = fmaf(s1, ut[k], s2 * kLn2);
        const float dr = a.softplus ? (t < n ? ds * sigmoid(raw[k]) : 0.f) : (t < n ? ds : 0.f);
        store_vec<E, 1>(du + t * a.D, FloatV<1>{{t < n ? fmaf(s1, s[k], skip * dyg) : 0.f}});
        store_vec<E, 1>(dd + t * a.D, FloatV<1>{{dr}});
        if (z)
          store_vec<E, 1>(dz + t * a.D,
                          FloatV<1>{{t < n ? dyt * fmaf(skip, ut[k], yo) * sg *
                                                 fmaf(zt, 1.f - sg, 1.f)
                                           : 0.f}});
        dD = fmaf(dyg, ut[k], dD);
        dbias += dr;
      }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < kTile * 2 * N4; i += kWarps * 32) {
      const int64_t t = t0 + i / (2 * N4);
      float v = 0.f;
      for (int x = 0; x < kWarps; ++x) v += (&bc[x][0][0][0])[i];
      if (t < a.T)
        ws[l.dbc + (((part * a.B + b) * a.T + t) * a.G + g) * 2 * N4 + i % (2 * N4)] = v;
    }
    __syncthreads();
  }
  if (!live) return;
  *reinterpret_cast<float4*>(ws + l.dA + (b * a.D + d) * N4 + n0) =
      make_float4(dA[0], dA[1], dA[2], dA[3]);
  if (a.dh0)
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (n0 + i < a.N) a.dh0[(b * a.D + d) * a.N + n0 + i] = gc[i];
  if (q == 0) {
    ws[l.dD + b * a.D + d] = dD;
    ws[l.dbias + b * a.D + d] = dbias;
  }
}

template <typename E>
__global__ void scan_bwd_bc_kernel(ScanArgs a, const float* ws, Layout l) {
  const int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  const int64_t rows = a.B * a.T * a.G;
  if (i >= rows * 2 * l.N4) return;
  const int64_t row = i / (2 * l.N4), k = i - row * 2 * l.N4;
  const int64_t n = k % l.N4;
  if (n >= a.N) return;
  float v = 0.f;
  for (int64_t p = 0; p < l.parts; ++p) v += ws[l.dbc + p * rows * 2 * l.N4 + i];
  store_vec<E, 1>(static_cast<E*>(k < l.N4 ? a.dB : a.dC) + row * a.N + n, FloatV<1>{{v}});
}

__global__ void scan_bwd_param_kernel(ScanArgs a, const float* ws, Layout l) {
  const int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  if (i < (int64_t)a.D * a.N) {
    const int64_t d = i / a.N, n = i - d * a.N;
    float v = 0.f;
    for (int64_t b = 0; b < a.B; ++b) v += ws[l.dA + (b * a.D + d) * l.N4 + n];
    a.dA[i] = v;
  }
  if (i < a.D) {
    float v = 0.f, w = 0.f;
    for (int64_t b = 0; b < a.B; ++b) {
      v += ws[l.dD + b * a.D + i];
      w += ws[l.dbias + b * a.D + i];
    }
    if (a.dDskip) a.dDskip[i] = v;
    if (a.ddelta_bias) a.ddelta_bias[i] = w;
  }
}

template <typename E, int LN>
cudaError_t bwd_lanes(const ScanArgs& a, cudaStream_t stream) {
  const Layout l(a.B, a.T, a.D, a.G, a.N);
  float* ws = static_cast<float*>(a.ws);
  scan_bwd_kernel<E, LN>
      <<<dim3((unsigned)(a.G * l.parts), (unsigned)a.B), kWarps * 32, 0, stream>>>(a, ws, l);
  cudaError_t e = cudaGetLastError();
  const int64_t bc = a.B * a.T * a.G * 2 * l.N4, pa = (int64_t)a.D * a.N;
  if (e == cudaSuccess && bc > 0) {
    scan_bwd_bc_kernel<E><<<(unsigned)((bc + 255) / 256), 256, 0, stream>>>(a, ws, l);
    e = cudaGetLastError();
  }
  if (e != cudaSuccess) return e;
  scan_bwd_param_kernel<<<(unsigned)((pa + 127) / 128), 128, 0, stream>>>(a, ws, l);
  return cudaGetLastError();
}

template <typename E>
cudaError_t bwd_typed(const ScanArgs& a, cudaStream_t stream) {
  switch (lanes_of(a.N)) {
    case 1: return bwd_lanes<E, 1>(a, stream);
    case 2: return bwd_lanes<E, 2>(a, stream);
    case 4: return bwd_lanes<E, 4>(a, stream);
    case 8: return bwd_lanes<E, 8>(a, stream);
    case 16: return bwd_lanes<E, 16>(a, stream);
    case 32: return bwd_lanes<E, 32>(a, stream);
  }
  return cudaErrorInvalidValue;
}

}  // namespace

size_t scan_bwd_workspace_bytes(const falcon_scan_shape& s) {
  return sizeof(float) * Layout(s.B, s.T, s.D, s.G, s.N).total;
}

cudaError_t launch_scan_bwd(const ScanArgs& a, cudaStream_t stream) {
  return a.dtype == FALCON_BF16 ? bwd_typed<__nv_bfloat16>(a, stream)
                                : bwd_typed<float>(a, stream);
}

}  // namespace falcon
