// Selective scan over prompts:
//   s_t = softplus(delta_t + bias),  h_t = exp(s_t A) h_{t-1} + s_t u_t B_t,
//   y_t = (<C_t, h_t> + Dskip u_t) silu(z_t)
// for every channel with its N states.
//
// A warp owns 2 * 32 / LN channels: LN = ceil(N / 4) lanes (a power of two) share
// two channels, four states each, in registers as f32x2 pairs.  It walks the
// tokens in tiles: a lane turns the u and delta of LN-th tokens of its channel
// pair into (s, s u) in shared memory, where the LN lanes of the pair read them,
// B and C lie there in fp32, and the next tile's loads are in flight while the
// tile is computed.  Two channels a lane, because every lane reads B_t and C_t
// (32 bytes for its four states): shared memory delivers 128 bytes a clock to
// an SM, so one channel a lane would be held at 16 states a clock by these reads
// alone, below the 32 that the exponential unit does.  <C_t, h_t> is
// summed over the LN lanes for LN tokens at a time, halving the tokens a lane
// keeps at each exchange, so that a lane ends with the token it stores.
//
// With few channels the tokens are split over a cluster of K warps: each first
// finds its segment's end state from a zero start and the sum of its steps (the
// decay of the whole segment is exp(A sum s)), reads those of the segments before
// it through distributed shared memory, and then runs the segment from its
// true start.

#include <cooperative_groups.h>

#include <type_traits>

#include "ssm.cuh"

namespace falcon {
namespace {

namespace cg = cooperative_groups;

template <int LN>
struct Cfg {
  static constexpr int kGroups = 32 / LN;        // channel pairs of a warp
  static constexpr int kChannels = 2 * kGroups;  // channels of a warp
  static constexpr int kTile = LN <= 2 ? 8 : LN <= 16 ? 16 : 32;  // tokens of a tile
  static constexpr int kItems = kTile / LN;      // (token, pair) items of a lane
  static constexpr int kN4 = 4 * LN;
  static constexpr int kQuads = kTile * 2 * LN;  // quads of B and C in a tile
  static constexpr int kLaneQuads = (kQuads + 31) / 32;
  static constexpr bool kAhead = kLaneQuads <= 8;  // the next tile's quads wait in registers
};

template <typename E, int LN, bool SPLIT>
__global__ void __launch_bounds__(32) scan_fwd_kernel(ScanArgs a) {
  typedef Cfg<LN> C;
  typedef typename Raw<E>::Pair Pair;
  typedef typename Raw<E>::Quad Quad;
  __shared__ __align__(16) float bc[C::kTile][2][C::kN4];
  __shared__ float4 step[C::kTile][C::kGroups];  // s of both channels, s u of both
  __shared__ __align__(16) float end_h[SPLIT ? C::kChannels : 1][C::kN4];
  __shared__ float2 end_s[SPLIT ? C::kGroups : 1];

  const int lane = threadIdx.x, pair = lane / LN, q = lane % LN, n0 = q * 4;
  const int R = a.D / a.G;
  const int blocks = (R + C::kChannels - 1) / C::kChannels;
  int K = 1, rank = 0;
  if (SPLIT) {
    K = (int)cg::this_cluster().num_blocks();
    rank = (int)cg::this_cluster().block_rank();
  }
  const int blk = blockIdx.x / K, g = blk / blocks;
  const int r0 = (blk - g * blocks) * C::kChannels + pair * 2;
  const int have = r0 >= R ? 0 : (r0 + 1 < R ? 2 : 1);  // live channels of the pair
  const int d = g * R + (have ? r0 : 0);
  const int64_t b = blockIdx.y;
  const int64_t n = row_length(a.lengths, b, a.T);
  const int64_t tiles = (n + C::kTile - 1) / C::kTile, per = (tiles + K - 1) / K;
  const int64_t begin = rank * per * C::kTile < n ? rank * per * C::kTile : n;
  const int64_t end = begin + per * C::kTile < n ? begin + per * C::kTile : n;

  f32x2 A2[2][2], h[2][2], first[2][2];
  float bias[2], skip[2];
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    const bool live = c < have;
    float v[4], w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const bool in = live && n0 + i < a.N;
      v[i] = in ? a.A[(int64_t)(d + c) * a.N + n0 + i] * kLog2e : 0.f;
      w[i] = in && a.h0 ? a.h0[(b * a.D + d + c) * a.N + n0 + i] : 0.f;
    }
    A2[c][0] = pack2(v[0], v[1]), A2[c][1] = pack2(v[2], v[3]);
    first[c][0] = pack2(w[0], w[1]), first[c][1] = pack2(w[2], w[3]);
    bias[c] = live && a.delta_bias ? a.delta_bias[d + c] : 0.f;
    skip[c] = live && a.Dskip ? a.Dskip[d + c] : 0.f;
  }
  const E* u = static_cast<const E*>(a.u) + b * a.us.batch + d;
  const E* dl = static_cast<const E*>(a.delta) + b * a.ds.batch + d;
  const E* z = a.z ? static_cast<const E*>(a.z) + b * a.zs.batch + d : nullptr;
  const E* Bm = static_cast<const E*>(a.Bm) + b * a.bs.batch + g * a.bs.head;
  const E* Cm = static_cast<const E*>(a.Cm) + b * a.cs.batch + g * a.cs.head;
  E* y = static_cast<E*>(a.y) + b * a.ys.batch + d;

  Pair ru[C::kItems], rd[C::kItems], rz[C::kItems];
  Quad rq[C::kAhead ? C::kLaneQuads : 1];
  auto quad_at = [&](int64_t t0, int i) {  // i-th quad of the tile
    const int k = i / (2 * LN), w = i % (2 * LN), s = (w % LN) * 4;
    const int64_t t = t0 + k;
    const E* p = w < LN ? Bm + t * a.bs.time : Cm + t * a.cs.time;
    return load_quad<E>(p + s, a.vec_bc, t < end ? a.N - s : 0);
  };
  auto fetch = [&](int64_t t0, bool gate) {
#pragma unroll
    for (int i = 0; i < C::kItems; ++i) {
      const int64_t t = t0 + i * LN + q;
      const int k = t < end ? have : 0;
      ru[i] = load_pair<E>(u + t * a.us.time, a.vec_ch, k);
      rd[i] = load_pair<E>(dl + t * a.ds.time, a.vec_ch, k);
      if (gate) rz[i] = load_pair<E>(z + t * a.zs.time, a.vec_ch, k);
    }
    if (C::kAhead) {
#pragma unroll
      for (int i = 0; i < C::kLaneQuads; ++i)
        if (i * 32 + lane < C::kQuads) rq[i] = quad_at(t0, i * 32 + lane);
    }
  };

  // One walk over the segment.  OUT: with outputs; otherwise only h and the
  // sum of the steps.
  float2 sum = make_float2(0.f, 0.f);
  auto walk = [&](auto out) {
    constexpr bool OUT = decltype(out)::value;
    const bool gate = OUT && z != nullptr;
    if (begin < end) fetch(begin, gate);
    for (int64_t t0 = begin; t0 < end; t0 += C::kTile) {
      float2 cu[C::kItems];
      Pair cz[C::kItems];
#pragma unroll
      for (int i = 0; i < C::kItems; ++i) {
        const int k = i * LN + q;
        cu[i] = widen(ru[i]);
        cz[i] = rz[i];
        float2 s = widen(rd[i]);
        s.x += bias[0], s.y += bias[1];
        if (a.softplus) s.x = softplus(s.x), s.y = softplus(s.y);
        if (t0 + k >= end) s = make_float2(0.f, 0.f);
        if (!OUT) sum.x += s.x, sum.y += s.y;
        step[k][pair] = make_float4(s.x, s.y, s.x * cu[i].x, s.y * cu[i].y);
      }
#pragma unroll
      for (int i = 0; i < C::kLaneQuads; ++i) {
        const int k = i * 32 + lane;
        if (k < C::kQuads)
          *reinterpret_cast<float4*>(&bc[0][0][0] + 4 * k) =
              widen(C::kAhead ? rq[C::kAhead ? i : 0] : quad_at(t0, k));
      }
      __syncwarp();
      if (t0 + C::kTile < end) fetch(t0 + C::kTile, gate);

#pragma unroll
      for (int i = 0; i < C::kItems; ++i) {
        float2 o[LN];  // <C_t, h_t> of LN tokens, this lane's states
#pragma unroll
        for (int j = 0; j < LN; ++j) {
          const int k = i * LN + j;
          const float4 s = step[k][pair];
          const ulonglong2 B = *reinterpret_cast<const ulonglong2*>(&bc[k][0][n0]);
          const f32x2 s0 = pack2(s.x, s.x), s1 = pack2(s.y, s.y);
          const f32x2 v0 = pack2(s.z, s.z), v1 = pack2(s.w, s.w);
          h[0][0] = fma2(decay2(s0, A2[0][0]), h[0][0], mul2(v0, B.x));
          h[0][1] = fma2(decay2(s0, A2[0][1]), h[0][1], mul2(v0, B.y));
          h[1][0] = fma2(decay2(s1, A2[1][0]), h[1][0], mul2(v1, B.x));
          h[1][1] = fma2(decay2(s1, A2[1][1]), h[1][1], mul2(v1, B.y));
          if (OUT) {
            const ulonglong2 Ct = *reinterpret_cast<const ulonglong2*>(&bc[k][1][n0]);
            const float2 p0 = unpack2(fma2(Ct.y, h[0][1], mul2(Ct.x, h[0][0])));
            const float2 p1 = unpack2(fma2(Ct.y, h[1][1], mul2(Ct.x, h[1][0])));
            o[j] = make_float2(p0.x + p0.y, p1.x + p1.y);
          }
        }
        if (OUT) {
#pragma unroll
          for (int w = LN / 2; w > 0; w >>= 1) {
            const bool up = q & w;
#pragma unroll
            for (int j = 0; j < w; ++j) {
              const float2 give = up ? o[j] : o[j + w], keep = up ? o[j + w] : o[j];
              o[j].x = keep.x + __shfl_xor_sync(0xffffffffu, give.x, w);
              o[j].y = keep.y + __shfl_xor_sync(0xffffffffu, give.y, w);
            }
          }
          float2 v = make_float2(fmaf(skip[0], cu[i].x, o[0].x), fmaf(skip[1], cu[i].y, o[0].y));
          if (gate) {
            const float2 zt = widen(cz[i]);
            v.x *= zt.x * sigmoid(zt.x);
            v.y *= zt.y * sigmoid(zt.y);
          }
          const int64_t t = t0 + i * LN + q;
          if (t < end) store_pair<E>(y + t * a.ys.time, a.vec_ch, have, v);
        }
      }
      __syncwarp();
    }
  };

  if (SPLIT) {
#pragma unroll
    for (int c = 0; c < 2; ++c) h[c][0] = h[c][1] = pack2(0.f, 0.f);
    if (rank + 1 < K) walk(std::false_type());
#pragma unroll
    for (int w = LN / 2; w > 0; w >>= 1) {
      sum.x += __shfl_xor_sync(0xffffffffu, sum.x, w);
      sum.y += __shfl_xor_sync(0xffffffffu, sum.y, w);
    }
    if (q == 0) end_s[pair] = sum;
#pragma unroll
    for (int c = 0; c < 2; ++c)
      *reinterpret_cast<ulonglong2*>(&end_h[pair * 2 + c][n0]) = make_ulonglong2(h[c][0], h[c][1]);
    cg::this_cluster().sync();
    for (int k = 0; k < rank; ++k) {
      const float2 s = *cg::this_cluster().map_shared_rank(&end_s[pair], k);
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const ulonglong2 e = *reinterpret_cast<const ulonglong2*>(
            cg::this_cluster().map_shared_rank(&end_h[pair * 2 + c][n0], k));
        const float sc = c ? s.y : s.x;
        first[c][0] = fma2(decay2(pack2(sc, sc), A2[c][0]), first[c][0], e.x);
        first[c][1] = fma2(decay2(pack2(sc, sc), A2[c][1]), first[c][1], e.y);
      }
    }
    cg::this_cluster().barrier_arrive();  // this warp has read the others' memory
  }
#pragma unroll
  for (int c = 0; c < 2; ++c) h[c][0] = first[c][0], h[c][1] = first[c][1];
  walk(std::true_type());

  for (int64_t t = n + rank * LN + q; t < a.T; t += K * LN)
    store_pair<E>(y + t * a.ys.time, a.vec_ch, have, make_float2(0.f, 0.f));
  if (rank == K - 1) {
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const float2 v0 = unpack2(h[c][0]), v1 = unpack2(h[c][1]);
      const float v[4] = {v0.x, v0.y, v1.x, v1.y};
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (c < have && n0 + i < a.N) a.h_out[(b * a.D + d + c) * a.N + n0 + i] = v[i];
    }
  }
  if (SPLIT) cg::this_cluster().barrier_wait();  // until the others have read this one's
}

// Warps that fill the GPU: about six an SM.  With fewer, the tokens are split
// while a segment keeps at least two tiles.
constexpr int64_t kFullWarps = 152 * 6;

template <typename E, int LN>
cudaError_t fwd_lanes(const ScanArgs& a, cudaStream_t stream) {
  typedef Cfg<LN> C;
  const int R = a.D / a.G;
  const int64_t blocks = (int64_t)a.G * ((R + C::kChannels - 1) / C::kChannels);
  const int64_t tiles = (a.T + C::kTile - 1) / C::kTile;
  int K = 1;
  while (K < 16 && blocks * a.B * K * 2 <= kFullWarps * 2 && tiles >= 4 * K) K *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(blocks * K), (unsigned)a.B);
  cfg.blockDim = dim3(32);
  cfg.stream = stream;
  if (K == 1) return cudaLaunchKernelEx(&cfg, scan_fwd_kernel<E, LN, false>, a);
  if (K > 8) {
    const cudaError_t e = cudaFuncSetAttribute(scan_fwd_kernel<E, LN, true>,
                                               cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
  }
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = (unsigned)K;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, scan_fwd_kernel<E, LN, true>, a);
}

template <typename E>
cudaError_t fwd_typed(const ScanArgs& a, cudaStream_t stream) {
  switch (scan_lanes(a.N)) {
    case 1: return fwd_lanes<E, 1>(a, stream);
    case 2: return fwd_lanes<E, 2>(a, stream);
    case 4: return fwd_lanes<E, 4>(a, stream);
    case 8: return fwd_lanes<E, 8>(a, stream);
    case 16: return fwd_lanes<E, 16>(a, stream);
    default: return fwd_lanes<E, 32>(a, stream);
  }
}

}  // namespace

// Whether pointer and strides keep every access of `elems` elements aligned.
bool scan_rows_fit(const void* p, const falcon_strides& s, int elems, int esz) {
  return reinterpret_cast<uintptr_t>(p) % (uintptr_t)(elems * esz) == 0 && s.batch % elems == 0 &&
         s.time % elems == 0 && s.head % elems == 0;
}

cudaError_t launch_scan_fwd(const ScanArgs& in, cudaStream_t stream) {
  ScanArgs a = in;
  const int esz = a.dtype == FALCON_BF16 ? 2 : 4;
  a.us.head = a.ds.head = a.zs.head = a.ys.head = 0;  // unused
  a.vec_ch = a.D / a.G % 2 == 0 && scan_rows_fit(a.u, a.us, 2, esz) &&
             scan_rows_fit(a.delta, a.ds, 2, esz) && scan_rows_fit(a.z, a.zs, 2, esz) &&
             scan_rows_fit(a.y, a.ys, 2, esz);
  a.vec_bc = a.N % 4 == 0 && scan_rows_fit(a.Bm, a.bs, 4, esz) &&
             scan_rows_fit(a.Cm, a.cs, 4, esz);
  return a.dtype == FALCON_BF16 ? fwd_typed<__nv_bfloat16>(a, stream)
                                : fwd_typed<float>(a, stream);
}

}  // namespace falcon
