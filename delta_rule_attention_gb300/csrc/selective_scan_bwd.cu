// Gradient of the selective scan.  With a_t = exp(s_t A), g_t the adjoint of h_t,
// dy_t after the gate:
//   g_t = C_t dy_t + a_{t+1} g_{t+1},   w_t = g_t a_t h_{t-1}
//   dC_t = sum_d dy_t h_t,  dB_t = sum_d g_t s_t u_t,  dA = sum_t w_t s_t,
//   du_t = s_t <g_t, B_t> + Dskip dy_t,  ds_t = <w_t, A> + <g_t, B_t> u_t.
//
// Tokens are cut into chunks of kChunk, which run in parallel:
//   1. every chunk by itself: its end state from a zero start, the adjoint it hands to
//      the chunk before it from a zero end, and the sum of its steps (the
//      decay of the whole chunk is exp(A sum s));
//   2. a walk over the chunks turns these into the state entering and the adjoint
//      leaving every chunk (one thread for four states of a channel);
//   3. every chunk again, from its true ends: a forward sweep keeps the state before
//      each group of kSub tokens in shared memory, then the groups are walked back,
//      each one's states and decays recomputed into registers;
//   4. sums: dB and dC over the blocks of channels, dA, dDskip and ddelta_bias over
//      the blocks of tokens, in a fixed order.
// Where the terms of dB and dC of all blocks of channels would take more than kTermBytes,
// steps 3 and 4 run once for each set of blocks whose terms fit.
// A warp owns 2 * 32 / LN channels: LN lanes share two channels, four states each, as
// f32x2 pairs.  <g, B>, <w, A> and <C, h> are summed over the LN lanes for kSub
// tokens at once, halving the tokens a lane keeps at each exchange; dB and dC are
// added up over the lane's two channels in registers, over the warp's lanes through
// shared memory, and over the block's warps when the chunk ends.
//
// B8 T2048 D2048 N16 bf16: 0.87 ms, of which step 1 takes 198 us, step 2 39, step 3 614,
// step 4 21; its bytes would take 70 us.  Steps 1 and 3 are bound by instruction issue and
// shared memory together (67% and 70% busy in step 1, 60% and 73% in step 3, whose
// 168 registers and 77 KB leave three blocks an SM): about ten and 27 instructions a
// lane for each (token, channel, state), three exponentials among them.  A chunk of 32
// costs step 2 a state and an adjoint for every 32 tokens (0.2 GB there and back); a group
// of four tokens is what fits the registers with its states and decays.  Measured and not
// kept: scalar arithmetic instead of doubled scalars in pairs (954 us).

#include <initializer_list>

#include "ssm.cuh"

namespace falcon {
namespace {

constexpr int kChunk = 32;
constexpr int kSub = 4;
constexpr int kSubs = kChunk / kSub;

int lanes_of(int N) {
  int ln = 1;
  while (ln * 4 < N) ln *= 2;
  return ln;
}
__host__ __device__ constexpr int warps_of(int LN) { return LN <= 8 ? 4 : LN == 16 ? 2 : 1; }

template <int LN>
struct Cfg {
  static constexpr int kWarps = warps_of(LN);
  static constexpr int kGroups = 32 / LN;        // channel pairs of a warp
  static constexpr int kChannels = 2 * kGroups;  // channels of a warp
  static constexpr int kNP = 4 * LN;             // states, padded
  static constexpr int kRow = kGroups;
  // A lane brings the tokens i * LN + q of channel pair `pair ^ turn(q)`, so that the
  // eight lanes of a store phase, whose rows begin in the same bank, store to
  // different places of them.
  __host__ __device__ static constexpr int turn(int q) {
    return LN == 2 ? q << 2 : LN == 4 ? q << 1 : LN == 8 ? q >> 1 : LN == 16 ? (q >> 2) & 1 : 0;
  }
  static constexpr int kBase = kGroups * kNP + 16;  // one token's dB (or dC) terms, padded
  // the chunk's dB and dC of a warp lie over its used steps where they fit
  static constexpr bool kOver = kRow * 4 >= 2 * kNP;
};

template <int LN>
struct WarpShared {
  typedef Cfg<LN> C;
  float4 sv[kChunk][C::kRow];   // s of both channels, s u of both
  float2 dyg[kChunk][C::kRow];  // dy after the gate
};
template <int LN>
struct GradShared {
  typedef Cfg<LN> C;
  float4 kept[kSubs - 1][2][32];         // state before each group but the first, by lane
  float terms[kSub][2][C::kBase];        // dB and dC terms by lane group
  float sums[C::kOver || C::kWarps == 1 ? 1 : kChunk][2 * C::kNP];
};

// Bytes of dB and dC terms that are kept at a time.  A block covers 64 channels with 16
// states and 2 with 128, so that the terms of all blocks would grow past any tensor of
// the call (17 GB for B8 T2048 D2048 N128).  Each pass has a last wave of its own: that
// call takes 26.6 ms in eight passes, 27.4 with 512 MB at a time and 25.8 with all terms
// kept; one with 64 states, whose terms are 2 GB, 5.19 ms, and 5.47 with 512 MB.
constexpr int64_t kTermBytes = 2LL << 30;

// Parts of the workspace, in floats.
struct Layout {
  int64_t chunks, parts, groups, per, NP;
  // parts of a pass of step 3, and the place of its first one's terms: 1 where there are
  // several passes, whose sum so far lies in place 0
  int64_t at_once, place0;
  size_t hin, gin, sums, dbc, dA, dD, dbias, total;
  Layout(int64_t B, int64_t T, int D, int G, int N) {
    const int ln = lanes_of(N), ch = 64 / ln * warps_of(ln);
    NP = 4 * ln;
    chunks = (T + kChunk - 1) / kChunk;
    parts = (D / G + ch - 1) / ch;
    const int64_t rows = B * T * G * 2 * NP, most = kTermBytes / 4 / (rows > 0 ? rows : 1);
    const int64_t passes = most >= parts ? 1 : most < 1 ? parts : (parts + most - 1) / most;
    at_once = (parts + passes - 1) / passes;
    place0 = passes > 1;
    // chunks a block walks in step 3: as many as leave four blocks a resident slot
    per = 1;
    while (per < 8 && G * at_once * B * (chunks / (2 * per)) >= 152 * 3 * 8) per *= 2;
    groups = (chunks + per - 1) / per;
    size_t at = 0;
    auto take = [&](int64_t n) {
      const size_t p = at;
      at += (size_t)((n + 63) / 64 * 64);
      return p;
    };
    hin = take(B * chunks * D * NP);
    gin = take(B * chunks * D * NP);
    sums = take(B * chunks * D);
    dbc = take((place0 + at_once) * rows);
    dA = take(groups * B * D * NP);
    dD = take(groups * B * D);
    dbias = take(groups * B * D);
    total = at;
  }
};

// What a warp knows of its place.
template <typename E, int LN>
struct Place {
  typedef Cfg<LN> C;
  int lane, warp, pair, q, n0, g, part, have, d;
  int64_t b, n;
  bool whole;
  float bias[2];
  // the channel pair whose tokens this lane brings, its live channels, how far its
  // channels are from d, and their biases
  int brings, its_have, off;
  float its_bias[2];
  const E *u, *dl, *z, *dy, *Bm, *Cm;

  // blocks of `parts` parts from part0 on
  __device__ __forceinline__ Place(const ScanArgs& a, int parts, int part0) {
    lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    pair = lane / LN, q = lane % LN, n0 = q * 4;
    const int R = a.D / a.G;
    const int blk = blockIdx.x % (a.G * parts);
    g = blk / parts, part = part0 + blk - g * parts;
    const int w0 = (part * C::kWarps + warp) * C::kChannels, r0 = w0 + pair * 2;
    have = r0 >= R ? 0 : (r0 + 1 < R ? 2 : 1);
    d = g * R + (have ? r0 : 0);
    b = blockIdx.y;
    n = row_length(a.lengths, b, a.T);
    whole = a.vec_ch && w0 + C::kChannels <= R;
    bias[0] = have > 0 && a.delta_bias ? a.delta_bias[d] : 0.f;
    bias[1] = have > 1 && a.delta_bias ? a.delta_bias[d + 1] : 0.f;
    brings = pair ^ C::turn(q);
    const int r1 = w0 + brings * 2;
    its_have = r1 >= R ? 0 : (r1 + 1 < R ? 2 : 1);
    off = g * R + (its_have ? r1 : 0) - d;
    its_bias[0] = its_have > 0 && a.delta_bias ? a.delta_bias[d + off] : 0.f;
    its_bias[1] = its_have > 1 && a.delta_bias ? a.delta_bias[d + off + 1] : 0.f;
    u = static_cast<const E*>(a.u) + b * a.us.batch + d;
    dl = static_cast<const E*>(a.delta) + b * a.ds.batch + d;
    z = a.z ? static_cast<const E*>(a.z) + b * a.zs.batch + d : nullptr;
    dy = static_cast<const E*>(a.dy) + b * a.dys.batch + d;
    Bm = static_cast<const E*>(a.Bm) + b * a.bs.batch + g * a.bs.head;
    Cm = static_cast<const E*>(a.Cm) + b * a.cs.batch + g * a.cs.head;
  }
  // A in units of log2(e), two states a pair
  __device__ __forceinline__ void decays(const ScanArgs& a, f32x2 (&A2)[2][2]) const {
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      float v[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        v[i] = c < have && n0 + i < a.N ? rate_log2(a.A[(int64_t)(d + c) * a.N + n0 + i]) : 0.f;
      A2[c][0] = pack2(v[0], v[1]), A2[c][1] = pack2(v[2], v[3]);
    }
  }
};

// Brings the tokens t0 .. of a chunk into shared memory; adds up the lane's steps.
// A whole chunk's loads are all under way before the first is used.
template <typename E, int LN>
__device__ __forceinline__ float2 stage_chunk(const ScanArgs& a, const Place<E, LN>& p, int64_t t0,
                                              float (&bc)[kChunk][2][4 * LN],
                                              WarpShared<LN>& ws) {
  typedef Cfg<LN> C;
  typedef typename Raw<E>::Pair Pair;
  typedef typename Raw<E>::Quad Quad;
  constexpr int kItems = kChunk / LN, kBatch = kItems < 8 ? kItems : 8;
  constexpr int kQuads = kChunk * 2 * LN / (C::kWarps * 32) > 0
                             ? kChunk * 2 * LN / (C::kWarps * 32) : 1;
  constexpr int kQuadBatch = kQuads < 4 ? kQuads : 4;
  const bool full = p.whole && t0 + kChunk <= p.n;
  auto quad_at = [&](int i) {
    const int k = i / (2 * LN), w = i % (2 * LN), s = w % LN * 4;
    const int64_t t = t0 + k;
    const E* src = w < LN ? p.Bm + t * a.bs.time : p.Cm + t * a.cs.time;
    return load_quad<E>(src + s, a.vec_bc, t < p.n ? a.N - s : 0);
  };
  float2 sum = make_float2(0.f, 0.f);
  auto put = [&](int k, float2 ut, float2 s, float2 o, float2 zt) {
    s.x += p.its_bias[0], s.y += p.its_bias[1];
    if (a.softplus) s = softplus2(s);
    if (p.z) o.x *= zt.x * sigmoid(zt.x), o.y *= zt.y * sigmoid(zt.y);
    if (!full) {  // no token, or a pair without a second (or any) channel
      const int have = t0 + k < p.n ? p.its_have : 0;
      if (have < 2) s.y = o.y = 0.f;
      if (have < 1) s.x = o.x = 0.f;
    }
    sum.x += s.x, sum.y += s.y;
    ws.sv[k][p.brings] = make_float4(s.x, s.y, s.x * ut.x, s.y * ut.y);
    ws.dyg[k][p.brings] = o;
  };
  for (int i0 = 0; i0 < kQuads; i0 += kQuadBatch) {
    Quad rq[kQuadBatch];
#pragma unroll
    for (int i = 0; i < kQuadBatch; ++i) {
      const int e = (i0 + i) * C::kWarps * 32 + threadIdx.x;
      if (kChunk * 2 * LN % (C::kWarps * 32) == 0 || e < kChunk * 2 * LN) rq[i] = quad_at(e);
    }
    if (i0 == 0) {
#pragma unroll 1
      for (int j0 = 0; j0 < kItems; j0 += kBatch) {
        Pair ru[kBatch], rd[kBatch], ro[kBatch], rz[kBatch];
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
          const int64_t t = t0 + (j0 + i) * LN + p.q;
          rz[i] = Pair();
          if (full) {
            ru[i] = *reinterpret_cast<const Pair*>(p.u + p.off + t * a.us.time);
            rd[i] = *reinterpret_cast<const Pair*>(p.dl + p.off + t * a.ds.time);
            ro[i] = *reinterpret_cast<const Pair*>(p.dy + p.off + t * a.dys.time);
            if (p.z) rz[i] = *reinterpret_cast<const Pair*>(p.z + p.off + t * a.zs.time);
          } else {
            const int have = t < p.n ? p.its_have : 0;
            ru[i] = load_pair<E>(p.u + p.off + t * a.us.time, a.vec_ch, have);
            rd[i] = load_pair<E>(p.dl + p.off + t * a.ds.time, a.vec_ch, have);
            ro[i] = load_pair<E>(p.dy + p.off + t * a.dys.time, a.vec_ch, have);
            if (p.z) rz[i] = load_pair<E>(p.z + p.off + t * a.zs.time, a.vec_ch, have);
          }
        }
#pragma unroll
        for (int i = 0; i < kBatch; ++i)
          put((j0 + i) * LN + p.q, widen(ru[i]), widen(rd[i]), widen(ro[i]), widen(rz[i]));
      }
    }
#pragma unroll
    for (int i = 0; i < kQuadBatch; ++i) {
      const int e = (i0 + i) * C::kWarps * 32 + threadIdx.x;
      if (kChunk * 2 * LN % (C::kWarps * 32) == 0 || e < kChunk * 2 * LN)
        reinterpret_cast<float4*>(bc)[e] = widen(rq[i]);
    }
  }
  return sum;
}

__device__ __forceinline__ f32x2 dup2(float v) { return pack2(v, v); }
__device__ __forceinline__ f32x2 decay_pair(f32x2 s, f32x2 A2) {
  const float2 e = decay2(s, A2, dup2(kDecayLift));
  return pack2(e.x, e.y);
}

// Step 1.
template <typename E, int LN>
__global__ void __launch_bounds__(Cfg<LN>::kWarps * 32)
    scan_bwd_chunk_kernel(const __grid_constant__ ScanArgs a, float* ws,
                          const __grid_constant__ Layout l) {
  typedef Cfg<LN> C;
  extern __shared__ __align__(16) unsigned char bytes[];
  auto& bc = *reinterpret_cast<float(*)[kChunk][2][C::kNP]>(bytes);
  const Place<E, LN> p(a, (int)l.parts, 0);
  WarpShared<LN>& sh = reinterpret_cast<WarpShared<LN>*>(bytes + sizeof(bc))[p.warp];
  const int64_t chunk = blockIdx.x / (unsigned)(a.G * l.parts), t0 = chunk * kChunk;
  if (t0 >= p.n) return;
  f32x2 A2[2][2], h[2][2], P[2][2], r[2][2];
  p.decays(a, A2);
#pragma unroll
  for (int c = 0; c < 2; ++c)
#pragma unroll
    for (int x = 0; x < 2; ++x) h[c][x] = r[c][x] = dup2(0.f), P[c][x] = dup2(1.f);
  float2 sum = stage_chunk<E, LN>(a, p, t0, bc, sh);
  __syncthreads();
#pragma unroll 4
  for (int k = 0; k < kChunk; ++k) {
    const float4 sv = sh.sv[k][p.pair];
    const float2 o = sh.dyg[k][p.pair];
    const ulonglong2 B = *reinterpret_cast<const ulonglong2*>(&bc[k][0][p.n0]);
    const ulonglong2 Ct = *reinterpret_cast<const ulonglong2*>(&bc[k][1][p.n0]);
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const f32x2 s2 = dup2(c ? sv.y : sv.x), v2 = dup2(c ? sv.w : sv.z), o2 = dup2(c ? o.y : o.x);
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const f32x2 at = decay_pair(s2, A2[c][x]);
        h[c][x] = fma2(at, h[c][x], mul2(v2, x ? B.y : B.x));
        P[c][x] = mul2(at, P[c][x]);
        r[c][x] = fma2(P[c][x], mul2(o2, x ? Ct.y : Ct.x), r[c][x]);
      }
    }
  }
  // over the LN lanes that brought a pair's tokens; the lane with q = 0 brought its own's
#pragma unroll
  for (int w = LN / 2; w > 0; w >>= 1) {
    sum.x += __shfl_xor_sync(0xffffffffu, sum.x, C::turn(w) * LN + w);
    sum.y += __shfl_xor_sync(0xffffffffu, sum.y, C::turn(w) * LN + w);
  }
  const int64_t row = (p.b * l.chunks + chunk) * a.D + p.d;
#pragma unroll
  for (int c = 0; c < 2; ++c)
    if (c < p.have) {
      *reinterpret_cast<ulonglong2*>(ws + l.hin + (row + c) * C::kNP + p.n0) =
          make_ulonglong2(h[c][0], h[c][1]);
      *reinterpret_cast<ulonglong2*>(ws + l.gin + (row + c) * C::kNP + p.n0) =
          make_ulonglong2(r[c][0], r[c][1]);
      if (p.q == 0) ws[l.sums + row + c] = c ? sum.y : sum.x;
    }
}

// Step 2: hin[c] becomes the state entering chunk c (blockIdx.z = 0), gin[c] the
// adjoint entering it from behind (blockIdx.z = 1), four chunks' loads ahead.
__global__ void __launch_bounds__(128)
    scan_bwd_chain_kernel(const __grid_constant__ ScanArgs a, float* ws,
                          const __grid_constant__ Layout l) {
  const int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  const int64_t quads = l.NP / 4;
  if (i >= (int64_t)a.D * quads) return;
  const bool back = blockIdx.z == 1;
  const int64_t d = i / quads, b = blockIdx.y;
  const int n0 = (int)(i - d * quads) * 4;
  const int64_t n = row_length(a.lengths, b, a.T);
  const int count = (int)((n + kChunk - 1) / kChunk);
  const float* from = back ? a.dh_T : a.h0;
  float A2[4], h[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const bool in = n0 + k < a.N;
    A2[k] = in ? rate_log2(a.A[d * a.N + n0 + k]) : 0.f;
    h[k] = in && from ? from[(b * a.D + d) * a.N + n0 + k] : 0.f;
  }
  // the walk's first chunk and its direction
  const int64_t start = back ? count - 1 : 0, dir = back ? -1 : 1;
  const int64_t step = dir * a.D * l.NP, sstep = dir * a.D;
  float* hp = ws + (back ? l.gin : l.hin) + ((b * l.chunks + start) * a.D + d) * l.NP + n0;
  const float* sp = ws + l.sums + (b * l.chunks + start) * a.D + d;
  constexpr int kAhead = 4;
  for (int c0 = 0; c0 < count; c0 += kAhead) {
    float4 hv[kAhead];
    float hs[kAhead];
#pragma unroll
    for (int k = 0; k < kAhead; ++k)
      if (c0 + k < count) {
        hv[k] = *reinterpret_cast<const float4*>(hp + k * step);
        hs[k] = sp[k * sstep];
      }
#pragma unroll
    for (int k = 0; k < kAhead; ++k)
      if (c0 + k < count) {
        *reinterpret_cast<float4*>(hp + k * step) = make_float4(h[0], h[1], h[2], h[3]);
        const float ha[4] = {hv[k].x, hv[k].y, hv[k].z, hv[k].w};
#pragma unroll
        for (int x = 0; x < 4; ++x) h[x] = fmaf(decay(hs[k], A2[x]), h[x], ha[x]);
      }
    hp += kAhead * step;
    sp += kAhead * sstep;
  }
  if (back && a.dh0)
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (n0 + k < a.N) a.dh0[(b * a.D + d) * a.N + n0 + k] = h[k];
}

// Step 3.
template <typename E, int LN>
__global__ void __launch_bounds__(Cfg<LN>::kWarps * 32, LN == 4 ? 3 : 1)
    scan_bwd_grad_kernel(const __grid_constant__ ScanArgs a, float* ws,
                         const __grid_constant__ Layout l, int part0, int parts) {
  typedef Cfg<LN> C;
  typedef typename Raw<E>::Pair Pair;
  constexpr int kMine = LN >= kSub ? 1 : kSub / LN;  // tokens of a group a lane finishes
  extern __shared__ __align__(16) unsigned char bytes[];
  auto& bc = *reinterpret_cast<float(*)[kChunk][2][C::kNP]>(bytes);
  const Place<E, LN> p(a, parts, part0);
  WarpShared<LN>* all = reinterpret_cast<WarpShared<LN>*>(bytes + sizeof(bc));
  GradShared<LN>* grads = reinterpret_cast<GradShared<LN>*>(all + C::kWarps);
  WarpShared<LN>& sh = all[p.warp];
  GradShared<LN>& gs = grads[p.warp];
  auto sums_row = [&](int warp, int k) -> float* {
    return C::kOver ? reinterpret_cast<float*>(all[warp].sv[k]) : grads[warp].sums[k];
  };
  const float skip0 = p.have > 0 && a.Dskip ? a.Dskip[p.d] : 0.f;
  const float skip1 = p.have > 1 && a.Dskip ? a.Dskip[p.d + 1] : 0.f;
  f32x2 A2[2][2], dA[2][2];
  p.decays(a, A2);
#pragma unroll
  for (int c = 0; c < 2; ++c) dA[c][0] = dA[c][1] = dup2(0.f);
  float2 dD = make_float2(0.f, 0.f), dbias = dD;
  // first token of a group that this lane finishes, and whether it stores it
  const int mine = LN >= 4 ? (p.q & (LN / 2) ? 2 : 0) + (p.q & (LN / 4) ? 1 : 0)
                           : (LN == 2 ? p.q * 2 : 0);
  const bool stores = LN <= 4 || (p.q & (LN / 4 - 1)) == 0;
  E* du = static_cast<E*>(a.du) + p.b * a.T * a.D + p.d;
  E* dd = static_cast<E*>(a.ddelta) + p.b * a.T * a.D + p.d;
  E* dz = a.z ? static_cast<E*>(a.dz) + p.b * a.T * a.D + p.d : nullptr;

  const int64_t group = blockIdx.x / (unsigned)(a.G * parts);
  const int64_t place = l.place0 + p.part - part0;  // of this part's dB and dC terms
  for (int64_t chunk = group * l.per; chunk < (group + 1) * l.per && chunk < l.chunks; ++chunk) {
    const int64_t t0 = chunk * kChunk;
    if (t0 >= p.n) {  // behind the row's end
      for (int k = p.q; k < kChunk && t0 + k < a.T; k += LN) {
        const float2 none = make_float2(0.f, 0.f);
        store_pair<E>(du + (t0 + k) * a.D, a.vec_ch, p.have, none);
        store_pair<E>(dd + (t0 + k) * a.D, a.vec_ch, p.have, none);
        if (dz) store_pair<E>(dz + (t0 + k) * a.D, a.vec_ch, p.have, none);
      }
      continue;
    }
    const bool full = p.whole && t0 + kChunk <= p.n;
    stage_chunk<E, LN>(a, p, t0, bc, sh);
    __syncthreads();
    const int64_t row = (p.b * l.chunks + chunk) * a.D + p.d;
    f32x2 h[2][2], g[2][2];
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      ulonglong2 hv = make_ulonglong2(0, 0), gv = hv;
      if (c < p.have) {
        hv = *reinterpret_cast<const ulonglong2*>(ws + l.hin + (row + c) * C::kNP + p.n0);
        gv = *reinterpret_cast<const ulonglong2*>(ws + l.gin + (row + c) * C::kNP + p.n0);
      }
      h[c][0] = hv.x, h[c][1] = hv.y, g[c][0] = gv.x, g[c][1] = gv.y;
    }
    auto forward = [&](int k, f32x2 (&hc)[2][2], f32x2 (&at)[2][2]) {
      const float4 sv = sh.sv[k][p.pair];
      const ulonglong2 B = *reinterpret_cast<const ulonglong2*>(&bc[k][0][p.n0]);
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const f32x2 s2 = dup2(c ? sv.y : sv.x), v2 = dup2(c ? sv.w : sv.z);
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          at[c][x] = decay_pair(s2, A2[c][x]);
          hc[c][x] = fma2(at[c][x], hc[c][x], mul2(v2, x ? B.y : B.x));
        }
      }
    };
    auto keep = [&](int sub) {
#pragma unroll
      for (int c = 0; c < 2; ++c)
        *reinterpret_cast<ulonglong2*>(&gs.kept[sub][c][p.lane]) =
            make_ulonglong2(h[c][0], h[c][1]);
    };
    const f32x2 h0[2][2] = {{h[0][0], h[0][1]}, {h[1][0], h[1][1]}};
#pragma unroll 1
    for (int sub = 0; sub + 1 < kSubs; ++sub) {
#pragma unroll
      for (int k = 0; k < kSub; ++k) {
        f32x2 at[2][2];
        forward(sub * kSub + k, h, at);
      }
      keep(sub);  // before group sub + 1
    }

#pragma unroll 1
    for (int sub = kSubs - 1; sub >= 0; --sub) {
      const int k0 = sub * kSub;
      f32x2 hs[kSub + 1][2][2], at[kSub][2][2];
      // what this lane needs to finish its tokens, on its way meanwhile
      Pair ru[kMine], rd[kMine], ro[kMine], rz[kMine];
#pragma unroll
      for (int m = 0; m < kMine; ++m) {
        const int64_t t = t0 + k0 + mine + m;
        rz[m] = Pair();
        if (full) {
          ru[m] = *reinterpret_cast<const Pair*>(p.u + t * a.us.time);
          rd[m] = *reinterpret_cast<const Pair*>(p.dl + t * a.ds.time);
          ro[m] = *reinterpret_cast<const Pair*>(p.dy + t * a.dys.time);
          if (dz) rz[m] = *reinterpret_cast<const Pair*>(p.z + t * a.zs.time);
        } else {
          const int have = t < p.n ? p.have : 0;
          ru[m] = load_pair<E>(p.u + t * a.us.time, a.vec_ch, have);
          rd[m] = load_pair<E>(p.dl + t * a.ds.time, a.vec_ch, have);
          ro[m] = load_pair<E>(p.dy + t * a.dys.time, a.vec_ch, have);
          if (dz) rz[m] = load_pair<E>(p.z + t * a.zs.time, a.vec_ch, have);
        }
      }
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        if (sub > 0) {
          const ulonglong2 v = *reinterpret_cast<const ulonglong2*>(&gs.kept[sub - 1][c][p.lane]);
          hs[0][c][0] = v.x, hs[0][c][1] = v.y;
        } else {
          hs[0][c][0] = h0[c][0], hs[0][c][1] = h0[c][1];
        }
      }
#pragma unroll
      for (int k = 0; k < kSub; ++k) {
#pragma unroll
        for (int c = 0; c < 2; ++c)
          hs[k + 1][c][0] = hs[k][c][0], hs[k + 1][c][1] = hs[k][c][1];
        forward(k0 + k, hs[k + 1], at[k]);
      }
      float2 gB[kSub], wA[kSub], yC[kSub];  // of both channels, this lane's states
#pragma unroll
      for (int k = kSub - 1; k >= 0; --k) {
        const float4 sv = sh.sv[k0 + k][p.pair];
        const float2 o = sh.dyg[k0 + k][p.pair];
        const ulonglong2 Bq = *reinterpret_cast<const ulonglong2*>(&bc[k0 + k][0][p.n0]);
        const ulonglong2 Cq = *reinterpret_cast<const ulonglong2*>(&bc[k0 + k][1][p.n0]);
        f32x2 vB[2], vC[2];
        float part[3][2];
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const f32x2 s2 = dup2(c ? sv.y : sv.x), v2 = dup2(c ? sv.w : sv.z),
                      o2 = dup2(c ? o.y : o.x);
          f32x2 acc[3];
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const f32x2 Bx = x ? Bq.y : Bq.x, Cx = x ? Cq.y : Cq.x, now = hs[k + 1][c][x];
            const f32x2 gt = fma2(o2, Cx, g[c][x]);
            const f32x2 gn = mul2(gt, at[k][c][x]);
            const f32x2 w = mul2(gn, hs[k][c][x]);
            g[c][x] = gn;
            dA[c][x] = fma2(w, s2, dA[c][x]);
            acc[0] = x ? fma2(gt, Bx, acc[0]) : mul2(gt, Bx);
            acc[1] = x ? fma2(w, A2[c][x], acc[1]) : mul2(w, A2[c][x]);
            acc[2] = x ? fma2(Cx, now, acc[2]) : mul2(Cx, now);
            vB[x] = c ? fma2(gt, v2, vB[x]) : mul2(gt, v2);
            vC[x] = c ? fma2(o2, now, vC[x]) : mul2(o2, now);
          }
#pragma unroll
          for (int m = 0; m < 3; ++m) {
            const float2 v = unpack2(acc[m]);
            part[m][c] = v.x + v.y;
          }
        }
        gB[k] = make_float2(part[0][0], part[0][1]);
        wA[k] = make_float2(part[1][0], part[1][1]);
        yC[k] = make_float2(part[2][0], part[2][1]);
        *reinterpret_cast<ulonglong2*>(&gs.terms[k][0][p.pair * C::kNP + p.n0]) =
            make_ulonglong2(vB[0], vB[1]);
        *reinterpret_cast<ulonglong2*>(&gs.terms[k][1][p.pair * C::kNP + p.n0]) =
            make_ulonglong2(vC[0], vC[1]);
      }
      // <g, B>, <w, A>, <C, h>: after the exchanges this lane has token `mine`
      auto exchange = [&](float2(&v)[kSub]) {
        if (LN >= 2) {
          const bool up = p.q & (LN / 2);
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const float2 give = up ? v[k] : v[k + 2], have = up ? v[k + 2] : v[k];
            v[k].x = have.x + __shfl_xor_sync(0xffffffffu, give.x, LN / 2);
            v[k].y = have.y + __shfl_xor_sync(0xffffffffu, give.y, LN / 2);
          }
        }
        if (LN >= 4) {
          const bool up = p.q & (LN / 4);
          const float2 give = up ? v[0] : v[1], have = up ? v[1] : v[0];
          v[0].x = have.x + __shfl_xor_sync(0xffffffffu, give.x, LN / 4);
          v[0].y = have.y + __shfl_xor_sync(0xffffffffu, give.y, LN / 4);
        }
#pragma unroll
        for (int w = LN / 8; w > 0; w >>= 1) {
          v[0].x += __shfl_xor_sync(0xffffffffu, v[0].x, w);
          v[0].y += __shfl_xor_sync(0xffffffffu, v[0].y, w);
        }
      };
      exchange(gB);
      exchange(wA);
      exchange(yC);
      if (stores) {
#pragma unroll
        for (int m = 0; m < kMine; ++m) {
          const int k = k0 + mine + m;
          const int64_t t = t0 + k;
          if (t < a.T) {
            float2 vu = make_float2(0.f, 0.f), vd = vu, vz = vu;
            if (t < p.n) {
              const float4 sv = sh.sv[k][p.pair];
              const float2 o = sh.dyg[k][p.pair];
              const float2 ut = widen(ru[m]);
              vu = make_float2(fmaf(gB[m].x, sv.x, skip0 * o.x), fmaf(gB[m].y, sv.y, skip1 * o.y));
              vd = make_float2(fmaf(gB[m].x, ut.x, wA[m].x * kLn2),
                               fmaf(gB[m].y, ut.y, wA[m].y * kLn2));
              if (a.softplus) {
                const float2 raw = widen(rd[m]);
                vd.x *= sigmoid(raw.x + p.bias[0]);
                vd.y *= sigmoid(raw.y + p.bias[1]);
              }
              if (dz) {
                const float2 zt = widen(rz[m]), yt = widen(ro[m]);
                const float q0 = sigmoid(zt.x), q1 = sigmoid(zt.y);
                vz.x = yt.x * fmaf(skip0, ut.x, yC[m].x) * q0 * fmaf(zt.x, 1.f - q0, 1.f);
                vz.y = yt.y * fmaf(skip1, ut.y, yC[m].y) * q1 * fmaf(zt.y, 1.f - q1, 1.f);
              }
              dD.x = fmaf(o.x, ut.x, dD.x), dD.y = fmaf(o.y, ut.y, dD.y);
              dbias.x += vd.x, dbias.y += vd.y;
            }
            store_pair<E>(du + t * a.D, a.vec_ch, p.have, vu);
            store_pair<E>(dd + t * a.D, a.vec_ch, p.have, vd);
            if (dz) store_pair<E>(dz + t * a.D, a.vec_ch, p.have, vz);
          }
        }
      }
      __syncwarp();
      // dB and dC of the group's tokens over the warp's channel pairs, four states a lane
#pragma unroll
      for (int i = 0; i < (kSub * 2 * LN + 31) / 32; ++i) {
        const int e = i * 32 + p.lane;
        if (kSub * 2 * LN % 32 == 0 || e < kSub * 2 * LN) {
          const int k = e / (2 * LN), w = e % (2 * LN);
          const float* from = &gs.terms[k][w / LN][w % LN * 4];
          ulonglong2 v = *reinterpret_cast<const ulonglong2*>(from);
#pragma unroll
          for (int j = 1; j < C::kGroups; ++j) {
            const ulonglong2 m = *reinterpret_cast<const ulonglong2*>(from + j * C::kNP);
            v.x = add2(v.x, m.x), v.y = add2(v.y, m.y);
          }
          if (C::kWarps > 1)
            *reinterpret_cast<ulonglong2*>(sums_row(p.warp, k0 + k) + w * 4) = v;
          else if (t0 + k0 + k < p.n)
            *reinterpret_cast<ulonglong2*>(
                ws + l.dbc +
                (((place * a.B + p.b) * a.T + t0 + k0 + k) * a.G + p.g) * 2 * C::kNP + w * 4) = v;
        }
      }
      __syncwarp();
    }
    __syncthreads();
    if (C::kWarps > 1) {
      for (int i = threadIdx.x; i < kChunk * 2 * LN; i += C::kWarps * 32) {
        const int k = i / (2 * LN), w = i % (2 * LN);
        if (t0 + k < p.n) {
          ulonglong2 v = *reinterpret_cast<const ulonglong2*>(sums_row(0, k) + w * 4);
#pragma unroll
          for (int m = 1; m < C::kWarps; ++m) {
            const ulonglong2 e = *reinterpret_cast<const ulonglong2*>(sums_row(m, k) + w * 4);
            v.x = add2(v.x, e.x), v.y = add2(v.y, e.y);
          }
          *reinterpret_cast<ulonglong2*>(
              ws + l.dbc +
              (((place * a.B + p.b) * a.T + t0 + k) * a.G + p.g) * 2 * C::kNP + w * 4) = v;
        }
      }
      __syncthreads();
    }
  }
#pragma unroll
  for (int w = LN / 2; w > 0; w >>= 1) {
    dD.x += __shfl_xor_sync(0xffffffffu, dD.x, w);
    dD.y += __shfl_xor_sync(0xffffffffu, dD.y, w);
    dbias.x += __shfl_xor_sync(0xffffffffu, dbias.x, w);
    dbias.y += __shfl_xor_sync(0xffffffffu, dbias.y, w);
  }
  const int64_t out = (group * a.B + p.b) * a.D + p.d;
#pragma unroll
  for (int c = 0; c < 2; ++c)
    if (c < p.have) {
      *reinterpret_cast<ulonglong2*>(ws + l.dA + (out + c) * C::kNP + p.n0) =
          make_ulonglong2(dA[c][0], dA[c][1]);
      if (p.q == 0) {
        ws[l.dD + out + c] = c ? dD.y : dD.x;
        ws[l.dbias + out + c] = c ? dbias.y : dbias.x;
      }
    }
}

// Rows of `width` values summed over `parts`: a warp's lanes hold neighbouring
// values, a block's eight warps an eighth of the parts each.
__device__ __forceinline__ float sum_parts(const float* from, int64_t width, int64_t at,
                                           int64_t parts, float (&sh)[8][32]) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  float v = 0.f;
  if (at < width) {
#pragma unroll 8
    for (int64_t p = warp; p < parts; p += 8) v += from[p * width + at];
  }
  __syncthreads();
  sh[warp][lane] = v;
  __syncthreads();
  v = 0.f;
#pragma unroll
  for (int w = 0; w < 8; ++w) v += sh[w][lane];
  return v;
}

// Step 4: the first `first` blocks sum the padded [D,NP] values of dA, the next ones up
// to `second` the D of dDskip and ddelta_bias, the others the terms of dB and dC in the
// places from..to - 1: into place 0, or when `last` into dB and dC.
template <typename E>
__global__ void __launch_bounds__(256)
    scan_bwd_sum_kernel(const __grid_constant__ ScanArgs a, float* ws,
                        const __grid_constant__ Layout l, int64_t first, int64_t second,
                        int from, int to, bool last) {
  __shared__ float sh[8][32];
  const int64_t parts = l.groups * a.B, width = (int64_t)a.D * l.NP;
  const int lane = threadIdx.x & 31;
  if (blockIdx.x < first) {
    const int64_t at = (int64_t)blockIdx.x * 32 + lane, d = at / l.NP, n = at - d * l.NP;
    const float v = sum_parts(ws + l.dA, width, at, parts, sh);
    if (threadIdx.x < 32 && at < width && n < a.N) a.dA[d * a.N + n] = v;
    return;
  }
  if (blockIdx.x < second) {
    const int64_t d = (blockIdx.x - first) * 32 + lane;
    const float v = sum_parts(ws + l.dD, a.D, d, parts, sh);
    const float w = sum_parts(ws + l.dbias, a.D, d, parts, sh);
    if (threadIdx.x < 32 && d < a.D) {
      if (a.dDskip) a.dDskip[d] = v;
      if (a.ddelta_bias) a.ddelta_bias[d] = w;
    }
    return;
  }
  const int64_t i = (blockIdx.x - second) * 256 + threadIdx.x;
  const int64_t rows = a.B * a.T * a.G, quads = 2 * l.NP / 4;
  if (i >= rows * quads) return;
  const int64_t row = i / quads;
  const int w = (int)(i - row * quads), n0 = w * 4 % (int)l.NP;
  const int64_t bt = row / a.G, b = bt / a.T;
  float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
  if (bt - b * a.T < row_length(a.lengths, b, a.T)) {
    const float* terms = ws + l.dbc + i * 4;
#pragma unroll 8
    for (int64_t p = from; p < to; ++p) {
      const float4 e = *reinterpret_cast<const float4*>(terms + p * rows * 2 * l.NP);
      v.x += e.x, v.y += e.y, v.z += e.z, v.w += e.w;
    }
    if (!last) *reinterpret_cast<float4*>(ws + l.dbc + i * 4) = v;
  }
  if (!last) return;
  E* out = static_cast<E*>(w * 4 < l.NP ? a.dB : a.dC) + row * a.N + n0;
  const float f[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int k = 0; k < 4; ++k)
    if (n0 + k < a.N) store_vec<E, 1>(out + k, FloatV<1>{{f[k]}});
}

template <typename E, int LN>
cudaError_t bwd_lanes(const ScanArgs& a, cudaStream_t stream) {
  typedef Cfg<LN> C;
  const Layout l(a.B, a.T, a.D, a.G, a.N);
  float* ws = static_cast<float*>(a.ws);
  const int bc = kChunk * 2 * C::kNP * 4;
  const int bytes1 = bc + C::kWarps * (int)sizeof(WarpShared<LN>);
  const int bytes3 = bytes1 + C::kWarps * (int)sizeof(GradShared<LN>);
  static std::atomic<uint64_t> done1, done3;
  cudaError_t e = allow_shared(scan_bwd_chunk_kernel<E, LN>, bytes1, &done1);
  if (e == cudaSuccess) e = allow_shared(scan_bwd_grad_kernel<E, LN>, bytes3, &done3);
  if (e != cudaSuccess) return e;
  const int64_t blocks = a.G * l.parts;
  if (blocks * l.chunks > 0x7fffffffLL) return cudaErrorInvalidValue;
  const dim3 chunks((unsigned)(blocks * l.chunks), (unsigned)a.B);
  if (l.chunks > 0) {
    scan_bwd_chunk_kernel<E, LN><<<chunks, C::kWarps * 32, bytes1, stream>>>(a, ws, l);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
  }
  const int64_t quads = (int64_t)a.D * LN;
  scan_bwd_chain_kernel<<<dim3((unsigned)((quads + 127) / 128), (unsigned)a.B, 2), 128, 0,
                          stream>>>(a, ws, l);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  const int64_t terms = (a.B * a.T * a.G * 2 * LN + 255) / 256;
  for (int64_t part0 = 0; part0 < l.parts; part0 += l.at_once) {
    const int parts = (int)(l.parts - part0 < l.at_once ? l.parts - part0 : l.at_once);
    if (l.chunks > 0) {
      const dim3 groups((unsigned)(a.G * parts * l.groups), (unsigned)a.B);
      scan_bwd_grad_kernel<E, LN>
          <<<groups, C::kWarps * 32, bytes3, stream>>>(a, ws, l, (int)part0, parts);
      if ((e = cudaGetLastError()) != cudaSuccess) return e;
    }
    const bool last = part0 + parts == l.parts;
    const int64_t first = last ? ((int64_t)a.D * l.NP + 31) / 32 : 0;
    const int64_t second = last ? first + (a.D + 31) / 32 : 0;
    const int from = part0 > 0 ? 0 : (int)l.place0, to = (int)l.place0 + parts;
    if (second + terms > 0)
      scan_bwd_sum_kernel<E><<<(unsigned)(second + terms), 256, 0, stream>>>(a, ws, l, first,
                                                                            second, from, to, last);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
  }
  return cudaSuccess;
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

cudaError_t launch_scan_bwd(const ScanArgs& in, cudaStream_t stream) {
  ScanArgs a = in;
  scan_access(&a);
  // the dense outputs' pairs as well
  const int pair = a.dtype == FALCON_BF16 ? 4 : 8;
  for (const void* p : {(const void*)a.du, (const void*)a.ddelta, (const void*)a.dz})
    a.vec_ch = a.vec_ch && reinterpret_cast<uintptr_t>(p) % pair == 0;
  return a.dtype == FALCON_BF16 ? bwd_typed<__nv_bfloat16>(a, stream)
                                : bwd_typed<float>(a, stream);
}

}  // namespace falcon
