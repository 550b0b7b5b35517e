// Selective scan over prompts:
//   s_t = softplus(delta_t + bias),  h_t = exp(s_t A) h_{t-1} + s_t u_t B_t,
//   y_t = (<C_t, h_t> + Dskip u_t) silu(z_t)
// for every channel with its N states.
//
// A warp owns 2 * 32 / LN channels: LN lanes share two channels, NS states each,
// in registers, and walk the tokens two at a time: the exponents of tokens t and
// t + 1, s u B, and <C, h> are f32x2 operations on the pair (A is kept doubled), only
// h_t = a_t h_{t-1} + b_t runs token by token.  Pairs of tokens need no copies of
// a value into both halves and no sum of the halves, which pairs of states do.
//
// Tokens come in tiles: a lane turns u and delta of its channel pair and token pair
// into s and s u in shared memory, where the LN lanes of the channels read them; B and
// C lie there in fp32, by token pairs.  While a tile runs, the next one's softplus
// and gates are computed in registers (they fill the waits of the recurrence) and the
// loads of the one after it are in flight.  Two channels a lane, because every lane reads
// B_t and C_t of its states: shared memory delivers 128 bytes a clock to an SM, so one
// channel a lane would be held at 16 states a clock by these reads alone, below the 32
// that the exponential unit does.  <C_t, h_t> is summed over the LN lanes for LN token
// pairs at a time, halving the tokens a lane keeps at each exchange, so that a lane ends
// with the tokens it stores.
//
// B8 T2048 D2048 N16 bf16: 229 us (1.18 TB/s); 40 us would move its bytes and 57 us run its
// exponentials.  With 1.6 warps a scheduler the issue slots are 57% busy, shared
// memory 59%, the exponential unit 30%: bound by the latency of a warp's own chain;
// with four times the rows the same work takes 188 us.  Measured and not kept: a second
// warp a block for loads and gates (275 us), scalar instead of paired arithmetic (250),
// the loop unrolled by two tiles (252, instruction cache), eight tokens a tile ahead of a
// split walk (1.50 ms for T 65536 instead of 1.35).
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

// sigmoid() with its exponent held at 128, which changes no gate (2^128 is infinite) but
// the kernel's registers with bf16 and N = 16: 127, and 130 without, with which 32 x 512
// tokens of 2048 channels take 199 us instead of 188.
__device__ __forceinline__ float gate_sigmoid(float x) {
  return rcp_approx(1.f + exp2_approx(fminf(-x * kLog2e, 128.f)));
}

template <int LN, int NS, bool SPLIT>
struct Cfg {
  static constexpr int kGroups = 32 / LN;        // channel pairs of a warp
  static constexpr int kChannels = 2 * kGroups;  // channels of a warp
  // Tokens of a tile.  With N = 16 and many rows, 8 of them leave registers for twice the
  // warps (187 us for 32 x 512 x 2048 tokens and channels, 241 with 16); a split walk
  // has few warps and gains from the longer tile (T 65536: 1.35 ms, 1.50 with 8).
  static constexpr int kTile = LN <= 2 ? 8 : LN == 4 ? (SPLIT ? 16 : 8) : LN == 8 ? 16 : 32;
  static constexpr int kItems = kTile / 2 / LN;  // (token pair, channel pair) items of a lane
  static constexpr int kNP = NS * LN;            // states, padded
  // rows of steps and gains: padded so that the eight lanes of a store phase (LN
  // token pairs of their channel pairs) fall in different banks
  static constexpr int kRow = kGroups + (LN == 1 ? 0 : LN == 2 ? 4 : LN == 4 ? 2 : 1);
  static constexpr int kNQ = kNP / 4;
  static constexpr int kUnits = kTile * kNQ;     // (token pair, B or C, quad of states)
  static constexpr int kLaneUnits = (kUnits + 31) / 32;
  static constexpr bool kAhead = kLaneUnits <= 4;  // the next tile's quads wait in registers
  static_assert(kItems >= 1 && NS % 4 == 0, "tile");
};

template <typename E, int LN, int NS, bool SPLIT>
__global__ void __launch_bounds__(32) scan_fwd_kernel(const __grid_constant__ ScanArgs a) {
  typedef Cfg<LN, NS, SPLIT> C;
  typedef typename Raw<E>::Pair Pair;
  typedef typename Raw<E>::Quad Quad;
  __shared__ __align__(16) float bc[C::kTile / 2][2][C::kNP][2];
  __shared__ float4 steps[C::kTile / 2][C::kRow];  // s: channel 0 at t, t+1, channel 1
  __shared__ float4 gains[C::kTile / 2][C::kRow];  // s u
  __shared__ __align__(16) float end_h[SPLIT ? C::kChannels : 1][C::kNP];
  __shared__ float2 end_s[SPLIT ? C::kGroups : 1];

  const int lane = threadIdx.x, pair = lane / LN, q = lane % LN, n0 = q * NS;
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

  f32x2 A2[2][NS];
  float h[2][NS], first[2][NS], bias[2], skip[2];
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    const bool live = c < have;
#pragma unroll
    for (int i = 0; i < NS; ++i) {
      const bool in = live && n0 + i < a.N;
      const float v = in ? rate_log2(a.A[(int64_t)(d + c) * a.N + n0 + i]) : 0.f;
      A2[c][i] = opaque2(pack2(v, v));
      first[c][i] = in && a.h0 ? a.h0[(b * a.D + d + c) * a.N + n0 + i] : 0.f;
    }
    bias[c] = live && a.delta_bias ? a.delta_bias[d + c] : 0.f;
    skip[c] = live && a.Dskip ? a.Dskip[d + c] : 0.f;
  }
  // every lane's channels and states exist: no access needs a test of its own
  const bool whole = a.fast && a.N == C::kNP &&
                     (blk - g * blocks + 1) * C::kChannels <= R;
  const bool has_z = a.z != nullptr;
  const E* u = static_cast<const E*>(a.u) + b * a.us.batch;
  const E* dl = static_cast<const E*>(a.delta) + b * a.ds.batch;
  const E* z = static_cast<const E*>(a.z) + (has_z ? b * a.zs.batch : 0);
  const E* Bm = static_cast<const E*>(a.Bm) + b * a.bs.batch + g * a.bs.head;
  const E* Cm = static_cast<const E*>(a.Cm) + b * a.cs.batch + g * a.cs.head;
  E* y = static_cast<E*>(a.y) + b * a.ys.batch;

  // A tile's inputs on their way: this lane's items and its units of B and C.
  struct Ahead {
    Pair u[C::kItems][2], dl[C::kItems][2], z[C::kItems][2];
    Quad bc[C::kAhead ? C::kLaneUnits : 1][2];
  };
  // quads of unit i (of the tile's) at its two tokens
  auto load_unit = [&](int64_t t0, int i, bool full, Quad (&v)[2]) {
    const int tp = i / (2 * C::kNQ), w = i % (2 * C::kNQ), s = w % C::kNQ * 4;
    const bool isB = w < C::kNQ;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int k = 2 * tp + e;
      if (full) {
        const E* p = isB ? Bm + t0 * a.bs.time : Cm + t0 * a.cs.time;
        const unsigned off = (unsigned)(k * (int)(isB ? a.bs.time : a.cs.time) + s);
        v[e] = *reinterpret_cast<const Quad*>(p + off);
      } else {
        const int64_t t = t0 + k;
        const E* p = isB ? Bm + t * a.bs.time : Cm + t * a.cs.time;
        v[e] = load_quad<E>(p + s, a.vec_bc, t < end ? a.N - s : 0);
      }
    }
  };
  auto fetch = [&](int64_t t0, bool gate, Ahead& r) {
    const bool full = whole && t0 + C::kTile <= end;
    if (full) {
      const E *pu = u + t0 * a.us.time, *pd = dl + t0 * a.ds.time, *pz = z + t0 * a.zs.time;
#pragma unroll
      for (int i = 0; i < C::kItems; ++i)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int k = 2 * (i * LN + q) + e;
          r.u[i][e] = *reinterpret_cast<const Pair*>(pu + (unsigned)(k * (int)a.us.time + d));
          r.dl[i][e] = *reinterpret_cast<const Pair*>(pd + (unsigned)(k * (int)a.ds.time + d));
          if (gate)
            r.z[i][e] = *reinterpret_cast<const Pair*>(pz + (unsigned)(k * (int)a.zs.time + d));
        }
    } else {
#pragma unroll
      for (int i = 0; i < C::kItems; ++i)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int64_t t = t0 + 2 * (i * LN + q) + e;
          const int k = t < end ? have : 0;
          r.u[i][e] = load_pair<E>(u + t * a.us.time + d, a.vec_ch, k);
          r.dl[i][e] = load_pair<E>(dl + t * a.ds.time + d, a.vec_ch, k);
          if (gate) r.z[i][e] = load_pair<E>(z + t * a.zs.time + d, a.vec_ch, k);
        }
    }
    if (C::kAhead) {
#pragma unroll
      for (int i = 0; i < C::kLaneUnits; ++i)
        if (C::kUnits % 32 == 0 || i * 32 + lane < C::kUnits)
          load_unit(t0, i * 32 + lane, full, r.bc[C::kAhead ? i : 0]);
    }
  };
  // What a tile needs of this lane's items: s and s u for the recurrence, the gate
  // and its product with the skip term for the output.  Without branches, so that it
  // shares a basic block with the tile before it and fills that one's waits.
  struct Ready {
    float4 s[C::kItems], v[C::kItems], gate[C::kItems], skip[C::kItems];
  };
  auto prepare = [&](int64_t t0, bool gate, const Ahead& r, Ready& o) {
#pragma unroll
    for (int i = 0; i < C::kItems; ++i) {
      float2 s[2], v[2], g[2], k[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float2 ut = widen(r.u[i][e]), zt = widen(r.z[i][e]);
        const float2 x = unpack2(add2(pair2(widen(r.dl[i][e])), pack2(bias[0], bias[1])));
        const float2 sp = softplus2(x);
        const bool in = t0 + 2 * (i * LN + q) + e < end;
        s[e].x = in ? (a.softplus ? sp.x : x.x) : 0.f;
        s[e].y = in ? (a.softplus ? sp.y : x.y) : 0.f;
        v[e] = unpack2(mul2(pair2(s[e]), pair2(ut)));
        const float2 sg = make_float2(gate_sigmoid(zt.x), gate_sigmoid(zt.y));
        const float2 silu = unpack2(mul2(pair2(zt), pair2(sg)));
        g[e] = make_float2(gate ? silu.x : 1.f, gate ? silu.y : 1.f);
        k[e] = unpack2(mul2(mul2(pack2(skip[0], skip[1]), pair2(ut)), pair2(g[e])));
      }
      o.s[i] = make_float4(s[0].x, s[1].x, s[0].y, s[1].y);
      o.v[i] = make_float4(v[0].x, v[1].x, v[0].y, v[1].y);
      o.gate[i] = make_float4(g[0].x, g[1].x, g[0].y, g[1].y);
      o.skip[i] = make_float4(k[0].x, k[1].x, k[0].y, k[1].y);
    }
  };
  auto put = [&](int64_t t0, const Ahead& r, const Ready& o) {
#pragma unroll
    for (int i = 0; i < C::kItems; ++i) {
      steps[i * LN + q][pair] = o.s[i];
      gains[i * LN + q][pair] = o.v[i];
    }
    const bool full = whole && t0 + C::kTile <= end;
#pragma unroll
    for (int i = 0; i < C::kLaneUnits; ++i) {
      const int k = i * 32 + lane;
      if (C::kUnits % 32 == 0 || k < C::kUnits) {
        Quad now[2];
        if (!C::kAhead) load_unit(t0, k, full, now);
        const float4 v0 = widen(C::kAhead ? r.bc[C::kAhead ? i : 0][0] : now[0]);
        const float4 v1 = widen(C::kAhead ? r.bc[C::kAhead ? i : 0][1] : now[1]);
        float4* to = reinterpret_cast<float4*>(&bc[0][0][0][0] + 8 * k);
        to[0] = make_float4(v0.x, v1.x, v0.y, v1.y);
        to[1] = make_float4(v0.z, v1.z, v0.w, v1.w);
      }
    }
  };

  // One walk over the segment.  OUT: with outputs; otherwise only h and the
  // sum of the steps.
  const f32x2 lift = opaque2(pack2(kDecayLift, kDecayLift));
  float2 sum = make_float2(0.f, 0.f);
  auto add_steps = [&](const Ready& r) {  // steps behind the segment's end are zero
#pragma unroll
    for (int i = 0; i < C::kItems; ++i)
      sum.x += r.s[i].x + r.s[i].y, sum.y += r.s[i].z + r.s[i].w;
  };
  auto walk = [&](auto out) {
    constexpr bool OUT = decltype(out)::value;
    const bool gate = OUT && has_z;
    if (begin >= end) return;
    Ahead next;
#pragma unroll
    for (int i = 0; i < C::kItems; ++i) next.z[i][0] = next.z[i][1] = Pair();
    Ready now;
    fetch(begin, gate, next);
    prepare(begin, gate, next, now);
    put(begin, next, now);
    if (begin + C::kTile < end) fetch(begin + C::kTile, gate, next);
    if (!OUT) add_steps(now);
    __syncwarp();
    for (int64_t t0 = begin; t0 < end; t0 += C::kTile) {
      const int64_t t1 = t0 + C::kTile;
      Ahead after = next;
      if (t1 + C::kTile < end) fetch(t1 + C::kTile, gate, after);
      Ready then;
      prepare(t1, gate, next, then);
      if (!OUT) add_steps(then);
      float4 y2[C::kItems];
#pragma unroll
      for (int i = 0; i < C::kItems; ++i) {
        float2 o[LN][2];  // <C, h> of LN token pairs, two channels, this lane's states
#pragma unroll
        for (int j = 0; j < LN; ++j) {
          const int tp = i * LN + j;
          const ulonglong2 s = *reinterpret_cast<const ulonglong2*>(&steps[tp][pair]);
          const ulonglong2 v = *reinterpret_cast<const ulonglong2*>(&gains[tp][pair]);
          // level by level over the lane's 2 NS chains, so that neighbouring
          // instructions do not wait for one another
          f32x2 Bt[NS], Ct[NS], acc[2];
#pragma unroll
          for (int k = 0; k < NS; k += 2) {
            const ulonglong2 x = *reinterpret_cast<const ulonglong2*>(&bc[tp][0][n0 + k][0]);
            Bt[k] = x.x, Bt[k + 1] = x.y;
            if (OUT) {
              const ulonglong2 w = *reinterpret_cast<const ulonglong2*>(&bc[tp][1][n0 + k][0]);
              Ct[k] = w.x, Ct[k + 1] = w.y;
            }
          }
          float2 at[2][NS], bt[2][NS];
#pragma unroll
          for (int k = 0; k < NS; ++k)
#pragma unroll
            for (int c = 0; c < 2; ++c) at[c][k] = decay2(c ? s.y : s.x, A2[c][k], lift);
#pragma unroll
          for (int k = 0; k < NS; ++k)
#pragma unroll
            for (int c = 0; c < 2; ++c) bt[c][k] = unpack2(mul2(c ? v.y : v.x, Bt[k]));
          float h0[2][NS];
#pragma unroll
          for (int k = 0; k < NS; ++k)
#pragma unroll
            for (int c = 0; c < 2; ++c) h0[c][k] = fmaf(at[c][k].x, h[c][k], bt[c][k].x);
#pragma unroll
          for (int k = 0; k < NS; ++k)
#pragma unroll
            for (int c = 0; c < 2; ++c) h[c][k] = fmaf(at[c][k].y, h0[c][k], bt[c][k].y);
          if (OUT) {
#pragma unroll
            for (int k = 0; k < NS; ++k)
#pragma unroll
              for (int c = 0; c < 2; ++c) {
                const f32x2 hp = pack2(h0[c][k], h[c][k]);
                acc[c] = k == 0 ? mul2(Ct[k], hp) : fma2(Ct[k], hp, acc[c]);
              }
            o[j][0] = unpack2(acc[0]), o[j][1] = unpack2(acc[1]);
          }
        }
        if (OUT) {
#pragma unroll
          for (int w = LN / 2; w > 0; w >>= 1) {
            const bool up = q & w;
#pragma unroll
            for (int j = 0; j < w; ++j)
#pragma unroll
              for (int c = 0; c < 2; ++c) {
                const float2 give = up ? o[j][c] : o[j + w][c], keep = up ? o[j + w][c] : o[j][c];
                o[j][c].x = keep.x + __shfl_xor_sync(0xffffffffu, give.x, w);
                o[j][c].y = keep.y + __shfl_xor_sync(0xffffffffu, give.y, w);
              }
          }
          y2[i] = make_float4(fmaf(o[0][0].x, now.gate[i].x, now.skip[i].x),
                              fmaf(o[0][0].y, now.gate[i].y, now.skip[i].y),
                              fmaf(o[0][1].x, now.gate[i].z, now.skip[i].z),
                              fmaf(o[0][1].y, now.gate[i].w, now.skip[i].w));
        }
      }
      __syncwarp();
      put(t1, next, then);
      if (OUT) {
        E* py = y + t0 * a.ys.time;
        if (whole && t1 <= end) {
#pragma unroll
          for (int i = 0; i < C::kItems; ++i) {
            const int k = 2 * (i * LN + q);
            *reinterpret_cast<Pair*>(py + (unsigned)(k * (int)a.ys.time + d)) =
                narrow(make_float2(y2[i].x, y2[i].z), Pair());
            *reinterpret_cast<Pair*>(py + (unsigned)((k + 1) * (int)a.ys.time + d)) =
                narrow(make_float2(y2[i].y, y2[i].w), Pair());
          }
        } else {
#pragma unroll
          for (int i = 0; i < C::kItems; ++i)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int k = 2 * (i * LN + q) + e;
              if (t0 + k < end)
                store_pair<E>(py + k * a.ys.time + d, a.vec_ch, have,
                              e ? make_float2(y2[i].y, y2[i].w) : make_float2(y2[i].x, y2[i].z));
            }
        }
      }
      now = then;
      next = after;
      __syncwarp();
    }
  };

  if (SPLIT) {
#pragma unroll
    for (int c = 0; c < 2; ++c)
#pragma unroll
      for (int i = 0; i < NS; ++i) h[c][i] = 0.f;
    if (rank + 1 < K) walk(std::false_type());
#pragma unroll
    for (int w = LN / 2; w > 0; w >>= 1) {
      sum.x += __shfl_xor_sync(0xffffffffu, sum.x, w);
      sum.y += __shfl_xor_sync(0xffffffffu, sum.y, w);
    }
    if (q == 0) end_s[pair] = sum;
#pragma unroll
    for (int c = 0; c < 2; ++c)
#pragma unroll
      for (int i = 0; i < NS; i += 4)
        *reinterpret_cast<float4*>(&end_h[pair * 2 + c][n0 + i]) =
            make_float4(h[c][i], h[c][i + 1], h[c][i + 2], h[c][i + 3]);
    cg::this_cluster().sync();
    for (int k = 0; k < rank; ++k) {
      const float2 s = *cg::this_cluster().map_shared_rank(&end_s[pair], k);
#pragma unroll
      for (int c = 0; c < 2; ++c)
#pragma unroll
        for (int i = 0; i < NS; i += 4) {
          const float4 e = *reinterpret_cast<const float4*>(
              cg::this_cluster().map_shared_rank(&end_h[pair * 2 + c][n0 + i], k));
          const float ev[4] = {e.x, e.y, e.z, e.w};
#pragma unroll
          for (int x = 0; x < 4; ++x)
            first[c][i + x] = fmaf(decay(c ? s.y : s.x, unpack2(A2[c][i + x]).x), first[c][i + x],
                                   ev[x]);
        }
    }
    cg::this_cluster().barrier_arrive();  // this warp has read the others' memory
  }
#pragma unroll
  for (int c = 0; c < 2; ++c)
#pragma unroll
    for (int i = 0; i < NS; ++i) h[c][i] = first[c][i];
  walk(std::true_type());

  for (int64_t t = n + rank * LN + q; t < a.T; t += K * LN)
    store_pair<E>(y + t * a.ys.time + d, a.vec_ch, have, make_float2(0.f, 0.f));
  if (rank == K - 1) {
#pragma unroll
    for (int c = 0; c < 2; ++c)
#pragma unroll
      for (int i = 0; i < NS; ++i)
        if (c < have && n0 + i < a.N) a.h_out[(b * a.D + d + c) * a.N + n0 + i] = h[c][i];
  }
  if (SPLIT) cg::this_cluster().barrier_wait();  // until the others have read this one's
}

// Segments of a row's tokens.  A warp alone takes about 80 ns a token, whatever else
// runs, up to about seven warps an SM; beyond that, a split only adds its first walk.
// The rule: the most segments that stay within twelve warps an SM (eight of the split
// kernel's fit at a time), each of two tiles at least, but never just two.  Measured at
// 8192 tokens, N = 16, bf16: 32 warps (512 channels) 68 us with 16 segments, 120 with 8,
// 619 with 1; 128 warps 181 us with 8, 239 with 4, 244 with 16, 732 with 1; 256 warps
// 350 us with 4, 360 with 8, 739 with 1.  Not the best everywhere: 512 warps of 4096
// tokens take 382 us unsplit and 350 with 2; and over 224 shapes (80 to 600 warps, 256 to
// 4096 tokens, 4 to 128 states, both types) the rule is 12% above the best of 1, 2, 4,
// 8 and 16 segments on average and 73% at worst (80 warps of 256 tokens, 42 us with 16
// segments and 24 with 8), where no split at all is 34% and 290% above.
int segments(int64_t warps, int64_t tiles) {
  int K = 1;
  while (K < 16 && warps * K * 2 <= 152 * 12 && tiles >= 4 * K) K *= 2;
  return K == 2 ? 1 : K;
}

template <typename E, int LN, int NS>
cudaError_t fwd_lanes(const ScanArgs& a, cudaStream_t stream) {
  typedef Cfg<LN, NS, true> C;
  const int R = a.D / a.G;
  const int64_t blocks = (int64_t)a.G * ((R + C::kChannels - 1) / C::kChannels);
  const int64_t tiles = (a.T + C::kTile - 1) / C::kTile;
  const int K = segments(blocks * a.B, tiles);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(blocks * K), (unsigned)a.B);
  cfg.blockDim = dim3(32);
  cfg.stream = stream;
  if (K == 1) return cudaLaunchKernelEx(&cfg, scan_fwd_kernel<E, LN, NS, false>, a);
  if (K > 8) {
    const cudaError_t e = cudaFuncSetAttribute(scan_fwd_kernel<E, LN, NS, true>,
                                               cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
  }
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = (unsigned)K;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, scan_fwd_kernel<E, LN, NS, true>, a);
}

template <typename E>
cudaError_t fwd_typed(const ScanArgs& a, cudaStream_t stream) {
  if (a.N <= 4) return fwd_lanes<E, 1, 4>(a, stream);
  if (a.N <= 8) return fwd_lanes<E, 2, 4>(a, stream);
  if (a.N <= 16) return fwd_lanes<E, 4, 4>(a, stream);
  if (a.N <= 32) return fwd_lanes<E, 8, 4>(a, stream);
  if (a.N <= 64) return fwd_lanes<E, 16, 4>(a, stream);
  return fwd_lanes<E, 16, 8>(a, stream);
}

// Whether pointer and strides keep every access of `elems` elements aligned.
bool rows_fit(const void* p, const falcon_strides& s, int elems, int esz) {
  return reinterpret_cast<uintptr_t>(p) % (uintptr_t)(elems * esz) == 0 && s.batch % elems == 0 &&
         s.time % elems == 0 && s.head % elems == 0;
}

}  // namespace

void scan_access(ScanArgs* a) {
  const int esz = a->dtype == FALCON_BF16 ? 2 : 4;
  a->us.head = a->ds.head = a->zs.head = a->ys.head = a->dys.head = 0;  // unused
  a->vec_ch = a->D / a->G % 2 == 0 && rows_fit(a->u, a->us, 2, esz) &&
              rows_fit(a->delta, a->ds, 2, esz) && rows_fit(a->z, a->zs, 2, esz) &&
              rows_fit(a->y, a->ys, 2, esz) && rows_fit(a->dy, a->dys, 2, esz);
  a->vec_bc = a->N % 4 == 0 && rows_fit(a->Bm, a->bs, 4, esz) && rows_fit(a->Cm, a->cs, 4, esz);
  const int64_t most = (0x7fffffffLL - a->D) / 32;
  a->fast = a->vec_ch && a->vec_bc && a->us.time < most && a->ds.time < most &&
            a->zs.time < most && a->ys.time < most && a->dys.time < most && a->bs.time < most &&
            a->cs.time < most;
}

cudaError_t launch_scan_fwd(const ScanArgs& in, cudaStream_t stream) {
  ScanArgs a = in;
  scan_access(&a);
  return a.dtype == FALCON_BF16 ? fwd_typed<__nv_bfloat16>(a, stream)
                                : fwd_typed<float>(a, stream);
}

}  // namespace falcon
