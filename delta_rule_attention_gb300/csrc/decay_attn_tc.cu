// Attention with a fixed decay a head on the tensor cores (tcgen05): bf16 activations
// whose rows TMA can read.  The same three steps as decay_attn.cu, in chunks of 128 tokens:
//
//   states: per 128 tokens of a run, D[key][value] += (Diag(w) K)^T V in TMEM, where w_j is
//     gamma to the number of tokens behind j in the run.  The weighted keys are split
//     into three bf16 terms (their sum has the 24 bits of fp32), so that a state
//     carries fp32's precision although the operands are bf16.
//   join: decay_attn.cu.
//   reads: per chunk, P = Q K^T and O = Q X (X the state entering the chunk, rounded to
//     bf16); P is weighted by gamma^{i-j}, masked, rounded to bf16 and put back into TMEM
//     as an operand, O is weighted by gamma^{i+1} in TMEM; O += P V and, where another
//     chunk of the run follows, X' = gamma^len X + (Diag(w) K)^T V with two terms.
//
// Rounding.  What a run adds and the states between runs (S_T, the gradient's dS0) are
// fp32.  An output is a sum of terms that are rounded once to bf16, as operands of a
// product (a weighted q k, or an entry of the state read), and is rounded once itself:
// 2.3e-3 of its norm off, against 1.7e-3 of the one rounding that fp32 throughout would
// leave.  Two terms for both operands would leave that one, for twice the products D and B
// and 32 KB more of shared memory with 128 x 128, which is not there.  The state carried from
// chunk to chunk inside a run has 16 bits of a weighted key (two terms), and what the tensor
// cores cut off in adding to it (kDecayTcRun): below 1e-4 of an output together.  In the
// gradient the same holds of dO v^T and v dO^T, with S and G in the state's place.
//
// Keys of up to 64 (M = 64) and up to 128 channels (M = 128), values likewise (N): TMA
// fills the missing channels with zeros.  All accumulators have 128 lanes; for N = 64 the
// second half of V^T as an A operand is the tile behind it in shared memory, which lands
// in lanes 64..127 that nobody reads.
//
// Measured (96 heads of 64, 2048 tokens; 16 heads of 128, 65536 tokens): a call 51 us, of
// which the states take 18 and the reads 28 (floor of the call's bytes: 15); 291 us, 99 and
// 175 (158).  The states are bound by shared memory, through which three terms of every
// key go to the tensor cores.  The reads of 64 channels take 8 us for the launch's start and
// end, 1.7 us (3500 cycles) a chunk, where memory needs 1.5, and 1.1 for a block's second
// run: the chain from one chunk's state to the next is about as long as memory takes.
// One block an SM whose warps have roles took the place
// of two blocks an SM that went through the phases together: 68 us and 609.
#include <cuda_bf16.h>

#include "linear.cuh"
#include "linear_tc.cuh"
#include "tc_ptx.cuh"
#include "tc_util.cuh"
#include "tmap.cuh"

namespace falcon {
namespace {

using namespace tc;
using tcu::align1024;
using tcu::flag_error;

constexpr int kC = 128;                // tokens of a chunk
constexpr uint32_t kTile = kC * 128;   // a chunk of 64 channels

// A block's warps: two groups of eight that work on rows (a warp's TMEM lanes are its
// number modulo 4, its half of the columns or channels the bit above), one warp that loads
// and one or two that issue the products.
constexpr int kStateThreads = 576, kReadThreads = 608;
constexpr int kLoader = 16, kIssuer = 17;

struct TcArgs {
  DecayPass p;
  int* err;
  int items;  // runs of all heads
  int wide_o;  // output rows lie on 32-byte boundaries
  // 0 where the tensor is broadcast along heads or batches
  int qh, qb, kh, kb, vh, vb;
};
struct TcMaps {
  CUtensorMap q, k, v;    // boxes of 128 tokens
  CUtensorMap ks, vs;     // of the states' chunks
};

// Barriers of a block.  A wait that gave up sets `fail`, after which nobody waits.
template <int BARS>
struct Control {
  uint64_t bar[BARS];
  uint32_t tmem;
  volatile int fail;
};
// The part that waits is not inlined: the roles of a block run side by side, and with
// everything unrolled their code did not fit the instruction cache (most of the warps'
// time went into fetching it).
__device__ __noinline__ void wait_on(uint64_t* bar, uint32_t parity, volatile int* fail) {
  if (!*fail && !mbar_wait(bar, parity)) *fail = 1;
}
template <int BARS>
__device__ __forceinline__ void wait(Control<BARS>& c, int which, uint32_t phase) {
  if (!mbar_try_wait(&c.bar[which], phase & 1)) wait_on(&c.bar[which], phase & 1, &c.fail);
}
// The same for all lanes of a warp, which go on together.
template <int BARS>
__device__ __forceinline__ void wait_warp(Control<BARS>& c, int which, uint32_t phase) {
  wait(c, which, phase);
  __syncwarp();
}
// A warp's part of a barrier that counts warps.
template <int BARS>
__device__ __forceinline__ void arrive_warp(Control<BARS>& c, int which) {
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(&c.bar[which]);
}

// At a block's end: the last phases of a ring of barriers that n uses went through.  Copies
// and the arrivals that products send are asynchronous, and the shared memory that they
// come to is the next block's once this one has ended.  After a wait that gave up, what is
// on its way still gets a while to land.
constexpr uint64_t kSettleNs = 10000000ull;
template <int BARS>
__device__ __forceinline__ void settle(Control<BARS>& c, int ring, int stages, int n) {
#pragma unroll 1
  for (int s = 0; s < stages && s < n; ++s)
    if (!mbar_wait(&c.bar[ring + s], last_phase(n, stages, s) & 1,
                   c.fail ? kSettleNs : kWaitLimitNs))
      c.fail = 1;
}

// a and b (of x) as sums of two or three bf16 terms.  All but the last of two are cut
// off, not rounded: each takes 8 of the 24 bits, so that three are exact.
__device__ __forceinline__ uint32_t upper_halves(float a, float b) {
  return __byte_perm(__float_as_uint(a), __float_as_uint(b), 0x7632);
}
__device__ __forceinline__ float2 rest_of(float2 x) {
  const f32x2 cut = pack2(-__uint_as_float(__float_as_uint(x.x) & 0xffff0000u),
                          -__uint_as_float(__float_as_uint(x.y) & 0xffff0000u));
  return unpack2(add2(pair2(x), cut));
}
__device__ __forceinline__ void split2(float2 x, uint32_t& hi, uint32_t& mid) {
  hi = upper_halves(x.x, x.y);
  const float2 r = rest_of(x);
  mid = pack_bf16(r.x, r.y);
}
__device__ __forceinline__ void split3(float2 x, uint32_t& hi, uint32_t& mid, uint32_t& lo) {
  hi = upper_halves(x.x, x.y);
  const float2 r = rest_of(x);
  mid = upper_halves(r.x, r.y);
  const float2 q = rest_of(r);
  lo = upper_halves(q.x, q.y);
}

// 16-byte chunk c of row r of a swizzled tile.
__device__ __forceinline__ unsigned char* chunk_of(unsigned char* tile, int r, int c) {
  return tile + r * 128 + ((c ^ (r & 7)) << 4);
}

// CHUNKS 16-byte chunks from `first` on of row r of every 64 keys, times w: the first
// term, in place or elsewhere, and those behind it.  Tiles are TILE bytes apart.
template <int ATOMS, int TERMS, int CHUNKS, uint32_t TILE>
__device__ __forceinline__ void weigh_keys(unsigned char* k, unsigned char* hi,
                                           unsigned char* mid, unsigned char* lo, int r,
                                           int first, float w) {
  const f32x2 w2 = pack2(w, w);
#pragma unroll 1
  for (int at = 0; at < ATOMS; ++at)
#pragma unroll 2
    for (int cc = 0; cc < CHUNKS; ++cc) {
      const int c = first + cc;
      const uint4 x = *reinterpret_cast<const uint4*>(chunk_of(k + at * TILE, r, c));
      const uint32_t in[4] = {x.x, x.y, x.z, x.w};
      uint32_t t[3][4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 y = unpack2(mul2(pack2(bf16_lo(in[e]), bf16_hi(in[e])), w2));
        if constexpr (TERMS == 3)
          split3(y, t[0][e], t[1][e], t[2][e]);
        else
          split2(y, t[0][e], t[1][e]);
      }
      *reinterpret_cast<uint4*>(chunk_of(hi + at * TILE, r, c)) =
          make_uint4(t[0][0], t[0][1], t[0][2], t[0][3]);
      *reinterpret_cast<uint4*>(chunk_of(mid + at * TILE, r, c)) =
          make_uint4(t[1][0], t[1][1], t[1][2], t[1][3]);
      if constexpr (TERMS == 3)
        *reinterpret_cast<uint4*>(chunk_of(lo + at * TILE, r, c)) =
            make_uint4(t[2][0], t[2][1], t[2][2], t[2][3]);
    }
}

template <int ATOMS, int CHUNKS = 4, uint32_t TILE = kTile>
__device__ __forceinline__ void clear_row(unsigned char* tile, int r, int first) {
#pragma unroll 1
  for (int at = 0; at < ATOMS; ++at)
#pragma unroll 1
    for (int c = 0; c < CHUNKS; ++c)
      *reinterpret_cast<uint4*>(chunk_of(tile + at * TILE, r, first + c)) = make_uint4(0, 0, 0, 0);
}

// The issuing warp stays together (what it computes is then the same in all lanes, and
// an operand's description costs one addition); one lane sends the products: sent by a
// lane that runs by itself, a product of 128 x 64 x 16 took about 90 cycles, most of them
// for its description.
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile(
      "{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}" : "=r"(r));
  return r != 0;
}
// Low word of a tile's description (the address moves by bytes / 16); the high word says
// 1024 bytes between groups of eight rows, and the 128-byte swizzle.
__device__ __forceinline__ uint32_t desc_low(uint32_t saddr, uint32_t lbo) {
  return (saddr >> 4) | (lbo >> 4) << 16;
}
constexpr uint32_t kDescHigh = (1024 >> 4) | 1u << 14 | 2u << 29;
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc,
                                       bool accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n .reg .b64 x, y;\n setp.ne.b32 p, %4, 0;\n mov.b64 x, {%1, %5};\n"
      " mov.b64 y, {%2, %5};\n tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, p;\n}" ::"r"(d),
      "r"(a), "r"(b), "r"(idesc), "r"((uint32_t)accumulate), "n"(kDescHigh)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a_tmem, uint32_t b, uint32_t idesc,
                                       bool accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n .reg .b64 y;\n setp.ne.b32 p, %4, 0;\n mov.b64 y, {%2, %5};\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], y, %3, p;\n}" ::"r"(d),
      "r"(a_tmem), "r"(b), "r"(idesc), "r"((uint32_t)accumulate), "n"(kDescHigh)
      : "memory");
}

// D (+)= A^T B over the C tokens of tiles [token][channel]; N channels of B.
template <int N, int C = kC>
__device__ __forceinline__ void mma_tokens(uint32_t d, uint32_t a, uint32_t b, bool accumulate) {
  const uint32_t da = desc_low(a, C * 128), db = desc_low(b, C * 128);
#pragma unroll
  for (int ks = 0; ks < C / 16; ++ks)
    mma_ss(d, da + ks * kStepMN, db + ks * kStepMN, idesc_bf16(128, N, true, true),
           accumulate || ks > 0);
}

// A run of one head: where its tokens lie.
struct Item {
  int64_t bh;
  int run, b, h, n, first, end, chunks;  // chunks that hold tokens
  float g;
  __device__ __forceinline__ Item(const DecayPass& p, int item) {
    const unsigned head = (unsigned)item / (unsigned)p.runs, heads = (unsigned)p.H;
    run = item - (int)head * p.runs;
    bh = head;
    b = (int)(head / heads), h = (int)(head - b * heads);
    n = (int)row_length(p.lengths, b, p.T);
    first = (int)(run * p.run_len);
    end = (int)(first + p.run_len < p.T ? first + p.run_len : p.T);
    const int left = min(n, end) - first;
    chunks = left > 0 ? (left + kC - 1) / kC : 0;
    g = decay_rate(p.log_decay, h);
  }
};

// ---- states -----------------------------------------------------------------
// D[value][key] = V^T (Diag(w) K), so that the three terms of a key share a thread's
// lane.  Shared memory's bandwidth is what these products take (4 KB of A and 32 bytes a
// column of B for 16 tokens): terms lie side by side and one product takes as many of them
// as it can, all three with 64 keys, the smaller two with 128.
//
// The tensor cores add into an accumulator without rounding to nearest: over a long run
// the error grows with the number of additions (1.3e-5 of a state of 65536 tokens at a rate
// of 2^-12).  So sums are taken out after every 256 tokens and added in registers; with
// 128 keys only the first term's, the other two, smaller by 2^8 and 2^16, stay in TMEM
// for the whole run.
//
// Sixteen warps weigh and split the keys of a chunk while the products of the chunk before
// run; the same warps take out the sums.  (Two sets of eight, a chunk each: 20.7 us for
// 18.7.)
template <int M, int N>
struct StatePlan {
  static constexpr bool kSide = M == 64;            // terms side by side
  static constexpr int kTokens = kSide ? 128 : 64;  // of a chunk here
  static constexpr int kGroup = 256 / kTokens;      // chunks whose sums stay in TMEM
  static constexpr uint32_t kTile = kTokens * 128;
  static constexpr uint32_t kK = M / 64 * kTile, kV = N / 64 * kTile;
  static constexpr int kStages = M + N == 192 && kSide ? 2 : 4;
  static constexpr uint32_t kT = (kSide ? 3 : 2) * kK;  // a chunk's terms
  static constexpr uint32_t V = 0, K = kStages * kV, T = K + kStages * kK;
  static constexpr uint32_t kBytes = T + 2 * kT + 1024;
  // TMEM columns: two groups' sums, and with 128 keys the smaller terms' two
  static constexpr uint32_t kSumCols = kSide ? 3 * M : M, kCols = 512;
  static constexpr int kFull = 0, kEmpty = kStages, kSplit = 2 * kStages,
                       kSplitFree = kSplit + 2, kSum = kSplit + 4, kSumFree = kSplit + 6,
                       kBars = kSplit + 8;
};

// Chunks [from, to) of a run whose weights are not all zero in fp32 (e^-104 is).
template <int C>
__device__ __forceinline__ void weighed_chunks(const Item& it, bool rev, int len, int* from,
                                               int* to) {
  *from = 0, *to = (len + C - 1) / C;
  if (!(it.g < 0.f)) return;
  const float reach = -104.f / it.g;
  if (!(reach < (float)len)) return;
  const int tokens = (int)reach + 2;
  if (rev)
    *to = min(*to, (tokens + C - 1) / C);
  else
    *from = max(0, len - tokens) / C;
}

template <int M, int N>
__global__ void __launch_bounds__(kStateThreads, 1)
    decay_states_tc(const __grid_constant__ TcArgs a, const __grid_constant__ TcMaps maps) {
  using L = StatePlan<M, N>;
  extern __shared__ unsigned char raw[];
  __shared__ Control<L::kBars> ctl;
  unsigned char* sm = align1024(raw);
  const DecayPass& p = a.p;
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  if (tid == 0) {
    for (int i = 0; i < L::kStages; ++i)
      mbar_init(&ctl.bar[L::kFull + i], 1), mbar_init(&ctl.bar[L::kEmpty + i], 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&ctl.bar[L::kSplit + i], 16), mbar_init(&ctl.bar[L::kSplitFree + i], 1);
      mbar_init(&ctl.bar[L::kSum + i], 1), mbar_init(&ctl.bar[L::kSumFree + i], 16);
    }
    ctl.fail = 0;
    fence_mbar_init();
  }
  if (warp == 0) tmem_alloc(&ctl.tmem, L::kCols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, ctl.tmem, 0), base = smem_addr(sm);
  constexpr int C = L::kTokens;
  // behind the pass before, which reads the states that this one writes
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  int c = 0, group = 0;  // chunks, and groups of them, of all items so far
  int loaded = 0;        // chunks that were copied
  for (int item = blockIdx.x; item < a.items; item += gridDim.x) {
    const Item it(p, item);
    const int len = max(min(it.n, it.end) - it.first, 0);
    int from, to;
    weighed_chunks<C>(it, p.rev, len, &from, &to);
    if (warp < 16) {
      constexpr int kOwn = M / 4;  // keys of a thread's sums
      const int j = 32 * (warp & 3) + lane, i0 = (warp >> 2) * kOwn;
      const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
      // a row of the keys, and the 16-byte chunks of it that this thread splits
      constexpr int kChunks = 8 * C / 512;
      const int r = tid & (C - 1), first = tid / C * kChunks;
      float sum[kOwn];
#pragma unroll
      for (int i = 0; i < kOwn; ++i) sum[i] = 0.f;
      auto add = [&](uint32_t col) {
        float x[kOwn];
        if constexpr (kOwn == 32)
          tmem_ld32(tmem + lanes + col + i0, x);
        else
          tmem_ld16(tmem + lanes + col + i0, x);
#pragma unroll
        for (int i = 0; i < kOwn; ++i) sum[i] += x[i];
      };
      auto take_out = [&](bool last) {
        const int g = group & 1;
        wait_warp(ctl, L::kSum + g, group >> 1);
        ++group;
        tc_fence_after();
        // the smallest first
        if constexpr (L::kSide) {
          add(g * L::kSumCols + 2 * M);
          add(g * L::kSumCols + M);
        } else if (last) {
          add(2 * L::kSumCols + M);
          add(2 * L::kSumCols);
        }
        add(g * L::kSumCols);
        tc_fence_before();
        arrive_warp(ctl, L::kSumFree + g);
      };
      for (int k = from; k < to; ++k, ++c) {
        const int s = c % L::kStages, t = c & 1, at = k * C + r;
        const float w = p.w * decay_power(it.g, (float)(p.rev ? at + 1 : len - 1 - at));
        unsigned char* key = sm + L::K + s * L::kK;
        unsigned char* terms = sm + L::T + t * L::kT;
        unsigned char* hi = L::kSide ? terms : key;
        unsigned char* mid = L::kSide ? terms + L::kK : terms;
        wait_warp(ctl, L::kFull + s, c / L::kStages);
        if (c >= 2) wait_warp(ctl, L::kSplitFree + t, (c >> 1) - 1);
        if (at < len) {
          weigh_keys<M / 64, 3, kChunks, L::kTile>(key, hi, mid, mid + L::kK, r, first, w);
        } else {  // rows that the sequence does not hold
          clear_row<M / 64, kChunks, L::kTile>(hi, r, first);
          clear_row<M / 64, kChunks, L::kTile>(mid, r, first);
          clear_row<M / 64, kChunks, L::kTile>(mid + L::kK, r, first);
          clear_row<N / 64, kChunks, L::kTile>(sm + L::V + s * L::kV, r, first);
        }
        fence_async_smem();
        arrive_warp(ctl, L::kSplit + t);
        if (k > from && (k - from) % L::kGroup == 0) take_out(false);  // the group before
      }
      if (to > from) take_out(true);
      float* out = p.states + (it.bh * p.runs + it.run) * p.m * p.dv + j;
      if (j < p.dv) {
#pragma unroll
        for (int i = 0; i < kOwn; ++i)
          if (i0 + i < p.m) out[(i0 + i) * p.dv] = sum[i];
      }
    } else if (warp == kLoader) {
      for (int k = from; k < to; ++k, ++c) {
        const int s = c % L::kStages, t = it.first + k * C;
        if (lane != 0) continue;
        if (c >= L::kStages) wait(ctl, L::kEmpty + s, c / L::kStages - 1);
        if (ctl.fail) continue;
        loaded = c + 1;
        uint64_t* bar = &ctl.bar[L::kFull + s];
        mbar_expect_tx(bar, L::kK + L::kV);
#pragma unroll
        for (int i = 0; i < M / 64; ++i)
          tma_load_4d(sm + L::K + s * L::kK + i * L::kTile, &maps.ks, 64 * i, t, it.h * a.kh,
                      it.b * a.kb, bar);
#pragma unroll
        for (int i = 0; i < N / 64; ++i)
          tma_load_4d(sm + L::V + s * L::kV + i * L::kTile, &maps.vs, 64 * i, t, it.h * a.vh,
                      it.b * a.vb, bar);
      }
    } else {
      for (int k = from; k < to; ++k, ++c) {
        const int s = c % L::kStages, t = c & 1, g = group & 1;
        const bool opens = (k - from) % L::kGroup == 0;
        wait_warp(ctl, L::kSplit + t, c >> 1);
        if (opens && group >= 2) wait_warp(ctl, L::kSumFree + g, (group >> 1) - 1);
        // the smaller terms' sums of the run before have been read
        if (k == from && group >= 1) wait_warp(ctl, L::kSumFree + (g ^ 1), (group - 1) >> 1);
        tc_fence_after();
        const uint32_t v = base + L::V + s * L::kV, terms = base + L::T + t * L::kT;
        const uint32_t d = tmem + g * L::kSumCols;
        const bool closes = (k + 1 - from) % L::kGroup == 0 || k + 1 == to;
        if (elect_one()) {
          if constexpr (L::kSide) {
            mma_tokens<3 * M, C>(d, v, terms, !opens);
          } else {
            mma_tokens<M, C>(d, v, base + L::K + s * L::kK, !opens);
            mma_tokens<2 * M, C>(tmem + 2 * L::kSumCols, v, terms, k > from);
          }
          mma_commit(&ctl.bar[L::kEmpty + s]);
          mma_commit(&ctl.bar[L::kSplitFree + t]);
          if (closes) mma_commit(&ctl.bar[L::kSum + g]);
        }
        __syncwarp();
        if (closes) ++group;
      }
    }
  }
  if (warp == kLoader && lane == 0) {
    settle(ctl, L::kFull, L::kStages, loaded);
    settle(ctl, L::kEmpty, L::kStages, c);
    settle(ctl, L::kSplitFree, 2, c);
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 0) tmem_dealloc(tmem, L::kCols);
  if (tid == 0 && ctl.fail) flag_error(a.err);
}

// ---- reads --------------------------------------------------------------------
// Per chunk, four products, sent by two warps, so that neither chain waits for the other:
//   A  P = Q K^T            -> weighted, masked and rounded by the first eight warps
//   B  Oi = Q X             X the state entering the chunk, rounded to bf16
//   C  X^T += V^T Kd        weighted keys in two terms; only where another chunk follows
//   D  O = P V              P read from TMEM
// One warp sends A and D, the other B and C.
// The other eight warps write gamma^{i+1} Oi + O and carry X.  (C sent before B, and the state
// taken out before the outputs: 208 us for 175 with 128 channels, 29.6 for 28.5 with 64.)
template <int M, int N>
struct ReadPlan {
  static constexpr bool kSide = M == 64;  // the two terms side by side, one product
  static constexpr uint32_t kQ = M / 64 * kTile, kK = kQ, kV = N / 64 * kTile;
  static constexpr uint32_t kSAtom = N * 128;  // the state [value][key], 64 keys of it
  static constexpr int kQs = M + N == 256 ? 1 : 2, kKs = M + N == 128 ? 3 : 2;  // stages
  static constexpr int kPs = N == 64 ? 2 : 1;  // P: the next chunk's beside this one's
  // V first: the tile behind its last one is read too (and ignored) where N = 64
  static constexpr uint32_t V = 0, Q = kKs * kV, K = Q + kQs * kQ, Lo = K + kKs * kK,
                            S = Lo + (kSide ? 2 : 1) * kK;
  static constexpr uint32_t kBytes = S + M / 64 * kSAtom + 1024;
  // TMEM columns: P (fp32, then bf16), O, Oi, X
  static constexpr uint32_t P = 0, O = kPs * 128, Oi = O + N, X = Oi + N, kCols = 512;
  static_assert(X + (kSide ? 2 * M : M) <= kCols, "columns of TMEM");
  static constexpr int kFullQ = 0, kEmptyQ = 2, kFullK = 4, kEmptyK = 7, kFullV = 10,
                       kEmptyV = 13, kA = 16, kB = 18, kC_ = 19, kD = 20, kClear = 21,
                       kPReady = 25, kKReady = 27, kSReady = 28, kOFree = 29, kBars = 30;
};
// How far one warp runs ahead of another decides how many barriers a step needs (a wait
// looks at a phase's parity): A, P's readiness and the clearing of padding may be one or
// two chunks ahead of the warp that sends B, the others not one.

// The chunks of an item in the order of the work, and whether rows of one have to be
// cleared in shared memory (padding that is not the tensor's end).
template <bool rev>
struct ChunkOf {
  int t0, have;
  bool clear;
  __device__ __forceinline__ ChunkOf(const Item& it, const DecayPass& p, int i) {
    t0 = it.first + (rev ? it.chunks - 1 - i : i) * kC;
    have = min(it.n - t0, kC);
    clear = have < kC && it.n < p.T;
  }
};

template <int M, int N, bool rev>
__global__ void __launch_bounds__(kReadThreads, 1)
    decay_read_tc(const __grid_constant__ TcArgs a, const __grid_constant__ TcMaps maps) {
  using L = ReadPlan<M, N>;
  using Chunk = ChunkOf<rev>;
  extern __shared__ unsigned char raw[];
  __shared__ Control<L::kBars> ctl;
  __shared__ float nears[4][64];
  unsigned char* sm = align1024(raw);
  const DecayPass& p = a.p;
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  if (tid == 0) {
    // what both issuing warps read is free when both have said so
    for (int i = 0; i < L::kBars; ++i) {
      const bool two = (i >= L::kEmptyQ && i < L::kFullK) || (i >= L::kEmptyK && i < L::kFullV) ||
                       (i >= L::kEmptyV && i < L::kA);
      mbar_init(&ctl.bar[i], i >= L::kClear ? 8 : two ? 2 : 1);
    }
    ctl.fail = 0;
    fence_mbar_init();
  }
  if (warp == 0) tmem_alloc(&ctl.tmem, L::kCols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, ctl.tmem, 0), base = smem_addr(sm);
  // behind the join; inputs that are read before were written before this pass began
  if (warp >= 8 && warp < 16) asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int row = 32 * (warp & 3) + lane;  // TMEM lane: a token, or a value
  const int part = warp >> 2 & 1;          // half of the columns
  const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;

  if (warp < 8) {
    int c = 0, carried = 0, cleared = 0;
    for (int item = blockIdx.x; item < a.items; item += gridDim.x) {
      const Item it(p, item);
      const float g2 = fmaxf(it.g * kLog2e, -kLargest);
      auto power = [&](int gap) { return exp2_approx(g2 * (float)gap); };
      const float intra = p.inter * p.w;
      f32x2 table[8];  // gamma^k from the far end of 16 columns
#pragma unroll
      for (int j = 0; j < 8; ++j)
        table[j] = rev ? pack2(power(2 * j), power(2 * j + 1))
                       : pack2(power(15 - 2 * j), power(14 - 2 * j));
      // intra gamma^k, zero for k < 0, for the square of 32 tokens on the diagonal
      // that half of these warps meet
      float* near = nears[warp & 3];
      __syncwarp();
      if (part == (warp & 3) >> 1) {
        near[lane] = lane == 31 ? intra : 0.f;
        near[32 + lane] = lane == 31 ? 0.f : intra * power(lane + 1);
      }
      __syncwarp();
      for (int i = 0; i < it.chunks; ++i, ++c) {
        const Chunk ch(it, p, i);
        const bool more = i + 1 < it.chunks;
        const int ks = c % L::kKs, qs = c % L::kQs, ps = c % L::kPs;
        const uint32_t at_p = tmem + lanes + L::P + ps * 128;
        unsigned char* key = sm + L::K + ks * L::kK;
        if (ch.clear) {
          wait_warp(ctl, L::kFullQ + qs, c / L::kQs);
          wait_warp(ctl, L::kFullK + ks, c / L::kKs);
          wait_warp(ctl, L::kFullV + ks, c / L::kKs);
          if (row >= ch.have) {
            clear_row<M / 64>(sm + L::Q + qs * L::kQ, row, 4 * part);
            clear_row<M / 64>(key, row, 4 * part);
            clear_row<N / 64>(sm + L::V + ks * L::kV, row, 4 * part);
          }
          fence_async_smem();
          arrive_warp(ctl, L::kClear + (cleared++ & 3));
        }
        wait_warp(ctl, L::kA + ps, c / L::kPs);
        tc_fence_after();
        {
          // columns 64 part .. 64 part + 63, to bf16 in place
          const int low = 32 * (warp & 3);
#pragma unroll 1
          for (int q = 0; q < 2; ++q) {
            const int c0 = 64 * part + 32 * q;  // against this warp's rows: one kind
            uint32_t to[16];
            if (rev ? c0 < low : c0 > low) {
#pragma unroll
              for (int j = 0; j < 16; ++j) to[j] = 0;
            } else {
              float x[32];
              tmem_ld32(at_p + c0, x);
              if (c0 == low) {
                const float* f = near + 31 + (rev ? -lane : lane);
#pragma unroll
                for (int j = 0; j < 16; ++j)
                  to[j] = rev ? pack_bf16(x[2 * j] * f[2 * j], x[2 * j + 1] * f[2 * j + 1])
                              : pack_bf16(x[2 * j] * f[-2 * j], x[2 * j + 1] * f[-2 * j - 1]);
              } else {
#pragma unroll
                for (int blk = 0; blk < 2; ++blk) {
                  const int j0 = c0 + 16 * blk;
                  const float f = intra * power(rev ? j0 - row : row - j0 - 15);
                  const f32x2 f2 = pack2(f, f);
#pragma unroll
                  for (int j = 0; j < 8; ++j) {
                    const float2 z =
                        unpack2(mul2(pack2(x[16 * blk + 2 * j], x[16 * blk + 2 * j + 1]),
                                     mul2(f2, table[j])));
                    to[8 * blk + j] = pack_bf16(z.x, z.y);
                  }
                }
              }
            }
            tmem_st16(at_p + 64 * part + 16 * q, to);
          }
          tmem_st_wait();
          tc_fence_before();
          arrive_warp(ctl, L::kPReady + ps);
        }
        if (more) {
          const float w = p.w * power(rev ? row + 1 : max(ch.have - 1 - row, 0));
          if (carried > 0) wait_warp(ctl, L::kC_, carried - 1);  // the second terms are free
          weigh_keys<M / 64, 2, 4, kTile>(key, L::kSide ? sm + L::Lo : key,
                                          L::kSide ? sm + L::Lo + L::kK : sm + L::Lo, nullptr,
                                          row, 4 * part, w);
          fence_async_smem();
          arrive_warp(ctl, L::kKReady);
          ++carried;
        }
      }
    }
  } else if (warp < 16) {
    int c = 0, carried = 0;
    const bool state_row = 32 * (warp & 3) < N;
    // keys 32 cb .. of value `row`: an operand, and what the next sum starts from
    auto put_state = [&](const float* x, int cb, const Carry& carry) {
      unsigned char* tile = sm + L::S + (cb >> 1) * L::kSAtom;
#pragma unroll
      for (int e = 0; e < 4; ++e)
        *reinterpret_cast<uint4*>(chunk_of(tile, row, 4 * (cb & 1) + e)) =
            tcu::pack8(x + 8 * e, 1.f);
      uint32_t w[32];
      const float keep = carry.near ? 1.f : 0.f;
      const f32x2 f2 = pack2(carry.f, carry.f), keep2 = pack2(keep, keep);
#pragma unroll
      for (int j = 0; j < 16; ++j) {  // carry.of() of two at a time
        const f32x2 y = pack2(x[2 * j], x[2 * j + 1]);
        const float2 z = unpack2(fma2(f2, y, mul2(keep2, y)));
        w[2 * j] = __float_as_uint(z.x), w[2 * j + 1] = __float_as_uint(z.y);
      }
      tmem_st32(tmem + lanes + L::X + 32 * cb, w);
      if constexpr (L::kSide) {  // the second term's sum
#pragma unroll
        for (int j = 0; j < 32; ++j) w[j] = 0u;
        tmem_st32(tmem + lanes + L::X + M + 32 * cb, w);
      }
    };
    auto state_ready = [&]() {
      tmem_st_wait();
      fence_async_smem();
      tc_fence_before();
      arrive_warp(ctl, L::kSReady);
    };
    for (int item = blockIdx.x; item < a.items; item += gridDim.x) {
      const Item it(p, item);
      const float g2 = fmaxf(it.g * kLog2e, -kLargest);
      auto power = [&](int gap) { return exp2_approx(g2 * (float)gap); };
      __nv_bfloat16* out =
          static_cast<__nv_bfloat16*>(p.o) + it.b * p.os.batch + it.h * p.os.head;
      const Carries carries(it.g, kC, (unsigned)max(min(it.n, it.end) - it.first, 0));
      if (it.chunks > 0) {
        if (state_row) {
          const Carry carry = carries.after(Chunk(it, p, 0).have, kC);
          const float* X = p.states + (it.bh * p.runs + it.run) * p.m * p.dv + row * p.xj;
#pragma unroll 1
          for (int q = 0; q < M / 64; ++q) {
            const int cb = part * (M / 64) + q;
            float x[32];
#pragma unroll
            for (int j = 0; j < 32; ++j) {
              const int i = 32 * cb + j;
              x[j] = i < p.m && row < p.dv ? X[i * p.xi] : 0.f;
            }
            put_state(x, cb, carry);
          }
        }
        state_ready();
      }
      // rows behind the last chunk that holds tokens
      const int eighths = p.dv / 8;
      const int64_t dead = (int64_t)max(it.end - it.first - it.chunks * kC, 0) * eighths;
      for (int64_t e = tid - 256; e < dead; e += 256)
        *reinterpret_cast<uint4*>(out + (it.first + it.chunks * kC + e / eighths) * p.os.time +
                                  e % eighths * 8) = make_uint4(0, 0, 0, 0);
      for (int i = 0; i < it.chunks; ++i, ++c) {
        const Chunk ch(it, p, i);
        const bool more = i + 1 < it.chunks;
        const float far = p.inter * power(rev ? max(ch.have - 1 - row, 0) : row + 1);
        const bool live = row < ch.have;
        wait_warp(ctl, L::kD, c);
        wait_warp(ctl, L::kB, c);
        tc_fence_after();
#pragma unroll 1
        for (int q = 0; q < N / 64; ++q) {
          const int col = 32 * (part * (N / 64) + q);
          float x[32], y[32];
          tmem_ld32(tmem + lanes + L::O + col, x);
          tmem_ld32(tmem + lanes + L::Oi + col, y);
          if (q + 1 == N / 64) {
            tc_fence_before();
            arrive_warp(ctl, L::kOFree);
          }
          if (ch.t0 + row < it.end) {
            uint32_t z[16];
#pragma unroll
            for (int j = 0; j < 16; ++j)
              z[j] = live ? pack_bf16(fmaf(far, y[2 * j], x[2 * j]),
                                      fmaf(far, y[2 * j + 1], x[2 * j + 1]))
                          : 0u;
            __nv_bfloat16* to = out + (ch.t0 + row) * p.os.time + col;
            if (a.wide_o) {
#pragma unroll
              for (int e = 0; e < 2; ++e)
                if (col + 16 * e < p.dv)
                  asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(
                                   to + 16 * e),
                               "r"(z[8 * e]), "r"(z[8 * e + 1]), "r"(z[8 * e + 2]),
                               "r"(z[8 * e + 3]), "r"(z[8 * e + 4]), "r"(z[8 * e + 5]),
                               "r"(z[8 * e + 6]), "r"(z[8 * e + 7])
                               : "memory");
            } else {
#pragma unroll
              for (int e = 0; e < 4; ++e)
                if (col + 8 * e < p.dv)
                  *reinterpret_cast<uint4*>(to + 8 * e) =
                      make_uint4(z[4 * e], z[4 * e + 1], z[4 * e + 2], z[4 * e + 3]);
            }
          }
          __syncwarp();
        }
        if (more) {
          const Carry carry = carries.after(Chunk(it, p, i + 1).have, kC);
          wait_warp(ctl, L::kC_, carried);
          ++carried;
          tc_fence_after();
          if (state_row) {
#pragma unroll 1
            for (int q = 0; q < M / 64; ++q) {
              const int cb = part * (M / 64) + q;
              float x[32];
              tmem_ld32(tmem + lanes + L::X + 32 * cb, x);
              if constexpr (L::kSide) {
                float y[32];
                tmem_ld32(tmem + lanes + L::X + M + 32 * cb, y);
#pragma unroll
                for (int j = 0; j < 32; ++j) x[j] += y[j];
              }
              put_state(x, cb, carry);
            }
          }
          state_ready();
        }
      }
    }
  } else if (warp == kLoader) {
    int c = 0, loaded_k = 0, loaded_v = 0, loaded_q = 0;
    auto free = [&](int ring, int stages) {
      if (c >= stages) wait(ctl, ring + c % stages, c / stages - 1);
      return ctl.fail == 0;
    };
    for (int item = blockIdx.x; item < a.items && lane == 0; item += gridDim.x) {
      const Item it(p, item);
      for (int i = 0; i < it.chunks; ++i, ++c) {
        const int t = Chunk(it, p, i).t0;
        if (L::kQs == 1) {  // its tile is still in use: as far as L2
#pragma unroll
          for (int x = 0; x < M / 64; ++x)
            tma_prefetch_4d(&maps.q, 64 * x, t, it.h * a.qh, it.b * a.qb);
        }
        const int ks = c % L::kKs, qs = c % L::kQs;
        if (free(L::kEmptyK, L::kKs)) {
          loaded_k = c + 1;
          mbar_expect_tx(&ctl.bar[L::kFullK + ks], L::kK);
#pragma unroll
          for (int x = 0; x < M / 64; ++x)
            tma_load_4d(sm + L::K + ks * L::kK + x * kTile, &maps.k, 64 * x, t, it.h * a.kh,
                        it.b * a.kb, &ctl.bar[L::kFullK + ks]);
        }
        if (free(L::kEmptyV, L::kKs)) {
          loaded_v = c + 1;
          mbar_expect_tx(&ctl.bar[L::kFullV + ks], L::kV);
#pragma unroll
          for (int x = 0; x < N / 64; ++x)
            tma_load_4d(sm + L::V + ks * L::kV + x * kTile, &maps.v, 64 * x, t, it.h * a.vh,
                        it.b * a.vb, &ctl.bar[L::kFullV + ks]);
        }
        if (free(L::kEmptyQ, L::kQs)) {
          loaded_q = c + 1;
          mbar_expect_tx(&ctl.bar[L::kFullQ + qs], L::kQ);
#pragma unroll
          for (int x = 0; x < M / 64; ++x)
            tma_load_4d(sm + L::Q + qs * L::kQ + x * kTile, &maps.q, 64 * x, t, it.h * a.qh,
                        it.b * a.qb, &ctl.bar[L::kFullQ + qs]);
        }
      }
    }
    if (lane == 0) {
      settle(ctl, L::kFullK, L::kKs, loaded_k);
      settle(ctl, L::kFullV, L::kKs, loaded_v);
      settle(ctl, L::kFullQ, L::kQs, loaded_q);
      settle(ctl, L::kEmptyK, L::kKs, c);
      settle(ctl, L::kEmptyV, L::kKs, c);
      settle(ctl, L::kEmptyQ, L::kQs, c);
    }
  } else if (warp == kIssuer) {
    int c = 0, cleared = 0;
    auto send_a = [&](int cc, bool clear) {
      const int ks = cc % L::kKs, qs = cc % L::kQs, ps = cc % L::kPs;
      wait_warp(ctl, L::kFullK + ks, cc / L::kKs);
      wait_warp(ctl, L::kFullQ + qs, cc / L::kQs);
      if (clear) wait_warp(ctl, L::kClear + (cleared & 3), cleared >> 2), ++cleared;
      tc_fence_after();
      const uint32_t q = desc_low(base + L::Q + qs * L::kQ, 16),
                     k = desc_low(base + L::K + ks * L::kK, 16);
      if (elect_one()) {  // behind the D that read this P
#pragma unroll
        for (int s = 0; s < M / 16; ++s) {
          const uint32_t at = (s >> 2) * (kTile >> 4) + (s & 3) * kStepK;
          mma_ss(tmem + L::P + ps * 128, q + at, k + at, idesc_bf16(128, 128, false, false),
                 s > 0);
        }
        mma_commit(&ctl.bar[L::kA + ps]);
        mma_commit(&ctl.bar[L::kEmptyQ + qs]);
      }
      __syncwarp();
    };
    for (int item = blockIdx.x; item < a.items; item += gridDim.x) {
      const Item it(p, item);
      if (it.chunks > 0) send_a(c, Chunk(it, p, 0).clear);
      for (int i = 0; i < it.chunks; ++i, ++c) {
        const int ks = c % L::kKs, ps = c % L::kPs;
        const bool more = i + 1 < it.chunks;
        if (L::kPs == 2 && more) send_a(c + 1, Chunk(it, p, i + 1).clear);
        const uint32_t v = desc_low(base + L::V + ks * L::kV, kTile);
        wait_warp(ctl, L::kFullV + ks, c / L::kKs);
        if (c > 0) wait_warp(ctl, L::kOFree, c - 1);
        wait_warp(ctl, L::kPReady + ps, c / L::kPs);
        tc_fence_after();
        if (elect_one()) {
#pragma unroll
          for (int s = 0; s < kC / 16; ++s)
            mma_ts(tmem + L::O, tmem + L::P + ps * 128 + (s >> 2) * 64 + (s & 3) * 8,
                   v + s * kStepMN, idesc_bf16(128, N, false, true), s > 0);
          mma_commit(&ctl.bar[L::kD]);
          mma_commit(&ctl.bar[L::kEmptyK + ks]);
          mma_commit(&ctl.bar[L::kEmptyV + ks]);
        }
        __syncwarp();
        if (L::kPs == 1 && more) send_a(c + 1, Chunk(it, p, i + 1).clear);
      }
    }
  } else {
    int c = 0, carried = 0, cleared = 0;
    for (int item = blockIdx.x; item < a.items; item += gridDim.x) {
      const Item it(p, item);
      for (int i = 0; i < it.chunks; ++i, ++c) {
        const int ks = c % L::kKs, qs = c % L::kQs;
        const uint32_t q = desc_low(base + L::Q + qs * L::kQ, 16),
                       s = desc_low(base + L::S, 16);
        wait_warp(ctl, L::kFullQ + qs, c / L::kQs);
        if (Chunk(it, p, i).clear)
          wait_warp(ctl, L::kClear + (cleared & 3), cleared >> 2), ++cleared;
        if (c > 0) wait_warp(ctl, L::kOFree, c - 1);
        wait_warp(ctl, L::kSReady, c);
        tc_fence_after();
        if (elect_one()) {
#pragma unroll
          for (int k = 0; k < M / 16; ++k)
            mma_ss(tmem + L::Oi, q + (k >> 2) * (kTile >> 4) + (k & 3) * kStepK,
                   s + (k >> 2) * (L::kSAtom >> 4) + (k & 3) * kStepK,
                   idesc_bf16(128, N, false, false), k > 0);
          mma_commit(&ctl.bar[L::kB]);
          mma_commit(&ctl.bar[L::kEmptyQ + qs]);
        }
        __syncwarp();
        if (i + 1 < it.chunks) {
          wait_warp(ctl, L::kFullV + ks, c / L::kKs);
          wait_warp(ctl, L::kKReady, carried++);
          tc_fence_after();
          const uint32_t v = base + L::V + ks * L::kV;
          if (elect_one()) {
            if constexpr (L::kSide) {
              mma_tokens<2 * M>(tmem + L::X, v, base + L::Lo, true);
            } else {
              mma_tokens<M>(tmem + L::X, v, base + L::K + ks * L::kK, true);
              mma_tokens<M>(tmem + L::X, v, base + L::Lo, true);
            }
            mma_commit(&ctl.bar[L::kC_]);
          }
          __syncwarp();
        }
        if (elect_one()) {
          mma_commit(&ctl.bar[L::kEmptyK + ks]);
          mma_commit(&ctl.bar[L::kEmptyV + ks]);
        }
        __syncwarp();
      }
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 0) tmem_dealloc(tmem, L::kCols);
  if (tid == 0 && ctl.fail) flag_error(a.err);
}

// ---- host -----------------------------------------------------------------------
bool heads_map(CUtensorMap* map, const void* x, const falcon_strides& s, int64_t B, int64_t H,
               int64_t T, int channels, int tokens, int* by_head, int* by_row) {
  const uintptr_t at = reinterpret_cast<uintptr_t>(x);
  if (at % 16 || s.batch % 8 || s.head % 8 || s.time % 8 || (T > 1 && s.time == 0)) return false;
  const bool hs = H > 1 && s.head != 0, bs = B > 1 && s.batch != 0;
  *by_head = hs, *by_row = bs;
  return encode_heads_bf16(map, x, channels, T, hs ? H : 1, bs ? B : 1, s.time, s.head, s.batch,
                           tokens);
}

template <int M, int N>
cudaError_t run_tc(const TcArgs& a, const TcMaps& maps, bool reads, cudaStream_t stream) {
  static std::atomic<uint64_t> allowed[3];
  const auto read = a.p.rev ? decay_read_tc<M, N, true> : decay_read_tc<M, N, false>;
  const unsigned grid = (unsigned)(a.items < kDecayTcBlocks ? a.items : kDecayTcBlocks);
  constexpr int ss = StatePlan<M, N>::kBytes, rs = ReadPlan<M, N>::kBytes;
  static_assert(ss + 1024 <= 232448 && rs + 1280 <= 232448, "shared memory of a block");
  cudaError_t e = reads ? allow_shared(read, rs, &allowed[a.p.rev])
                        : allow_shared(decay_states_tc<M, N>, ss, &allowed[2]);
  if (e != cudaSuccess) return e;
  return reads ? launch_behind(a.p.behind_reads, read, grid, kReadThreads, rs, stream, a, maps)
               : launch_behind(a.p.behind_states, decay_states_tc<M, N>, grid, kStateThreads, ss,
                               stream, a, maps);
}

cudaError_t run_tc_any(const TcArgs& a, const TcMaps& maps, bool reads, cudaStream_t stream) {
  if (a.p.m <= 64)
    return a.p.dv <= 64 ? run_tc<64, 64>(a, maps, reads, stream)
                        : run_tc<64, 128>(a, maps, reads, stream);
  return a.p.dv <= 64 ? run_tc<128, 64>(a, maps, reads, stream)
                      : run_tc<128, 128>(a, maps, reads, stream);
}

}  // namespace

bool decay_tc_pass(const DecayPass& p, cudaError_t* status, cudaStream_t stream) {
  if (p.dtype != FALCON_BF16 || p.m % 8 || p.dv % 8 || p.runs == 0 || p.T > (1 << 30) ||
      p.B * p.H * p.runs > 0x7fffffff)
    return false;
  TcArgs a = {};
  TcMaps maps;
  const int sum_tokens =
      p.m <= 64 ? StatePlan<64, 64>::kTokens : StatePlan<128, 64>::kTokens;
  if (!heads_map(&maps.q, p.q, p.qs, p.B, p.H, p.T, p.m, kC, &a.qh, &a.qb) ||
      !heads_map(&maps.k, p.k, p.ks, p.B, p.H, p.T, p.m, kC, &a.kh, &a.kb) ||
      !heads_map(&maps.v, p.v, p.vs, p.B, p.H, p.T, p.dv, kC, &a.vh, &a.vb) ||
      !heads_map(&maps.ks, p.k, p.ks, p.B, p.H, p.T, p.m, sum_tokens, &a.kh, &a.kb) ||
      !heads_map(&maps.vs, p.v, p.vs, p.B, p.H, p.T, p.dv, sum_tokens, &a.vh, &a.vb) ||
      reinterpret_cast<uintptr_t>(p.o) % 16 || p.os.batch % 8 || p.os.head % 8 || p.os.time % 8)
    return false;
  a.p = p;
  a.items = (int)(p.B * p.H * p.runs);
  a.wide_o = reinterpret_cast<uintptr_t>(p.o) % 32 == 0 && p.os.batch % 16 == 0 &&
             p.os.head % 16 == 0 && p.os.time % 16 == 0 && p.dv % 16 == 0;
  a.err = device_error_word_of_current();
  if (p.sums) *status = run_tc_any(a, maps, false, stream);
  if (p.sums && *status == cudaSuccess) *status = launch_decay_join(p, true, stream);
  if (*status == cudaSuccess) *status = run_tc_any(a, maps, true, stream);
  return true;
}

}  // namespace falcon
