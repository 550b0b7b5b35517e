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
// Rounding: an output is a sum of terms rounded once to bf16 (a weight times q k, or a
// state), and is rounded once itself; weights, sums and states are fp32.
//
// Keys of up to 64 (M = 64) and up to 128 channels (M = 128), values likewise (N): TMA
// fills the missing channels with zeros.  All accumulators have 128 lanes; for M = 64 the
// A operand's second half is the tile behind it in shared memory, which lands in lanes
// 64..127 that nobody reads.
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

constexpr int kThreads = 256;
constexpr int kC = 128;                // tokens of a chunk
constexpr uint32_t kTile = kC * 128;   // a chunk of 64 channels

struct TcArgs {
  DecayPass p;
  int* err;
  // 0 where the tensor is broadcast along heads or batches
  int qh, qb, kh, kb, vh, vb;
};
struct TcMaps {
  CUtensorMap q, k, v, o;
};

struct Control {
  uint64_t bar[4];
  uint32_t tmem;
  volatile int fail;
};

__device__ __forceinline__ void wait(Control& c, int which, uint32_t phase) {
  if (!c.fail && !mbar_wait(&c.bar[which], phase)) c.fail = 1;
}

// x as three bf16 terms; their sum keeps 24 bits.
__device__ __forceinline__ void split2(float a, float b, uint32_t& hi, uint32_t& mid) {
  hi = pack_bf16(a, b);
  mid = pack_bf16(a - bf16_lo(hi), b - bf16_hi(hi));
}
__device__ __forceinline__ void split3(float a, float b, uint32_t& hi, uint32_t& mid,
                                       uint32_t& lo) {
  hi = pack_bf16(a, b);
  const float ra = a - bf16_lo(hi), rb = b - bf16_hi(hi);
  mid = pack_bf16(ra, rb);
  lo = pack_bf16(ra - bf16_lo(mid), rb - bf16_hi(mid));
}

// One row's share of a thread: 64 / (256 / 128) channels of every 64-wide tile.
__device__ __forceinline__ unsigned char* chunk_of(unsigned char* tile, int r, int c) {
  return tile + r * 128 + ((c ^ (r & 7)) << 4);
}

// Weighted keys of row r (in place: the first term), and the terms behind it.
template <int ATOMS, int TERMS>
__device__ __forceinline__ void weigh_keys(unsigned char* k, unsigned char* mid,
                                           unsigned char* lo, int r, int half, float w) {
#pragma unroll
  for (int at = 0; at < ATOMS; ++at)
#pragma unroll
    for (int c = 4 * half; c < 4 * half + 4; ++c) {
      uint4* p = reinterpret_cast<uint4*>(chunk_of(k + at * kTile, r, c));
      const uint4 x = *p;
      const uint32_t in[4] = {x.x, x.y, x.z, x.w};
      uint32_t t[3][4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float a = bf16_lo(in[e]) * w, b = bf16_hi(in[e]) * w;
        if constexpr (TERMS == 3)
          split3(a, b, t[0][e], t[1][e], t[2][e]);
        else
          split2(a, b, t[0][e], t[1][e]);
      }
      *p = make_uint4(t[0][0], t[0][1], t[0][2], t[0][3]);
      *reinterpret_cast<uint4*>(chunk_of(mid + at * kTile, r, c)) =
          make_uint4(t[1][0], t[1][1], t[1][2], t[1][3]);
      if constexpr (TERMS == 3)
        *reinterpret_cast<uint4*>(chunk_of(lo + at * kTile, r, c)) =
            make_uint4(t[2][0], t[2][1], t[2][2], t[2][3]);
    }
}

template <int ATOMS>
__device__ __forceinline__ void clear_row(unsigned char* tile, int r, int half) {
#pragma unroll
  for (int at = 0; at < ATOMS; ++at)
#pragma unroll
    for (int c = 4 * half; c < 4 * half + 4; ++c)
      *reinterpret_cast<uint4*>(chunk_of(tile + at * kTile, r, c)) = make_uint4(0, 0, 0, 0);
}

// D += A^T B over 128 tokens: A and B tiles [token][channel], M (or 64) and N channels.
template <int N>
__device__ __forceinline__ void mma_tokens(uint32_t d, uint32_t a, uint32_t b, bool accumulate) {
  const uint32_t id = idesc_bf16(128, N, true, true);
  const uint64_t da = sw128_desc(a, kTile, 1024), db = sw128_desc(b, kTile, 1024);
#pragma unroll
  for (int ks = 0; ks < kC / 16; ++ks)
    mma_bf16(d, da + (uint64_t)(ks * kStepMN), db + (uint64_t)(ks * kStepMN), id,
             accumulate || ks > 0);
}

// ---- states -----------------------------------------------------------------
template <int M, int N>
struct StateSmem {
  static constexpr uint32_t kK = M / 64 * kTile, kV = N / 64 * kTile;
  static constexpr uint32_t kMid = 0, kLo = kK, kStage = 2 * kK, kStageBytes = kK + kV;
  static constexpr uint32_t kBytes = kStage + 2 * kStageBytes + 1024;
};

template <int M, int N>
__global__ void __launch_bounds__(kThreads, M + N == 128 ? 2 : 1)
    decay_states_tc(const __grid_constant__ TcArgs a, const __grid_constant__ TcMaps maps) {
  using L = StateSmem<M, N>;
  extern __shared__ unsigned char raw[];
  __shared__ Control ctl;
  unsigned char* sm = align1024(raw);
  const DecayPass& p = a.p;
  const int tid = threadIdx.x, warp = tid >> 5;
  const int run = blockIdx.x % p.runs;
  const int64_t bh = blockIdx.x / p.runs;
  const int b = (int)(bh / p.H), h = (int)(bh % p.H);
  const int64_t n = row_length(p.lengths, b, p.T);
  const int64_t t0 = run * p.run_len, len = run_tokens(n, run, p.run_len);
  const int chunks = (int)((len + kC - 1) / kC);
  if (tid == 0) {
    for (int i = 0; i < 3; ++i) mbar_init(&ctl.bar[i], 1);
    ctl.fail = 0;
    fence_mbar_init();
  }
  if (warp == 0) tmem_alloc(&ctl.tmem, N);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ctl.tmem;
  auto load = [&](int c) {
    unsigned char* st = sm + L::kStage + (c & 1) * L::kStageBytes;
    uint64_t* bar = &ctl.bar[c & 1];
    mbar_expect_tx(bar, L::kStageBytes);
    const int t = (int)t0 + c * kC;
#pragma unroll
    for (int i = 0; i < M / 64; ++i)
      tma_load_4d(st + i * kTile, &maps.k, 64 * i, t, h * a.kh, b * a.kb, bar);
#pragma unroll
    for (int i = 0; i < N / 64; ++i)
      tma_load_4d(st + L::kK + i * kTile, &maps.v, 64 * i, t, h * a.vh, b * a.vb, bar);
  };
  if (tid == 0)
    for (int c = 0; c < 2 && c < chunks; ++c) load(c);
  const float g = decay_rate(p.log_decay, h);
  const int r = tid & (kC - 1), half = tid >> 7;
  for (int c = 0; c < chunks; ++c) {
    unsigned char* st = sm + L::kStage + (c & 1) * L::kStageBytes;
    const int have = (int)(len - (int64_t)c * kC < kC ? len - (int64_t)c * kC : kC);
    const float w = p.w * decay_power(g, (float)(p.rev ? (int64_t)c * kC + r + 1
                                                       : len - 1 - (int64_t)c * kC - r));
    wait(ctl, c & 1, (c >> 1) & 1);
    if (c > 0) {
      wait(ctl, 2, (c - 1) & 1);  // the products of the last chunk: its tiles are free
      if (tid == 0 && c + 1 < chunks) load(c + 1);
    }
    if (r < have) {
      weigh_keys<M / 64, 3>(st, sm + L::kMid, sm + L::kLo, r, half, w);
    } else {  // rows that the sequence does not hold
      clear_row<M / 64>(st, r, half);
      clear_row<M / 64>(sm + L::kMid, r, half);
      clear_row<M / 64>(sm + L::kLo, r, half);
      clear_row<N / 64>(st + L::kK, r, half);
    }
    fence_async_smem();
    __syncthreads();
    if (tid == 0) {
      tc_fence_after();
      const uint32_t k = smem_addr(st), v = k + L::kK;
      mma_tokens<N>(tmem, k, v, c > 0);
      mma_tokens<N>(tmem, smem_addr(sm + L::kMid), v, true);
      mma_tokens<N>(tmem, smem_addr(sm + L::kLo), v, true);
      mma_commit(&ctl.bar[2]);
    }
  }
  if (chunks > 0) wait(ctl, 2, (chunks - 1) & 1);
  tc_fence_after();
  const int i = 32 * (warp & 3) + (tid & 31);
  float* out = p.states + ((bh * p.runs + run) * p.m + i) * p.dv;
  if (32 * (warp & 3) < M) {
#pragma unroll
    for (int cb = 0; cb < N / 64; ++cb) {
      const int j0 = (warp >> 2) * (N / 2) + cb * 32;
      float v[32];
      tmem_ld32(tmem + ((uint32_t)(32 * (warp & 3)) << 16) + j0, v);
      if (i < p.m) {
#pragma unroll
        for (int j = 0; j < 32; j += 4)
          if (j0 + j < p.dv)
            *reinterpret_cast<float4*>(out + j0 + j) =
                chunks > 0 ? make_float4(v[j], v[j + 1], v[j + 2], v[j + 3])
                           : make_float4(0.f, 0.f, 0.f, 0.f);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 0) tmem_dealloc(tmem, N);
  if (tid == 0 && ctl.fail) flag_error(a.err);
}

// ---- reads --------------------------------------------------------------------
template <int M, int N>
struct ReadSmem {
  static constexpr uint32_t kK = M / 64 * kTile, kV = N / 64 * kTile;
  static constexpr uint32_t kSAtom = M * 128;  // 64 values of the state
  static constexpr uint32_t Q = 0, K = kK, Lo = 2 * kK, V = 3 * kK, O = V + kV, S = O + kV;
  static constexpr uint32_t kBytes = S + N / 64 * kSAtom + 1024;
  // TMEM columns: P (fp32, then bf16), O, X
  static constexpr uint32_t P = 0, Od = 128, X = Od + N, kCols = X + N <= 256 ? 256 : 512;
};

template <int M, int N>
__global__ void __launch_bounds__(kThreads, M + N == 128 ? 2 : 1)
    decay_read_tc(const __grid_constant__ TcArgs a, const __grid_constant__ TcMaps maps) {
  using L = ReadSmem<M, N>;
  extern __shared__ unsigned char raw[];
  __shared__ Control ctl;
  unsigned char* sm = align1024(raw);
  const DecayPass& p = a.p;
  const int tid = threadIdx.x, warp = tid >> 5;
  const int run = blockIdx.x % p.runs;
  const int64_t bh = blockIdx.x / p.runs;
  const int b = (int)(bh / p.H), h = (int)(bh % p.H);
  const int n = (int)row_length(p.lengths, b, p.T);
  const int first = (int)(run * p.run_len);
  const int end = (int)(first + p.run_len < p.T ? first + p.run_len : p.T);
  const int chunks = (end - first + kC - 1) / kC;
  const bool rev = p.rev;
  enum { kQK = 0, kVb = 1, kMma = 2 };
  if (tid == 0) {
    for (int i = 0; i < 3; ++i) mbar_init(&ctl.bar[i], 1);
    ctl.fail = 0;
    fence_mbar_init();
  }
  if (warp == 0) tmem_alloc(&ctl.tmem, L::kCols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ctl.tmem;

  auto token = [&](int c) { return first + (rev ? chunks - 1 - c : c) * kC; };
  auto held = [&](int c) { return min(max(n - token(c), 0), kC); };
  auto load_q = [&](int c) {
    mbar_expect_tx(&ctl.bar[kQK], 2 * L::kK);
#pragma unroll
    for (int i = 0; i < M / 64; ++i)
      tma_load_4d(sm + L::Q + i * kTile, &maps.q, 64 * i, token(c), h * a.qh, b * a.qb,
                  &ctl.bar[kQK]);
  };
  auto load_kv = [&](int c) {
#pragma unroll
    for (int i = 0; i < M / 64; ++i)
      tma_load_4d(sm + L::K + i * kTile, &maps.k, 64 * i, token(c), h * a.kh, b * a.kb,
                  &ctl.bar[kQK]);
    mbar_expect_tx(&ctl.bar[kVb], L::kV);
#pragma unroll
    for (int i = 0; i < N / 64; ++i)
      tma_load_4d(sm + L::V + i * kTile, &maps.v, 64 * i, token(c), h * a.vh, b * a.vb,
                  &ctl.bar[kVb]);
  };
  // chunks behind the row's last token come first (backward) or last (forward)
  int live = 0, live0 = 0;
  for (int c = 0; c < chunks; ++c)
    if (held(c) > 0) {
      if (live == 0) live0 = c;
      ++live;
    }
  if (tid == 0 && live > 0) {
    load_q(live0);
    load_kv(live0);
  }

  const float g = decay_rate(p.log_decay, h);
  const float g2 = fmaxf(g * kLog2e, -kLargest);
  auto power = [&](int gap) { return exp2_approx(g2 * (float)gap); };
  const float intra = p.inter * p.w;
  const int lane = tid & 31, i = 32 * (warp & 3) + lane;  // TMEM lane: a token, or a key
  const int part = warp >> 2;                             // half of the columns
  const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
  const int r = tid & (kC - 1), half = tid >> 7;  // a row of a staged tile, half of it

  // the state entering the run: as an operand, and weighted for the sum
  const bool state_row = 32 * (warp & 3) < M;
  auto put_state = [&](float* x, int cb, float lost) {
    // columns 32 cb .. of key i
    unsigned char* tile = sm + L::S + (cb >> 1) * L::kSAtom;
#pragma unroll
    for (int c = 0; c < 4; ++c)
      *reinterpret_cast<uint4*>(chunk_of(tile, i, 4 * (cb & 1) + c)) = tcu::pack8(x + 8 * c, 1.f);
    uint32_t w[32];
#pragma unroll
    for (int j = 0; j < 32; ++j) w[j] = __float_as_uint(fmaf(lost, x[j], x[j]));
    tmem_st32(tmem + lanes + L::X + 32 * cb, w);
  };
  if (live > 0 && state_row) {
    const float lost = expm1f(g * (float)held(live0));
    const float* X = p.states + ((bh * p.runs + run) * p.m + (i < p.m ? i : 0)) * p.dv;
#pragma unroll
    for (int q = 0; q < N / 64; ++q) {
      const int cb = part * (N / 64) + q;
      float x[32];
#pragma unroll
      for (int j = 0; j < 32; j += 4) {
        const int col = 32 * cb + j;
        const float4 y = i < p.m && col < p.dv ? *reinterpret_cast<const float4*>(X + col)
                                               : make_float4(0.f, 0.f, 0.f, 0.f);
        x[j] = y.x, x[j + 1] = y.y, x[j + 2] = y.z, x[j + 3] = y.w;
      }
      put_state(x, cb, lost);
    }
    tmem_st_wait();
  }

  float table[16];  // gamma^k, from the far end of 16 columns
#pragma unroll
  for (int j = 0; j < 16; ++j) table[j] = power(rev ? j : 15 - j);

  int done = 0;         // chunks worked on
  uint32_t mma = 0;     // phase of the products' barrier
  for (int c = 0; c < chunks; ++c) {
    const int t0 = token(c), have = held(c);
    if (have > 0) {
      const bool more = done + 1 < live;
      wait(ctl, kQK, done & 1);
      if (have < kC) {
        wait(ctl, kVb, done & 1);
        if (r >= have) {
          clear_row<M / 64>(sm + L::Q, r, half);
          clear_row<M / 64>(sm + L::K, r, half);
          clear_row<N / 64>(sm + L::V, r, half);
        }
      }
      fence_async_smem();
      tc_fence_before();
      __syncthreads();
      if (tid == 0) {
        tc_fence_after();
        const uint32_t q = smem_addr(sm + L::Q), k = smem_addr(sm + L::K),
                       s = smem_addr(sm + L::S);
#pragma unroll
        for (int ks = 0; ks < M / 16; ++ks) {
          const uint32_t at = (ks >> 2) * kTile + (ks & 3) * 32;
          mma_bf16(tmem + L::P, sw128_desc(q + at, 16, 1024), sw128_desc(k + at, 16, 1024),
                   idesc_bf16(128, 128, false, false), ks > 0);
        }
#pragma unroll
        for (int ks = 0; ks < M / 16; ++ks)
          mma_bf16(tmem + L::Od,
                   sw128_desc(q + (ks >> 2) * kTile + (ks & 3) * 32, 16, 1024),
                   sw128_desc(s + ks * 2048, L::kSAtom, 1024), idesc_bf16(128, N, false, true),
                   ks > 0);
        mma_commit(&ctl.bar[kMma]);
      }
      const float far = p.inter * power(rev ? max(have - 1 - i, 0) : i + 1);
      const float wk = more ? p.w * power(rev ? r + 1 : max(have - 1 - r, 0)) : 0.f;
      wait(ctl, kMma, mma);
      mma ^= 1;
      tc_fence_after();
      if (tid == 0 && more) load_q(live0 + done + 1);
      // O: the state's part
#pragma unroll
      for (int q = 0; q < N / 64; ++q) {
        const uint32_t at = tmem + lanes + L::Od + part * (N / 2) + 32 * q;
        float x[32];
        tmem_ld32(at, x);
        uint32_t w[32];
#pragma unroll
        for (int j = 0; j < 32; ++j) w[j] = __float_as_uint(x[j] * far);
        tmem_st32(at, w);
      }
      // P: weights and mask, columns 64 part .. 64 part + 63, to bf16 in place
      {
        uint32_t w[32];
        const int low = 32 * (warp & 3);
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          float x[32];
          tmem_ld32(tmem + lanes + L::P + 64 * part + 32 * q, x);
#pragma unroll
          for (int blk = 0; blk < 2; ++blk) {
            const int j0 = 64 * part + 32 * q + 16 * blk;
            float* y = x + 16 * blk;
            uint32_t* to = w + 16 * q + 8 * blk;
            const int least = rev ? j0 - low - 31 : low - j0 - 15;
            const int most = rev ? j0 + 15 - low : low + 31 - j0;
            if (most < 0) {
#pragma unroll
              for (int j = 0; j < 8; ++j) to[j] = 0;
            } else if (least >= 0) {
              const float f = intra * power(rev ? j0 - i : i - j0 - 15);
#pragma unroll
              for (int j = 0; j < 8; ++j)
                to[j] = pack_bf16(y[2 * j] * (f * table[2 * j]),
                                  y[2 * j + 1] * (f * table[2 * j + 1]));
            } else {
#pragma unroll
              for (int j = 0; j < 16; ++j) {
                const int gap = rev ? j0 + j - i : i - j0 - j;
                y[j] = gap >= 0 ? y[j] * (intra * power(gap)) : 0.f;
              }
#pragma unroll
              for (int j = 0; j < 8; ++j) to[j] = pack_bf16(y[2 * j], y[2 * j + 1]);
            }
          }
        }
        tmem_st32(tmem + lanes + L::P + 64 * part, w);
      }
      if (more) weigh_keys<M / 64, 2>(sm + L::K, sm + L::Lo, nullptr, r, half, wk);
      tmem_st_wait();
      fence_async_smem();
      tc_fence_before();
      __syncthreads();
      wait(ctl, kVb, done & 1);
      if (tid == 0) {
        tc_fence_after();
        const uint64_t v = sw128_desc(smem_addr(sm + L::V), kTile, 1024);
#pragma unroll
        for (int ks = 0; ks < kC / 16; ++ks)
          mma_bf16_ta(tmem + L::Od, tmem + L::P + (ks >> 2) * 64 + (ks & 3) * 8,
                      v + (uint64_t)(ks * kStepMN), idesc_bf16(128, N, false, true), 1);
        if (more) {
          mma_tokens<N>(tmem + L::X, smem_addr(sm + L::K), smem_addr(sm + L::V), true);
          mma_tokens<N>(tmem + L::X, smem_addr(sm + L::Lo), smem_addr(sm + L::V), true);
        }
        mma_commit(&ctl.bar[kMma]);
        bulk_wait_read<0>();  // the last chunk's outputs have left their tiles
      }
      wait(ctl, kMma, mma);
      mma ^= 1;
      tc_fence_after();
      if (tid == 0 && more) load_kv(live0 + done + 1);
      __syncthreads();
#pragma unroll
      for (int q = 0; q < N / 64; ++q) {
        const int cb = part * (N / 64) + q;
        float x[32];
        tmem_ld32(tmem + lanes + L::Od + 32 * cb, x);
        if (i >= have) {
#pragma unroll
          for (int j = 0; j < 32; ++j) x[j] = 0.f;
        }
        unsigned char* tile = sm + L::O + (cb >> 1) * kTile;
#pragma unroll
        for (int e = 0; e < 4; ++e)
          *reinterpret_cast<uint4*>(chunk_of(tile, i, 4 * (cb & 1) + e)) =
              tcu::pack8(x + 8 * e, 1.f);
      }
      if (more && state_row) {
        const float lost = expm1f(g * (float)held(live0 + done + 1));
#pragma unroll
        for (int q = 0; q < N / 64; ++q) {
          const int cb = part * (N / 64) + q;
          float x[32];
          tmem_ld32(tmem + lanes + L::X + 32 * cb, x);
          put_state(x, cb, lost);
        }
        tmem_st_wait();
      }
      ++done;
    } else {  // no token: zeros
      if (tid == 0) bulk_wait_read<0>();
      __syncthreads();
      clear_row<N / 64>(sm + L::O, r, half);
    }
    fence_async_smem();
    tc_fence_before();
    __syncthreads();
    if (tid == 0) {
#pragma unroll
      for (int q = 0; q < N / 64; ++q)
        if (64 * q < p.dv) tma_store_4d(&maps.o, sm + L::O + q * kTile, 64 * q, t0, h, b);
      bulk_commit();
    }
  }
  if (tid == 0) bulk_wait<0>();
  __syncthreads();
  if (warp == 0) tmem_dealloc(tmem, L::kCols);
  if (tid == 0 && ctl.fail) flag_error(a.err);
}

// ---- host -----------------------------------------------------------------------
bool heads_map(CUtensorMap* map, const void* x, const falcon_strides& s, int64_t B, int64_t H,
               int64_t T, int channels, bool output, int* by_head, int* by_row) {
  const uintptr_t at = reinterpret_cast<uintptr_t>(x);
  if (at % 16 || s.batch % 8 || s.head % 8 || s.time % 8 || (T > 1 && s.time == 0)) return false;
  const bool hs = H > 1 && s.head != 0, bs = B > 1 && s.batch != 0;
  *by_head = output || hs, *by_row = output || bs;
  return encode_heads_bf16(map, x, channels, T, hs ? H : 1, bs ? B : 1, s.time, s.head, s.batch,
                           kC);
}

template <int M, int N>
cudaError_t run_tc(const TcArgs& a, const TcMaps& maps, bool reads, cudaStream_t stream) {
  static std::atomic<uint64_t> allowed[2];
  const unsigned grid = (unsigned)(a.p.B * a.p.H * a.p.runs);
  constexpr int ss = StateSmem<M, N>::kBytes, rs = ReadSmem<M, N>::kBytes;
  static_assert(ss <= 232448 && rs <= 232448, "shared memory of a block");
  cudaError_t e = reads ? allow_shared(decay_read_tc<M, N>, rs, &allowed[0])
                        : allow_shared(decay_states_tc<M, N>, ss, &allowed[1]);
  if (e != cudaSuccess) return e;
  if (reads)
    decay_read_tc<M, N><<<grid, kThreads, rs, stream>>>(a, maps);
  else
    decay_states_tc<M, N><<<grid, kThreads, ss, stream>>>(a, maps);
  return cudaGetLastError();
}

cudaError_t run_tc_any(const TcArgs& a, const TcMaps& maps, bool reads, cudaStream_t stream) {
  if (a.p.m <= 64)
    return a.p.dv <= 64 ? run_tc<64, 64>(a, maps, reads, stream)
                        : run_tc<64, 128>(a, maps, reads, stream);
  return a.p.dv <= 64 ? run_tc<128, 64>(a, maps, reads, stream)
                      : run_tc<128, 128>(a, maps, reads, stream);
}

}  // namespace

int64_t decay_tc_blocks(int m, int dv) { return m <= 64 && dv <= 64 ? 2 * 152 : 152; }

bool decay_tc_pass(const DecayPass& p, cudaError_t* status, cudaStream_t stream) {
  if (p.dtype != FALCON_BF16 || p.m % 8 || p.dv % 8 || p.runs == 0 || p.T > (1 << 30))
    return false;
  TcArgs a = {};
  TcMaps maps;
  int oh, ob;
  if (!heads_map(&maps.q, p.q, p.qs, p.B, p.H, p.T, p.m, false, &a.qh, &a.qb) ||
      !heads_map(&maps.k, p.k, p.ks, p.B, p.H, p.T, p.m, false, &a.kh, &a.kb) ||
      !heads_map(&maps.v, p.v, p.vs, p.B, p.H, p.T, p.dv, false, &a.vh, &a.vb) ||
      !heads_map(&maps.o, p.o, p.os, p.B, p.H, p.T, p.dv, true, &oh, &ob))
    return false;
  a.p = p;
  a.err = device_error_word_of_current();
  *status = run_tc_any(a, maps, false, stream);
  if (*status == cudaSuccess) *status = launch_decay_join(p, stream);
  if (*status == cudaSuccess) *status = run_tc_any(a, maps, true, stream);
  return true;
}

}  // namespace falcon
