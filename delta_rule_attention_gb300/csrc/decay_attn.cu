// Attention with a fixed decay a head, in fp32 on the CUDA cores: any type, any m and dv
// up to 128, any strides.  The tensor-core kernels take the bf16 shapes that they fit.
//
// The sum o_t = sum_{j <= t} gamma^{t-j} (q_t . k_j) v_j is split by runs of tokens, so
// that every run can be worked on at once although the state goes from token to token:
//   1. states: what a run adds to the state, U_r = sum_j gamma^{e-1-j} k_j v_j^T
//      (weights relative to the run's end e: all at most 1);
//   2. join: the state entering each run, X_{r+1} = gamma^{len_r} X_r + U_r;
//   3. reads: chunk by chunk inside a run, o = ((q k^T) * gamma^{i-j}) v + gamma^{i+1} q X,
//      X carried on.
// Every power of gamma is of a number of tokens >= 0, so none overflows, and heads that
// forget within a chunk (gamma^64 = 0) need no care of their own.
//
// Bound by the CUDA cores and the shared memory that feeds them: a thread's 4 x 4 corner
// takes two 16-byte reads for 16 multiply-adds.  fp32, 96 heads of 64 channels and 2048
// tokens: 323 us, 25 TFLOP/s of the 80 that the cores have (gradient 945 us); 32 heads of 128
// and 4096 tokens 607 us (1820).  64 keys a step, all loads of a chunk under way at once:
// 319 for 336 us with 32 keys, 607 for 715.
#include "linear.cuh"
#include "linear_tc.cuh"

namespace falcon {

namespace {

constexpr int kThreads = 256;
constexpr int kTile = 64;         // rows and columns of a block's tile
constexpr int kLd = kTile + 4;    // row stride in shared memory
constexpr int kStep = 32;         // tokens staged at a time (states)
constexpr int kKeys = 64;         // keys staged at a time (reads)
constexpr int kChunk = 64;        // tokens of a chunk
constexpr int kWholeTokens = 128;  // rows of at most so many are one run
constexpr int kTcFrom = 64;        // longer rows go to the tensor cores

// acc[i][j] += sum_{k < n} a[k][i] b[k][j] for this thread's 4 x 4 corner of the tile
__device__ __forceinline__ void outer_sum(float (&acc)[4][4], const float* a, const float* b,
                                          int n) {
#pragma unroll 8
  for (int k = 0; k < n; ++k) {
    const float4 x = *reinterpret_cast<const float4*>(a + k * kLd);
    const float4 y = *reinterpret_cast<const float4*>(b + k * kLd);
    const float xs[4] = {x.x, x.y, x.z, x.w}, ys[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(xs[i], ys[j], acc[i][j]);
  }
}

// Four channels from c on of a row with `width` of them, zeros behind.
template <typename E>
__device__ __forceinline__ float4 row_quad(const E* row, int c, int width, bool vec) {
  const int have = width - c;
  return widen(load_quad<E>(row + c, vec && have >= 4, have < 0 ? 0 : (have < 4 ? have : 4)));
}

template <typename E>
__global__ void __launch_bounds__(kThreads)
    decay_states_kernel(const __grid_constant__ DecayPass a) {
  __shared__ float ks[kStep * kLd], vs[kStep * kLd];
  const int run = blockIdx.x % a.runs;
  const int64_t bh = blockIdx.x / a.runs, b = bh / a.H;
  const int h = (int)(bh % a.H), tid = threadIdx.x;
  const int tiles = (a.dv + kTile - 1) / kTile;
  const int i0 = blockIdx.y / tiles * kTile, j0 = blockIdx.y % tiles * kTile;
  const int64_t n = row_length(a.lengths, b, a.T);
  const int64_t t0 = run * a.run_len, len = run_tokens(n, run, a.run_len);
  const float g = decay_rate(a.log_decay, h);
  const E* k = static_cast<const E*>(a.k) + b * a.ks.batch + h * a.ks.head;
  const E* v = static_cast<const E*>(a.v) + b * a.vs.batch + h * a.vs.head;
  const int ti = (tid >> 4) * 4, tj = (tid & 15) * 4;
  float acc[4][4] = {};
  for (int64_t s = 0; s < len; s += kStep) {
    const int have = (int)(len - s < kStep ? len - s : kStep);
    __syncthreads();
    for (int e = tid; e < kStep * (kTile / 4); e += kThreads) {
      const int r = e / (kTile / 4), c = e % (kTile / 4) * 4;
      float4 x = make_float4(0.f, 0.f, 0.f, 0.f), y = x;
      if (r < have) {
        const int64_t t = t0 + s + r;
        const float wt = a.w * decay_power(g, (float)(a.rev ? s + r + 1 : len - 1 - s - r));
        x = row_quad<E>(k + t * a.ks.time, i0 + c, a.m, a.vec_k);
        y = row_quad<E>(v + t * a.vs.time, j0 + c, a.dv, a.vec_v);
        x.x *= wt, x.y *= wt, x.z *= wt, x.w *= wt;
      }
      *reinterpret_cast<float4*>(ks + r * kLd + c) = x;
      *reinterpret_cast<float4*>(vs + r * kLd + c) = y;
    }
    __syncthreads();
    outer_sum(acc, ks + ti, vs + tj, have);
  }
  float* out = a.states + (bh * a.runs + run) * a.m * a.dv;
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (i0 + ti + i < a.m && j0 + tj + j < a.dv)
        out[(i0 + ti + i) * a.dv + j0 + tj + j] = acc[i][j];
}

// The state entering each run, in the order of time (rev: from the last run back), in
// place of what the run adds; one thread an element.
constexpr int kAhead = 8;
__global__ void __launch_bounds__(kThreads)
    decay_join_kernel(const __grid_constant__ DecayPass a) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const unsigned size = a.m * a.dv, tiles = (size + kThreads - 1) / kThreads;
  const unsigned bh = blockIdx.x / tiles, b = bh / (unsigned)a.H;
  const unsigned e = (blockIdx.x - bh * tiles) * kThreads + threadIdx.x;
  if (e >= size) return;
  const unsigned i = e / (unsigned)a.dv, j = e - i * a.dv;
  const int64_t n = row_length(a.lengths, b, a.T);
  const float g = decay_rate(a.log_decay, (int)(bh - b * (unsigned)a.H));
  const int64_t seat = (int64_t)bh * size + i * a.si + j * a.sj;
  float X = a.S_init ? a.S_init[seat] : 0.f;
  const Carries carries(g, (unsigned)a.run_len, (unsigned)n);
  float* st = a.states + (int64_t)bh * a.runs * size + e;
  for (int s0 = 0; s0 < a.runs; s0 += kAhead) {
    float U[kAhead];
#pragma unroll
    for (int s = 0; s < kAhead; ++s)
      if (s0 + s < a.runs) U[s] = st[(int64_t)(a.rev ? a.runs - 1 - s0 - s : s0 + s) * size];
#pragma unroll
    for (int s = 0; s < kAhead; ++s) {
      if (s0 + s >= a.runs) break;
      const int r = a.rev ? a.runs - 1 - s0 - s : s0 + s;
      st[(int64_t)r * size] = X;
      const int64_t len = run_tokens(n, r, a.run_len);
      X = (len > 0 ? carries.after(len, a.run_len).of(X) : X) + U[s];
    }
  }
  if (a.S_out) a.S_out[seat] = X;
}

struct ReadSmem {
  float q[kKeys * kLd], k[kKeys * kLd];  // transposed: [key][token]
  float v[kChunk * kLd];                 // [token][value]
  float p[kChunk * kLd];                 // [source][token]; then weighted keys [token][key]
  float S[128 * kLd];                    // [key][value]
};

template <typename E>
__global__ void __launch_bounds__(kThreads)
    decay_read_kernel(const __grid_constant__ DecayPass a) {
  extern __shared__ __align__(16) unsigned char raw[];
  ReadSmem& sm = *reinterpret_cast<ReadSmem*>(raw);
  const int run = blockIdx.x % a.runs;
  const int64_t bh = blockIdx.x / a.runs, b = bh / a.H;
  const int h = (int)(bh % a.H), tid = threadIdx.x, j0 = blockIdx.y * kTile;
  const int64_t n = row_length(a.lengths, b, a.T);
  const float g = decay_rate(a.log_decay, h);
  const E* q = static_cast<const E*>(a.q) + b * a.qs.batch + h * a.qs.head;
  const E* k = static_cast<const E*>(a.k) + b * a.ks.batch + h * a.ks.head;
  const E* v = static_cast<const E*>(a.v) + b * a.vs.batch + h * a.vs.head;
  E* o = static_cast<E*>(a.o) + b * a.os.batch + h * a.os.head;
  const int ti = (tid >> 4) * 4, tj = (tid & 15) * 4;
  const int mpad = (a.m + kKeys - 1) / kKeys * kKeys;
  const int64_t first = run * a.run_len;
  const int64_t end = first + a.run_len < a.T ? first + a.run_len : a.T;
  const int chunks = (int)((end - first + kChunk - 1) / kChunk);
  // the state entering the run; where a row is one run, the call's own
  const float* X = a.whole ? a.S_init : a.states + (bh * a.runs + run) * a.m * a.dv;
  const int si = a.whole ? a.si : a.dv, sj = a.whole ? a.sj : 1;
  const int64_t seat = a.whole ? bh * a.m * a.dv : 0;
  for (int e = tid; e < mpad * kTile; e += kThreads) {
    const int i = e / kTile, j = e % kTile;
    sm.S[i * kLd + j] =
        X && i < a.m && j0 + j < a.dv ? X[seat + i * si + (j0 + j) * sj] : 0.f;
  }
  for (int cc = 0; cc < chunks; ++cc) {
    const int64_t t0 = first + (int64_t)(a.rev ? chunks - 1 - cc : cc) * kChunk;
    const int have = (int)run_tokens(n, 0, t0 + kChunk) - (int)(n < t0 ? n : t0);
    const int rows = (int)(end - t0 < kChunk ? end - t0 : kChunk);
    float P[4][4] = {}, O[4][4] = {};
    if (have > 0) {
      constexpr int kEach = kChunk * kTile / 4 / kThreads;  // quads of a thread
      for (int mk = 0; mk < a.m; mk += kKeys) {
        // all loads under way before the first is stored
        float4 x[kEach], y[kEach], z[kEach];
#pragma unroll
        for (int u = 0; u < kEach; ++u) {
          const int e = tid + u * kThreads, r = e % kChunk, c = e / kChunk * 4;
          const int vr = e / (kTile / 4), vc = e % (kTile / 4) * 4;
          x[u] = y[u] = z[u] = make_float4(0.f, 0.f, 0.f, 0.f);
          if (r < have) {
            x[u] = row_quad<E>(q + (t0 + r) * a.qs.time, mk + c, a.m, a.vec_q);
            y[u] = row_quad<E>(k + (t0 + r) * a.ks.time, mk + c, a.m, a.vec_k);
          }
          if (mk == 0 && vr < have)
            z[u] = row_quad<E>(v + (t0 + vr) * a.vs.time, j0 + vc, a.dv, a.vec_v);
        }
        __syncthreads();
#pragma unroll
        for (int u = 0; u < kEach; ++u) {
          const int e = tid + u * kThreads, r = e % kChunk, c = e / kChunk * 4;
          sm.q[c * kLd + r] = x[u].x, sm.q[(c + 1) * kLd + r] = x[u].y;
          sm.q[(c + 2) * kLd + r] = x[u].z, sm.q[(c + 3) * kLd + r] = x[u].w;
          sm.k[c * kLd + r] = y[u].x, sm.k[(c + 1) * kLd + r] = y[u].y;
          sm.k[(c + 2) * kLd + r] = y[u].z, sm.k[(c + 3) * kLd + r] = y[u].w;
          if (mk == 0)
            *reinterpret_cast<float4*>(sm.v + e / (kTile / 4) * kLd + e % (kTile / 4) * 4) = z[u];
        }
        __syncthreads();
        const int keys = a.m - mk < kKeys ? a.m - mk : kKeys;
        outer_sum(P, sm.q + ti, sm.k + tj, keys);
        outer_sum(O, sm.q + ti, sm.S + mk * kLd + tj, keys);
      }
      const float intra = a.inter * a.w;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = ti + i;
        const float far = a.inter * decay_power(g, (float)(a.rev ? max(have - 1 - r, 0) : r + 1));
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          O[i][j] *= far;
          const int gap = a.rev ? tj + j - r : r - tj - j;
          P[i][j] = gap >= 0 ? P[i][j] * intra * decay_power(g, (float)gap) : 0.f;
        }
      }
#pragma unroll
      for (int j = 0; j < 4; ++j)
        *reinterpret_cast<float4*>(sm.p + (tj + j) * kLd + ti) =
            make_float4(P[0][j], P[1][j], P[2][j], P[3][j]);
      __syncthreads();
      outer_sum(O, sm.p + ti, sm.v + tj, kChunk);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = ti + i;
      if (r >= rows) break;
      E* to = o + (t0 + r) * a.os.time + j0 + tj;
      const int cols = a.dv - j0 - tj;
      const bool live = r < have;
      if (a.vec_o && cols >= 4) {
        *reinterpret_cast<typename Raw<E>::Quad*>(to) =
            narrow(live ? make_float4(O[i][0], O[i][1], O[i][2], O[i][3])
                        : make_float4(0.f, 0.f, 0.f, 0.f),
                   typename Raw<E>::Quad());
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (j < cols) store_vec<E, 1>(to + j, FloatV<1>{{live ? O[i][j] : 0.f}});
      }
    }
    if (have > 0 && (cc + 1 < chunks || (a.whole && a.S_out))) {
      const Carry carry(g, (float)have);
      for (int mk = 0; mk < a.m; mk += kTile) {
        __syncthreads();
        for (int e = tid; e < kChunk * (kTile / 4); e += kThreads) {
          const int r = e / (kTile / 4), c = e % (kTile / 4) * 4;
          float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
          if (r < have) {
            x = row_quad<E>(k + (t0 + r) * a.ks.time, mk + c, a.m, a.vec_k);
            const float wt = a.w * decay_power(g, (float)(a.rev ? r + 1 : have - 1 - r));
            x.x *= wt, x.y *= wt, x.z *= wt, x.w *= wt;
          }
          *reinterpret_cast<float4*>(sm.p + r * kLd + c) = x;
        }
        __syncthreads();
        float U[4][4] = {};
        outer_sum(U, sm.p + ti, sm.v + tj, kChunk);
        if (mk + ti < mpad) {
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              float& S = sm.S[(mk + ti + i) * kLd + tj + j];
              S = carry.of(S) + U[i][j];
            }
        }
      }
      __syncthreads();
    }
  }
  if (a.whole && a.S_out) {
    __syncthreads();
    for (int e = tid; e < a.m * kTile; e += kThreads) {
      const int i = e / kTile, j = e % kTile;
      if (j0 + j < a.dv) a.S_out[seat + i * si + (j0 + j) * sj] = sm.S[i * kLd + j];
    }
  }
}

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Runs of a row, of whole chunks: as many as make the last block's work shortest when
// `want` blocks take the runs of all heads in turn, a run costing its chunks and `extra`
// of one: its set-up, and the state that is written, joined and read back.  96 heads of 16
// chunks over 152 blocks: 3 runs of 6 chunks, of which a block takes up to two (10.1 chunks
// a block would be even).  No run has more than `longest` chunks.
void split_runs(DecayPass* p, int chunk, int64_t want, double extra, int64_t longest) {
  const int64_t chunks = ceil_div(p->T, chunk), heads = p->B * p->H;
  int64_t best = chunks ? chunks : 1;
  double least = -1.;
  const int64_t first = ceil_div(heads, want);
  for (int64_t t = first; t < first + 4 && chunks; ++t) {
    const int64_t most = t * want / heads, few = ceil_div(chunks, longest);
    const int64_t runs = most < few ? few : most < chunks ? most : chunks;
    const int64_t each = ceil_div(chunks, runs);
    const double cost =
        (double)ceil_div(heads * ceil_div(chunks, each), want) * ((double)each + extra);
    if (least < 0. || cost < least) least = cost, best = each;
  }
  p->run_len = best * chunk;
  p->runs = (int)ceil_div(p->T, p->run_len);
}

constexpr int64_t kSimtBlocks = 608;  // four blocks for each of 152 SMs

DecayPass shape_pass(const falcon_decay_shape& s, int m, int dv, bool tc) {
  DecayPass p = {};
  p.B = s.B, p.H = s.H, p.T = s.T;
  p.m = m, p.dv = dv, p.dtype = s.dtype;
  if (tc)
    split_runs(&p, kDecayTcChunk, kDecayTcBlocks, 0.5, kDecayTcRun);
  else
    split_runs(&p, kChunk, kSimtBlocks, 1., p.T);
  return p;
}
bool quads(const void* p, const falcon_strides& s, int dtype) {
  const uintptr_t bytes = dtype == FALCON_BF16 ? 8 : 16;
  return reinterpret_cast<uintptr_t>(p) % bytes == 0 && s.batch % 4 == 0 && s.head % 4 == 0 &&
         s.time % 4 == 0;
}

template <typename E>
cudaError_t run_pass(DecayPass& p, cudaStream_t stream) {
  static std::atomic<uint64_t> allowed{0};
  p.vec_q = quads(p.q, p.qs, p.dtype), p.vec_k = quads(p.k, p.ks, p.dtype);
  p.vec_v = quads(p.v, p.vs, p.dtype), p.vec_o = quads(p.o, p.os, p.dtype);
  const int64_t bh = p.B * p.H;
  // Rows that are one run carry their state themselves: one launch instead of three.  Of
  // few chunks they are made one (fp32, 2 heads of 64: T 64 13.8 us for 18.3 in a graph, T
  // 128 25.1 for 18.5, but a call by itself 18.5 for the host's 25; 1024 heads 82.7 for 128 and
  // 166 for 229).
  if (p.T > 0 && p.T <= kWholeTokens) p.runs = 1, p.run_len = kWholeTokens;
  p.whole = p.runs == 1;
  const unsigned grid = (unsigned)(bh * p.runs);
  const unsigned vt = (unsigned)ceil_div(p.dv, kTile), mt = (unsigned)ceil_div(p.m, kTile);
  if (p.runs > 0 && !p.whole)
    decay_states_kernel<E><<<dim3(grid, mt * vt), kThreads, 0, stream>>>(p);
  cudaError_t e = p.whole ? cudaSuccess : launch_decay_join(p, false, stream);
  if (e != cudaSuccess) return e;
  if (p.runs > 0) {
    e = allow_shared(decay_read_kernel<E>, sizeof(ReadSmem), &allowed);
    if (e != cudaSuccess) return e;
    decay_read_kernel<E><<<dim3(grid, vt), kThreads, sizeof(ReadSmem), stream>>>(p);
  }
  return cudaGetLastError();
}

// A pass with its tensors set, on the tensor cores; false where they do not fit.
// Rows of one chunk here take one launch, against three there: a call by itself takes the
// host 19 us for 26 (in a graph 15 us here for 9 there with 2 heads of 64, 83 for 75 with
// 1024; longer rows 27 for 9.6 and 156 for 77).
bool tc_pass(const falcon_decay_shape& s, DecayPass p, cudaError_t* e, cudaStream_t stream) {
  if (p.T <= kTcFrom) return false;
  const DecayPass split = shape_pass(s, p.m, p.dv, true);
  p.runs = split.runs, p.run_len = split.run_len;
  return decay_tc_pass(p, e, stream);
}
cudaError_t simt_pass(const falcon_decay_shape& s, DecayPass p, cudaStream_t stream) {
  const DecayPass split = shape_pass(s, p.m, p.dv, false);
  p.runs = split.runs, p.run_len = split.run_len;
  return p.dtype == FALCON_BF16 ? run_pass<__nv_bfloat16>(p, stream) : run_pass<float>(p, stream);
}

}  // namespace

cudaError_t launch_decay_join(const DecayPass& p, bool early, cudaStream_t stream) {
  const int64_t blocks = p.B * p.H * ceil_div((int64_t)p.m * p.dv, kThreads);
  return launch_behind(early, decay_join_kernel, (unsigned)blocks, kThreads, 0, stream, p);
}

// Room for either path: which one a pass takes goes by its pointers and strides too.  The
// gradient's passes use the same room one after another.
size_t decay_workspace_bytes(const falcon_decay_shape& s) {
  const int runs[2] = {shape_pass(s, s.m, s.dv, false).runs, shape_pass(s, s.m, s.dv, true).runs};
  const size_t most = (size_t)(runs[0] > runs[1] ? runs[0] : runs[1]);
  return ((size_t)s.B * s.H * most * s.m * s.dv * 4 + 255) / 256 * 256;
}

cudaError_t launch_decay_fwd(const DecayCall& c, cudaStream_t stream) {
  DecayPass p = shape_pass(c.s, c.s.m, c.s.dv, false);
  p.q = c.q, p.k = c.k, p.v = c.v, p.o = c.o;
  p.qs = c.qs, p.ks = c.ks, p.vs = c.vs, p.os = c.os;
  p.log_decay = c.log_decay, p.lengths = c.lengths;
  p.S_init = c.S0, p.S_out = c.S_out;
  p.si = c.s.dv, p.sj = 1;
  p.inter = c.s.scale, p.w = 1.f;
  p.states = static_cast<float*>(c.ws);
  p.sums = true, p.behind_reads = true;
  p.xi = c.s.dv, p.xj = 1;
  cudaError_t e = cudaSuccess;
  return tc_pass(c.s, p, &e, stream) ? e : simt_pass(c.s, p, stream);
}

cudaError_t launch_decay_bwd(const DecayCall& c, cudaStream_t stream) {
  const int m = c.s.m, dv = c.s.dv;
  // dq = scale S_t dO_t: the forward pass with (dO, v, k), its state transposed
  DecayPass p = shape_pass(c.s, dv, m, false);
  p.log_decay = c.log_decay, p.lengths = c.lengths;
  p.states = static_cast<float*>(c.ws);
  p.q = c.dO, p.k = c.v, p.v = c.k, p.o = c.dq;
  p.qs = c.dos, p.ks = c.vs, p.vs = c.ks, p.os = c.dqs;
  p.S_init = c.S0;
  p.si = 1, p.sj = dv;
  p.inter = c.s.scale, p.w = 1.f;
  p.sums = true, p.behind_reads = true;
  p.xi = m, p.xj = 1;
  cudaError_t e = cudaSuccess;
  const bool behind = tc_pass(c.s, p, &e, stream);
  if (!behind) e = simt_pass(c.s, p, stream);
  if (e != cudaSuccess) return e;
  p.rev = 1;
  p.inter = 1.f, p.w = c.s.scale;
  p.S_init = c.dS_T;
  // dv = G_t^T k_t, backward in time with (k, q, dO)
  DecayPass v = p;
  v.m = m, v.dv = dv;
  v.q = c.k, v.k = c.q, v.v = c.dO, v.o = c.dv;
  v.qs = c.ks, v.ks = c.qs, v.vs = c.dos, v.os = c.dvs;
  v.S_out = c.dS0;
  v.si = dv, v.sj = 1;
  v.xi = dv, v.xj = 1;
  // dk = G_t v_t, backward in time with (v, dO, q)
  DecayPass k = p;
  k.m = dv, k.dv = m;
  k.q = c.v, k.k = c.dO, k.v = c.q, k.o = c.dk;
  k.qs = c.vs, k.ks = c.dos, k.vs = c.qs, k.os = c.dks;
  k.si = 1, k.sj = dv;
  k.xi = m, k.xj = 1;
  if (c.dS_T && c.dS0 == c.dS_T) {  // in place: nothing reads dS_T behind the pass that writes dS0
    k.behind_states = behind;
    const bool first = tc_pass(c.s, k, &e, stream);
    if (!first) e = simt_pass(c.s, k, stream);
    if (e != cudaSuccess) return e;
    v.behind_states = first;
    return tc_pass(c.s, v, &e, stream) ? e : simt_pass(c.s, v, stream);
  }
  v.behind_states = behind;
  const bool kept = tc_pass(c.s, v, &e, stream);  // its states serve dk too
  if (!kept) e = simt_pass(c.s, v, stream);
  if (e != cudaSuccess) return e;
  DecayPass last = k;  // forms its own where dv's tensors did not fit
  if (kept) last.sums = false, last.xi = 1, last.xj = dv;
  return tc_pass(c.s, last, &e, stream) ? e : simt_pass(c.s, k, stream);
}

}  // namespace falcon
