// C ABI of the selective state space block (declared in include/falcon.h):
// argument checks, empty problems, and dispatch.  Nothing is launched when an
// argument is rejected.
#include <math.h>
#include <stdint.h>

#include <algorithm>
#include <memory>
#include <new>

#include "ssm.cuh"

namespace {

constexpr int64_t kMostGrid = 0x7fffffffLL;

bool element_aligned(const void* p, int bytes) {
  return reinterpret_cast<uintptr_t>(p) % (uintptr_t)bytes == 0;
}
bool negative(const falcon_strides* s) {
  return s && (s->batch < 0 || s->head < 0 || s->time < 0);
}
// An output's rows must not lie on one another.
bool on_itself(const falcon_strides* s, int64_t B, int64_t H, int64_t T) {
  return (B > 1 && s->batch == 0) || (H > 1 && s->head == 0) || (T > 1 && s->time == 0);
}
int to_status(cudaError_t e) { return e == cudaSuccess ? FALCON_OK : FALCON_ERR_CUDA; }

template <int N>
bool any_misaligned(const void* const (&p)[N], int bytes) {
  for (const void* q : p)
    if (!element_aligned(q, bytes)) return true;
  return false;
}

int check_conv(const falcon_conv_shape* s) {
  if (!s) return FALCON_ERR_NULL_PTR;
  if (s->B < 0 || s->H < 0 || s->T < 0 || s->m < 1 || s->width < 2 || s->width > 4)
    return FALCON_ERR_BAD_SHAPE;
  if (s->B > kMostGrid || s->T > kMostGrid || s->H > kMostGrid / s->m) return FALCON_ERR_BAD_SHAPE;
  if (s->dtype != FALCON_BF16 && s->dtype != FALCON_F32) return FALCON_ERR_BAD_DTYPE;
  if (s->activation != FALCON_ACT_IDENTITY && s->activation != FALCON_ACT_SILU)
    return FALCON_ERR_BAD_ARG;
  return FALCON_OK;
}

int check_scan(int64_t B, int64_t T, int32_t D, int32_t G, int32_t N, int32_t dtype) {
  if (B < 0 || T < 0 || D < 0 || G < 1 || D % G != 0 || N < 1 || N > 128)
    return FALCON_ERR_BAD_SHAPE;
  if (B > 65535 || T > kMostGrid) return FALCON_ERR_BAD_SHAPE;
  if (dtype != FALCON_BF16 && dtype != FALCON_F32) return FALCON_ERR_BAD_DTYPE;
  return FALCON_OK;
}

int esize(int dtype) { return dtype == FALCON_BF16 ? 2 : 4; }

// A clipped gradient's place.
struct Place {
  uintptr_t first, end;
  int64_t index;
};
Place place_of(const falcon_grad& g, const void* p, int64_t index) {
  const uintptr_t at = reinterpret_cast<uintptr_t>(p);
  return {at, at + (uintptr_t)g.count * (uintptr_t)esize(g.dtype), index};
}

// Every result must have its place to itself, and share it with no gradient but its own:
// blocks scale their parts in no order.
int check_clip_places(const falcon_grad* grads, int64_t tensors) {
  // results in rising order, in place or all apart from the gradients: no need to sort
  bool rising = true, in_place = true;
  uintptr_t last = 0, lo[2] = {UINTPTR_MAX, UINTPTR_MAX}, hi[2] = {0, 0};
  for (int64_t i = 0; i < tensors; ++i) {
    const falcon_grad& g = grads[i];
    if (g.count == 0) continue;
    const Place from = place_of(g, g.grad, i), to = place_of(g, g.out, i);
    rising = rising && to.first >= last;
    last = to.end;
    in_place = in_place && from.first == to.first;
    lo[0] = std::min(lo[0], from.first), hi[0] = std::max(hi[0], from.end);
    lo[1] = std::min(lo[1], to.first), hi[1] = std::max(hi[1], to.end);
  }
  const bool apart = hi[0] <= lo[1] || hi[1] <= lo[0];
  if (rising && (in_place || apart)) return FALCON_OK;
  const std::unique_ptr<Place[]> out(new (std::nothrow) Place[(size_t)tensors]);
  if (!out) return FALCON_ERR_WORKSPACE;
  int64_t n = 0;
  for (int64_t i = 0; i < tensors; ++i)
    if (grads[i].count > 0) out[n++] = place_of(grads[i], grads[i].out, i);
  std::sort(out.get(), out.get() + n,
            [](const Place& a, const Place& b) { return a.first < b.first; });
  for (int64_t i = 1; i < n; ++i)
    if (out[i].first < out[i - 1].end) return FALCON_ERR_BAD_ARG;
  if (in_place || apart) return FALCON_OK;
  for (int64_t i = 0; i < tensors; ++i) {
    if (grads[i].count == 0) continue;
    const Place g = place_of(grads[i], grads[i].grad, i);
    const Place* p = std::upper_bound(out.get(), out.get() + n, g.first,
                                      [](uintptr_t at, const Place& q) { return at < q.end; });
    if (p != out.get() + n && p->first < g.end && (p->index != i || p->first != g.first))
      return FALCON_ERR_BAD_ARG;
  }
  return FALCON_OK;
}

falcon::ConvArgs conv_args(const falcon_conv_shape* s) {
  falcon::ConvArgs a = {};
  a.B = s->B;
  a.H = s->H;
  a.T = s->T;
  a.m = s->m;
  a.width = s->width;
  a.dtype = s->dtype;
  a.act = s->activation;
  a.C = s->H * s->m;
  return a;
}

}  // namespace

extern "C" {

int falcon_short_conv_fwd(const falcon_conv_shape* s, const void* x, const falcon_strides* xs,
                          const float* weight, const float* bias, const void* state,
                          const int32_t* lengths, void* y, const falcon_strides* ys,
                          void* state_out, cudaStream_t stream) {
  int rc = check_conv(s);
  if (rc) return rc;
  if (s->B == 0 || s->H == 0) return FALCON_OK;
  if (!xs || !ys || !weight || (s->T > 0 && (!x || !y))) return FALCON_ERR_NULL_PTR;
  if (negative(xs) || negative(ys) || (state && state == state_out)) return FALCON_ERR_BAD_ARG;
  const void* acts[] = {x, y, state, state_out};
  const void* words[] = {weight, bias, lengths};
  if (any_misaligned(acts, esize(s->dtype)) || any_misaligned(words, 4))
    return FALCON_ERR_MISALIGNED;
  // a run reads rows that the run before it would have written
  if (s->T > 0 && (x == y || on_itself(ys, s->B, s->H, s->T))) return FALCON_ERR_BAD_ARG;
  rc = falcon::check_sm103_device();
  if (rc) return rc;
  falcon::ConvArgs a = conv_args(s);
  a.xs = *xs;
  a.ys = *ys;
  a.x = x;
  a.weight = weight;
  a.bias = bias;
  a.state = state;
  a.lengths = lengths;
  a.y = y;
  a.state_out = state_out;
  return to_status(falcon::launch_conv_fwd(a, stream));
}

size_t falcon_short_conv_bwd_workspace_bytes(const falcon_conv_shape* s) {
  if (check_conv(s) != FALCON_OK) return 0;
  return falcon::conv_bwd_workspace_bytes(s->B, s->T, s->H * s->m, s->width);
}

int falcon_short_conv_bwd(const falcon_conv_shape* s, const void* x, const falcon_strides* xs,
                          const float* weight, const float* bias, const void* state,
                          const int32_t* lengths, const void* dy, const falcon_strides* dys,
                          const void* dstate_out, void* dx, const falcon_strides* dxs,
                          float* dweight, float* dbias, void* dstate, void* workspace,
                          size_t workspace_bytes, cudaStream_t stream) {
  int rc = check_conv(s);
  if (rc) return rc;
  if (s->H == 0) return FALCON_OK;
  if (!xs || !dys || !dxs || !weight || !dweight) return FALCON_ERR_NULL_PTR;
  if (s->B > 0 && s->T > 0 && (!x || !dy || !dx)) return FALCON_ERR_NULL_PTR;
  if (negative(xs) || negative(dys) || negative(dxs)) return FALCON_ERR_BAD_ARG;
  if (dstate && (dstate == dstate_out || dstate == state)) return FALCON_ERR_BAD_ARG;
  const void* acts[] = {x, dy, dx, state, dstate_out, dstate};
  const void* words[] = {weight, bias, lengths, dweight, dbias};
  if (any_misaligned(acts, esize(s->dtype)) || any_misaligned(words, 4))
    return FALCON_ERR_MISALIGNED;
  const size_t need = falcon_short_conv_bwd_workspace_bytes(s);
  if (need > 0 && (!workspace || workspace_bytes < need)) return FALCON_ERR_WORKSPACE;
  if (!element_aligned(workspace, 16)) return FALCON_ERR_MISALIGNED;
  if (s->B > 0 && s->T > 0 && (dx == x || dx == dy || on_itself(dxs, s->B, s->H, s->T)))
    return FALCON_ERR_BAD_ARG;
  rc = falcon::check_sm103_device();
  if (rc) return rc;
  falcon::ConvArgs a = conv_args(s);
  a.xs = *xs;
  a.dys = *dys;
  a.dxs = *dxs;
  a.x = x;
  a.weight = weight;
  a.bias = bias;
  a.state = state;
  a.lengths = lengths;
  a.dy = dy;
  a.dstate_out = dstate_out;
  a.dx = dx;
  a.dstate = dstate;
  a.dweight = dweight;
  a.dbias = dbias;
  a.ws = static_cast<float*>(workspace);
  return to_status(falcon::launch_conv_bwd(a, stream));
}

int falcon_short_conv_step(int64_t N, int32_t C, int32_t width, int32_t dtype, int32_t activation,
                           const void* x, int64_t x_stride, const float* weight,
                           const float* bias, void* state, int64_t pool, const int32_t* slots,
                           const uint8_t* fresh, void* y, cudaStream_t stream) {
  if (N < 0 || C < 0 || pool < 0 || width < 2 || width > 4) return FALCON_ERR_BAD_SHAPE;
  if (dtype != FALCON_BF16 && dtype != FALCON_F32) return FALCON_ERR_BAD_DTYPE;
  if (activation != FALCON_ACT_IDENTITY && activation != FALCON_ACT_SILU)
    return FALCON_ERR_BAD_ARG;
  if (x_stride < 0) return FALCON_ERR_BAD_ARG;
  if (N == 0 || C == 0) return FALCON_OK;
  if (N > kMostGrid / C) return FALCON_ERR_BAD_SHAPE;
  if (!x || !weight || !y || (pool > 0 && !state)) return FALCON_ERR_NULL_PTR;
  const void* acts[] = {x, y, state};
  const void* words[] = {weight, bias, slots};
  if (any_misaligned(acts, esize(dtype)) || any_misaligned(words, 4)) return FALCON_ERR_MISALIGNED;
  int rc = falcon::check_sm103_device();
  if (rc) return rc;
  falcon::ConvStepArgs a = {};
  a.N = N;
  a.pool = pool;
  a.x_stride = x_stride;
  a.C = C;
  a.width = width;
  a.dtype = dtype;
  a.act = activation;
  a.x = x;
  a.weight = weight;
  a.bias = bias;
  a.state = state;
  a.slots = slots;
  a.fresh = fresh;
  a.y = y;
  return to_status(falcon::launch_conv_step(a, stream));
}

int falcon_selective_scan_fwd(const falcon_scan_shape* s, const void* u, const falcon_strides* us,
                              const void* delta, const falcon_strides* ds, const float* A,
                              const void* Bm, const falcon_strides* bs, const void* Cm,
                              const falcon_strides* cs, const float* Dskip, const void* z,
                              const falcon_strides* zs, const float* delta_bias, const float* h0,
                              const int32_t* lengths, void* y, const falcon_strides* ys,
                              float* h_out, cudaStream_t stream) {
  if (!s) return FALCON_ERR_NULL_PTR;
  int rc = check_scan(s->B, s->T, s->D, s->G, s->N, s->dtype);
  if (rc) return rc;
  if (s->B == 0 || s->D == 0) return FALCON_OK;
  if (!us || !ds || !bs || !cs || !ys || (z && !zs) || !A || !h_out) return FALCON_ERR_NULL_PTR;
  if (s->T > 0 && (!u || !delta || !Bm || !Cm || !y)) return FALCON_ERR_NULL_PTR;
  if (negative(us) || negative(ds) || negative(bs) || negative(cs) || negative(ys) ||
      (z && negative(zs)))
    return FALCON_ERR_BAD_ARG;
  const void* acts[] = {u, delta, Bm, Cm, z, y};
  const void* words[] = {A, Dskip, delta_bias, h0, h_out, lengths};
  if (any_misaligned(acts, esize(s->dtype)) || any_misaligned(words, 4))
    return FALCON_ERR_MISALIGNED;
  if (s->T > 0 && on_itself(ys, s->B, 1, s->T)) return FALCON_ERR_BAD_ARG;
  rc = falcon::check_sm103_device();
  if (rc) return rc;
  falcon::ScanArgs a = {};
  a.B = s->B;
  a.T = s->T;
  a.D = s->D;
  a.G = s->G;
  a.N = s->N;
  a.dtype = s->dtype;
  a.softplus = s->softplus != 0;
  a.us = *us;
  a.ds = *ds;
  a.bs = *bs;
  a.cs = *cs;
  a.ys = *ys;
  if (z) a.zs = *zs;
  a.u = u;
  a.delta = delta;
  a.Bm = Bm;
  a.Cm = Cm;
  a.z = z;
  a.A = A;
  a.Dskip = Dskip;
  a.delta_bias = delta_bias;
  a.h0 = h0;
  a.lengths = lengths;
  a.y = y;
  a.h_out = h_out;
  return to_status(falcon::launch_scan_fwd(a, stream));
}

size_t falcon_selective_scan_bwd_workspace_bytes(const falcon_scan_shape* s) {
  if (!s || check_scan(s->B, s->T, s->D, s->G, s->N, s->dtype) != FALCON_OK) return 0;
  if (s->B == 0 || s->D == 0) return 0;
  return falcon::scan_bwd_workspace_bytes(*s);
}

int falcon_selective_scan_bwd(const falcon_scan_shape* s, const void* u, const falcon_strides* us,
                              const void* delta, const falcon_strides* ds, const float* A,
                              const void* Bm, const falcon_strides* bs, const void* Cm,
                              const falcon_strides* cs, const float* Dskip, const void* z,
                              const falcon_strides* zs, const float* delta_bias, const float* h0,
                              const int32_t* lengths, const void* dy, const falcon_strides* dys,
                              const float* dh_T, void* du, void* ddelta, float* dA, void* dB,
                              void* dC, float* dDskip, void* dz, float* ddelta_bias, float* dh0,
                              void* workspace, size_t workspace_bytes, cudaStream_t stream) {
  if (!s) return FALCON_ERR_NULL_PTR;
  int rc = check_scan(s->B, s->T, s->D, s->G, s->N, s->dtype);
  if (rc) return rc;
  if (s->D == 0) return FALCON_OK;
  if (!us || !ds || !bs || !cs || !dys || (z && !zs) || !A || !dA) return FALCON_ERR_NULL_PTR;
  if (s->B > 0 && s->T > 0 &&
      (!u || !delta || !Bm || !Cm || !dy || !du || !ddelta || !dB || !dC || (z && !dz)))
    return FALCON_ERR_NULL_PTR;
  if (negative(us) || negative(ds) || negative(bs) || negative(cs) || negative(dys) ||
      (z && negative(zs)) || (!z && dz))
    return FALCON_ERR_BAD_ARG;
  if (dh0 && dh0 == h0) return FALCON_ERR_BAD_ARG;  // written while other blocks read h0
  const void* acts[] = {u, delta, Bm, Cm, z, dy, du, ddelta, dB, dC, dz};
  const void* words[] = {A, Dskip, delta_bias, h0, lengths, dh_T, dA, dDskip, ddelta_bias, dh0};
  if (any_misaligned(acts, esize(s->dtype)) || any_misaligned(words, 4))
    return FALCON_ERR_MISALIGNED;
  const size_t need = falcon_selective_scan_bwd_workspace_bytes(s);
  if (need > 0 && (!workspace || workspace_bytes < need)) return FALCON_ERR_WORKSPACE;
  if (!element_aligned(workspace, 256)) return FALCON_ERR_MISALIGNED;
  rc = falcon::check_sm103_device();
  if (rc) return rc;
  if (s->B == 0) {  // no row: the parameters' gradients are zero
    cudaError_t e = cudaMemsetAsync(dA, 0, sizeof(float) * (size_t)s->D * s->N, stream);
    if (e == cudaSuccess && dDskip) e = cudaMemsetAsync(dDskip, 0, sizeof(float) * s->D, stream);
    if (e == cudaSuccess && ddelta_bias)
      e = cudaMemsetAsync(ddelta_bias, 0, sizeof(float) * s->D, stream);
    return to_status(e);
  }
  falcon::ScanArgs a = {};
  a.B = s->B;
  a.T = s->T;
  a.D = s->D;
  a.G = s->G;
  a.N = s->N;
  a.dtype = s->dtype;
  a.softplus = s->softplus != 0;
  a.us = *us;
  a.ds = *ds;
  a.bs = *bs;
  a.cs = *cs;
  a.dys = *dys;
  if (z) a.zs = *zs;
  a.u = u;
  a.delta = delta;
  a.Bm = Bm;
  a.Cm = Cm;
  a.z = z;
  a.A = A;
  a.Dskip = Dskip;
  a.delta_bias = delta_bias;
  a.h0 = h0;
  a.lengths = lengths;
  a.dy = dy;
  a.dh_T = dh_T;
  a.du = du;
  a.ddelta = ddelta;
  a.dA = dA;
  a.dB = dB;
  a.dC = dC;
  a.dDskip = dDskip;
  a.dz = dz;
  a.ddelta_bias = ddelta_bias;
  a.dh0 = dh0;
  a.ws = workspace;
  return to_status(falcon::launch_scan_bwd(a, stream));
}

int falcon_selective_scan_step(int64_t N, int32_t D, int32_t G, int32_t S, int32_t dtype,
                               int32_t softplus, const void* u, int64_t u_stride,
                               const void* delta, int64_t delta_stride, const float* A,
                               const void* Bm, const falcon_strides* bs, const void* Cm,
                               const falcon_strides* cs, const float* Dskip, const void* z,
                               int64_t z_stride, const float* delta_bias, float* h, int64_t pool,
                               const int32_t* slots, const uint8_t* fresh, void* y,
                               cudaStream_t stream) {
  int rc = check_scan(0, 0, D, G, S, dtype);
  if (rc) return rc;
  if (N < 0 || pool < 0) return FALCON_ERR_BAD_SHAPE;
  if (N == 0 || D == 0) return FALCON_OK;
  // rows along x, 128 lanes of channel pairs along y of the grid
  if (N > kMostGrid / D || D > (1 << 18)) return FALCON_ERR_BAD_SHAPE;
  if (!u || !delta || !A || !Bm || !Cm || !bs || !cs || !y || (pool > 0 && !h))
    return FALCON_ERR_NULL_PTR;
  if (u_stride < 0 || delta_stride < 0 || (z && z_stride < 0) || negative(bs) || negative(cs))
    return FALCON_ERR_BAD_ARG;
  const void* acts[] = {u, delta, Bm, Cm, z, y};
  const void* words[] = {A, Dskip, delta_bias, h, slots};
  if (any_misaligned(acts, esize(dtype)) || any_misaligned(words, 4)) return FALCON_ERR_MISALIGNED;
  rc = falcon::check_sm103_device();
  if (rc) return rc;
  falcon::ScanStepArgs a = {};
  a.N = N;
  a.pool = pool;
  a.u_stride = u_stride;
  a.delta_stride = delta_stride;
  a.z_stride = z_stride;
  a.D = D;
  a.G = G;
  a.S = S;
  a.dtype = dtype;
  a.softplus = softplus != 0;
  a.bs = *bs;
  a.cs = *cs;
  a.u = u;
  a.delta = delta;
  a.Bm = Bm;
  a.Cm = Cm;
  a.z = z;
  a.A = A;
  a.Dskip = Dskip;
  a.delta_bias = delta_bias;
  a.h = h;
  a.slots = slots;
  a.fresh = fresh;
  a.y = y;
  return to_status(falcon::launch_scan_step(a, stream));
}

size_t falcon_clip_workspace_bytes(const falcon_grad* grads, int64_t tensors) {
  if (tensors < 0 || (tensors > 0 && !grads)) return 0;
  return falcon::clip_workspace_bytes(grads, tensors);
}

int falcon_clip_grad_norm(const falcon_grad* grads, int64_t tensors, float max_norm, float eps,
                          float* norm, void* workspace, size_t workspace_bytes,
                          cudaStream_t stream) {
  if (tensors < 0) return FALCON_ERR_BAD_SHAPE;
  if ((tensors > 0 && !grads) || !norm) return FALCON_ERR_NULL_PTR;
  if (!(max_norm >= 0.f) || !(eps >= 0.f)) return FALCON_ERR_BAD_ARG;
  if (!element_aligned(norm, 4)) return FALCON_ERR_MISALIGNED;
  for (int64_t i = 0; i < tensors; ++i) {
    const falcon_grad& g = grads[i];
    if (g.count < 0) return FALCON_ERR_BAD_SHAPE;
    if (g.dtype != FALCON_BF16 && g.dtype != FALCON_F32) return FALCON_ERR_BAD_DTYPE;
    if (g.count > 0 && (!g.grad || !g.out)) return FALCON_ERR_NULL_PTR;
    if (!element_aligned(g.grad, esize(g.dtype)) || !element_aligned(g.out, esize(g.dtype)))
      return FALCON_ERR_MISALIGNED;
  }
  int rc = check_clip_places(grads, tensors);
  if (rc) return rc;
  const size_t need = falcon_clip_workspace_bytes(grads, tensors);
  if (!workspace || workspace_bytes < need) return FALCON_ERR_WORKSPACE;
  if (!element_aligned(workspace, 16)) return FALCON_ERR_MISALIGNED;
  rc = falcon::check_sm103_device();
  if (rc) return rc;
  return to_status(falcon::launch_clip(grads, tensors, max_norm, eps, norm, workspace, stream));
}

}  // extern "C"
