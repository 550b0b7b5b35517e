// C ABI of the linear attention block (declared in include/falcon.h): argument checks,
// empty problems, and dispatch.  Nothing is launched when an argument is rejected.
#include <math.h>
#include <stdint.h>

#include "linear.cuh"

namespace {

constexpr int64_t kMostGrid = 0x7fffffffLL;
constexpr int kMostWidth = 128, kMostRow = 8192;

bool aligned(const void* p, int bytes) {
  return reinterpret_cast<uintptr_t>(p) % (uintptr_t)bytes == 0;
}
template <int N>
bool any_misaligned(const void* const (&p)[N], int bytes) {
  for (const void* q : p)
    if (!aligned(q, bytes)) return true;
  return false;
}
template <int N>
bool any_negative(const falcon_strides* const (&s)[N]) {
  for (const falcon_strides* q : s)
    if (q && (q->batch < 0 || q->head < 0 || q->time < 0)) return true;
  return false;
}
template <int N>
bool among(const void* p, const void* const (&list)[N]) {
  if (!p) return false;
  for (const void* q : list)
    if (p == q) return true;
  return false;
}
// An output's rows must not lie on one another.
bool on_itself(const falcon_strides* s, int64_t B, int64_t H, int64_t T) {
  return (B > 1 && s->batch == 0) || (H > 1 && s->head == 0) || (T > 1 && s->time == 0);
}
bool same(const falcon_strides* x, const falcon_strides* y, int64_t B, int64_t T) {
  return (B <= 1 || x->batch == y->batch) && (T <= 1 || x->time == y->time);
}
int to_status(cudaError_t e) { return e == cudaSuccess ? FALCON_OK : FALCON_ERR_CUDA; }
int esize(int dtype) { return dtype == FALCON_BF16 ? 2 : 4; }
falcon_strides of(const falcon_strides* s) { return s ? *s : falcon_strides{0, 0, 0}; }

int check_decay(const falcon_decay_shape* s) {
  if (!s) return FALCON_ERR_NULL_PTR;
  if (s->B < 0 || s->H < 0 || s->T < 0 || s->m < 1 || s->dv < 1 || s->m > kMostWidth ||
      s->dv > kMostWidth)
    return FALCON_ERR_BAD_SHAPE;
  if (s->B > kMostGrid || s->H > kMostGrid || s->T > kMostGrid) return FALCON_ERR_BAD_SHAPE;
  // a block for every head and run of 64 tokens, a thread for every element of a state
  if (s->H > 0 && s->B > (1LL << 31) / s->H) return FALCON_ERR_BAD_SHAPE;
  const int64_t runs = s->T / 64 + 1;
  if (s->B * s->H > kMostGrid / (runs < 608 ? runs : 608)) return FALCON_ERR_BAD_SHAPE;
  if (s->B * s->H > kMostGrid / 64) return FALCON_ERR_BAD_SHAPE;
  if (s->dtype != FALCON_BF16 && s->dtype != FALCON_F32) return FALCON_ERR_BAD_DTYPE;
  if (!isfinite(s->scale)) return FALCON_ERR_BAD_ARG;
  return FALCON_OK;
}

int check_norm(const falcon_norm_shape* s) {
  if (!s) return FALCON_ERR_NULL_PTR;
  if (s->B < 0 || s->H < 1 || s->T < 0 || s->m < 1 || s->H > kMostRow ||
      s->H * s->m > kMostRow)
    return FALCON_ERR_BAD_SHAPE;
  if (s->B > kMostGrid || s->T > kMostGrid || (s->T > 0 && s->B > kMostGrid / s->T))
    return FALCON_ERR_BAD_SHAPE;
  if (s->dtype != FALCON_BF16 && s->dtype != FALCON_F32) return FALCON_ERR_BAD_DTYPE;
  if (s->gate != FALCON_ACT_IDENTITY && s->gate != FALCON_ACT_SILU &&
      s->gate != FALCON_ACT_SIGMOID)
    return FALCON_ERR_BAD_ARG;
  if (!(s->eps > 0.f) || !isfinite(s->eps)) return FALCON_ERR_BAD_ARG;
  return FALCON_OK;
}

falcon::NormArgs norm_args(const falcon_norm_shape* s) {
  falcon::NormArgs a = {};
  a.B = s->B, a.T = s->T, a.H = (int)s->H, a.m = s->m, a.D = (int)(s->H * s->m);
  a.dtype = s->dtype, a.gate = s->gate, a.eps = s->eps;
  return a;
}

}  // namespace

extern "C" {

size_t falcon_decay_attn_workspace_bytes(const falcon_decay_shape* s) {
  if (check_decay(s) != FALCON_OK || s->B == 0 || s->H == 0) return 0;
  return falcon::decay_workspace_bytes(*s);
}

int falcon_decay_attn_fwd(const falcon_decay_shape* s, const void* q, const falcon_strides* qs,
                          const void* k, const falcon_strides* ks, const void* v,
                          const falcon_strides* vs, const float* log_decay, const float* S0,
                          const int32_t* lengths, void* o, const falcon_strides* os,
                          float* S_out, void* workspace, size_t workspace_bytes,
                          cudaStream_t stream) {
  int rc = check_decay(s);
  if (rc) return rc;
  if (s->B == 0 || s->H == 0) return FALCON_OK;
  if (!qs || !ks || !vs || !os || !log_decay) return FALCON_ERR_NULL_PTR;
  if (s->T > 0 && (!q || !k || !v || !o)) return FALCON_ERR_NULL_PTR;
  const falcon_strides* strides[] = {qs, ks, vs, os};
  if (any_negative(strides)) return FALCON_ERR_BAD_ARG;
  const void* acts[] = {q, k, v, o};
  const void* words[] = {log_decay, S0, lengths, S_out};
  if (any_misaligned(acts, esize(s->dtype)) || any_misaligned(words, 4))
    return FALCON_ERR_MISALIGNED;
  const void* inputs[] = {q, k, v, S0, log_decay};
  if (s->T > 0 && (among(o, inputs) || o == S_out || on_itself(os, s->B, s->H, s->T)))
    return FALCON_ERR_BAD_ARG;
  if (S_out && (S_out == q || S_out == k || S_out == v || S_out == log_decay))
    return FALCON_ERR_BAD_ARG;
  const size_t need = falcon_decay_attn_workspace_bytes(s);
  if (need > 0 && (!workspace || workspace_bytes < need)) return FALCON_ERR_WORKSPACE;
  if (!aligned(workspace, 256)) return FALCON_ERR_MISALIGNED;
  rc = falcon::check_sm103_device();
  if (rc) return rc;
  falcon::DecayCall c = {};
  c.s = *s;
  c.q = q, c.k = k, c.v = v, c.o = o;
  c.qs = *qs, c.ks = *ks, c.vs = *vs, c.os = *os;
  c.log_decay = log_decay, c.S0 = S0, c.lengths = lengths, c.S_out = S_out;
  c.ws = workspace;
  return to_status(falcon::launch_decay_fwd(c, stream));
}

size_t falcon_decay_attn_bwd_workspace_bytes(const falcon_decay_shape* s) {
  if (check_decay(s) != FALCON_OK || s->B == 0 || s->H == 0) return 0;
  return falcon::decay_workspace_bytes(*s);
}

int falcon_decay_attn_bwd(const falcon_decay_shape* s, const void* q, const falcon_strides* qs,
                          const void* k, const falcon_strides* ks, const void* v,
                          const falcon_strides* vs, const float* log_decay, const float* S0,
                          const int32_t* lengths, const void* dO, const falcon_strides* dos,
                          const float* dS_T, void* dq, const falcon_strides* dqs, void* dk,
                          const falcon_strides* dks, void* dv, const falcon_strides* dvs,
                          float* dS0, void* workspace, size_t workspace_bytes,
                          cudaStream_t stream) {
  int rc = check_decay(s);
  if (rc) return rc;
  if (s->B == 0 || s->H == 0) return FALCON_OK;
  if (!qs || !ks || !vs || !dos || !dqs || !dks || !dvs || !log_decay)
    return FALCON_ERR_NULL_PTR;
  if (s->T > 0 && (!q || !k || !v || !dO || !dq || !dk || !dv)) return FALCON_ERR_NULL_PTR;
  const falcon_strides* strides[] = {qs, ks, vs, dos, dqs, dks, dvs};
  if (any_negative(strides)) return FALCON_ERR_BAD_ARG;
  const void* acts[] = {q, k, v, dO, dq, dk, dv};
  const void* words[] = {log_decay, S0, lengths, dS_T, dS0};
  if (any_misaligned(acts, esize(s->dtype)) || any_misaligned(words, 4))
    return FALCON_ERR_MISALIGNED;
  const void* inputs[] = {q, k, v, dO, S0, log_decay};
  if (s->T > 0) {
    if (among(dq, inputs) || among(dk, inputs) || among(dv, inputs)) return FALCON_ERR_BAD_ARG;
    const void* states[] = {dS_T, dS0};
    if (among(dq, states) || among(dk, states) || among(dv, states)) return FALCON_ERR_BAD_ARG;
    if (dq == dk || dq == dv || dk == dv) return FALCON_ERR_BAD_ARG;
    if (on_itself(dqs, s->B, s->H, s->T) || on_itself(dks, s->B, s->H, s->T) ||
        on_itself(dvs, s->B, s->H, s->T))
      return FALCON_ERR_BAD_ARG;
  }
  if (among(dS0, inputs)) return FALCON_ERR_BAD_ARG;
  const size_t need = falcon_decay_attn_bwd_workspace_bytes(s);
  if (need > 0 && (!workspace || workspace_bytes < need)) return FALCON_ERR_WORKSPACE;
  if (!aligned(workspace, 256)) return FALCON_ERR_MISALIGNED;
  rc = falcon::check_sm103_device();
  if (rc) return rc;
  falcon::DecayCall c = {};
  c.s = *s;
  c.q = q, c.k = k, c.v = v, c.dO = dO;
  c.qs = *qs, c.ks = *ks, c.vs = *vs, c.dos = *dos;
  c.log_decay = log_decay, c.S0 = S0, c.dS_T = dS_T, c.lengths = lengths;
  c.dq = dq, c.dk = dk, c.dv = dv, c.dS0 = dS0;
  c.dqs = *dqs, c.dks = *dks, c.dvs = *dvs;
  c.ws = workspace;
  return to_status(falcon::launch_decay_bwd(c, stream));
}

int falcon_decay_attn_step(const falcon_decay_shape* s, const void* q, const falcon_strides* qs,
                           const void* k, const falcon_strides* ks, const void* v,
                           const falcon_strides* vs, const float* log_decay, float* S,
                           int64_t pool, const int32_t* slots, const uint8_t* fresh, void* o,
                           cudaStream_t stream) {
  if (!s) return FALCON_ERR_NULL_PTR;
  falcon_decay_shape one = *s;
  one.T = 1;
  int rc = check_decay(&one);
  if (rc) return rc;
  if (pool < 0 || (!slots && pool < s->B)) return FALCON_ERR_BAD_SHAPE;
  if (s->B == 0 || s->H == 0) return FALCON_OK;
  if (!q || !k || !v || !qs || !ks || !vs || !log_decay || !o || (pool > 0 && !S))
    return FALCON_ERR_NULL_PTR;
  const falcon_strides* strides[] = {qs, ks, vs};
  if (any_negative(strides)) return FALCON_ERR_BAD_ARG;
  const void* acts[] = {q, k, v, o};
  const void* words[] = {log_decay, S, slots};
  if (any_misaligned(acts, esize(s->dtype)) || any_misaligned(words, 4))
    return FALCON_ERR_MISALIGNED;
  const void* inputs[] = {q, k, v, S, log_decay};
  if (among(o, inputs)) return FALCON_ERR_BAD_ARG;
  rc = falcon::check_sm103_device();
  if (rc) return rc;
  falcon::DecayStepArgs a = {};
  a.N = s->B, a.pool = pool;
  a.H = (int)s->H, a.m = s->m, a.dv = s->dv, a.dtype = s->dtype, a.scale = s->scale;
  a.qs = *qs, a.ks = *ks, a.vs = *vs;
  a.q = q, a.k = k, a.v = v;
  a.log_decay = log_decay, a.S = S, a.slots = slots, a.fresh = fresh, a.o = o;
  return to_status(falcon::launch_decay_step(a, stream));
}

int falcon_gated_norm_fwd(const falcon_norm_shape* s, const void* h, const falcon_strides* hs,
                          const float* weight, const void* z, const falcon_strides* zs,
                          const float* scale, const void* x, const falcon_strides* xs,
                          const float* next_weight, const int32_t* lengths, void* out,
                          const falcon_strides* os, void* next, const falcon_strides* ns,
                          cudaStream_t stream) {
  int rc = check_norm(s);
  if (rc) return rc;
  if (s->B == 0 || s->T == 0) return FALCON_OK;
  if (!h && (out || weight || scale || z)) return FALCON_ERR_BAD_ARG;
  if (h ? (!hs || !out || !os) : (!x || !next)) return FALCON_ERR_NULL_PTR;
  if ((z && !zs) || (x && !xs) || (next && !ns) || (next == nullptr) != (next_weight == nullptr))
    return FALCON_ERR_NULL_PTR;
  const falcon_strides* strides[] = {hs, zs, xs, os, ns};
  if (any_negative(strides)) return FALCON_ERR_BAD_ARG;
  const void* acts[] = {h, z, x, out, next};
  const void* words[] = {weight, scale, next_weight, lengths};
  if (any_misaligned(acts, esize(s->dtype)) || any_misaligned(words, 4))
    return FALCON_ERR_MISALIGNED;
  const void* others[] = {h, z, weight, scale, next_weight};
  if (among(out, others) || among(next, others) || (next && (next == out || next == x)))
    return FALCON_ERR_BAD_ARG;
  if (out && out == x && !same(os, xs, s->B, s->T)) return FALCON_ERR_BAD_ARG;
  if ((out && on_itself(os, s->B, 1, s->T)) || (next && on_itself(ns, s->B, 1, s->T)))
    return FALCON_ERR_BAD_ARG;
  rc = falcon::check_sm103_device();
  if (rc) return rc;
  falcon::NormArgs a = norm_args(s);
  a.h = h, a.z = z, a.x = x, a.out = out, a.next = next;
  a.hs = of(hs), a.zs = of(zs), a.xs = of(xs), a.os = of(os), a.ns = of(ns);
  a.weight = weight, a.scale = scale, a.next_weight = next_weight, a.lengths = lengths;
  return to_status(falcon::launch_norm_fwd(a, stream));
}

size_t falcon_gated_norm_bwd_workspace_bytes(const falcon_norm_shape* s) {
  if (check_norm(s) != FALCON_OK) return 0;
  return falcon::norm_bwd_workspace_bytes(*s);
}

int falcon_gated_norm_bwd(const falcon_norm_shape* s, const void* h, const falcon_strides* hs,
                          const float* weight, const void* z, const falcon_strides* zs,
                          const float* scale, const void* out, const falcon_strides* os,
                          const float* next_weight, const int32_t* lengths, const void* dout,
                          const falcon_strides* dos, const void* dnext,
                          const falcon_strides* dns, void* dx, const falcon_strides* dxs,
                          void* dh, const falcon_strides* dhs, void* dz,
                          const falcon_strides* dzs, float* dweight, float* dscale,
                          float* dnext_weight, void* workspace, size_t workspace_bytes,
                          cudaStream_t stream) {
  int rc = check_norm(s);
  if (rc) return rc;
  if ((dscale && !scale) || (dnext_weight && !next_weight)) return FALCON_ERR_BAD_ARG;
  if (s->B > 0 && s->T > 0) {
    if (!h && (weight || scale || z || dweight)) return FALCON_ERR_BAD_ARG;
    if (!h && !next_weight) return FALCON_ERR_NULL_PTR;
    if (!dout && !dnext) return FALCON_ERR_NULL_PTR;
    if ((h && (!hs || !dh || !dhs)) || (!h && dh)) return FALCON_ERR_NULL_PTR;
    if ((z == nullptr) != (dz == nullptr) || (z && (!zs || !dzs))) return FALCON_ERR_NULL_PTR;
    if (next_weight ? (!out || !os || !dnext || !dns) : dnext != nullptr)
      return FALCON_ERR_NULL_PTR;
    if ((dout && !dos) || (dx && !dxs)) return FALCON_ERR_NULL_PTR;
  }
  const falcon_strides* strides[] = {hs, zs, os, dos, dns, dxs, dhs, dzs};
  if (any_negative(strides)) return FALCON_ERR_BAD_ARG;
  const void* acts[] = {h, z, out, dout, dnext, dx, dh, dz};
  const void* words[] = {weight, scale, next_weight, lengths, dweight, dscale, dnext_weight};
  if (any_misaligned(acts, esize(s->dtype)) || any_misaligned(words, 4))
    return FALCON_ERR_MISALIGNED;
  const void* inputs[] = {h, z, out, dnext, weight, scale, next_weight};
  if (s->B > 0 && s->T > 0) {
    if (among(dx, inputs) || among(dh, inputs) || among(dz, inputs) || (dh && dh == dout) ||
        (dz && dz == dout) || (dh && (dh == dx || dh == dz)) || (dz && dz == dx))
      return FALCON_ERR_BAD_ARG;
    if (dx && dx == dout && !same(dxs, dos, s->B, s->T)) return FALCON_ERR_BAD_ARG;
    if ((dx && on_itself(dxs, s->B, 1, s->T)) || (dh && on_itself(dhs, s->B, s->H, s->T)) ||
        (dz && on_itself(dzs, s->B, 1, s->T)))
      return FALCON_ERR_BAD_ARG;
  }
  if (among(dweight, inputs) || among(dscale, inputs) || among(dnext_weight, inputs) ||
      (dweight && (dweight == dscale || dweight == dnext_weight)) ||
      (dscale && dscale == dnext_weight))
    return FALCON_ERR_BAD_ARG;
  const size_t need = falcon_gated_norm_bwd_workspace_bytes(s);
  if (need > 0 && (!workspace || workspace_bytes < need)) return FALCON_ERR_WORKSPACE;
  if (!aligned(workspace, 16)) return FALCON_ERR_MISALIGNED;
  rc = falcon::check_sm103_device();
  if (rc) return rc;
  falcon::NormArgs a = norm_args(s);
  a.h = h, a.z = z, a.y = out, a.dout = dout, a.dnext = dnext;
  a.hs = of(hs), a.zs = of(zs), a.os = of(os), a.dos = of(dos), a.dns = of(dns);
  a.weight = weight, a.scale = scale, a.next_weight = next_weight, a.lengths = lengths;
  a.dx = dx, a.dh = dh, a.dz = dz;
  a.dxs = of(dxs), a.dhs = of(dhs), a.dzs = of(dzs);
  a.dweight = dweight, a.dscale = dscale, a.dnext_weight = dnext_weight;
  a.ws = static_cast<float*>(workspace);
  return to_status(falcon::launch_norm_bwd(a, stream));
}

}  // extern "C"
