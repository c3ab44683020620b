// The C ABI of cross attention and of the 8-bit cache (include/sa2.h): argument checks, workspace
// layout, tensor maps and launches.
#include <algorithm>
#include <cmath>

#include "cross_internal.h"

namespace sa2 {

// SMs of the current device (152 where there is none, so that sizes can be asked for on any host).
int sm_count() {
  static std::atomic<int> known[64];
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 152;
  sms = known[dev].load(std::memory_order_relaxed);
  if (sms == 0) {
    if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || sms < 1) return 152;
    known[dev].store(sms, std::memory_order_relaxed);
  }
  return sms;
}

sa2_status cuda_status(cudaError_t e) { return e == cudaSuccess ? SA2_OK : SA2_ERR_CUDA; }

// Checks a token tensor of B x heads x tokens x d elements of which G heads share a key head; strides of
// dimensions of size 1 are replaced by d, so that a tensor map sees legal ones.
sa2_status check_tensor(const sa2_tensor* t, int B, int heads, int G, int tokens, int d, int esz, TokenRef* r) {
  if (!t || !t->data) return SA2_ERR_INVALID_ARG;
  if (!aligned16(t->data)) return SA2_ERR_ALIGNMENT;
  r->p = t->data;
  r->sn = tokens > 1 ? t->stride_n : d;
  r->sh = heads > 1 ? t->stride_h : d;
  r->sb = B > 1 ? t->stride_b : d;
  if (r->sn < d || r->sh < 1 || r->sb < 1) return SA2_ERR_INVALID_ARG;
  if (r->sn * esz % 16 || r->sh * esz % 16 || r->sb * esz % 16) return SA2_ERR_ALIGNMENT;
  // a tensor map's strides are below 2^40 bytes; that of the key heads' groups is one of them
  const int64_t most = ((int64_t)1 << 40) / esz;
  if (r->sn >= most || r->sh >= (heads > G ? most / G : most) || r->sb >= most) return SA2_ERR_UNSUPPORTED;
  return SA2_OK;
}

bool misaligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) != 0; }

}  // namespace sa2

using namespace sa2;

namespace {

constexpr int kMaxGridYZ = 32767;  // B and Hkv are grid dimensions (B twice over)

sa2_status check_cross(const sa2_cross_shape* x, CrossShape* s) {
  if (!x) return SA2_ERR_INVALID_ARG;
  if (x->B < 1 || x->H < 1 || x->Hkv < 1 || x->N < 1 || x->M < 1 || x->reserved != 0) return SA2_ERR_INVALID_ARG;
  if (x->H % x->Hkv) return SA2_ERR_INVALID_ARG;
  if (x->dtype != SA2_BF16 && x->dtype != SA2_FP16) return SA2_ERR_UNSUPPORTED;
  if (x->d != 64 && x->d != 128) return SA2_ERR_UNSUPPORTED;
  if (x->N >= kMaxTokens || x->M >= kMaxTokens || x->B > kMaxGridYZ || x->Hkv > kMaxGridYZ ||
      x->H / x->Hkv > kMaxGroup)
    return SA2_ERR_UNSUPPORTED;
  s->B = x->B;
  s->H = x->H;
  s->Hkv = x->Hkv;
  s->G = x->H / x->Hkv;
  s->N = x->N;
  s->M = x->M;
  s->d = x->d;
  s->dtype = x->dtype;
  wait_settings(&s->wait_ns, &s->stall_ns);
  return SA2_OK;
}

sa2_status check_cache(const sa2_cache8* x, CacheRef* c) {
  if (!x || !x->k || !x->v || !x->k_scale || !x->v_scale) return SA2_ERR_INVALID_ARG;
  if (x->B < 1 || x->Hkv < 1 || x->C < 1) return SA2_ERR_INVALID_ARG;
  if (x->d != 64 && x->d != 128) return SA2_ERR_UNSUPPORTED;
  if (x->C >= kMaxTokens || x->B > kMaxGridYZ || x->Hkv > kMaxGridYZ) return SA2_ERR_UNSUPPORTED;
  const sa2_tensor k{x->k, x->stride_b, x->stride_h, x->stride_n};
  TokenRef r;
  const sa2_status st = check_tensor(&k, x->B, x->Hkv, 1, x->C, x->d, 1, &r);
  if (st != SA2_OK) return st;
  if (!aligned16(x->v) || (reinterpret_cast<uintptr_t>(x->k_scale) & 3u) ||
      (reinterpret_cast<uintptr_t>(x->v_scale) & 3u))
    return SA2_ERR_ALIGNMENT;
  c->k = static_cast<uint8_t*>(x->k);
  c->v = static_cast<uint8_t*>(x->v);
  c->ks = x->k_scale;
  c->vs = x->v_scale;
  c->sb = r.sb;
  c->sh = r.sh;
  c->sn = r.sn;
  c->C = x->C;
  c->nsb = (x->C + 63) / 64;
  return SA2_OK;
}

// What the two forward calls share: q, o, lse, kv_len, the plan and its workspace.
sa2_status fwd_args(const CrossShape& s, const sa2_tensor* q, const int32_t* kv_len, float scale, const sa2_tensor* o,
                    float* lse, void* ws, size_t ws_bytes, FwdPlan* plan, CrossFwdArgs* a) {
  if (!lse || !std::isfinite(scale)) return SA2_ERR_INVALID_ARG;
  sa2_status st = check_tensor(q, s.B, s.H, s.G, s.N, s.d, 2, &a->q);
  if (st == SA2_OK) st = check_tensor(o, s.B, s.H, s.G, s.N, s.d, 2, &a->o);
  if (st != SA2_OK) return st;
  if (misaligned4(lse) || misaligned4(kv_len) || !aligned16(ws)) return SA2_ERR_ALIGNMENT;
  *plan = cross_fwd_plan(s, sm_count());
  if (plan->segs < 0) return SA2_ERR_UNSUPPORTED;
  const size_t floats = cross_fwd_partials(s, *plan);
  if (floats && (!ws || ws_bytes < floats * sizeof(float))) return SA2_ERR_WORKSPACE;
  a->kv_len = kv_len;
  a->lse = lse;
  a->part_o = static_cast<float*>(ws);
  a->part_l = floats ? a->part_o + (size_t)(plan->grid + plan->segs) * plan->rows * s.d : nullptr;
  const float sc = scale > 0.f ? scale : (float)(1.0 / std::sqrt((double)s.d));
  a->scale_log2 = sc * 1.4426950408889634f;
  a->status = status_word();
  return SA2_OK;
}

}  // namespace

extern "C" {

size_t sa2_cross_fwd_workspace_size(const sa2_cross_shape* shape) {
  CrossShape s;
  if (check_cross(shape, &s) != SA2_OK) return 0;
  const FwdPlan p = cross_fwd_plan(s, sm_count());
  return p.segs < 0 ? 0 : cross_fwd_partials(s, p) * sizeof(float);
}

sa2_status sa2_cross_attn_fwd(const sa2_cross_shape* shape, const sa2_tensor* q, const sa2_tensor* k,
                              const sa2_tensor* v, const int32_t* kv_len, float scale, const sa2_tensor* o,
                              float* lse, void* ws, size_t ws_bytes, void* stream) {
  CrossShape s;
  sa2_status st = check_cross(shape, &s);
  if (st != SA2_OK) return st;
  TokenRef kr, vr;
  st = check_tensor(k, s.B, s.Hkv, 1, s.M, s.d, 2, &kr);
  if (st == SA2_OK) st = check_tensor(v, s.B, s.Hkv, 1, s.M, s.d, 2, &vr);
  if (st != SA2_OK) return st;
  FwdPlan plan;
  CrossFwdArgs a;
  st = fwd_args(s, q, kv_len, scale, o, lse, ws, ws_bytes, &plan, &a);
  if (st != SA2_OK) return st;
  if (plan.few)
    return cuda_status(launch_few_rows(s, plan, kr, vr, CacheRef{}, false, a, static_cast<cudaStream_t>(stream)));
  CUtensorMap mq, mk, mv, mo;
  const bool f16 = s.dtype == SA2_FP16;
  if (!make_group_map(&mq, a.q, s.B, s.H, s.G, s.N, s.d, s.G, plan.nb, f16) ||
      !make_group_map(&mo, a.o, s.B, s.H, s.G, s.N, s.d, s.G, plan.nb, f16) ||
      !make_group_map(&mk, kr, s.B, s.Hkv, 1, s.M, s.d, 1, kKeyBlock, f16) ||
      !make_group_map(&mv, vr, s.B, s.Hkv, 1, s.M, s.d, 1, kKeyBlock, f16))
    return SA2_ERR_CUDA;
  return cuda_status(launch_cross_fwd(s, plan, mq, mk, mv, mo, a, static_cast<cudaStream_t>(stream)));
}

size_t sa2_cross_bwd_workspace_size(const sa2_cross_shape* shape) {
  CrossShape s;
  if (check_cross(shape, &s) != SA2_OK || s.dtype != SA2_BF16) return 0;
  size_t stats;
  return cross_bwd_floats(s, cross_bwd_plan(s, sm_count()), &stats) * sizeof(float);
}

sa2_status sa2_cross_attn_bwd(const sa2_cross_shape* shape, const sa2_tensor* q, const sa2_tensor* k,
                              const sa2_tensor* v, const sa2_tensor* o, const float* lse, const sa2_tensor* dO,
                              const int32_t* kv_len, float scale, const sa2_tensor* dq, const sa2_tensor* dk,
                              const sa2_tensor* dv, void* ws, size_t ws_bytes, void* stream) {
  CrossShape s;
  sa2_status st = check_cross(shape, &s);
  if (st != SA2_OK) return st;
  if (s.dtype != SA2_BF16) return SA2_ERR_UNSUPPORTED;
  if (!lse || !std::isfinite(scale)) return SA2_ERR_INVALID_ARG;
  CrossBwdArgs a;
  TokenRef qr, kr, vr;
  st = check_tensor(q, s.B, s.H, s.G, s.N, s.d, 2, &qr);
  if (st == SA2_OK) st = check_tensor(k, s.B, s.Hkv, 1, s.M, s.d, 2, &kr);
  if (st == SA2_OK) st = check_tensor(v, s.B, s.Hkv, 1, s.M, s.d, 2, &vr);
  if (st == SA2_OK) st = check_tensor(o, s.B, s.H, s.G, s.N, s.d, 2, &a.o);
  if (st == SA2_OK) st = check_tensor(dO, s.B, s.H, s.G, s.N, s.d, 2, &a.dO);
  if (st == SA2_OK) st = check_tensor(dq, s.B, s.H, s.G, s.N, s.d, 2, &a.dq);
  if (st == SA2_OK) st = check_tensor(dk, s.B, s.Hkv, 1, s.M, s.d, 2, &a.dk);
  if (st == SA2_OK) st = check_tensor(dv, s.B, s.Hkv, 1, s.M, s.d, 2, &a.dv);
  if (st != SA2_OK) return st;
  if (misaligned4(lse) || misaligned4(kv_len) || !aligned16(ws)) return SA2_ERR_ALIGNMENT;
  const BwdPlan plan = cross_bwd_plan(s, sm_count());
  // (grid dimensions; tensors of so many tiles or key blocks have terabytes)
  if ((int64_t)s.B * s.Hkv * std::max(plan.tiles, plan.kblocks) > INT32_MAX) return SA2_ERR_UNSUPPORTED;
  size_t stats;
  const size_t floats = cross_bwd_floats(s, plan, &stats);
  if (!ws || ws_bytes < floats * sizeof(float)) return SA2_ERR_WORKSPACE;
  CUtensorMap mq, mk, mv, mdo;
  if (!make_group_map(&mq, qr, s.B, s.H, s.G, s.N, s.d, s.G, plan.nb, false) ||
      !make_group_map(&mdo, a.dO, s.B, s.H, s.G, s.N, s.d, s.G, plan.nb, false) ||
      !make_group_map(&mk, kr, s.B, s.Hkv, 1, s.M, s.d, 1, kKeyBlock, false) ||
      !make_group_map(&mv, vr, s.B, s.Hkv, 1, s.M, s.d, 1, kKeyBlock, false))
    return SA2_ERR_CUDA;
  a.kv_len = kv_len;
  a.lse = lse;
  a.stats = static_cast<float*>(ws);
  a.part = a.stats + stats;
  a.scale = scale > 0.f ? scale : (float)(1.0 / std::sqrt((double)s.d));
  a.scale_log2 = a.scale * 1.4426950408889634f;
  a.status = status_word();
  return cuda_status(launch_cross_bwd(s, plan, mq, mk, mv, mdo, a, static_cast<cudaStream_t>(stream)));
}

sa2_status sa2_cache8_append(const sa2_cache8* cache, int32_t n, int32_t dtype, const sa2_tensor* k,
                             const sa2_tensor* v, const int32_t* pos, const int32_t* n_new, void* stream) {
  CacheRef c;
  sa2_status st = check_cache(cache, &c);
  if (st != SA2_OK) return st;
  if (n < 1 || !pos) return SA2_ERR_INVALID_ARG;
  if (n >= kMaxTokens || (dtype != SA2_BF16 && dtype != SA2_FP16)) return SA2_ERR_UNSUPPORTED;
  TokenRef kr, vr;
  st = check_tensor(k, cache->B, cache->Hkv, 1, n, cache->d, 2, &kr);
  if (st == SA2_OK) st = check_tensor(v, cache->B, cache->Hkv, 1, n, cache->d, 2, &vr);
  if (st != SA2_OK) return st;
  if (misaligned4(pos) || misaligned4(n_new)) return SA2_ERR_ALIGNMENT;
  return cuda_status(launch_cache_append(c, cache->B, cache->Hkv, cache->d, n, dtype == SA2_FP16, kr, vr, pos, n_new,
                                         status_word(), static_cast<cudaStream_t>(stream)));
}

sa2_status sa2_cache8_read(const sa2_cache8* cache, int32_t n, int32_t dtype, const sa2_tensor* k,
                           const sa2_tensor* v, const int32_t* pos, void* stream) {
  CacheRef c;
  sa2_status st = check_cache(cache, &c);
  if (st != SA2_OK) return st;
  if (n < 1 || !pos) return SA2_ERR_INVALID_ARG;
  if (n >= kMaxTokens || (dtype != SA2_BF16 && dtype != SA2_FP16)) return SA2_ERR_UNSUPPORTED;
  TokenRef kr, vr;
  st = check_tensor(k, cache->B, cache->Hkv, 1, n, cache->d, 2, &kr);
  if (st == SA2_OK) st = check_tensor(v, cache->B, cache->Hkv, 1, n, cache->d, 2, &vr);
  if (st != SA2_OK) return st;
  if (misaligned4(pos)) return SA2_ERR_ALIGNMENT;
  return cuda_status(launch_cache_read(c, cache->B, cache->Hkv, cache->d, n, dtype == SA2_FP16, kr, vr, pos,
                                       status_word(), static_cast<cudaStream_t>(stream)));
}

sa2_status sa2_cache8_attn(const sa2_cross_shape* shape, const sa2_tensor* q, const sa2_cache8* cache,
                           const int32_t* kv_len, float scale, const sa2_tensor* o, float* lse, void* ws,
                           size_t ws_bytes, void* stream) {
  CrossShape s;
  sa2_status st = check_cross(shape, &s);
  if (st != SA2_OK) return st;
  CacheRef c;
  st = check_cache(cache, &c);
  if (st != SA2_OK) return st;
  if (!kv_len || cache->B != s.B || cache->Hkv != s.Hkv || cache->C != s.M || cache->d != s.d)
    return SA2_ERR_INVALID_ARG;
  FwdPlan plan;
  CrossFwdArgs a;
  st = fwd_args(s, q, kv_len, scale, o, lse, ws, ws_bytes, &plan, &a);
  if (st != SA2_OK) return st;
  if (plan.few)
    return cuda_status(launch_few_rows(s, plan, TokenRef{}, TokenRef{}, c, true, a, static_cast<cudaStream_t>(stream)));
  CUtensorMap mk, mv;
  if (!make_cache_map(&mk, c.k, c, s.B, s.Hkv, s.d, kKeyBlock) || !make_cache_map(&mv, c.v, c, s.B, s.Hkv, s.d, kKeyBlock))
    return SA2_ERR_CUDA;
  return cuda_status(launch_cache_fwd(s, plan, mk, mv, c, a, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
