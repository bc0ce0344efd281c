// eqlin_attn_api.cu -- argument checks and dispatch of the document attention.
#include <math.h>

#include "eqlin_attn.cuh"

using namespace eqlin;

namespace {

bool bad16(const void* p) { return ((uintptr_t)p & 15u) != 0; }
bool bad4(const void* p) { return ((uintptr_t)p & 3u) != 0; }

// Checks common to both directions; fills what they share.
eqlin_status_t describe(const eqlin_attention_t* a, eqlin_dtype_t dtype, attn::Params& p) {
  if (!a || (dtype != EQLIN_F32 && dtype != EQLIN_F16 && dtype != EQLIN_BF16)) return EQLIN_ERR_INVALID_ARG;
  if (a->tokens < 0 || a->docs < 0 || a->max_len < 0 || a->heads < 1 || a->kv_heads < 1 || a->head_dim < 1)
    return EQLIN_ERR_INVALID_ARG;
  if (a->heads % a->kv_heads) return EQLIN_ERR_INVALID_ARG;
  if (!isfinite(a->scale) || !(a->scale > 0.f) || !isfinite(a->cap) || a->cap < 0.f) return EQLIN_ERR_INVALID_ARG;
  if (a->axes < 0 || (a->axes > 0 && !a->slopes)) return EQLIN_ERR_INVALID_ARG;
  if (a->axes > attn::kMaxAxes) return EQLIN_ERR_UNSUPPORTED;
  // what the kernels scale scores by stays a normal FP32 number
  auto far = [](float x) { return x < 0x1p-120f || x > 0x1p120f; };
  if (far(a->scale) || (a->cap > 0.f && (far(a->cap) || far(a->scale / a->cap) || far(a->cap / a->scale))))
    return EQLIN_ERR_UNSUPPORTED;
  if (a->heads > 65536 || a->head_dim > attn::kMaxHeadDim || a->tokens > 0x7fffff00)   // a tile's end fits 32 bits
    return EQLIN_ERR_UNSUPPORTED;
  const int64_t es = dtype == EQLIN_F32 ? 4 : 2;
  if (a->head_dim * es % 16) return EQLIN_ERR_MISALIGNED;
  if (!a->offsets) {
    if (a->tokens > 0 && (a->docs < 1 || a->tokens % a->docs)) return EQLIN_ERR_INVALID_ARG;
  }
  if (a->docs > 0x7fffffff || (a->docs + 1) * a->heads > 0x7fffffff) return EQLIN_ERR_UNSUPPORTED;
  if (bad4(a->offsets) || bad4(a->pos) || bad4(a->slopes) || bad4(a->err)) return EQLIN_ERR_MISALIGNED;
  p = attn::Params{};
  p.N = a->tokens;
  p.H = (int)a->heads;
  p.K = (int)a->kv_heads;
  p.D = (int)a->head_dim;
  p.offsets = a->offsets;
  p.docs = a->docs;
  if (!a->offsets) {
    p.len = a->docs ? a->tokens / a->docs : 0;
  } else {
    // spreads the work; every length is right with any value
    p.len = a->max_len ? a->max_len : (a->docs ? (a->tokens + a->docs - 1) / a->docs : 1);
    if (p.len > a->tokens) p.len = a->tokens;
  }
  p.pos = a->pos;
  p.slopes = a->slopes;
  p.axes = a->axes;
  p.scale = a->scale;
  p.cap = a->cap;
  p.err = a->err;
  p.wait_limit = a->wait_limit == 0 ? kDefaultWaitLimit : a->wait_limit == UINT32_MAX ? 0 : a->wait_limit;
  return EQLIN_OK;
}

// A per-token row stride: wide enough for its heads, a multiple of 16 bytes.
eqlin_status_t stride_ok(int64_t stride, int64_t heads, const attn::Params& p, eqlin_dtype_t dtype) {
  if (stride < heads * p.D) return EQLIN_ERR_INVALID_ARG;
  return stride * (dtype == EQLIN_F32 ? 4 : 2) % 16 ? EQLIN_ERR_MISALIGNED : EQLIN_OK;
}

eqlin_status_t done(cudaError_t e) { return e == cudaSuccess ? EQLIN_OK : EQLIN_ERR_CUDA; }

}  // namespace

extern "C" eqlin_status_t eqlin_attention_forward(const eqlin_attention_t* a, eqlin_dtype_t dtype, const void* q,
                                                  const void* k, const void* v, void* o, float* lse, void* stream) {
  attn::Params p;
  eqlin_status_t st = describe(a, dtype, p);
  if (st != EQLIN_OK) return st;
  if ((st = stride_ok(a->q_stride, p.H, p, dtype)) != EQLIN_OK) return st;
  if ((st = stride_ok(a->k_stride, p.K, p, dtype)) != EQLIN_OK) return st;
  if ((st = stride_ok(a->v_stride, p.K, p, dtype)) != EQLIN_OK) return st;
  if ((st = stride_ok(a->o_stride, p.H, p, dtype)) != EQLIN_OK) return st;
  if (p.N == 0) return EQLIN_OK;
  if (!q || !k || !v || !o || !lse || (p.axes && !p.pos)) return EQLIN_ERR_INVALID_ARG;
  if (bad16(q) || bad16(k) || bad16(v) || bad16(o) || bad4(lse)) return EQLIN_ERR_MISALIGNED;
  p.q = q;
  p.k = k;
  p.v = v;
  p.o = o;
  p.lse = lse;
  p.qs = a->q_stride;
  p.ks = a->k_stride;
  p.vs = a->v_stride;
  p.os = a->o_stride;
  cudaStream_t cs = static_cast<cudaStream_t>(stream);
  return done(dtype == EQLIN_F32 ? launch_attn_simt_forward(p, cs) : launch_attn_tc_forward(p, dtype, cs));
}

extern "C" eqlin_status_t eqlin_attention_backward(const eqlin_attention_t* a, eqlin_dtype_t dtype, const void* go,
                                                   int64_t go_stride, const void* q, const void* k, const void* v,
                                                   const void* o, const float* lse, void* dq, int64_t dq_stride,
                                                   void* dk, int64_t dk_stride, void* dv, int64_t dv_stride,
                                                   float* delta, void* stream) {
  attn::Params p;
  eqlin_status_t st = describe(a, dtype, p);
  if (st != EQLIN_OK) return st;
  const int64_t wide[4] = {a->q_stride, a->o_stride, go_stride, dq_stride};
  const int64_t narrow[4] = {a->k_stride, a->v_stride, dk_stride, dv_stride};
  for (int i = 0; i < 4; ++i) {
    if ((st = stride_ok(wide[i], p.H, p, dtype)) != EQLIN_OK) return st;
    if ((st = stride_ok(narrow[i], p.K, p, dtype)) != EQLIN_OK) return st;
  }
  if (p.N == 0) return EQLIN_OK;
  if (!go || !q || !k || !v || !o || !lse || !dq || !dk || !dv || !delta || (p.axes && !p.pos))
    return EQLIN_ERR_INVALID_ARG;
  if (bad16(go) || bad16(q) || bad16(k) || bad16(v) || bad16(o) || bad16(dq) || bad16(dk) || bad16(dv) ||
      bad4(lse) || bad4(delta))
    return EQLIN_ERR_MISALIGNED;
  p.q = q;
  p.k = k;
  p.v = v;
  p.go = go;
  p.o = const_cast<void*>(o);
  p.lse = const_cast<float*>(lse);
  p.dq = dq;
  p.dk = dk;
  p.dv = dv;
  p.delta = delta;
  p.qs = a->q_stride;
  p.ks = a->k_stride;
  p.vs = a->v_stride;
  p.os = a->o_stride;
  p.gos = go_stride;
  p.dqs = dq_stride;
  p.dks = dk_stride;
  p.dvs = dv_stride;
  cudaStream_t cs = static_cast<cudaStream_t>(stream);
  if (dtype == EQLIN_F32) return done(launch_attn_simt_backward(p, cs));
  const cudaError_t e = launch_attn_tc_dq(p, dtype, cs);
  return done(e != cudaSuccess ? e : launch_attn_tc_dkv(p, dtype, cs));
}
