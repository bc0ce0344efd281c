// eqlin_attn.cuh -- what the attention kernels share: the call's parameters,
// the documents, and the score function.
//
// Tokens lie in one packed sequence [N]; a document is a contiguous range of
// them, and a token attends to the tokens of its document.  With u = scale
// q_i.k_j (natural units throughout, base-2 inside the kernels):
//
//   c = cap tanh(u / cap)   (cap > 0),   c = u   (cap = 0)
//   s = c - slope_h sum_a |pos[i, a] - pos[j, a]|
//   lse_i = log sum_j exp s_ij,   P = exp(s - lse),   o_i = sum_j P_ij v_j
//
//   dv_j = sum_i P_ij do_i,   dP = do.v,   delta_i = do_i.o_i
//   ds = P (dP - delta),      du = ds (1 - tanh^2(u / cap))
//   dq_i = scale sum_j du k_j,   dk_j = scale sum_i du q_i
//
// Rows outside every document get o = 0, lse = 0 and zero gradients.
#pragma once

#include "eqlin_internal.cuh"

namespace eqlin {
namespace attn {

constexpr int kMaxAxes = 3;
constexpr int kMaxHeadDim = 128;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

struct Params {
  const void* q;
  const void* k;
  const void* v;
  const void* go;
  void* o;                // read by the backward
  void* dq;
  void* dk;
  void* dv;
  float* lse;             // [H][N]
  float* delta;           // [H][N]
  int64_t qs, ks, vs, os, gos, dqs, dks, dvs;   // elements per token
  int64_t N;
  const int32_t* offsets; // [docs + 1], or null: documents of `len` tokens
  int64_t docs, len;
  const float* pos;       // [N][axes]
  const float* slopes;    // [H]
  int axes;               // 0: no bias
  int H, K, D;
  int hint;               // f32: blocks per (document, head), each walks the tiles hint apart;
                          // else tiles per document (equal lengths) or 128-token slots (packed)
  uint32_t items;         // work items in all
  float scale, cap;
  int* err;               // error record (eqlin_wait.cuh), or null
  uint32_t wait_limit;
};

// A document's tokens [lo, hi).  Offsets are forced into [0, N] and into
// order, so that wrong ones cannot lead out of the tensors.
__device__ __forceinline__ void doc_range(const Params& p, int64_t doc, int64_t& lo, int64_t& hi) {
  if (!p.offsets) {
    lo = doc * p.len;
    hi = lo + p.len;
    return;
  }
  lo = min(max((int64_t)p.offsets[doc], (int64_t)0), p.N);
  hi = min(max((int64_t)p.offsets[doc + 1], lo), p.N);
}

}  // namespace attn

// f32: CUDA cores.
cudaError_t launch_attn_simt_forward(const attn::Params& p, cudaStream_t st);
cudaError_t launch_attn_simt_backward(const attn::Params& p, cudaStream_t st);

// f16 and bf16: tcgen05.
cudaError_t launch_attn_tc_forward(const attn::Params& p, eqlin_dtype_t dt, cudaStream_t st);
// dq and delta first, then dk and dv, which read delta.
cudaError_t launch_attn_tc_dq(const attn::Params& p, eqlin_dtype_t dt, cudaStream_t st);
cudaError_t launch_attn_tc_dkv(const attn::Params& p, eqlin_dtype_t dt, cudaStream_t st);

}  // namespace eqlin
