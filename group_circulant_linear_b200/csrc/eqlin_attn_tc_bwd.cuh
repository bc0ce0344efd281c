// eqlin_attn_tc_bwd.cuh -- document attention, backward, on the tensor cores.
//
// Two kernels of one template.  KEYS = false owns 128 query rows and passes
// over the keys: dq, and delta = do.o on the way.  KEYS = true owns 128 key
// rows and passes over the queries of every head that shares them: dk, dv.
// Both form the scores again; in exchange no sum crosses blocks, so there are
// no atomics and results are the same in every run.  With own tiles (A0, A1) =
// (Q, dO) or (K, V) and moving tiles (X, Y) = (K, V) or (Q, dO):
//
//   S = A0 X^T,  dP = A1 Y^T          TMEM accumulators
//   P = 2^(s - lse),  du = P (dP - delta) (1 - tanh^2)   FP32 registers
//   dq += du X        or       dv += P Y,  dk += du X     A from TMEM, 16 bits
//
// P and du are rounded to the inputs' type as operands of those products, half
// a step each; sums are FP32 in TMEM.  In f16 P carries a factor 2^8 on its
// way to dv, so that probabilities of long documents (1e-5 and less) stay out
// of the subnormals.
//
// A thread owns one row and 64 columns of a tile (NWG warpgroups of rows, the
// 32-column chunks dealt out in turn).  Where TMEM allows, P and du have
// columns of their own (SEP) and the next tile's scores are issued as soon as
// the present ones are in registers; else they lie over the scores they came
// from, chunk by chunk, and the SM's other block fills the gap.
#pragma once

#include "eqlin_attn_tc.cuh"

namespace eqlin {
namespace attn_tc {

template <int DP, bool KEYS> struct BwdCfg {
  // up to 64 features: 64-row moving tiles in 256 TMEM columns, two blocks per
  // SM; above, 128-row tiles, 512 columns, one block with two warpgroups
  static constexpr int CW = DP > 64 ? 128 : 64;
  static constexpr int NWG = CW / 64;
  static constexpr int BLOCKS = DP > 64 ? 1 : 2;
  static constexpr int THREADS = NWG * 128 + 64;
  static constexpr int TMEM = DP > 64 ? 512 : 256;
  static constexpr bool SEP = !KEYS;
  static constexpr int S_COL = 0, DP_COL = CW, ACC0 = 2 * CW;   // dq, or dv
  static constexpr int ACC1 = ACC0 + DP;                        // KEYS: dk;  else: du's columns
  static constexpr int OWN = DP / 64 * PANEL;                   // bytes of one own tile
  static constexpr int MOV_PANEL = CW * 128;
  static constexpr int MOV = DP / 64 * MOV_PANEL;               // bytes of one moving tile
  static constexpr int SLOTS = DP > 64 ? 2 : 4;
  static constexpr int SIDE = (kMaxAxes * ROWS + (KEYS ? 2 * ROWS : 0)) * 4;   // positions, lse, delta of a slot
  static constexpr int NBAR = 2 + 2 * SLOTS + 5;
  static constexpr int SMEM = 2 * OWN + SLOTS * (2 * MOV + SIDE) + NBAR * 8 + 64 + 1024;
  static_assert(ACC1 + (KEYS ? DP : CW / 2) <= TMEM, "TMEM columns");
  static_assert(BLOCKS * SMEM <= 227 * 1024, "shared memory");
};

template <int DP, typename E, int AXES, bool CAP, bool KEYS>
__global__ void __launch_bounds__(BwdCfg<DP, KEYS>::THREADS, BwdCfg<DP, KEYS>::BLOCKS)
attn_tc_bwd_kernel(const __grid_constant__ Params p) {
  using C = BwdCfg<DP, KEYS>;
  constexpr int CW = C::CW, NWG = C::NWG;
  constexpr uint32_t KID = KEYS ? K_ATTN_DKV : K_ATTN_DQ;
  constexpr bool F16 = Pair<E>::fmt == 0;
  constexpr float kUp = F16 ? 8.f : 0.f;             // P's factor, as an exponent
  constexpr float kDown = F16 ? 1.f / 256.f : 1.f;
  constexpr int MMA = NWG * 4, LOAD = NWG * 4 + 1;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  uint8_t* ring = smem + 2 * C::OWN;
  float* side = reinterpret_cast<float*>(ring + C::SLOTS * 2 * C::MOV);
  constexpr int SIDE_F = C::SIDE / 4;
  uint64_t* bars = reinterpret_cast<uint64_t*>(side + C::SLOTS * SIDE_F);
  uint64_t* own_full = bars;
  uint64_t* own_empty = bars + 1;
  uint64_t* full = bars + 2;
  uint64_t* empty = full + C::SLOTS;
  uint64_t* s_full = empty + C::SLOTS;
  uint64_t* s_free = s_full + 1;
  uint64_t* p_full = s_free + 1;
  uint64_t* acc_full = p_full + 1;
  uint64_t* drain = acc_full + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + C::NBAR);
  int* abort_word = reinterpret_cast<int*>(tmem_slot + 1);
  int* local_err = abort_word + 1;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  grid_dep_wait();
  const int rep = p.H / p.K;
  const Work w = work_of(p, KEYS ? p.K : p.H);
  const int64_t kh = (int64_t)(KEYS ? w.head : w.head / rep) * p.D;
  const int64_t qh0 = (int64_t)(KEYS ? w.head * rep : w.head) * p.D;
  if (w.doc == p.docs) {
    outside_rows(p, w.tile, [&](int64_t r) {
      for (int d = threadIdx.x; d < p.D; d += C::THREADS) {
        if (KEYS) {
          static_cast<E*>(p.dk)[r * p.dks + kh + d] = Elem<E>::from_f(0.f);
          static_cast<E*>(p.dv)[r * p.dvs + kh + d] = Elem<E>::from_f(0.f);
        } else {
          static_cast<E*>(p.dq)[r * p.dqs + qh0 + d] = Elem<E>::from_f(0.f);
        }
      }
    });
    return;
  }
  int64_t lo, hi;
  doc_range(p, w.doc, lo, hi);
  if (lo + (int64_t)w.tile * ROWS >= hi) return;

  if (threadIdx.x == 0) {
    mbar_init(own_full, 32);
    mbar_init(own_empty, 1);
    for (int i = 0; i < C::SLOTS; ++i) {
      mbar_init(full + i, 32);
      mbar_init(empty + i, 1);
    }
    mbar_init(s_full, 1);
    mbar_init(s_free, NWG * 128);
    mbar_init(p_full, NWG * 128);
    mbar_init(acc_full, 1);
    mbar_init(drain, 1);
    *abort_word = 0;
    for (int i = 0; i < 4; ++i) local_err[i] = 0;
    fence_barrier_init();
  }
  if (warp == MMA) {
    tmem_alloc(tmem_slot, C::TMEM);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  grid_dep_launch();                                 // after the allocation, as in the forward
  volatile int* abort_flag = abort_word;
  int* err = p.err ? p.err : local_err;
  const uint32_t limit = p.wait_limit;
  const int d16 = (p.D + 15) / 16;
  const int64_t first = lo + (int64_t)w.tile * ROWS, stride = (int64_t)p.hint * ROWS;
  const int passes = KEYS ? rep : 1;                 // query heads that pass by
  auto width = [&](int64_t c0) { return (int)(hi - c0 < CW ? hi - c0 : CW); };

  if (warp == LOAD) {
    Pending pend;
    uint32_t item = 0, tile_no = 0;
    bool ok = true;
    for (int64_t r0 = first; ok && r0 < hi; r0 += stride, ++tile_no) {
      ok = claim(pend, own_empty, (tile_no & 1) ^ 1, limit, abort_flag, lane, err, site(KID, 2, 0), tile_no);
      if (!ok) break;
      load_rows<DP, E>(smem_u32(smem), KEYS ? p.k : p.q, KEYS ? p.ks : p.qs, KEYS ? kh : qh0, r0, hi, ROWS, p.D, 2 * d16,
                       lane);
      load_rows<DP, E>(smem_u32(smem + C::OWN), KEYS ? p.v : p.go, KEYS ? p.vs : p.gos, KEYS ? kh : qh0, r0, hi, ROWS,
                       p.D, 2 * d16, lane);
      cp_async_commit();
      announce_later(pend, own_full);
      for (int g = 0; ok && g < passes; ++g) {
        const int64_t qh = qh0 + (int64_t)g * p.D;
        for (int64_t c0 = lo; c0 < hi; c0 += CW, ++item) {
          const int nc = width(c0), rows = (nc + 15) & ~15, slot = item % C::SLOTS;
          ok = claim(pend, empty + slot, ((item / C::SLOTS) & 1) ^ 1, limit, abort_flag, lane, err, site(KID, 2, 1), item);
          if (!ok) break;
          const uint32_t to = smem_u32(ring + slot * 2 * C::MOV);
          load_rows<DP, E, CW>(to, KEYS ? p.q : p.k, KEYS ? p.qs : p.ks, KEYS ? qh : kh, c0, hi, rows, p.D, 2 * d16, lane);
          load_rows<DP, E, CW>(to + C::MOV, KEYS ? p.go : p.v, KEYS ? p.gos : p.vs, KEYS ? qh : kh, c0, hi, rows, p.D,
                               2 * d16, lane);
          float* sd = side + slot * SIDE_F;
          const int rows32 = (nc + 31) & ~31;
          if (AXES) load_positions(sd, p, c0, hi, rows32, lane);
          if (KEYS) {
            const int64_t at = (int64_t)(w.head * rep + g) * p.N + c0;
            for (int r = lane; r < rows32; r += 32) {
              sd[kMaxAxes * ROWS + r] = r < nc ? fmaf(p.lse[at + r], kLog2e, -kUp) : 0.f;
              sd[kMaxAxes * ROWS + ROWS + r] = r < nc ? p.delta[at + r] * kDown : 0.f;
            }
          }
          cp_async_commit();
          announce_later(pend, full + slot);
        }
      }
    }
    announce_all(pend);
    if (!ok && lane == 0) raise_abort(abort_flag, err);
  } else if (warp == MMA) {
    if (lane == 0) {
      uint32_t item = 0, tile_no = 0;
      bool ok = true;
      const uint32_t a0 = smem_u32(smem), a1 = smem_u32(smem + C::OWN);
      const uint32_t id_acc = idesc_f16(Pair<E>::fmt, (uint32_t)(16 * d16)) | kBTransposed;
      auto p_col = [](uint32_t base, int s) { return base + 32 * (s >> 1) + 8 * (s & 1); };   // over the scores' chunks
      auto scores = [&](uint32_t it, int64_t c0) -> bool {
        const int slot = it % C::SLOTS;
        if (!bwait(full + slot, (it / C::SLOTS) & 1, limit, abort_flag, err, site(KID, 1, 1), it)) return false;
        if (C::SEP && !bwait(s_free, (it & 1) ^ 1, limit, abort_flag, err, site(KID, 1, 2), it)) return false;
        tc_fence_after();
        const uint32_t id = idesc_f16(Pair<E>::fmt, (uint32_t)((width(c0) + 15) & ~15));
        const uint32_t x = smem_u32(ring + slot * 2 * C::MOV);
        for (int d = 0; d < d16; ++d) {
          const uint32_t oa = (d >> 2) * PANEL + (d & 3) * 32, ob = (d >> 2) * C::MOV_PANEL + (d & 3) * 32;
          mma_f16_ss(tmem + C::S_COL, smem_desc(a0 + oa, 128), smem_desc(x + ob, 128), id, d > 0);
        }
        for (int d = 0; d < d16; ++d) {
          const uint32_t oa = (d >> 2) * PANEL + (d & 3) * 32, ob = (d >> 2) * C::MOV_PANEL + (d & 3) * 32;
          mma_f16_ss(tmem + C::DP_COL, smem_desc(a1 + oa, 128), smem_desc(x + C::MOV + ob, 128), id, d > 0);
        }
        mma_commit(s_full);
        return true;
      };
      for (int64_t r0 = first; ok && r0 < hi; r0 += stride, ++tile_no) {
        ok = bwait(own_full, tile_no & 1, limit, abort_flag, err, site(KID, 1, 0), tile_no) && scores(item, lo);
        bool fresh = true;                           // accumulators start from zero
        for (int g = 0; ok && g < passes; ++g) {
          for (int64_t c0 = lo; ok && c0 < hi; c0 += CW, ++item) {
            const bool more = c0 + CW < hi || g + 1 < passes;
            const int64_t next = c0 + CW < hi ? c0 + CW : lo;
            if (C::SEP && more) ok = scores(item + 1, next);
            ok = ok && bwait(p_full, item & 1, limit, abort_flag, err, site(KID, 1, 3), item);
            if (!ok) break;
            tc_fence_after();
            const int steps = (width(c0) + 15) / 16, slot = item % C::SLOTS;
            const uint32_t x = smem_u32(ring + slot * 2 * C::MOV), y = x + C::MOV;
            if (KEYS) {
              for (int s = 0; s < steps; ++s)
                mma_f16_ts(tmem + C::ACC0, p_col(tmem + C::S_COL, s), smem_desc_mn(y + s * 2048, C::MOV_PANEL, 1024),
                           id_acc, !fresh || s > 0);
              for (int s = 0; s < steps; ++s)
                mma_f16_ts(tmem + C::ACC1, p_col(tmem + C::DP_COL, s), smem_desc_mn(x + s * 2048, C::MOV_PANEL, 1024),
                           id_acc, !fresh || s > 0);
            } else {
              for (int s = 0; s < steps; ++s)
                mma_f16_ts(tmem + C::ACC0, tmem + C::ACC1 + s * 8, smem_desc_mn(x + s * 2048, C::MOV_PANEL, 1024), id_acc,
                           !fresh || s > 0);
            }
            fresh = false;
            mma_commit(acc_full);
            mma_commit(empty + slot);
            if (!more) mma_commit(own_empty);
            if (!C::SEP && more) ok = scores(item + 1, next);
          }
        }
      }
      if (!ok) raise_abort(abort_flag, err);
      mma_commit(drain);
      mbar_wait(drain, 0, kDefaultWaitLimit);
    }
    __syncwarp();
  } else {
    const int wg = warp >> 2, quarter = warp & 3;
    const uint32_t my = tmem + ((uint32_t)(quarter * 32) << 16);
    uint32_t item = 0;
    bool ok = true;
    for (int64_t r0 = first; ok && r0 < hi; r0 += stride) {
      const int64_t row = r0 + quarter * 32 + lane;
      const bool any = r0 + quarter * 32 < hi, live = row < hi;
      float own[AXES ? AXES : 1];
#pragma unroll
      for (int a = 0; a < AXES; ++a) own[a] = live ? p.pos[row * AXES + a] : 0.f;
      float lse2 = 0.f, delta = 0.f;                 // of the own row (queries own)
      if (!KEYS && live) {
        const uint4* a = reinterpret_cast<const uint4*>(static_cast<const E*>(p.go) + row * p.gos + qh0);
        const uint4* b = reinterpret_cast<const uint4*>(static_cast<const E*>(p.o) + row * p.os + qh0);
        for (int c = 0; c < p.D / 8; ++c) {
          const uint4 u = a[c], v = b[c];
          const E* x = reinterpret_cast<const E*>(&u);
          const E* y = reinterpret_cast<const E*>(&v);
#pragma unroll
          for (int k = 0; k < 8; ++k) delta = fmaf(Elem<E>::to_f(x[k]), Elem<E>::to_f(y[k]), delta);
        }
        lse2 = p.lse[(int64_t)w.head * p.N + row] * kLog2e;
        if (wg == 0) p.delta[(int64_t)w.head * p.N + row] = delta;
      }
      for (int g = 0; ok && g < passes; ++g) {
        const Score sc = score_of(p, KEYS ? w.head * rep + g : w.head);
        for (int64_t c0 = lo; c0 < hi; c0 += CW, ++item) {
          const int nc = width(c0), slot = item % C::SLOTS;
          ok = wwait(s_full, item & 1, limit, abort_flag, lane, err, site(KID, 0, 0), item);
          if ((AXES || KEYS) && ok)
            ok = wwait_all(full + slot, (item / C::SLOTS) & 1, limit, abort_flag, err, site(KID, 0, 1), item);
          if (!ok) break;
          tc_fence_after();
          // this warpgroup's chunks: wg, wg + NWG
          uint32_t rs[2][32], rd[2][32];
          if (any) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const int c = wg + i * NWG;
              if (c * 32 < nc) {
                tmem_ld32(my + C::S_COL + c * 32, rs[i]);
                tmem_ld32(my + C::DP_COL + c * 32, rd[i]);
              }
            }
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              tie32(rs[i]);
              tie32(rd[i]);
            }
          }
          if (C::SEP) {
            tc_fence_before();
            mbar_arrive(s_free);
            if (item > 0) {                          // du's columns are free once the last product is done
              ok = wwait(acc_full, (item - 1) & 1, limit, abort_flag, lane, err, site(KID, 0, 2), item);
              if (!ok) break;
              tc_fence_after();
            }
          }
          if (any) {
            const float* sd = side + slot * SIDE_F;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const int c = wg + i * NWG;
              if (c * 32 >= nc) continue;
              const bool edge = c * 32 + 32 > nc;
              uint32_t pp[16], pd[16];
#pragma unroll
              for (int j = 0; j < 32; j += 4) {
                float dist[4] = {0.f, 0.f, 0.f, 0.f}, ls[4], dl[4], pr[4], du[4];
                if (AXES) distances<AXES>(sd, c * 32 + j, own, dist);
                if (KEYS) {
                  *reinterpret_cast<float4*>(ls) = *reinterpret_cast<const float4*>(sd + kMaxAxes * ROWS + c * 32 + j);
                  *reinterpret_cast<float4*>(dl) =
                      *reinterpret_cast<const float4*>(sd + kMaxAxes * ROWS + ROWS + c * 32 + j);
                }
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                  const float raw = __uint_as_float(rs[i][j + k]), dp = __uint_as_float(rd[i][j + k]);
                  const float off = KEYS ? ls[k] : lse2;
                  float t = 0.f, x;
                  if (CAP) {
                    t = tanh_raw(raw, sc);
                    x = fmaf(sc.cap2, t, -off);
                  } else {
                    x = fmaf(raw, sc.scale2, -off);
                  }
                  if (AXES) x = fmaf(-sc.slope2, dist[k], x);
                  pr[k] = ex2(x);
                  // KEYS: pr carries 2^kUp, delta and dP its inverse
                  const float diff = KEYS ? (F16 ? fmaf(dp, kDown, -dl[k]) : dp - dl[k]) : dp - delta;
                  du[k] = pr[k] * diff;
                  if (CAP) du[k] *= fmaf(-t, t, 1.f);
                  if (edge && c * 32 + j + k >= nc) pr[k] = du[k] = 0.f;
                }
                if (KEYS) {
                  pp[j / 2] = Pair<E>::pack(pr[0], pr[1]);
                  pp[j / 2 + 1] = Pair<E>::pack(pr[2], pr[3]);
                }
                pd[j / 2] = Pair<E>::pack(du[0], du[1]);
                pd[j / 2 + 1] = Pair<E>::pack(du[2], du[3]);
              }
              if (KEYS) {
                tmem_st_32x32b_x16(my + C::S_COL + c * 32, pp);
                tmem_st_32x32b_x16(my + C::DP_COL + c * 32, pd);
              } else {
                tmem_st_32x32b_x16(my + C::ACC1 + c * 16, pd);
              }
            }
            tmem_wait_st();
          }
          tc_fence_before();
          mbar_arrive(p_full);
        }
      }
      if (!ok) break;
      ok = wwait(acc_full, (item - 1) & 1, limit, abort_flag, lane, err, site(KID, 0, 3), item);
      if (!ok) break;
      tc_fence_after();
      if (any) {
#pragma unroll
        for (int which = 0; which < (KEYS ? 2 : 1); ++which) {
          const float mul = KEYS && which == 0 ? kDown : p.scale;
          E* out = KEYS ? (which == 0 ? static_cast<E*>(p.dv) + row * p.dvs + kh : static_cast<E*>(p.dk) + row * p.dks + kh)
                        : static_cast<E*>(p.dq) + row * p.dqs + qh0;
#pragma unroll
          for (int c = 0; c < DP / 16; ++c) {
            if (c >= d16 || c % NWG != wg) continue;
            uint32_t o[16], pk[8];
            tmem_ld_32x32b_x16(my + (which ? C::ACC1 : C::ACC0) + c * 16, o);
            tmem_wait_ld();
            tie16(o);
#pragma unroll
            for (int i = 0; i < 16; i += 2)
              pk[i / 2] = Pair<E>::pack(__uint_as_float(o[i]) * mul, __uint_as_float(o[i + 1]) * mul);
            if (live) {
              *reinterpret_cast<uint4*>(out + c * 16) = make_uint4(pk[0], pk[1], pk[2], pk[3]);
              if (c * 16 + 8 < p.D) *reinterpret_cast<uint4*>(out + c * 16 + 8) = make_uint4(pk[4], pk[5], pk[6], pk[7]);
            }
          }
        }
      }
      tc_fence_before();
    }
    if (!ok && lane == 0) raise_abort(abort_flag, err);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == MMA) tmem_dealloc(tmem, C::TMEM);
}

template <int DP, typename E, bool CAP, bool KEYS>
cudaError_t backward_axes(const Params& p, cudaStream_t st) {
  using C = BwdCfg<DP, KEYS>;
  const int heads = KEYS ? p.K : p.H;
  switch (p.axes) {
    case 0: return launch_rows(attn_tc_bwd_kernel<DP, E, 0, CAP, KEYS>, C::SMEM, p, heads, st, C::THREADS);
    case 1: return launch_rows(attn_tc_bwd_kernel<DP, E, 1, CAP, KEYS>, C::SMEM, p, heads, st, C::THREADS);
    case 2: return launch_rows(attn_tc_bwd_kernel<DP, E, 2, CAP, KEYS>, C::SMEM, p, heads, st, C::THREADS);
    default: return launch_rows(attn_tc_bwd_kernel<DP, E, 3, CAP, KEYS>, C::SMEM, p, heads, st, C::THREADS);
  }
}
template <int DP, typename E, bool KEYS>
cudaError_t backward_cap(const Params& p, cudaStream_t st) {
  return p.cap > 0.f ? backward_axes<DP, E, true, KEYS>(p, st) : backward_axes<DP, E, false, KEYS>(p, st);
}
template <bool KEYS>
cudaError_t backward_pick(const Params& p, eqlin_dtype_t dt, cudaStream_t st) {
  if (dt == EQLIN_F16)
    return p.D <= 64 ? backward_cap<64, __half, KEYS>(p, st) : backward_cap<128, __half, KEYS>(p, st);
  return p.D <= 64 ? backward_cap<64, __nv_bfloat16, KEYS>(p, st) : backward_cap<128, __nv_bfloat16, KEYS>(p, st);
}

}  // namespace attn_tc
}  // namespace eqlin
