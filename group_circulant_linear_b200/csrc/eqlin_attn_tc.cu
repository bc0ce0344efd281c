// eqlin_attn_tc.cu -- document attention, forward, on the tensor cores.
//
// Per own tile of 128 queries, one pass over the document's keys in tiles of
// up to CW (trimmed to 16): S = Q K^T into TMEM, a thread per row reads its
// scores, keeps the running maximum m and sum l in FP32, and writes
// P = 2^(s - m) back as 16-bit pairs, which the tensor core takes from TMEM
// for O += P V.  P's rounding to 16 bits is the operand type's own (half a
// step of the inputs'); l sums the unrounded values.
//
// The output is rescaled only when a row's maximum grows by more than 2^8
// (kLag): until then P is at most 256, far inside both types, and O and l
// share the older m, so the quotient is the same.  (A refinement, published
// since, of the online softmax of Milakov and Gimelshein, 2018.)  In f16 P and l
// carry 2^7 more: P is then at most 2^15, and what f16's smallest step loses of a
// small P is 2^-32 of the row's largest, so that a hundred thousand keys which
// share little of a row still count.
//
// Bound by the exponentials (128 x 128 of them take the four schedulers' MUFU
// pipes 1024 cycles, the products 512) and by latency: TMEM and the registers
// of a row per thread leave room for two blocks per SM.  Two forms:
//   CW = 64    S, then P in its place, then the next S.
//   CW = 128   P has columns of its own and the next S is issued while P is
//              formed; half the hand-overs, but its 128 scores per thread only
//              stay in registers in whole tiles away from the cap and, without a
//              cap and a bias, in a document's last tile.
// CW = 128 is taken for heads of up to 64 features (its columns need them) in
// documents that are long on average: from 384 tokens, with a cap or a bias from
// 768.  CW 128 against 64, heads of 64, us, inputs cold: 12544 tokens, 6 heads 373 :
// 539 (two-axis bias 542 : 701, capped 634 : 758); 30 x 900 tokens, 6 heads 100 :
// 118 (capped and biased 206 : 197); 30 x 500, 12 heads 70 : 74 (150 : 120); 30 x
// 384, 12 heads 44 : 48 (77 : 79); 30 x 300, 12 heads 45 : 41; 64 x 197, 12 heads
// 49 : 47 (105 : 74).
#include <float.h>

#include "eqlin_attn_tc.cuh"

namespace eqlin {
namespace attn_tc {

constexpr float kLag = 8.f;
template <typename E> constexpr float kLift = Pair<E>::fmt == 0 ? 7.f : 0.f;

template <int DP, int CW_> struct FwdCfg {
  static constexpr int CW = CW_;                              // keys of a tile
  static constexpr bool SEP = CW == 128;                      // P has its own columns
  static constexpr int OWN = DP / 64 * PANEL;
  static constexpr int MOV_PANEL = CW * 128;
  static constexpr int MOV = DP / 64 * MOV_PANEL;
  static constexpr int SLOTS = MOV > 8192 ? 4 : 6;            // K and V tiles in turn
  static constexpr int NBAR = 2 + 3 * SLOTS + 5;
  static constexpr int P_COL = SEP ? CW : 0, O_COL = SEP ? CW + CW / 2 : CW;
  static constexpr int TMEM = O_COL + DP <= 128 ? 128 : 256;
  static constexpr int POS = (SLOTS / 2) * kMaxAxes * CW * 4;
  static constexpr int SMEM = OWN + SLOTS * MOV + POS + 4 * STAGE + NBAR * 8 + 32 + kListInts * 4 + 1024;
  static_assert(O_COL + DP <= TMEM, "TMEM columns");
  static_assert(2 * (SMEM + 1024) <= 228 * 1024, "shared memory");
};
constexpr int kWideFrom = 384, kWideFromBiased = 768;         // average tokens of a document

template <int DP, int CW, typename E, int AXES, bool CAP>
__global__ void __launch_bounds__(kThreads, 2) attn_tc_fwd_kernel(const __grid_constant__ Params p,
                                                                 const __grid_constant__ Maps maps) {
  using C = FwdCfg<DP, CW>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  uint8_t* ring = smem + C::OWN;
  float* spos = reinterpret_cast<float*>(ring + C::SLOTS * C::MOV);
  uint8_t* stage = reinterpret_cast<uint8_t*>(spos) + C::POS;
  uint64_t* bars = reinterpret_cast<uint64_t*>(stage + 4 * STAGE);
  uint64_t* q_full = bars;
  uint64_t* q_empty = bars + 1;
  uint64_t* kv_full = bars + 2;
  uint64_t* kv_empty = kv_full + C::SLOTS;
  uint64_t* land = kv_empty + C::SLOTS;
  uint64_t* s_full = land + C::SLOTS;
  uint64_t* s_free = s_full + 1;
  uint64_t* p_full = s_free + 1;
  uint64_t* o_full = p_full + 1;
  uint64_t* drain = o_full + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + C::NBAR);
  int* abort_word = reinterpret_cast<int*>(tmem_slot + 1);
  int* local_err = abort_word + 1;
  int* list = local_err + 4;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  grid_dep_wait();
  const uint32_t count = begin(p, p.H, list, [&](int head, int64_t r) {
        for (int d = threadIdx.x; d < p.D; d += kThreads)
          static_cast<E*>(p.o)[r * p.os + (int64_t)head * p.D + d] = Elem<E>::from_f(0.f);
        if (threadIdx.x == 0) p.lse[(int64_t)head * p.N + r] = 0.f;
      });
  if (count == 0) return;
  const int rep = p.H / p.K;

  if (threadIdx.x == 0) {
    mbar_init(q_full, 32);
    mbar_init(q_empty, 1);
    for (int i = 0; i < C::SLOTS; ++i) {
      mbar_init(kv_full + i, 32);
      mbar_init(kv_empty + i, 1);
      mbar_init(land + i, 1);
    }
    mbar_init(s_full, 1);
    mbar_init(s_free, 128);
    mbar_init(p_full, 128);
    mbar_init(o_full, 1);
    mbar_init(drain, 1);
    *abort_word = 0;
    for (int i = 0; i < 4; ++i) local_err[i] = 0;
    fence_barrier_init();
  }
  if (warp == MMA_WARP) {
    tmem_alloc(tmem_slot, C::TMEM);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = uniform(*tmem_slot);
  // after the allocation: a dependent kernel's block that takes TMEM columns
  // early must not be able to starve one of these
  grid_dep_launch();
  volatile int* abort_flag = abort_word;
  int* err = p.err ? p.err : local_err;
  const uint32_t limit = p.wait_limit;
  const int d16 = (p.D + 15) / 16;                            // 16-feature steps

  if (warp == LOAD_WARP) {
    const Waits wait{limit, abort_flag, err};
    Tails tails;
    Side<AXES, false, CW> sidev;
    uint32_t item = 0, owns = 0;
    bool ok = true;
    for (uint32_t i = 0; ok && i < count; ++i) {
      const Tile w = tile_at(p, p.H, list, i);
      const int lo = w.lo, hi = w.hi, kv_head = w.head / rep, key_tiles = (hi - lo - 1) / CW + 1;
      if (AXES) sidev.fetch(p, w.head, lo, hi, lane);
      ok = claim<DP, CW, 1>(tails, q_empty, (owns & 1) ^ 1, ring, land, kv_full, wait, site(K_ATTN_FWD, 2, 0), owns, lane);
      if (!ok) break;
      if (lane == 0) {
        expect_bytes(q_full, C::OWN);
        tma_rows<DP, ROWS>(smem, &maps.m[0], w.head, w.first, q_full);
      }
      mbar_arrive(q_full);
      ++owns;
      for (int j = 0; ok && j < key_tiles; ++j) {
        const int c0 = lo + j * CW, nc = min(hi - c0, CW);
#pragma unroll 1
        for (int kv = 0; ok && kv < 2; ++kv) {
          const uint32_t slot = item % C::SLOTS;
          ok = claim<DP, CW, 1>(tails, kv_empty + slot, ((item / C::SLOTS) & 1) ^ 1, ring, land, kv_full, wait,
                                  site(K_ATTN_FWD, 2, 1), item, lane);
          if (!ok) break;
          // positions go with V: its slot is free once the softmax has used them
          if (AXES && kv) {
            sidev.store(spos + (slot >> 1) * kMaxAxes * CW, 0.f, lane);
            if (j + 1 < key_tiles) sidev.fetch(p, w.head, c0 + CW, hi, lane);
          }
          ok = bring<DP, CW, 1>(tails, slot, ring, land, kv_full, &maps.m[1 + kv], kv_head, c0, nc, wait,
                                  site(K_ATTN_FWD, 2, 2), lane);
          ++item;
        }
      }
    }
    if (ok) ok = settle<DP, CW, 1>(tails, tails.count, ring, land, kv_full, wait, site(K_ATTN_FWD, 2, 2), lane);
    if (!ok && lane == 0) raise_abort(abort_flag, err);
    drain_loads(tails, land, q_full, owns, kv_full, item, C::SLOTS);
  } else if (warp == MMA_WARP) {
    const uint32_t leader = lane == 0;
    uint32_t item = 0, step = 0, owns = 0;                    // step: key tiles since the start
    bool ok = true;
    int lo = 0, hi = 0;
    const uint64_t q_desc = smem_desc(smem_u32(smem), 128);
    const uint32_t q_lo = lo32(q_desc), k_hi = hi32(q_desc), v_hi = hi32(smem_desc_mn(0, C::MOV_PANEL, 1024));
    const uint32_t ring_k = lo32(smem_desc(smem_u32(ring), 128)), ring_v = lo32(smem_desc_mn(smem_u32(ring), C::MOV_PANEL, 1024));
    const uint32_t id_o = idesc_f16(Pair<E>::fmt, (uint32_t)(16 * d16)) | kBTransposed;
    // scores of key tile j, step n, whose K is item `it`
    auto qk = [&](int j, uint32_t it, uint32_t n) -> bool {
      const int slot = it % C::SLOTS;
      if (!wwait_all(kv_full + slot, (it / C::SLOTS) & 1, limit, abort_flag, err, site(K_ATTN_FWD, 1, 1), it)) return false;
      // S is free once every thread has read the previous scores (P over S: once PV, in order, is issued)
      if (C::SEP && !wwait_all(s_free, (n & 1) ^ 1, limit, abort_flag, err, site(K_ATTN_FWD, 1, 2), n)) return false;
      tc_fence_after();
      const uint32_t id = idesc_f16(Pair<E>::fmt, (uint32_t)((min(hi - lo - j * CW, CW) + 15) & ~15));
      const uint32_t k_lo = ring_k + slot * (C::MOV >> 4);
#pragma unroll
      for (int d = 0; d < DP / 16; ++d)
        if (d < d16)
          mma_ss(leader, tmem, q_lo + (((d >> 2) * PANEL + (d & 3) * 32) >> 4),
                 k_lo + (((d >> 2) * C::MOV_PANEL + (d & 3) * 32) >> 4), k_hi, id, d > 0);
      commit(leader, s_full);
      commit(leader, kv_empty + slot);
      return true;
    };
    for (; ok && owns < count; ++owns) {
      const Tile w = tile_at(p, p.H, list, owns);
      lo = w.lo;
      hi = w.hi;
      const int key_tiles = (hi - lo - 1) / CW + 1;
      ok = wwait_all(q_full, owns & 1, limit, abort_flag, err, site(K_ATTN_FWD, 1, 0), owns) && qk(0, item, step);
      for (int j = 0; ok && j < key_tiles; ++j, item += 2, ++step) {
        const bool more = j + 1 < key_tiles;
        if (C::SEP && more) ok = qk(j + 1, item + 2, step + 1);
        if (!more) commit(leader, q_empty);                 // every product with this Q is issued
        const uint32_t vi = item + 1;
        const int slot = vi % C::SLOTS;
        ok = ok && wwait_all(kv_full + slot, (vi / C::SLOTS) & 1, limit, abort_flag, err, site(K_ATTN_FWD, 1, 1), vi) &&
             wwait_all(p_full, step & 1, limit, abort_flag, err, site(K_ATTN_FWD, 1, 3), step);
        if (!ok) break;
        tc_fence_after();
        const int steps = (min(hi - lo - j * CW, CW) + 15) / 16;
        const uint32_t v_lo = ring_v + slot * (C::MOV >> 4);
#pragma unroll
        for (int s = 0; s < CW / 16; ++s)
          if (s < steps)
            mma_ts(leader, tmem + C::O_COL, tmem + (C::SEP ? C::P_COL + 8 * s : 32 * (s >> 1) + 8 * (s & 1)), v_lo + s * (2048 >> 4), v_hi, id_o,
                   j > 0 || s > 0);
        commit(leader, o_full);
        commit(leader, kv_empty + slot);
        if (!C::SEP && more) ok = qk(j + 1, item + 2, step + 1);   // in order behind the product that reads P
      }
    }
    if (!ok && lane == 0) raise_abort(abort_flag, err);
    commit(leader, drain);
    mbar_wait(drain, 0, kDefaultWaitLimit);
    __syncwarp();
  } else {
    const uint32_t my = tmem + ((uint32_t)(warp * 32) << 16);
    uint32_t step = 0;
    bool ok = true;
    for (uint32_t i = 0; ok && i < count; ++i) {
      const Tile w = tile_at(p, p.H, list, i);
      const int lo = w.lo, hi = w.hi, key_tiles = (hi - lo - 1) / CW + 1;
      const int64_t qh = (int64_t)w.head * p.D;
      const Score sc = score_of(p, w.head);
      const int r0 = w.first + warp * 32;   // the warp's first row
      const bool any = r0 < hi, live = lane < hi - r0;
      const int64_t row = (int64_t)r0 + lane;
      float own[AXES ? AXES : 1];
#pragma unroll
      for (int a = 0; a < AXES; ++a) own[a] = live ? p.pos[row * AXES + a] : 0.f;
      float m = -INFINITY, l = 0.f;                           // m in base-2 units, kLift below the maximum
      for (int j = 0; j < key_tiles; ++j, ++step) {
        const int nc = min(hi - lo - j * CW, CW);
        // S is there; without SEP with it, in order, every earlier product
        ok = wwait_all(s_full, step & 1, limit, abort_flag, err, site(K_ATTN_FWD, 0, 0), step);
        const uint32_t vi = 2 * step + 1;
        if (AXES && ok)
          ok = wwait_all(kv_full + vi % C::SLOTS, (vi / C::SLOTS) & 1, limit, abort_flag, err, site(K_ATTN_FWD, 0, 1), step);
        if (!ok) break;
        tc_fence_after();
        uint32_t raw[CW];
        float* s = reinterpret_cast<float*>(raw);
        if (any) {
          const float* pos = spos + ((vi % C::SLOTS) >> 1) * kMaxAxes * CW;
          auto load = [&] {
#pragma unroll
            for (int c = 0; c < CW / 32; ++c)
              if (c * 32 < nc) tmem_ld32(my + c * 32, raw + c * 32);
            tmem_wait_ld();
#pragma unroll
            for (int c = 0; c < CW / 32; ++c) tie32(raw + c * 32);
          };
          // cap, bias and -inf past the document's end for one chunk of which `left` columns are inside
          auto chunk = [&](float* v, int c, int left) {
            if (CAP && left < 32) {                         // what lies past the end must not choose the tanh
#pragma unroll
              for (int i = 0; i < 32; ++i)
                if (i >= left) v[i] = 0.f;
            }
            transform32<AXES, CAP, CW>(v, pos, c * 32, own, sc, CAP && all_small<32>(v, sc, live));
            if (left < 32) {
#pragma unroll
              for (int i = 0; i < 32; ++i)
                if (i >= left) v[i] = -INFINITY;
            }
          };
          if constexpr (!C::SEP) {
            load();
#pragma unroll
            for (int c = 0; c < CW / 32; ++c)
              if (c * 32 < nc) chunk(s + c * 32, c, nc - c * 32);
          } else {
            constexpr bool PLAIN = !CAP && AXES == 0;
            bool fast = PLAIN || nc == CW;
            if (fast) {
              load();
              if (PLAIN && nc < CW) {                       // the document ends in this tile
#pragma unroll
                for (int i = 0; i < CW; ++i)
                  if (i >= nc) s[i] = -INFINITY;
              }
              if (CAP) fast = all_small<CW>(s, sc, live);
            }
            if (fast) {
#pragma unroll
              for (int c = 0; c < CW / 32; ++c) transform32<AXES, CAP, CW>(s + c * 32, pos, c * 32, own, sc, true);
            } else {
              // a document's last tile, or scores near the cap: through TMEM in a rolled loop (both forms of the
              // tanh unrolled over 128 columns would not fit the instruction cache)
#pragma unroll 1
              for (int c = 0; c * 32 < nc; ++c) {
                uint32_t r[32];
                tmem_ld32(my + c * 32, r);
                tmem_wait_ld();
                tie32(r);
                chunk(reinterpret_cast<float*>(r), c, nc - c * 32);
                tmem_st_32x32b_x16(my + c * 32, r);
                tmem_st_32x32b_x16(my + c * 32 + 16, r + 16);
              }
              tmem_wait_st();
              load();
            }
          }
        }
        if (C::SEP) {
          tc_fence_before();
          mbar_arrive(s_free);
        }
        float top = -INFINITY;
        if (any) {
#pragma unroll
          for (int c = 0; c < CW / 32; ++c) {
            if (c * 32 >= nc) continue;
            const float* v = s + c * 32;
            float t0 = top, t1 = v[0];
#pragma unroll
            for (int i = 1; i < 31; i += 3) {               // three-way maxima, two chains
              t0 = fmaxf(fmaxf(t0, v[i]), v[i + 1]);
              t1 = fmaxf(t1, v[i + 2]);
            }
            top = fmaxf(fmaxf(t0, t1), v[31]);
          }
          top = kLift<E> > 0.f ? fmaf(top, sc.scale2, -kLift<E>) : top * sc.scale2;          // scale > 0
          if (AXES) top = fmaxf(top, -FLT_MAX);             // where every key of the tile is infinitely far away
        }
        if (C::SEP && j > 0) {                              // P's columns, and O, are free once the last product is done
          ok = wwait_all(o_full, (step - 1) & 1, limit, abort_flag, err, site(K_ATTN_FWD, 0, 2), step);
          if (!ok) break;
          tc_fence_after();
        }
        if (any) {
          if (j == 0) {
            m = top;
          } else {
            const bool grow = top > m + kLag;
            if (__any_sync(0xffffffffu, grow)) {
              const float fix = grow ? ex2(m - top) : 1.f;
              l *= fix;
              if (grow) m = top;
#pragma unroll 1
              for (int c = 0; c < d16; ++c) {
                uint32_t o[16];
                tmem_ld_32x32b_x16(my + C::O_COL + c * 16, o);
                tmem_wait_ld();
                tie16(o);
#pragma unroll
                for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * fix);
                tmem_st_32x32b_x16(my + C::O_COL + c * 16, o);
              }
            }
          }
          const uint64_t k2 = pk2(sc.scale2, sc.scale2), off = pk2(-m, -m);
          uint64_t l0 = 0, l1 = 0;
#pragma unroll
          for (int c = 0; c < CW / 32; ++c) {
            if (c * 32 >= nc) continue;
            uint32_t pk[16];
#pragma unroll
            for (int i = 0; i < 32; i += 4) {
              float a, b, d, e;
              unpk2(fma2(pk2(s[c * 32 + i], s[c * 32 + i + 1]), k2, off), a, b);
              unpk2(fma2(pk2(s[c * 32 + i + 2], s[c * 32 + i + 3]), k2, off), d, e);
              a = ex2(a);
              b = ex2(b);
              d = ex2(d);
              e = ex2(e);
              l0 = add2(l0, pk2(a, b));
              l1 = add2(l1, pk2(d, e));
              pk[i / 2] = Pair<E>::pack(a, b);
              pk[i / 2 + 1] = Pair<E>::pack(d, e);
            }
            tmem_st_32x32b_x16(my + (C::SEP ? C::P_COL + c * 16 : c * 32), pk);
          }
          float a, b;
          unpk2(add2(l0, l1), a, b);
          l += a + b;
          tmem_wait_st();
        }
        tc_fence_before();
        mbar_arrive(p_full);
      }
      if (!ok) break;
      ok = wwait_all(o_full, (step - 1) & 1, limit, abort_flag, err, site(K_ATTN_FWD, 0, 3), step);
      if (!ok) break;
      tc_fence_after();
      if (any) {
        const float inv = 1.f / l;
        E* out = static_cast<E*>(p.o) + (int64_t)r0 * p.os + qh;
#pragma unroll
        for (int c = 0; c < DP / 32; ++c) {
          if (c * 32 >= p.D) continue;
          uint32_t o[32], pk[16];
          tmem_ld32(my + C::O_COL + c * 32, o);
          tmem_wait_ld();
          tie32(o);
#pragma unroll
          for (int i = 0; i < 32; i += 2)
            pk[i / 2] = Pair<E>::pack(__uint_as_float(o[i]) * inv, __uint_as_float(o[i + 1]) * inv);
          store32(stage + warp * STAGE, pk, out, p.os, hi - r0, c * 32, p.D, lane);
        }
        if (live) p.lse[(int64_t)w.head * p.N + row] = (m + log2f(l)) * kLn2;
      }
      tc_fence_before();
    }
    if (!ok && lane == 0) raise_abort(abort_flag, err);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == MMA_WARP) tmem_dealloc(tmem, C::TMEM);
}

template <int DP, int CW, typename E, bool CAP>
cudaError_t forward_axes(const Params& p, const Maps& maps, cudaStream_t st) {
  constexpr int smem = FwdCfg<DP, CW>::SMEM;
  switch (p.axes) {
    case 0: return launch_rows(attn_tc_fwd_kernel<DP, CW, E, 0, CAP>, smem, p, maps, p.H, kThreads, 2, st);
    case 1: return launch_rows(attn_tc_fwd_kernel<DP, CW, E, 1, CAP>, smem, p, maps, p.H, kThreads, 2, st);
    case 2: return launch_rows(attn_tc_fwd_kernel<DP, CW, E, 2, CAP>, smem, p, maps, p.H, kThreads, 2, st);
    default: return launch_rows(attn_tc_fwd_kernel<DP, CW, E, 3, CAP>, smem, p, maps, p.H, kThreads, 2, st);
  }
}
template <int DP, int CW, typename E>
cudaError_t forward_cap(const Params& p, cudaStream_t st) {
  Maps maps;
  cudaError_t e = enter_context();
  if (e == cudaSuccess) e = make_map(&maps.m[0], p.q, Pair<E>::fmt, p, p.H, p.qs, ROWS);
  if (e == cudaSuccess) e = make_map(&maps.m[1], p.k, Pair<E>::fmt, p, p.K, p.ks, CW);
  if (e == cudaSuccess) e = make_map(&maps.m[2], p.v, Pair<E>::fmt, p, p.K, p.vs, CW);
  if (e != cudaSuccess) return e;
  maps.m[3] = maps.m[0];
  return p.cap > 0.f ? forward_axes<DP, CW, E, true>(p, maps, st) : forward_axes<DP, CW, E, false>(p, maps, st);
}
template <typename E>
cudaError_t forward_dim(const Params& p, cudaStream_t st) {
  if (p.D > 64) return forward_cap<128, 64, E>(p, st);
  // by the average length, not by max_len: results do not depend on that
  const int64_t from = p.cap > 0.f || p.axes ? kWideFromBiased : kWideFrom;
  return p.N >= from * p.docs ? forward_cap<64, 128, E>(p, st) : forward_cap<64, 64, E>(p, st);
}

}  // namespace attn_tc

cudaError_t launch_attn_tc_forward(const attn::Params& p, eqlin_dtype_t dt, cudaStream_t st) {
  return dt == EQLIN_F16 ? attn_tc::forward_dim<__half>(p, st) : attn_tc::forward_dim<__nv_bfloat16>(p, st);
}

}  // namespace eqlin
