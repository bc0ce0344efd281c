// eqlin_attn_tc_bwd.cuh -- document attention, backward, on the tensor cores.
//
// Two kernels of one template.  KEYS = false owns 128 query rows and passes
// over the keys: dq, and delta on the way.  KEYS = true owns 128 key rows and
// passes over the queries of every head that shares them: dk, dv.  Both form
// the scores again; in exchange no sum crosses blocks, so there are no atomics
// and results are the same in every run.  With own tiles (A0, A1) = (Q, dO) or
// (K, V) and moving tiles (X, Y) = (K, V) or (Q, dO):
//
//   S = A0 X^T,  dP = A1 Y^T          TMEM accumulators
//   P = 2^(s - lse),  du = P (dP - delta) g,  g = 1 - tanh^2    FP32 registers
//   KEYS:  dv += P Y,  dk += du X     A from TMEM, 16 bits
//   else:  e += (P g) X,  dq += du X
//
// P and du are rounded to the inputs' type as operands of those products, half
// a step each; sums are FP32 in TMEM.  f16's range is narrow: du is about the
// gradient over the document's length, below 6e-5 it loses bits, and under a
// loss scale dP alone can pass 65504.  So in f16 both carry powers of two, which
// the FP32 results are freed of.  P, at most 1, has 2^12.  A row of du has its
// own, f: with top the row's largest |dP| + |delta| in a tile, f top is brought
// to 2^12 .. 2^13 in the first tile and again in any tile where it passes 2^14
// (so is du f then, with room for a P that rounding puts above 1), and what the
// row has summed up follows.  A row's results are then off by at most 2^-37 of
// its largest top for each of its du, beside the roundings.  The other look at dP
// costs an f16 backward 9 to 14 % (12544 tokens, 6 heads of 64: 1.24 to 1.38 ms;
// 64 x 197 tokens, 12 heads, capped, two-axis bias: 175 to 193 us; 2048 windows of
// 49 tokens, 3 heads of 32: 161 to 181 us).  Bounds from max|do| and max|v|, found
// in shared memory before the scores, cost long documents 2 to 6 % and short ones
// up to 25 %.
//
// delta = do.o from the stored o would carry o's rounding (its own and that of
// P in the forward) into every du; for short documents that is more than all
// other roundings together.  It only serves as a first guess d0 here: the
// dq kernel sums eps = sum_j P (dP - d0), so delta = d0 + eps exactly in FP32,
// which is what the dk, dv kernel reads, and corrects its own result by
// dq = sum du0 k - eps sum P g k.  That second product costs a quarter of the
// kernel's MMAs; another pass for delta would cost twice that.
//
// A thread owns one row and 64 columns of a tile (NWG warpgroups of rows, the
// 32-column chunks dealt out in turn).  P and du lie over the scores they came
// from, chunk by chunk: the accumulators take the rest of the columns, and the
// SM's other block fills the gap until the next scores.  Measured, bf16, both
// kernels: 12544 tokens, 6 heads of 64, 1.23 ms (490 TFLOP/s of the formula's five
// products); 64 x 197 tokens, 12 heads, capped, two-axis bias, 179 us; one tile of
// 64 moving rows takes an SM about 1550 cycles, 512 of them exponentials.
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
  static constexpr int S_COL = 0, DP_COL = CW, ACC0 = 2 * CW;   // ACC0: dv, or e
  static constexpr int ACC1 = ACC0 + DP;                        // dk, or dq
  static constexpr int OWN = DP / 64 * PANEL;                   // bytes of one own tile
  static constexpr int MOV_PANEL = CW * 128;
  static constexpr int MOV = DP / 64 * MOV_PANEL;               // bytes of one moving tile
  static constexpr int SLOTS = DP > 64 ? 2 : 4;
  // positions, lse, delta and the largest |delta| (in 16 bytes) of a slot
  static constexpr int SIDE = (kMaxAxes + (KEYS ? 2 : 0)) * CW * 4 + (KEYS ? 16 : 0);
  static constexpr int NBAR = 2 + 3 * SLOTS + 6;
  static constexpr int EPS = NWG == 2 ? 4 * ROWS * 4 : 0;       // eps and top of the two warpgroups
  static constexpr int SMEM = 2 * OWN + SLOTS * (2 * MOV + SIDE) + EPS + NWG * 4 * STAGE + NBAR * 8 + 32 + kListInts * 4 + 1024;
  static_assert(ACC1 + DP <= TMEM, "TMEM columns");
  static_assert(BLOCKS * SMEM <= 227 * 1024, "shared memory");
};

// One 32-column chunk of a row: raw scores rs and dP rd in, packed P and du out.
//   KEYS: -lse and delta belong to the columns (in shared memory, in base 2 and
//   scaled), else to the row.
// FMA-pipe operations per element, which bound this under a cap: 8 for the tanh
// and its derivative, 2 axes for the bias, 5 for the rest.  Two signs cancel to
// save two more: under a cap diff is delta - dP and gain tanh^2 - 1, so that du
// is right, while eps and P g (KEYS = false) come out negated, and so does not
// their product.
// In f16 P comes out times 2^kUp, du and the terms of eps times the row's f.
constexpr float kUp16 = 12.f, kDown16 = 1.f / 4096.f;     // P's power of two in f16, and its inverse
template <int AXES, bool CAP, bool KEYS, bool SMALL, bool EDGE, int CW, typename E>
__device__ __forceinline__ void grad32(const uint32_t* rs, const uint32_t* rd, const float* side, int c0, const float* own,
                                       float lse2, float delta, float f, const Score& sc, int left, uint64_t& eps,
                                       uint32_t* pp, uint32_t* pd) {
  constexpr bool F16 = Pair<E>::fmt == 0;
  const float fd = F16 ? f * kDown16 : 1.f;          // of dP and delta: P brings the rest
  const uint64_t plus_f = pk2(fd, fd), minus_f = pk2(-fd, -fd);
  const uint64_t k2 = CAP ? pk2(sc.cap2, sc.cap2) : pk2(sc.scale2, sc.scale2);
  const uint64_t in = pk2(sc.in, sc.in), slope = pk2(-sc.slope2, -sc.slope2);
  const uint64_t minus = pk2(-1.f, -1.f);
  const float off_row = F16 ? kUp16 - lse2 : -lse2, delta_row = CAP ? delta * fd : -delta * fd;
  const uint64_t row_off = pk2(off_row, off_row), row_delta = pk2(delta_row, delta_row);
#pragma unroll
  for (int j = 0; j < 32; j += 4) {
    float d[4];
    if (AXES) distances<AXES, CW>(side, c0 + j, own, d);
    ulonglong2 ls, dl;
    if (KEYS) {
      ls = *reinterpret_cast<const ulonglong2*>(side + kMaxAxes * CW + c0 + j);
      dl = *reinterpret_cast<const ulonglong2*>(side + (kMaxAxes + 1) * CW + c0 + j);
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int i = j + 2 * h;
      uint64_t x = pk2(__uint_as_float(rs[i]), __uint_as_float(rs[i + 1]));
      const uint64_t dp = pk2(__uint_as_float(rd[i]), __uint_as_float(rd[i + 1]));
      uint64_t gain = minus;                         // tanh^2 - 1
      if (CAP) {
        if (SMALL) {
          x = mul2(x, in);
          x = mul2(x, q_small2(x));
        } else {
          float a, b;
          unpk2(x, a, b);
          tanh_any2(a, b, sc);
          x = pk2(a, b);
        }
        gain = fma2(x, x, minus);
      }
      uint64_t off = KEYS ? (h ? ls.y : ls.x) : row_off;
      if (AXES) off = fma2(slope, pk2(d[2 * h], d[2 * h + 1]), off);
      float a, b;
      unpk2(fma2(x, k2, off), a, b);
      a = ex2(a);
      b = ex2(b);
      if (EDGE) {                                    // no probability past the document's end
        if (i >= left) a = 0.f;
        if (i + 1 >= left) b = 0.f;
      }
      // delta - dP under a cap, else dP - delta (the factors are powers of two: their products are exact)
      uint64_t diff;
      if (KEYS) {
        const uint64_t de = h ? dl.y : dl.x;
        if (CAP) diff = F16 ? fma2(de, plus_f, mul2(dp, minus_f)) : fma2(dp, minus, de);
        else diff = F16 ? fma2(de, minus_f, mul2(dp, plus_f)) : fma2(de, minus, dp);
      } else if (F16) {
        diff = fma2(dp, CAP ? minus_f : plus_f, row_delta);
      } else {
        diff = CAP ? fma2(dp, minus, row_delta) : add2(dp, row_delta);
      }
      uint64_t prob = pk2(a, b);
      if (!KEYS) eps = fma2(prob, diff, eps);
      if (!KEYS && CAP) prob = mul2(prob, gain);     // KEYS: dv takes P itself
      uint64_t du = mul2(prob, diff);
      if (KEYS && CAP) du = mul2(du, gain);
      float e, f;
      unpk2(prob, a, b);
      unpk2(du, e, f);
      pp[i / 2] = Pair<E>::pack(a, b);
      pd[i / 2] = Pair<E>::pack(e, f);
    }
  }
}

// The largest magnitude of a row's 64 values x, y, of which `left` and `left` - `apart` are inside.
__device__ __forceinline__ float top64(uint32_t* x, uint32_t* y, int left, int apart) {
  if (left < 32 + apart) {
#pragma unroll
    for (int i = 0; i < 32; ++i) {
      if (i >= left) x[i] = 0u;
      if (i >= left - apart) y[i] = 0u;
    }
  }
  float a = 0.f, b = 0.f, c = 0.f, d = 0.f;
#pragma unroll
  for (int i = 0; i < 32; i += 4) {
    a = fmaxf(fmaxf(a, fabsf(__uint_as_float(x[i]))), fabsf(__uint_as_float(x[i + 1])));
    b = fmaxf(fmaxf(b, fabsf(__uint_as_float(x[i + 2]))), fabsf(__uint_as_float(x[i + 3])));
    c = fmaxf(fmaxf(c, fabsf(__uint_as_float(y[i]))), fabsf(__uint_as_float(y[i + 1])));
    d = fmaxf(fmaxf(d, fabsf(__uint_as_float(y[i + 2]))), fabsf(__uint_as_float(y[i + 3])));
  }
  return fmaxf(fmaxf(a, b), fmaxf(c, d));
}
// The power of two that brings top into [2^12, 2^13), at most 2^100, and its inverse.
__device__ __forceinline__ uint32_t top_exponent(float top) { return max((__float_as_uint(top) >> 23) & 255u, 39u); }
__device__ __forceinline__ float factor_of(uint32_t e) { return __uint_as_float((266u - e) << 23); }
__device__ __forceinline__ float inverse_of(uint32_t e) { return __uint_as_float((e - 12u) << 23); }

template <int DP, typename E, int AXES, bool CAP, bool KEYS>
__global__ void __launch_bounds__(BwdCfg<DP, KEYS>::THREADS, BwdCfg<DP, KEYS>::BLOCKS)
attn_tc_bwd_kernel(const __grid_constant__ Params p, const __grid_constant__ Maps maps) {
  using C = BwdCfg<DP, KEYS>;
  constexpr int CW = C::CW, NWG = C::NWG;
  constexpr uint32_t KID = KEYS ? K_ATTN_DKV : K_ATTN_DQ;
  constexpr bool F16 = Pair<E>::fmt == 0;
  constexpr float kUp = F16 ? kUp16 : 0.f, kDown = F16 ? kDown16 : 1.f;   // P's factor (as an exponent), its inverse
  constexpr int MMA = NWG * 4, LOAD = NWG * 4 + 1;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  uint8_t* ring = smem + 2 * C::OWN;
  float* side = reinterpret_cast<float*>(ring + C::SLOTS * 2 * C::MOV);
  constexpr int SIDE_F = C::SIDE / 4;
  float* eps_sum = side + C::SLOTS * SIDE_F;         // [2][ROWS]
  float* tops = eps_sum + 2 * ROWS;                  // [2][ROWS]
  uint8_t* stage = reinterpret_cast<uint8_t*>(eps_sum + C::EPS / 4);
  uint64_t* bars = reinterpret_cast<uint64_t*>(stage + NWG * 4 * STAGE);
  uint64_t* own_full = bars;
  uint64_t* own_empty = bars + 1;
  uint64_t* full = bars + 2;
  uint64_t* empty = full + C::SLOTS;
  uint64_t* land = empty + C::SLOTS;
  uint64_t* s_full = land + C::SLOTS;
  uint64_t* p_full = s_full + 1;
  uint64_t* acc_full = p_full + 1;
  uint64_t* eps_full = acc_full + 1;
  uint64_t* top_full = eps_full + 1;
  uint64_t* drain = top_full + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + C::NBAR);
  int* abort_word = reinterpret_cast<int*>(tmem_slot + 1);
  int* local_err = abort_word + 1;
  int* list = local_err + 4;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  grid_dep_wait();
  const int rep = p.H / p.K, heads = KEYS ? p.K : p.H;
  const int passes = KEYS ? rep : 1;                 // query heads that pass by
  const uint32_t count = begin(p, heads, list, [&](int head, int64_t r) {
        for (int d = threadIdx.x; d < p.D; d += C::THREADS) {
          const int64_t at = (int64_t)head * p.D + d;
          if (KEYS) {
            static_cast<E*>(p.dk)[r * p.dks + at] = Elem<E>::from_f(0.f);
            static_cast<E*>(p.dv)[r * p.dvs + at] = Elem<E>::from_f(0.f);
          } else {
            static_cast<E*>(p.dq)[r * p.dqs + at] = Elem<E>::from_f(0.f);
          }
        }
      });
  if (count == 0) return;

  if (threadIdx.x == 0) {
    mbar_init(own_full, 32);
    mbar_init(own_empty, 1);
    for (int i = 0; i < C::SLOTS; ++i) {
      mbar_init(full + i, 32);
      mbar_init(empty + i, 1);
      mbar_init(land + i, 1);
    }
    mbar_init(s_full, 1);
    mbar_init(p_full, NWG * 128);
    mbar_init(acc_full, 1);
    mbar_init(eps_full, NWG * 128);
    mbar_init(top_full, NWG * 128);
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
  const uint32_t tmem = uniform(*tmem_slot);
  grid_dep_launch();                                 // after the allocation, as in the forward
  volatile int* abort_flag = abort_word;
  int* err = p.err ? p.err : local_err;
  const uint32_t limit = p.wait_limit;
  const int d16 = (p.D + 15) / 16;

  if (warp == LOAD) {
    const Waits wait{limit, abort_flag, err};
    Tails tails;
    Side<AXES, KEYS, CW> sides;
    uint32_t item = 0, owns = 0;
    bool ok = true;
    for (uint32_t i = 0; ok && i < count; ++i) {
      const Tile w = tile_at(p, heads, list, i);
      const int kv_head = KEYS ? w.head : w.head / rep, q_head = KEYS ? w.head * rep : w.head;
      const int lo = w.lo, hi = w.hi, tiles = (hi - lo - 1) / CW + 1;   // moving tiles of one head
      sides.fetch(p, q_head, lo, hi, lane);
      ok = claim<DP, CW, 2>(tails, own_empty, (owns & 1) ^ 1, ring, land, full, wait, site(KID, 2, 0), owns, lane);
      if (!ok) break;
      if (lane == 0) {
        const int head = KEYS ? kv_head : q_head;
        expect_bytes(own_full, 2 * C::OWN);
        tma_rows<DP, ROWS>(smem, &maps.m[0], head, w.first, own_full);
        tma_rows<DP, ROWS>(smem + C::OWN, &maps.m[1], head, w.first, own_full);
      }
      mbar_arrive(own_full);
      ++owns;
      for (int g = 0; ok && g < passes; ++g)
        for (int j = 0; ok && j < tiles; ++j) {
          const int c0 = lo + j * CW, nc = min(hi - c0, CW);
          const uint32_t slot = item % C::SLOTS;
          ok = claim<DP, CW, 2>(tails, empty + slot, ((item / C::SLOTS) & 1) ^ 1, ring, land, full, wait,
                                site(KID, 2, 1), item, lane);
          if (!ok) break;
          if (AXES || KEYS) {
            sides.store(side + slot * SIDE_F, kUp, lane);
            if constexpr (KEYS && F16) sides.store_top(side + slot * SIDE_F, lane);
            const bool last = j + 1 == tiles;
            if (!last || g + 1 < passes) sides.fetch(p, q_head + g + (last ? 1 : 0), last ? lo : c0 + CW, hi, lane);
          }
          ok = bring<DP, CW, 2>(tails, slot, ring, land, full, &maps.m[2], KEYS ? q_head + g : kv_head, c0, nc, wait,
                                site(KID, 2, 2), lane);
          ++item;
        }
    }
    if (ok) ok = settle<DP, CW, 2>(tails, tails.count, ring, land, full, wait, site(KID, 2, 2), lane);
    if (!ok && lane == 0) raise_abort(abort_flag, err);
    drain_loads(tails, land, own_full, owns, full, item, C::SLOTS);
  } else if (warp == MMA) {
    const uint32_t leader = lane == 0;
    uint32_t item = 0, owns = 0;
    bool ok = true;
    int lo = 0, hi = 0;
    const uint64_t own_desc = smem_desc(smem_u32(smem), 128);
    const uint32_t a0 = lo32(own_desc), a1 = a0 + (C::OWN >> 4), k_hi = hi32(own_desc);
    const uint32_t ring_k = lo32(smem_desc(smem_u32(ring), 128));
    const uint64_t mn_desc = smem_desc_mn(smem_u32(ring), C::MOV_PANEL, 1024);
    const uint32_t ring_mn = lo32(mn_desc), mn_hi = hi32(mn_desc);
    const uint32_t id_acc = idesc_f16(Pair<E>::fmt, (uint32_t)(16 * d16)) | kBTransposed;
    auto scores = [&](uint32_t it, int j) -> bool {
      const int slot = it % C::SLOTS;
      if (!wwait_all(full + slot, (it / C::SLOTS) & 1, limit, abort_flag, err, site(KID, 1, 1), it)) return false;
      tc_fence_after();
      const uint32_t id = idesc_f16(Pair<E>::fmt, (uint32_t)((min(hi - lo - j * CW, CW) + 15) & ~15));
      const uint32_t x = ring_k + slot * (2 * C::MOV >> 4);
#pragma unroll
      for (int d = 0; d < DP / 16; ++d)
        if (d < d16) {
          const uint32_t oa = ((d >> 2) * PANEL + (d & 3) * 32) >> 4, ob = ((d >> 2) * C::MOV_PANEL + (d & 3) * 32) >> 4;
          mma_ss(leader, tmem + C::S_COL, a0 + oa, x + ob, k_hi, id, d > 0);
        }
#pragma unroll
      for (int d = 0; d < DP / 16; ++d)
        if (d < d16) {
          const uint32_t oa = ((d >> 2) * PANEL + (d & 3) * 32) >> 4, ob = ((d >> 2) * C::MOV_PANEL + (d & 3) * 32) >> 4;
          mma_ss(leader, tmem + C::DP_COL, a1 + oa, x + (C::MOV >> 4) + ob, k_hi, id, d > 0);
        }
      commit(leader, s_full);
      return true;
    };
    for (; ok && owns < count; ++owns) {
      const Tile w = tile_at(p, heads, list, owns);
      lo = w.lo;
      hi = w.hi;
      const int tiles = (hi - lo - 1) / CW + 1;      // moving tiles of one head
      ok = wwait_all(own_full, owns & 1, limit, abort_flag, err, site(KID, 1, 0), owns) && scores(item, 0);
      const int all = passes * tiles;
      if (ok && all == 1) commit(leader, own_empty);
      int j = 0;                                     // moving tile of the present pass
      for (int i = 0; ok && i < all; ++i, ++item) {
        const bool more = i + 1 < all;
        const int next = j + 1 < tiles ? j + 1 : 0;
        ok = wwait_all(p_full, item & 1, limit, abort_flag, err, site(KID, 1, 3), item);
        if (!ok) break;
        tc_fence_after();
        const int steps = (min(hi - lo - j * CW, CW) + 15) / 16, slot = item % C::SLOTS;
        const uint32_t x = ring_mn + slot * (2 * C::MOV >> 4), y = x + (C::MOV >> 4);
        // P and du lie over the scores' chunks
        const uint32_t b0 = KEYS ? y : x;
#pragma unroll
        for (int s = 0; s < CW / 16; ++s)
          if (s < steps)
            mma_ts(leader, tmem + C::ACC0, tmem + C::S_COL + 32 * (s >> 1) + 8 * (s & 1),
                   b0 + s * (2048 >> 4), mn_hi, id_acc, i > 0 || s > 0);
#pragma unroll
        for (int s = 0; s < CW / 16; ++s)
          if (s < steps)
            mma_ts(leader, tmem + C::ACC1, tmem + C::DP_COL + 32 * (s >> 1) + 8 * (s & 1),
                   x + s * (2048 >> 4), mn_hi, id_acc, i > 0 || s > 0);
        commit(leader, acc_full);
        commit(leader, empty + slot);
        if (more) ok = scores(item + 1, next);   // in order behind the products that read P and du
        if (i + 2 == all) commit(leader, own_empty);   // every product with the own tiles is issued
        j = next;
      }
    }
    if (!ok && lane == 0) raise_abort(abort_flag, err);
    commit(leader, drain);
    mbar_wait(drain, 0, kDefaultWaitLimit);
    __syncwarp();
  } else {
    const int wg = warp >> 2, quarter = warp & 3;
    const uint32_t my = tmem + ((uint32_t)(quarter * 32) << 16);
    uint32_t item = 0;
    bool ok = true;
    // A tile's own rows: positions and, where queries own, lse (base 2) and the
    // first guess of delta.  Read while the tile before ends.
    Tile w;
    float own[AXES ? AXES : 1], lse2 = 0.f, delta = 0.f;
    auto enter = [&](uint32_t i) {
      w = tile_at(p, heads, list, i);
      const int r0 = w.first + quarter * 32;
      const int64_t row = (int64_t)r0 + lane;
      const bool live = row < w.hi;
#pragma unroll
      for (int a = 0; a < AXES; ++a) own[a] = live ? p.pos[row * AXES + a] : 0.f;
      if (!KEYS && r0 < w.hi) {
        const int64_t at = (int64_t)w.head * p.D;
        delta = row_dots(static_cast<const E*>(p.go) + (int64_t)r0 * p.gos + at, p.gos,
                         static_cast<const E*>(p.o) + (int64_t)r0 * p.os + at, p.os, w.hi - r0, p.D, lane);
        lse2 = live ? p.lse[(int64_t)w.head * p.N + row] * kLog2e : 0.f;
      }
    };
    enter(0);
    for (uint32_t i = 0; ok && i < count; ++i) {
      const int kv_head = KEYS ? w.head : w.head / rep, q_head = KEYS ? w.head * rep : w.head;
      const int64_t kh = (int64_t)kv_head * p.D, qh0 = (int64_t)q_head * p.D;
      const int lo = w.lo, hi = w.hi, tiles = (hi - lo - 1) / CW + 1;   // moving tiles of one head
      const int r0 = w.first + quarter * 32;
      const bool any = r0 < hi, live = lane < hi - r0;
      const int64_t row = (int64_t)r0 + lane;
      uint64_t eps2 = 0;
      uint32_t fe = 0;                               // the row's factor in f16: factor_of(fe)
      for (int g = 0; ok && g < passes; ++g) {
        const Score sc = score_of(p, q_head + g);
        for (int j = 0; j < tiles; ++j, ++item) {
          const int nc = min(hi - lo - j * CW, CW), slot = item % C::SLOTS;
          const float* sd = side + slot * SIDE_F;
          ok = wwait_all(s_full, item & 1, limit, abort_flag, err, site(KID, 0, 0), item);
          if ((AXES || KEYS) && ok)
            ok = wwait_all(full + slot, (item / C::SLOTS) & 1, limit, abort_flag, err, site(KID, 0, 1), item);
          if (!ok) break;
          tc_fence_after();
          if constexpr (F16) {
            float top = 0.f;
            if (any) {                               // this warpgroup's two chunks
              uint32_t x[32], y[32];
              tmem_ld32(my + C::DP_COL + wg * 32, x);
              tmem_ld32(my + C::DP_COL + (wg + NWG) * 32, y);
              tmem_wait_ld();
              tie32(x);
              tie32(y);
              top = top64(x, y, nc - wg * 32, NWG * 32);
            }
            if (NWG == 2) {                          // and the other's, as with eps below
              tops[wg * ROWS + quarter * 32 + lane] = top;
              mbar_arrive(top_full);
              ok = wwait_all(top_full, item & 1, limit, abort_flag, err, site(KID, 0, 5), item);
              if (!ok) break;
              top = fmaxf(tops[quarter * 32 + lane], tops[ROWS + quarter * 32 + lane]);
            }
            top += KEYS ? sd[(kMaxAxes + 2) * CW] : fabsf(delta);
            if (g == 0 && j == 0) {
              fe = top_exponent(top);
            } else if (any) {
              const bool grow = top * factor_of(fe) > 16384.f;
              if (__any_sync(0xffffffffu, grow)) {
                // every product before these scores is done: the sums may be changed
                const uint32_t now = grow ? top_exponent(top) : fe;
                const float fix = factor_of(now) * inverse_of(fe);
                fe = now;
                eps2 = mul2(eps2, pk2(fix, fix));
#pragma unroll 1
                for (int c = wg; c < d16; c += NWG) {
                  uint32_t x[16];
                  tmem_ld_32x32b_x16(my + C::ACC1 + c * 16, x);
                  tmem_wait_ld();
                  tie16(x);
#pragma unroll
                  for (int k = 0; k < 16; ++k) x[k] = __float_as_uint(__uint_as_float(x[k]) * fix);
                  tmem_st_32x32b_x16(my + C::ACC1 + c * 16, x);
                }
              }
            }
          }
          if (any) {
            const float f = F16 ? factor_of(fe) : 1.f;
            // this warpgroup's chunks: wg, wg + NWG
#pragma unroll 1
            for (int c = wg; c * 32 < nc; c += NWG) {
              uint32_t rs[32], rd[32], pp[16], pd[16];
              tmem_ld32(my + C::S_COL + c * 32, rs);
              tmem_ld32(my + C::DP_COL + c * 32, rd);
              tmem_wait_ld();
              tie32(rs);
              tie32(rd);
              // Past the document's end dP = delta, and P = 0 by a raw score of -inf or, where a cap would bring that
              // back to -cap, by EDGE.  KEYS: lse is +inf there, so any finite score will do.
              const int left = nc - c * 32;
              if ((!KEYS || CAP) && left < 32) {
#pragma unroll
                for (int k = 0; k < 32; ++k)
                  if (k >= left) {
                    rs[k] = KEYS || CAP ? 0u : __float_as_uint(-INFINITY);
                    if (!KEYS) rd[k] = __float_as_uint(delta);
                  }
              }
              if (CAP && !KEYS && left < 32)
                grad32<AXES, CAP, KEYS, false, CAP && !KEYS, CW, E>(rs, rd, sd, c * 32, own, lse2, delta, f, sc, left, eps2,
                                                                    pp, pd);
              else if (CAP && all_small<32>(reinterpret_cast<const float*>(rs), sc, live))
                grad32<AXES, CAP, KEYS, true, false, CW, E>(rs, rd, sd, c * 32, own, lse2, delta, f, sc, 32, eps2, pp, pd);
              else
                grad32<AXES, CAP, KEYS, false, false, CW, E>(rs, rd, sd, c * 32, own, lse2, delta, f, sc, 32, eps2, pp, pd);
              tmem_st_32x32b_x16(my + C::S_COL + c * 32, pp);
              tmem_st_32x32b_x16(my + C::DP_COL + c * 32, pd);
            }
            tmem_wait_st();
          }
          tc_fence_before();
          mbar_arrive(p_full);
        }
      }
      if (!ok) break;
      const float guess = delta, inv_f = F16 ? inverse_of(fe) : 1.f;
      if (i + 1 < count) enter(i + 1);
      ok = wwait_all(acc_full, (item - 1) & 1, limit, abort_flag, err, site(KID, 0, 3), item);
      if (!ok) break;
      tc_fence_after();
      float eps = 0.f;
      if (!KEYS) {
        float a, b;
        unpk2(eps2, a, b);
        eps = a + b;
        if (NWG == 2) {                              // the two halves of the row's columns
          // (a bounded wait, not a block barrier: a warp that gave up does not come here; the next tile's sums are
          // written after every warp has passed this one's scores, and so this)
          eps_sum[wg * ROWS + quarter * 32 + lane] = eps;
          mbar_arrive(eps_full);
          ok = wwait_all(eps_full, i & 1, limit, abort_flag, err, site(KID, 0, 4), item);
          if (!ok) break;
          eps = eps_sum[quarter * 32 + lane] + eps_sum[ROWS + quarter * 32 + lane];
        }
        if (live && wg == 0) p.delta[(int64_t)q_head * p.N + row] = CAP ? guess - eps * inv_f : guess + eps * inv_f;
      }
      if (any) {
#pragma unroll
        for (int c = 0; c < DP / 32; ++c) {
          if (c * 32 >= p.D || c % NWG != wg) continue;
          const float fix = p.scale * inv_f;
          uint32_t x[32], y[32], pk[16];
          tmem_ld32(my + C::ACC0 + c * 32, x);
          tmem_ld32(my + C::ACC1 + c * 32, y);
          tmem_wait_ld();
          tie32(x);
          tie32(y);
          uint8_t* st = stage + warp * STAGE;
          if (KEYS) {
#pragma unroll
            for (int i = 0; i < 32; i += 2)
              pk[i / 2] = Pair<E>::pack(__uint_as_float(x[i]) * kDown, __uint_as_float(x[i + 1]) * kDown);
            store32(st, pk, static_cast<E*>(p.dv) + (int64_t)r0 * p.dvs + kh, p.dvs, hi - r0, c * 32, p.D, lane);
          }
#pragma unroll
          for (int i = 0; i < 32; i += 2) {
            float a = __uint_as_float(y[i]), b = __uint_as_float(y[i + 1]);
            if (!KEYS) {
              a = fmaf(-eps * kDown, __uint_as_float(x[i]), a);
              b = fmaf(-eps * kDown, __uint_as_float(x[i + 1]), b);
            }
            pk[i / 2] = Pair<E>::pack(a * fix, b * fix);
          }
          if (KEYS) store32(st, pk, static_cast<E*>(p.dk) + (int64_t)r0 * p.dks + kh, p.dks, hi - r0, c * 32, p.D, lane);
          else store32(st, pk, static_cast<E*>(p.dq) + (int64_t)r0 * p.dqs + qh0, p.dqs, hi - r0, c * 32, p.D, lane);
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
cudaError_t backward_axes(const Params& p, const Maps& maps, cudaStream_t st) {
  using C = BwdCfg<DP, KEYS>;
  const int heads = KEYS ? p.K : p.H;
  switch (p.axes) {
    case 0: return launch_rows(attn_tc_bwd_kernel<DP, E, 0, CAP, KEYS>, C::SMEM, p, maps, heads, C::THREADS, C::BLOCKS, st);
    case 1: return launch_rows(attn_tc_bwd_kernel<DP, E, 1, CAP, KEYS>, C::SMEM, p, maps, heads, C::THREADS, C::BLOCKS, st);
    case 2: return launch_rows(attn_tc_bwd_kernel<DP, E, 2, CAP, KEYS>, C::SMEM, p, maps, heads, C::THREADS, C::BLOCKS, st);
    default: return launch_rows(attn_tc_bwd_kernel<DP, E, 3, CAP, KEYS>, C::SMEM, p, maps, heads, C::THREADS, C::BLOCKS, st);
  }
}
template <int DP, typename E, bool KEYS>
cudaError_t backward_cap(const Params& p, cudaStream_t st) {
  constexpr uint32_t fmt = Pair<E>::fmt;
  constexpr int CW = BwdCfg<DP, KEYS>::CW;
  Maps maps;                                         // own tiles A0, A1, moving tiles X, Y
  cudaError_t e = enter_context();
  if (e == cudaSuccess) e = make_map(&maps.m[KEYS ? 2 : 0], p.q, fmt, p, p.H, p.qs, KEYS ? CW : ROWS);
  if (e == cudaSuccess) e = make_map(&maps.m[KEYS ? 3 : 1], p.go, fmt, p, p.H, p.gos, KEYS ? CW : ROWS);
  if (e == cudaSuccess) e = make_map(&maps.m[KEYS ? 0 : 2], p.k, fmt, p, p.K, p.ks, KEYS ? ROWS : CW);
  if (e == cudaSuccess) e = make_map(&maps.m[KEYS ? 1 : 3], p.v, fmt, p, p.K, p.vs, KEYS ? ROWS : CW);
  if (e != cudaSuccess) return e;
  return p.cap > 0.f ? backward_axes<DP, E, true, KEYS>(p, maps, st) : backward_axes<DP, E, false, KEYS>(p, maps, st);
}
template <bool KEYS>
cudaError_t backward_pick(const Params& p, eqlin_dtype_t dt, cudaStream_t st) {
  if (dt == EQLIN_F16)
    return p.D <= 64 ? backward_cap<64, __half, KEYS>(p, st) : backward_cap<128, __half, KEYS>(p, st);
  return p.D <= 64 ? backward_cap<64, __nv_bfloat16, KEYS>(p, st) : backward_cap<128, __nv_bfloat16, KEYS>(p, st);
}

}  // namespace attn_tc
}  // namespace eqlin
