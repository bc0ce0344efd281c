// eqlin_attn_tc.cuh -- parts shared by the tensor-core attention kernels.
//
// All of them have one shape: 128 rows stay ("own" rows: queries, or keys in
// the kernel for dk and dv), the other side passes by in tiles of up to 128
// ("moving" rows).  A block is six warps, or ten with two threads per own row:
//
//   warps 0-3   one thread per own row: scores out of TMEM, softmax (or its
//               gradient) in FP32 registers, 16-bit probabilities back into
//               TMEM as the next product's A operand
//   warp 4      issues the MMAs: the whole warp runs the loops, so that
//               descriptors stay in uniform registers, and one lane's predicate
//               is set on the instruction itself; the warp allocates TMEM
//   warp 5      brings tiles into shared memory with TMA (a 3D map over
//               features, heads, tokens: features past D read as zero) and
//               clears the rows between a document's end and the next multiple
//               of 16 in its last moving tile, which the products still read: a
//               neighbour's rows must not be there, since a product with P = 0
//               would spread their infinities and NaNs.  (Own rows past the end
//               are whatever lies there: a row's results stay in that row.)
//
// Shared tiles are panels of 64 features: 128 rows of 128 bytes in the
// 128-byte swizzle (16-byte chunk j of row r at chunk j ^ (r & 7)).  The same
// image serves as a K-major operand (contraction over features) and as an
// MN-major one (contraction over rows).
#pragma once

#include <cudaTypedefs.h>

#include "eqlin_attn.cuh"
#include "eqlin_ptx.cuh"
#include "eqlin_wait.cuh"

namespace eqlin {
namespace attn_tc {

using namespace attn;
using namespace ptx;
using namespace waits;

constexpr int ROWS = 128;
constexpr int PANEL = ROWS * 128;         // bytes of a panel
constexpr int kThreads = 192;
constexpr int MMA_WARP = 4, LOAD_WARP = 5;

// kernels in the error record
enum : uint32_t { K_ATTN_FWD = 4, K_ATTN_DQ = 5, K_ATTN_DKV = 6 };

template <typename E> struct Pair;
template <> struct Pair<__half> {
  static constexpr uint32_t fmt = 0;
  static __device__ __forceinline__ uint32_t pack(float lo, float hi) {
    const __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
  }
};
template <> struct Pair<__nv_bfloat16> {
  static constexpr uint32_t fmt = 1;
  static __device__ __forceinline__ uint32_t pack(float lo, float hi) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
  }
};

// The MMAs below are issued by the lane whose `leader` is set; every lane of
// the warp executes the statement, so operands stay warp-uniform.
// Descriptors are passed as their low word (address and leading offset), which
// advances by one 32-bit addition per step, and the constant high word.
// D[tmem] (+)= A[tmem] * B[smem]: A holds 16-bit pairs, row = lane, two
// consecutive k per column.
__device__ __forceinline__ void mma_ts(uint32_t leader, uint32_t d, uint32_t a, uint32_t b_lo, uint32_t b_hi,
                                       uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t.reg .b64 db;\n\t"
      "mov.b64 db, {%2, %3};\n\t"
      "setp.ne.b32 p, %5, 0;\n\t"
      "setp.ne.b32 q, %6, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], db, %4, p;\n\t}"
      ::"r"(d), "r"(a), "r"(b_lo), "r"(b_hi), "r"(idesc), "r"(accumulate), "r"(leader) : "memory");
}
// D[tmem] (+)= A[smem] * B[smem]^T, both K-major (one high word)
__device__ __forceinline__ void mma_ss(uint32_t leader, uint32_t d, uint32_t a_lo, uint32_t b_lo, uint32_t hi,
                                       uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t.reg .b64 da, db;\n\t"
      "mov.b64 da, {%1, %3};\n\t"
      "mov.b64 db, {%2, %3};\n\t"
      "setp.ne.b32 p, %5, 0;\n\t"
      "setp.ne.b32 q, %6, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %4, p;\n\t}"
      ::"r"(d), "r"(a_lo), "r"(b_lo), "r"(hi), "r"(idesc), "r"(accumulate), "r"(leader) : "memory");
}
__device__ __forceinline__ uint32_t lo32(uint64_t v) { return (uint32_t)v; }
__device__ __forceinline__ uint32_t hi32(uint64_t v) { return (uint32_t)(v >> 32); }
__device__ __forceinline__ void commit(uint32_t leader, uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .pred q;\n\t"
      "setp.ne.b32 q, %1, 0;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}"
      ::"r"(smem_u32(bar)), "r"(leader) : "memory");
}
// A value that is the same in every lane, in a uniform register.
__device__ __forceinline__ uint32_t uniform(uint32_t v) { return __reduce_max_sync(0xffffffffu, v); }

// B operand with its N index contiguous (MN-major).
constexpr uint32_t kBTransposed = 1u << 16;

#define EQLIN_R8(r, o) "=r"(r[o]), "=r"(r[o + 1]), "=r"(r[o + 2]), "=r"(r[o + 3]), "=r"(r[o + 4]), "=r"(r[o + 5]), "=r"(r[o + 6]), "=r"(r[o + 7])
#define EQLIN_T8(r, o) "+r"(r[o]), "+r"(r[o + 1]), "+r"(r[o + 2]), "+r"(r[o + 3]), "+r"(r[o + 4]), "+r"(r[o + 5]), "+r"(r[o + 6]), "+r"(r[o + 7])
// 32 lanes x 32 bits, 32 consecutive columns per thread.
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : EQLIN_R8(r, 0), EQLIN_R8(r, 8), EQLIN_R8(r, 16), EQLIN_R8(r, 24) : "r"(taddr));
}
// After tmem_wait_ld: keeps every use of the loaded registers behind the wait.
__device__ __forceinline__ void tie32(uint32_t* r) {
  asm volatile("" : EQLIN_T8(r, 0), EQLIN_T8(r, 8), EQLIN_T8(r, 16), EQLIN_T8(r, 24));
}
__device__ __forceinline__ void tie16(uint32_t* r) { asm volatile("" : EQLIN_T8(r, 0), EQLIN_T8(r, 8)); }

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// TILE_ROWS rows from token r0 on, all panels, announced on `bar` by the copy's
// bytes (call from one lane, which arrives on `bar` afterwards).
template <int DP, int TILE_ROWS>
__device__ __forceinline__ void tma_rows(void* dst, const CUtensorMap* map, int head, int r0, uint64_t* bar) {
#pragma unroll
  for (int pn = 0; pn < DP / 64; ++pn)
    tma_load_3d(static_cast<uint8_t*>(dst) + pn * TILE_ROWS * 128, map, pn * 64, head, r0, bar);
}
__device__ __forceinline__ void expect_bytes(uint64_t* bar, uint32_t bytes) {
  asm volatile("mbarrier.expect_tx.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(smem_u32(bar)), "r"(bytes) : "memory");
}

// What a tile needs beside its operands, one row per lane and round: negated
// positions [axes][rows] and, for moving queries, -lse (base 2) and delta.  The
// loads are issued a tile ahead and stored when the slot is free.
template <int AXES, bool STAT, int TILE_ROWS> struct Side {
  static constexpr int R = TILE_ROWS / 32;
  float pos[AXES ? AXES * R : 1], lse[STAT ? R : 1], delta[STAT ? R : 1];
  __device__ __forceinline__ void fetch(const Params& p, int head, int r0, int hi, int lane) {
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const int r = r0 + lane + 32 * i;
      const bool on = r < hi;
#pragma unroll
      for (int a = 0; a < AXES; ++a) pos[a * R + i] = on ? p.pos[(int64_t)r * AXES + a] : 0.f;
      if (STAT) {
        lse[i] = on ? p.lse[(int64_t)head * p.N + r] : INFINITY;
        delta[i] = on ? p.delta[(int64_t)head * p.N + r] : 0.f;
      }
    }
  }
  // delta's largest magnitude, behind the rest
  __device__ __forceinline__ void store_top(float* dst, int lane) const {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < R; ++i) m = max(m, __float_as_uint(fabsf(delta[i])));   // ordered as the floats are
    m = __reduce_max_sync(0xffffffffu, m);
    if (lane == 0) dst[(kMaxAxes + 2) * TILE_ROWS] = __uint_as_float(m);
  }
  __device__ __forceinline__ void store(float* dst, float up, int lane) const {
#pragma unroll
    for (int i = 0; i < R; ++i) {
#pragma unroll
      for (int a = 0; a < AXES; ++a) dst[a * TILE_ROWS + lane + 32 * i] = -pos[a * R + i];
      if (STAT) {
        // past the document's end lse is +inf: P = 0 there
        dst[kMaxAxes * TILE_ROWS + lane + 32 * i] = fmaf(lse[i], -kLog2e, up);
        dst[(kMaxAxes + 1) * TILE_ROWS + lane + 32 * i] = delta[i];
      }
    }
  }
};

// Moving tiles whose last rows are to be cleared once the copy has landed: the
// loading warp settles them when it has nothing else to issue, at the latest
// when three wait.  land[slot] counts the copy's bytes, full[slot] the warp's
// 32 arrivals.
struct Tails {
  int count = 0;
  uint32_t phases = 0;    // of land, one bit per slot
  uint32_t slot[3];
  int from[3];            // first row to clear
};
// What every wait of a role needs to know.
struct Waits {
  uint32_t limit;
  volatile int* abort_flag;
  int* err;
  __device__ __forceinline__ bool on(uint64_t* bar, uint32_t parity, uint32_t where, uint32_t iter) const {
    return wwait_all(bar, parity, limit, abort_flag, err, where, iter);
  }
};
// Settle the oldest `n` of the waiting tiles (NT tiles of TILE_ROWS rows per slot).
template <int DP, int TILE_ROWS, int NT>
__device__ __forceinline__ bool settle(Tails& q, int n, uint8_t* ring, uint64_t* land, uint64_t* full, const Waits& w,
                                       uint32_t where, int lane) {
  constexpr int TILE = DP / 64 * TILE_ROWS * 128;
  for (; n > 0; --n) {
    const uint32_t slot = q.slot[0];
    const int from = q.from[0], rows = ((from + 15) & ~15) - from;
    if (!w.on(land + slot, (q.phases >> slot) & 1, where, slot)) return false;
    q.phases ^= 1u << slot;
    uint8_t* base = ring + slot * NT * TILE + from * 128;
#pragma unroll
    for (int t = 0; t < NT * DP / 64; ++t)           // panels of the slot
      for (int i = lane; i < rows * 8; i += 32)
        *reinterpret_cast<uint4*>(base + t * TILE_ROWS * 128 + i * 16) = make_uint4(0, 0, 0, 0);
    fence_proxy_async_smem();
    mbar_arrive(full + slot);
    q.slot[0] = q.slot[1];
    q.from[0] = q.from[1];
    q.slot[1] = q.slot[2];
    q.from[1] = q.from[2];
    --q.count;
  }
  return true;
}
// Start a moving tile's copies on slot `slot`, which is free; maps and heads of its NT
// tiles, token c0, nc rows of the document.  What the lanes stored for the
// tile before is announced with it.
template <int DP, int TILE_ROWS, int NT>
__device__ __forceinline__ bool bring(Tails& q, uint32_t slot, uint8_t* ring, uint64_t* land, uint64_t* full,
                                      const CUtensorMap* map, int head, int c0, int nc, const Waits& w, uint32_t where,
                                      int lane) {
  constexpr int TILE = DP / 64 * TILE_ROWS * 128;
  const bool whole = (nc & 15) == 0;
  uint64_t* bar = whole ? full + slot : land + slot;
  if (lane == 0) {
    if (whole) expect_bytes(bar, NT * TILE);
    else mbar_arrive_expect_tx(bar, NT * TILE);
#pragma unroll
    for (int t = 0; t < NT; ++t) tma_rows<DP, TILE_ROWS>(ring + slot * NT * TILE + t * TILE, map + t, head, c0, bar);
  }
  if (whole) {
    mbar_arrive(bar);
    return true;
  }
#pragma unroll
  for (int i = 0; i < 3; ++i)
    if (i == q.count) {
      q.slot[i] = slot;
      q.from[i] = nc;
    }
  return ++q.count < 3 || settle<DP, TILE_ROWS, NT>(q, 1, ring, land, full, w, where, lane);
}
// Before writing into a slot: wait until it is free, settling what waits first
// if that takes time.  Uniform over the warp; false on abort.
template <int DP, int TILE_ROWS, int NT>
__device__ __forceinline__ bool claim(Tails& q, uint64_t* empty, uint32_t parity, uint8_t* ring, uint64_t* land,
                                      uint64_t* full, const Waits& w, uint32_t where, uint32_t iter, int lane) {
  if (__all_sync(0xffffffffu, mbar_test_wait(empty, parity))) return true;
  return settle<DP, TILE_ROWS, NT>(q, q.count, ring, land, full, w, where, lane) && w.on(empty, parity, where, iter);
}

// No copy of this block may be in flight when it exits: wait for those of the
// tiles not settled (after a wait ran out; nothing reads them any more), the
// last `slots` tiles of the ring and the last own tile.
__device__ __forceinline__ void drain_loads(Tails& q, uint64_t* land, uint64_t* own_full, uint32_t own_count,
                                            uint64_t* full, uint32_t items, uint32_t slots) {
  for (int i = 0; i < q.count; ++i) {
    mbar_wait(land + q.slot[i], (q.phases >> q.slot[i]) & 1, kDefaultWaitLimit);
    mbar_arrive(full + q.slot[i]);
  }
  for (uint32_t k = items > slots ? items - slots : 0; k < items; ++k)
    mbar_wait(full + k % slots, (k / slots) & 1, kDefaultWaitLimit);
  if (own_count) mbar_wait(own_full, (own_count - 1) & 1, kDefaultWaitLimit);
}

// A warp's 32 rows x 32 features (16 packed words per lane, lane = row) into
// global rows: through 2 KB of shared memory, so that four lanes write 64
// consecutive bytes of a row.  Lanes writing 16 bytes of 32 rows each would
// take the load/store unit a cycle per row and store.  Chunk j of row r lies
// at chunk j ^ (r / 2 % 4) of its 64 bytes: no bank conflicts either way.
constexpr int STAGE = 2048;
template <typename E>
__device__ __forceinline__ void store32(uint8_t* stage, const uint32_t* words, E* out, int64_t stride, int rows, int col,
                                        int D, int lane) {
#pragma unroll
  for (int j = 0; j < 4; ++j)
    *reinterpret_cast<uint4*>(stage + lane * 64 + ((j ^ ((lane >> 1) & 3)) << 4)) =
        make_uint4(words[4 * j], words[4 * j + 1], words[4 * j + 2], words[4 * j + 3]);
  __syncwarp();
  const int j = lane & 3;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = 8 * i + (lane >> 2);
    const uint4 v = *reinterpret_cast<const uint4*>(stage + r * 64 + ((j ^ ((r >> 1) & 3)) << 4));
    if (r < rows && col + j * 8 < D) *reinterpret_cast<uint4*>(out + r * stride + col + j * 8) = v;
  }
  __syncwarp();
}

// Dot products of a warp's 32 rows of two tensors, one result per lane: eight
// lanes read 128 consecutive bytes of a row.
template <typename E>
__device__ __forceinline__ float row_dots(const E* a, int64_t as, const E* b, int64_t bs, int rows, int D, int lane) {
  float mine = 0.f, d[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) d[i] = 0.f;
  for (int c = (lane & 7) * 8; c < ((D + 63) & ~63); c += 64) {
    uint4 u[8], v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int r = 4 * i + (lane >> 3);
      u[i] = v[i] = make_uint4(0, 0, 0, 0);
      if (r < rows && c < D) {
        u[i] = *reinterpret_cast<const uint4*>(a + r * as + c);
        v[i] = *reinterpret_cast<const uint4*>(b + r * bs + c);
      }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const E* x = reinterpret_cast<const E*>(&u[i]);
      const E* y = reinterpret_cast<const E*>(&v[i]);
#pragma unroll
      for (int k = 0; k < 8; ++k) d[i] = fmaf(Elem<E>::to_f(x[k]), Elem<E>::to_f(y[k]), d[i]);
    }
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    d[i] += __shfl_xor_sync(0xffffffffu, d[i], 1);
    d[i] += __shfl_xor_sync(0xffffffffu, d[i], 2);
    d[i] += __shfl_xor_sync(0xffffffffu, d[i], 4);
    const float x = __shfl_sync(0xffffffffu, d[i], (lane & 3) * 8);
    if ((lane >> 2) == i) mine = x;
  }
  return mine;
}

// Scores in units of the raw product q.k (the softmax multiplies by scale2 =
// scale log2 e): x = cap/scale tanh(raw scale/cap) - slope/scale distance.
struct Score {
  float scale2;
  float in, out;          // scale / cap, cap / scale
  float cap2, slope2;     // cap log2 e, slope log2 e
  float twoin;            // 2 log2 e scale / cap: e^{2u/cap} = 2^(raw twoin)
  float slope;            // slope / scale
};
__device__ __forceinline__ Score score_of(const Params& p, int head) {
  Score s;
  s.scale2 = p.scale * kLog2e;
  s.in = p.cap > 0.f ? p.scale / p.cap : 0.f;
  s.out = p.cap > 0.f ? p.cap / p.scale : 0.f;
  s.twoin = 2.f * kLog2e * s.in;
  s.cap2 = p.cap * kLog2e;
  s.slope = p.axes ? p.slopes[head] / p.scale : 0.f;
  s.slope2 = p.axes ? p.slopes[head] * kLog2e : 0.f;
  return s;
}

// tanh, for two arguments.  Where all of a warp's arguments are small (|x| <=
// kSmall, the usual case below a cap) an odd polynomial, x q(x^2): 2.8e-8 off at
// most, the FP32 roundings apart (with them 4.5e-7 relative), which under a cap of
// 30 is less than the FP32 step of a score of 8 to 16 (coefficients: a weighted
// least-squares fit of tanh(x)/x refined to equal ripple), 3 instructions per
// score on the FMA pipes.  Otherwise 1 - 2 / (1 + e^{2x}) for the arguments that
// are not: a few 2^-24 off in absolute terms, which cap times over would be too
// much for a small one (under a cap of 1e6 a score of 1 would be off by 0.2).  The
// forward makes the difference above kLargeCap alone: at that cap it is 6e-5 of a
// score, an eighth of f16's half step in P (12544 tokens, 6 heads of 64, scores of
// spread 2 under a cap of 3: 1.18 ms, 1.67 below it, too; the backward takes 2.22
// ms, 2.09 without the difference, which is not worth a third form there).  The
// two MUFU operations (8 cycles of a scheduler each) for every score would be two
// thirds of the softmax's time.  tanh.approx would be one, but is only good to
// 2^-11.
constexpr float kSmall = 0.6f, kLargeCap = 256.f;
__device__ __forceinline__ uint64_t q_small2(uint64_t x) {      // tanh(x) / x
  const uint64_t z = mul2(x, x);
  uint64_t q = pk2(0.01497695967555046f, 0.01497695967555046f);
  q = fma2(q, z, pk2(-0.051696743816137314f, -0.051696743816137314f));
  q = fma2(q, z, pk2(0.13299210369586945f, 0.13299210369586945f));
  q = fma2(q, z, pk2(-0.33331209421157837f, -0.33331209421157837f));
  return fma2(q, z, pk2(0.9999996423721313f, 0.9999996423721313f));
}
__device__ __forceinline__ float tanh_large(float raw, const Score& s) {
  return fmaf(-2.f, rcp(1.f + ex2(raw * s.twoin)), 1.f);
}
__device__ __forceinline__ void tanh_any2(float& a, float& b, const Score& s) {      // raw scores in
  const uint64_t x = mul2(pk2(a, b), pk2(s.in, s.in));
  float xa, xb, pa, pb;
  unpk2(x, xa, xb);
  unpk2(mul2(x, q_small2(x)), pa, pb);
  a = fabsf(xa) <= kSmall ? pa : tanh_large(a, s);
  b = fabsf(xb) <= kSmall ? pb : tanh_large(b, s);
}
// Are all of the warp's raw scores, N per row, small enough for the polynomial?
// Only live rows count: results must not depend on what lies behind a document.
template <int N>
__device__ __forceinline__ bool all_small(const float* raw, const Score& s, bool live) {
  float a = fabsf(raw[0]), b = fabsf(raw[1]);
#pragma unroll
  for (int i = 2; i < N; i += 2) {
    a = fmaxf(a, fabsf(raw[i]));
    b = fmaxf(b, fabsf(raw[i + 1]));
  }
  return __all_sync(0xffffffffu, !live || fmaxf(a, b) * s.in <= kSmall);   // a NaN survives either way
}

// City-block distances of four moving rows c0 .. c0+3 (their positions are
// stored negated) from the own row.
template <int AXES, int TILE_ROWS>
__device__ __forceinline__ void distances(const float* pos, int c0, const float* own, float (&d)[4]) {
#pragma unroll
  for (int a = 0; a < AXES; ++a) {
    const ulonglong2 v = *reinterpret_cast<const ulonglong2*>(pos + a * TILE_ROWS + c0);
    const uint64_t o = pk2(own[a], own[a]);
    float e[4];
    unpk2(add2(o, v.x), e[0], e[1]);
    unpk2(add2(o, v.y), e[2], e[3]);
#pragma unroll
    for (int k = 0; k < 4; ++k) d[k] = a == 0 ? fabsf(e[k]) : d[k] + fabsf(e[k]);
  }
}

// Cap and bias of a row's 32 raw scores, in place; `small` as all_small says.
template <int AXES, bool CAP, int TILE_ROWS>
__device__ __forceinline__ void transform32(float* s, const float* pos, int c0, const float* own, const Score& sc,
                                            bool small) {
  if constexpr (CAP) {
    if (small) {
      const uint64_t in = pk2(sc.in, sc.in);
#pragma unroll
      for (int i = 0; i < 32; i += 2) {
        const uint64_t v = pk2(s[i], s[i + 1]);
        unpk2(mul2(v, q_small2(mul2(v, in))), s[i], s[i + 1]);
      }
    } else if (sc.cap2 <= kLargeCap * kLog2e) {
#pragma unroll
      for (int i = 0; i < 32; ++i) s[i] = sc.out * tanh_large(s[i], sc);
    } else {
#pragma unroll
      for (int i = 0; i < 32; i += 2) {
        tanh_any2(s[i], s[i + 1], sc);
        s[i] *= sc.out;
        s[i + 1] *= sc.out;
      }
    }
  }
  if constexpr (AXES > 0) {
    const uint64_t slope = pk2(-sc.slope, -sc.slope);
#pragma unroll
    for (int i = 0; i < 32; i += 4) {
      float d[4];
      distances<AXES, TILE_ROWS>(pos, c0 + i, own, d);
      unpk2(fma2(slope, pk2(d[0], d[1]), pk2(s[i], s[i + 1])), s[i], s[i + 1]);
      unpk2(fma2(slope, pk2(d[2], d[3]), pk2(s[i + 2], s[i + 3])), s[i + 2], s[i + 3]);
    }
  }
}

// ------------------------------------------------------------------- launch

struct Maps {
  CUtensorMap m[4];
};

// Make the current device's context current in this host thread, too: one that
// has only selected the device (an autograd worker, say) may not have it yet,
// and encoding a tensor map needs it.
inline cudaError_t enter_context() {
  int dev = 0;
  const cudaError_t e = cudaGetDevice(&dev);
  return e != cudaSuccess ? e : cudaSetDevice(dev);
}

// A map over [N][heads][D] for boxes of 64 features x one head x `rows` tokens.
inline cudaError_t make_map(CUtensorMap* map, const void* base, uint32_t fmt, const Params& p, int heads, int64_t stride,
                            int rows) {
  const auto encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(tensor_map_encoder());
  if (!encode) return cudaErrorNotSupported;
  const cuuint64_t dims[3] = {(cuuint64_t)p.D, (cuuint64_t)heads, (cuuint64_t)p.N};
  const cuuint64_t strides[2] = {(cuuint64_t)p.D * 2, (cuuint64_t)stride * 2};
  const cuuint32_t box[3] = {64, 1, (cuuint32_t)rows};       // what lies outside the tensor reads as zero
  const cuuint32_t ones[3] = {1, 1, 1};
  const CUresult r =
      encode(map, fmt ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, const_cast<void*>(base),
             dims, strides, box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

// One own tile: rows from `first` on of the document [lo, hi), first < hi.
struct Tile {
  int head, lo, hi, first;
};

// The own tiles of a block, in the order in which every role meets them.
//
// Documents of one length: item = (document, head, tile), tiles fastest, so
// that blocks which share keys run together; as many blocks as fit the SMs
// walk all items, and one item's loads run under the previous one's products
// and stores.
//
// Packed documents: item = (slot, head), a slot being 128 tokens of the packed
// sequence, a block per item.  Its own tiles are those that start in the slot:
// at most one of a document that began earlier, and the first one of every
// document that begins there.  So the grid is as large as the work, whatever
// the lengths are, and short documents share a block.  Warp 0 lists them in
// shared memory, finding the first document by a search over the offsets, 32
// ways at a time.  (The roles' own loops stay free of data-dependent control
// flow: with it the compiler keeps the MMA warp's descriptors out of uniform
// registers, a tenth of the backward's time.)  Offsets are forced into [0, N]
// and into order, so that wrong ones cannot lead out of the tensors.
constexpr int kListInts = 1 + 3 * (ROWS + 1);        // count; lo, hi, first of each
__device__ __forceinline__ int offset_at(const Params& p, int64_t i) { return min(max(p.offsets[i], 0), (int)p.N); }

// First of the docs + 1 offsets that is at least `from`; for a whole warp.
__device__ __forceinline__ int64_t first_offset(const Params& p, int from) {
  const int lane = threadIdx.x & 31;
  int64_t l = 0, r = p.docs + 1;
  while (l < r) {
    const int64_t step = (r - l + 31) / 32, at = l + lane * step;
    const bool below = at < r && p.offsets[at] < from;
    const int c = __popc(__ballot_sync(0xffffffffu, below));
    if (c == 0) break;
    const int64_t next = l + c * step;               // not below, if there is one
    l += (c - 1) * step + 1;
    if (next < r) r = next;
  }
  return l;
}
// Warp 0: the own tiles that start in tokens [from, to).
__device__ __forceinline__ void list_tiles(const Params& p, int from, int to, int* list) {
  const int lane = threadIdx.x & 31;
  int64_t doc = first_offset(p, from);
  int n = 0;
  if (doc >= 1 && doc <= p.docs) {                   // the document that began before the slot
    const int lo = offset_at(p, doc - 1), hi = max(offset_at(p, doc), lo);
    const int first = lo + (from - lo + ROWS - 1) / ROWS * ROWS;
    if (first >= from && first < to && first < hi) {
      if (lane == 0) {
        list[1] = lo;
        list[2] = hi;
        list[3] = first;
      }
      n = 1;
    }
  }
  for (; doc < p.docs; doc += 32) {
    const int64_t d = doc + lane;
    const int lo = d < p.docs ? offset_at(p, d) : to, hi = d < p.docs ? max(offset_at(p, d + 1), lo) : to;
    const bool inside = lo >= from && lo < to;
    const uint32_t mask = __ballot_sync(0xffffffffu, inside && hi > lo);
    const int at = n + __popc(mask & ((1u << lane) - 1u));
    if (inside && hi > lo && at <= ROWS) {           // at most one tile a token, unless offsets are out of order
      list[1 + 3 * at] = lo;
      list[2 + 3 * at] = hi;
      list[3 + 3 * at] = lo;
    }
    n = min(n + __popc(mask), ROWS + 1);
    if (!__all_sync(0xffffffffu, inside)) break;
  }
  if (lane == 0) list[0] = n;
}

// Before anything else, by the whole block: the number of its own tiles.
// Packed calls also clear the rows of the slot that no document holds.
template <typename F>
__device__ __forceinline__ uint32_t begin(const Params& p, int heads, int* list, F&& clear) {
  if (!p.offsets) return (p.items - blockIdx.x + gridDim.x - 1) / gridDim.x;
  const int slot = (int)(blockIdx.x / (uint32_t)heads), head = (int)(blockIdx.x - (uint32_t)slot * (uint32_t)heads);
  const int from = slot * ROWS, to = min(from + ROWS, (int)p.N);
  const int a = offset_at(p, 0), b = max(offset_at(p, p.docs), a);
  for (int r = from; r < min(to, a); ++r) clear(head, (int64_t)r);
  for (int r = max(from, b); r < to; ++r) clear(head, (int64_t)r);
  if (threadIdx.x < 32) list_tiles(p, from, to, list);
  __syncthreads();
  return uniform((uint32_t)list[0]);
}
// Own tile i of the block, in warp-uniform values.
__device__ __forceinline__ Tile tile_at(const Params& p, int heads, const int* list, uint32_t i) {
  uint32_t head, lo, hi, first;
  if (p.offsets) {
    head = blockIdx.x % (uint32_t)heads;
    lo = (uint32_t)list[1 + 3 * i];
    hi = (uint32_t)list[2 + 3 * i];
    first = (uint32_t)list[3 + 3 * i];
  } else {
    const uint32_t work = blockIdx.x + i * gridDim.x, rest = work / (uint32_t)p.hint, d = rest / (uint32_t)heads;
    head = rest - d * (uint32_t)heads;
    lo = d * (uint32_t)p.len;
    hi = lo + (uint32_t)p.len;
    first = lo + (work - rest * (uint32_t)p.hint) * ROWS;
  }
  return Tile{(int)uniform(head), (int)uniform(lo), (int)uniform(hi), (int)uniform(first)};
}

inline cudaError_t launch_rows(void (*k)(Params, Maps), int smem, Params p, const Maps& maps, int heads, int threads,
                               int blocks_per_sm, cudaStream_t st) {
  // tiles of a document, or slots of the packed sequence
  p.hint = (int)(((p.offsets ? p.N : p.len) + ROWS - 1) / ROWS);
  const int64_t items = (p.offsets ? 1 : p.docs) * heads * (int64_t)p.hint;
  if (items == 0) return cudaSuccess;
  if (items > 0x7fffffff) return cudaErrorInvalidValue;
  p.items = (uint32_t)items;
  uint32_t grid = p.items;
  if (!p.offsets) {
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    const uint32_t most = (uint32_t)(sms * blocks_per_sm);
    if (grid > most) grid = most;
  }
  cudaError_t e = set_smem_limit(reinterpret_cast<const void*>(k), smem);
  if (e == cudaSuccess) e = launch_pdl(k, dim3(grid), dim3(threads), (size_t)smem, st, p, maps);
  if (e == cudaSuccess) count_launches(1);
  return e;
}

}  // namespace attn_tc
}  // namespace eqlin
