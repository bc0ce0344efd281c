// eqlin_attn_tc.cuh -- parts shared by the tensor-core attention kernels.
//
// All of them have one shape: 128 rows stay ("own" rows: queries, or keys in
// the kernel for dk and dv), the other side passes by in tiles of up to 128
// ("moving" rows).  A block is six warps:
//
//   warps 0-3   one thread per own row: scores out of TMEM, softmax (or its
//               gradient) in FP32 registers, 16-bit probabilities back into
//               TMEM as the next product's A operand
//   warp 4      issues the MMAs: the whole warp runs the loops, so that
//               descriptors stay in uniform registers, and one lane's predicate
//               is set on the instruction itself; the warp allocates TMEM
//   warp 5      brings tiles into shared memory: whole tiles with TMA (a 3D map
//               over features, heads, tokens: features past D read as zero), the
//               last, partial tile of a document with 16-byte asynchronous
//               copies that write zeros past its end.  A neighbour's rows must
//               not be in the tile at all: a product with P = 0 would spread
//               their infinities and NaNs.
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
// D[tmem] (+)= A[tmem] * B[smem]: A holds 16-bit pairs, row = lane, two
// consecutive k per column.
__device__ __forceinline__ void mma_ts(uint32_t leader, uint32_t d, uint32_t a, uint64_t b_desc, uint32_t idesc,
                                       uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "setp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}"
      ::"r"(d), "r"(a), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"(leader) : "memory");
}
// D[tmem] (+)= A[smem] * B[smem]^T
__device__ __forceinline__ void mma_ss(uint32_t leader, uint32_t d, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                       uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "setp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}"
      ::"r"(d), "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"(leader) : "memory");
}
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

// Two FP32 operations per instruction.
__device__ __forceinline__ uint64_t pk2(float a, float b) {
  uint64_t v;
  asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(a), "f"(b));
  return v;
}
__device__ __forceinline__ void unpk2(uint64_t v, float& a, float& b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v)); }
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t v;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(v) : "l"(a), "l"(b));
  return v;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t v;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(v) : "l"(a), "l"(b));
  return v;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t v;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(v) : "l"(a), "l"(b), "l"(c));
  return v;
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// One warp copies `rows` rows (<= TILE_ROWS) from token r0 on of one head into the
// panels at dst; rows at or past `hi`, and features at or past D, read as zero.
// chunks: 16-byte chunks of a row that any product reads (ceil(D / 16) * 2).
template <int DP, typename E, int TILE_ROWS = ROWS>
__device__ __forceinline__ void load_rows(uint32_t dst, const void* src, int64_t stride, int64_t head_off, int r0,
                                          int hi, int rows, int D, int chunks, int lane) {
  const int sub = lane >> 3, ch0 = lane & 7;
  const char* base = reinterpret_cast<const char*>(static_cast<const E*>(src) + head_off);
  const int64_t step = stride * (int64_t)sizeof(E);
  const int left = min(hi - r0, TILE_ROWS);
#pragma unroll
  for (int pn = 0; pn < DP / 64; ++pn) {
    const int ch = pn * 8 + ch0;
    if (ch >= chunks) continue;
    const bool live_ch = ch * 8 < D;
    const char* from = base + (int64_t)(r0 + sub) * step + ch * 16;
    const uint32_t to = dst + pn * TILE_ROWS * 128;
#pragma unroll 4
    for (int r = sub; r < rows; r += 4, from += 4 * step) {
      const bool on = live_ch && r < left;
      cp_async16(to + r * 128 + ((ch0 ^ (r & 7)) << 4), on ? from : base, on ? 16u : 0u);
    }
  }
}

// Whole tiles: TILE_ROWS rows from token r0 on, all panels, announced on `bar`
// by the copy's bytes (call from one lane, which arrives on `bar` afterwards).
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
// positions [axes][128] and, for moving queries, lse (base 2) and delta.  The
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
  __device__ __forceinline__ void store(float* dst, float up, float down, int lane) const {
#pragma unroll
    for (int i = 0; i < R; ++i) {
#pragma unroll
      for (int a = 0; a < AXES; ++a) dst[a * ROWS + lane + 32 * i] = -pos[a * R + i];
      if (STAT) {
        // past the document's end +inf: P = 0 there
        dst[kMaxAxes * ROWS + lane + 32 * i] = fmaf(lse[i], kLog2e, -up);
        dst[kMaxAxes * ROWS + ROWS + lane + 32 * i] = delta[i] * down;
      }
    }
  }
};

// The loading warp's asynchronous copies that are not yet announced: a tile is
// announced (32 arrivals) once its copies have landed and been made visible to
// the tensor core, at the latest when the warp has nothing else to issue.
struct Pending {
  int count = 0;
  uint64_t* bar[3];
};
__device__ __forceinline__ void announce_all(Pending& q) {
  if (!q.count) return;
  cp_async_wait<0>();
  fence_proxy_async_smem();
#pragma unroll
  for (int i = 0; i < 3; ++i)
    if (i < q.count) mbar_arrive(q.bar[i]);
  q.count = 0;
}
// After an issue and its commit: at most two groups stay in flight unannounced.
__device__ __forceinline__ void announce_later(Pending& q, uint64_t* bar) {
#pragma unroll
  for (int i = 0; i < 3; ++i)
    if (i == q.count) q.bar[i] = bar;
  if (++q.count == 3) {
    cp_async_wait<2>();
    fence_proxy_async_smem();
    mbar_arrive(q.bar[0]);
    q.bar[0] = q.bar[1];
    q.bar[1] = q.bar[2];
    q.count = 2;
  }
}
// Before writing into a slot: wait until it is free, announcing what is in
// flight first if that takes time.  Uniform over the warp; false on abort.
__device__ __forceinline__ bool claim(Pending& q, uint64_t* empty, uint32_t parity, uint32_t limit,
                                      volatile int* abort_flag, int* err, uint32_t where, uint32_t iter) {
  if (__all_sync(0xffffffffu, mbar_test_wait(empty, parity))) return true;
  announce_all(q);
  return wwait_all(empty, parity, limit, abort_flag, err, where, iter);
}

// No copy of this block may be in flight when it exits: wait for the last
// `slots` tiles of the ring and the last own tile (long done unless a wait ran
// out somewhere).
__device__ __forceinline__ void drain_loads(uint64_t* own_full, uint32_t own_count, uint64_t* full, uint32_t items,
                                            uint32_t slots) {
  for (uint32_t k = items > slots ? items - slots : 0; k < items; ++k)
    mbar_wait(full + k % slots, (k / slots) & 1, kDefaultWaitLimit);
  if (own_count) mbar_wait(own_full, (own_count - 1) & 1, kDefaultWaitLimit);
}

// Scores in units of the raw product q.k (the softmax multiplies by scale2 =
// scale log2 e): x = cap/scale tanh(raw scale/cap) - slope/scale distance.
struct Score {
  float scale2;
  float in, out;          // scale / cap, cap / scale
  float twoin;            // 2 log2 e scale / cap: e^{2u/cap} = 2^(raw twoin)
  float slope;            // slope / scale
};
__device__ __forceinline__ Score score_of(const Params& p, int head) {
  Score s;
  s.scale2 = p.scale * kLog2e;
  s.in = p.cap > 0.f ? p.scale / p.cap : 0.f;
  s.out = p.cap > 0.f ? p.cap / p.scale : 0.f;
  s.twoin = 2.f * kLog2e * s.in;
  s.slope = p.axes ? p.slopes[head] / p.scale : 0.f;
  return s;
}

// tanh, for two arguments.  Where all of a warp's arguments are small (|x| <=
// kSmall, the usual case below a cap) an odd polynomial, x q(x^2): 4e-9 off at
// most (coefficients: a weighted least-squares fit of tanh(x)/x refined to
// equal ripple), 3.5 instructions per score on the FMA pipes.  Otherwise
// 1 - 2 / (1 + e^{2x}), a few 2^-24 off in absolute terms everywhere, which is
// what a score needs; its two MUFU operations (8 cycles of a scheduler each)
// would otherwise be two thirds of the softmax's time.  tanh.approx would be
// one, but is only good to 2^-11.
constexpr float kSmall = 0.7f;
__device__ __forceinline__ uint64_t q_small2(uint64_t x) {      // tanh(x) / x
  const uint64_t z = mul2(x, x);
  uint64_t q = pk2(-0.004874242004007101f, -0.004874242004007101f);
  q = fma2(q, z, pk2(0.01973520778119564f, 0.01973520778119564f));
  q = fma2(q, z, pk2(-0.053383808583021164f, -0.053383808583021164f));
  q = fma2(q, z, pk2(0.1332535296678543f, 0.1332535296678543f));
  q = fma2(q, z, pk2(-0.33332860469818115f, -0.33332860469818115f));
  return fma2(q, z, pk2(0.9999999403953552f, 0.9999999403953552f));
}
__device__ __forceinline__ float tanh_any(float raw, const Score& s) {
  return fmaf(-2.f, rcp(1.f + ex2(raw * s.twoin)), 1.f);
}
// Are all the warp's 32 x 32 raw scores small enough for the polynomial?
__device__ __forceinline__ bool all_small(const float* raw, const Score& s) {
  float a = fabsf(raw[0]), b = fabsf(raw[1]);
#pragma unroll
  for (int i = 2; i < 32; i += 2) {
    a = fmaxf(a, fabsf(raw[i]));
    b = fmaxf(b, fabsf(raw[i + 1]));
  }
  return __all_sync(0xffffffffu, fmaxf(a, b) * s.in <= kSmall);   // a NaN is left out by fmaxf and survives either way
}

// City-block distances of four moving rows c0 .. c0+3 (their positions are
// stored negated) from the own row.
template <int AXES>
__device__ __forceinline__ void distances(const float* pos, int c0, const float* own, float (&d)[4]) {
#pragma unroll
  for (int a = 0; a < AXES; ++a) {
    const ulonglong2 v = *reinterpret_cast<const ulonglong2*>(pos + a * ROWS + c0);
    const uint64_t o = pk2(own[a], own[a]);
    float e[4];
    unpk2(add2(o, v.x), e[0], e[1]);
    unpk2(add2(o, v.y), e[2], e[3]);
#pragma unroll
    for (int k = 0; k < 4; ++k) d[k] = a == 0 ? fabsf(e[k]) : d[k] + fabsf(e[k]);
  }
}

// Cap and bias of a row's 32 raw scores, in place; a and b pairs.
template <int AXES, bool CAP>
__device__ __forceinline__ void transform32(float* s, const float* pos, int c0, const float* own, const Score& sc) {
  if constexpr (CAP) {
    if (all_small(s, sc)) {
      const uint64_t in = pk2(sc.in, sc.in);
#pragma unroll
      for (int i = 0; i < 32; i += 2) {
        const uint64_t v = pk2(s[i], s[i + 1]);
        unpk2(mul2(v, q_small2(mul2(v, in))), s[i], s[i + 1]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 32; ++i) s[i] = sc.out * tanh_any(s[i], sc);
    }
  }
  if constexpr (AXES > 0) {
    const uint64_t slope = pk2(-sc.slope, -sc.slope);
#pragma unroll
    for (int i = 0; i < 32; i += 4) {
      float d[4];
      distances<AXES>(pos, c0 + i, own, d);
      unpk2(fma2(slope, pk2(d[0], d[1]), pk2(s[i], s[i + 1])), s[i], s[i + 1]);
      unpk2(fma2(slope, pk2(d[2], d[3]), pk2(s[i + 2], s[i + 3])), s[i + 2], s[i + 3]);
    }
  }
}

// ------------------------------------------------------------------- launch

struct Maps {
  CUtensorMap m[4];
};

// A map over [N][heads][D] for boxes of 64 features x one head x `rows` tokens.
inline cudaError_t make_map(CUtensorMap* map, const void* base, uint32_t fmt, const Params& p, int heads, int64_t stride,
                            int rows) {
  const auto encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(tensor_map_encoder());
  if (!encode) return cudaErrorNotSupported;
  const cuuint64_t dims[3] = {(cuuint64_t)p.D, (cuuint64_t)heads, (cuuint64_t)p.N};
  const cuuint64_t strides[2] = {(cuuint64_t)p.D * 2, (cuuint64_t)stride * 2};
  const cuuint32_t box[3] = {64, 1, (cuuint32_t)(rows < p.N ? rows : p.N)};   // a shorter sequence has no whole tile
  const cuuint32_t ones[3] = {1, 1, 1};
  const CUresult r =
      encode(map, fmt ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, const_cast<void*>(base),
             dims, strides, box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

// A work item in the kernels' 32-bit coordinates: own rows first, first + step,
// ... below hi (`tiles` of them) of the document [lo, hi).
struct Item {
  int head, lo, hi, first, tiles;
};
template <bool UNIFORM>
__device__ __forceinline__ Item item_of(const Params& p, uint32_t item, int heads) {
  const Work w = work_of(p, item, heads);
  int64_t lo, hi;
  doc_range(p, w.doc, lo, hi);
  Item i;
  i.head = w.head;
  i.lo = UNIFORM ? (int)uniform((uint32_t)lo) : (int)lo;
  i.hi = UNIFORM ? (int)uniform((uint32_t)hi) : (int)hi;
  const int64_t first = lo + (int64_t)w.tile * ROWS, step = (int64_t)p.hint * ROWS;
  i.first = first < hi ? (int)first : (int)hi;
  i.tiles = (int)((hi - i.first + step - 1) / step);
  if (UNIFORM) {
    i.first = (int)uniform((uint32_t)i.first);
    i.tiles = (int)uniform((uint32_t)i.tiles);
  }
  return i;
}

// Documents of one length: as many blocks as fit the SMs walk all items, so
// that one item's loads run under the previous one's products and its stores.
// Packed documents: a block per item, many of which may be empty.
inline cudaError_t launch_rows(void (*k)(Params, Maps), int smem, Params p, const Maps& maps, int heads, int threads,
                               int blocks_per_sm, cudaStream_t st) {
  int64_t tiles = (p.len + ROWS - 1) / ROWS;
  if (tiles < 1) tiles = 1;
  const int64_t items = (p.docs + (p.offsets ? 1 : 0)) * heads;
  if (items == 0) return cudaSuccess;
  if (items > 0x7fffffff) return cudaErrorInvalidValue;
  const int64_t room = 0x7fffffff / items;
  p.hint = (int)(tiles < room ? tiles : room);
  p.items = (uint32_t)(items * p.hint);
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
