// eqlin_attn_tc.cuh -- parts shared by the tensor-core attention kernels.
//
// All of them have one shape: 128 rows stay ("own" rows: queries, or keys in
// the kernel for dk and dv), the other side passes by in tiles of up to 128
// ("moving" rows).  A block is six warps:
//
//   warps 0-3   one thread per own row: scores out of TMEM, softmax (or its
//               gradient) in FP32 registers, 16-bit probabilities back into
//               TMEM as the next product's A operand
//   warp 4      lane 0 issues the MMAs; the warp allocates TMEM
//   warp 5      brings tiles into shared memory with 16-byte asynchronous
//               copies that write zeros past the document's end and past the
//               head's features
//
// Copies rather than TMA tensor loads, because a tile may end inside a
// document's neighbour: its rows must read as zero (a product with P = 0 would
// spread a neighbour's infinity or NaN), and documents start at any token.
//
// Shared tiles are panels of 64 features: 128 rows of 128 bytes in the
// 128-byte swizzle (16-byte chunk j of row r at chunk j ^ (r & 7)).  The same
// image serves as a K-major operand (contraction over features) and as an
// MN-major one (contraction over rows).
#pragma once

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

// D[tmem] (+)= A[tmem] * B[smem]: A holds 16-bit pairs, row = lane, two
// consecutive k per column.
__device__ __forceinline__ void mma_f16_ts(uint32_t d, uint32_t a, uint64_t b_desc, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}"
      ::"r"(d), "r"(a), "l"(b_desc), "r"(idesc), "r"(accumulate) : "memory");
}
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
__device__ __forceinline__ void load_rows(uint32_t dst, const void* src, int64_t stride, int64_t head_off, int64_t r0,
                                          int64_t hi, int rows, int D, int chunks, int lane) {
  const int sub = lane >> 3, ch0 = lane & 7;
  const char* base = reinterpret_cast<const char*>(static_cast<const E*>(src) + head_off);
  const int64_t step = stride * (int64_t)sizeof(E);
  const int left = (int)(hi - r0 < TILE_ROWS ? hi - r0 : TILE_ROWS);
#pragma unroll
  for (int pn = 0; pn < DP / 64; ++pn) {
    const int ch = pn * 8 + ch0;
    if (ch >= chunks) continue;
    const bool live_ch = ch * 8 < D;
    const char* from = base + (r0 + sub) * step + ch * 16;
    const uint32_t to = dst + pn * TILE_ROWS * 128;
#pragma unroll 4
    for (int r = sub; r < rows; r += 4, from += 4 * step) {
      const bool on = live_ch && r < left;
      cp_async16(to + r * 128 + ((ch0 ^ (r & 7)) << 4), on ? from : base, on ? 16u : 0u);
    }
  }
}

// Positions of moving rows into [axes][128].
__device__ __forceinline__ void load_positions(float* dst, const Params& p, int64_t r0, int64_t hi, int rows, int lane) {
  for (int a = 0; a < p.axes; ++a)
    for (int r = lane; r < rows; r += 32) dst[a * ROWS + r] = r0 + r < hi ? p.pos[(r0 + r) * p.axes + a] : 0.f;
}

// The loading warp's side of a ring of slots: copies are announced once they
// have landed and been made visible to the tensor core, at the latest when the
// warp has nothing else to issue.
struct Pending {
  int count = 0;
  uint64_t* bar[3];
};
__device__ __forceinline__ void announce_all(Pending& q) {
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
                                      volatile int* abort_flag, int lane, int* err, uint32_t where, uint32_t iter) {
  int ready = 0;
  if (lane == 0) ready = mbar_test_wait(empty, parity) ? 1 : 0;
  if (__shfl_sync(0xffffffffu, ready, 0)) {
    __syncwarp();
    return true;
  }
  announce_all(q);
  return wwait(empty, parity, limit, abort_flag, lane, err, where, iter);
}

// Scores in base 2 from raw products: u2 = raw * scale * log2 e, capped and
// biased.  tanh(x) = 1 - 2 / (1 + e^{2x}): its absolute error is a few 2^-24
// everywhere, which is what a score needs (two MUFU operations; tanh.approx
// would be one, but is only good to 2^-11).
struct Score {
  float scale2;           // scale * log2 e
  float twocap;           // 2 scale log2 e / cap: e^{2u/cap} = 2^(raw * twocap)
  float cap2;             // cap * log2 e
  float slope2;           // slope * log2 e
};
__device__ __forceinline__ Score score_of(const Params& p, int head) {
  Score s;
  s.scale2 = p.scale * kLog2e;
  s.cap2 = p.cap * kLog2e;
  s.twocap = p.cap > 0.f ? 2.f * p.scale * kLog2e / p.cap : 0.f;
  s.slope2 = p.axes ? p.slopes[head] * kLog2e : 0.f;
  return s;
}
__device__ __forceinline__ float tanh_raw(float raw, const Score& s) { return fmaf(-2.f, rcp(1.f + ex2(raw * s.twocap)), 1.f); }

// City-block distances of 32 moving rows from one own row.
template <int AXES>
__device__ __forceinline__ void distances(const float* pos, int c0, const float* own, float (&d)[4]) {
  // four columns c0 .. c0+3
#pragma unroll
  for (int a = 0; a < AXES; ++a) {
    const float4 v = *reinterpret_cast<const float4*>(pos + a * ROWS + c0);
    if (a == 0) {
      d[0] = fabsf(own[0] - v.x);
      d[1] = fabsf(own[0] - v.y);
      d[2] = fabsf(own[0] - v.z);
      d[3] = fabsf(own[0] - v.w);
    } else {
      d[0] += fabsf(own[a] - v.x);
      d[1] += fabsf(own[a] - v.y);
      d[2] += fabsf(own[a] - v.z);
      d[3] += fabsf(own[a] - v.w);
    }
  }
}

inline cudaError_t launch_rows(void (*k)(Params), int smem, Params p, int heads, cudaStream_t st,
                               int threads = kThreads) {
  int64_t tiles = (p.len + ROWS - 1) / ROWS;
  if (tiles < 1) tiles = 1;
  const int64_t items = (p.docs + (p.offsets ? 1 : 0)) * heads;
  if (items == 0) return cudaSuccess;
  if (items > 0x7fffffff) return cudaErrorInvalidValue;
  const int64_t room = 0x7fffffff / items;
  p.hint = (int)(tiles < room ? tiles : room);
  cudaError_t e = set_smem_limit(reinterpret_cast<const void*>(k), smem);
  if (e == cudaSuccess) e = launch_pdl(k, dim3((unsigned)(items * p.hint)), dim3(threads), (size_t)smem, st, p);
  if (e == cudaSuccess) count_launches(1);
  return e;
}

}  // namespace attn_tc
}  // namespace eqlin
