// eqlin_norm.cu -- group layer norm, forward and backward.
//
// Features are [C', T] per token; the statistics run over all F = C'T of them
// and the affine parameters w, b [C'] are shared along the group axis:
//
//   s = x + r (r optional),  mu = mean_f s,  rstd = (mean_f (s - mu)^2 + eps)^-1/2
//   y[n, cT+t] = (s - mu) rstd w[c] + b[c]
//
// and, with xh = (s - mu) rstd and g = gy w,
//
//   ds = rstd (g - mean_f g - xh mean_f(g xh)) + gs       (gs: gradient of s itself, optional)
//   dw[c] = sum_n sum_t gy xh,    db[c] = sum_n sum_t gy
//
// The backward forms s = x + r again from both, unrounded: reading the stored
// sum instead would save one of its six tensors but put the sum's rounding
// (half a step of the type, relative) into xh, and with it into dw.
//
// All sums are FP32; the variance is taken about the mean in a second pass
// over registers, not as E[s^2] - mu^2, which cancels when |mu| >> sigma.
//
// The work is bound by memory: a row is read once into registers (16-byte
// vectors, kept packed in the element type) and everything follows from there.
// A row belongs to `lpr` lanes of a warp (a power of two) holding VPT vectors
// each, or to a whole block when it is longer than 32 lanes hold.  lpr
// and VPT are the pair that leaves the fewest lanes idle (F = 96 in 16 bits:
// 12 vectors = 4 lanes x 3; 768: 32 x 3), so short rows share a warp.  Each
// thread keeps the same columns over all its rows, so w and b are read once
// per thread and the column sums of dw and db stay in registers until the end.
// 12608 x 768 bf16 with a residual, inputs beyond L2: forward 15.8 us (4.9 TB/s),
// backward 23.9 us (4.1 TB/s) with its second launch; 401408 x 96 f16 without:
// 28.9 us (5.3 TB/s) and 48.1 us (4.8 TB/s).
#include "eqlin_internal.cuh"

namespace eqlin {
namespace norm {

// Forward blocks per SM: what the registers of two rows leave.  12608 x 768
// with a residual, inputs beyond L2: 15.8 us at 5 blocks, 19.5 at 8 (spilled);
// 50000 x 120: 9.3 us at 8, 12.8 at 5.
constexpr int kFwdThreads = 128;
constexpr int fwd_blocks(int vpt) { return vpt == 1 ? 8 : vpt == 2 ? 6 : 5; }
constexpr int kBwdThreads = 128, kBwdBlocks = 3;   // backward: room for two rows in registers, 12 warps an SM
// Threads of a block that shares one row, at most: 4 vectors each cover 8192
// features, and the backward's column sums fit its registers.
template <typename E> constexpr int kBlockThreads = sizeof(E) == 4 ? 512 : 256;
inline int block_threads(eqlin_dtype_t dt) { return dt == EQLIN_F32 ? kBlockThreads<float> : kBlockThreads<__half>; }

struct Params {
  const void* x;
  const void* res;
  const void* w;
  const void* b;
  const void* gy;
  const void* gs;
  void* sum;
  void* y;              // y (forward) or ds (backward)
  float* mean;
  float* rstd;
  float* part;          // [blocks][2][Cp] partial column sums (backward)
  int64_t N;
  int F, T, Cp;
  int nvec;             // 16-byte vectors per row
  int lpr;              // lanes per row (threads per row in block mode)
  float eps;
};

// 16-byte load that is not kept in L1 (each row is read once).
__device__ __forceinline__ uint4 ld_stream(const uint4* p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p) : "memory");
  return v;
}

template <typename E>
__device__ __forceinline__ void unpack(const uint4& u, float* f) {
  constexpr int V = 16 / sizeof(E);
  const E* e = reinterpret_cast<const E*>(&u);
#pragma unroll
  for (int i = 0; i < V; ++i) f[i] = Elem<E>::to_f(e[i]);
}
template <typename E>
__device__ __forceinline__ void add(const uint4& u, float* f) {
  constexpr int V = 16 / sizeof(E);
  const E* e = reinterpret_cast<const E*>(&u);
#pragma unroll
  for (int i = 0; i < V; ++i) f[i] += Elem<E>::to_f(e[i]);
}
template <typename E>
__device__ __forceinline__ uint4 pack(const float* f) {
  constexpr int V = 16 / sizeof(E);
  uint4 u;
  E* e = reinterpret_cast<E*>(&u);
#pragma unroll
  for (int i = 0; i < V; ++i) e[i] = Elem<E>::from_f(f[i]);
  return u;
}

// Sums of K values over the threads of a row.  Every thread of the warp (block
// mode: of the block) calls it.
template <bool BLOCK, int K>
__device__ __forceinline__ void row_sum(float (&v)[K], int lpr, float* red) {
  const int steps = BLOCK ? 32 : lpr;
  for (int o = steps >> 1; o > 0; o >>= 1) {
#pragma unroll
    for (int k = 0; k < K; ++k) v[k] += __shfl_xor_sync(0xffffffffu, v[k], o);
  }
  if constexpr (BLOCK) {
    const int warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
    __syncthreads();                       // the previous call's readers are done
    if ((threadIdx.x & 31) == 0)
#pragma unroll
      for (int k = 0; k < K; ++k) red[k * 32 + warp] = v[k];
    __syncthreads();
#pragma unroll
    for (int k = 0; k < K; ++k) {
      float s = 0.f;
      for (int i = 0; i < nw; ++i) s += red[k * 32 + i];
      v[k] = s;
    }
  }
}

// The rows of a thread: its first one, the distance to the next, and its
// place in the row.
struct Place {
  int64_t row, step;
  int lane;             // in the row's lanes
};
template <bool BLOCK>
__device__ __forceinline__ Place place(const Params& p) {
  Place q;
  if constexpr (BLOCK) {
    q.row = blockIdx.x;
    q.step = gridDim.x;
    q.lane = threadIdx.x;
  } else {
    const int per_block = blockDim.x / p.lpr;
    q.row = (int64_t)blockIdx.x * per_block + threadIdx.x / p.lpr;
    q.step = (int64_t)gridDim.x * per_block;
    q.lane = threadIdx.x % p.lpr;
  }
  return q;
}

// TT is the number of neighbouring features known to share a channel: 4 when
// 4 divides T (w, b and the column sums then take a quarter of the registers),
// else 1.
template <typename E, int VPT, int TT, bool BLOCK>
__global__ void __launch_bounds__(BLOCK ? kBlockThreads<E> : kFwdThreads, BLOCK ? 1 : fwd_blocks(VPT))
norm_fwd_kernel(const __grid_constant__ Params p) {
  constexpr int V = 16 / sizeof(E), CG = V / TT;
  __shared__ float red[32];
  const Place at = place<BLOCK>(p);
  grid_dep_launch();
  grid_dep_wait();
  float w[VPT][CG], b[VPT][CG];
#pragma unroll
  for (int j = 0; j < VPT; ++j) {
    const int vec = at.lane + j * p.lpr;
#pragma unroll
    for (int i = 0; i < CG; ++i) {
      const int c = (vec * V + i * TT) / p.T;
      w[j][i] = vec < p.nvec ? Elem<E>::to_f(static_cast<const E*>(p.w)[c]) : 0.f;
      b[j][i] = vec < p.nvec ? Elem<E>::to_f(static_cast<const E*>(p.b)[c]) : 0.f;
    }
  }
  const float inv = 1.f / (float)p.F;
  // the loop's trip count is the same for all threads of a warp: shuffles stay whole
  const int64_t first = at.row - (BLOCK ? 0 : (threadIdx.x & 31) / p.lpr);
  // the next row is on its way while this one is worked on: a warp's own loads
  // are what keeps memory busy
  uint4 x[VPT], r[VPT];
  auto load = [&](int64_t row) {
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      const int vec = at.lane + j * p.lpr;
      const int64_t off = row * p.nvec + vec;
      x[j] = r[j] = make_uint4(0, 0, 0, 0);
      if (row < p.N && vec < p.nvec) {
        x[j] = ld_stream(static_cast<const uint4*>(p.x) + off);
        if (p.res) r[j] = ld_stream(static_cast<const uint4*>(p.res) + off);
      }
    }
  };
  load(at.row);
  for (int64_t base = first, row = at.row; base < p.N; base += at.step, row += at.step) {
    const bool live = row < p.N;
    float s[VPT][V];
    float acc[1] = {0.f};
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      unpack<E>(x[j], s[j]);
      if (p.res) add<E>(r[j], s[j]);
    }
    load(row + at.step);
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      const int vec = at.lane + j * p.lpr;
      if (p.res && live && vec < p.nvec) static_cast<uint4*>(p.sum)[row * p.nvec + vec] = pack<E>(s[j]);
#pragma unroll
      for (int i = 0; i < V; ++i) acc[0] += s[j][i];
    }
    row_sum<BLOCK>(acc, p.lpr, red);
    const float mu = acc[0] * inv;
    acc[0] = 0.f;
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      const bool on = at.lane + j * p.lpr < p.nvec;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        s[j][i] = on ? s[j][i] - mu : 0.f;
        acc[0] = fmaf(s[j][i], s[j][i], acc[0]);
      }
    }
    row_sum<BLOCK>(acc, p.lpr, red);
    const float rstd = 1.f / sqrtf(fmaf(acc[0], inv, p.eps));
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      const int vec = at.lane + j * p.lpr;
#pragma unroll
      for (int i = 0; i < V; ++i) s[j][i] = fmaf(s[j][i] * rstd, w[j][i / TT], b[j][i / TT]);
      if (live && vec < p.nvec) static_cast<uint4*>(p.y)[row * p.nvec + vec] = pack<E>(s[j]);
    }
    if (live && at.lane == 0) {
      p.mean[row] = mu;
      p.rstd[row] = rstd;
    }
  }
}

// What the backward reads of a row: x, gy, and where given res and gs.
template <int VPT, bool RES> struct Row {
  uint4 x[VPT], g[VPT], s[VPT], r[RES ? VPT : 1];
  float mean, rstd;
  __device__ __forceinline__ void load(const Params& p, int64_t row, int lane) {
    const bool live = row < p.N;
    mean = live ? p.mean[row] : 0.f;
    rstd = live ? p.rstd[row] : 0.f;
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      const int vec = lane + j * p.lpr;
      const int64_t at = row * p.nvec + vec;
      x[j] = g[j] = s[j] = make_uint4(0, 0, 0, 0);
      if (RES) r[j] = x[j];
      if (live && vec < p.nvec) {
        x[j] = ld_stream(static_cast<const uint4*>(p.x) + at);
        g[j] = ld_stream(static_cast<const uint4*>(p.gy) + at);
        if (RES) r[j] = ld_stream(static_cast<const uint4*>(p.res) + at);
        if (p.gs) s[j] = ld_stream(static_cast<const uint4*>(p.gs) + at);
      }
    }
  }
};

template <typename E, int VPT, int TT, bool BLOCK, bool RES>
__global__ void __launch_bounds__(BLOCK ? kBlockThreads<E> : kBwdThreads,
                                  BLOCK ? (sizeof(E) == 2 && VPT <= 2 ? 2 : 1) : kBwdBlocks)
norm_bwd_kernel(const __grid_constant__ Params p) {
  constexpr int V = 16 / sizeof(E), CG = V / TT;
  extern __shared__ float colsum[];        // [2][F / TT]: dw, db of this block
  __shared__ float red[64];
  const Place at = place<BLOCK>(p);
  grid_dep_launch();
  grid_dep_wait();
  float w[VPT][CG], dw[VPT][CG], db[VPT][CG];
#pragma unroll
  for (int j = 0; j < VPT; ++j) {
    const int vec = at.lane + j * p.lpr;
#pragma unroll
    for (int i = 0; i < CG; ++i) {
      const int c = (vec * V + i * TT) / p.T;
      w[j][i] = vec < p.nvec ? Elem<E>::to_f(static_cast<const E*>(p.w)[c]) : 0.f;
      dw[j][i] = db[j][i] = 0.f;
    }
  }
  const float inv = 1.f / (float)p.F;
  const int64_t first = at.row - (BLOCK ? 0 : (threadIdx.x & 31) / p.lpr);
  // Rows are kept packed, and the next one is on its way while this one is
  // worked on: a warp's own loads are what keeps memory busy.
  Row<VPT, RES> cur, nxt;
  cur.load(p, at.row, at.lane);
  for (int64_t base = first, row = at.row; base < p.N; base += at.step, row += at.step) {
    const bool live = row < p.N;
    nxt.load(p, row + at.step, at.lane);
    const float mu = cur.mean, rstd = cur.rstd;
    float m[2] = {0.f, 0.f};
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      if (!(live && at.lane + j * p.lpr < p.nvec)) continue;
      float x[V], g[V];
      unpack<E>(cur.x[j], x);
      if (RES) add<E>(cur.r[j], x);
      unpack<E>(cur.g[j], g);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const float xh = (x[i] - mu) * rstd, gw = g[i] * w[j][i / TT];
        m[0] += gw;
        m[1] = fmaf(gw, xh, m[1]);
        db[j][i / TT] += g[i];
        dw[j][i / TT] = fmaf(g[i], xh, dw[j][i / TT]);
      }
    }
    row_sum<BLOCK>(m, p.lpr, red);
    m[0] *= inv;
    m[1] *= inv;
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      const int vec = at.lane + j * p.lpr;
      if (!(live && vec < p.nvec)) continue;
      float x[V], g[V];
      unpack<E>(cur.x[j], x);
      if (RES) add<E>(cur.r[j], x);
      unpack<E>(cur.g[j], g);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const float xh = (x[i] - mu) * rstd;
        x[i] = rstd * (fmaf(g[i], w[j][i / TT], -m[0]) - xh * m[1]);
      }
      if (p.gs) add<E>(cur.s[j], x);
      static_cast<uint4*>(p.y)[row * p.nvec + vec] = pack<E>(x);
    }
    cur = nxt;
  }
  // Column sums of the block in a fixed order: rows that share a warp by
  // shuffles, then the warps one after the other.
  const int groups = p.F / TT;
  if constexpr (!BLOCK) {
    for (int o = 16; o >= p.lpr; o >>= 1)
#pragma unroll
      for (int j = 0; j < VPT; ++j)
#pragma unroll
        for (int i = 0; i < CG; ++i) {
          dw[j][i] += __shfl_xor_sync(0xffffffffu, dw[j][i], o);
          db[j][i] += __shfl_xor_sync(0xffffffffu, db[j][i], o);
        }
    const int warp = threadIdx.x >> 5;
    for (int turn = 0; turn < (int)(blockDim.x >> 5); ++turn) {
      if (warp == turn && (threadIdx.x & 31) < p.lpr) {
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
          const int vec = at.lane + j * p.lpr;
          if (vec >= p.nvec) continue;
#pragma unroll
          for (int i = 0; i < CG; ++i) {
            const int f = vec * CG + i;
            colsum[f] = dw[j][i] + (turn ? colsum[f] : 0.f);
            colsum[groups + f] = db[j][i] + (turn ? colsum[groups + f] : 0.f);
          }
        }
      }
      __syncthreads();
    }
  } else {
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      const int vec = at.lane + j * p.lpr;
      if (vec >= p.nvec) continue;
#pragma unroll
      for (int i = 0; i < CG; ++i) {
        colsum[vec * CG + i] = dw[j][i];
        colsum[groups + vec * CG + i] = db[j][i];
      }
    }
    __syncthreads();
  }
  const int per = p.T / TT;                // column groups per channel
  for (int i = threadIdx.x; i < 2 * p.Cp; i += blockDim.x) {
    const int which = i / p.Cp, c = i - which * p.Cp;
    float s = 0.f;
    for (int t = 0; t < per; ++t) s += colsum[which * groups + c * per + t];
    p.part[(int64_t)blockIdx.x * 2 * p.Cp + i] = s;
  }
}

// dw, db from the blocks' partial sums, in a fixed order: 32 columns by 32
// slices of the blocks, the slices then added by a tree.
__global__ void __launch_bounds__(1024) norm_cols_kernel(const float* part, int blocks, int Cp, float* dw, float* db) {
  __shared__ float red[32][33];
  const int col = blockIdx.x * 32 + threadIdx.x, cols = 2 * Cp;
  grid_dep_launch();
  grid_dep_wait();
  float s = 0.f;
  if (col < cols)
    for (int g = threadIdx.y; g < blocks; g += 32) s += part[(int64_t)g * cols + col];
  red[threadIdx.y][threadIdx.x] = s;
  __syncthreads();
  // warp y reduces column y over the slices
  s = red[threadIdx.x][threadIdx.y];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  const int out = blockIdx.x * 32 + threadIdx.y;
  if (threadIdx.x == 0 && out < cols) {
    if (out < Cp) dw[out] = s;
    else db[out - Cp] = s;
  }
}

// ------------------------------------------------------------------ launch

constexpr int kMaxF = 8192;
// Blocks of the backward at most, kBwdBlocks for each SM of a B200; the
// partial sums are as many rows.
constexpr int kMaxParts = 148 * kBwdBlocks;

struct Shape {
  int vpt, lpr;
  bool block;
};
inline Shape shape_of(int nvec, int T, int max_threads) {
  // vectors per thread whose two rows and column sums fit the backward's registers
  const int most = T % 4 == 0 ? 3 : 2;
  Shape best{0, 0, false};
  if (nvec <= 32 * most) {
    int waste = 1 << 30;
    for (int vpt = 1; vpt <= most; ++vpt) {
      int lpr = 1;
      while (lpr * vpt < nvec) lpr *= 2;
      if (lpr > 32) continue;
      if (lpr * vpt - nvec < waste) {      // fewer vectors per thread on a tie: more threads for short inputs
        waste = lpr * vpt - nvec;
        best = Shape{vpt, lpr, false};
      }
    }
    return best;
  }
  // a block per row: at least two vectors a thread (fewer warps wait at the row's barriers)
  int vpt = (nvec + max_threads - 1) / max_threads;
  if (vpt < 2) vpt = 2;
  const int threads = ((nvec + vpt - 1) / vpt + 31) / 32 * 32;
  return Shape{vpt, threads, true};
}

int sm_count() {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
  return n;
}

template <typename E, int TT, int VPT>
cudaError_t launch_vpt(const Params& p, const Shape& s, bool bwd, int blocks, cudaStream_t st) {
  const int threads = s.block ? s.lpr : bwd ? kBwdThreads : kFwdThreads;
  const size_t smem = bwd ? (size_t)2 * (p.F / TT) * sizeof(float) : 0;
  void (*k)(Params) = bwd ? (p.res ? (s.block ? norm_bwd_kernel<E, VPT, TT, true, true>
                                              : norm_bwd_kernel<E, VPT, TT, false, true>)
                                   : (s.block ? norm_bwd_kernel<E, VPT, TT, true, false>
                                              : norm_bwd_kernel<E, VPT, TT, false, false>))
                          : (s.block ? norm_fwd_kernel<E, VPT, TT, true> : norm_fwd_kernel<E, VPT, TT, false>);
  if (smem > 40 * 1024) {
    const cudaError_t e = set_smem_limit(reinterpret_cast<const void*>(k), 2 * kMaxF * (int)sizeof(float));
    if (e != cudaSuccess) return e;
  }
  const cudaError_t e = launch_pdl(k, dim3(blocks), dim3(threads), smem, st, p);
  if (e == cudaSuccess) count_launches(1);
  return e;
}

template <typename E, int TT>
cudaError_t launch_tt(const Params& p, const Shape& s, bool bwd, int blocks, cudaStream_t st) {
  switch (s.vpt) {
    case 1: return launch_vpt<E, TT, 1>(p, s, bwd, blocks, st);
    case 2: return launch_vpt<E, TT, 2>(p, s, bwd, blocks, st);
    case 3: return launch_vpt<E, TT, 3>(p, s, bwd, blocks, st);
    default: return launch_vpt<E, TT, 4>(p, s, bwd, blocks, st);   // a block per row
  }
}

template <typename E>
cudaError_t launch(const Params& p, const Shape& s, bool bwd, int blocks, cudaStream_t st) {
  return p.T % 4 == 0 ? launch_tt<E, 4>(p, s, bwd, blocks, st) : launch_tt<E, 1>(p, s, bwd, blocks, st);
}

cudaError_t dispatch(eqlin_dtype_t dt, const Params& p, const Shape& s, bool bwd, int blocks, cudaStream_t st) {
  switch (dt) {
    case EQLIN_F32: return launch<float>(p, s, bwd, blocks, st);
    case EQLIN_F16: return launch<__half>(p, s, bwd, blocks, st);
    default: return launch<__nv_bfloat16>(p, s, bwd, blocks, st);
  }
}

bool bad16(const void* p) { return ((uintptr_t)p & 15u) != 0; }
bool bad4(const void* p) { return ((uintptr_t)p & 3u) != 0; }
bool bad_elem(const void* p, eqlin_dtype_t dt) { return ((uintptr_t)p & (dt == EQLIN_F32 ? 3u : 1u)) != 0; }

eqlin_status_t check(int T, int64_t Cp, eqlin_dtype_t dt, int64_t N) {
  if (dt != EQLIN_F32 && dt != EQLIN_F16 && dt != EQLIN_BF16) return EQLIN_ERR_INVALID_ARG;
  if (T < 1 || Cp < 1 || N < 0) return EQLIN_ERR_INVALID_ARG;
  if (T > 16 || Cp > kMaxF || Cp * T > kMaxF) return EQLIN_ERR_UNSUPPORTED;
  if ((Cp * T * (dt == EQLIN_F32 ? 4 : 2)) % 16) return EQLIN_ERR_MISALIGNED;
  return EQLIN_OK;
}

Params describe(int T, int64_t Cp, eqlin_dtype_t dt, int64_t N) {
  Params p = {};
  p.N = N;
  p.T = T;
  p.Cp = (int)Cp;
  p.F = (int)Cp * T;
  p.nvec = p.F * (dt == EQLIN_F32 ? 4 : 2) / 16;
  return p;
}

int64_t parts_of(int64_t N) { return N < kMaxParts ? N : kMaxParts; }

}  // namespace norm
}  // namespace eqlin

using namespace eqlin;

extern "C" eqlin_status_t eqlin_norm_forward(int T, int64_t Cp, eqlin_dtype_t dtype, const void* x, const void* res,
                                             const void* w, const void* b, float eps, void* sum, void* y,
                                             float* mean, float* rstd, int64_t N, void* stream) {
  const eqlin_status_t st = norm::check(T, Cp, dtype, N);
  if (st != EQLIN_OK) return st;
  if (!w || !b || !(eps >= 0.f) || (res == nullptr) != (sum == nullptr)) return EQLIN_ERR_INVALID_ARG;
  if (N == 0) return EQLIN_OK;
  if (!x || !y || !mean || !rstd) return EQLIN_ERR_INVALID_ARG;
  if (norm::bad16(x) || norm::bad16(res) || norm::bad16(sum) || norm::bad16(y) || norm::bad_elem(w, dtype) ||
      norm::bad_elem(b, dtype) || norm::bad4(mean) || norm::bad4(rstd))
    return EQLIN_ERR_MISALIGNED;
  norm::Params p = norm::describe(T, Cp, dtype, N);
  p.x = x;
  p.res = res;
  p.w = w;
  p.b = b;
  p.sum = sum;
  p.y = y;
  p.mean = mean;
  p.rstd = rstd;
  p.eps = eps;
  const norm::Shape s = norm::shape_of(p.nvec, T, norm::block_threads(dtype));
  p.lpr = s.lpr;
  const int64_t rows = s.block ? 1 : norm::kFwdThreads / s.lpr;
  const int64_t want = (N + rows - 1) / rows, cap = norm::fwd_blocks(s.vpt) * (int64_t)norm::sm_count();
  if (cap == 0) return EQLIN_ERR_CUDA;
  const cudaError_t e = norm::dispatch(dtype, p, s, false, (int)(want < cap ? want : cap),
                                       static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? EQLIN_OK : EQLIN_ERR_CUDA;
}

extern "C" int64_t eqlin_norm_workspace_bytes(int T, int64_t Cp, int64_t N) {
  if (T < 1 || T > 16 || Cp < 1 || Cp > norm::kMaxF || Cp * T > norm::kMaxF || N < 0) return -1;
  return norm::parts_of(N) * 2 * Cp * (int64_t)sizeof(float);
}

extern "C" eqlin_status_t eqlin_norm_backward(int T, int64_t Cp, eqlin_dtype_t dtype, const void* gy, const void* gsum,
                                              const void* x, const void* res, const void* w, const float* mean, const float* rstd,
                                              void* dx, float* dw, float* db, void* workspace, int64_t N,
                                              void* stream) {
  const eqlin_status_t st = norm::check(T, Cp, dtype, N);
  if (st != EQLIN_OK) return st;
  if (!w || !dw || !db) return EQLIN_ERR_INVALID_ARG;
  if (norm::bad_elem(w, dtype) || norm::bad4(dw) || norm::bad4(db)) return EQLIN_ERR_MISALIGNED;
  cudaStream_t cs = static_cast<cudaStream_t>(stream);
  if (N == 0) {
    cudaError_t e = cudaMemsetAsync(dw, 0, (size_t)Cp * sizeof(float), cs);
    if (e == cudaSuccess) e = cudaMemsetAsync(db, 0, (size_t)Cp * sizeof(float), cs);
    return e == cudaSuccess ? EQLIN_OK : EQLIN_ERR_CUDA;
  }
  if (!gy || !x || !mean || !rstd || !dx || !workspace) return EQLIN_ERR_INVALID_ARG;
  if (norm::bad16(gy) || norm::bad16(gsum) || norm::bad16(x) || norm::bad16(res) || norm::bad16(dx) || norm::bad16(workspace) ||
      norm::bad4(mean) || norm::bad4(rstd))
    return EQLIN_ERR_MISALIGNED;
  norm::Params p = norm::describe(T, Cp, dtype, N);
  p.x = x;
  p.res = res;
  p.gy = gy;
  p.gs = gsum;
  p.w = w;
  p.mean = const_cast<float*>(mean);
  p.rstd = const_cast<float*>(rstd);
  p.y = dx;
  p.part = static_cast<float*>(workspace);
  const norm::Shape s = norm::shape_of(p.nvec, T, norm::block_threads(dtype));
  p.lpr = s.lpr;
  const int64_t rows = s.block ? 1 : norm::kBwdThreads / s.lpr;
  const int64_t want = (N + rows - 1) / rows, cap = norm::kMaxParts;
  const int blocks = (int)(want < cap ? want : cap);
  cudaError_t e = norm::dispatch(dtype, p, s, true, blocks, cs);
  if (e == cudaSuccess)
    e = launch_pdl(norm::norm_cols_kernel, dim3((unsigned)((2 * Cp + 31) / 32)), dim3(32, 32), 0, cs,
                   (const float*)p.part, blocks, (int)Cp, dw, db);
  if (e == cudaSuccess) count_launches(1);
  return e == cudaSuccess ? EQLIN_OK : EQLIN_ERR_CUDA;
}
