// eqlin_attn_simt.cu -- document attention of f32 tensors, on the CUDA cores.
//
// One block owns 64 rows of one head of one document and walks the other
// side in tiles of 64, with one pass over it: the forward keeps each row's
// running maximum and sum and rescales its output when the maximum grows.
// The backward is two kernels of the same shape, so no sum needs atomics and
// results do not depend on the order in which blocks run: one owns query rows
// (dq, and delta on the way), the other key rows (dk, dv, over all query
// heads that share them).
//
// Threads form a grid 16 wide; thread (ty, tx) owns R rows from R ty on and,
// of a 64 x 64 product, columns tx + 16j: reads of the moving operand are then
// 16 rows apart by D + 4 floats, free of bank conflicts, and those of the rows
// broadcast.  Products take two FMAs an instruction, stop at a document's last
// column (in steps of 16, or 4), and warps without rows skip them: the last
// tile of 197 tokens costs 5 columns, not 64.
// A warp alone reads and writes its rows of P, so only tiles need block
// barriers.  tanhf and expf, at some 60 instructions a score together, would
// cost as much as one product each; tanh_fast and exp_fast take a third.
#include "eqlin_attn.cuh"
#include "eqlin_ptx.cuh"

namespace eqlin {
namespace attn_simt {

using namespace attn;
using ptx::fma2;
using ptx::pk2;
using ptx::unpk2;

constexpr int B = 64;                     // rows and columns of a tile
constexpr int LDP = B + 4;

// AHEAD: the next moving tile is read into registers while this one is worked
// on.  Not at 64 features: two blocks of 128 registers hide the reads better
// than the spills cost (16 x 197 tokens, 6 heads of 64: backward 165 us against
// 188; 512 windows of 49, 3 heads of 32: 135 with, 156 without).
template <int DP> struct Cfg {
  static constexpr int R = 4;              // rows per thread
  static constexpr int THREADS = 16 * (B / R);
  static constexpr bool AHEAD = DP != 64;
  static constexpr int LD = DP + 4;
  static constexpr int TILE = B * LD;     // floats
  static constexpr int DC = (DP + 63) / 64;   // float4 groups of a thread's output columns
};

// Blocks whose document index is `docs` (packed calls only) clear the rows
// outside all documents: [0, first offset) and [last offset, N).
template <typename F>
__device__ __forceinline__ void outside_rows(const Params& p, int tile, F&& clear) {
  const int64_t a = min(max((int64_t)p.offsets[0], (int64_t)0), p.N);
  const int64_t b = min(max((int64_t)p.offsets[p.docs], a), p.N);
  for (int64_t r = tile; r < a; r += p.hint) clear(r);
  for (int64_t r = b + tile; r < p.N; r += p.hint) clear(r);
}

struct Work {
  int64_t doc;
  int head, tile;
};
// A block's work: the first tile of every document and head before any second
// one, so that the short last tiles fill the gaps of the last wave (197 tokens
// of 16 images in 6 heads are 288 full tiles, one wave, and 96 of 5 rows).
__device__ __forceinline__ Work work_of_row(const Params& p, int heads) {
  const uint32_t each = p.items / (uint32_t)p.hint;
  Work w;
  w.tile = (int)(blockIdx.x / each);
  const uint32_t rest = blockIdx.x - (uint32_t)w.tile * each, d = rest / (uint32_t)heads;
  w.head = (int)(rest - d * (uint32_t)heads);
  w.doc = d;
  return w;
}

// Rows [r0, r0 + 64) of a head, zero past `hi` and past D: global to registers
// and registers to shared memory.
template <int DP> struct Rows {
  static constexpr int N = B * (DP / 4) / Cfg<DP>::THREADS;
  float4 v[N];
  __device__ __forceinline__ void read(const void* src, int64_t stride, int64_t head_off, int64_t r0, int64_t hi, int D) {
#pragma unroll
    for (int k = 0; k < N; ++k) {
      const int i = threadIdx.x + k * Cfg<DP>::THREADS, r = i / (DP / 4), c = (i - r * (DP / 4)) * 4;
      v[k] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (r0 + r < hi && c < D)
        v[k] = *reinterpret_cast<const float4*>(static_cast<const float*>(src) + (r0 + r) * stride + head_off + c);
    }
  }
  __device__ __forceinline__ void write(float* dst, float mul) const {
#pragma unroll
    for (int k = 0; k < N; ++k) {
      const int i = threadIdx.x + k * Cfg<DP>::THREADS, r = i / (DP / 4), c = (i - r * (DP / 4)) * 4;
      *reinterpret_cast<float4*>(dst + r * Cfg<DP>::LD + c) =
          make_float4(v[k].x * mul, v[k].y * mul, v[k].z * mul, v[k].w * mul);
    }
  }
};
template <int DP>
__device__ __forceinline__ void load_tile(float* dst, const void* src, int64_t stride, int64_t head_off, int64_t r0,
                                          int64_t hi, int D, float mul) {
  Rows<DP> rows;
  rows.read(src, stride, head_off, r0, hi, D);
  rows.write(dst, mul);
}

// acc[i][j] = A[row R ty + i] . Bm[row tx + 16j] over DP features; columns from
// nc on are left at 0.
template <int DP, int J>
__device__ __forceinline__ void mm_nt_cols(const float* A, const float* Bm, float (&acc)[Cfg<DP>::R][4]) {
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  constexpr int R = Cfg<DP>::R;
  uint64_t sum[R][J];                      // even and odd features apart: one instruction for two products
#pragma unroll
  for (int i = 0; i < R; ++i)
#pragma unroll
    for (int j = 0; j < J; ++j) sum[i][j] = 0;
#pragma unroll 4
  for (int d = 0; d < DP; d += 4) {
    ulonglong2 a[R], b[J];
#pragma unroll
    for (int i = 0; i < R; ++i) a[i] = *reinterpret_cast<const ulonglong2*>(A + (R * ty + i) * Cfg<DP>::LD + d);
#pragma unroll
    for (int j = 0; j < J; ++j) b[j] = *reinterpret_cast<const ulonglong2*>(Bm + (tx + 16 * j) * Cfg<DP>::LD + d);
#pragma unroll
    for (int i = 0; i < R; ++i)
#pragma unroll
      for (int j = 0; j < J; ++j) sum[i][j] = fma2(a[i].y, b[j].y, fma2(a[i].x, b[j].x, sum[i][j]));
  }
#pragma unroll
  for (int i = 0; i < R; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float x = 0.f, y = 0.f;
      if (j < J) unpk2(sum[i][j], x, y);
      acc[i][j] = x + y;
    }
}

template <int DP>
__device__ __forceinline__ void mm_nt(const float* A, const float* Bm, int nc, float (&acc)[Cfg<DP>::R][4]) {
  if (nc > 48) mm_nt_cols<DP, 4>(A, Bm, acc);
  else if (nc > 32) mm_nt_cols<DP, 3>(A, Bm, acc);
  else if (nc > 16) mm_nt_cols<DP, 2>(A, Bm, acc);
  else mm_nt_cols<DP, 1>(A, Bm, acc);
}

// out[i][c] += sum_j P[R ty + i][j] M[j][4tx + 64c ..] over the first nc rows of M
template <int DP>
__device__ __forceinline__ void mm_nn(const float* P, const float* M, int nc, uint64_t (&out)[Cfg<DP>::R][Cfg<DP>::DC][2]) {
  constexpr int R = Cfg<DP>::R;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  if (4 * tx >= DP) return;
#pragma unroll 2
  for (int j = 0; j < nc; j += 4) {
    float4 a[R];
#pragma unroll
    for (int i = 0; i < R; ++i) a[i] = *reinterpret_cast<const float4*>(P + (R * ty + i) * LDP + j);
#pragma unroll
    for (int jj = 0; jj < 4; ++jj)
#pragma unroll
      for (int c = 0; c < Cfg<DP>::DC; ++c) {
        const ulonglong2 m = *reinterpret_cast<const ulonglong2*>(M + (j + jj) * Cfg<DP>::LD + 4 * tx + 64 * c);
#pragma unroll
        for (int i = 0; i < R; ++i) {
          const float w = jj == 0 ? a[i].x : jj == 1 ? a[i].y : jj == 2 ? a[i].z : a[i].w;
          const uint64_t w2 = pk2(w, w);
          out[i][c][0] = fma2(w2, m.x, out[i][c][0]);
          out[i][c][1] = fma2(w2, m.y, out[i][c][1]);
        }
      }
  }
}

// Row i times mul[i].
template <int DP>
__device__ __forceinline__ void store_rows(void* dst, int64_t stride, int64_t head_off, int64_t r0, int64_t hi, int D,
                                           const uint64_t (&v)[Cfg<DP>::R][Cfg<DP>::DC][2], const float (&mul)[Cfg<DP>::R]) {
  constexpr int R = Cfg<DP>::R;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const int64_t r = r0 + R * ty + i;
    if (r >= hi) continue;
#pragma unroll
    for (int c = 0; c < Cfg<DP>::DC; ++c) {
      const int d = 4 * tx + 64 * c;
      if (d >= D) continue;               // D is a multiple of 4
      float4 f;
      unpk2(v[i][c][0], f.x, f.y);
      unpk2(v[i][c][1], f.z, f.w);
      f.x *= mul[i];
      f.y *= mul[i];
      f.z *= mul[i];
      f.w *= mul[i];
      *reinterpret_cast<float4*>(static_cast<float*>(dst) + r * stride + head_off + d) = f;
    }
  }
}

__device__ __forceinline__ void clear_row(void* dst, int64_t stride, int64_t head_off, int64_t r, int D) {
  for (int d = threadIdx.x; d < D; d += blockDim.x) static_cast<float*>(dst)[r * stride + head_off + d] = 0.f;
}

// What goes with a tile's rows: positions [axes][64] and, for moving queries,
// lse [64] and delta [64].
template <int DP, bool STAT> struct Side {
  static constexpr int T = Cfg<DP>::THREADS, N = (kMaxAxes * B + T - 1) / T;
  float pos[N], lse, delta;
  __device__ __forceinline__ void read(const Params& p, int head, int64_t r0, int64_t hi) {
#pragma unroll
    for (int k = 0; k < N; ++k) {
      const int i = threadIdx.x + k * T, a = i / B, r = i - a * B;
      pos[k] = a < p.axes && r0 + r < hi ? p.pos[(r0 + r) * p.axes + a] : 0.f;
    }
    if (STAT) {
      const bool on = threadIdx.x < B && r0 + threadIdx.x < hi;
      lse = on ? p.lse[(int64_t)head * p.N + r0 + threadIdx.x] : 0.f;
      delta = on ? p.delta[(int64_t)head * p.N + r0 + threadIdx.x] : 0.f;
    }
  }
  __device__ __forceinline__ void write(float* dst, float* stat) const {
#pragma unroll
    for (int k = 0; k < N; ++k)
      if (threadIdx.x + k * T < kMaxAxes * B) dst[threadIdx.x + k * T] = pos[k];
    if (STAT && threadIdx.x < B) {
      stat[threadIdx.x] = lse;
      stat[B + threadIdx.x] = delta;
    }
  }
};
// City-block distances of the thread's R x 4 scores, times mul.
template <int R>
__device__ __forceinline__ void distances(const Params& p, const float* pr, const float* pc, float mul, float (&d)[R][4]) {
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
#pragma unroll
  for (int i = 0; i < R; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) d[i][j] = 0.f;
#pragma unroll
  for (int a = 0; a < kMaxAxes; ++a) {
    if (a >= p.axes) break;
    float c[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) c[j] = pc[a * B + tx + 16 * j];
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const float r = pr[a * B + R * ty + i];
#pragma unroll
      for (int j = 0; j < 4; ++j) d[i][j] += fabsf(r - c[j]);
    }
  }
#pragma unroll
  for (int i = 0; i < R; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) d[i][j] *= mul;
}

// ------------------------------------------------------------- exponentials

// e^x for x <= 0 or so: the product with log2 e is taken to twice FP32's
// precision, so that the error stays at ex2.approx's 2^-22 for any x; a third
// of expf's instructions.
__device__ __forceinline__ float exp_fast(float x) {
  const float h = x * kLog2e, l = fmaf(x, kLog2e, -h) + x * 1.925963033500e-8f;
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(h));
  // h = -inf (masked) leaves l a NaN
  return y > 0.f ? fmaf(y, l * kLn2, y) : y;
}
// tanh: below 0.7 an odd polynomial (a weighted least-squares fit of tanh(x)/x),
// 2.0e-8 off at most, the FP32 roundings apart (with them 1.5e-7 relative); the
// usual case below a cap; tanhf elsewhere.
__device__ __forceinline__ float tanh_fast(float x) {
  const float z = x * x;
  if (z > 0.49f) return tanhf(x);
  float q = fmaf(-0.004874242004007101f, z, 0.01973520778119564f);
  q = fmaf(q, z, -0.053383808583021164f);
  q = fmaf(q, z, 0.1332535296678543f);
  q = fmaf(q, z, -0.33332860469818115f);
  q = fmaf(q, z, 0.9999999403953552f);
  return q * x;
}

// ------------------------------------------------------------------ forward

template <int DP>
__global__ void __launch_bounds__(Cfg<DP>::THREADS, DP > 64 ? 1 : 2) attn_simt_fwd_kernel(const __grid_constant__ Params p) {
  extern __shared__ __align__(16) float sm[];
  float* Q = sm;
  float* K = Q + Cfg<DP>::TILE;
  float* V = K + Cfg<DP>::TILE;
  float* P = V + Cfg<DP>::TILE;
  float* pq = P + B * LDP;
  float* pk = pq + kMaxAxes * B;
  constexpr int R = Cfg<DP>::R;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  grid_dep_launch();
  grid_dep_wait();
  const Work w = work_of_row(p, p.H);
  const int64_t qh = (int64_t)w.head * p.D, kh = (int64_t)(w.head / (p.H / p.K)) * p.D;
  if (w.doc == p.docs) {
    outside_rows(p, w.tile, [&](int64_t r) {
      clear_row(p.o, p.os, qh, r, p.D);
      if (threadIdx.x == 0) p.lse[(int64_t)w.head * p.N + r] = 0.f;
    });
    return;
  }
  int64_t lo, hi;
  doc_range(p, w.doc, lo, hi);
  const float slope = p.axes ? p.slopes[w.head] : 0.f;
  const float icap = p.cap > 0.f ? 1.f / p.cap : 0.f;
  for (int64_t r0 = lo + (int64_t)w.tile * B; r0 < hi; r0 += (int64_t)p.hint * B) {
    __syncthreads();
    load_tile<DP>(Q, p.q, p.qs, qh, r0, hi, p.D, p.scale);
    Side<DP, false> side;
    side.read(p, w.head, r0, hi);
    side.write(pq, nullptr);
    const bool busy = r0 + 2 * R * (threadIdx.x >> 5) < hi;       // does the warp have a row
    float m[R], l[R];
    uint64_t o[R][Cfg<DP>::DC][2];
#pragma unroll
    for (int i = 0; i < R; ++i) {
      m[i] = -INFINITY;
      l[i] = 0.f;
#pragma unroll
      for (int c = 0; c < Cfg<DP>::DC; ++c) o[i][c][0] = o[i][c][1] = 0;
    }
    Rows<DP> kr, vr;                       // the next moving tile
    auto read = [&](int64_t c0) {
      kr.read(p.k, p.ks, kh, c0, hi, p.D);
      vr.read(p.v, p.vs, kh, c0, hi, p.D);
      side.read(p, w.head, c0, hi);
    };
    if (Cfg<DP>::AHEAD) read(lo);
    for (int64_t c0 = lo; c0 < hi; c0 += B) {
      __syncthreads();
      if (!Cfg<DP>::AHEAD) read(c0);
      kr.write(K, 1.f);
      vr.write(V, 1.f);
      side.write(pk, nullptr);
      __syncthreads();
      if (Cfg<DP>::AHEAD && c0 + B < hi) read(c0 + B);
      if (!busy) continue;
      const int nc = (int)(hi - c0 < B ? hi - c0 : B);
      float s[R][4];
      mm_nt<DP>(Q, K, nc, s);
      float bias[R][4];
      distances(p, pq, pk, slope, bias);
#pragma unroll
      for (int i = 0; i < R; ++i) {
        float top = m[i];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if (p.cap > 0.f) s[i][j] = p.cap * tanh_fast(s[i][j] * icap);
          s[i][j] -= bias[i][j];
          if (c0 + tx + 16 * j >= hi) s[i][j] = -INFINITY;
          top = fmaxf(top, s[i][j]);
        }
#pragma unroll
        for (int x = 8; x > 0; x >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
        const float base = top == -INFINITY ? 0.f : top;
        const float fix = exp_fast(m[i] - base);
        m[i] = top;
        float sum = 0.f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          s[i][j] = exp_fast(s[i][j] - base);
          sum += s[i][j];
          P[(R * ty + i) * LDP + tx + 16 * j] = s[i][j];
        }
        l[i] = l[i] * fix + sum;          // this thread's columns; joined at the end
        const uint64_t fix2 = pk2(fix, fix);
#pragma unroll
        for (int c = 0; c < Cfg<DP>::DC; ++c)
#pragma unroll
          for (int k = 0; k < 2; ++k) o[i][c][k] = ptx::mul2(o[i][c][k], fix2);
      }
      __syncwarp();
      mm_nn<DP>(P, V, nc, o);
      __syncwarp();
    }
    float inv[R];
#pragma unroll
    for (int i = 0; i < R; ++i) {
#pragma unroll
      for (int x = 8; x > 0; x >>= 1) l[i] += __shfl_xor_sync(0xffffffffu, l[i], x);
      inv[i] = 1.f / l[i];
      const int64_t r = r0 + R * ty + i;
      if (tx == 0 && r < hi) p.lse[(int64_t)w.head * p.N + r] = m[i] + logf(l[i]);
    }
    store_rows<DP>(p.o, p.os, qh, r0, hi, p.D, o, inv);
  }
}

// ----------------------------------------------------------------- backward

// P and du of one 64 x 64 tile from its raw products u (rows and columns as in
// mm_nt), dP, and the softmax statistics of the query side.
__device__ __forceinline__ void tile_grad(const Params& p, float u, float dp, float bias, float lse, float delta,
                                          bool on, float icap, float& prob, float& du) {
  float slope_u = 1.f, s = u;
  if (p.cap > 0.f) {
    const float t = tanh_fast(u * icap);
    s = p.cap * t;
    slope_u = 1.f - t * t;
  }
  s -= bias;
  prob = on ? exp_fast(s - lse) : 0.f;
  du = on ? prob * (dp - delta) * slope_u : 0.f;
}

template <int DP>
__global__ void __launch_bounds__(Cfg<DP>::THREADS, DP > 64 ? 1 : 2) attn_simt_dq_kernel(const __grid_constant__ Params p) {
  extern __shared__ __align__(16) float sm[];
  float* Q = sm;
  float* G = Q + Cfg<DP>::TILE;
  float* K = G + Cfg<DP>::TILE;
  float* V = K + Cfg<DP>::TILE;
  float* P = V + Cfg<DP>::TILE;
  float* pq = P + B * LDP;
  float* pk = pq + kMaxAxes * B;
  float* dl = pk + kMaxAxes * B;
  constexpr int R = Cfg<DP>::R;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  grid_dep_launch();
  grid_dep_wait();
  const Work w = work_of_row(p, p.H);
  const int64_t qh = (int64_t)w.head * p.D, kh = (int64_t)(w.head / (p.H / p.K)) * p.D;
  if (w.doc == p.docs) {
    outside_rows(p, w.tile, [&](int64_t r) { clear_row(p.dq, p.dqs, qh, r, p.D); });
    return;
  }
  int64_t lo, hi;
  doc_range(p, w.doc, lo, hi);
  const float slope = p.axes ? p.slopes[w.head] : 0.f;
  const float icap = p.cap > 0.f ? 1.f / p.cap : 0.f;
  for (int64_t r0 = lo + (int64_t)w.tile * B; r0 < hi; r0 += (int64_t)p.hint * B) {
    __syncthreads();
    load_tile<DP>(K, p.o, p.os, qh, r0, hi, p.D, 1.f);   // o, for delta
    load_tile<DP>(G, p.go, p.gos, qh, r0, hi, p.D, 1.f);
    load_tile<DP>(Q, p.q, p.qs, qh, r0, hi, p.D, p.scale);
    Side<DP, false> side;
    side.read(p, w.head, r0, hi);
    side.write(pq, nullptr);
    __syncthreads();
    {   // delta, TR threads a row
      constexpr int TR = Cfg<DP>::THREADS / B;
      const int r = threadIdx.x / TR;
      float d = 0.f;
      for (int c = threadIdx.x % TR; c < DP; c += TR) d = fmaf(G[r * Cfg<DP>::LD + c], K[r * Cfg<DP>::LD + c], d);
#pragma unroll
      for (int x = 1; x < TR; x *= 2) d += __shfl_xor_sync(0xffffffffu, d, x);
      if (threadIdx.x % TR == 0) {
        dl[r] = d;
        if (r0 + r < hi) p.delta[(int64_t)w.head * p.N + r0 + r] = d;
      }
    }
    __syncthreads();
    const bool busy = r0 + 2 * R * (threadIdx.x >> 5) < hi;
    float lse[R], delta[R];
    uint64_t acc[R][Cfg<DP>::DC][2];
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const int64_t r = r0 + R * ty + i;
      lse[i] = r < hi ? p.lse[(int64_t)w.head * p.N + r] : 0.f;
      delta[i] = dl[R * ty + i];
#pragma unroll
      for (int c = 0; c < Cfg<DP>::DC; ++c) acc[i][c][0] = acc[i][c][1] = 0;
    }
    Rows<DP> kr, vr;                       // the next moving tile
    auto read = [&](int64_t c0) {
      kr.read(p.k, p.ks, kh, c0, hi, p.D);
      vr.read(p.v, p.vs, kh, c0, hi, p.D);
      side.read(p, w.head, c0, hi);
    };
    if (Cfg<DP>::AHEAD) read(lo);
    for (int64_t c0 = lo; c0 < hi; c0 += B) {
      __syncthreads();
      if (!Cfg<DP>::AHEAD) read(c0);
      kr.write(K, 1.f);
      vr.write(V, 1.f);
      side.write(pk, nullptr);
      __syncthreads();
      if (Cfg<DP>::AHEAD && c0 + B < hi) read(c0 + B);
      if (!busy) continue;
      const int nc = (int)(hi - c0 < B ? hi - c0 : B);
      float u[R][4], dp[R][4];
      mm_nt<DP>(Q, K, nc, u);
      mm_nt<DP>(G, V, nc, dp);
      float bias[R][4];
      distances(p, pq, pk, slope, bias);
#pragma unroll
      for (int i = 0; i < R; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int c = tx + 16 * j, r = R * ty + i;
          float prob, du;
          tile_grad(p, u[i][j], dp[i][j], bias[i][j], lse[i], delta[i], r0 + r < hi && c0 + c < hi, icap, prob, du);
          P[r * LDP + c] = du;
        }
      __syncwarp();
      mm_nn<DP>(P, K, nc, acc);
      __syncwarp();
    }
    float mul[R];
#pragma unroll
    for (int i = 0; i < R; ++i) mul[i] = p.scale;
    store_rows<DP>(p.dq, p.dqs, qh, r0, hi, p.D, acc, mul);
  }
}

template <int DP>
__global__ void __launch_bounds__(Cfg<DP>::THREADS, DP > 64 ? 1 : 2) attn_simt_dkv_kernel(const __grid_constant__ Params p) {
  extern __shared__ __align__(16) float sm[];
  float* K = sm;
  float* V = K + Cfg<DP>::TILE;
  float* Q = V + Cfg<DP>::TILE;
  float* G = Q + Cfg<DP>::TILE;
  float* P = G + Cfg<DP>::TILE;
  float* pq = P + B * LDP;
  float* pk = pq + kMaxAxes * B;
  float* stat = pk + kMaxAxes * B;         // lse [64], delta [64]
  constexpr int R = Cfg<DP>::R;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  grid_dep_launch();
  grid_dep_wait();
  const Work w = work_of_row(p, p.K);
  const int rep = p.H / p.K;
  const int64_t kh = (int64_t)w.head * p.D;
  if (w.doc == p.docs) {
    outside_rows(p, w.tile, [&](int64_t r) {
      clear_row(p.dk, p.dks, kh, r, p.D);
      clear_row(p.dv, p.dvs, kh, r, p.D);
    });
    return;
  }
  int64_t lo, hi;
  doc_range(p, w.doc, lo, hi);
  const float icap = p.cap > 0.f ? 1.f / p.cap : 0.f;
  for (int64_t r0 = lo + (int64_t)w.tile * B; r0 < hi; r0 += (int64_t)p.hint * B) {
    __syncthreads();
    load_tile<DP>(K, p.k, p.ks, kh, r0, hi, p.D, 1.f);
    load_tile<DP>(V, p.v, p.vs, kh, r0, hi, p.D, 1.f);
    Side<DP, true> side;
    side.read(p, w.head * rep, r0, hi);
    side.write(pk, stat);                  // stat comes with each moving tile
    const bool busy = r0 + 2 * R * (threadIdx.x >> 5) < hi;
    uint64_t dk[R][Cfg<DP>::DC][2], dv[R][Cfg<DP>::DC][2];
#pragma unroll
    for (int i = 0; i < R; ++i)
#pragma unroll
      for (int c = 0; c < Cfg<DP>::DC; ++c)
#pragma unroll
        for (int k = 0; k < 2; ++k) dk[i][c][k] = dv[i][c][k] = 0;
    Rows<DP> qr, gr;                       // the next moving tile
    auto read = [&](int head, int64_t c0) {
      qr.read(p.q, p.qs, (int64_t)head * p.D, c0, hi, p.D);
      gr.read(p.go, p.gos, (int64_t)head * p.D, c0, hi, p.D);
      side.read(p, head, c0, hi);
    };
    if (Cfg<DP>::AHEAD) read(w.head * rep, lo);
    for (int g = 0; g < rep; ++g) {
      const int head = w.head * rep + g;
      const float slope = p.axes ? p.slopes[head] : 0.f;
      for (int64_t c0 = lo; c0 < hi; c0 += B) {
        __syncthreads();
        if (!Cfg<DP>::AHEAD) read(head, c0);
        qr.write(Q, p.scale);
        gr.write(G, 1.f);
        side.write(pq, stat);
        __syncthreads();
        if (Cfg<DP>::AHEAD && c0 + B < hi) read(head, c0 + B);
        else if (Cfg<DP>::AHEAD && g + 1 < rep) read(head + 1, lo);
        if (!busy) continue;
        const int nc = (int)(hi - c0 < B ? hi - c0 : B);
        float u[R][4], dp[R][4];
        mm_nt<DP>(K, Q, nc, u);
        mm_nt<DP>(V, G, nc, dp);
        float bias[R][4];
        distances(p, pk, pq, slope, bias);
#pragma unroll
        for (int i = 0; i < R; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int c = tx + 16 * j, r = R * ty + i;
            float prob, du;
            tile_grad(p, u[i][j], dp[i][j], bias[i][j], stat[c], stat[B + c], r0 + r < hi && c0 + c < hi, icap, prob,
                      du);
            P[r * LDP + c] = prob;
            dp[i][j] = du;
          }
        __syncwarp();
        mm_nn<DP>(P, G, nc, dv);
        __syncwarp();
#pragma unroll
        for (int i = 0; i < R; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) P[(R * ty + i) * LDP + tx + 16 * j] = dp[i][j];
        __syncwarp();
        mm_nn<DP>(P, Q, nc, dk);           // Q carries the scale
        __syncwarp();
      }
    }
    float one[R];
#pragma unroll
    for (int i = 0; i < R; ++i) one[i] = 1.f;
    store_rows<DP>(p.dk, p.dks, kh, r0, hi, p.D, dk, one);
    store_rows<DP>(p.dv, p.dvs, kh, r0, hi, p.D, dv, one);
  }
}

// ------------------------------------------------------------------- launch

template <int DP> constexpr int smem_bytes(int tiles) {
  return (tiles * Cfg<DP>::TILE + B * LDP + 2 * kMaxAxes * B + 2 * B) * (int)sizeof(float);
}

cudaError_t run(void (*k)(Params), int smem, int threads, Params p, int heads, cudaStream_t st) {
  const int64_t longest = p.len;           // the document length that sets the blocks per head
  int64_t tiles = (longest + B - 1) / B;
  if (tiles < 1) tiles = 1;
  const int64_t items = (p.docs + (p.offsets ? 1 : 0)) * heads;
  if (items == 0) return cudaSuccess;
  if (items > 0x7fffffff) return cudaErrorInvalidValue;
  const int64_t room = 0x7fffffff / items;
  p.hint = (int)(tiles < room ? tiles : room);
  p.items = (uint32_t)(items * p.hint);
  cudaError_t e = set_smem_limit(reinterpret_cast<const void*>(k), smem);
  if (e == cudaSuccess) e = launch_pdl(k, dim3(p.items), dim3(threads), (size_t)smem, st, p);
  if (e == cudaSuccess) count_launches(1);
  return e;
}

template <int DP>
cudaError_t forward(const Params& p, cudaStream_t st) {
  return run(attn_simt_fwd_kernel<DP>, smem_bytes<DP>(3), Cfg<DP>::THREADS, p, p.H, st);
}
template <int DP>
cudaError_t backward(const Params& p, cudaStream_t st) {
  const cudaError_t e = run(attn_simt_dq_kernel<DP>, smem_bytes<DP>(4), Cfg<DP>::THREADS, p, p.H, st);
  return e != cudaSuccess ? e : run(attn_simt_dkv_kernel<DP>, smem_bytes<DP>(4), Cfg<DP>::THREADS, p, p.K, st);
}

cudaError_t dispatch(const Params& p, bool bwd, cudaStream_t st) {
  if (p.D <= 32) return bwd ? backward<32>(p, st) : forward<32>(p, st);
  if (p.D <= 64) return bwd ? backward<64>(p, st) : forward<64>(p, st);
  return bwd ? backward<128>(p, st) : forward<128>(p, st);
}

}  // namespace attn_simt

cudaError_t launch_attn_simt_forward(const attn::Params& p, cudaStream_t st) { return attn_simt::dispatch(p, false, st); }
cudaError_t launch_attn_simt_backward(const attn::Params& p, cudaStream_t st) { return attn_simt::dispatch(p, true, st); }

}  // namespace eqlin
