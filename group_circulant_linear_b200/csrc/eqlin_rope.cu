// eqlin_rope.cu -- rotary positions with several axes, on equivariant heads.
//
// A head's features are [Ch, T], index c*T + t.  Channel i < Ch/2 forms a
// plane with channel i + Ch/2, at every group position t, and is turned by
// the angle a_i = pos[n, axis_i] * f_i:
//
//   y1 = x1 cos a_i - x2 sin a_i,    y2 = x2 cos a_i + x1 sin a_i
//
// The angle does not depend on t, so the operator commutes with a cyclic
// shift of the group axis.  Each axis (time, height, width) owns a run of
// channels; channels past the last run are copied.  The inverse turns by
// -a_i, which is also the gradient (the map is orthogonal).
//
// Angles of far positions: a product pos * f in FP32 is off by up to half a
// unit in its last place, 0.004 rad at an angle of 1e5.  So frequencies are
// kept in turns (f / 2 pi) as two floats hi + lo of the 64-bit value, the
// product's rounding error is recovered with one FMA, whole turns are removed
// exactly, and sincospi takes the remainder: 1e-7 turns up to 2^23 turns.
//
// Bound by memory: one read and one write of the rotated heads.  A thread
// keeps one vector of channels of one token, works out its sines once, and
// walks HPT heads with them, so all HPT x 2 loads are in flight together.
// 25088 tokens, 24 heads of 64 in f16: 25.4 us, 6.1 TB/s, 0.94 of a copy.
#include <math.h>
#include <new>

#include "eqlin_internal.cuh"

namespace eqlin {
namespace rope {

constexpr int kMaxPairs = 128;
constexpr int kMaxAxes = 4;
constexpr int kThreads = 256;
constexpr int HPT = 4;

// The plan lives in host memory and travels with each launch (1.2 KB of
// kernel parameters), so it belongs to no device or stream.
struct Plan {
  int T, Ch, axes;
  float hi[kMaxPairs], lo[kMaxPairs];      // turns per unit of position
  int8_t axis[kMaxPairs];                  // -1: copied
};

struct Params {
  const float* pos;
  const void* src;
  void* dst;
  int64_t src_stride, dst_stride;          // elements per token
  int64_t N;
  int heads;
  int nvec;                                // vectors per half head
  int groups;                              // ceil(heads / HPT)
  int tokens;                              // tokens per block
  float sign;
};

template <int B> struct Raw;
template <> struct Raw<16> { using type = uint4; };
template <> struct Raw<8> { using type = uint2; };
template <> struct Raw<4> { using type = uint32_t; };
template <> struct Raw<2> { using type = uint16_t; };

// V elements of type E per vector; TT as in the norm: neighbouring elements
// known to share a channel.
template <typename E, int V, int TT>
__global__ void __launch_bounds__(kThreads) rope_kernel(const __grid_constant__ Plan plan,
                                                        const __grid_constant__ Params p) {
  using R = typename Raw<V * (int)sizeof(E)>::type;
  constexpr int CG = V / TT;
  const int per = p.nvec * p.groups;       // threads per token
  const int half = plan.Ch / 2 * plan.T;
  grid_dep_launch();
  grid_dep_wait();
  for (int item = threadIdx.x; item < p.tokens * per; item += kThreads) {
    const int tok = item / per, rest = item - tok * per;
    const int group = rest / p.nvec, vec = rest - group * p.nvec;
    const int64_t n = (int64_t)blockIdx.x * p.tokens + tok;
    if (n >= p.N) break;
    const int h0 = group * HPT, h1 = min(h0 + HPT, p.heads);
    const E* src = static_cast<const E*>(p.src) + n * p.src_stride + (int64_t)h0 * 2 * half + vec * V;
    E* dst = static_cast<E*>(p.dst) + n * p.dst_stride + (int64_t)h0 * 2 * half + vec * V;
    R a[HPT], b[HPT];
#pragma unroll
    for (int h = 0; h < HPT; ++h)
      if (h0 + h < h1) {
        a[h] = *reinterpret_cast<const R*>(src + h * 2 * half);
        b[h] = *reinterpret_cast<const R*>(src + h * 2 * half + half);
      }
    float c[CG], s[CG];
    bool turn[CG];
#pragma unroll
    for (int i = 0; i < CG; ++i) {
      const int ch = (vec * V + i * TT) / plan.T;
      const int ax = plan.axis[ch];
      turn[i] = ax >= 0;
      c[i] = 1.f;
      s[i] = 0.f;
      if (ax >= 0) {
        const float x = p.pos[n * plan.axes + ax];
        const float t = x * plan.hi[ch];
        const float err = fmaf(x, plan.hi[ch], -t);
        const float r = (t - rintf(t)) + fmaf(x, plan.lo[ch], err);
        sincospif(2.f * r, &s[i], &c[i]);
        s[i] *= p.sign;
      }
    }
#pragma unroll
    for (int h = 0; h < HPT; ++h)
      if (h0 + h < h1) {
        E* x1 = reinterpret_cast<E*>(&a[h]);
        E* x2 = reinterpret_cast<E*>(&b[h]);
#pragma unroll
        for (int i = 0; i < V; ++i) {
          if (!turn[i / TT]) continue;     // copied bit for bit: a product with 0 would spread an infinity
          const float u = Elem<E>::to_f(x1[i]), v = Elem<E>::to_f(x2[i]);
          x1[i] = Elem<E>::from_f(u * c[i / TT] - v * s[i / TT]);
          x2[i] = Elem<E>::from_f(v * c[i / TT] + u * s[i / TT]);
        }
        *reinterpret_cast<R*>(dst + h * 2 * half) = a[h];
        *reinterpret_cast<R*>(dst + h * 2 * half + half) = b[h];
      }
  }
}

template <typename E, int V>
cudaError_t launch(const Plan& plan, Params p, cudaStream_t st) {
  p.nvec = plan.Ch / 2 * plan.T / V;
  p.groups = (p.heads + HPT - 1) / HPT;
  const int64_t per = (int64_t)p.nvec * p.groups;
  p.tokens = per >= kThreads ? 1 : (int)(kThreads / per);
  const int64_t blocks = (p.N + p.tokens - 1) / p.tokens;
  if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
  void (*k)(Plan, Params) = rope_kernel<E, V, 1>;
  if constexpr (V >= 4) {
    if (plan.T % 4 == 0) k = rope_kernel<E, V, 4>;
  }
  const cudaError_t e = launch_pdl(k, dim3((unsigned)blocks), dim3(kThreads), 0, st, plan, p);
  if (e == cudaSuccess) count_launches(1);
  return e;
}

// The widest vector that the half head, the strides and the pointers allow.
template <typename E>
cudaError_t dispatch(const Plan& plan, const Params& p, cudaStream_t st) {
  const uint64_t bits = (uint64_t)(uintptr_t)p.src | (uint64_t)(uintptr_t)p.dst |
                        (uint64_t)(p.src_stride * (int64_t)sizeof(E)) | (uint64_t)(p.dst_stride * (int64_t)sizeof(E)) |
                        (uint64_t)(plan.Ch / 2 * plan.T * (int)sizeof(E));
  if (bits % 16 == 0) return launch<E, 16 / sizeof(E)>(plan, p, st);
  if (bits % 8 == 0) return launch<E, 8 / sizeof(E)>(plan, p, st);
  if constexpr (sizeof(E) == 2) {
    if (bits % 4 == 0) return launch<E, 2>(plan, p, st);
  }
  return launch<E, 1>(plan, p, st);
}

}  // namespace rope
}  // namespace eqlin

using namespace eqlin;

struct eqlin_rope {
  rope::Plan plan;
};

extern "C" eqlin_status_t eqlin_rope_create(int T, int64_t Ch, int axes, const int64_t* sections, const double* freqs,
                                            eqlin_rope_t* out) {
  if (!out || !sections || T < 1 || Ch < 2 || axes < 1) return EQLIN_ERR_INVALID_ARG;
  if (Ch % 2) return EQLIN_ERR_INVALID_ARG;
  if (T > 16 || Ch > 2 * rope::kMaxPairs || axes > rope::kMaxAxes) return EQLIN_ERR_UNSUPPORTED;
  int64_t pairs = 0;
  for (int a = 0; a < axes; ++a) {
    if (sections[a] < 0 || sections[a] > Ch / 2) return EQLIN_ERR_INVALID_ARG;
    pairs += sections[a];
  }
  if (pairs > Ch / 2 || (pairs > 0 && !freqs)) return EQLIN_ERR_INVALID_ARG;
  for (int64_t i = 0; i < pairs; ++i)
    if (!isfinite(freqs[i])) return EQLIN_ERR_INVALID_ARG;
  eqlin_rope* r = new (std::nothrow) eqlin_rope;
  if (!r) return EQLIN_ERR_OOM;
  r->plan = rope::Plan{};
  r->plan.T = T;
  r->plan.Ch = (int)Ch;
  r->plan.axes = axes;
  int i = 0;
  for (int a = 0; a < axes; ++a)
    for (int64_t k = 0; k < sections[a]; ++k, ++i) {
      const double turns = freqs[i] / 6.283185307179586476925286766559;
      r->plan.hi[i] = (float)turns;
      r->plan.lo[i] = (float)(turns - (double)r->plan.hi[i]);
      r->plan.axis[i] = (int8_t)a;
    }
  for (; i < rope::kMaxPairs; ++i) r->plan.axis[i] = -1;
  *out = r;
  return EQLIN_OK;
}

extern "C" void eqlin_rope_destroy(eqlin_rope_t r) { delete r; }

extern "C" eqlin_status_t eqlin_rope_apply(eqlin_rope_t r, eqlin_dtype_t dtype, const float* pos, const void* src,
                                           int64_t src_stride, void* dst, int64_t dst_stride, int64_t heads,
                                           int inverse, int64_t N, void* stream) {
  if (!r || (dtype != EQLIN_F32 && dtype != EQLIN_F16 && dtype != EQLIN_BF16)) return EQLIN_ERR_INVALID_ARG;
  if (N < 0 || heads < 1) return EQLIN_ERR_INVALID_ARG;
  if (heads > 65536) return EQLIN_ERR_UNSUPPORTED;
  const int64_t width = heads * r->plan.Ch * r->plan.T;
  if (src_stride < width || dst_stride < width) return EQLIN_ERR_INVALID_ARG;
  if (N == 0) return EQLIN_OK;
  if (!pos || !src || !dst || (src == dst && src_stride != dst_stride)) return EQLIN_ERR_INVALID_ARG;
  const int64_t es = dtype == EQLIN_F32 ? 4 : 2;
  if ((uintptr_t)src % es || (uintptr_t)dst % es || (uintptr_t)pos % 4) return EQLIN_ERR_MISALIGNED;
  rope::Params p = {};
  p.pos = pos;
  p.src = src;
  p.dst = dst;
  p.src_stride = src_stride;
  p.dst_stride = dst_stride;
  p.N = N;
  p.heads = (int)heads;
  p.sign = inverse ? -1.f : 1.f;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  switch (dtype) {
    case EQLIN_F32: e = rope::dispatch<float>(r->plan, p, st); break;
    case EQLIN_F16: e = rope::dispatch<__half>(r->plan, p, st); break;
    default: e = rope::dispatch<__nv_bfloat16>(r->plan, p, st); break;
  }
  return e == cudaSuccess ? EQLIN_OK : EQLIN_ERR_CUDA;
}
