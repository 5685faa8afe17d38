// Layer norm and RMS norm over rows, forward and backward.
//   y = (x - mean) r w + b,  r = 1 / sqrt(mean((x - mean)^2) + eps)
//   g = dy w, h = (x - mean) r:  dx = r (g - mean(g) - h mean(g h)),
//   dw = sum_rows dy h,  db = sum_rows dy            (RMS: mean = 0, no b)
// Bound by memory: the forward reads x and writes y, the backward reads x and
// dy and writes dx, each once; a row stays in registers between its sums and
// its output. The backward's CTAs walk over the rows and keep dw and db of
// their columns in registers, so that x and dy are not read again for the
// column sums: those leave one partial row pair a CTA, joined in a fixed order.
#include <cuda_bf16.h>

#include "internal.h"

namespace grpo {

namespace {

template <typename T>
__device__ __forceinline__ float ldf(const T* p, int64_t i);
template <>
__device__ __forceinline__ float ldf<float>(const float* p, int64_t i) {
  return p[i];
}
template <>
__device__ __forceinline__ float ldf<__nv_bfloat16>(const __nv_bfloat16* p, int64_t i) {
  return __bfloat162float(p[i]);
}
__device__ __forceinline__ void stf(float* p, int64_t i, float v) { p[i] = v; }
__device__ __forceinline__ void stf(__nv_bfloat16* p, int64_t i, float v) {
  p[i] = __float2bfloat16_rn(v);
}

// Piece of N consecutive values: one access of N elements, 16 bytes at most.
template <typename T, int N>
struct Piece;
template <>
struct Piece<float, 4> {
  uint4 raw;
  __device__ __forceinline__ float get(int e) const {
    return __uint_as_float(e == 0 ? raw.x : e == 1 ? raw.y : e == 2 ? raw.z : raw.w);
  }
  __device__ __forceinline__ void set(const float* v) {
    raw = make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
  }
};
template <>
struct Piece<float, 1> {
  uint32_t raw;
  __device__ __forceinline__ float get(int) const { return __uint_as_float(raw); }
  __device__ __forceinline__ void set(const float* v) { raw = __float_as_uint(v[0]); }
};
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 p = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&p);
}
template <>
struct Piece<__nv_bfloat16, 8> {
  uint4 raw;
  __device__ __forceinline__ float get(int e) const {
    const uint32_t w = e < 2 ? raw.x : e < 4 ? raw.y : e < 6 ? raw.z : raw.w;
    return __uint_as_float((e & 1) ? (w & 0xFFFF0000u) : (w << 16));
  }
  __device__ __forceinline__ void set(const float* v) {
    raw = make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
  }
};
template <>
struct Piece<__nv_bfloat16, 4> {
  uint2 raw;
  __device__ __forceinline__ float get(int e) const {
    const uint32_t w = e < 2 ? raw.x : raw.y;
    return __uint_as_float((e & 1) ? (w & 0xFFFF0000u) : (w << 16));
  }
  __device__ __forceinline__ void set(const float* v) {
    raw = make_uint2(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]));
  }
};
template <>
struct Piece<__nv_bfloat16, 1> {
  unsigned short raw;
  __device__ __forceinline__ float get(int) const {
    return __uint_as_float(static_cast<uint32_t>(raw) << 16);
  }
  __device__ __forceinline__ void set(const float* v) {
    raw = __bfloat16_as_ushort(__float2bfloat16_rn(v[0]));
  }
};
template <typename T, int N>
__device__ __forceinline__ Piece<T, N> load_piece(const T* p) {
  return *reinterpret_cast<const Piece<T, N>*>(p);
}
template <typename T, int N>
__device__ __forceinline__ void store_piece(T* p, const Piece<T, N>& v) {
  *reinterpret_cast<Piece<T, N>*>(p) = v;
}

// Sum of (a, b) over a group of G threads (a power of two from 32 on that
// divides the CTA), returned to each of them. `slot` alternates between calls,
// so that one barrier a call is enough.
template <int G, bool BOTH>
__device__ __forceinline__ float2 group_sum(float a, float b, float2* part, int slot) {
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) {
    a += __shfl_xor_sync(0xffffffffu, a, o);
    if (BOTH) b += __shfl_xor_sync(0xffffffffu, b, o);
  }
  if (G == 32) return make_float2(a, b);
  const int warp = threadIdx.x >> 5, first = warp / (G / 32) * (G / 32);
  float2* mine = part + slot * 32;
  if ((threadIdx.x & 31) == 0) mine[warp] = make_float2(a, b);
  __syncthreads();
  a = b = 0.f;
#pragma unroll
  for (int w = 0; w < G / 32; ++w) {
    const float2 p = mine[first + w];
    a += p.x;
    if (BOTH) b += p.y;
  }
  return make_float2(a, b);
}

// ---------------------------------------------------------------- forward
// A group of G threads takes a row, R rows a CTA; each thread holds NV pieces of
// N values of it (G N NV >= d).
template <typename T, typename P, int N, int NV, int G, int R>
__global__ void __launch_bounds__(G * R) k_norm_fwd(NormArgs a) {
  __shared__ float2 part[2 * 32];
  const int tid = threadIdx.x % G;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * R + threadIdx.x / G;
  const bool live = row < a.rows;  // every thread takes part in the barriers
  const int d = static_cast<int>(a.d);
  const T* x = static_cast<const T*>(a.x) + (live ? row : 0) * a.ld_x;
  Piece<T, N> v[NV];
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    const int i = (k * G + tid) * N;
    if (i < d) v[k] = load_piece<T, N>(x + i);
  }
  const float inv_d = 1.f / d;
  float mean = 0.f;
  if (!a.rms) {
    float s = 0.f;
#pragma unroll
    for (int k = 0; k < NV; ++k)
      if ((k * G + tid) * N < d)
#pragma unroll
        for (int e = 0; e < N; ++e) s += v[k].get(e);
    mean = group_sum<G, false>(s, 0.f, part, 0).x * inv_d;
  }
  float q = 0.f;
#pragma unroll
  for (int k = 0; k < NV; ++k)
    if ((k * G + tid) * N < d)
#pragma unroll
      for (int e = 0; e < N; ++e) {
        const float c = v[k].get(e) - mean;
        q = fmaf(c, c, q);
      }
  const float r = rsqrtf(group_sum<G, false>(q, 0.f, part, 1).x * inv_d + a.eps);
  if (!live) return;
  T* y = static_cast<T*>(a.y) + row * a.ld_y;
  const P* w = static_cast<const P*>(a.weight);
  const P* b = static_cast<const P*>(a.bias);
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    const int i = (k * G + tid) * N;
    if (i < d) {
      float o[N];
#pragma unroll
      for (int e = 0; e < N; ++e) o[e] = (v[k].get(e) - mean) * r;
      if (N == 8 || N == 4) {
        constexpr int M = N > 1 && sizeof(P) == 4 ? 4 : N;  // of a 16-byte load at most
#pragma unroll
        for (int e = 0; e < N; e += M) {
          const Piece<P, M> ww = load_piece<P, M>(w + i + e);
#pragma unroll
          for (int f = 0; f < M; ++f) o[e + f] *= ww.get(f);
          if (b) {
            const Piece<P, M> bb = load_piece<P, M>(b + i + e);
#pragma unroll
            for (int f = 0; f < M; ++f) o[e + f] += bb.get(f);
          }
        }
      } else {
#pragma unroll
        for (int e = 0; e < N; ++e) o[e] = b ? fmaf(o[e], ldf(w, i + e), ldf(b, i + e)) : o[e] * ldf(w, i + e);
      }
      Piece<T, N> p;
      p.set(o);
      store_piece<T, N>(y + i, p);
    }
  }
  if (tid == 0) {
    if (a.mean) a.mean[row] = mean;
    if (a.rstd) a.rstd[row] = r;
  }
}

// --------------------------------------------------------------- backward
// A CTA of G threads walks over rows blockIdx.x, + gridDim.x, ...; each thread
// holds NV pieces of N columns: their values of a row and their column sums.
// The next row is loaded before this one's sums are joined.
template <typename T, typename P, int N, int NV, int G>
__global__ void __launch_bounds__(G) k_norm_bwd(NormArgs a) {
  __shared__ float2 part[2 * 32];
  const int tid = threadIdx.x, d = static_cast<int>(a.d);
  const T* x = static_cast<const T*>(a.x);
  const T* dy = static_cast<const T*>(a.dy);
  const P* w = static_cast<const P*>(a.weight);
  float dw[NV][N], db[NV][N];
#pragma unroll
  for (int k = 0; k < NV; ++k)
#pragma unroll
    for (int e = 0; e < N; ++e) dw[k][e] = db[k][e] = 0.f;
  Piece<T, N> xv[NV], gv[NV];
  float mean = 0.f, r = 0.f;
  auto fetch = [&](int64_t row) {
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int i = (k * G + tid) * N;
      if (i < d) {
        xv[k] = load_piece<T, N>(x + row * a.ld_x + i);
        gv[k] = load_piece<T, N>(dy + row * a.ld_dy + i);
      }
    }
    mean = a.rms ? 0.f : a.mean[row];
    r = a.rstd[row];
  };
  const float inv_d = 1.f / d;
  int slot = 0;
  int64_t row = blockIdx.x;
  if (row < a.rows) fetch(row);
  for (; row < a.rows; row += gridDim.x) {
    float sg = 0.f, sgh = 0.f;
    Piece<T, N> x0[NV], g0[NV];
    const float m0 = mean, r0 = r;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      x0[k] = xv[k];
      g0[k] = gv[k];
    }
    if (row + gridDim.x < a.rows) fetch(row + gridDim.x);
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int i = (k * G + tid) * N;
      if (i < d) {
#pragma unroll
        for (int e = 0; e < N; ++e) {
          const float g = g0[k].get(e), h = (x0[k].get(e) - m0) * r0;
          dw[k][e] = fmaf(g, h, dw[k][e]);
          db[k][e] += g;
          const float gw = g * ldf(w, i + e);
          sg += gw;
          sgh = fmaf(gw, h, sgh);
        }
      }
    }
    float2 s = group_sum<G, true>(sg, sgh, part, slot);
    slot ^= 1;
    s.x = a.rms ? 0.f : s.x * inv_d;
    s.y *= inv_d;
    T* dx = static_cast<T*>(a.dx) + row * a.ld_dx;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int i = (k * G + tid) * N;
      if (i < d) {
        float o[N];
#pragma unroll
        for (int e = 0; e < N; ++e) {
          const float gw = g0[k].get(e) * ldf(w, i + e), h = (x0[k].get(e) - m0) * r0;
          o[e] = r0 * (gw - s.x - h * s.y);
        }
        Piece<T, N> p;
        p.set(o);
        store_piece<T, N>(dx + i, p);
      }
    }
  }
  if (!a.partial) return;
  float* pw = a.partial + 2 * static_cast<int64_t>(blockIdx.x) * d;
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    const int i = (k * G + tid) * N;
    if (i < d) {
#pragma unroll
      for (int e = 0; e < N; ++e) {
        pw[i + e] = dw[k][e];
        pw[d + i + e] = db[k][e];
      }
    }
  }
}

// Rows too long for registers: three passes, the later ones from cache.
constexpr int kLong = 1024;
template <typename T, typename P>
__global__ void __launch_bounds__(kLong) k_norm_fwd_long(NormArgs a) {
  __shared__ float2 part[2 * 32];
  const int64_t row = blockIdx.x;
  const T* x = static_cast<const T*>(a.x) + row * a.ld_x;
  T* y = static_cast<T*>(a.y) + row * a.ld_y;
  const P* w = static_cast<const P*>(a.weight);
  const P* b = static_cast<const P*>(a.bias);
  const int d = static_cast<int>(a.d);
  float mean = 0.f;
  if (!a.rms) {
    float s = 0.f;
    for (int i = threadIdx.x; i < d; i += kLong) s += ldf(x, i);
    mean = group_sum<kLong, false>(s, 0.f, part, 0).x / d;
  }
  float q = 0.f;
  for (int i = threadIdx.x; i < d; i += kLong) {
    const float c = ldf(x, i) - mean;
    q = fmaf(c, c, q);
  }
  const float r = rsqrtf(group_sum<kLong, false>(q, 0.f, part, 1).x / d + a.eps);
  for (int i = threadIdx.x; i < d; i += kLong) {
    float v = (ldf(x, i) - mean) * r * ldf(w, i);
    if (b) v += ldf(b, i);
    stf(y, i, v);
  }
  if (threadIdx.x == 0) {
    if (a.mean) a.mean[row] = mean;
    if (a.rstd) a.rstd[row] = r;
  }
}

// The same for the backward; the column sums are in the partial rows of the CTA
// from its first row on.
template <typename T, typename P>
__global__ void __launch_bounds__(kLong) k_norm_bwd_long(NormArgs a) {
  __shared__ float2 part[2 * 32];
  const int d = static_cast<int>(a.d);
  const P* w = static_cast<const P*>(a.weight);
  float* pw = a.partial ? a.partial + 2 * static_cast<int64_t>(blockIdx.x) * d : nullptr;
  int slot = 0;
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const T* x = static_cast<const T*>(a.x) + row * a.ld_x;
    const T* dy = static_cast<const T*>(a.dy) + row * a.ld_dy;
    T* dx = static_cast<T*>(a.dx) + row * a.ld_dx;
    const float mean = a.rms ? 0.f : a.mean[row], r = a.rstd[row];
    const bool first = row == blockIdx.x;
    float sg = 0.f, sgh = 0.f;
    for (int i = threadIdx.x; i < d; i += kLong) {
      const float g = ldf(dy, i), h = (ldf(x, i) - mean) * r, gw = g * ldf(w, i);
      sg += gw;
      sgh = fmaf(gw, h, sgh);
      if (pw) {
        pw[i] = fmaf(g, h, first ? 0.f : pw[i]);
        pw[d + i] = g + (first ? 0.f : pw[d + i]);
      }
    }
    float2 s = group_sum<kLong, true>(sg, sgh, part, slot);
    slot ^= 1;
    s.x = a.rms ? 0.f : s.x / d;
    s.y /= d;
    for (int i = threadIdx.x; i < d; i += kLong) {
      const float gw = ldf(dy, i) * ldf(w, i);
      stf(dx, i, r * (gw - s.x - (ldf(x, i) - mean) * r * s.y));
    }
  }
}

// Joins the partial column sums: 32 columns a CTA, the warps take every eighth
// part, and add up in a fixed order.
__global__ void __launch_bounds__(256) k_norm_colsum(NormArgs a, int parts) {
  __shared__ float2 s[8][33];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t col = static_cast<int64_t>(blockIdx.x) * 32 + lane;
  float sw = 0.f, sb = 0.f;
  if (col < a.d) {
#pragma unroll 4
    for (int p = warp; p < parts; p += 8) {
      const float* q = a.partial + 2 * static_cast<int64_t>(p) * a.d + col;
      sw += q[0];
      sb += q[a.d];
    }
  }
  s[warp][lane] = make_float2(sw, sb);
  __syncthreads();
  if (warp == 0 && col < a.d) {
    for (int k = 1; k < 8; ++k) {
      sw += s[k][lane].x;
      sb += s[k][lane].y;
    }
    if (a.dweight) a.dweight[col] = sw;
    if (a.dbias) a.dbias[col] = sb;
  }
}

// How a row is spread over threads: pieces of N values if every row starts on a
// 16-byte boundary and d is whole pieces, else single values.
struct Shape {
  int n;       // values a piece: 16 bytes, or 1
  int pieces;  // of a row
};
Shape shape_of(const NormArgs& a, bool fwd) {
  const int es = a.bf16 ? 2 : 4, vec = 16 / es, ps = a.param_bf16 ? 2 : 4;
  auto on16 = [&](const void* p, int64_t ld, int size) {
    return reinterpret_cast<uintptr_t>(p) % 16 == 0 && ld * size % 16 == 0;
  };
  bool ok = a.d % vec == 0 && on16(a.x, a.ld_x, es) && on16(a.weight, 0, ps);
  if (fwd) ok = ok && on16(a.y, a.ld_y, es) && on16(a.bias, 0, ps);
  else ok = ok && on16(a.dy, a.ld_dy, es) && on16(a.dx, a.ld_dx, es);
  Shape s;
  s.n = ok ? vec : 1;
  s.pieces = static_cast<int>((a.d + s.n - 1) / s.n);
  return s;
}

template <typename T, typename P, int N, int NV, int G, int R>
cudaError_t fwd(const NormArgs& a, cudaStream_t s) {
  const unsigned grid = static_cast<unsigned>((a.rows + R - 1) / R);
  k_norm_fwd<T, P, N, NV, G, R><<<grid, G * R, 0, s>>>(a);
  return cudaGetLastError();
}
template <typename T, typename P, int N>
cudaError_t fwd_n(const NormArgs& a, int pieces, cudaStream_t s) {
  if (pieces <= 32) return fwd<T, P, N, 1, 32, 4>(a, s);
  if (pieces <= 64) return fwd<T, P, N, 2, 32, 4>(a, s);
  if (pieces <= 128) return fwd<T, P, N, 4, 32, 4>(a, s);
  if (pieces <= 256) return fwd<T, P, N, 2, 128, 1>(a, s);
  if (pieces <= 512) return fwd<T, P, N, 4, 128, 1>(a, s);
  if (pieces <= 1024) return fwd<T, P, N, 4, 256, 1>(a, s);
  if (pieces <= 2048) return fwd<T, P, N, 4, 512, 1>(a, s);
  if (pieces <= 4096) return fwd<T, P, N, 4, 1024, 1>(a, s);
  if (pieces <= 8192) return fwd<T, P, N, 8, 1024, 1>(a, s);
  k_norm_fwd_long<T, P><<<static_cast<unsigned>(a.rows), kLong, 0, s>>>(a);
  return cudaGetLastError();
}

template <typename T, typename P, int N, int NV, int G>
cudaError_t bwd(const NormArgs& a, int parts, cudaStream_t s) {
  k_norm_bwd<T, P, N, NV, G><<<parts, G, 0, s>>>(a);
  return cudaGetLastError();
}
template <typename T, typename P, int N>
cudaError_t bwd_n(const NormArgs& a, int pieces, int parts, cudaStream_t s) {
  if (pieces <= 64) return bwd<T, P, N, 1, 64>(a, parts, s);
  if (pieces <= 128) return bwd<T, P, N, 1, 128>(a, parts, s);
  if (pieces <= 256) return bwd<T, P, N, 1, 256>(a, parts, s);
  if (pieces <= 384) return bwd<T, P, N, 1, 384>(a, parts, s);
  if (pieces <= 512) return bwd<T, P, N, 1, 512>(a, parts, s);
  if (pieces <= 768) return bwd<T, P, N, 1, 768>(a, parts, s);
  if (pieces <= 1024) return bwd<T, P, N, 1, 1024>(a, parts, s);
  if constexpr (N == 1) {
    if (pieces <= 2048) return bwd<T, P, N, 2, 1024>(a, parts, s);
    if (pieces <= 4096) return bwd<T, P, N, 4, 1024>(a, parts, s);
  }
  k_norm_bwd_long<T, P><<<parts, kLong, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace

int norm_parts(const NormArgs& a, int sms) {
  const int most = (a.d <= 4096 ? 4 : 2) * sms;
  return static_cast<int>(a.rows < 1 ? 1 : a.rows < most ? a.rows : most);
}

// The statements after `a` for the element types T and P of `a`.
#define NORM_TYPES(a, ...)                                         \
  do {                                                             \
    if ((a).bf16) {                                                \
      using T = __nv_bfloat16;                                     \
      if ((a).param_bf16) { using P = __nv_bfloat16; __VA_ARGS__; } \
      else { using P = float; __VA_ARGS__; }          \
    } else {                                                       \
      using T = float;                                             \
      if ((a).param_bf16) { using P = __nv_bfloat16; __VA_ARGS__; } \
      else { using P = float; __VA_ARGS__; }          \
    }                                                              \
  } while (0)

cudaError_t launch_norm_fwd(const NormArgs& a, int, cudaStream_t s) {
  const Shape f = shape_of(a, true);
  NORM_TYPES(a, {
    constexpr int V = 16 / sizeof(T);
    return f.n > 1 ? fwd_n<T, P, V>(a, f.pieces, s) : fwd_n<T, P, 1>(a, f.pieces, s);
  });
}

cudaError_t launch_norm_bwd(const NormArgs& a, int sms, cudaStream_t s) {
  const Shape f = shape_of(a, false);
  const int parts = norm_parts(a, sms);
  NORM_TYPES(a, {
    constexpr int V = 16 / sizeof(T);
    return f.n > 1 ? bwd_n<T, P, V>(a, f.pieces, parts, s) : bwd_n<T, P, 1>(a, f.pieces, parts, s);
  });
}

cudaError_t launch_norm_colsum(const NormArgs& a, int sms, cudaStream_t s) {
  k_norm_colsum<<<static_cast<unsigned>((a.d + 31) / 32), 256, 0, s>>>(a, norm_parts(a, sms));
  return cudaGetLastError();
}

}  // namespace grpo
