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

#include <atomic>

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
template <>
struct Piece<float, 2> {
  uint2 raw;
  __device__ __forceinline__ float get(int e) const { return __uint_as_float(e == 0 ? raw.x : raw.y); }
  __device__ __forceinline__ void set(const float* v) {
    raw = make_uint2(__float_as_uint(v[0]), __float_as_uint(v[1]));
  }
};
template <>
struct Piece<__nv_bfloat16, 2> {
  uint32_t raw;
  __device__ __forceinline__ float get(int e) const {
    return __uint_as_float(e ? raw & 0xFFFF0000u : raw << 16);
  }
  __device__ __forceinline__ void set(const float* v) { raw = pack_bf16(v[0], v[1]); }
};
template <typename T, int N>
__device__ __forceinline__ Piece<T, N> load_piece(const T* p) {
  return *reinterpret_cast<const Piece<T, N>*>(p);
}
template <typename T, int N>
__device__ __forceinline__ void store_piece(T* p, const Piece<T, N>& v) {
  *reinterpret_cast<Piece<T, N>*>(p) = v;
}
// Pairs of floats in one register pair: one instruction for both.
__device__ __forceinline__ uint64_t pair_of(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ float2 of_pair(uint64_t p) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(p));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// N weights (or biases) from element i on; their type is the same for a launch.
template <int N>
__device__ __forceinline__ void load_params(const void* p, int bf16, int i, float* v) {
  if (bf16) {
    const Piece<__nv_bfloat16, N> q = load_piece<__nv_bfloat16, N>(static_cast<const __nv_bfloat16*>(p) + i);
#pragma unroll
    for (int e = 0; e < N; ++e) v[e] = q.get(e);
  } else {
    constexpr int M = N < 4 ? N : 4;
#pragma unroll
    for (int f = 0; f < N; f += M) {
      const Piece<float, M> q = load_piece<float, M>(static_cast<const float*>(p) + i + f);
#pragma unroll
      for (int e = 0; e < M; ++e) v[f + e] = q.get(e);
    }
  }
}

__device__ __forceinline__ float param(const void* p, int bf16, int i) {
  return bf16 ? ldf(static_cast<const __nv_bfloat16*>(p), i) : ldf(static_cast<const float*>(p), i);
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
  const int lane = threadIdx.x & 31;
  if (lane == 0) mine[warp] = make_float2(a, b);
  __syncthreads();
  // each lane takes one warp's sums
  constexpr int W = G / 32, P = W <= 2 ? 2 : W <= 4 ? 4 : W <= 8 ? 8 : W <= 16 ? 16 : 32;
  const float2 p = (lane & (P - 1)) < W ? mine[first + (lane & (P - 1))] : make_float2(0.f, 0.f);
  a = p.x;
  b = p.y;
#pragma unroll
  for (int o = P / 2; o >= 1; o >>= 1) {
    a += __shfl_xor_sync(0xffffffffu, a, o);
    if (BOTH) b += __shfl_xor_sync(0xffffffffu, b, o);
  }
  return make_float2(a, b);
}

// ---------------------------------------------------------------- forward
// A group of G threads takes a row, R rows a CTA; each thread holds NV pieces of
// N values of it (G N NV >= d).
template <typename T, int N, int NV, int G, int R>
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
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    const int i = (k * G + tid) * N;
    if (i < d) {
      float o[N], w[N];
      load_params<N>(a.weight, a.param_bf16, i, w);
#pragma unroll
      for (int e = 0; e < N; ++e) o[e] = (v[k].get(e) - mean) * r * w[e];
      if (a.bias) {
        load_params<N>(a.bias, a.param_bf16, i, w);
#pragma unroll
        for (int e = 0; e < N; ++e) o[e] += w[e];
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
// Copies a piece into shared memory while the thread goes on.
template <int BYTES>
__device__ __forceinline__ void copy_async(void* to, const void* from) {
  const uint32_t at = static_cast<uint32_t>(__cvta_generic_to_shared(to));
  if constexpr (BYTES == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(at), "l"(from) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(at), "l"(from), "n"(BYTES) : "memory");
}

// A group of G threads walks over the rows group, + groups, ... (R groups a CTA);
// each thread holds NV pieces of N columns: their values of a row and their column
// sums. Its pieces of the next S - 1 rows are on their way into shared memory:
// S 16-byte pieces of x and of dy a thread keep HBM busy where registers for them
// would halve the threads (1075 us for 163840 x 4096 bf16 with one row ahead in
// registers). A thread reads back what it copied itself, so no barrier is needed
// for them.
template <typename T, int N, int NV, int G, int R, int S>
__global__ void __launch_bounds__(G * R) k_norm_bwd(NormArgs a) {
  constexpr int B = N * static_cast<int>(sizeof(T));
  using V = Piece<T, N>;
  extern __shared__ __align__(16) unsigned char ring_raw[];
  __shared__ float2 part[2 * 32];
  V* ring = reinterpret_cast<V*>(ring_raw) + threadIdx.x;  // [S][2][NV][threads]
  const int tid = threadIdx.x % G, d = static_cast<int>(a.d);
  const int64_t groups = static_cast<int64_t>(gridDim.x) * R;
  const int64_t row0 = static_cast<int64_t>(blockIdx.x) * R + threadIdx.x / G;
  const T* x = static_cast<const T*>(a.x);
  const T* dy = static_cast<const T*>(a.dy);
  // columns in pairs (a column alone has a pair of its own)
  constexpr int H = (N + 1) / 2;
  uint64_t dw[NV][H], db[NV][H], w[NV][H];
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    const int i = (k * G + tid) * N;
    float ww[2 * H] = {};
    if (i < d) load_params<N>(a.weight, a.param_bf16, i, ww);
#pragma unroll
    for (int e = 0; e < H; ++e) {
      dw[k][e] = db[k][e] = pair_of(0.f, 0.f);
      w[k][e] = pair_of(ww[2 * e], ww[2 * e + 1]);
    }
  }
  auto slot_of = [&](int s, int which, int k) -> V& {
    return ring[((s * 2 + which) * NV + k) * (G * R)];
  };
  auto fetch = [&](int64_t row, int s) {
    if (row < a.rows) {
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        const int i = (k * G + tid) * N;
        if (i < d) {
          if constexpr (B >= 4) {
            copy_async<B>(&slot_of(s, 0, k), x + row * a.ld_x + i);
            copy_async<B>(&slot_of(s, 1, k), dy + row * a.ld_dy + i);
          } else {
            slot_of(s, 0, k) = load_piece<T, N>(x + row * a.ld_x + i);
            slot_of(s, 1, k) = load_piece<T, N>(dy + row * a.ld_dy + i);
          }
        }
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  const float inv_d = 1.f / d;
  // every group of a CTA makes the same number of turns: barriers are the CTA's
  const int64_t first = static_cast<int64_t>(blockIdx.x) * R;
  const int64_t turns = first < a.rows ? (a.rows - first + groups - 1) / groups : 0;
#pragma unroll
  for (int s = 0; s < S - 1; ++s) fetch(row0 + s * groups, s);
  float mean_next = 0.f, rstd_next = 0.f;
  if (row0 < a.rows) {
    mean_next = a.rms ? 0.f : a.mean[row0];
    rstd_next = a.rstd[row0];
  }
  int at = 0, parity = 0;
  int64_t row = row0;
  for (int64_t n = 0; n < turns; ++n, row += groups) {
    const bool live = row < a.rows;
    const int to = at == 0 ? S - 1 : at - 1;  // the slot read last
    fetch(row + (S - 1) * groups, to);
    asm volatile("cp.async.wait_group %0;" ::"n"(S - 1) : "memory");
    const float mean = mean_next, r = rstd_next;
    if (row + groups < a.rows) {
      mean_next = a.rms ? 0.f : a.mean[row + groups];
      rstd_next = a.rstd[row + groups];
    }
    uint64_t gw[NV][H], h[NV][H], sg = pair_of(0.f, 0.f), sgh = sg;
    if (live) {
      // (x - mean) r, the difference first: x and mean may be large and close
      const uint64_t rr = pair_of(r, r), shift = pair_of(-mean, -mean);
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        if ((k * G + tid) * N < d) {
          const V xv = slot_of(at, 0, k), gv = slot_of(at, 1, k);
#pragma unroll
          for (int e = 0; e < H; ++e) {
            const bool two = 2 * e + 1 < N;
            const uint64_t g = pair_of(gv.get(2 * e), two ? gv.get(2 * e + 1) : 0.f);
            const uint64_t x2 = pair_of(xv.get(2 * e), two ? xv.get(2 * e + 1) : 0.f);
            h[k][e] = mul2(add2(x2, shift), rr);
            dw[k][e] = fma2(g, h[k][e], dw[k][e]);
            db[k][e] = add2(db[k][e], g);
            gw[k][e] = mul2(g, w[k][e]);
            sg = add2(sg, gw[k][e]);
            sgh = fma2(gw[k][e], h[k][e], sgh);
          }
        }
      }
    }
    const float2 pg = of_pair(sg), ph = of_pair(sgh);
    float2 s = group_sum<G, true>(pg.x + pg.y, ph.x + ph.y, part, parity);
    parity ^= 1;
    s.x = a.rms ? 0.f : s.x * inv_d;
    s.y *= inv_d;
    if (live) {
      const uint64_t rr = pair_of(r, r), c1 = pair_of(-s.x, -s.x), c2 = pair_of(-s.y, -s.y);
      T* dx = static_cast<T*>(a.dx) + row * a.ld_dx;
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        const int i = (k * G + tid) * N;
        if (i < d) {
          float o[2 * H];
#pragma unroll
          for (int e = 0; e < H; ++e) {
            const float2 q = of_pair(mul2(fma2(h[k][e], c2, add2(gw[k][e], c1)), rr));
            o[2 * e] = q.x;
            o[2 * e + 1] = q.y;
          }
          V p;
          p.set(o);
          store_piece<T, N>(dx + i, p);
        }
      }
    }
    at = at == S - 1 ? 0 : at + 1;
  }
  if (!a.partial) return;
  float* pw = a.partial + 2 * row0 * d;  // one pair of rows a group
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    const int i = (k * G + tid) * N;
    if (i < d) {
#pragma unroll
      for (int e = 0; e < H; ++e) {
        const float2 p = of_pair(dw[k][e]), q = of_pair(db[k][e]);
        pw[i + 2 * e] = p.x;
        pw[d + i + 2 * e] = q.x;
        if (2 * e + 1 < N) {
          pw[i + 2 * e + 1] = p.y;
          pw[d + i + 2 * e + 1] = q.y;
        }
      }
    }
  }
}

// Rows too long for registers: three passes, the later ones from cache.
constexpr int kLong = 1024;
template <typename T>
__global__ void __launch_bounds__(kLong) k_norm_fwd_long(NormArgs a) {
  __shared__ float2 part[2 * 32];
  const int64_t row = blockIdx.x;
  const T* x = static_cast<const T*>(a.x) + row * a.ld_x;
  T* y = static_cast<T*>(a.y) + row * a.ld_y;
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
    float v = (ldf(x, i) - mean) * r * param(a.weight, a.param_bf16, i);
    if (a.bias) v += param(a.bias, a.param_bf16, i);
    stf(y, i, v);
  }
  if (threadIdx.x == 0) {
    if (a.mean) a.mean[row] = mean;
    if (a.rstd) a.rstd[row] = r;
  }
}

// The same for the backward; the column sums are in the partial rows of the CTA
// from its first row on.
template <typename T>
__global__ void __launch_bounds__(kLong) k_norm_bwd_long(NormArgs a) {
  __shared__ float2 part[2 * 32];
  const int d = static_cast<int>(a.d);
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
      const float g = ldf(dy, i), h = (ldf(x, i) - mean) * r, gw = g * param(a.weight, a.param_bf16, i);
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
      const float gw = ldf(dy, i) * param(a.weight, a.param_bf16, i);
      stf(dx, i, r * (gw - s.x - (ldf(x, i) - mean) * r * s.y));
    }
  }
}

// Joins the partial column sums: 32 columns a CTA, each warp takes every 32nd
// part; added up in a fixed order.
__global__ void __launch_bounds__(1024) k_norm_colsum(NormArgs a, int parts) {
  __shared__ float2 s[32][33];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t col = static_cast<int64_t>(blockIdx.x) * 32 + lane;
  float sw = 0.f, sb = 0.f;
  if (col < a.d) {
#pragma unroll 8
    for (int p = warp; p < parts; p += 32) {
      const float* q = a.partial + 2 * static_cast<int64_t>(p) * a.d + col;
      sw += q[0];
      sb += q[a.d];
    }
  }
  s[warp][lane] = make_float2(sw, sb);
  __syncthreads();
  const float2 v = s[lane][warp];  // part `lane` of column `warp`
  sw = v.x;
  sb = v.y;
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) {
    sw += __shfl_xor_sync(0xffffffffu, sw, o);
    sb += __shfl_xor_sync(0xffffffffu, sb, o);
  }
  const int64_t to = static_cast<int64_t>(blockIdx.x) * 32 + warp;
  if (lane == 0 && to < a.d) {
    if (a.dweight) a.dweight[to] = sw;
    if (a.dbias) a.dbias[to] = sb;
  }
}

// Values a piece: as many of 8, 4, 2 and 1 (up to 16 bytes) as divide d and find
// every row of every operand on a boundary of their size.
int piece_of(const NormArgs& a, bool fwd) {
  const int es = a.bf16 ? 2 : 4, ps = a.param_bf16 ? 2 : 4;
  uint64_t rows = 0, params = reinterpret_cast<uintptr_t>(a.weight);  // low bits of all addresses
  auto add = [&](const void* p, int64_t ld) {
    rows |= reinterpret_cast<uintptr_t>(p) | static_cast<uint64_t>(ld) * es;
  };
  add(a.x, a.ld_x);
  if (fwd) {
    add(a.y, a.ld_y);
    params |= reinterpret_cast<uintptr_t>(a.bias);
  } else {
    add(a.dy, a.ld_dy);
    add(a.dx, a.ld_dx);
  }
  int n = 16 / es;
  while (n > 1 && (a.d % n || rows % (n * es) || params % (n * ps < 16 ? n * ps : 16))) n /= 2;
  return n;
}

// The backward's threads: G a row, R rows a CTA at a time, NV pieces a thread; 0
// where a row does not fit.
struct BwdShape {
  int n, g, r, nv;
};
BwdShape bwd_shape(const NormArgs& a) {
  BwdShape s;
  s.n = piece_of(a, false);
  const int pieces = static_cast<int>((a.d + s.n - 1) / s.n);
  s.nv = 1;
  s.r = 1;
  if (pieces <= 32) s.g = 32, s.r = 8;
  else if (pieces <= 64) s.g = 32, s.r = 8, s.nv = 2;
  else if (pieces <= 128) s.g = 128, s.r = 2;
  else if (pieces <= 256) s.g = 256;
  else if (pieces <= 384) s.g = 384;
  else if (pieces <= 512) s.g = 512;
  else if (pieces <= 768) s.g = 384, s.nv = 2;
  else if (pieces <= 1024) s.g = 512, s.nv = 2;
  else if (pieces <= 2048) s.g = 1024, s.nv = 2;
  else if (s.n <= 2 && pieces <= 4096) s.g = 1024, s.nv = 4;
  else s.g = 0;
  return s;
}

template <typename T, int N, int NV, int G, int R>
cudaError_t fwd(const NormArgs& a, cudaStream_t s) {
  const unsigned grid = static_cast<unsigned>((a.rows + R - 1) / R);
  k_norm_fwd<T, N, NV, G, R><<<grid, G * R, 0, s>>>(a);
  return cudaGetLastError();
}
template <typename T, int N>
cudaError_t fwd_n(const NormArgs& a, cudaStream_t s) {
  const int64_t pieces = (a.d + N - 1) / N;
  if (pieces <= 32) return fwd<T, N, 1, 32, 4>(a, s);
  if (pieces <= 64) return fwd<T, N, 2, 32, 4>(a, s);
  if (pieces <= 128) return fwd<T, N, 4, 32, 4>(a, s);
  if (pieces <= 256) return fwd<T, N, 2, 128, 1>(a, s);
  if (pieces <= 512) return fwd<T, N, 4, 128, 1>(a, s);
  if (pieces <= 1024) return fwd<T, N, 4, 256, 1>(a, s);
  if (pieces <= 2048) return fwd<T, N, 4, 512, 1>(a, s);
  if (pieces <= 4096) return fwd<T, N, 4, 1024, 1>(a, s);
  if (pieces <= 8192) return fwd<T, N, 8, 1024, 1>(a, s);
  k_norm_fwd_long<T><<<static_cast<unsigned>(a.rows), kLong, 0, s>>>(a);
  return cudaGetLastError();
}

// CTAs of the backward: what the SMs hold at a time (by threads and the ring's
// shared memory), so that each walks over its share of the rows once.
int bwd_ctas_per_sm(const BwdShape& b) {
  if (b.g == 0) return 2;
  const int by_threads = 1024 / (b.g * b.r);
  return by_threads < 1 ? 1 : by_threads;
}
int bwd_grid(const NormArgs& a, const BwdShape& b, int sms) {
  const int64_t need = (a.rows + (b.g ? b.r : 1) - 1) / (b.g ? b.r : 1);
  const int64_t most = static_cast<int64_t>(bwd_ctas_per_sm(b)) * sms;
  return static_cast<int>(need < 1 ? 1 : need < most ? need : most);
}

template <typename T, int N, int NV, int G, int R>
cudaError_t bwd(const NormArgs& a, int grid, cudaStream_t s) {
  constexpr int slot = 2 * NV * N * static_cast<int>(sizeof(T)) * G * R;
  constexpr int S = 4 * slot <= 200 * 1024 ? 4 : 3;
  constexpr int smem = S * slot;
  if constexpr (smem > 40 * 1024) {  // (48 KB with the static part need no attribute)
    static std::atomic<uint64_t> configured{0};  // one bit a device
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = 1ull << (dev & 63);
    if (!(configured.load() & bit)) {
      e = cudaFuncSetAttribute(k_norm_bwd<T, N, NV, G, R, S>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
      if (e != cudaSuccess) return e;
      configured.fetch_or(bit);
    }
  }
  k_norm_bwd<T, N, NV, G, R, S><<<grid, G * R, smem, s>>>(a);
  return cudaGetLastError();
}
template <typename T, int N>
cudaError_t bwd_n(const NormArgs& a, const BwdShape& b, int grid, cudaStream_t s) {
  if (b.g == 32 && b.nv == 1) return bwd<T, N, 1, 32, 8>(a, grid, s);
  if (b.g == 32) return bwd<T, N, 2, 32, 8>(a, grid, s);
  if (b.g == 128) return bwd<T, N, 1, 128, 2>(a, grid, s);
  if (b.g == 256) return bwd<T, N, 1, 256, 1>(a, grid, s);
  if (b.g == 384 && b.nv == 1) return bwd<T, N, 1, 384, 1>(a, grid, s);
  if (b.g == 512 && b.nv == 1) return bwd<T, N, 1, 512, 1>(a, grid, s);
  if (b.g == 384) return bwd<T, N, 2, 384, 1>(a, grid, s);
  if (b.g == 512) return bwd<T, N, 2, 512, 1>(a, grid, s);
  if (b.g == 1024 && b.nv == 2) return bwd<T, N, 2, 1024, 1>(a, grid, s);
  if constexpr (N <= 2) {
    if (b.g == 1024) return bwd<T, N, 4, 1024, 1>(a, grid, s);
  }
  k_norm_bwd_long<T><<<grid, kLong, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace

// Rows of partial column sums that the workspace holds.
int norm_parts(const NormArgs& a, int sms) {
  // A bound that does not depend on addresses (the workspace is sized before they
  // are known): up to 8 groups a CTA, 32 an SM for short rows and 8 for others.
  const int64_t most = 8ll * sms * (a.d <= 512 ? 4 : 1), need = (a.rows + 7) / 8 * 8;
  return static_cast<int>(need < 8 ? 8 : need < most ? need : most);
}

cudaError_t launch_norm_fwd(const NormArgs& a, int, cudaStream_t s) {
  const int n = piece_of(a, true);
  if (a.bf16)
    return n == 8   ? fwd_n<__nv_bfloat16, 8>(a, s)
           : n == 4 ? fwd_n<__nv_bfloat16, 4>(a, s)
           : n == 2 ? fwd_n<__nv_bfloat16, 2>(a, s)
                    : fwd_n<__nv_bfloat16, 1>(a, s);
  return n == 4 ? fwd_n<float, 4>(a, s) : n == 2 ? fwd_n<float, 2>(a, s) : fwd_n<float, 1>(a, s);
}

cudaError_t launch_norm_bwd(const NormArgs& a, int sms, cudaStream_t s) {
  const BwdShape b = bwd_shape(a);
  const int grid = bwd_grid(a, b, sms);
  if (a.bf16)
    return b.n == 8   ? bwd_n<__nv_bfloat16, 8>(a, b, grid, s)
           : b.n == 4 ? bwd_n<__nv_bfloat16, 4>(a, b, grid, s)
           : b.n == 2 ? bwd_n<__nv_bfloat16, 2>(a, b, grid, s)
                      : bwd_n<__nv_bfloat16, 1>(a, b, grid, s);
  return b.n == 4 ? bwd_n<float, 4>(a, b, grid, s)
         : b.n == 2 ? bwd_n<float, 2>(a, b, grid, s)
                    : bwd_n<float, 1>(a, b, grid, s);
}

cudaError_t launch_norm_colsum(const NormArgs& a, int sms, cudaStream_t s) {
  k_norm_colsum<<<static_cast<unsigned>((a.d + 31) / 32), 1024, 0, s>>>(
      a, bwd_grid(a, bwd_shape(a), sms) * (bwd_shape(a).g ? bwd_shape(a).r : 1));
  return cudaGetLastError();
}

}  // namespace grpo
