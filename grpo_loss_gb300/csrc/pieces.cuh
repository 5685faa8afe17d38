// Rows of float32 or bf16 values by pieces of up to 16 bytes, parameters beside them, and
// sums over the threads that hold a row.
#pragma once

#include <cuda_bf16.h>
#include <stdint.h>

namespace grpo {

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

__device__ __forceinline__ float param(const void* p, int bf16, int64_t i) {
  return bf16 ? ldf(static_cast<const __nv_bfloat16*>(p), i) : ldf(static_cast<const float*>(p), i);
}

// Sums over a group of G threads (a part of a warp, or a multiple of 32 that
// divides the CTA or is it), returned to each of them. `slot` alternates between calls, so that one
// barrier a call is enough.
template <int G>
__device__ __forceinline__ float group_sum(float a, float* part, int slot) {
#pragma unroll
  for (int o = G < 32 ? G / 2 : 16; o >= 1; o >>= 1) a += __shfl_xor_sync(0xffffffffu, a, o);
  if constexpr (G > 32) {
    constexpr int W = G / 32, P = W <= 2 ? 2 : W <= 4 ? 4 : W <= 8 ? 8 : W <= 16 ? 16 : 32;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    float* mine = part + slot * 128;
    if (lane == 0) mine[warp] = a;
    __syncthreads();
    // each lane takes one warp's sum
    const int w = lane & (P - 1);
    a = w < W ? mine[warp / W * W + w] : 0.f;
#pragma unroll
    for (int o = P / 2; o >= 1; o >>= 1) a += __shfl_xor_sync(0xffffffffu, a, o);
  }
  return a;
}
// 2, 4 or 8 sums at once. While the lanes are halved, so are the sums that a lane
// carries: first the lanes of either half take half of the sums each, and so on.
template <int G, int M>
__device__ __forceinline__ void group_sums(float (&v)[M], float* part, int slot) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int o = 16;
#pragma unroll
  for (int m = M / 2; m >= 1; m /= 2, o /= 2) {
    const bool up = lane & o;
#pragma unroll
    for (int i = 0; i < m; ++i) {
      const float give = up ? v[i] : v[i + m], keep = up ? v[i + m] : v[i];
      v[i] = keep + __shfl_xor_sync(0xffffffffu, give, o);
    }
  }
  // each of M runs of `run` lanes holds one sum, in the order of the runs
  constexpr int run = 32 / M;
  float a = v[0];
#pragma unroll
  for (int p = run / 2; p >= 1; p /= 2) a += __shfl_xor_sync(0xffffffffu, a, p);
  if (G > 32) {
    constexpr int W = G / 32;
    float* mine = part + slot * (M < 4 ? 128 : 32 * M) + lane / run * 32;  // the run's sum of every warp
    if (lane % run == 0) mine[warp] = a;
    __syncthreads();
    a = 0.f;
#pragma unroll
    for (int w = 0; w < W; w += run)
      if (w + lane % run < W) a += mine[warp / W * W + w + lane % run];
#pragma unroll
    for (int p = run / 2; p >= 1; p /= 2) a += __shfl_xor_sync(0xffffffffu, a, p);
  }
#pragma unroll
  for (int i = 0; i < M; ++i) v[i] = __shfl_sync(0xffffffffu, a, i * run);
}

// Copies a piece into shared memory while the thread goes on.
template <int BYTES>
__device__ __forceinline__ void copy_async(void* to, const void* from) {
  const uint32_t at = static_cast<uint32_t>(__cvta_generic_to_shared(to));
  if constexpr (BYTES == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(at), "l"(from) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(at), "l"(from), "n"(BYTES) : "memory");
}

// The same of the first `bytes` bytes; the others are 0.
__device__ __forceinline__ void copy_async_zero(void* to, const void* from, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                   static_cast<uint32_t>(__cvta_generic_to_shared(to))),
               "l"(from), "r"(bytes)
               : "memory");
}

}  // namespace grpo
