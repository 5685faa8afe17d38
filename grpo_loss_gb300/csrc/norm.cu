// Layer norm and RMS norm over rows, forward and backward.
//   y = (x - mean) r w + b,  r = 1 / sqrt(mean((x - mean)^2) + eps)
//   g = dy w, h = (x - mean) r:  dx = r (g - mean(g) - h mean(g h)),
//   dw = sum_rows dy h,  db = sum_rows dy            (RMS: mean = 0, no b)
// Bound by memory: the forward reads x and writes y, the backward reads x and
// dy and writes dx; the column sums add a few rows' worth of partials.
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

constexpr int kThreads = 256;

// Sum of (a, b) over the CTA, returned to every thread.
__device__ __forceinline__ float2 block_sum2(float a, float b) {
  __shared__ float2 part[32];
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) {
    a += __shfl_xor_sync(0xffffffffu, a, o);
    b += __shfl_xor_sync(0xffffffffu, b, o);
  }
  __syncthreads();  // the previous call's readers are done
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = make_float2(a, b);
  __syncthreads();
  float2 s = make_float2(0.f, 0.f);
  for (int w = 0; w < kThreads / 32; ++w) {
    s.x += part[w].x;
    s.y += part[w].y;
  }
  return s;
}

// One CTA per row; the row is read three times (mean, variance, output), the
// later two from cache.
template <typename T, typename P>
__global__ void __launch_bounds__(kThreads) k_norm_fwd(NormArgs a) {
  const int64_t row = blockIdx.x;
  const T* x = static_cast<const T*>(a.x) + row * a.ld_x;
  T* y = static_cast<T*>(a.y) + row * a.ld_y;
  const P* w = static_cast<const P*>(a.weight);
  const P* b = static_cast<const P*>(a.bias);
  const int d = static_cast<int>(a.d);
  float mean = 0.f;
  if (!a.rms) {
    float s = 0.f;
    for (int i = threadIdx.x; i < d; i += kThreads) s += ldf(x, i);
    mean = block_sum2(s, 0.f).x / d;
  }
  float q = 0.f;
  for (int i = threadIdx.x; i < d; i += kThreads) {
    const float c = ldf(x, i) - mean;
    q += c * c;
  }
  const float r = 1.0f / sqrtf(block_sum2(q, 0.f).x / d + a.eps);
  for (int i = threadIdx.x; i < d; i += kThreads) {
    float v = (ldf(x, i) - mean) * r * ldf(w, i);
    if (b) v += ldf(b, i);
    stf(y, i, v);
  }
  if (threadIdx.x == 0) {
    if (a.mean) a.mean[row] = mean;
    if (a.rstd) a.rstd[row] = r;
  }
}

// One CTA per row: the two row sums, then dx.
template <typename T, typename P>
__global__ void __launch_bounds__(kThreads) k_norm_bwd(NormArgs a) {
  const int64_t row = blockIdx.x;
  const T* x = static_cast<const T*>(a.x) + row * a.ld_x;
  const T* dy = static_cast<const T*>(a.dy) + row * a.ld_dy;
  T* dx = static_cast<T*>(a.dx) + row * a.ld_dx;
  const P* w = static_cast<const P*>(a.weight);
  const int d = static_cast<int>(a.d);
  const float mean = a.mean ? a.mean[row] : 0.f, r = a.rstd[row];
  float sg = 0.f, sgh = 0.f;
  for (int i = threadIdx.x; i < d; i += kThreads) {
    const float g = ldf(dy, i) * ldf(w, i);
    sg += g;
    sgh += g * ((ldf(x, i) - mean) * r);
  }
  float2 s = block_sum2(sg, sgh);
  s.x = a.rms ? 0.f : s.x / d;
  s.y /= d;
  for (int i = threadIdx.x; i < d; i += kThreads) {
    const float g = ldf(dy, i) * ldf(w, i);
    stf(dx, i, r * (g - s.x - (ldf(x, i) - mean) * r * s.y));
  }
}

// Partial column sums of one group of rows: one thread a column, in row order.
template <typename T>
__global__ void __launch_bounds__(kThreads) k_norm_partial(NormArgs a, int parts) {
  const int64_t col = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
  if (col >= a.d) return;
  const int64_t r0 = a.rows * blockIdx.y / parts, r1 = a.rows * (blockIdx.y + 1) / parts;
  const T* x = static_cast<const T*>(a.x);
  const T* dy = static_cast<const T*>(a.dy);
  float sw = 0.f, sb = 0.f;
  for (int64_t r = r0; r < r1; ++r) {
    const float g = ldf(dy, r * a.ld_dy + col);
    const float mean = a.mean ? a.mean[r] : 0.f;
    sw += g * ((ldf(x, r * a.ld_x + col) - mean) * a.rstd[r]);
    sb += g;
  }
  a.partial[(2 * static_cast<int64_t>(blockIdx.y)) * a.d + col] = sw;
  a.partial[(2 * static_cast<int64_t>(blockIdx.y) + 1) * a.d + col] = sb;
}

__global__ void __launch_bounds__(kThreads) k_norm_colsum(NormArgs a, int parts) {
  const int64_t col = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
  if (col >= a.d) return;
  float sw = 0.f, sb = 0.f;
  for (int p = 0; p < parts; ++p) {
    sw += a.partial[(2 * static_cast<int64_t>(p)) * a.d + col];
    sb += a.partial[(2 * static_cast<int64_t>(p) + 1) * a.d + col];
  }
  if (a.dweight) a.dweight[col] = sw;
  if (a.dbias) a.dbias[col] = sb;
}

}  // namespace

int norm_parts(const NormArgs& a, int sms) {
  return static_cast<int>(a.rows < 1 ? 1 : a.rows < 2 * sms ? a.rows : 2 * sms);
}

// Calls F.template operator()<T, P>() for the element types of `a`.
#define NORM_TYPES(a, call)                                        \
  do {                                                             \
    if ((a).bf16) {                                                \
      using T = __nv_bfloat16;                                     \
      if ((a).param_bf16) { using P = __nv_bfloat16; call; }       \
      else { using P = float; call; }                              \
    } else {                                                       \
      using T = float;                                             \
      if ((a).param_bf16) { using P = __nv_bfloat16; call; }       \
      else { using P = float; call; }                              \
    }                                                              \
  } while (0)

cudaError_t launch_norm_fwd(const NormArgs& a, int, cudaStream_t s) {
  NORM_TYPES(a, (k_norm_fwd<T, P><<<static_cast<unsigned>(a.rows), kThreads, 0, s>>>(a)));
  return cudaGetLastError();
}

cudaError_t launch_norm_bwd(const NormArgs& a, int sms, cudaStream_t s) {
  // the column sums first: dx may overwrite dy or x
  if (a.partial) {
    const int parts = norm_parts(a, sms);
    const dim3 grid(static_cast<unsigned>((a.d + kThreads - 1) / kThreads), parts);
    if (a.bf16)
      k_norm_partial<__nv_bfloat16><<<grid, kThreads, 0, s>>>(a, parts);
    else
      k_norm_partial<float><<<grid, kThreads, 0, s>>>(a, parts);
  }
  NORM_TYPES(a, (k_norm_bwd<T, P><<<static_cast<unsigned>(a.rows), kThreads, 0, s>>>(a)));
  return cudaGetLastError();
}

cudaError_t launch_norm_colsum(const NormArgs& a, int sms, cudaStream_t s) {
  k_norm_colsum<<<static_cast<unsigned>((a.d + kThreads - 1) / kThreads), kThreads, 0, s>>>(
      a, norm_parts(a, sms));
  return cudaGetLastError();
}

}  // namespace grpo
