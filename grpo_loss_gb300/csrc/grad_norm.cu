// The norm of many tensors taken as one vector, and their scaling by the clip factor
//   factor = min(1, max_norm / (norm + eps)).
// The norm reads every element once; the factor needs all of them, so that clipping
// reads them a second time and writes them.
#include <cuda_bf16.h>

#include "internal.h"

namespace grpo {

namespace {

constexpr int kThreads = 256;
constexpr int kChunk = 8192;  // elements a CTA takes at a time

// The table of one launch, a kernel parameter (a captured launch holds its own).
struct GradTable {
  int n;
  uint32_t chunks;
  GradTensor t[kGradMaxTensors];
};
static_assert(sizeof(GradTable) + 256 <= 32764, "kernel parameters");

__device__ __forceinline__ int tensor_of(const GradTable& tab, uint32_t chunk) {
  int lo = 0, hi = tab.n - 1;  // the last tensor whose first chunk is not past this one
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (tab.t[mid].chunk0 <= chunk) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}
__device__ __forceinline__ float value(const GradTensor& t, int64_t i) {
  return t.bf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(t.grad)[i]) : static_cast<const float*>(t.grad)[i];
}

// The larger, and NaN where either is.
__device__ __forceinline__ double larger(double a, double b) { return a != a || a > b ? a : b; }

__device__ double cta_join(double v, int inf) {
  __shared__ double part[32];
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) {
    const double u = __shfl_xor_sync(0xffffffffu, v, o);
    v = inf ? larger(v, u) : v + u;
  }
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
  __syncthreads();
  v = 0.0;
  for (int w = 0; w < kThreads / 32; ++w) v = inf ? larger(v, part[w]) : v + part[w];
  __syncthreads();
  return v;
}

__global__ void __launch_bounds__(kThreads) k_grad_norm(const __grid_constant__ GradTable tab, int inf, double* partial) {
  double sum = 0.0;
  for (uint32_t chunk = blockIdx.x; chunk < tab.chunks; chunk += gridDim.x) {
    const GradTensor& t = tab.t[tensor_of(tab, chunk)];
    const int64_t i0 = static_cast<int64_t>(chunk - t.chunk0) * kChunk;
    const int64_t end = t.n - i0 < kChunk ? t.n : i0 + kChunk;
    for (int64_t i = i0 + threadIdx.x; i < end; i += kThreads) {
      const double g = value(t, i);
      sum = inf ? larger(sum, fabs(g)) : sum + g * g;
    }
  }
  sum = cta_join(sum, inf);
  if (threadIdx.x == 0) partial[blockIdx.x] = sum;
}

__global__ void __launch_bounds__(kThreads) k_grad_join(const double* partial, int parts, int inf, double max_norm, double eps,
                                                        float* norm, float* factor, double* fold) {
  double sum = 0.0;
  for (int i = threadIdx.x; i < parts; i += kThreads) sum = inf ? larger(sum, partial[i]) : sum + partial[i];
  sum = cta_join(sum, inf);
  if (threadIdx.x == 0 && fold) *fold = sum;
  if (threadIdx.x == 0 && !fold) {
    if (!inf) sum = sqrt(sum);
    norm[0] = static_cast<float>(sum);
    if (factor) {
      const double f = max_norm / (sum + eps);
      factor[0] = f > 1.0 || max_norm == INFINITY ? 1.f : static_cast<float>(f);
    }
  }
}

__global__ void __launch_bounds__(kThreads) k_grad_scale(const __grid_constant__ GradTable tab, const float* factor) {
  const float f = *factor;
  for (uint32_t chunk = blockIdx.x; chunk < tab.chunks; chunk += gridDim.x) {
    const GradTensor& t = tab.t[tensor_of(tab, chunk)];
    if (f == 1.f && t.out == t.grad) continue;
    const int64_t i0 = static_cast<int64_t>(chunk - t.chunk0) * kChunk;
    const int64_t end = t.n - i0 < kChunk ? t.n : i0 + kChunk;
    for (int64_t i = i0 + threadIdx.x; i < end; i += kThreads) {
      const float v = value(t, i) * f;
      if (t.bf16) static_cast<__nv_bfloat16*>(t.out)[i] = __float2bfloat16_rn(v);
      else static_cast<float*>(t.out)[i] = v;
    }
  }
}

void fill(GradTable& tab, const GradTensor* t, int n) {
  tab.n = n;
  tab.chunks = 0;
  for (int i = 0; i < n; ++i) {
    tab.t[i] = t[i];
    tab.t[i].chunk0 = tab.chunks;
    tab.chunks += static_cast<uint32_t>((t[i].n + kChunk - 1) / kChunk);
  }
}

}  // namespace

// CTAs of one launch, and partial norms that a launch leaves, at most.
int grad_parts(int sms) { return 8 * sms; }

cudaError_t launch_grad_norm(const GradTensor* t, int n, int inf, int sms, double* partial, int* parts, cudaStream_t s) {
  GradTable tab;
  fill(tab, t, n);
  *parts = static_cast<int>(tab.chunks < static_cast<uint32_t>(grad_parts(sms)) ? tab.chunks : grad_parts(sms));
  k_grad_norm<<<*parts, kThreads, 0, s>>>(tab, inf, partial);
  return cudaGetLastError();
}
cudaError_t launch_grad_join(const double* partial, int parts, int inf, double max_norm, double eps, float* norm, float* factor,
                             cudaStream_t s) {
  k_grad_join<<<1, kThreads, 0, s>>>(partial, parts, inf, max_norm, eps, norm, factor, nullptr);
  return cudaGetLastError();
}
cudaError_t launch_grad_fold(double* partial, int parts, int inf, cudaStream_t s) {
  k_grad_join<<<1, kThreads, 0, s>>>(partial, parts, inf, 0.0, 0.0, nullptr, nullptr, partial);
  return cudaGetLastError();
}
cudaError_t launch_grad_scale(const GradTensor* t, int n, const float* factor, int sms, cudaStream_t s) {
  GradTable tab;
  fill(tab, t, n);
  const int64_t most = grad_parts(sms);
  k_grad_scale<<<static_cast<unsigned>(tab.chunks < most ? tab.chunks : most), kThreads, 0, s>>>(tab, factor);
  return cudaGetLastError();
}

}  // namespace grpo
