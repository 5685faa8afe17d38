// The norm of many tensors taken as one vector, and their scaling by the clip factor
//   factor = min(1, max_norm / (norm + eps)).
// Bound by memory: the norm reads every element once; the factor needs all of them, so
// that clipping reads them a second time and writes them. Short lists, whose time is the
// launches', take one: a cluster of CTAs that joins its parts over shared memory. Others
// take a launch for the parts of the norm, each CTA one, and one that joins them: it writes
// the norm, or scales, each of its CTAs joining them again in the same order. 151936 x 1536
// float32: norm 136 us (6.9 TB/s), clipping into another buffer 437 us (6.4 TB/s over its
// three passes; stores that leave L2 at once 454).
#include <cooperative_groups.h>
#include <cuda_bf16.h>

#include <type_traits>

#include "f32x2.cuh"
#include "internal.h"

namespace cg = cooperative_groups;

namespace grpo {

namespace {

constexpr int kThreads = 256;
constexpr int kPieces = 8;                              // 16-byte loads of a thread in flight
constexpr int kChunkBytes = kThreads * kPieces * 16;    // what a CTA takes at a time
constexpr int kNormCtas = 3, kScaleCtas = 4;            // of an SM, at a time
constexpr int kCluster = 8;
// Lists of up to so many chunks take the one launch.
constexpr int kSmallChunks = 2 * kCluster;
// Tables of a launch: a kernel's parameters are copied whole.
constexpr int kSmallTensors = 32, kSomeTensors = 128;

// The table of one launch, a kernel parameter (a captured launch holds its own).
template <int MOST>
struct GradTable {
  int n;
  uint32_t chunks;
  GradTensor t[MOST];
};
static_assert(sizeof(GradTable<kGradMaxTensors>) + 256 <= 32764, "kernel parameters");

// A tensor is cut at the 16-byte boundaries of its gradient: elements before the first of
// these, and behind the last, are taken one by one with the first and the last chunk.
__host__ __device__ __forceinline__ int head_of(const GradTensor& t) {
  const int es = t.bf16 ? 2 : 4, off = static_cast<int>(reinterpret_cast<uintptr_t>(t.grad) & 15);
  const int64_t head = off ? (16 - off) / es : 0;
  return static_cast<int>(head < t.n ? head : t.n);
}

struct Chunk {
  const GradTensor* t;
  int64_t from;       // its first piece's first element
  int pieces, last;   // whole pieces, and elements behind them
  int head;           // elements before the tensor's first piece
};
template <int MOST>
__device__ __forceinline__ Chunk chunk_of(const GradTable<MOST>& tab, uint32_t chunk) {
  int lo = 0, hi = tab.n - 1;  // the last tensor whose first chunk is not past this one
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (tab.t[mid].chunk0 <= chunk) lo = mid;
    else hi = mid - 1;
  }
  Chunk c;
  c.t = &tab.t[lo];
  const int each = c.t->bf16 ? 8 : 4, head = head_of(*c.t);
  const int64_t many = static_cast<int64_t>(chunk - c.t->chunk0) * (kThreads * kPieces);
  const int64_t left = (c.t->n - head) / each - many;
  c.from = head + many * each;
  c.pieces = static_cast<int>(left < kThreads * kPieces ? left : kThreads * kPieces);
  c.last = left <= kThreads * kPieces ? static_cast<int>((c.t->n - head) % each) : 0;
  c.head = chunk == c.t->chunk0 ? head : 0;
  return c;
}

__device__ __forceinline__ float value(const GradTensor& t, int64_t i) {
  return t.bf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(t.grad)[i]) : static_cast<const float*>(t.grad)[i];
}
__device__ __forceinline__ uint64_t pair_in(uint32_t w) { return pair_of(w << 16, w & 0xFFFF0000u); }  // of two bf16

// The larger, and NaN where either is.
__device__ __forceinline__ double larger(double a, double b) { return a != a || a > b ? a : b; }

// Joins the threads' values in a fixed order; every thread gets the result.
__device__ double cta_join(double v, int inf) {
  __shared__ double part[kThreads / 32];
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) {
    const double u = __shfl_xor_sync(0xffffffffu, v, o);
    v = inf ? larger(v, u) : v + u;
  }
  __syncthreads();
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
  __syncthreads();
  v = part[0];
#pragma unroll
  for (int w = 1; w < kThreads / 32; ++w) v = inf ? larger(v, part[w]) : v + part[w];
  return v;
}

// The sum of the squares of up to kPieces pieces, in float32 with four sums; where that
// may have lost something (squares that overflow, or a sum so small that squares underflow
// beside it) again with the values scaled by a power of two. Sums of all zeros, as of rows
// of an embedding that no token had, are known by their bits.
template <bool BF16>
__device__ __forceinline__ double squares(const uint4 (&v)[kPieces]) {
  auto sum = [&](uint64_t scale, auto scaled) {
    uint64_t s[2] = {pair_of(0.f), pair_of(0.f)};
#pragma unroll
    for (int j = 0; j < kPieces; ++j) {
      const uint32_t w[4] = {v[j].x, v[j].y, v[j].z, v[j].w};
#pragma unroll
      for (int e = 0; e < (BF16 ? 4 : 2); ++e) {
        uint64_t p = BF16 ? pair_in(w[e]) : pair_of(w[2 * (e & 1)], w[2 * (e & 1) + 1]);
        if constexpr (decltype(scaled)::value) p = mul2(p, scale);
        s[e & 1] = fma2(p, p, s[e & 1]);
      }
    }
    const float2 a = of_pair(s[0]), b = of_pair(s[1]);
    return (a.x + a.y) + (b.x + b.y);
  };
  const float s = sum(0, std::false_type());
  if (s >= 0x1p-60f && s <= 0x1p100f) return s;
  uint32_t top = 0;  // the largest magnitude's bits
#pragma unroll
  for (int j = 0; j < kPieces; ++j) {
    const uint32_t w[4] = {v[j].x, v[j].y, v[j].z, v[j].w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if (BF16) top = max(top, max((w[e] << 16) & 0x7FFFFFFFu, w[e] & 0x7FFF0000u));
      else top = max(top, w[e] & 0x7FFFFFFFu);
    }
  }
  if (top == 0) return 0.0;
  if (top >= 0x7F800000u) return s;  // an infinity, or a NaN
  const int up = max(min(254 - static_cast<int>(top >> 23), 253), 1);  // exponent byte of the scale: values below 2
  const float t = sum(pair_of(__uint_as_float(static_cast<uint32_t>(up) << 23)), std::true_type());
  return ldexp(static_cast<double>(t), 2 * (127 - up));
}
template <bool BF16>
__device__ __forceinline__ uint32_t largest(const uint4 (&v)[kPieces]) {
  uint32_t top = 0;
#pragma unroll
  for (int j = 0; j < kPieces; ++j) {
    const uint32_t w[4] = {v[j].x, v[j].y, v[j].z, v[j].w};
#pragma unroll
    for (int e = 0; e < 4; ++e) top = BF16 ? __vmaxu2(top, w[e] & 0x7FFF7FFFu) : max(top, w[e] & 0x7FFFFFFFu);
  }
  return BF16 ? max(top << 16, top & 0xFFFF0000u) : top;
}

// Adds a chunk to a thread's part of the norm.
__device__ __forceinline__ void add_chunk(const Chunk& c, int inf, double& sum) {
  const bool bf16 = c.t->bf16;
  uint4 v[kPieces];
  const uint4* p = reinterpret_cast<const uint4*>(static_cast<const char*>(c.t->grad) + c.from * (bf16 ? 2 : 4));
  const int live = c.pieces;
#pragma unroll
  for (int j = 0; j < kPieces; ++j) {
    const int i = j * kThreads + threadIdx.x;
    v[j] = i < live ? p[i] : make_uint4(0, 0, 0, 0);
  }
  if (c.head + c.last > 0 && static_cast<int>(threadIdx.x) < c.head + c.last) {
    const int i = threadIdx.x;
    const int64_t at = i < c.head ? i : c.from + static_cast<int64_t>(c.pieces) * (bf16 ? 8 : 4) + (i - c.head);
    const double g = value(*c.t, at);
    sum = inf ? larger(sum, fabs(g)) : sum + g * g;
  }
  if (inf) {
    const float top = __uint_as_float(bf16 ? largest<true>(v) : largest<false>(v));
    sum = larger(sum, static_cast<double>(top));
  } else {
    sum += bf16 ? squares<true>(v) : squares<false>(v);
  }
}

__device__ __forceinline__ float factor_of(double norm, double max_norm, double eps) {
  if (norm != norm) return __int_as_float(0x7FFFFFFF);  // whatever the bound
  const double f = max_norm / (norm + eps);
  return f > 1.0 || max_norm == INFINITY ? 1.f : static_cast<float>(f);
}

// Scales a chunk. Outputs that lie in their 16-byte granules as the gradients do are
// written by pieces, others one by one.
__device__ __forceinline__ void scale_chunk(const Chunk& c, float f) {
  const bool bf16 = c.t->bf16;
  const int es = bf16 ? 2 : 4, each = 16 / es;
  if (f == 1.f && c.t->out == c.t->grad) return;
  auto put = [&](int64_t i) {
    const float v = value(*c.t, i) * f;
    if (bf16) static_cast<__nv_bfloat16*>(c.t->out)[i] = __float2bfloat16_rn(v);
    else static_cast<float*>(c.t->out)[i] = v;
  };
  const int ends = c.head + c.last;
  if (static_cast<int>(threadIdx.x) < ends)
    put(static_cast<int>(threadIdx.x) < c.head ? threadIdx.x : c.from + static_cast<int64_t>(c.pieces) * each + (threadIdx.x - c.head));
  if (((reinterpret_cast<uintptr_t>(c.t->out) ^ reinterpret_cast<uintptr_t>(c.t->grad)) & 15) != 0) {
    for (int i = threadIdx.x; i < c.pieces * each; i += kThreads) put(c.from + i);
    return;
  }
  const uint4* p = reinterpret_cast<const uint4*>(static_cast<const char*>(c.t->grad) + c.from * es);
  uint4* o = reinterpret_cast<uint4*>(static_cast<char*>(c.t->out) + c.from * es);
  uint4 v[kPieces];
#pragma unroll
  for (int j = 0; j < kPieces; ++j) {
    const int i = j * kThreads + threadIdx.x;
    if (i < c.pieces) v[j] = p[i];
  }
  const uint64_t ff = pair_of(f);
#pragma unroll
  for (int j = 0; j < kPieces; ++j) {
    const int i = j * kThreads + threadIdx.x;
    if (i >= c.pieces) break;
    uint32_t w[4] = {v[j].x, v[j].y, v[j].z, v[j].w};
    if (bf16) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 q = of_pair(mul2(pair_in(w[e]), ff));
        const __nv_bfloat162 b = __floats2bfloat162_rn(q.x, q.y);
        w[e] = *reinterpret_cast<const uint32_t*>(&b);
      }
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) w[e] = __float_as_uint(__uint_as_float(w[e]) * f);
    }
    o[i] = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

template <int MOST>
__global__ void __launch_bounds__(kThreads, kNormCtas) k_grad_norm(const __grid_constant__ GradTable<MOST> tab, int inf, double* partial) {
  double sum = 0.0;
  for (uint32_t chunk = blockIdx.x; chunk < tab.chunks; chunk += gridDim.x) add_chunk(chunk_of(tab, chunk), inf, sum);
  sum = cta_join(sum, inf);
  if (threadIdx.x == 0) partial[blockIdx.x] = sum;
}

__device__ __forceinline__ double join_parts(const double* partial, int parts, int inf) {
  double sum = 0.0;
  for (int i = threadIdx.x; i < parts; i += kThreads) sum = inf ? larger(sum, partial[i]) : sum + partial[i];
  return cta_join(sum, inf);
}

// The norm and the factor of the parts; or, with `fold`, the parts joined to one.
__global__ void __launch_bounds__(kThreads) k_grad_join(const double* partial, int parts, int inf, double max_norm, double eps,
                                                        float* norm, float* factor, double* fold) {
  double sum = join_parts(partial, parts, inf);
  if (threadIdx.x != 0) return;
  if (fold) {
    *fold = sum;
    return;
  }
  if (!inf) sum = sqrt(sum);
  norm[0] = static_cast<float>(sum);
  if (factor) factor[0] = factor_of(sum, max_norm, eps);
}

// The chunks are taken from the last one on: the norm read it last, and it may be in L2.
template <int MOST>
__global__ void __launch_bounds__(kThreads, kScaleCtas) k_grad_scale(const __grid_constant__ GradTable<MOST> tab, const double* partial, int parts,
                                                                int inf, double max_norm, double eps, float* norm, float* factor) {
  double sum = join_parts(partial, parts, inf);
  if (!inf) sum = sqrt(sum);
  const float f = factor_of(sum, max_norm, eps);
  if (norm && blockIdx.x == 0 && threadIdx.x == 0) {
    norm[0] = static_cast<float>(sum);
    if (factor) factor[0] = f;
  }
  for (uint32_t chunk = blockIdx.x; chunk < tab.chunks; chunk += gridDim.x) scale_chunk(chunk_of(tab, tab.chunks - 1 - chunk), f);
}

// All of it for a short list.
__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kThreads)
    k_grad_small(const __grid_constant__ GradTable<kSmallTensors> tab, int inf, double max_norm, double eps, float* norm, float* factor, int scale) {
  __shared__ double parts[kCluster];
  cg::cluster_group cluster = cg::this_cluster();
  const unsigned rank = cluster.block_rank();
  double sum = 0.0;
  for (uint32_t chunk = rank; chunk < tab.chunks; chunk += kCluster) add_chunk(chunk_of(tab, chunk), inf, sum);
  sum = cta_join(sum, inf);
  cluster.sync();  // every CTA runs: its shared memory may be written
  if (threadIdx.x < kCluster) *cluster.map_shared_rank(&parts[rank], threadIdx.x) = sum;
  cluster.sync();
  sum = parts[0];
#pragma unroll
  for (int i = 1; i < kCluster; ++i) sum = inf ? larger(sum, parts[i]) : sum + parts[i];
  if (!inf) sum = sqrt(sum);
  const float f = factor_of(sum, max_norm, eps);
  if (rank == 0 && threadIdx.x == 0) {
    norm[0] = static_cast<float>(sum);
    if (factor) factor[0] = f;
  }
  if (scale)
    for (uint32_t chunk = rank; chunk < tab.chunks; chunk += kCluster) scale_chunk(chunk_of(tab, chunk), f);
}

uint32_t chunks_of(const GradTensor& t) {
  const int64_t pieces = (t.n - head_of(t)) / (t.bf16 ? 8 : 4);
  const int64_t n = (pieces + kThreads * kPieces - 1) / (kThreads * kPieces);
  return static_cast<uint32_t>(n < 1 ? 1 : n);
}
template <int MOST>
void fill(GradTable<MOST>& tab, const GradTensor* t, int n) {
  tab.n = n;
  tab.chunks = 0;
  for (int i = 0; i < n; ++i) {
    tab.t[i] = t[i];
    tab.t[i].chunk0 = tab.chunks;
    tab.chunks += chunks_of(t[i]);
  }
}
unsigned grid_of(uint32_t chunks, int most) { return chunks < static_cast<uint32_t>(most) ? chunks : most; }

template <int MOST>
cudaError_t norm_launch(const GradTensor* t, int n, int inf, int sms, double* partial, int* parts, cudaStream_t s) {
  GradTable<MOST> tab;
  fill(tab, t, n);
  *parts = static_cast<int>(grid_of(tab.chunks, grad_parts(sms)));
  k_grad_norm<MOST><<<*parts, kThreads, 0, s>>>(tab, inf, partial);
  return cudaGetLastError();
}
template <int MOST>
cudaError_t scale_launch(const GradTensor* t, int n, const GradJoin& j, int sms, cudaStream_t s) {
  GradTable<MOST> tab;
  fill(tab, t, n);
  k_grad_scale<MOST><<<grid_of(tab.chunks, kScaleCtas * sms), kThreads, 0, s>>>(tab, j.partial, j.parts, j.inf, j.max_norm, j.eps, j.norm, j.factor);
  return cudaGetLastError();
}

}  // namespace

// Parts of a norm that a launch leaves, at most.
int grad_parts(int sms) { return kNormCtas * sms; }

bool grad_small(const GradTensor* t, int n) {
  if (n > kSmallTensors) return false;
  uint32_t chunks = 0;
  for (int i = 0; i < n; ++i) {
    if (t[i].n > kSmallChunks * (kChunkBytes / 2)) return false;
    chunks += chunks_of(t[i]);
  }
  return chunks <= kSmallChunks;
}
cudaError_t launch_grad_small(const GradTensor* t, int n, const GradJoin& j, int scale, cudaStream_t s) {
  GradTable<kSmallTensors> tab;
  fill(tab, t, n);
  k_grad_small<<<kCluster, kThreads, 0, s>>>(tab, j.inf, j.max_norm, j.eps, j.norm, j.factor, scale);
  return cudaGetLastError();
}
cudaError_t launch_grad_norm(const GradTensor* t, int n, int inf, int sms, double* partial, int* parts, cudaStream_t s) {
  return n <= kSmallTensors  ? norm_launch<kSmallTensors>(t, n, inf, sms, partial, parts, s)
         : n <= kSomeTensors ? norm_launch<kSomeTensors>(t, n, inf, sms, partial, parts, s)
                             : norm_launch<kGradMaxTensors>(t, n, inf, sms, partial, parts, s);
}
cudaError_t launch_grad_join(const GradJoin& j, cudaStream_t s) {
  k_grad_join<<<1, kThreads, 0, s>>>(j.partial, j.parts, j.inf, j.max_norm, j.eps, j.norm, j.factor, nullptr);
  return cudaGetLastError();
}
cudaError_t launch_grad_fold(double* partial, int parts, int inf, cudaStream_t s) {
  k_grad_join<<<1, kThreads, 0, s>>>(partial, parts, inf, 0.0, 0.0, nullptr, nullptr, partial);
  return cudaGetLastError();
}
cudaError_t launch_grad_scale(const GradTensor* t, int n, const GradJoin& j, int sms, cudaStream_t s) {
  return n <= kSmallTensors  ? scale_launch<kSmallTensors>(t, n, j, sms, s)
         : n <= kSomeTensors ? scale_launch<kSomeTensors>(t, n, j, sms, s)
                             : scale_launch<kGradMaxTensors>(t, n, j, sms, s);
}

}  // namespace grpo
