// Clipped policy loss with a KL term, and its gradient by every token's log-probability:
//   w = logp - old (or its mean over the sequence), r = e^w,  x = ref - logp
//   l = -A min(r, 1 + hi) for A > 0,  -A max(min(r, dual), 1 - lo) for A < 0
//   loss = sum c (l + beta (e^x - 1 - x)),  dlogp = c (-A r [not clipped] - beta (e^x - 1))
// The weight c of a token needs the number of valid tokens (of its sequence, or of all),
// so that the mask is read first: a launch that counts, and one that does the rest.
#include "internal.h"

namespace grpo {

namespace {

constexpr int kThreads = 256;
constexpr int kChunk = 2048;  // tokens a CTA takes at a time, at most

// log of a bound in two floats: the sign of w - bound is that of exact numbers but for
// differences below 2^-48 of the bound.
struct Wide {
  float hi, lo;
};

__device__ __forceinline__ Wide two_diff(float a, float b) {  // a - b, exactly
  const float s = __fsub_rn(a, b), v = __fsub_rn(s, a);
  return {s, __fsub_rn(__fsub_rn(a, __fsub_rn(s, v)), __fadd_rn(b, v))};
}
__device__ __forceinline__ bool above(const Wide& w, float hi, float lo) {
  return w.hi > hi || (w.hi == hi && w.lo > lo);
}
__device__ __forceinline__ bool below(const Wide& w, float hi, float lo) {
  return w.hi < hi || (w.hi == hi && w.lo < lo);
}

// e^x - 1 - x, which has lost most digits near 0 when it is formed from e^x - 1: there
// the series x^2 (1/2 + x/6 + ...), whose next term is below 2^-26 of it for |x| < 1/2.
__device__ __forceinline__ float kl_term(float x, float em1) {
  if (fabsf(x) >= 0.5f) return em1 - x;
  float p = 1.f / 3628800.f;
  p = fmaf(p, x, 1.f / 362880.f);
  p = fmaf(p, x, 1.f / 40320.f);
  p = fmaf(p, x, 1.f / 5040.f);
  p = fmaf(p, x, 1.f / 720.f);
  p = fmaf(p, x, 1.f / 120.f);
  p = fmaf(p, x, 1.f / 24.f);
  p = fmaf(p, x, 1.f / 6.f);
  p = fmaf(p, x, 0.5f);
  return p * x * x;
}

__device__ __forceinline__ double warp_sum(double v) {
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Sums of a CTA in a fixed order, returned to thread 0.
template <int M>
__device__ void cta_sums(double (&v)[M]) {
  __shared__ double part[M][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
#pragma unroll
  for (int m = 0; m < M; ++m) {
    v[m] = warp_sum(v[m]);
    if (lane == 0) part[m][warp] = v[m];
  }
  __syncthreads();
  if (warp == 0) {
#pragma unroll
    for (int m = 0; m < M; ++m) v[m] = warp_sum(lane < warps ? part[m][lane] : 0.0);
  }
  __syncthreads();
}

// A chunk: `rows` sequences of a piece of `len` tokens each (one sequence, or a piece of
// one, or several whole short ones).
struct Chunk {
  int64_t row0;
  int t0, rows, len, seg0;  // seg0: the first's segment
};
__device__ __forceinline__ Chunk chunk_of(const PolicyArgs& a, int64_t c) {
  Chunk k;
  if (a.pieces > 1) {
    k.row0 = c / a.pieces;
    const int64_t p = c - k.row0 * a.pieces;
    k.t0 = static_cast<int>(p * a.T / a.pieces);
    k.len = static_cast<int>((p + 1) * a.T / a.pieces) - k.t0;
    k.rows = 1;
  } else {
    k.row0 = c * a.rows_per_chunk;
    k.rows = static_cast<int>(a.B - k.row0 < a.rows_per_chunk ? a.B - k.row0 : a.rows_per_chunk);
    k.t0 = 0;
    k.len = static_cast<int>(a.T);
  }
  return k;
}

// Valid tokens of every segment (a sequence's piece), and the sum of w of these.
__global__ void __launch_bounds__(kThreads) k_policy_count(PolicyArgs a) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = kThreads / 32;
  if (blockIdx.x == 0 && threadIdx.x == 0) *a.ticket = 0;
  double total[1] = {0.0};
  for (int64_t c = blockIdx.x; c < a.chunks; c += gridDim.x) {
    const Chunk k = chunk_of(a, c);
    if (k.rows == 1) {
      double v[2] = {0.0, 0.0};
      const uint8_t* m = a.mask + k.row0 * a.ld_mask + k.t0;
      const float *q = a.logp + k.row0 * a.ld_logp + k.t0, *o = a.old + k.row0 * a.ld_old + k.t0;
      int n = 0;
      for (int t = threadIdx.x; t < k.len; t += kThreads) {
        if (m[t]) {
          ++n;
          if (a.sequence_ratio) v[1] += static_cast<double>(q[t]) - static_cast<double>(o[t]);
        }
      }
      v[0] = n;
      cta_sums(v);
      if (threadIdx.x == 0) {
        const int64_t s = a.pieces > 1 ? c : k.row0;
        a.seg_count[s] = static_cast<int>(v[0]);
        if (a.sequence_ratio) a.seg_w[s] = v[1];
        total[0] += v[0];
      }
    } else {
      for (int r = warp; r < k.rows; r += warps) {
        const int64_t row = k.row0 + r;
        const uint8_t* m = a.mask + row * a.ld_mask;
        int n = 0;
        double w = 0.0;
        for (int t = lane; t < k.len; t += 32) {
          if (m[t]) {
            ++n;
            if (a.sequence_ratio)
              w += static_cast<double>(a.logp[row * a.ld_logp + t]) - static_cast<double>(a.old[row * a.ld_old + t]);
          }
        }
        n = __reduce_add_sync(0xffffffffu, n);
        if (a.sequence_ratio) w = warp_sum(w);
        if (lane == 0) {
          a.seg_count[row] = n;
          if (a.sequence_ratio) a.seg_w[row] = w;
          total[0] += n;
        }
      }
    }
  }
  cta_sums(total);
  if (threadIdx.x == 0) a.cta_count[blockIdx.x] = static_cast<int64_t>(total[0]);
}

enum : int { S_LOSS, S_KL, S_RATIO, S_LOW, S_HIGH, S_VALID, S_ALL };

__global__ void __launch_bounds__(kThreads) k_policy_loss(PolicyArgs a) {
  __shared__ double s_total;
  __shared__ bool s_last;
  double v[1] = {0.0};
  if (a.reduce == 1) {
    for (int i = threadIdx.x; i < a.count_ctas; i += kThreads) v[0] += static_cast<double>(a.cta_count[i]);
    cta_sums(v);
    if (threadIdx.x == 0) s_total = v[0];
    __syncthreads();
  }
  double sums[S_ALL] = {};
  for (int64_t c = blockIdx.x; c < a.chunks; c += gridDim.x) {
    const Chunk k = chunk_of(a, c);
    for (int i = threadIdx.x; i < k.rows * k.len; i += kThreads) {
      const int r = k.rows == 1 ? 0 : i / k.len, t = k.t0 + (i - r * k.len);
      const int64_t row = k.row0 + r;
      float d = 0.f;
      if (a.mask[row * a.ld_mask + t]) {
        double n = 1.0, ws = 0.0;
        if (a.reduce == 0 || a.sequence_ratio) {
          n = 0.0;
          for (int p = 0; p < a.pieces; ++p) {
            n += a.seg_count[row * a.pieces + p];
            if (a.sequence_ratio) ws += a.seg_w[row * a.pieces + p];
          }
        }
        const double cd = a.reduce == 0 ? 1.0 / (static_cast<double>(a.B) * n) : a.reduce == 1 ? 1.0 / s_total : a.inv_divisor;
        const float weight = static_cast<float>(cd);
        const float q = a.logp[row * a.ld_logp + t];
        const float A = a.adv[a.token_adv ? row * a.ld_adv + t : row];
        Wide w = {0.f, 0.f};
        if (a.sequence_ratio) {
          const double m = ws / n;
          w.hi = static_cast<float>(m);
          w.lo = static_cast<float>(m - static_cast<double>(w.hi));
        } else if (a.old) {
          w = two_diff(q, a.old[row * a.ld_old + t]);
        }
        float ratio = expf(w.hi);
        ratio = isfinite(w.lo) && isfinite(ratio) ? fmaf(ratio, w.lo, ratio) : ratio;
        const bool up = above(w, a.up_hi, a.up_lo), down = below(w, a.down_hi, a.down_lo), far = above(w, a.far_hi, a.far_lo);
        const bool high = A > 0.f ? up : A < 0.f && far, low = A < 0.f && down;
        const float held = A > 0.f ? (up ? a.r_up : ratio) : down ? a.r_down : far ? a.r_far : ratio;
        float l = A == 0.f ? 0.f : -A * held;
        float g = high || low || A == 0.f ? 0.f : -A * ratio;
        float kl = 0.f;
        if (a.ref) {
          const float x = a.ref[row * a.ld_ref + t] - q, e = expm1f(x);
          kl = kl_term(x, e);
          l = fmaf(a.beta, kl, l);
          g = fmaf(-a.beta, e, g);
        }
        d = weight * g;
        sums[S_LOSS] += cd * static_cast<double>(l);
        sums[S_KL] += kl;
        sums[S_RATIO] += ratio;
        sums[S_LOW] += low;
        sums[S_HIGH] += high;
        sums[S_VALID] += 1.0;
      }
      if (a.dlogp) a.dlogp[row * a.ld_dlogp + t] = d;
    }
  }
  cta_sums(sums);
  if (threadIdx.x == 0) {
#pragma unroll
    for (int m = 0; m < S_ALL; ++m) a.partial[S_ALL * blockIdx.x + m] = sums[m];
    __threadfence();
    s_last = atomicAdd(a.ticket, 1u) == gridDim.x - 1;
  }
  __syncthreads();
  if (!s_last) return;
  __threadfence();
#pragma unroll
  for (int m = 0; m < S_ALL; ++m) sums[m] = 0.0;
  for (int i = threadIdx.x; i < static_cast<int>(gridDim.x); i += kThreads)
#pragma unroll
    for (int m = 0; m < S_ALL; ++m) sums[m] += a.partial[S_ALL * i + m];
  cta_sums(sums);
  if (threadIdx.x == 0) {
    const double n = sums[S_VALID] > 1.0 ? sums[S_VALID] : 1.0;
    a.loss[0] = static_cast<float>(sums[S_LOSS]);
    if (a.stats) {
      a.stats[0] = static_cast<float>(sums[S_KL] / n);
      a.stats[1] = static_cast<float>(sums[S_LOW] / n);
      a.stats[2] = static_cast<float>(sums[S_HIGH] / n);
      a.stats[3] = static_cast<float>(sums[S_RATIO] / n);
    }
  }
}

}  // namespace

// Fills in how the tokens are cut into chunks, and the places in the workspace.
size_t policy_plan(PolicyArgs& a, int sms, void* workspace) {
  a.pieces = a.T > kChunk ? (a.T + kChunk - 1) / kChunk : 1;
  a.rows_per_chunk = a.T >= kChunk / 2 || a.T < 1 ? 1 : kChunk / a.T;
  a.chunks = a.pieces > 1 ? a.B * a.pieces : (a.B + a.rows_per_chunk - 1) / a.rows_per_chunk;
  const int64_t most = 8ll * sms;
  a.count_ctas = static_cast<int>(a.chunks < most ? a.chunks : most);
  size_t at = 0;
  auto take = [&](size_t bytes) {
    char* p = static_cast<char*>(workspace) + at;
    at += (bytes + 255) / 256 * 256;
    return static_cast<void*>(p);
  };
  const size_t segs = static_cast<size_t>(a.B) * a.pieces;
  a.ticket = static_cast<unsigned*>(take(4));
  a.cta_count = static_cast<int64_t*>(take(8 * most));
  a.partial = static_cast<double*>(take(8 * S_ALL * most));
  a.seg_count = static_cast<int*>(take(4 * segs));
  a.seg_w = static_cast<double*>(take(a.sequence_ratio ? 8 * segs : 0));
  return at;
}

cudaError_t launch_policy_count(const PolicyArgs& a, cudaStream_t s) {
  k_policy_count<<<a.count_ctas, kThreads, 0, s>>>(a);
  return cudaGetLastError();
}
cudaError_t launch_policy_loss(const PolicyArgs& a, cudaStream_t s) {
  k_policy_loss<<<a.count_ctas, kThreads, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace grpo
