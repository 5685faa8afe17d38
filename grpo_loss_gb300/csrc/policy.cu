// Clipped policy loss with a KL term, and its gradient by every token's log-probability:
//   w = logp - old (or its mean over the sequence), r = e^w,  x = ref - logp
//   l = -A min(r, 1 + hi) for A > 0,  -A max(min(r, dual), 1 - lo) for A < 0
//   loss = sum c (l + beta (e^x - 1 - x)),  dlogp = c (-A r [not clipped] - beta (e^x - 1))
// The weight c of a token needs the number of valid tokens (of its sequence, or of all),
// so that the mask is read first: a launch that counts, and one that does the rest; for few
// tokens one cluster of CTAs does both, with a barrier between.
// Bound by memory for many tokens (21 bytes each), with some 70 instructions each beside it.
#include <cooperative_groups.h>

#include "f32x2.cuh"
#include "internal.h"

namespace cg = cooperative_groups;

namespace grpo {

namespace {

constexpr int kThreads = 256;
constexpr int kTokens = 8;                   // of a thread at a time: their loads are in flight together
constexpr int kChunk = kThreads * kTokens;   // tokens a CTA takes at a time, at most
constexpr int kCluster = 8;
constexpr int kSmall = 16 * kChunk;          // tokens that one cluster takes

// ---------------------------------------------------------------- numbers
// The rounding error of s = a - b.
__device__ __forceinline__ float diff_error(float a, float b, float s) {
  const float v = __fsub_rn(s, a);
  return __fsub_rn(__fsub_rn(a, __fsub_rn(s, v)), __fadd_rn(b, v));
}
// A sum in two floats: what a float loses is kept in the second.
struct Sum2 {
  float hi = 0.f, lo = 0.f;
  __device__ __forceinline__ void add(float v) {
    const float s = __fadd_rn(hi, v), z = __fsub_rn(s, hi);
    lo += __fadd_rn(__fsub_rn(hi, __fsub_rn(s, z)), __fsub_rn(v, z));
    hi = s;
  }
  __device__ __forceinline__ double value() const { return static_cast<double>(hi) + static_cast<double>(lo); }
};

// e^x - 1 - x, of which e^x - 1 keeps too few digits near 0: there by the series
// x^2 (1/2 + x/6 + ... + x^8/10!), whose next term is below 2^-27 of it for |x| < 1/2; of
// two numbers at once.
__device__ __forceinline__ uint64_t series2(uint64_t x) {
  uint64_t p = pair_of(1.f / 3628800.f);
  p = fma2(p, x, pair_of(1.f / 362880.f));
  p = fma2(p, x, pair_of(1.f / 40320.f));
  p = fma2(p, x, pair_of(1.f / 5040.f));
  p = fma2(p, x, pair_of(1.f / 720.f));
  p = fma2(p, x, pair_of(1.f / 120.f));
  p = fma2(p, x, pair_of(1.f / 24.f));
  p = fma2(p, x, pair_of(1.f / 6.f));
  p = fma2(p, x, pair_of(0.5f));
  return mul2(mul2(x, x), p);
}
// {e^x - 1, e^x - 1 - x} of each of the pair.
__device__ __forceinline__ void exponentials(float x0, float x1, float (&em1)[2], float (&k)[2]) {
  const float2 s = of_pair(series2(pair_of(x0, x1)));
  k[0] = s.x, k[1] = s.y;
  em1[0] = x0 + k[0], em1[1] = x1 + k[1];
  if (!(fabsf(x0) < 0.5f)) {
    em1[0] = expm1f(x0);
    k[0] = em1[0] - x0;
  }
  if (!(fabsf(x1) < 0.5f)) {
    em1[1] = expm1f(x1);
    k[1] = em1[1] - x1;
  }
}

// ----------------------------------------------------------------- chunks
// A chunk: whole sequences of up to half its tokens, or a piece of a longer one.
struct Chunk {
  int64_t row0;
  int t0, rows, len;
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

__device__ __forceinline__ double warp_sum(double v) {
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
// Sums of a CTA in a fixed order, returned to its first warp.
template <int M>
__device__ void cta_sums(double (&v)[M]) {
  __shared__ double part[M][kThreads / 32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  __syncthreads();
#pragma unroll
  for (int m = 0; m < M; ++m) {
    v[m] = warp_sum(v[m]);
    if (lane == 0) part[m][warp] = v[m];
  }
  __syncthreads();
  if (warp == 0) {
#pragma unroll
    for (int m = 0; m < M; ++m) {
      v[m] = lane < kThreads / 32 ? part[m][lane] : 0.0;
#pragma unroll
      for (int o = kThreads / 64; o >= 1; o >>= 1) v[m] += __shfl_xor_sync(0xffffffffu, v[m], o);
    }
  }
}

// -------------------------------------------------------------- the count
__device__ __forceinline__ int nonzero_bytes(uint32_t w) {
  return __popc((((w & 0x7F7F7F7Fu) + 0x7F7F7F7Fu) | w) & 0x80808080u);
}
// Valid tokens among `len` bytes from p on: a lane's part.
__device__ __forceinline__ int count_bytes(const uint8_t* p, int len, int lane) {
  int n = 0, head = static_cast<int>(-reinterpret_cast<uintptr_t>(p) & 15);
  if (head > len) head = len;
  const int pieces = (len - head) / 16, last = (len - head) % 16;
  if (lane < head) n += p[lane] != 0;
  if (lane < last) n += p[head + 16 * pieces + lane] != 0;
  const uint4* q = reinterpret_cast<const uint4*>(p + head);
#pragma unroll 4
  for (int i = lane; i < pieces; i += 32) {
    const uint4 v = q[i];
    n += nonzero_bytes(v.x) + nonzero_bytes(v.y) + nonzero_bytes(v.z) + nonzero_bytes(v.w);
  }
  return n;
}

// Valid tokens of every segment (a sequence, or its piece), and with a sequence's ratio the
// sum of w of these: a warp a segment. Rows of few tokens: a thread a row.
__device__ void count_phase(const PolicyArgs& a, int cta, int ctas, bool w_too) {
  const int lane = threadIdx.x & 31;
  const int64_t segs = a.B * a.pieces, warps = static_cast<int64_t>(ctas) * (kThreads / 32);
  double total[1] = {0.0};
  const bool thin = a.T < 16;
  for (int64_t i = thin ? static_cast<int64_t>(cta) * kThreads + threadIdx.x
                        : static_cast<int64_t>(cta) * (kThreads / 32) + (threadIdx.x >> 5);
       i < segs; i += thin ? static_cast<int64_t>(ctas) * kThreads : warps) {
    const int64_t row = i / a.pieces, p = i - row * a.pieces;
    const int t0 = static_cast<int>(p * a.T / a.pieces), len = static_cast<int>((p + 1) * a.T / a.pieces) - t0;
    const uint8_t* m = a.mask + row * a.ld_mask + t0;
    const int step = thin ? 1 : 32, first = thin ? 0 : lane;
    int n = 0;
    Sum2 w;
    if (w_too) {
      const float *q = a.logp + row * a.ld_logp + t0, *o = a.old + row * a.ld_old + t0;
#pragma unroll 8
      for (int t = first; t < len; t += step) {
        const bool valid = m[t] != 0;
        const float u = q[t], v = o[t], s = __fsub_rn(u, v);
        n += valid;
        const float z = valid ? s : 0.f;
        w.add(z);
        const float e = diff_error(u, v, s);
        if (valid && isfinite(s)) w.lo += e;
      }
    } else if (thin) {
      for (int t = 0; t < len; ++t) n += m[t] != 0;
    } else {
      n = count_bytes(m, len, lane);
    }
    double sum = 0.0;
    if (w_too) {
      // (a sum that is not finite has no second part)
      sum = isfinite(w.hi) ? w.value() : static_cast<double>(w.hi);
      if (!thin) sum = warp_sum(sum);
    }
    if (!thin) n = __reduce_add_sync(0xffffffffu, n);
    if (thin || lane == 0) {
      a.seg_count[i] = n;
      if (w_too) a.seg_w[i] = sum;
      total[0] += n;
    }
  }
  cta_sums(total);
  if (threadIdx.x == 0) a.cta_count[cta] = static_cast<int64_t>(total[0]);
}

// --------------------------------------------------------------- the loss
enum : int { S_LOSS, S_KL, S_RATIO, S_LOW, S_HIGH, S_VALID, S_ALL };
enum : int { W_NONE, W_TOKEN, W_SEQUENCE };

// What a sequence's tokens share: the weight c, the advantage where it is one for all, and
// the ratio where that is (its sides of the bounds in three bits).
struct Row {
  float c, em1;
  int sides;
};

// Which bounds w is beyond: 1 above the upper, 2 below the lower, 4 above the dual one. w
// rounds a difference (lo: what it lost) and a bound's log is held in two floats: where the
// first ones are equal the second decide.
__device__ __forceinline__ int sides_of(const PolicyArgs& a, float w, float lo) {
  auto above = [&](float hi, float l) { return w > hi || (w == hi && lo > l); };
  return (above(a.up_hi, a.up_lo) ? 1 : 0) | (w < a.down_hi || (w == a.down_hi && lo < a.down_lo) ? 2 : 0) |
         (above(a.far_hi, a.far_lo) ? 4 : 0);
}

template <int W, bool REF>
__device__ void loss_phase(const PolicyArgs& a, int cta, int ctas, double (&sums)[S_ALL]) {
  __shared__ Row s_row[kChunk];
  __shared__ double s_total;
  __shared__ int s_valid;
  if (a.reduce == 1) {
    double v[1] = {0.0};
    for (int i = threadIdx.x; i < a.count_ctas; i += kThreads) v[0] += static_cast<double>(a.cta_count[i]);
    cta_sums(v);
    if (threadIdx.x == 0) s_total = v[0];
    __syncthreads();
  }
#pragma unroll
  for (int m = 0; m < S_ALL; ++m) sums[m] = 0.0;
  const double same = a.reduce == 1 ? 1.0 / s_total : a.inv_divisor;  // (unused with a weight for each sequence)
  for (int64_t ch = cta; ch < a.chunks; ch += ctas) {
    const Chunk k = chunk_of(a, ch);
    __syncthreads();  // the last chunk's rows have been read
    if (threadIdx.x == 0) s_valid = 0;
    __syncthreads();
    // the rows of the chunk, a thread each (a piece's sequence: one warp, a lane a piece)
    if (k.rows == 1) {
      if (threadIdx.x < 32) {
        double n = 0.0, w = 0.0;
        for (int64_t p = threadIdx.x; p < a.pieces; p += 32) {
          n += a.seg_count[k.row0 * a.pieces + p];
          if (W == W_SEQUENCE) w += a.seg_w[k.row0 * a.pieces + p];
        }
        n = warp_sum(n);
        if (W == W_SEQUENCE) w = warp_sum(w);
        const int here = a.seg_count[a.pieces > 1 ? ch : k.row0];
        if (threadIdx.x == 0 && here > 0) {
          const double c = a.reduce == 0 ? 1.0 / (static_cast<double>(a.B) * n) : same;
          Row r = {static_cast<float>(c), 0.f, 0};
          if (W == W_SEQUENCE) {
            const double mean = w / n;
            const float hi = static_cast<float>(mean);
            r.em1 = static_cast<float>(expm1(mean));
            r.sides = sides_of(a, hi, static_cast<float>(mean - static_cast<double>(hi)));
          }
          s_row[0] = r;
          s_valid = here;
          sums[S_VALID] += here;
          if (!a.token_adv) sums[S_LOSS] -= c * here * static_cast<double>(a.adv[k.row0]);
        }
      }
    } else {
      int some = 0;
      for (int i = threadIdx.x; i < k.rows; i += kThreads) {
        const int n = a.seg_count[k.row0 + i];
        if (n == 0) continue;
        const double c = a.reduce == 0 ? 1.0 / (static_cast<double>(a.B) * n) : same;
        Row r = {static_cast<float>(c), 0.f, 0};
        if (W == W_SEQUENCE) {
          const double mean = a.seg_w[k.row0 + i] / n;
          const float hi = static_cast<float>(mean);
          r.em1 = static_cast<float>(expm1(mean));
          r.sides = sides_of(a, hi, static_cast<float>(mean - static_cast<double>(hi)));
        }
        s_row[i] = r;
        some = 1;
        sums[S_VALID] += n;
        if (!a.token_adv) sums[S_LOSS] -= c * n * static_cast<double>(a.adv[k.row0 + i]);
      }
      if (some) s_valid = 1;
    }
    __syncthreads();
    const int all = k.rows * k.len;
    if (s_valid == 0) {  // nothing but the gradient's zeros
      if (a.dlogp)
        for (int i = threadIdx.x; i < all; i += kThreads) {
          const int r = k.rows == 1 ? 0 : i / k.len;
          a.dlogp[(k.row0 + r) * a.ld_dlogp + k.t0 + (i - r * k.len)] = 0.f;
        }
      continue;
    }
    float q[kTokens], o[kTokens], p[kTokens], A[kTokens];
    bool valid[kTokens];
    int at[kTokens], of[kTokens];  // token and row of the chunk
#pragma unroll
    for (int j = 0; j < kTokens; ++j) {
      const int i = j * kThreads + threadIdx.x;
      of[j] = k.rows == 1 ? 0 : i / k.len;
      at[j] = k.t0 + (i - of[j] * k.len);
      valid[j] = i < all;
      q[j] = o[j] = p[j] = A[j] = 0.f;
      if (valid[j]) {
        const int64_t row = k.row0 + of[j];
        valid[j] = a.mask[row * a.ld_mask + at[j]] != 0;
        q[j] = a.logp[row * a.ld_logp + at[j]];
        if (W == W_TOKEN) o[j] = a.old[row * a.ld_old + at[j]];
        if (REF) p[j] = a.ref[row * a.ld_ref + at[j]];
        A[j] = a.adv[a.token_adv ? row * a.ld_adv + at[j] : row];
      }
    }
    // float32 sums of a thread's few tokens
    float loss = 0.f, kls = 0.f, rs = 0.f;
    Sum2 base;
    int low = 0, high = 0;
#pragma unroll
    for (int j = 0; j < kTokens; j += 2) {
      float em1[2] = {0.f, 0.f}, k0[2], x1[2], kl[2] = {0.f, 0.f};
      float w[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        w[e] = valid[j + e] ? __fsub_rn(q[j + e], o[j + e]) : 0.f;
        x1[e] = REF && valid[j + e] ? p[j + e] - q[j + e] : 0.f;
      }
      if (W == W_TOKEN) exponentials(w[0], w[1], em1, k0);
      if (REF) exponentials(x1[0], x1[1], x1, kl);  // x1: now e^x - 1
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const Row r = s_row[of[j + e]];
        float d = 0.f;
        if (valid[j + e]) {
          int sides = 0;
          if (W == W_SEQUENCE) {
            em1[e] = r.em1;
            sides = r.sides;
          } else if (W == W_TOKEN) {
            float lo = 0.f;
            if (w[e] == a.up_hi || w[e] == a.down_hi || w[e] == a.far_hi) lo = diff_error(q[j + e], o[j + e], w[e]);
            sides = sides_of(a, w[e], lo);
          }
          const float Ae = A[j + e];
          const bool up = Ae > 0.f && (sides & 1), down = Ae < 0.f && (sides & 2), far = Ae < 0.f && (sides & 4) && !down;
          const float held = up ? a.e_up : down ? a.e_down : far ? a.e_far : em1[e];  // less 1
          float l = Ae == 0.f ? 0.f : -Ae * held;
          float g = up || down || far || Ae == 0.f ? 0.f : -fmaf(Ae, em1[e], Ae);
          if (REF) {
            l = fmaf(a.beta, kl[e], l);
            g = fmaf(-a.beta, x1[e], g);
          }
          d = r.c * g;
          if (a.token_adv) base.add(k.rows == 1 ? Ae : r.c * Ae);
          loss += k.rows == 1 ? l : r.c * l;
          kls += kl[e];
          rs += em1[e];
          low += down;
          high += up || far;
        }
        if (a.dlogp && (j + e) * kThreads + static_cast<int>(threadIdx.x) < all)
          a.dlogp[(k.row0 + of[j + e]) * a.ld_dlogp + at[j + e]] = d;
      }
    }
    double l = static_cast<double>(loss);
    if (a.token_adv) l -= base.value();
    if (k.rows == 1) l *= a.reduce == 0 ? static_cast<double>(s_row[0].c) : same;
    sums[S_LOSS] += l;
    if (REF) sums[S_KL] += static_cast<double>(kls);
    if (W != W_NONE) sums[S_RATIO] += static_cast<double>(rs);
    sums[S_LOW] += low;
    sums[S_HIGH] += high;
  }
  cta_sums(sums);
}

// By the first thread of the CTA that has every CTA's sums.
__device__ void finish(const PolicyArgs& a, const double (&sums)[S_ALL]) {
  const double n = sums[S_VALID] > 1.0 ? sums[S_VALID] : 1.0;
  a.loss[0] = static_cast<float>(sums[S_LOSS]);
  if (a.stats) {
    a.stats[0] = static_cast<float>(sums[S_KL] / n);
    a.stats[1] = static_cast<float>(sums[S_LOW] / n);
    a.stats[2] = static_cast<float>(sums[S_HIGH] / n);
    a.stats[3] = static_cast<float>((sums[S_VALID] + sums[S_RATIO]) / n);
  }
}

__global__ void __launch_bounds__(kThreads) k_policy_count(PolicyArgs a) {
  if (blockIdx.x == 0 && threadIdx.x == 0) *a.ticket = 0;
  count_phase(a, blockIdx.x, gridDim.x, a.sequence_ratio);
}

template <int W, bool REF>
__global__ void __launch_bounds__(kThreads) k_policy_loss(PolicyArgs a) {
  __shared__ bool s_last;
  double sums[S_ALL];
  loss_phase<W, REF>(a, blockIdx.x, gridDim.x, sums);
  if (threadIdx.x == 0) {
#pragma unroll
    for (int m = 0; m < S_ALL; ++m) a.partial[S_ALL * blockIdx.x + m] = sums[m];
    __threadfence();
    s_last = atomicAdd(a.ticket, 1u) == gridDim.x - 1;
  }
  __syncthreads();
  if (!s_last) return;  // the last CTA joins what all have left, in their order
  __threadfence();
#pragma unroll
  for (int m = 0; m < S_ALL; ++m) sums[m] = 0.0;
  for (int i = threadIdx.x; i < static_cast<int>(gridDim.x); i += kThreads)
#pragma unroll
    for (int m = 0; m < S_ALL; ++m) sums[m] += a.partial[S_ALL * i + m];
  cta_sums(sums);
  if (threadIdx.x == 0) finish(a, sums);
}

// Both for few tokens.
template <int W, bool REF>
__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kThreads) k_policy_small(PolicyArgs a) {
  __shared__ double parts[kCluster][S_ALL];
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = static_cast<int>(cluster.block_rank());
  count_phase(a, rank, kCluster, W == W_SEQUENCE);
  __threadfence();
  cluster.sync();
  double sums[S_ALL];
  loss_phase<W, REF>(a, rank, kCluster, sums);
  if (threadIdx.x == 0) {
    double* to = cluster.map_shared_rank(&parts[0][0], 0);
#pragma unroll
    for (int m = 0; m < S_ALL; ++m) to[rank * S_ALL + m] = sums[m];
  }
  cluster.sync();
  if (rank == 0 && threadIdx.x == 0) {
#pragma unroll
    for (int m = 0; m < S_ALL; ++m) {
      sums[m] = 0.0;
      for (int i = 0; i < kCluster; ++i) sums[m] += parts[i][m];
    }
    finish(a, sums);
  }
}

bool small(const PolicyArgs& a) { return a.B * a.T <= kSmall; }

template <int W, bool REF>
cudaError_t loss_launch(const PolicyArgs& a, cudaStream_t s) {
  if (small(a)) k_policy_small<W, REF><<<kCluster, kThreads, 0, s>>>(a);
  else k_policy_loss<W, REF><<<a.loss_ctas, kThreads, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace

// Fills in how the tokens are cut into chunks, and the places in the workspace.
size_t policy_plan(PolicyArgs& a, int sms, void* workspace) {
  a.pieces = a.T > kChunk ? (a.T + kChunk - 1) / kChunk : 1;
  a.rows_per_chunk = a.T > kChunk / 2 || a.T < 1 ? 1 : kChunk / a.T;
  a.chunks = a.pieces > 1 ? a.B * a.pieces : (a.B + a.rows_per_chunk - 1) / a.rows_per_chunk;
  const int64_t most = 8ll * sms;
  a.loss_ctas = static_cast<int>(a.chunks < 3ll * sms ? a.chunks : 3ll * sms);
  const int64_t segs = a.B * a.pieces, want = (segs + kThreads / 32 - 1) / (kThreads / 32);
  a.count_ctas = small(a) ? kCluster : static_cast<int>(want < most ? want : most);
  size_t at = 0;
  auto take = [&](size_t bytes) {
    char* p = static_cast<char*>(workspace) + at;
    at += (bytes + 255) / 256 * 256;
    return static_cast<void*>(p);
  };
  a.ticket = static_cast<unsigned*>(take(4));
  a.cta_count = static_cast<int64_t*>(take(8 * most));
  a.partial = static_cast<double*>(take(8 * S_ALL * most));
  a.seg_count = static_cast<int*>(take(4 * segs));
  a.seg_w = static_cast<double*>(take(a.sequence_ratio ? 8 * segs : 0));
  return at;
}

bool policy_counts_first(const PolicyArgs& a) { return !small(a); }
cudaError_t launch_policy_count(const PolicyArgs& a, cudaStream_t s) {
  k_policy_count<<<a.count_ctas, kThreads, 0, s>>>(a);
  return cudaGetLastError();
}
cudaError_t launch_policy_loss(const PolicyArgs& a, cudaStream_t s) {
  const int w = !a.old ? W_NONE : a.sequence_ratio ? W_SEQUENCE : W_TOKEN;
  if (a.ref)
    return w == W_NONE    ? loss_launch<W_NONE, true>(a, s)
           : w == W_TOKEN ? loss_launch<W_TOKEN, true>(a, s)
                          : loss_launch<W_SEQUENCE, true>(a, s);
  return w == W_NONE    ? loss_launch<W_NONE, false>(a, s)
         : w == W_TOKEN ? loss_launch<W_TOKEN, false>(a, s)
                        : loss_launch<W_SEQUENCE, false>(a, s);
}

}  // namespace grpo
