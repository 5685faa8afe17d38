// Clipped policy loss with a KL term, and its gradient by every token's log-probability:
//   w = logp - old (or its mean over the sequence), r = e^w,  x = ref - logp
//   l = -A min(r, 1 + hi) for A > 0,  -A max(min(r, dual), 1 - lo) for A < 0
//   loss = sum c (l + beta (e^x - 1 - x)),  dlogp = c (-A r [not clipped] - beta (e^x - 1))
// The weight c of a token needs the number of valid tokens (of its sequence, or of all),
// so that the mask is read first: a launch that counts, and one that does the rest; for few
// tokens one cluster of CTAs does both, with a barrier between.
// Bound by memory and by the instructions beside it for many tokens (21 bytes each).
#include <cooperative_groups.h>

#include "f32x2.cuh"
#include "internal.h"

namespace cg = cooperative_groups;

namespace grpo {

namespace {

constexpr int kThreads = 256;
constexpr int kTokens = 8;                   // of a thread at a time: their loads are in flight together
constexpr int kChunk = kThreads * kTokens;   // tokens a CTA takes at a time, at most
constexpr int kLossCtas = 3;                 // of an SM, at a time
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
  __device__ __forceinline__ void add_product(float a, float b) {
    const float v = __fmul_rn(a, b);
    add(v);
    lo += __fmaf_rn(a, b, -v);
  }
  __device__ __forceinline__ double value() const { return static_cast<double>(hi) + static_cast<double>(lo); }
};

// e^x - 1 and e^x - 1 - x of two numbers: x = n ln 2 + f with |f| <= ln 2 / 2 (Cody and
// Waite's reduction, ln 2 in two floats), e^f - 1 - f by its series f^2 (1/2 + f/6 + ... +
// f^6/8!), whose next term is below 2^-28 of it, and e^x - 1 = 2^n (e^f - 1) + 2^n - 1. Both
// keep their digits near 0, where e^x less 1 and less x would not.
template <bool K>
__device__ __forceinline__ void exponentials(float x0, float x1, float (&em1)[2], float (&k)[2]) {
  constexpr float kMagic = 12582912.f;  // 1.5 * 2^23: the sum's low bits are the nearest integer
  const uint64_t x = pair_of(x0, x1);
  const uint64_t t = fma2(x, pair_of(1.44269504f), pair_of(kMagic)), n = add2(t, pair_of(-kMagic));
  const uint64_t f = fma2(n, pair_of(1.90465421e-9f), fma2(n, pair_of(-0.693147182f), x));
  uint64_t p = pair_of(1.f / 40320.f);
  p = fma2(p, f, pair_of(1.f / 5040.f));
  p = fma2(p, f, pair_of(1.f / 720.f));
  p = fma2(p, f, pair_of(1.f / 120.f));
  p = fma2(p, f, pair_of(1.f / 24.f));
  p = fma2(p, f, pair_of(1.f / 6.f));
  p = fma2(p, f, pair_of(0.5f));
  const uint64_t kf = mul2(mul2(f, f), p);
  const float2 tt = of_pair(t), kk = of_pair(kf);
  const int t0 = __float_as_int(tt.x), t1 = __float_as_int(tt.y);
  const uint64_t two_n = pair_of(__int_as_float((t0 << 23) + 0x3F800000), __int_as_float((t1 << 23) + 0x3F800000));
  const float2 e = of_pair(fma2(two_n, add2(f, kf), add2(two_n, pair_of(-1.f))));
  em1[0] = e.x, em1[1] = e.y;
  if (K) {
    const int zero = __float_as_int(kMagic);
    k[0] = t0 == zero ? kk.x : em1[0] - x0;
    k[1] = t1 == zero ? kk.y : em1[1] - x1;
  }
  // 2^n beyond float32's range, and what is not a number
  if (!(fabsf(x0) < 80.f && fabsf(x1) < 80.f)) {
    if (!(fabsf(x0) < 80.f)) {
      em1[0] = expm1f(x0);
      if (K) k[0] = em1[0] - x0;
    }
    if (!(fabsf(x1) < 80.f)) {
      em1[1] = expm1f(x1);
      if (K) k[1] = em1[1] - x1;
    }
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
// Sums of a CTA in a fixed order, returned to its first thread.
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
  double total[1] = {0.0};  // (whole numbers)
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
  if (a.reduce != 1) return;
  cta_sums(total);
  if (threadIdx.x == 0) a.cta_count[cta] = static_cast<int64_t>(total[0]);
}

// --------------------------------------------------------------- the loss
enum : int { S_LOSS, S_KL, S_RATIO, S_LOW, S_HIGH, S_VALID, S_ALL };
enum : int { W_NONE, W_TOKEN, W_SEQUENCE };

// What a sequence's tokens share: the weight c, the advantage where it is one for all, and
// the ratio where that is: the difference w's two floats, e^w - 1.
struct Row {
  float c, A, w, lo, em1;
};
// Which bound a token's ratio is held by.
struct Side {
  bool above, below;
  float held;  // the ratio less 1, held
};
// w rounds a difference (lo gives what it lost) and a bound's log is held in two floats:
// where the first ones are equal the second decide.
template <typename Lo>
__device__ __forceinline__ Side side_of(const PolicyArgs& a, float A, float w, float em1, Lo lo) {
  // the upper bound is 1 + clip_high, or dual_clip for A < 0; the lower one is for A < 0 alone
  const bool neg = A < 0.f;
  const float top = neg ? a.far_hi : a.up_hi, bottom = neg ? a.down_hi : -INFINITY;
  Side s;
  s.above = w > top;
  s.below = w < bottom;
  if (w == top || w == bottom) {
    const float l = lo();
    s.above = w == top && l > (neg ? a.far_lo : a.up_lo);
    s.below = w == bottom && l < (neg ? a.down_lo : 0.f);
  }
  s.held = s.above ? (neg ? a.e_far : a.e_up) : s.below ? a.e_down : em1;
  return s;
}

// A thread's sums.
struct Sums {
  Sum2 loss, kl, ratio;  // ratio: of r - 1
  int low = 0, high = 0;
  int64_t valid = 0;
  double base = 0.0;     // of the loss: -c A of tokens with one advantage for their sequence
};

// Two tokens (all zeros where masked): their gradients over c, their terms of the loss over
// c into l, and the statistics.
template <int W, bool REF>
__device__ __forceinline__ void two_tokens(const PolicyArgs& a, const Row& r0, const Row& r1, const float (&q)[2], const float (&o)[2],
                                           const float (&p)[2], const float (&A)[2], float (&g)[2], float (&l)[2], float& kls, float& rs,
                                           Sums& sums) {
  float em1[2] = {W == W_SEQUENCE ? r0.em1 : 0.f, W == W_SEQUENCE ? r1.em1 : 0.f}, ex[2], kl[2] = {0.f, 0.f}, none[2];
  float w[2] = {r0.w, r1.w};
  if (W == W_TOKEN) {
    w[0] = __fsub_rn(q[0], o[0]), w[1] = __fsub_rn(q[1], o[1]);
    exponentials<false>(w[0], w[1], em1, none);
  }
  if (REF) exponentials<true>(p[0] - q[0], p[1] - q[1], ex, kl);
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const Row& r = e ? r1 : r0;
    Side s = {false, false, em1[e]};
    if (W != W_NONE) s = side_of(a, A[e], w[e], em1[e], [&] { return W == W_TOKEN ? diff_error(q[e], o[e], w[e]) : r.lo; });
    const bool some = A[e] != 0.f;
    l[e] = some ? -A[e] * s.held : 0.f;
    g[e] = some && !s.above && !s.below ? -fmaf(A[e], em1[e], A[e]) : 0.f;
    if (REF) {
      l[e] = fmaf(a.beta, kl[e], l[e]);
      g[e] = fmaf(-a.beta, ex[e], g[e]);
      kls += kl[e];
    }
    if (W == W_TOKEN) rs += em1[e];
    if (W != W_NONE) {
      sums.low += some && s.below;
      sums.high += some && s.above;
    }
  }
}

// Sequences of more than kChunk / 2 tokens, by their pieces: a CTA takes a run of these, so
// that what a sequence shares is mostly known from the piece before.
template <int W, bool REF>
__device__ __forceinline__ void long_rows(const PolicyArgs& a, int cta, int ctas, float same, Sums& sums) {
  const int64_t c0 = a.chunks * cta / ctas, c1 = a.chunks * (cta + 1) / ctas;
  const int lane = threadIdx.x & 31;
  int64_t row = -1;
  Row r = {same, 0.f, 0.f, 0.f, 0.f};
  for (int64_t ch = c0; ch < c1; ++ch) {
    const Chunk k = chunk_of(a, ch);
    const int here = a.seg_count[ch];
    if (k.row0 != row) {
      row = k.row0;
      if (a.reduce == 0 || W == W_SEQUENCE) {
        int n = 0;
        double w = 0.0;
        for (int64_t i = lane; i < a.pieces; i += 32) {
          n += a.seg_count[row * a.pieces + i];
          if (W == W_SEQUENCE) w += a.seg_w[row * a.pieces + i];
        }
        n = __reduce_add_sync(0xffffffffu, n);
        if (a.reduce == 0) r.c = 1.f / (static_cast<float>(a.B) * static_cast<float>(n));
        if (W == W_SEQUENCE && n > 0) {
          const double mean = warp_sum(w) / n;
          r.w = static_cast<float>(mean);
          r.lo = static_cast<float>(mean - static_cast<double>(r.w));
          r.em1 = static_cast<float>(expm1(mean));
        }
      }
      if (!a.token_adv) r.A = a.adv[row];
    }
    float* const d = a.dlogp ? a.dlogp + row * a.ld_dlogp + k.t0 : nullptr;
    if (here == 0) {  // nothing but the gradient's zeros
      if (d)
        for (int i = threadIdx.x; i < k.len; i += kThreads) d[i] = 0.f;
      continue;
    }
    if (threadIdx.x == 0) {
      sums.valid += here;
      if (!a.token_adv) sums.base -= static_cast<double>(r.c) * here * static_cast<double>(r.A);
      if (W == W_SEQUENCE) sums.ratio.add_product(r.em1, static_cast<float>(here));
    }
    const uint8_t* m = a.mask + row * a.ld_mask + k.t0;
    const float* q_in = a.logp + row * a.ld_logp + k.t0;
    const float* o_in = W == W_TOKEN ? a.old + row * a.ld_old + k.t0 : nullptr;
    const float* p_in = REF ? a.ref + row * a.ld_ref + k.t0 : nullptr;
    const float* A_in = a.token_adv ? a.adv + row * a.ld_adv + k.t0 : nullptr;
    float q[kTokens], o[kTokens], p[kTokens], A[kTokens];
    bool valid[kTokens];
#pragma unroll
    for (int j = 0; j < kTokens; ++j) {
      const int i = j * kThreads + threadIdx.x;
      valid[j] = i < k.len && m[i] != 0;
      q[j] = o[j] = p[j] = A[j] = 0.f;
      if (i < k.len) {
        q[j] = q_in[i];
        if (W == W_TOKEN) o[j] = o_in[i];
        if (REF) p[j] = p_in[i];
        if (a.token_adv) A[j] = A_in[i];
      }
    }
    float loss = 0.f, kls = 0.f, rs = 0.f;
#pragma unroll
    for (int j = 0; j < kTokens; j += 2) {
      float qq[2], oo[2], pp[2], AA[2], g[2], l[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        qq[e] = valid[j + e] ? q[j + e] : 0.f;
        oo[e] = W == W_TOKEN && valid[j + e] ? o[j + e] : 0.f;
        pp[e] = REF && valid[j + e] ? p[j + e] : 0.f;
        AA[e] = !valid[j + e] ? 0.f : a.token_adv ? A[j + e] : r.A;
      }
      two_tokens<W, REF>(a, r, r, qq, oo, pp, AA, g, l, kls, rs, sums);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        loss += l[e];
        if (a.token_adv) sums.loss.add_product(-AA[e], r.c);
        const int i = (j + e) * kThreads + threadIdx.x;
        if (d && i < k.len) d[i] = r.c * g[e];
      }
    }
    sums.loss.add_product(loss, r.c);
    if (REF) sums.kl.add(kls);
    if (W == W_TOKEN) sums.ratio.add(rs);
  }
}

// Shorter sequences, several whole ones a chunk; what they share stands in shared memory.
template <int W, bool REF>
__device__ __forceinline__ void short_rows(const PolicyArgs& a, int cta, int ctas, float same, Sums& sums) {
  __shared__ Row s_row[kChunk];
  const int len = static_cast<int>(a.T);
  const uint32_t inverse = len > 1 ? static_cast<uint32_t>(0x100000000ull / len) + 1 : 0;  // i / len = i inverse / 2^32 for i < 2^16
  for (int64_t ch = cta; ch < a.chunks; ch += ctas) {
    const Chunk k = chunk_of(a, ch);
    __syncthreads();  // the last chunk's rows have been read
    for (int i = threadIdx.x; i < k.rows; i += kThreads) {
      const int n = a.seg_count[k.row0 + i];
      if (n == 0) continue;
      Row r = {same, 0.f, 0.f, 0.f, 0.f};
      if (a.reduce == 0) r.c = 1.f / (static_cast<float>(a.B) * static_cast<float>(n));
      if (W == W_SEQUENCE) {
        const double mean = a.seg_w[k.row0 + i] / n;
        r.w = static_cast<float>(mean);
        r.lo = static_cast<float>(mean - static_cast<double>(r.w));
        r.em1 = static_cast<float>(expm1(mean));
        sums.ratio.add_product(r.em1, static_cast<float>(n));
      }
      if (!a.token_adv) {
        r.A = a.adv[k.row0 + i];
        sums.loss.add_product(-r.A * static_cast<float>(n), r.c);
      }
      sums.valid += n;
      s_row[i] = r;
    }
    __syncthreads();
    const int all = k.rows * len;
    float q[kTokens], o[kTokens], p[kTokens], A[kTokens];
    bool valid[kTokens];
    int of[kTokens], at[kTokens];
#pragma unroll
    for (int j = 0; j < kTokens; ++j) {
      const int i = j * kThreads + threadIdx.x;
      of[j] = len > 1 ? static_cast<int>(__umulhi(static_cast<uint32_t>(i), inverse)) : i;
      at[j] = i - of[j] * len;
      valid[j] = false;
      q[j] = o[j] = p[j] = A[j] = 0.f;
      if (i < all) {
        const int64_t row = k.row0 + of[j];
        valid[j] = a.mask[row * a.ld_mask + at[j]] != 0;
        q[j] = a.logp[row * a.ld_logp + at[j]];
        if (W == W_TOKEN) o[j] = a.old[row * a.ld_old + at[j]];
        if (REF) p[j] = a.ref[row * a.ld_ref + at[j]];
        if (a.token_adv) A[j] = a.adv[row * a.ld_adv + at[j]];
      }
    }
    float kls = 0.f, rs = 0.f;
#pragma unroll
    for (int j = 0; j < kTokens; j += 2) {
      float qq[2], oo[2], pp[2], AA[2], g[2], l[2];
      Row r[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        r[e] = {0.f, 0.f, 0.f, 0.f, 0.f};
        if (valid[j + e]) r[e] = s_row[of[j + e]];
        qq[e] = valid[j + e] ? q[j + e] : 0.f;
        oo[e] = W == W_TOKEN && valid[j + e] ? o[j + e] : 0.f;
        pp[e] = REF && valid[j + e] ? p[j + e] : 0.f;
        AA[e] = !valid[j + e] ? 0.f : a.token_adv ? A[j + e] : r[e].A;
      }
      two_tokens<W, REF>(a, r[0], r[1], qq, oo, pp, AA, g, l, kls, rs, sums);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        sums.loss.add_product(l[e], r[e].c);
        if (a.token_adv) sums.loss.add_product(-AA[e], r[e].c);
        if (a.dlogp && (j + e) * kThreads + static_cast<int>(threadIdx.x) < all)
          a.dlogp[(k.row0 + of[j + e]) * a.ld_dlogp + at[j + e]] = r[e].c * g[e];
      }
    }
    if (REF) sums.kl.add(kls);
    if (W == W_TOKEN) sums.ratio.add(rs);
  }
}

template <int W, bool REF>
__device__ void loss_phase(const PolicyArgs& a, int cta, int ctas, double (&out)[S_ALL]) {
  __shared__ float s_same;
  float same = a.inv_divisor;  // (unused with a weight for each sequence)
  if (a.reduce == 1) {
    double v[1] = {0.0};
    for (int i = threadIdx.x; i < a.count_ctas; i += kThreads) v[0] += static_cast<double>(a.cta_count[i]);
    cta_sums(v);
    if (threadIdx.x == 0) s_same = static_cast<float>(1.0 / v[0]);
    __syncthreads();
    same = s_same;
  }
  Sums sums;
  if (a.rows_per_chunk == 1) long_rows<W, REF>(a, cta, ctas, same, sums);
  else short_rows<W, REF>(a, cta, ctas, same, sums);
  // (a sum that is not finite has no second part)
  auto value = [](const Sum2& s) { return isfinite(s.hi) ? s.value() : static_cast<double>(s.hi); };
  out[S_LOSS] = value(sums.loss) + sums.base;
  out[S_KL] = value(sums.kl);
  out[S_RATIO] = value(sums.ratio);
  out[S_LOW] = sums.low;
  out[S_HIGH] = sums.high;
  out[S_VALID] = static_cast<double>(sums.valid);
  cta_sums(out);
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
__global__ void __launch_bounds__(kThreads, kLossCtas) k_policy_loss(PolicyArgs a) {
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
  a.loss_ctas = static_cast<int>(a.chunks < kLossCtas * sms ? a.chunks : kLossCtas * sms);
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
