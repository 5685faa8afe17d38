// Clipped policy loss with a KL term, and its gradient by every token's log-probability:
//   w = logp - old (or its mean over the sequence), r = e^w,  x = ref - logp
//   l = -A min(r, 1 + hi) for A > 0,  -A max(min(r, dual), 1 - lo) for A < 0
//   loss = sum c (l + beta (e^x - 1 - x)),  dlogp = c (-A r [not clipped] - beta (e^x - 1))
// (with the mean's ratio and an advantage for each token, dlogp is the gradient where token t
// has the ratio r times its own probability over itself held constant)
// The weight c of a token needs the number of valid tokens (of its sequence, or of all),
// so that the mask is read first: a launch that counts, and one that does the rest; for few
// tokens one cluster of CTAs does both, with a barrier between.
// Many tokens (17 bytes each with a KL term) are bound by the instructions and by latency at the
// 16 warps an SM holds beside the bytes: 256 x 32768 tokens 39 us for both launches in a graph,
// 3.6 TB/s (one token a thread at a time with float64 sums 207 us).
#include <cooperative_groups.h>

#include <atomic>

#include "f32x2.cuh"
#include "internal.h"

namespace cg = cooperative_groups;

namespace grpo {

namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kTokens = 8;               // of a thread at a time: their loads are in flight together
constexpr int kPiece = 2048;             // tokens of a sequence that are counted together
constexpr int kUnit = 32 * kTokens;      // tokens that a warp takes at a time
constexpr int kChunk = kThreads * kTokens;  // of short sequences, that a CTA takes at a time
constexpr int kShort = 128;              // sequences below this are taken several a CTA
// CTAs of an SM, at a time: the next unit's operands are registers (256 x 32768 tokens: two
// 46 us with the count, three 71; without the next unit ahead three 52, four 58).
constexpr int kLossCtas = 2;
constexpr int kCluster = 16;
// Tokens that one cluster takes: at 8 x 20480 its 16 SMs take 16.7 us where two launches over
// all take 13.3, but those cost the host a launch and a workspace more: a call 23.7 us for 28.3.
// (The limit is by that size alone; a call that is captured pays the difference.)
constexpr int64_t kSmall = 96 * kChunk;

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
  // (a sum that is not finite has no second part)
  __device__ __forceinline__ double value() const {
    return isfinite(hi) ? static_cast<double>(hi) + static_cast<double>(lo) : static_cast<double>(hi);
  }
};

// e^x - 1 and e^x - 1 - x of two numbers: x = n ln 2 + f with |f| <= ln 2 / 2 (Cody and
// Waite's reduction, ln 2 in two floats), e^f - 1 - f by its series f^2 (1/2 + f/6 + ... +
// f^6/8!), whose next term is below 2^-28 of it, and e^x - 1 = 2^n (e^f - 1) + 2^n - 1. Both
// keep their digits near 0, where e^x less 1 and less x would not. For |x| < 80, or NaN.
constexpr float kFar = 80.f;
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
}

__device__ __forceinline__ double warp_sum(double v) {
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
// Sums of a CTA in a fixed order, returned to its first thread.
template <int M>
__device__ void cta_sums(double (&v)[M]) {
  __shared__ double part[M][kWarps];
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
      v[m] = lane < kWarps ? part[m][lane] : 0.0;
#pragma unroll
      for (int o = kWarps / 2; o >= 1; o >>= 1) v[m] += __shfl_xor_sync(0xffffffffu, v[m], o);
    }
  }
}
// A sum of whole numbers, returned to every thread.
__device__ __forceinline__ int64_t cta_total(int64_t v) {
  __shared__ int64_t part[kWarps];
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
  __syncthreads();
  v = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) v += part[w];
  return v;
}

// A thread's sums.
struct Sums {
  Sum2 loss, kl, ratio;  // ratio: of r - 1
  int low = 0, high = 0;
  int64_t valid = 0;
};
// A warp's, in the order of the lanes' distances (in two floats: the float64 unit takes 16
// cycles for a warp's addition).
__device__ __forceinline__ double warp_total(Sum2 s) {
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) {
    const float hi = __shfl_xor_sync(0xffffffffu, s.hi, o), lo = __shfl_xor_sync(0xffffffffu, s.lo, o);
    s.add(hi);
    s.lo += lo;
  }
  return s.value();
}
// A CTA's, in the order of the warps; returned to its first thread.
__device__ __forceinline__ void cta_total(const Sums& sums, double (&out)[6]) {
  __shared__ double part[6][kWarps];
  const int warp = threadIdx.x >> 5;
  const double v[3] = {warp_total(sums.loss), warp_total(sums.kl), warp_total(sums.ratio)};
  const int low = __reduce_add_sync(0xffffffffu, sums.low), high = __reduce_add_sync(0xffffffffu, sums.high);
  const unsigned v0 = __reduce_add_sync(0xffffffffu, static_cast<unsigned>(sums.valid & 0xFFFFFF));
  const unsigned v1 = __reduce_add_sync(0xffffffffu, static_cast<unsigned>(sums.valid >> 24));
  if ((threadIdx.x & 31) == 0) {
#pragma unroll
    for (int m = 0; m < 3; ++m) part[m][warp] = v[m];
    part[3][warp] = low;
    part[4][warp] = high;
    part[5][warp] = static_cast<double>(v0) + 16777216.0 * static_cast<double>(v1);
  }
  __syncthreads();
  if (threadIdx.x < 6) {  // a thread a sum
    double t = 0.0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) t += part[threadIdx.x][w];
    part[threadIdx.x][0] = t;
  }
  __syncthreads();
#pragma unroll
  for (int m = 0; m < 6; ++m) out[m] = part[m][0];
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

// A sequence's tokens are cut at every kPiece and kUnit of them from `-shift` on: with VEC
// where quads of four tokens are on 16-byte boundaries, in every operand alike.
template <bool VEC>
__device__ __forceinline__ int shift_of(const PolicyArgs& a, int64_t row) {
  return VEC ? static_cast<int>(row * a.ld_logp & 3) : 0;
}
// Eight tokens of a lane, of the 256 from t0 on, of a sequence of T: two quads, or with
// VEC = false every 32nd.
template <bool VEC>
__device__ __forceinline__ int token_at(int t0, int j) {
  const int lane = threadIdx.x & 31;
  return VEC ? t0 + 128 * (j / 4) + 4 * lane + j % 4 : t0 + 32 * j + lane;
}
// Their values, in pairs; 0 beside the sequence.
struct Eight {
  uint64_t v[kTokens / 2];
  __device__ __forceinline__ float get(int j) const { return j % 2 ? of_pair(v[j / 2]).y : of_pair(v[j / 2]).x; }
};
template <bool VEC>
__device__ __forceinline__ void load_tokens(const float* p, int t0, int T, Eight& e) {
  if (VEC && t0 >= 0 && t0 + kUnit <= T) {
    const ulonglong2* q = reinterpret_cast<const ulonglong2*>(p + token_at<VEC>(t0, 0));
    const ulonglong2 a = q[0], b = q[32];
    e.v[0] = a.x, e.v[1] = a.y, e.v[2] = b.x, e.v[3] = b.y;
  } else {
    float v[kTokens];
#pragma unroll
    for (int j = 0; j < kTokens; ++j) {
      const int i = token_at<VEC>(t0, j);
      v[j] = i >= 0 && i < T ? p[i] : 0.f;
    }
#pragma unroll
    for (int j = 0; j < kTokens / 2; ++j) e.v[j] = pair_of(v[2 * j], v[2 * j + 1]);
  }
}
// The mask of the same tokens, a byte each.
struct Mask {
  uint32_t w[2];
  __device__ __forceinline__ bool operator[](int j) const { return (w[j / 4] & 0xFFu << 8 * (j % 4)) != 0; }
};
template <bool VEC>
__device__ __forceinline__ Mask load_mask(const uint8_t* p, int t0, int T) {
  Mask m;
  if (VEC && t0 >= 0 && t0 + kUnit <= T) {
    const uint32_t* q = reinterpret_cast<const uint32_t*>(p + token_at<VEC>(t0, 0));
    m.w[0] = q[0], m.w[1] = q[32];
  } else {
    m.w[0] = m.w[1] = 0;
#pragma unroll
    for (int j = 0; j < kTokens; ++j) {
      const int i = token_at<VEC>(t0, j);
      if (i >= 0 && i < T) m.w[j / 4] |= static_cast<uint32_t>(p[i]) << 8 * (j % 4);
    }
  }
  return m;
}

// Where the counts are: in the workspace, or in the shared memory of every CTA of a cluster.
struct Counts {
  int* n;         // of every piece
  double* w;      // sums of w
  int64_t* cta;   // totals of the CTAs that counted
};
constexpr int kSmallPieces = 1024;  // that shared memory holds

// Valid tokens of every piece of a sequence, and with a sequence's ratio the sum of w of
// these: a warp a piece. Sequences of few tokens: a thread each. put(pointer, i, value)
// writes a count.
template <bool VEC, bool WTOO, typename Put>
__device__ void count_phase(const PolicyArgs& a, const Counts& to_counts, int cta, int ctas, Put put) {
  const int lane = threadIdx.x & 31;
  const bool thin = a.T < 16;
  const int64_t pieces = a.B * a.pieces, step = static_cast<int64_t>(ctas) * (thin ? kThreads : kWarps);
  int64_t total = 0;
  for (int64_t i = static_cast<int64_t>(cta) * (thin ? kThreads : kWarps) + (thin ? threadIdx.x : threadIdx.x >> 5); i < pieces; i += step) {
    const int64_t row = a.pieces == 1 ? i : i / a.pieces;
    const int T = static_cast<int>(a.T), from = static_cast<int>(i - row * a.pieces) * kPiece - shift_of<VEC>(a, row);
    const int to = from + kPiece < T && a.pieces > 1 ? from + kPiece : T, t0 = from > 0 ? from : 0;
    const uint8_t* m = a.mask + row * a.ld_mask;
    const float *q = a.logp + row * a.ld_logp, *o = a.old + row * a.ld_old;
    int n = 0;
    double sum = 0.0;
    if (thin) {
      Sum2 w;
      for (int64_t t = 0; t < a.T; ++t) {
        const bool valid = m[t] != 0;
        n += valid;
        if (WTOO && valid) {
          const float s = __fsub_rn(q[t], o[t]);
          w.add(s);
          w.lo += diff_error(q[t], o[t], s);
        }
      }
      sum = w.value();
    } else if (WTOO) {
      Sum2 w;
#pragma unroll 2
      for (int u = from; u < to; u += kUnit) {
        Eight qs, os;
        const Mask valid = load_mask<VEC>(m, u, to);
        load_tokens<VEC>(q, u, to, qs);
        load_tokens<VEC>(o, u, to, os);
        n += nonzero_bytes(valid.w[0]) + nonzero_bytes(valid.w[1]);
#pragma unroll
        for (int j = 0; j < kTokens; ++j) {
          const float x = valid[j] ? qs.get(j) : 0.f, y = valid[j] ? os.get(j) : 0.f, s = __fsub_rn(x, y);
          w.add(s);
          w.lo += diff_error(x, y, s);
        }
      }
      sum = __shfl_sync(0xffffffffu, warp_total(w), 0);
    } else {
      n = count_bytes(m + t0, to - t0, lane);
    }
    if (!thin) n = __reduce_add_sync(0xffffffffu, n);
    put(to_counts.n, i, n, thin);
    if (WTOO) put(to_counts.w, i, sum, thin);
    if (thin || lane == 0) total += n;
  }
  if (a.reduce != 1) return;
  total = cta_total(total);
  if (threadIdx.x < 32) put(to_counts.cta, cta, total, false);
}

// --------------------------------------------------------------- the loss
enum : int { S_LOSS, S_KL, S_RATIO, S_LOW, S_HIGH, S_VALID, S_ALL };
enum : int { W_NONE, W_TOKEN, W_SEQUENCE };

// What holds the ratio of tokens of one advantage A: 1 + clip_high, or dual_clip for A < 0,
// from above, and 1 - clip_low from below for A < 0. w rounds a difference (lo: what it
// lost) and a bound's log is held in two floats: where the first are equal the second decide.
struct Bounds {
  float top, bottom, e_top;  // logs; the ratio less 1
};
__device__ __forceinline__ Bounds bounds_of(const PolicyArgs& a, float A) {
  const bool neg = A < 0.f;
  return {neg ? a.far_hi : a.up_hi, neg ? a.down_hi : -INFINITY, neg ? a.e_far : a.e_up};
}
__device__ __forceinline__ void sides_of(const PolicyArgs& a, float A, const Bounds& b, float w, float lo, bool& above, bool& below) {
  above = w > b.top || (w == b.top && lo > (A < 0.f ? a.far_lo : a.up_lo));
  below = w < b.bottom || (w == b.bottom && A < 0.f && lo < a.down_lo);
}

// What a sequence's tokens share: the weight c, the advantage A and the ratio where they are
// one for all (e^w - 1, and whether it is held).
struct Row {
  float c, A, em1;
  int held;  // 1 from above, 2 from below
};
// From the sums over its pieces. Its terms of the sums that every token shares are added by
// the caller that takes its `here` tokens.
template <int W, bool TADV>
__device__ __forceinline__ Row row_of(const PolicyArgs& a, float same, int64_t row, int n, double w) {
  Row r = {same, 0.f, 0.f, 0};
  if (a.reduce == 0) r.c = 1.f / (static_cast<float>(a.B) * static_cast<float>(n));
  if (!TADV) r.A = a.adv[row];
  if (W == W_SEQUENCE && n > 0) {
    // the mean in two floats, and e^mean - 1 of both (float64's functions would take longer
    // than the sequence's tokens)
    float hi = static_cast<float>(w) / static_cast<float>(n), lo = 0.f;
    if (isfinite(hi)) {
      const float rest = static_cast<float>(fma(-static_cast<double>(hi), static_cast<double>(n), w)) / static_cast<float>(n);
      lo = rest - ((hi + rest) - hi);
      hi += rest;
    }
    r.em1 = expm1f(hi);
    if (isfinite(r.em1)) r.em1 = fmaf(r.em1 + 1.f, lo, r.em1);
    if (!TADV) {
      bool above, below;
      sides_of(a, r.A, bounds_of(a, r.A), hi, lo, above, below);
      r.held = above ? 1 : below ? 2 : 0;
    } else {  // by the sign of the token's: bits 0 and 1 for A > 0, 2 and 3 for A < 0
      bool above, below;
      sides_of(a, 1.f, bounds_of(a, 1.f), hi, lo, above, below);
      r.held = above ? 1 : 0;
      sides_of(a, -1.f, bounds_of(a, -1.f), hi, lo, above, below);
      r.held |= above ? 4 : below ? 8 : 0;
    }
  }
  return r;
}
template <int W, bool TADV>
__device__ __forceinline__ void add_row(const PolicyArgs& a, const Row& r, int here, Sums& sums) {
  sums.valid += here;
  const float n = static_cast<float>(here);
  if (W == W_SEQUENCE) sums.ratio.add_product(r.em1, n);
  if (!TADV && r.A != 0.f) {
    const float cA = r.c * r.A;
    sums.loss.add_product(-cA, n);
    if (W == W_SEQUENCE) {
      sums.loss.add_product(-cA * (r.held == 0 ? r.em1 : r.held == 1 ? bounds_of(a, r.A).e_top : a.e_down), n);
      sums.high += r.held == 1 ? here : 0;
      sums.low += r.held == 2 ? here : 0;
    }
  }
}

// Where a sequence's tokens are.
struct Rows {
  const uint8_t* mask;
  const float *q, *o, *p, *A;
  float* d;
};
template <int W, bool REF, bool TADV>
__device__ __forceinline__ Rows rows_of(const PolicyArgs& a, int64_t row, int64_t t0) {
  return {a.mask + row * a.ld_mask + t0,
          a.logp + row * a.ld_logp + t0,
          W == W_TOKEN ? a.old + row * a.ld_old + t0 : nullptr,
          REF ? a.ref + row * a.ld_ref + t0 : nullptr,
          TADV ? a.adv + row * a.ld_adv + t0 : nullptr,
          a.dlogp ? a.dlogp + row * a.ld_dlogp + t0 : nullptr};
}

// One token's terms.
struct Term {
  float d, held, kl, em1;  // the gradient; the ratio less 1, held (0 for A = 0) and not
  bool above, below;
};
// A token whose numbers are too large for the series, infinite, or on a bound.
template <int W, bool REF>
__device__ __noinline__ Term far_token(const PolicyArgs& a, Row r, float A, float q, float o, float p) {
  Term t = {0.f, 0.f, 0.f, r.em1, false, false};
  if (W == W_TOKEN) {
    const float w = __fsub_rn(q, o);
    t.em1 = expm1f(w);
    if (A != 0.f) {
      const Bounds b = bounds_of(a, A);
      sides_of(a, A, b, w, diff_error(q, o, w), t.above, t.below);
      t.held = t.above ? b.e_top : t.below ? a.e_down : t.em1;
    }
  } else if (W == W_SEQUENCE) {
    t.held = A != 0.f ? t.em1 : 0.f;  // (the caller holds it)
  }
  const float cA = r.c * A;
  t.d = A != 0.f && !t.above && !t.below ? -fmaf(cA, t.em1, cA) : 0.f;
  if (REF) {
    const float x = p - q, e = expm1f(x);
    t.kl = e - x;
    t.d = fmaf(-r.c * a.beta, e, t.d);
  }
  return t;
}

// Units of a sequence's tokens.
__host__ __device__ __forceinline__ int64_t units_of(const PolicyArgs& a, bool vec) { return (a.T + (vec ? 3 : 0) + kUnit - 1) / kUnit; }

// The tokens of a thread, of a sequence each (row_for(j)). `at(j, i)`: where the sequence's
// are, and which of them token j is; `in(j)`: whether it is one.
template <int W, bool REF, bool TADV, typename In, typename At, typename RowOf>
__device__ __forceinline__ void tokens(const PolicyArgs& a, In in, At at, RowOf row_for, Sums& sums) {
  constexpr bool LOGP = W == W_TOKEN || REF;
  bool valid[kTokens];
  float w[kTokens], x[kTokens], A[kTokens];
  {
    float q[kTokens], o[kTokens], p[kTokens];
#pragma unroll
    for (int j = 0; j < kTokens; ++j) {
      valid[j] = false;
      q[j] = o[j] = p[j] = A[j] = 0.f;
      if (in(j)) {
        int i;
        const Rows g = at(j, i);
        valid[j] = g.mask[i] != 0;
        if (LOGP) q[j] = g.q[i];
        if (W == W_TOKEN) o[j] = g.o[i];
        if (REF) p[j] = g.p[i];
        if (TADV) A[j] = g.A[i];
      }
    }
#pragma unroll
    for (int j = 0; j < kTokens; ++j) {
      w[j] = W == W_TOKEN && valid[j] ? __fsub_rn(q[j], o[j]) : 0.f;
      x[j] = REF && valid[j] ? p[j] - q[j] : 0.f;
    }
  }
  // numbers that the series does not take, and differences on a bound
  float most = 0.f;
  bool far = false;
#pragma unroll
  for (int j = 0; j < kTokens; ++j) {
    most = fmaxf(most, fmaxf(fabsf(w[j]), fabsf(x[j])));
    if (W == W_TOKEN) far |= w[j] == a.up_hi || w[j] == a.down_hi || w[j] == a.far_hi;
  }
  far |= most >= kFar;
  float kls = 0.f, rs = 0.f;
#pragma unroll
  for (int j = 0; j < kTokens; j += 2) {
    float em1[2] = {0.f, 0.f}, ex[2], kl[2] = {0.f, 0.f}, none[2];
    if (W == W_TOKEN) exponentials<false>(w[j], w[j + 1], em1, none);
    if (REF) exponentials<true>(x[j], x[j + 1], ex, kl);
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const Row r = row_for(j + e);
      const float Ae = TADV ? A[j + e] : r.A;
      if (W == W_SEQUENCE) em1[e] = r.em1;
      Term t = {0.f, em1[e], kl[e], em1[e], false, false};
      const float cA = r.c * Ae;
      if (far && valid[j + e]) {
        int i;
        const Rows g = at(j + e, i);
        t = far_token<W, REF>(a, r, Ae, LOGP ? g.q[i] : 0.f, W == W_TOKEN ? g.o[i] : 0.f, REF ? g.p[i] : 0.f);
      } else {
        if (W == W_TOKEN) {
          const Bounds b = bounds_of(a, Ae);
          t.above = w[j + e] > b.top;
          t.below = w[j + e] < b.bottom;
          t.held = t.above ? b.e_top : t.below ? a.e_down : em1[e];
        }
        t.d = t.above || t.below ? 0.f : -fmaf(cA, em1[e], cA);
        if (Ae == 0.f) t.d = t.held = 0.f, t.above = t.below = false;
        if (REF) t.d = fmaf(-r.c * a.beta, ex[e], t.d);
      }
      if (W == W_SEQUENCE) {  // the ratio's side is known
        const int side = !TADV ? r.held : Ae > 0.f ? r.held & 3 : Ae < 0.f ? r.held >> 2 : 0;
        if (side) {
          t.d = REF ? -r.c * a.beta * (far ? expm1f(x[j + e]) : ex[e]) : 0.f;
          t.held = Ae == 0.f ? 0.f : side == 1 ? bounds_of(a, Ae).e_top : a.e_down;
          t.above = side == 1 && Ae != 0.f;
          t.below = side == 2 && Ae != 0.f;
        }
      }
      if (!valid[j + e]) t.d = 0.f;
      if (REF) kls += t.kl;
      if (W == W_TOKEN) rs += t.em1;
      // the loss: c (-A (1 + held) + beta kl); of one advantage for all, -c A n is the row's
      if (TADV) {
        if (valid[j + e] && Ae != 0.f) {
          sums.loss.add_product(-Ae, r.c);
          sums.loss.add_product(-Ae * t.held, r.c);
        }
      } else if (W == W_TOKEN) {
        sums.loss.add_product(t.held, -cA);
      }
      if (REF) sums.loss.add_product(t.kl, r.c * a.beta);
      if (W == W_TOKEN || (W == W_SEQUENCE && TADV)) {
        sums.low += valid[j + e] && t.below;
        sums.high += valid[j + e] && t.above;
      }
      if (a.dlogp && in(j + e)) {
        int i;
        const Rows g = at(j + e, i);
        g.d[i] = t.d;
      }
    }
  }
  if (REF) sums.kl.add(kls);
  if (W == W_TOKEN) sums.ratio.add(rs);
}

// Sums of a thread's tokens of one sequence, over its weight, for up to a piece of it (9
// units: 36 additions each, so that float32 loses 36 half steps of them at most).
struct RowSums {
  // pairs: of the held ratios less 1 (with an advantage for each token, times c A), of k, of r - 1
  uint64_t held, kl, ratio;
  __device__ __forceinline__ void clear() { held = kl = ratio = pair_of(0.f); }
};
template <int W, bool REF, bool TADV>
__device__ __forceinline__ void fold(const PolicyArgs& a, const Row& r, RowSums& s, Sums& sums) {
  const float2 h = of_pair(s.held);
  if (TADV) sums.loss.add(-(h.x + h.y));
  else if (W == W_TOKEN && r.A != 0.f) sums.loss.add_product(h.x + h.y, -r.c * r.A);
  if (REF) {
    const float2 k = of_pair(s.kl);
    sums.loss.add_product(k.x + k.y, r.c * a.beta);
    sums.kl.add(k.x + k.y);
  }
  if (W == W_TOKEN) {
    const float2 x = of_pair(s.ratio);
    sums.ratio.add(x.x + x.y);
  }
  s.clear();
}

// Eight tokens of a lane, of one sequence, of which some are too far for the series or on a
// bound: one by one. Their sums are returned, and the gradients written.
struct FarSums {
  float held, kl, ratio;
  Sum2 loss;  // with an advantage for each token
  int low, high;
};
template <bool VEC, int W, bool REF, bool TADV>
__device__ __noinline__ FarSums far_tokens(const PolicyArgs& a, Row r, Rows g, int t0, Mask valid) {
  FarSums s = {0.f, 0.f, 0.f, Sum2(), 0, 0};
#pragma unroll 1
  for (int j = 0; j < kTokens; ++j) {
    const int t = token_at<VEC>(t0, j);
    if (t < 0 || t >= a.T) continue;
    Term x = {0.f, 0.f, 0.f, 0.f, false, false};
    if (valid[j]) {
      const float A = TADV ? g.A[t] : r.A, q = W == W_TOKEN || REF ? g.q[t] : 0.f, p = REF ? g.p[t] : 0.f;
      x = far_token<W, REF>(a, r, A, q, W == W_TOKEN ? g.o[t] : 0.f, p);
      if (W == W_SEQUENCE) {
        const int side = A == 0.f ? 0 : !TADV ? r.held : A > 0.f ? r.held & 3 : r.held >> 2;
        if (side) {
          x.d = REF ? -r.c * a.beta * expm1f(p - q) : 0.f;
          x.held = side == 1 ? bounds_of(a, A).e_top : a.e_down;
          x.above = side == 1;
          x.below = side == 2;
        }
      }
      if (TADV && A != 0.f) {
        s.loss.add_product(-A, r.c);
        s.loss.add_product(-A * x.held, r.c);
      }
    }
    s.held += x.held;
    s.kl += x.kl;
    s.ratio += x.em1;
    s.low += x.below;
    s.high += x.above;
    if (g.d) g.d[t] = x.d;
  }
  return s;
}

// Eight tokens of a lane, all of one sequence.
template <bool VEC, int W, bool REF, bool TADV>
__device__ __forceinline__ void unit_tokens(const PolicyArgs& a, const Row& r, const Bounds& b, const Rows& g, int t0, const Mask& valid, Eight& q,
                                            Eight& o, Eight& p, Eight& A, RowSums& row, Sums& sums) {
  // the differences, of masked tokens 0, in the numbers' place
  const uint64_t minus = pair_of(-1.f);
  float most = 0.f;
  bool far = false;
#pragma unroll
  for (int j = 0; j < kTokens / 2; ++j) {
    if (REF) {
      const float2 x = of_pair(fma2(q.v[j], minus, p.v[j]));
      const float x0 = valid[2 * j] ? x.x : 0.f, x1 = valid[2 * j + 1] ? x.y : 0.f;
      most = fmaxf(most, fmaxf(fabsf(x0), fabsf(x1)));
      p.v[j] = pair_of(x0, x1);
    }
    if (W == W_TOKEN) {
      const float2 w = of_pair(fma2(o.v[j], minus, q.v[j]));
      const float w0 = valid[2 * j] ? w.x : 0.f, w1 = valid[2 * j + 1] ? w.y : 0.f;
      most = fmaxf(most, fmaxf(fabsf(w0), fabsf(w1)));
      if (TADV) far |= w0 == a.up_hi || w0 == a.down_hi || w0 == a.far_hi || w1 == a.up_hi || w1 == a.down_hi || w1 == a.far_hi;
      else far |= w0 == b.top || w0 == b.bottom || w1 == b.top || w1 == b.bottom;
      o.v[j] = pair_of(w0, w1);
    }
    if (TADV) A.v[j] = pair_of(valid[2 * j] ? A.get(2 * j) : 0.f, valid[2 * j + 1] ? A.get(2 * j + 1) : 0.f);
  }
  if (far || most >= kFar) {
    const FarSums s = far_tokens<VEC, W, REF, TADV>(a, r, g, t0, valid);
    if (!TADV) row.held = add2(row.held, pair_of(s.held, 0.f));
    row.kl = add2(row.kl, pair_of(s.kl, 0.f));
    row.ratio = add2(row.ratio, pair_of(s.ratio, 0.f));
    if (TADV) {
      sums.loss.add(s.loss.hi);
      sums.loss.lo += s.loss.lo;
    }
    if (W == W_TOKEN || (W == W_SEQUENCE && TADV)) {
      sums.low += s.low;
      sums.high += s.high;
    }
    return;
  }
  const bool none = r.A == 0.f;  // no advantage, no gradient, whatever the ratio
  const float cb = -r.c * a.beta, cA = none ? 0.f : r.c * r.A;
  float d[kTokens];
#pragma unroll
  for (int j = 0; j < kTokens; j += 2) {
    float em1[2] = {r.em1, r.em1}, ex[2], kl[2], dd[2];
    const float2 w = of_pair(o.v[j / 2]), x = of_pair(p.v[j / 2]);
    if (W == W_TOKEN) {
      float none[2];
      exponentials<false>(w.x, w.y, em1, none);
      row.ratio = add2(row.ratio, pair_of(em1[0], em1[1]));
    }
    if (REF) {
      exponentials<true>(x.x, x.y, ex, kl);
      row.kl = add2(row.kl, pair_of(kl[0], kl[1]));
    }
    if (!TADV) {
      if (W == W_TOKEN) {
        const float2 gr = of_pair(none ? pair_of(0.f) : fma2(pair_of(em1[0], em1[1]), pair_of(-cA), pair_of(-cA)));
        float held[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float we = e ? w.y : w.x;
          const bool above = we > b.top, below = we < b.bottom;
          held[e] = above ? b.e_top : below ? a.e_down : em1[e];
          dd[e] = above || below ? 0.f : e ? gr.y : gr.x;
          if (above) ++sums.high;
          if (below) ++sums.low;
        }
        row.held = add2(row.held, pair_of(held[0], held[1]));
      } else {
        dd[0] = dd[1] = none || (W == W_SEQUENCE && r.held) ? 0.f : -fmaf(cA, r.em1, cA);
      }
    } else {
      float more[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float Aj = A.get(j + e), cAj = r.c * Aj, we = e ? w.y : w.x;
        const Bounds bj = bounds_of(a, Aj);
        bool above = false, below = false;
        if (W == W_TOKEN) {
          above = we > bj.top;
          below = we < bj.bottom;
        } else if (W == W_SEQUENCE) {
          const int side = Aj > 0.f ? r.held & 3 : r.held >> 2;
          above = side == 1;
          below = side == 2;
        }
        const bool some = Aj != 0.f;
        const float held = above ? bj.e_top : below ? a.e_down : em1[e];
        dd[e] = above || below || !some ? 0.f : -fmaf(cAj, em1[e], cAj);
        if (some && above) ++sums.high;
        if (some && below) ++sums.low;
        // c A in full, and of it what the ratio adds
        sums.loss.add_product(-Aj, r.c);
        more[e] = some ? cAj * held : 0.f;
      }
      row.held = add2(row.held, pair_of(more[0], more[1]));
    }
    if (REF) {
      const float2 t = of_pair(fma2(pair_of(ex[0], ex[1]), pair_of(cb), pair_of(dd[0], dd[1])));
      dd[0] = t.x, dd[1] = t.y;
    }
    d[j] = valid[j] ? dd[0] : 0.f;
    d[j + 1] = valid[j + 1] ? dd[1] : 0.f;
  }
  if (!g.d) return;
  if (VEC && t0 >= 0 && t0 + kUnit <= a.T) {
    float4* to = reinterpret_cast<float4*>(g.d + token_at<VEC>(t0, 0));
    to[0] = make_float4(d[0], d[1], d[2], d[3]);
    to[32] = make_float4(d[4], d[5], d[6], d[7]);
  } else {
#pragma unroll
    for (int j = 0; j < kTokens; ++j) {
      const int i = token_at<VEC>(t0, j);
      if (i >= 0 && i < a.T) g.d[i] = d[j];
    }
  }
}

// A warp takes a run of units of its own, so that what a sequence shares is mostly known
// from the unit before, and no warp waits for another.
template <bool VEC, int W, bool REF, bool TADV>
__device__ __forceinline__ void long_rows(const PolicyArgs& a, const Counts& counts, int cta, int ctas, float same, Sums& sums) {
  const int lane = threadIdx.x & 31;
  const int64_t units = units_of(a, VEC), all = a.B * units;  // of a sequence, and of all
  const int64_t warps = static_cast<int64_t>(ctas) * kWarps, warp = static_cast<int64_t>(cta) * kWarps + (threadIdx.x >> 5);
  const int64_t u0 = all / warps * warp + (warp < all % warps ? warp : all % warps), u1 = u0 + all / warps + (warp < all % warps ? 1 : 0);
  if (u0 >= u1) return;
  const int T = static_cast<int>(a.T);
  // Where a unit is, and how many valid tokens its piece has; its operands. The next unit's
  // are on their way while one is worked on, and the count of the one behind it, which says
  // whether there is anything to load.
  struct Place {
    int64_t row;
    int unit;
  };
  struct Raw {
    Eight q, o, p, A;
    Mask valid;
  };
  auto step = [&](Place& x) {
    if (++x.unit == units) x.unit = 0, ++x.row;
  };
  auto count_of = [&](const Place& x) { return counts.n[x.row * a.pieces + (a.pieces > 1 ? x.unit / (kPiece / kUnit) : 0)]; };
  auto first_of = [&](const Place& x) { return x.unit * kUnit - shift_of<VEC>(a, x.row); };
  auto load = [&](const Place& x, int here, Raw& raw) {
    if (here == 0) return;
    const Rows g = rows_of<W, REF, TADV>(a, x.row, 0);
    const int t0 = first_of(x);
    raw.valid = load_mask<VEC>(g.mask, t0, T);
    if (W == W_TOKEN || REF) load_tokens<VEC>(g.q, t0, T, raw.q);
    if (W == W_TOKEN) load_tokens<VEC>(g.o, t0, T, raw.o);
    if (REF) load_tokens<VEC>(g.p, t0, T, raw.p);
    if (TADV) load_tokens<VEC>(g.A, t0, T, raw.A);
  };
  Place at = {u0 / units, 0}, ahead;
  at.unit = static_cast<int>(u0 - at.row * units);
  ahead = at;
  int here = count_of(at), here_next = 0;
  Raw raw, next;
  load(at, here, raw);
  if (u0 + 1 < u1) {
    step(ahead);
    here_next = count_of(ahead);
  }
  Row r = {0.f, 0.f, 0.f, 0};  // (no token yet)
  Bounds b = {INFINITY, -INFINITY, 0.f};
  RowSums row_sums;
  row_sums.clear();
  int64_t known = -1;  // the sequence that r is of
  for (int64_t u = u0; u < u1; ++u) {
    int here_after = 0;
    if (u + 1 < u1) {
      load(ahead, here_next, next);
      step(ahead);
      if (u + 2 < u1) here_after = count_of(ahead);
    }
    const bool begins = (a.pieces > 1 ? at.unit % (kPiece / kUnit) : at.unit) == 0;  // a piece, or a sequence
    if (here > 0 && (begins || at.row != known)) fold<W, REF, TADV>(a, r, row_sums, sums);
    if (here > 0 && at.row != known) {
      known = at.row;
      int n = 0;
      double w = 0.0;
      if (a.reduce == 0 || W == W_SEQUENCE) {
        for (int64_t i = lane; i < a.pieces; i += 32) {
          n += counts.n[known * a.pieces + i];
          if (W == W_SEQUENCE) w += counts.w[known * a.pieces + i];
        }
        n = __reduce_add_sync(0xffffffffu, n);
        if (W == W_SEQUENCE) w = warp_sum(w);
      }
      r = row_of<W, TADV>(a, same, known, n, w);
      b = bounds_of(a, r.A);
      if (r.A == 0.f) b.top = INFINITY;  // (nothing to hold, or to count)
    }
    const Rows g = rows_of<W, REF, TADV>(a, at.row, 0);
    const int t0 = first_of(at);
    if (here > 0) {
      // (what the piece's tokens share is added with its first unit)
      if (lane == 0 && begins) add_row<W, TADV>(a, r, here, sums);
      unit_tokens<VEC, W, REF, TADV>(a, r, b, g, t0, raw.valid, raw.q, raw.o, raw.p, raw.A, row_sums, sums);
    } else if (g.d) {  // nothing but the gradient's zeros
#pragma unroll
      for (int j = 0; j < kTokens; ++j) {
        const int i = token_at<VEC>(t0, j);
        if (i >= 0 && i < T) g.d[i] = 0.f;
      }
    }
    step(at);
    raw = next;
    here = here_next;
    here_next = here_after;
  }
  fold<W, REF, TADV>(a, r, row_sums, sums);
}

// Short sequences, several whole ones a chunk; what they share stands in shared memory.
template <int W, bool REF, bool TADV>
__device__ __forceinline__ void short_rows(const PolicyArgs& a, const Counts& counts, int cta, int ctas, float same, Sums& sums) {
  __shared__ Row s_row[kChunk];
  const int len = static_cast<int>(a.T), per = kChunk / len;
  const uint32_t inverse = len > 1 ? static_cast<uint32_t>(0x100000000ull / len) + 1 : 0;  // i / len = i inverse / 2^32 for i < 2^16
  for (int64_t row0 = static_cast<int64_t>(cta) * per; row0 < a.B; row0 += static_cast<int64_t>(ctas) * per) {
    const int rows = static_cast<int>(a.B - row0 < per ? a.B - row0 : per), all = rows * len;
    __syncthreads();  // the last chunk's rows have been read
    for (int i = threadIdx.x; i < rows; i += kThreads) {
      const int n = counts.n[row0 + i];
      Row r = {0.f, 0.f, 0.f, 0};
      if (n > 0) {
        r = row_of<W, TADV>(a, same, row0 + i, n, W == W_SEQUENCE ? counts.w[row0 + i] : 0.0);
        add_row<W, TADV>(a, r, n, sums);
      }
      s_row[i] = r;
    }
    __syncthreads();
    auto row_in = [&](int j) {
      const uint32_t i = j * kThreads + threadIdx.x;
      return len > 1 ? static_cast<int>(__umulhi(i, inverse)) : static_cast<int>(i);
    };
    auto in = [&](int j) { return j * kThreads + static_cast<int>(threadIdx.x) < all; };
    tokens<W, REF, TADV>(a, in, [&](int j, int& i) {
      const int k = row_in(j);
      i = j * kThreads + threadIdx.x - k * len;
      return rows_of<W, REF, TADV>(a, row0 + k, 0);
    }, [&](int j) { return in(j) ? s_row[row_in(j)] : Row{0.f, 0.f, 0.f, 0}; }, sums);
  }
}

template <bool VEC, int W, bool REF, bool TADV>
__device__ void loss_phase(const PolicyArgs& a, const Counts& counts, int cta, int ctas, double (&out)[S_ALL]) {
  float same = a.inv_divisor;  // (unused with a weight for each sequence)
  if (a.reduce == 1) {
    int64_t n = 0;
    for (int i = threadIdx.x; i < a.count_ctas; i += kThreads) n += counts.cta[i];
    same = 1.f / static_cast<float>(cta_total(n));
  }
  Sums sums;
  if (a.T < kShort) short_rows<W, REF, TADV>(a, counts, cta, ctas, same, sums);
  else long_rows<VEC, W, REF, TADV>(a, counts, cta, ctas, same, sums);
  static_assert(S_ALL == 6 && S_LOSS == 0 && S_KL == 1 && S_RATIO == 2 && S_LOW == 3 && S_HIGH == 4 && S_VALID == 5, "");
  cta_total(sums, out);
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

template <bool VEC, bool WTOO>
__global__ void __launch_bounds__(kThreads) k_policy_count(const __grid_constant__ PolicyArgs a) {
  let_next();
  if (blockIdx.x == 0 && threadIdx.x == 0) *a.ticket = 0;
  const bool first = (threadIdx.x & 31) == 0;
  count_phase<VEC, WTOO>(a, {a.piece_count, a.piece_w, a.cta_count}, blockIdx.x, gridDim.x, [&](auto* p, int64_t i, auto v, bool every) {
    if (every || first) p[i] = v;
  });
}

template <bool VEC, int W, bool REF, bool TADV>
__global__ void __launch_bounds__(kThreads, kLossCtas) k_policy_loss(const __grid_constant__ PolicyArgs a) {
  __shared__ bool s_last;
  after_previous();
  double sums[S_ALL];
  loss_phase<VEC, W, REF, TADV>(a, {a.piece_count, a.piece_w, a.cta_count}, blockIdx.x, gridDim.x, sums);
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

// Both for few tokens: every CTA of the cluster has all counts in its shared memory, and
// no workspace is needed.
template <bool VEC, int W, bool REF, bool TADV>
__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kThreads) k_policy_small(const __grid_constant__ PolicyArgs a) {
  __shared__ double parts[kCluster][S_ALL];
  __shared__ int s_n[kSmallPieces];
  __shared__ double s_w[W == W_SEQUENCE ? kSmallPieces : 1];
  __shared__ int64_t s_cta[kCluster];
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = static_cast<int>(cluster.block_rank()), lane = threadIdx.x & 31;
  const Counts counts = {s_n, s_w, s_cta};
  cluster.sync();  // every CTA runs: its shared memory may be written
  count_phase<VEC, W == W_SEQUENCE>(a, counts, rank, kCluster, [&](auto* p, int64_t i, auto v, bool every) {
    if (every) {
      for (int c = 0; c < kCluster; ++c) cluster.map_shared_rank(p, c)[i] = v;
    } else if (lane < kCluster) {
      cluster.map_shared_rank(p, lane)[i] = v;
    }
  });
  cluster.sync();
  double sums[S_ALL];
  loss_phase<VEC, W, REF, TADV>(a, counts, rank, kCluster, sums);
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

bool small(const PolicyArgs& a) { return a.B * a.T <= kSmall && a.B * a.pieces <= kSmallPieces; }

// Whether quads of tokens of every operand are on 16-byte boundaries alike.
bool by_quads(const PolicyArgs& a) {
  auto fits = [&](const void* p, int64_t ld, int size) {
    return !p || (reinterpret_cast<uintptr_t>(p) % (4 * size) == 0 && (ld - a.ld_logp) % 4 == 0);
  };
  return fits(a.logp, a.ld_logp, 4) && fits(a.old, a.ld_old, 4) && fits(a.ref, a.ld_ref, 4) &&
         fits(a.token_adv ? a.adv : nullptr, a.ld_adv, 4) && fits(a.mask, a.ld_mask, 1) && fits(a.dlogp, a.ld_dlogp, 4);
}

template <bool VEC, int W, bool REF, bool TADV>
cudaError_t loss_launch(const PolicyArgs& a, cudaStream_t s) {
  if (small(a)) {
    auto kernel = k_policy_small<VEC, W, REF, TADV>;
    // clusters of more than 8 are asked for once a device
    static std::atomic<uint64_t> configured{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    const uint64_t bit = 1ull << (dev & 63);
    if (e == cudaSuccess && !(configured.load() & bit)) {
      e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
      if (e == cudaSuccess) configured.fetch_or(bit);
    }
    if (e != cudaSuccess) return e;
    kernel<<<kCluster, kThreads, 0, s>>>(a);
    return cudaGetLastError();
  }
  return launch_after(k_policy_loss<VEC, W, REF, TADV>, dim3(static_cast<unsigned>(a.loss_ctas)), kThreads, 0, s, a);
}
template <bool VEC>
cudaError_t loss_of(const PolicyArgs& a, cudaStream_t s) {
  const int w = !a.old ? W_NONE : a.sequence_ratio ? W_SEQUENCE : W_TOKEN;
  switch (4 * w + (a.ref ? 2 : 0) + (a.token_adv ? 1 : 0)) {
#define POLICY_CASE(W)                                              \
  case 4 * W: return loss_launch<VEC, W, false, false>(a, s);       \
  case 4 * W + 1: return loss_launch<VEC, W, false, true>(a, s);    \
  case 4 * W + 2: return loss_launch<VEC, W, true, false>(a, s);    \
  case 4 * W + 3: return loss_launch<VEC, W, true, true>(a, s);
    POLICY_CASE(W_NONE)
    POLICY_CASE(W_TOKEN)
    POLICY_CASE(W_SEQUENCE)
#undef POLICY_CASE
  }
  return cudaErrorInvalidValue;
}

}  // namespace

// Fills in how the tokens are cut, and the places in the workspace.
size_t policy_plan(PolicyArgs& a, int sms, void* workspace) {
  a.pieces = a.T > kPiece ? (a.T + 3 + kPiece - 1) / kPiece : 1;  // (the first may begin up to 3 tokens early)
  const int64_t pieces = a.B * a.pieces, most = 8ll * sms, all = 1ll * kLossCtas * sms;
  const int64_t chunks = a.T < 1 ? 1 : a.T < kShort ? (a.B + kChunk / a.T - 1) / (kChunk / a.T)
                                                    : (a.B * units_of(a, true) + kWarps - 1) / kWarps;
  const int64_t want = (pieces + kWarps - 1) / kWarps;
  a.loss_ctas = static_cast<int>(chunks < all ? chunks : all);
  a.count_ctas = small(a) ? kCluster : static_cast<int>(want < most ? want : most);
  if (small(a)) return 0;
  size_t at = 0;
  auto take = [&](size_t bytes) {
    char* p = static_cast<char*>(workspace) + at;
    at += (bytes + 255) / 256 * 256;
    return static_cast<void*>(p);
  };
  a.ticket = static_cast<unsigned*>(take(4));
  a.cta_count = static_cast<int64_t*>(take(8 * most));
  a.partial = static_cast<double*>(take(8 * S_ALL * most));
  a.piece_count = static_cast<int*>(take(4 * pieces));
  a.piece_w = static_cast<double*>(take(a.sequence_ratio ? 8 * pieces : 0));
  return at;
}

bool policy_counts_first(const PolicyArgs& a) { return !small(a); }
cudaError_t launch_policy_count(const PolicyArgs& a, cudaStream_t s) {
  if (by_quads(a)) {
    if (a.sequence_ratio) k_policy_count<true, true><<<a.count_ctas, kThreads, 0, s>>>(a);
    else k_policy_count<true, false><<<a.count_ctas, kThreads, 0, s>>>(a);
  } else {
    if (a.sequence_ratio) k_policy_count<false, true><<<a.count_ctas, kThreads, 0, s>>>(a);
    else k_policy_count<false, false><<<a.count_ctas, kThreads, 0, s>>>(a);
  }
  return cudaGetLastError();
}
cudaError_t launch_policy_loss(const PolicyArgs& a, cudaStream_t s) { return by_quads(a) ? loss_of<true>(a, s) : loss_of<false>(a, s); }

}  // namespace grpo
