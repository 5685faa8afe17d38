// Token sampling with temperature, top-k, top-p and min-p from given uniforms.
//
// A row's weights w_i = exp((z_i - zmax) / T) are summed as integers of fixed
// point, W = w 2^B, so that sums do not depend on their order, and the token is
// the one that real numbers give: the draw compares u sum W with the running sum,
// and with 10^5 tokens of similar weight, sums of float32 weights (2^-22 off, or
// so) would pick a neighbour in one draw of ten. All three cut-offs keep a prefix
// of the order (logit descending, index ascending): what is kept is a threshold t
// on the logit's sort key and a number of ties at t, the first in index order.
//
// What bounds a call is not the bytes of a row (31 us of the 135 that 512 mixed rows of
// 201088 take) but the work on each logit, two to ten cycles of an SM for 32 of them and
// a pass, and for few rows the barriers between the questions that a row is asked.
// Three kernels share the parts below:
//
// - k_sample_counts (bf16 rows): the row as counts of its few distinct values, in
//   which every sum is exact and every cut-off is a search; a cluster of CTAs a row.
//   One row of 128256: 15 to 19 us; 64 rows: 24 to 31, but 68 to 780 where the logits
//   are almost equal (a spread of 0.05), whose counts meet in few counters.
// - k_sample (float32 rows, and short ones): two ways of weighing share one body. The
//   fast one takes 2^y from a polynomial and carries a bound E on the error of its
//   sums; where the draw or the top-p cut falls within E of a border, the row is
//   done again with weights from pairs of floats (2^-43), whose integer sums decide.
//   A trained model's rows (a few likely tokens) seldom need that. A cluster takes a
//   row, each CTA one slice of it that it copies into shared memory once, and every
//   question (maximum, sums, histogram, draw) reads that and is joined through
//   distributed shared memory. 8 rows of 128256: 15 us with no cut-off, 33 where a draw
//   falls near a border in one of them, 19 with few candidates; with top-p alone 74 (a
//   spread of 3) to 650 (0.05).
// - k_sample_rows (rows enough for every SM): a CTA a row in little more than a pass, for
//   what a list of a few candidates or the plain softmax decides; the others are left to
//   a second launch of the kernels above. 512 rows of 201088 in bf16: greedy and small
//   top-k 65 to 78 us, all rows left to the second launch (wide top-p) 295 to 321, or 2280
//   of almost equal logits. In float32: 95 and 110; left to the second launch 2150 (a
//   spread of 3) to 20000 (0.05).
#include <cooperative_groups.h>
#include <cuda_bf16.h>

#include <atomic>
#include <type_traits>

#include "f32x2.cuh"
#include "internal.h"
#include "ptx.cuh"

namespace cg = cooperative_groups;

namespace grpo {

namespace {

constexpr int kMaxThreads = 1024;              // of a CTA
constexpr int kMaxWarps = kMaxThreads / 32;
constexpr int kMaxCluster = 8;                 // the portable cluster size
constexpr int kBins = 1280;                    // (five a thread at most) 1/32 of a binary order each, down to 2^-40
constexpr int kCap = 1024;                     // candidates that one CTA sorts
constexpr int kGuess = 96;                      // candidates asked for with top-p alone
constexpr int kCount = 256;                    // and those that it sorts by counting
constexpr int kSliceBytes = 33 * 1024;         // of a row's slice kept in shared memory, with 256 threads
constexpr int kMaxSliceBytes = 192 * 1024;     // and with 512
constexpr int kMaxFast = 500000;              // elements of a slice that the bins' sums can take
constexpr float kCut = -40.f;                  // binary orders below the top that weigh nothing

// 2^(j/32), j = 0..31, each as the sum of two floats (2^x from a table and a short series
// on the remainder: Tang's method).
__constant__ float2 c_exp2_32[32] = {
    {0x1.0000000000000p+0f, 0x0.0p+0f}, {0x1.059b0e0000000p+0f, -0x1.9d4f520000000p-25f},
    {0x1.0b55860000000p+0f, 0x1.9f31220000000p-25f}, {0x1.11301e0000000p+0f, -0x1.fdb4960000000p-25f},
    {0x1.172b840000000p+0f, -0x1.c157420000000p-27f}, {0x1.1d48740000000p+0f, -0x1.d2e8ca0000000p-25f},
    {0x1.2387a60000000p+0f, 0x1.ceac480000000p-25f}, {0x1.29e9e00000000p+0f, -0x1.5c04240000000p-25f},
    {0x1.306fe00000000p+0f, 0x1.4636e20000000p-25f}, {0x1.371a740000000p+0f, -0x1.18aac60000000p-25f},
    {0x1.3dea640000000p+0f, 0x1.8246840000000p-25f}, {0x1.44e0860000000p+0f, 0x1.8624b40000000p-30f},
    {0x1.4bfdae0000000p+0f, -0x1.593abc0000000p-25f}, {0x1.5342b60000000p+0f, -0x1.2c56100000000p-25f},
    {0x1.5ab07e0000000p+0f, -0x1.5bd5ec0000000p-27f}, {0x1.6247ec0000000p+0f, -0x1.f8b5500000000p-25f},
    {0x1.6a09e60000000p+0f, 0x1.9fcef40000000p-26f}, {0x1.71f75e0000000p+0f, 0x1.1d8bee0000000p-25f},
    {0x1.7a11480000000p+0f, -0x1.829fd00000000p-25f}, {0x1.82589a0000000p+0f, -0x1.accc7c0000000p-26f},
    {0x1.8ace540000000p+0f, 0x1.15506e0000000p-27f}, {0x1.93737c0000000p+0f, -0x1.e647440000000p-25f},
    {0x1.9c49180000000p+0f, 0x1.51f8480000000p-27f}, {0x1.a5503c0000000p+0f, -0x1.b83b540000000p-25f},
    {0x1.ae89fa0000000p+0f, -0x1.a94b140000000p-26f}, {0x1.b7f7700000000p+0f, -0x1.a094380000000p-25f},
    {0x1.c199be0000000p+0f, -0x1.3d56b20000000p-27f}, {0x1.cb720e0000000p+0f, -0x1.8837cc0000000p-27f},
    {0x1.d5818e0000000p+0f, -0x1.822dbc0000000p-27f}, {0x1.dfc9740000000p+0f, -0x1.908c940000000p-25f},
    {0x1.ea4afa0000000p+0f, 0x1.52486c0000000p-27f}, {0x1.f507660000000p+0f, -0x1.246eb00000000p-26f},
};


__device__ __forceinline__ float to_f(float v) { return v; }
__device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
// NaN counts as -inf
__device__ __forceinline__ float clean(float z) { return fmaxf(z, -INFINITY); }
// sorts like the float; -0 ties with +0
__device__ __forceinline__ uint32_t key_of(float z) {
  const uint32_t b = __float_as_uint(z + 0.f);
  return b ^ ((b >> 31) ? 0xFFFFFFFFu : 0x80000000u);
}
__device__ __forceinline__ float float_of(uint32_t key) {
  return __uint_as_float(key ^ ((key >> 31) ? 0x80000000u : 0xFFFFFFFFu));
}

// The float z such that a logit is above it if and only if its key is above k.
// (Key 0x7FFFFFFF is that of -0, which no logit has: both zeros are above it.)
__device__ __forceinline__ float above_key(uint32_t k) {
  return k <= 0x007FFFFFu ? -INFINITY : float_of(k == 0x7FFFFFFFu ? 0x7FFFFFFEu : k);
}

// A 16-byte piece of a row.
template <typename T>
struct Vec {
  static constexpr int N = 16 / sizeof(T);
  uint4 raw;
  __device__ __forceinline__ float get(int e) const;
  __device__ __forceinline__ float max() const;  // NaN counts as -inf
  // elements 2 e and 2 e + 1 as they are
  __device__ __forceinline__ uint64_t pair(int e) const;
};
template <>
__device__ __forceinline__ uint64_t Vec<float>::pair(int e) const {
  return e == 0 ? pair_of(raw.x, raw.y) : pair_of(raw.z, raw.w);
}
template <>
__device__ __forceinline__ uint64_t Vec<__nv_bfloat16>::pair(int e) const {
  const uint32_t w = e == 0 ? raw.x : e == 1 ? raw.y : e == 2 ? raw.z : raw.w;
  return pair_of(w << 16, w & 0xFFFF0000u);
}
template <>
__device__ __forceinline__ float Vec<float>::get(int e) const {
  return clean(__uint_as_float(e == 0 ? raw.x : e == 1 ? raw.y : e == 2 ? raw.z : raw.w));
}
template <>
__device__ __forceinline__ float Vec<__nv_bfloat16>::get(int e) const {
  const uint32_t w = e < 2 ? raw.x : e < 4 ? raw.y : e < 6 ? raw.z : raw.w;
  return clean(__uint_as_float((e & 1) ? (w & 0xFFFF0000u) : (w << 16)));
}

template <>
__device__ __forceinline__ float Vec<float>::max() const {
  return fmaxf(fmaxf(get(0), get(1)), fmaxf(get(2), get(3)));
}
template <>
__device__ __forceinline__ float Vec<__nv_bfloat16>::max() const {
  auto h = [](uint32_t w) { return *reinterpret_cast<__nv_bfloat162*>(&w); };
  // of a number and a NaN this maximum is the number
  const __nv_bfloat162 m = __hmax2(__hmax2(h(raw.x), h(raw.y)), __hmax2(h(raw.z), h(raw.w)));
  return fmaxf(clean(__low2float(m)), __high2float(m));
}

// log2(e) and ln(2) as pairs of floats
constexpr float kLog2e = 0x1.715476p+0f, kLog2eLo = 0x1.4ae0cp-26f;
constexpr float kLn2 = 0x1.62e430p-1f, kLn2Lo = -0x1.05c610p-29f;

// 2^(p + pl) = 2^n (h + hl) to about 2^-46, for |pl| far below |p|, -41 < p <= 0
__device__ __forceinline__ void exp2_pair(const float2* tab, float p, float pl, int& n, float& h,
                                          float& hl) {
  // p = k / 32 + r, |r| <= 1/64
  const float kf = rintf(p * 32.f);
  const int k = static_cast<int>(kf);
  const float r0 = __fmaf_rn(kf, -0.03125f, p);
  const float r = __fadd_rn(r0, pl), rl = __fsub_rn(pl, __fsub_rn(r, r0));
  // s = 2^r - 1 = x + x^2/2 + x^3/6 + ..., x = r ln 2, the first two terms in pairs
  const float x = __fmul_rn(r, kLn2);
  const float xl = __fmaf_rn(r, kLn2, -x) + __fmaf_rn(r, kLn2Lo, rl * kLn2);
  const float xx = __fmul_rn(x, x);
  const float xxl = __fmaf_rn(x, x, -xx) + 2.f * x * xl;
  const float cubic = xx * x * __fmaf_rn(x, __fmaf_rn(x, __fmaf_rn(x, 1.f / 720.f, 1.f / 120.f), 1.f / 24.f), 1.f / 6.f);
  const float s = __fmaf_rn(xx, 0.5f, x);
  const float sl = __fmaf_rn(xx, 0.5f, __fsub_rn(x, s)) + (xl + 0.5f * xxl + cubic);
  // 2^(k/32) (1 + s)
  const float2 t = tab[k & 31];
  const float q = __fmul_rn(t.x, s);
  const float ql = __fmaf_rn(t.x, s, -q) + __fmaf_rn(t.x, sl, t.y * s);
  h = __fadd_rn(t.x, q);
  hl = __fsub_rn(q, __fsub_rn(h, t.x)) + (ql + t.y);
  n = k >> 5;
}

// What turns a logit into its weight: y = (z - zmax) log2(e) / T, log2(e) / T
// as a pair of floats, and the fixed point's scale.
struct Weigher {
  float zmax, c_hi, c_lo, one;  // one = 2^B
  float d_min;                  // z - zmax where y = -120
  int down;                     // 44 - B
  const float2* tab;
};

// W = round(2^(y + B)) of two logits, 0 below y = -40 and for NaN. The steps are
// those of exp2_pair, for both at once; the argument error is 2^-46 |y|. Every copy of
// this gives the same bits, so that the parts of a row add up to its sum wherever they
// are weighed: no sum here takes a product, which might be rounded together with it
// (see f32x2.cuh).
__device__ __forceinline__ void weight2(const Weigher& w, uint64_t z, uint64_t& w0, uint64_t& w1) {
  const uint64_t neg = pair_of(-1.f), c = pair_of(w.c_hi), top = pair_of(-w.zmax);
  // z - zmax without loss: the difference and what its rounding left
  const uint64_t d = add2(z, top), b = fma2(z, neg, d);
  const uint64_t dl = add2(fma2(fma2(b, neg, d), neg, z), fma2(b, neg, top));
  const uint64_t p = mul2(d, c);
  const uint64_t pl = add2(fma2(d, c, mul2(p, neg)), fma2(d, pair_of(w.c_lo), mul2(dl, c)));
  const float2 pf = of_pair(p);
  const uint64_t y = pair_of(__float_as_uint(fmaxf(pf.x, -41.f)), __float_as_uint(fmaxf(pf.y, -41.f)));
  // y = k / 32 + r, |r| <= 1/64
  const uint64_t kt = fma2(y, pair_of(32.f), pair_of(12582912.f));
  const uint64_t r0 = fma2(add2(kt, pair_of(-12582912.f)), pair_of(-0.03125f), y);
  const uint64_t r = add2(r0, pl), rl = fma2(fma2(r0, neg, r), neg, pl);
  const uint64_t ln2 = pair_of(kLn2), half = pair_of(0.5f);
  const uint64_t x = mul2(r, ln2);
  const uint64_t xl = add2(fma2(r, ln2, mul2(x, neg)), fma2(r, pair_of(kLn2Lo), mul2(rl, ln2)));
  const uint64_t xx = mul2(x, x);
  const uint64_t xxl = fma2(x, add2(xl, xl), fma2(x, x, mul2(xx, neg)));
  const uint64_t q3 = fma2(x, fma2(x, fma2(x, pair_of(1.f / 720.f), pair_of(1.f / 120.f)), pair_of(1.f / 24.f)),
                           pair_of(1.f / 6.f));
  const uint64_t s = fma2(xx, half, x);
  const uint64_t sl = add2(fma2(xx, half, fma2(s, neg, x)), fma2(xxl, half, fma2(mul2(xx, x), q3, xl)));
  const float2 ktf = of_pair(kt);
  const uint32_t k0 = __float_as_uint(ktf.x), k1 = __float_as_uint(ktf.y);  // 0x4B400000 + k
  const float2 t0 = w.tab[k0 & 31], t1 = w.tab[k1 & 31];
  const uint64_t tx = pair_of(__float_as_uint(t0.x), __float_as_uint(t1.x));
  const uint64_t ty = pair_of(__float_as_uint(t0.y), __float_as_uint(t1.y));
  const uint64_t q = mul2(tx, s);
  const uint64_t ql = add2(fma2(tx, s, mul2(q, neg)), fma2(tx, sl, mul2(ty, s)));
  const uint64_t h = fma2(tx, s, tx);
  const uint64_t hl = add2(fma2(fma2(tx, neg, h), neg, q), add2(ql, ty));
  // 2^44 (h + hl), h in [0.98, 2) with 24 bits behind the point at most; then
  // down by 44 - B - n
  const float2 hf = of_pair(mul2(h, pair_of(16777216.f))), lf = of_pair(mul2(hl, pair_of(17592186044416.f)));
  auto fixed = [&](float hi, float lo, uint32_t k, float pp, float zz) {
    const uint64_t v = (static_cast<uint64_t>(__float2uint_rn(hi)) << 20) + static_cast<int64_t>(__float2int_rn(lo));
    const int down = w.down - (static_cast<int>(k - 0x4B400000u) >> 5);
    const uint64_t r = (v + ((1ull << down) >> 1)) >> down;
    return zz == w.zmax ? static_cast<uint64_t>(__float2ll_rn(w.one)) : pp >= kCut ? r : 0;
  };
  const float2 zf = of_pair(z);
  w0 = fixed(hf.x, lf.x, k0, pf.x, zf.x);
  w1 = fixed(hf.y, lf.y, k1, pf.y, zf.y);
}
__device__ __noinline__ uint64_t weight(Weigher w, float z) {
  uint64_t a, b;
  weight2(w, pair_of(z), a, b);
  return a;
}

// floor and ceiling of f x for 0 <= f < 1: exact
__device__ __forceinline__ uint64_t mul_floor(float f, uint64_t x, bool& rest) {
  const uint32_t b = __float_as_uint(f), e = b >> 23;
  const uint64_t m = e ? (b & 0x7FFFFFu) | 0x800000u : b;
  const int sh = 150 - static_cast<int>(e ? e : 1);  // f = m 2^-sh, sh >= 24
  const uint64_t lo = m * x, hi = __umul64hi(m, x);
  if (sh < 64) {
    rest = (lo & ((1ull << sh) - 1)) != 0;
    return (lo >> sh) | (hi << (64 - sh));
  }
  if (sh < 128) {
    rest = lo != 0 || (hi & ((1ull << (sh - 64)) - 1)) != 0;
    return hi >> (sh - 64);
  }
  rest = (lo | hi) != 0;
  return 0;
}
__device__ __forceinline__ uint64_t mul_ceil(float f, uint64_t x) {
  bool rest;
  const uint64_t r = mul_floor(f, x, rest);
  return r + rest;
}
__device__ __forceinline__ uint64_t distance(uint64_t a, uint64_t b) { return a > b ? a - b : b - a; }

// y in single precision, for the bins.
__device__ __forceinline__ float fast_y(const Weigher& w, float z) { return (z - w.zmax) * w.c_hi; }

// The fast weight, 2^(n + f): n = round(d log2(e) / T) by adding 1.5 * 2^23, f what
// the product leaves, 2^f = 1 + f q(f) with q of degree 5, within 2^-25.9. In
// units of 2^-24 its error is 1.3 for 2^f, 0.4 for f and 0.7 |y| for d = z - zmax
// (exact for bf16 logits, but for |z| below 2^-16 |zmax|). It has no cut at 2^-40;
// what it has below is V 2^-40 at most. (The special-function unit's 2^y is four
// times less exact: one row in seven of a spread-out softmax was left to the exact
// weights.)
constexpr float kRound = 12582912.f;  // 1.5 * 2^23
#define SAMPLE_Q {0x1.62e430p-1f, 0x1.ebfbdcp-3f, 0x1.c6aee8p-5f, 0x1.3b2d4cp-7f, 0x1.5f3e58p-10f, 0x1.41fbc8p-13f}
__device__ __forceinline__ float fast_weight(const Weigher& w, float z) {
  const float d = fmaxf(z - w.zmax, w.d_min);
  const float t = __fmaf_rn(d, w.c_hi, kRound);
  const float f = __fmaf_rn(d, w.c_lo, __fmaf_rn(d, w.c_hi, -__fsub_rn(t, kRound)));
  const float k[6] = SAMPLE_Q;
  float q = k[5];
#pragma unroll
  for (int i = 4; i >= 0; --i) q = __fmaf_rn(q, f, k[i]);
  return __uint_as_float(__float_as_uint(__fmaf_rn(q, f, 1.f)) + (__float_as_uint(t) << 23));
}
// The same of two logits.
__device__ __forceinline__ uint64_t fast_weight2(uint64_t z, uint64_t top, float d_min, uint64_t c_hi,
                                                 uint64_t c_lo) {
  const float2 d0 = of_pair(add2(z, top));
  const uint64_t d = pair_of(__float_as_uint(fmaxf(d0.x, d_min)), __float_as_uint(fmaxf(d0.y, d_min)));
  const uint64_t t = fma2(d, c_hi, pair_of(kRound));
  const uint64_t n = add2(t, pair_of(-kRound));
  const uint64_t f = fma2(d, c_lo, fma2(d, c_hi, mul2(n, pair_of(-1.f))));
  const float k[6] = SAMPLE_Q;
  uint64_t q = pair_of(k[5]);
#pragma unroll
  for (int i = 4; i >= 0; --i) q = fma2(q, f, pair_of(k[i]));
  const float2 r = of_pair(fma2(q, f, pair_of(1.f))), e = of_pair(t);
  return pair_of(__float_as_uint(r.x) + (__float_as_uint(e.x) << 23),
                 __float_as_uint(r.y) + (__float_as_uint(e.y) << 23));
}

// The rough weights, from the special-function unit: 2^y to 2^-22.4, y off by its own
// rounding and c_hi's, 2^-24 |y|. (NaN weighs nothing.)
__device__ __forceinline__ uint64_t rough_weight2(uint64_t z, uint64_t top, uint64_t c_hi) {
  const float2 y = of_pair(mul2(add2(z, top), c_hi));
  return pair_of(__float_as_uint(ex2_approx(clean(y.x))), __float_as_uint(ex2_approx(clean(y.y))));
}

// Element weight as an integer.
template <bool EXACT>
__device__ __forceinline__ uint64_t weigh(const Weigher& w, float z) {
  if (EXACT) return weight(w, z);
  return static_cast<uint64_t>(__float2ll_rn(fast_weight(w, z) * w.one));
}

__device__ __forceinline__ uint64_t warp_sum(uint64_t v) {
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
__device__ __forceinline__ uint64_t warp_scan(uint64_t v, int lane) {  // inclusive
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint64_t n = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += n;
  }
  return v;
}

// Sum of floats without the growth of rounding errors: what each addition
// rounds away is kept beside the sum.
struct PairSum {
  float hi = 0.f, lo = 0.f;
  __device__ __forceinline__ void add(float v) {
    const float s = __fadd_rn(hi, v), b = __fsub_rn(s, hi);
    lo = __fadd_rn(lo, __fadd_rn(__fsub_rn(hi, __fsub_rn(s, b)), __fsub_rn(v, b)));
    hi = s;
  }
  __device__ __forceinline__ uint64_t fixed(float one) const {
    return static_cast<uint64_t>(__float2ll_rn(hi * one) + __float2ll_rn(lo * one));
  }
};

// What the parts of a row add up to.
struct Part {
  uint64_t mass = 0;
  uint32_t count = 0;
  uint32_t lo = 0xFFFFFFFFu, hi = 0;
  float sum = 0.f;
};
enum : int { P_MASS = 1, P_COUNT = 4, P_LO = 8, P_HI = 16, P_SUM = 32 };

struct Shared {
  float2 tab[32];
  uint64_t cand[kCap];              // this CTA's candidates, the leader's list: key, then ~index
  union {
    uint64_t wts[kCap];             // their weights
    uint32_t hist[kBins];           // masses of the bins (read before there are weights)
  };
  uint32_t n_cand;
  // the leader's answers to the cluster, alternating between rows
  struct {
    uint32_t t, ties;
    int bad;
  } ans[2];
  // this CTA's scratch
  uint32_t scan_u[kMaxWarps];
  // the draw: the warp that holds u, what is ahead of it, and its chunks
  int b;
  uint32_t base_ties;
  uint64_t base, chunk[kMaxWarps];
  uint32_t chunk_ties[kMaxWarps];
  uint32_t n_kept;
  // what the fast way leaves to the exact one: the top-p cut is behind the list;
  // it lies among the logits from z2 to z1
  int behind, found;
  float z1, z2;
  // the row's parameters
  Weigher w;
  float floor_z, top_p, u, temp;
  int top_k, warm, use_p, use_q;
};

template <typename T, bool ONE>
struct Row;
template <typename T, bool ONE>
__device__ __noinline__ ulonglong2 exact_mass(const Row<T, ONE> r, const Weigher w, float lo, float hi);

// One row, seen from one CTA. ONE: the row has one CTA and no cluster.
template <typename T, bool ONE>
struct Row {
  static constexpr int VE = Vec<T>::N;
  cg::cluster_group cl = cg::this_cluster();
  Shared& sh;
  Part* parts;         // [2][C of at most 8][warps], alternating between joins
  const uint4* slice;  // this CTA's slice in shared memory, or null: the logits are read again
  const uint4* global; // its first piece among the logits
  const T* row;
  int n_vec;           // 16-byte pieces of the slice
  int64_t pos0;        // row index of the slice's first element (may be below 0)
  int64_t V;
  int lane, warp, nt, nw, C, rank, turn = 0, par = 0;  // nt threads, nw warps
  int v0, v1;          // this warp's pieces
  float hist_bits = 13.f;  // of a bin's mass: no sum of them passes 2^32
  int full0, full1;    // pieces that lie inside the row

  __device__ __forceinline__ Row(Shared& s) : sh(s) {}

  // Piece v from global memory. The pieces at the row's ends hold other rows'
  // elements, or none: these are read one by one, with -inf in their place.
  __device__ __forceinline__ Vec<T> fetch(int v) const {
    Vec<T> x;
    if (v >= full0 && v < full1) {
      x.raw = __ldg(global + v);
    } else {
      const int64_t i0 = pos0 + static_cast<int64_t>(v) * VE;
      uint32_t w[4];
      T* e = reinterpret_cast<T*>(w);
#pragma unroll
      for (int i = 0; i < VE; ++i)
        e[i] = i0 + i >= 0 && i0 + i < V ? row[i0 + i] : static_cast<T>(-INFINITY);
      x.raw = make_uint4(w[0], w[1], w[2], w[3]);
    }
    return x;
  }
  // This CTA's slice of a row: 16-byte pieces from the one that holds the row's
  // first element. `to`: shared memory for it, or null (it is read again from L2).
  __device__ __forceinline__ void place(const SampleArgs& a, int64_t which, int slice_vecs, uint4* to) {
    const T* z = static_cast<const T*>(a.logits) + which * a.ld;
    const int off = static_cast<int>((reinterpret_cast<uintptr_t>(z) & 15) / sizeof(T));
    const int64_t all = (off + a.V + VE - 1) / VE;
    const int64_t p0 = static_cast<int64_t>(rank) * slice_vecs;
    n_vec = static_cast<int>(p0 >= all ? 0 : min(static_cast<int64_t>(slice_vecs), all - p0));
    pos0 = p0 * VE - off;
    const int per = (n_vec + nw - 1) / nw;
    v0 = min(n_vec, warp * per);
    v1 = min(n_vec, v0 + per);
    full0 = pos0 < 0 ? 1 : 0;
    full1 = static_cast<int>(min(static_cast<int64_t>(n_vec), a.V > pos0 ? (a.V - pos0) / VE : 0));
    V = a.V;
    row = z;
    global = reinterpret_cast<const uint4*>(z - off) + p0;
    slice = to;
  }

  // Copies the slice, taking this thread's maximum on the way (a warp reads back its own).
  __device__ __forceinline__ float copy_in() {
    uint4* to = const_cast<uint4*>(slice);
    float mx = -INFINITY;
    // the pieces that lie inside the row, all on their way at once
    const int f0 = max(v0, full0), f1 = min(v1, full1);
    if (to) {
      for (int v = f0 + lane; v < f1; v += 32)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                         static_cast<uint32_t>(__cvta_generic_to_shared(to + v))),
                     "l"(global + v)
                     : "memory");
      asm volatile("cp.async.commit_group;\n\tcp.async.wait_group 0;" ::: "memory");
    }
    for (int vb = f0 + lane; vb < f1; vb += 256) {  // (each lane reads its own copies)
      Vec<T> x[8];
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (vb + 32 * i < f1) x[i].raw = to ? to[vb + 32 * i] : __ldg(global + vb + 32 * i);
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (vb + 32 * i < f1) mx = fmaxf(mx, x[i].max());
    }
    // and the ones at its ends
    for (int v = v0 + lane; v < v1; v += 32) {
      if (v >= f0 && v < f1) continue;
      const Vec<T> x = fetch(v);
      if (to) to[v] = x.raw;
      mx = fmaxf(mx, x.max());
    }
    return mx;
  }

  __device__ __forceinline__ Vec<T> load(int v) const {
    if (slice == nullptr) return fetch(v);
    Vec<T> x;
    x.raw = slice[v];
    return x;
  }

  // f(piece, its number) for this warp's pieces, U loads at a time; (step, lane,
  // element) is their index order.
  template <int U = 1, typename F>
  __device__ __forceinline__ void pieces(F f) const {
#pragma unroll 1
    for (int vb = v0 + lane; vb < v1; vb += 32 * U) {
      Vec<T> x[U];
#pragma unroll
      for (int i = 0; i < U; ++i)
        if (vb + 32 * i < v1) x[i] = load(vb + 32 * i);
#pragma unroll
      for (int i = 0; i < U; ++i)
        if (vb + 32 * i < v1) f(x[i], vb + 32 * i);
    }
  }

  // Waits for the row's CTAs, whose writes are then seen.
  __device__ __forceinline__ void sync() {
    if (ONE) __syncthreads();
    else cl.sync();
  }
  template <typename U>
  __device__ __forceinline__ U* of_rank(U* p, int k) {
    return ONE ? p : cl.map_shared_rank(p, k);
  }

  template <int F>
  __device__ __forceinline__ static void add(Part& p, const Part& o) {
    if (F & P_MASS) p.mass += o.mass;
    if (F & P_SUM) p.sum += o.sum;
    if (F & P_COUNT) p.count += o.count;
    if (F & P_LO) p.lo = min(p.lo, o.lo);
    if (F & P_HI) p.hi = max(p.hi, o.hi);
  }
  template <int F>
  __device__ __forceinline__ static void put(Part& to, const Part& p) {
    if (F & P_MASS) to.mass = p.mass;
    if (F & P_SUM) to.sum = p.sum;
    if (F & P_COUNT) to.count = p.count;
    if (F & P_LO) to.lo = p.lo;
    if (F & P_HI) to.hi = p.hi;
  }
  // The fields F of the warp's Parts, in every lane. (A mass below 2^62 is added up
  // as three limbs: a reduction of 32 bits is one instruction, one of 64 ten shuffles.)
  template <int F>
  __device__ __forceinline__ static void lanes(Part& p) {
    constexpr uint32_t all = 0xffffffffu, limb = (1u << 27) - 1;
    if (F & P_MASS) {
      const uint32_t a = __reduce_add_sync(all, static_cast<uint32_t>(p.mass) & limb);
      const uint32_t b = __reduce_add_sync(all, static_cast<uint32_t>(p.mass >> 27) & limb);
      const uint32_t c = __reduce_add_sync(all, static_cast<uint32_t>(p.mass >> 54));
      p.mass = a + (static_cast<uint64_t>(b) << 27) + (static_cast<uint64_t>(c) << 54);
    }
    if (F & P_COUNT) p.count = __reduce_add_sync(all, p.count);
    if (F & P_LO) p.lo = __reduce_min_sync(all, p.lo);
    if (F & P_HI) p.hi = __reduce_max_sync(all, p.hi);
    if (F & P_SUM)
#pragma unroll
      for (int o = 16; o >= 1; o >>= 1) p.sum += __shfl_xor_sync(all, p.sum, o);
  }

  // Joins the fields F of every thread's Part over the cluster; each thread gets
  // the whole, `mine` its warp's and `before` what the warps ahead of its own
  // have. A warp pushes its sum into every CTA's shared memory, so that after
  // one barrier all is read at home (remote shared memory is slow to read: 128
  // Parts read by every warp took 16,000 cycles).
  template <int F>
  __device__ __forceinline__ Part join(Part p, Part* mine = nullptr, Part* before = nullptr) {
    lanes<F>(p);
    if (mine) *mine = p;
    const int n = C * nw, me = rank * nw + warp;
    Part* slots = parts + turn * C * nw;
    if (lane < C) put<F>(*of_rank(slots + me, lane), p);
    sync();
    Part all, ahead;
    for (int i = lane; i < n; i += 32) {
      Part o;
      put<F>(o, slots[i]);
      add<F>(all, o);
      if (before && i < me) add<F>(ahead, o);
    }
    lanes<F>(all);
    if (before) {
      lanes<F>(ahead);
      *before = ahead;
    }
    turn ^= 1;
    return all;
  }

  // f(z) for the pieces whose largest element passes `some`.
  template <typename P, typename F>
  __device__ __forceinline__ void each_if(P some, F f) const {
    pieces([&](const Vec<T>& x, int) {
      if (!some(x.max())) return;
#pragma unroll
      for (int e = 0; e < VE; ++e) f(x.get(e));
    });
  }

  // Number of tokens above key k, and their exact mass.
  template <bool MASS>
  __device__ Part above(const Weigher& w, uint32_t k) {
    Part p;
    each_if([&](float z) { return key_of(z) > k; }, [&](float z) { p.count += key_of(z) > k; });
    if (MASS) {
      p.mass = exact_mass(*this, w, above_key(k), INFINITY).x;
    }
    return join<MASS ? P_MASS | P_COUNT : P_COUNT>(p);
  }

  // Bin of a logit in steps of 1/32 of a binary order below the top.
  __device__ __forceinline__ static int bin_of(float y) { return static_cast<int>(-32.f * y); }

  // Adds an element to this CTA's list.
  __device__ __forceinline__ void list(float z, int v, int e) {
    const uint32_t at = atomicAdd(&sh.n_cand, 1u);
    const uint32_t idx = static_cast<uint32_t>(pos0 + static_cast<int64_t>(v) * VE + e);
    if (at < kCap) sh.cand[at] = (static_cast<uint64_t>(key_of(z)) << 32) | ~idx;
  }

  // Lists the elements from lo to hi; returns their number over the cluster.
  __device__ uint32_t gather(float lo, float hi) {
    Part p;
    pieces([&](const Vec<T>& x, int v) {
      if (!(x.max() >= lo)) return;
#pragma unroll
      for (int e = 0; e < VE; ++e) {
        const float z = x.get(e);
        if (z >= lo && z <= hi) {
          list(z, v, e);
          ++p.count;
        }
      }
    });
    return join<P_COUNT>(p).count;
  }

  // The leader fetches the other CTAs' lists, n <= kCap candidates in all.
  __device__ void fetch_lists(uint32_t n) {
    if (static_cast<int>(threadIdx.x) < C) sh.scan_u[threadIdx.x] = *of_rank(&sh.n_cand, threadIdx.x);
    __syncthreads();
    for (uint32_t i = sh.scan_u[0] + threadIdx.x; i < n; i += nt) {
      uint32_t j = i;
      int c = 0;
      while (j >= sh.scan_u[c]) j -= sh.scan_u[c++];
      sh.cand[i] = of_rank(sh.cand, c)[j];
    }
    __syncthreads();
  }

  // Sorts the leader's n candidates, largest first, and weighs them. A few by
  // counting the larger ones of each: a barrier of the CTA takes some 200 cycles
  // and a sorting network of 128 elements has 28 of them.
  __device__ void sort_and_weigh(uint32_t n) {
    if (n <= kCount) {
      uint64_t c = 0;
      uint32_t at = 0;
      if (threadIdx.x < n) {
        c = sh.cand[threadIdx.x];
        for (uint32_t j = 0; j < n; ++j) at += sh.cand[j] > c;
      }
      __syncthreads();
      if (threadIdx.x < n) {
        sh.cand[at] = c;
        sh.wts[at] = weight(sh.w, float_of(static_cast<uint32_t>(c >> 32)));
      }
    } else {
      sort_desc(sh.cand, n);
      for (uint32_t i = threadIdx.x; i < n; i += nt)
        sh.wts[i] = weight(sh.w, float_of(static_cast<uint32_t>(sh.cand[i] >> 32)));
    }
    __syncthreads();
  }

  // Sorts the first n of a list in shared memory, largest first (one CTA).
  __device__ void sort_desc(uint64_t* a, uint32_t n) {
    uint32_t n2 = 2;
    while (n2 < n) n2 <<= 1;
    for (uint32_t i = n + threadIdx.x; i < n2; i += nt) a[i] = 0;
    __syncthreads();
    for (uint32_t k = 2; k <= n2; k <<= 1)
      for (uint32_t j = k >> 1; j > 0; j >>= 1) {
        for (uint32_t i = threadIdx.x; i < n2 / 2; i += nt) {
          const uint32_t lo = 2 * i - (i & (j - 1)), hi = lo + j;
          const uint64_t x = a[lo], y = a[hi];
          if ((x < y) == ((lo & k) == 0)) {
            a[lo] = y;
            a[hi] = x;
          }
        }
        __syncthreads();
      }
  }
};

// The exact mass of this thread's elements above `lo`, and of those above `hi`; in
// a function of its own, whose registers are the weights'.
template <typename T, bool ONE>
__device__ __noinline__ ulonglong2 exact_mass(const Row<T, ONE> r, const Weigher w, float lo, float hi) {
  uint64_t m = 0, n = 0;
#pragma unroll 1
  for (int v = r.v0 + r.lane; v < r.v1; v += 32) {
    const Vec<T> x = r.load(v);
    if (!(x.max() > lo)) continue;
#pragma unroll 2
    for (int e = 0; e < Vec<T>::N / 2; ++e) {
      const uint64_t z = x.pair(e);
      uint64_t a, b;
      weight2(w, z, a, b);
      const float2 f = of_pair(z);
      m += (f.x > lo ? a : 0) + (f.y > lo ? b : 0);
      n += (f.x > hi ? a : 0) + (f.y > hi ? b : 0);
    }
  }
  return make_ulonglong2(m, n);
}

// Threshold and ties that the cut-offs keep.
struct Kept {
  uint32_t t = 0, ties = 0xFFFFFFFFu;
};

// The largest value of 16 leading bits that at least k of the warp's keys reach
// (N a lane); 0 if fewer do.
template <int N>
__device__ __forceinline__ uint32_t kth_from_below(const uint32_t (&key)[N], uint32_t k) {
  uint32_t prefix = 0;
#pragma unroll
  for (int bit = 31; bit >= 16; --bit) {
    const uint32_t t = prefix | (1u << bit);
    uint32_t n = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) n += __popc(__ballot_sync(0xffffffffu, key[i] >= t));
    if (n >= k) prefix = t;
  }
  return prefix;
}

// Bound on the error of any sum of fast weights, in units of W: 2^-24 sum w (1.7 +
// 0.7 |y|), and three roundings in the sum of a piece. The entropy of w / S is at
// most log2 V, so sum w |y| <= S log2(V / S); for bf16 the term with |y| is left
// only for logits around 0, whose weights are 2^(-zmax log2(e) / T).
// The rough weights' sums are off by 2^-24 sum w (3 + 0.7 |y| (1 + e)) beside what the
// difference's rounding leaves, for every type, and the same three roundings: y is
// rounded once, and its factor c_hi is e 2^-24 off, what c_lo holds.
template <typename T>
__device__ __forceinline__ uint64_t error_bound(const Weigher& w, uint64_t mass, int64_t V, bool rough = false) {
  const float s = static_cast<float>(mass) / w.one, v = static_cast<float>(V);
  const float y0 = fmaxf(0.f, w.zmax * w.c_hi), sum_y = s * fmaxf(0.f, log2f(v / s));
  float terms = s * 5.5f + (sizeof(T) == 4 ? 0.8f * sum_y : v * ex2_approx(-y0) * fminf(y0, 200.f));
  if (rough) terms += 0.7f * s + 0.7f * sum_y * (1.f + fabsf(w.c_lo) / w.c_hi * 16777216.f);
  return static_cast<uint64_t>(__float2ll_ru((terms * 6.0e-8f + v * 1e-12f) * w.one)) + 2 * V + 1024;
}

// The row's parameters (one thread; zmax and the min-p floor follow).
__device__ __forceinline__ void set_row(Shared& sh, float t, int k, float p, bool use_q, float u,
                                        int64_t V) {
  sh.behind = sh.found = 0;
  sh.n_cand = 0;
  sh.warm = t > 0.f;
  const float temp = sh.warm ? t : 1.f;
  sh.temp = temp;
  // log2(e) / T, kept within float's range (a T near 0, an infinite one)
  const float c = fminf(fmaxf(kLog2e / temp, 1.4e-45f), 3.4e38f);
  sh.w.c_hi = c;
  sh.w.c_lo = c > 1e-30f && c < 1e30f ? (__fmaf_rn(-c, temp, kLog2e) + kLog2eLo) / temp : 0.f;
  sh.w.d_min = -120.f / c;
  // V 2^B < 2^62
  const int bits = min(44, 62 - (32 - __clz(static_cast<int>(V))));
  sh.w.one = __uint_as_float(static_cast<uint32_t>(127 + bits) << 23);
  sh.w.down = 44 - bits;
  sh.w.tab = sh.tab;
  sh.top_k = k > 0 && k < V ? k : 0;
  sh.use_q = use_q;
  sh.use_p = p < 1.f;
  sh.top_p = fmaxf(p, 0.f);
  sh.u = fminf(fmaxf(u, 0.f), 1.f - 5.9604645e-8f);
}

// The token of a row and its log-probability (one thread).
template <typename T>
__device__ __forceinline__ void write_row(const SampleArgs& a, int64_t row, const T* logits, const Shared& sh,
                                          const Weigher& w, uint64_t mass, int par = 0) {
  // (an index that no draw has set stays in the row)
  const int64_t at = min(static_cast<int64_t>(sh.ans[par].t), a.V - 1);
  const float z = clean(to_f(logits[at]));
  const float d = z == w.zmax ? 0.f : (z - w.zmax) / sh.temp;
  // ln(mass): the sum as two floats
  const float hi = static_cast<float>(mass);
  const float lo = static_cast<float>(static_cast<int64_t>(mass - static_cast<uint64_t>(hi)));
  a.tokens[row] = static_cast<int32_t>(at);
  a.logp[row] = d - (logf(hi / w.one) + lo / hi);
}

constexpr int32_t kUndecided = -2, kClose = -3;  // mark rows that are left for a second launch

// How the leader's list served: the token is in ans.t; or u or the top-p cut is
// within the error of a border; or the top-p cut is behind the list's end.
enum : int { L_DONE = 0, L_CLOSE = 1, L_SHORT = 2 };

// The leader alone draws from its list of n candidates, exactly. With top-k the
// list holds the k first tokens, with `whole` every token that can stay. `own`: the
// top-p cut is taken of the list's mass; else of `base`, off by slack at most.
template <typename T, bool ONE>
__device__ __noinline__ void draw_from_list(Row<T, ONE> r, uint32_t n, bool warm, uint64_t base,
                                            uint64_t slack, bool whole, bool own) {
  Shared& sh = r.sh;
  const int lane = r.lane, warp = r.warp;
  const bool use_k = !warm || sh.top_k > 0, use_p = warm && sh.use_p;
  r.fetch_lists(n);
  r.sort_and_weigh(n);
  if (warp == 0) {
    const uint32_t floor_key = sh.use_q ? key_of(sh.floor_z) : 0;
    uint32_t n_l = n;
    if (use_k) n_l = min(n_l, warm ? static_cast<uint32_t>(sh.top_k) : 1u);
    if (sh.use_q) {  // those from the min-p floor on are the first of the order
      uint32_t m = 0;
      for (uint32_t i = lane; i < n_l; i += 32) m += static_cast<uint32_t>(sh.cand[i] >> 32) >= floor_key;
      m = __reduce_add_sync(0xffffffffu, m);
      whole |= m < n_l;
      n_l = m;
    }
    int state = L_DONE;
    if (use_p) {
      if (own || use_k) {
        base = 0;
        for (uint32_t i = lane; i < n_l; i += 32) base += sh.wts[i];
        base = warp_sum(base);
        slack = 0;
        whole = true;
      }
      const uint64_t want = mul_ceil(sh.top_p, base);
      uint64_t run = 0;
      uint32_t stay = 0;
      for (uint32_t i0 = 0; i0 < n_l; i0 += 32) {
        const uint32_t i = i0 + lane;
        const uint64_t x = i < n_l ? sh.wts[i] : 0;
        const uint64_t ahead = run + warp_scan(x, lane) - x;
        stay += __popc(__ballot_sync(0xffffffffu, i < n_l && ahead < want));
        if (__any_sync(0xffffffffu, slack && i < n_l && i > 0 && distance(ahead, want) <= slack)) state = L_CLOSE;
        run += warp_sum(x);
      }
      if (!whole && run <= want + slack) state = L_SHORT;
      else if (slack && run <= want + slack) state = L_CLOSE;
      n_l = max(1u, stay);
    }
    if (lane == 0) {
      sh.n_kept = n_l;
      sh.ans[r.par].bad = state;
      sh.ans[r.par].t = 0xFFFFFFFFu;
    }
  }
  __syncthreads();
  const uint32_t n_l = sh.n_kept;
  if (sh.ans[r.par].bad != L_DONE) return;
  // The draw runs in the row's own order. Of a few, each adds up the weights of
  // the indexes up to its own.
  if (n_l <= kCount) {
    if (warp * 32 < static_cast<int>(n_l)) {
      uint64_t total = 0, upto_me = 0;
      const bool in = threadIdx.x < n_l;
      const uint32_t me = in ? static_cast<uint32_t>(sh.cand[threadIdx.x]) : 0;
      for (uint32_t j = 0; j < n_l; ++j) {
        const uint64_t x = sh.wts[j];
        total += x;
        if (static_cast<uint32_t>(sh.cand[j]) >= me) upto_me += x;  // (~index)
      }
      bool rest;
      if (in && upto_me > mul_floor(sh.u, total, rest)) atomicMin(&sh.ans[r.par].t, ~me);
    }
  } else {
    for (uint32_t i = threadIdx.x; i < n_l; i += r.nt)
      sh.cand[i] = (sh.cand[i] << 32) | i;  // ~index descends as the index ascends
    __syncthreads();
    r.sort_desc(sh.cand, n_l);
    if (warp == 0) {
      uint64_t total = 0;
      for (uint32_t i = lane; i < n_l; i += 32) total += sh.wts[i];
      bool rest;
      const uint64_t target = mul_floor(sh.u, warp_sum(total), rest);
      uint64_t run = 0;
      for (uint32_t i0 = 0; i0 < n_l; i0 += 32) {
        const uint32_t i = i0 + lane;
        const uint64_t c = i < n_l ? sh.cand[i] : 0;
        const uint64_t x = i < n_l ? sh.wts[static_cast<uint32_t>(c)] : 0;
        const uint32_t hit = __ballot_sync(0xffffffffu, run + warp_scan(x, lane) > target);
        if (hit) {
          const uint32_t at =
              ~static_cast<uint32_t>(__shfl_sync(0xffffffffu, c, __ffs(hit) - 1) >> 32);
          if (lane == 0) sh.ans[r.par].t = at;
          break;
        }
        run += warp_sum(x);
      }
    }
  }
}

// The smallest key t from lo to hi that `enough` holds for (it holds for hi, and
// from some key on). bf16 logits differ in a key's upper half only.
template <typename T, typename F>
__device__ __forceinline__ uint32_t first_key(uint32_t lo, uint32_t hi, F enough) {
  constexpr int SH = sizeof(T) == 2 ? 16 : 0;
  auto whole = [](uint32_t k) { return SH == 0 ? k : k >= 0x8000u ? k << SH : (k << SH) | 0xFFFFu; };
  uint32_t a = lo >> SH, b = hi >> SH;
  while (a < b) {
    const uint32_t mid = a + (b - a) / 2;
    if (enough(whole(mid))) b = mid;
    else a = mid + 1;
  }
  return whole(a);
}

// Where the top-p cut falls, when `want` is to be kept: a threshold and its ties,
// from the mass ahead of the logits z2 to z1 and a look at these. Returns 1 where
// that is found, 0 where it is not among them, -1 within E of a border. *mine_a:
// this warp's mass above z1.
template <typename T, bool ONE, bool EXACT>
__device__ __noinline__ int cut_between(Row<T, ONE> r, int* turn, uint32_t* t, uint32_t* ties,
                                        uint64_t* mine_a, uint64_t above, uint64_t want, uint64_t E) {
  Shared& sh = r.sh;
  const Weigher w = sh.w;
  const float z1 = sh.z1, z2 = sh.z2;
  Part q;
  PairSum f;
  const uint64_t top = pair_of(-w.zmax), c_hi = pair_of(w.c_hi), c_lo = pair_of(w.c_lo);
  r.pieces([&](const Vec<T>& x, int) {
    if (!(x.max() >= z2)) return;
#pragma unroll
    for (int e = 0; e < Vec<T>::N / 2; ++e) {
      const uint64_t z = x.pair(e);
      const float2 v = of_pair(z);
      if (!EXACT) {
        const float2 m = of_pair(fast_weight2(z, top, w.d_min, c_hi, c_lo));
        f.add((v.x > z1 ? m.x : 0.f) + (v.y > z1 ? m.y : 0.f));
      }
      for (float y : {v.x, v.y}) {
        if (y >= z2 && y <= z1) {
          const uint32_t key = key_of(y);
          ++q.count;
          q.lo = min(q.lo, key);
          q.hi = max(q.hi, key);
        }
      }
    }
  });
  q.mass = EXACT ? above : f.fixed(w.one);
  Part mine;
  q = r.template join<P_MASS | P_COUNT | P_LO | P_HI>(q, &mine);
  *mine_a = mine.mass;
  int state = 0;
  if (q.count > 0 && want > q.mass) {
    const uint64_t rest = want - q.mass;
    if (q.lo != q.hi && q.count <= kCap) {
      // few enough to be sorted by the leader
      if (threadIdx.x == 0) sh.n_cand = 0;
      __syncthreads();
      r.gather(z2, z1);
      if (r.rank == 0) {
        r.fetch_lists(q.count);
        r.sort_and_weigh(q.count);
        if (r.warp == 0) {
          uint64_t run = 0;
          uint32_t stay = 0;
          bool close = false;
          for (uint32_t i0 = 0; i0 < q.count; i0 += 32) {
            const uint32_t i = i0 + r.lane;
            const uint64_t x = i < q.count ? sh.wts[i] : 0;
            const uint64_t ahead = run + warp_scan(x, r.lane) - x;
            stay += __popc(__ballot_sync(0xffffffffu, i < q.count && ahead < rest));
            close |= E && __any_sync(0xffffffffu, i < q.count && distance(ahead, rest) <= 2 * E);
            run += warp_sum(x);
          }
          close |= E && distance(run, rest) <= 2 * E;
          const uint32_t key = stay ? static_cast<uint32_t>(sh.cand[stay - 1] >> 32) : 0;
          uint32_t n = 0;
          for (uint32_t i = r.lane; i < stay; i += 32) n += static_cast<uint32_t>(sh.cand[i] >> 32) == key;
          n = __reduce_add_sync(0xffffffffu, n);
          if (r.lane == 0) {
            sh.ans[r.par].t = key;
            sh.ans[r.par].ties = n;
            sh.ans[r.par].bad = close ? -1 : stay == 0 || run < rest ? 0 : 1;
          }
        }
      }
      r.sync();
      const auto& lead = r.of_rank(&sh, 0)->ans[r.par];
      *t = lead.t;
      *ties = lead.ties;
      state = lead.bad;
      r.sync();  // all have read it
      if (threadIdx.x == 0) sh.ans[r.par].bad = 0;
    } else {
      // one value, or many: by halves of the keys between
      auto inside = [&](uint32_t k) {
        Part p;
        r.each_if([&](float z) { return z >= z2 && key_of(z) > k; }, [&](float z) {
          if (z >= z2 && z <= z1 && key_of(z) > k) p.mass += weight(w, z);
        });
        return r.template join<P_MASS>(p).mass;
      };
      uint32_t key = q.hi;
      uint64_t ahead = 0;
      if (q.lo != q.hi) {
        key = first_key<T>(q.lo, q.hi, [&](uint32_t k) { return inside(k) < rest; });
        ahead = inside(key);
      }
      const uint64_t each = max(static_cast<uint64_t>(1), weight(w, float_of(key)));
      const uint64_t n = (rest - ahead + each - 1) / each, over = n * each - (rest - ahead);
      *t = key;
      *ties = static_cast<uint32_t>(n);
      state = n > q.count ? 0 : E && (over <= 2 * E || each - over <= 2 * E) ? -1 : 1;
    }
  }
  *turn = r.turn;
  return state;
}

// The logits among which the top-p cut falls, from a histogram of the masses by
// bins of 1/32 of a binary order, into sh.z1 and sh.z2.
template <typename T, bool ONE>
__device__ __noinline__ int find_cut(Row<T, ONE> r, float mass) {
  Shared& sh = r.sh;
  const Weigher w = sh.w;
  const int lane = r.lane;
  const float floor_z = sh.floor_z;
  for (int i = threadIdx.x; i < kBins; i += r.nt) sh.hist[i] = 0;
  __syncthreads();
  // Tokens lighter than (1 - p) mass / V sum to less than (1 - p) mass.
  const float least = log2f(fmaxf(0.5f * (1.f - sh.top_p) * mass / static_cast<float>(r.V), 1e-30f));
  const float y_cut = fmaxf(least - 0.0625f, kCut);
  const int b_cut = min(Row<T, ONE>::bin_of(fminf(y_cut, 0.f)), kBins - 1);
  r.each_if([&](float z) { return fast_y(w, z) >= y_cut && z >= floor_z; }, [&](float z) {
    const float y = fast_y(w, z);
    if (y >= y_cut && z >= floor_z) {
      const int b = min(Row<T, ONE>::bin_of(y), kBins - 1);
      // the weight over the bin's own: 13 bits or more
      atomicAdd(&sh.hist[b], __float2uint_rn(ex2_approx(y + 0.03125f * b + r.hist_bits)));
    }
  });
  r.sync();
  // Running sums: this CTA adds up its share of the bins over the slices, five bins
  // a thread or fewer.
  const int share = (b_cut + r.C) / r.C, per = (share + r.nt - 1) / r.nt;
  const int first = r.rank * share;
  float m[5], n_m = 0.f;
#pragma unroll
  for (int i = 0; i < 5; ++i) {
    const int j = static_cast<int>(threadIdx.x) * per + i, b = first + j;
    m[i] = 0.f;
    if (i < per && j < share && b <= b_cut) {
      uint64_t mm = 0;
      for (int c = 0; c < r.C; ++c) mm += r.of_rank(sh.hist, c)[b];
      m[i] = static_cast<float>(mm) * ex2_approx(-r.hist_bits - 0.03125f * b);
    }
    n_m += m[i];
  }
  float m_at = n_m;  // inclusive over the warp, then with what is ahead of it
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const float x = __shfl_up_sync(0xffffffffu, m_at, o);
    if (lane >= o) m_at += x;
  }
  Part q, ahead;
  q.sum = n_m;
  r.template join<P_SUM>(q, nullptr, &ahead);
  m_at += ahead.sum - n_m;
  // the masses here are 2^-14 off for their 13 bits, and 2^-20 for the rest
  const float need = sh.top_p * mass;
  q.lo = kBins - 1;  // the first bin that may reach the mass, and that does
  uint32_t does = kBins - 1;
#pragma unroll
  for (int i = 0; i < 5; ++i) {
    const int j = static_cast<int>(threadIdx.x) * per + i;
    m_at += m[i];
    if (i >= per || j >= share || first + j > b_cut) continue;
    const uint32_t b = first + j;
    if (m_at * (1.f + 8e-5f) >= need) q.lo = min(q.lo, b);
    if (m_at * (1.f - 8e-5f) > need) does = min(does, b);
  }
  q.hi = kBins - 1 - does;  // (a minimum as a maximum)
  q = r.template join<P_LO | P_HI>(q);
  const int b1 = static_cast<int>(q.lo), b2 = static_cast<int>(kBins - 1 - q.hi);
  if (threadIdx.x == 0) {
    // the bins' edges, a little apart for their rounding
    const float step = 0.03125f * kLn2 * sh.temp;
    const float e1 = w.zmax - b1 * step, e2 = w.zmax - (b2 + 1) * step;
    sh.z1 = e1 + (fabsf(e1) + fabsf(w.zmax)) * 4e-7f;
    sh.z2 = b2 == kBins - 1 ? -3.4e38f : e2 - (fabsf(e2) + fabsf(w.zmax)) * 4e-7f;
    sh.z2 = fmaxf(sh.z2, floor_z);
    sh.found = 1;
  }
  __syncthreads();
  return r.turn;
}

// One row with one way of weighing. `from`: at least the k first tokens (a first
// guess of them, with top-p alone; all, with min-p and no top-k) are logits from it
// on; `listing`: they are few. Returns whether the token is decided; with EXACT it
// always is. Every thread of the cluster returns the same.
template <typename T, bool ONE, bool EXACT>
__device__ __forceinline__ bool decide(Row<T, ONE>& r, const SampleArgs& a, int64_t row, uint32_t kmax,
                                    bool bins, bool listing, float from) {
  constexpr int VE = Vec<T>::N;
  Shared& sh = r.sh;
  if (EXACT) {
    if (threadIdx.x == 0) {
      sh.ans[r.par].bad = 0;
      sh.n_cand = 0;
    }
    __syncthreads();
    listing = listing && !sh.behind;
  }
  Weigher w = sh.w;
  w.zmax = float_of(kmax);
  const int lane = r.lane;
  const bool warm = sh.warm != 0, use_k = sh.top_k > 0, use_p = sh.use_p != 0;

  // ---- the mass of all tokens, and the list
  Part p;
  uint64_t my_above = 0;
  auto list = [&](const Vec<T>& x, int v) {
    if (listing && x.max() >= from) {
#pragma unroll
      for (int e = 0; e < VE; ++e) {
        const float z = x.get(e);
        if (z >= from && z > -INFINITY) {
          r.list(z, v, e);
          ++p.count;
          p.sum += ex2_approx(fast_y(w, z));
        }
      }
    }
  };
  if (EXACT) {
    const ulonglong2 m = exact_mass(r, w, -INFINITY, sh.found ? sh.z1 : INFINITY);
    p.mass = m.x;
    my_above = m.y;
    if (listing) r.pieces(list);
  } else {
    PairSum all;
    const uint64_t top = pair_of(-w.zmax), c_hi = pair_of(w.c_hi), c_lo = pair_of(w.c_lo);
    r.pieces([&](const Vec<T>& x, int v) {
      uint64_t s[VE / 2];
#pragma unroll
      for (int i = 0; i < VE / 2; ++i) s[i] = fast_weight2(x.pair(i), top, w.d_min, c_hi, c_lo);
#pragma unroll
      for (int o = 1; o < VE / 2; o <<= 1)
#pragma unroll
        for (int i = 0; i + o < VE / 2; i += 2 * o) s[i] = add2(s[i], s[i + o]);
      const float2 t = of_pair(s[0]);
      all.add(t.x + t.y);
      list(x, v);
    });
    p.mass = all.fixed(w.one);
  }
  Part mine, before;
  const Part S = r.template join<P_MASS | P_COUNT | P_SUM>(p, &mine, &before);
  const float floor_z = sh.floor_z;  // min-p keeps logits from here on (-inf: off)
  const uint64_t E = EXACT || !warm ? 0 : error_bound<T>(w, S.mass, r.V);
  const bool floored = sh.use_q && !use_k;  // the list is of all logits from min-p's floor on
  const bool listed = listing && S.count <= kCap;
  // the mass that the top-p cut is taken of
  uint64_t mass_q = S.mass;
  if (use_p && floored && !listed) {
    Part q;
    if (EXACT) {
      q.mass = exact_mass(r, w, nextafterf(floor_z, -INFINITY), INFINITY).x;
    } else {
      PairSum kept;
      r.each_if([&](float z) { return z >= floor_z; }, [&](float z) {
        if (z >= floor_z) kept.add(fast_weight(w, z));
      });
      q.mass = kept.fixed(w.one);
    }
    mass_q = r.template join<P_MASS>(q).mass;
  }
  const float mass_f = static_cast<float>(mass_q) / w.one;

  Kept keep;
  bool drawn = false, synced = false;  // the leader has the token; and all know it
  // ---- few candidates: the leader finishes the row with exact weights
  if (listed && (!warm || use_k || floored || S.sum > 0.9999f * sh.top_p * mass_f)) {
    if (r.rank == 0) draw_from_list<T, ONE>(r, S.count, warm, mass_q, 2 * E, floored, floored);
    drawn = true;
    if (warm && !use_k && !floored) {  // (the top-p cut may fall behind the list)
      r.sync();
      const int state = r.of_rank(&sh, 0)->ans[r.par].bad;
      if (state == L_CLOSE) return false;
      drawn = synced = state == L_DONE;
      if (!drawn) {
        r.sync();  // all have read it
        if (threadIdx.x == 0) sh.ans[r.par].bad = 0;
      }
    }
  }
  bool between = false;  // mine_a is this warp's mass above sh.z1, and the cut is below
  uint64_t mine_a = 0;
  if (drawn) {
  } else if (!warm) {
    keep.t = kmax;
    keep.ties = 1;
  } else if (use_k || use_p) {
    int state = 0;
    if (use_k) {
      // ---- many of top-k's: the smallest t with fewer than k keys above it
      if (!EXACT && (use_p || sh.use_q)) return false;
      const uint32_t k = static_cast<uint32_t>(sh.top_k);
      keep.t = first_key<T>(key_of(from), kmax, [&](uint32_t t) { return r.template above<false>(w, t).count < k; });
      keep.ties = k - r.template above<false>(w, keep.t).count;
      if (sh.use_q && key_of(floor_z) > keep.t) {
        keep.t = key_of(floor_z);
        keep.ties = 0xFFFFFFFFu;
      }
      state = !use_p;
    } else if (bins) {
      // ---- many of top-p's: the cut falls among the logits of a bin or two
      if (threadIdx.x == 0) sh.behind = 1;
      if (!EXACT) r.turn = find_cut<T, ONE>(r, mass_f);
      if (!EXACT || sh.found)
        state = cut_between<T, ONE, EXACT>(r, &r.turn, &keep.t, &keep.ties, &mine_a, my_above,
                                           mul_ceil(sh.top_p, mass_q), E);
      between = state == 1;
    }
    if (state != 1) {
      // ---- by halves of the key's range: any row, any number of ties
      if (!EXACT) return false;
      if (!use_k) keep = Kept();
      if (floored && key_of(floor_z) > keep.t) keep.t = key_of(floor_z);
      const uint32_t t = keep.t;
      const Part over = r.template above<true>(w, t);
      // t = 0 has no ties: no logit has key 0
      const uint32_t from_t = t == 0 ? over.count : r.template above<false>(w, t - 1).count;
      const uint64_t at = min(keep.ties, from_t - over.count);
      const uint64_t need = mul_ceil(sh.top_p, over.mass + (t == 0 ? 0 : at * weight(w, float_of(t))));
      // the smallest key with less than `need` above it
      const uint32_t key = first_key<T>(t, kmax, [&](uint32_t k) { return r.template above<true>(w, k).mass < need; });
      const uint64_t ahead = r.template above<true>(w, key).mass;
      const uint64_t each = weight(w, float_of(key));
      uint32_t more = 0xFFFFFFFFu;  // ties before which there is less than `need`
      if (ahead >= need) more = 1;  // p <= 0: the first token alone
      else if (each > 0)
        more = static_cast<uint32_t>(min((need - ahead + each - 1) / each, static_cast<uint64_t>(0xFFFFFFFFu)));
      keep.ties = key > t ? more : min(keep.ties, more);
      keep.t = key;
    }
  } else if (sh.use_q) {
    keep.t = key_of(floor_z);
  }

  if (!drawn) {
    // ---- the draw: the mass and ties ahead of each warp, then the one that holds u
    Part all = S;
    if (keep.t != 0) {
      Part q;
      if (between) {  // the warp's mass above z1 is known
        const float z1 = sh.z1;
        r.each_if([&](float z) { return key_of(z) >= keep.t; }, [&](float z) {
          const uint32_t key = key_of(z);
          if (key > keep.t && z <= z1) q.mass += weight(w, z);
          q.count += key == keep.t;
        });
        if (lane == 0) q.mass += mine_a;
      } else {
        PairSum f;
        r.each_if([&](float z) { return key_of(z) >= keep.t; }, [&](float z) {
          const uint32_t key = key_of(z);
          if (!EXACT && key > keep.t) f.add(fast_weight(w, z));
          q.count += key == keep.t;
        });
        q.mass = EXACT ? exact_mass(r, w, above_key(keep.t), INFINITY).x : f.fixed(w.one);
      }
      all = r.template join<P_MASS | P_COUNT>(q, &mine, &before);
    } else {
      all.count = mine.count = before.count = 0;
    }
    auto* lead = &r.of_rank(&sh, 0)->ans[r.par];
    const uint32_t lim = keep.ties;
    const uint64_t wt = keep.t == 0 ? 0 : weigh<EXACT>(w, float_of(keep.t));
    bool rest;
    const uint64_t target = mul_floor(sh.u, all.mass + min(all.count, lim) * wt, rest);
    auto holds = [&](uint64_t m, uint32_t e, uint64_t dm, uint32_t de) {
      return m + min(e, lim) * wt <= target && m + dm + min(e + de, lim) * wt > target;
    };
    // the warp that holds u (CTAs and warps are in index order), then the chunk of its
    // pieces: every warp of its CTA takes one
    if (threadIdx.x == 0) sh.b = -1;
    __syncthreads();
    if (holds(before.mass, before.count, mine.mass, mine.count) && lane == 0) {
      sh.b = r.warp;
      sh.base = before.mass;
      sh.base_ties = before.count;
      if (!EXACT) lead->bad = 1;  // until the token is found
    }
    __syncthreads();
    if (sh.b >= 0) {
      // the mass and ties of a lane's piece
      auto piece = [&](int v, uint64_t& s, uint32_t& eq) {
        const Vec<T> x = r.load(v);
        if (keep.t != 0 && !(key_of(x.max()) >= keep.t)) return;
        float f = 0.f;
#pragma unroll 2
        for (int i = 0; i < VE / 2; ++i) {
          const float2 z = of_pair(x.pair(i));
          const uint32_t k0 = key_of(clean(z.x)), k1 = key_of(clean(z.y));
          if (EXACT) {
            uint64_t w0, w1;
            weight2(w, x.pair(i), w0, w1);
            s += (k0 > keep.t ? w0 : 0) + (k1 > keep.t ? w1 : 0);
          } else {
            f += (k0 > keep.t ? fast_weight(w, z.x) : 0.f) + (k1 > keep.t ? fast_weight(w, z.y) : 0.f);
          }
          eq += (k0 == keep.t) + (k1 == keep.t);
        }
        if (!EXACT) s += static_cast<uint64_t>(__float2ll_rn(f * w.one));
      };
      const int per = (r.n_vec + r.nw - 1) / r.nw, v0 = min(r.n_vec, sh.b * per), v1 = min(r.n_vec, v0 + per);
      const int chunk = (per + r.nw - 1) / r.nw;
      const int c0 = min(v1, v0 + r.warp * chunk), c1 = min(v1, c0 + chunk);
      uint64_t s = 0;
      uint32_t eq = 0;
#pragma unroll 1
      for (int v = c0 + lane; v < c1; v += 32) piece(v, s, eq);
      s = warp_sum(s);
      eq = __reduce_add_sync(0xffffffffu, eq);
      if (lane == 0) {
        sh.chunk[r.warp] = s;
        sh.chunk_ties[r.warp] = eq;
      }
      __syncthreads();
      uint64_t m = sh.base;
      uint32_t e = sh.base_ties;
      for (int i = 0; i < r.warp; ++i) {
        m += sh.chunk[i];
        e += sh.chunk_ties[i];
      }
      if (holds(m, e, s, eq)) {
        for (int vb = c0; vb < c1; vb += 32) {
          const int v = vb + lane;
          uint64_t s1 = 0;
          uint32_t e1 = 0;
          if (v < c1) piece(v, s1, e1);
          const uint64_t s_in = m + warp_scan(s1, lane);
          uint32_t e_in = e1;
#pragma unroll
          for (int o = 1; o < 32; o <<= 1) {
            const uint32_t y = __shfl_up_sync(0xffffffffu, e_in, o);
            if (lane >= o) e_in += y;
          }
          e_in += e;
          const uint32_t hit = __ballot_sync(0xffffffffu, s_in + min(e_in, lim) * wt > target);
          if (hit) {
            if (lane == __ffs(hit) - 1) {
              const Vec<T> x = r.load(v);
              uint64_t sm = s_in - s1;
              uint32_t se = e_in - e1;
              int at = 0;  // the piece's last token that stays, up to the one that passes u
#pragma unroll 1
              for (int i = 0; i < VE; ++i) {
                const float z = x.get(i);
                const uint32_t key = key_of(z);
                const uint64_t was = sm + min(se, lim) * wt;
                if (key > keep.t) sm += weigh<EXACT>(w, z);
                se += key == keep.t;
                const uint64_t now = sm + min(se, lim) * wt;
                if (now > was) at = i;
                if (now > target) {
                  // a border within E of u is left to the exact weights (as is a
                  // token that the float sums of pieces and of elements disagree on)
                  if (!EXACT && (!E || (now - target > 2 * E && distance(target, was) > 2 * E))) lead->bad = 0;
                  break;
                }
              }
              lead->t = static_cast<uint32_t>(r.pos0 + static_cast<int64_t>(v) * VE + at);
            }
            break;
          }
          m = __shfl_sync(0xffffffffu, s_in, 31);
          e = __shfl_sync(0xffffffffu, e_in, 31);
        }
      }
    }
  }
  if (!synced) {
    r.sync();
    if (!EXACT && r.of_rank(&sh, 0)->ans[r.par].bad) return false;
  }
  if (r.rank == 0 && threadIdx.x == 0) write_row(a, row, r.row, sh, w, S.mass, r.par);
  return true;
}

// The smallest float z with exp((z - zmax) / T) >= q, for 2^-40 <= q < 1.
__device__ __noinline__ float min_logit(Weigher w, float temp, float q) {
  // log2(q) = y + yl: what 2^y misses of q, relative to q, times log2(e)
  const float y = fminf(log2f(q), 0.f);
  int n;
  float h, hl;
  exp2_pair(w.tab, y, 0.f, n, h, hl);
  const float qs = q * __uint_as_float(static_cast<uint32_t>(127 - n) << 23);
  const float yl = __fsub_rn(__fsub_rn(qs, h), hl) / h * kLog2e;
  // zmax + (y + yl) T ln 2, rounded up
  const float t = __fmul_rn(temp, kLn2), tl = __fmaf_rn(temp, kLn2, -t) + temp * kLn2Lo;
  const float p = __fmul_rn(y, t), pl = __fmaf_rn(y, t, -p) + __fmaf_rn(y, tl, yl * t);
  const float s = __fadd_rn(w.zmax, p), b = __fsub_rn(s, w.zmax);
  const float sl = __fadd_rn(__fadd_rn(__fsub_rn(w.zmax, __fsub_rn(s, b)), __fsub_rn(p, b)), pl);
  if (!(fabsf(s) < INFINITY) || !(fabsf(sl) < INFINITY)) return s;
  const float f = __fadd_rn(s, sl);
  return __fsub_rn(sl, __fsub_rn(f, s)) > 0.f ? nextafterf(f, INFINITY) : f;
}

// The rare way, apart from the common one's registers.
template <typename T, bool ONE>
__device__ __noinline__ int decide_exact(Row<T, ONE> r, const SampleArgs& a, int64_t row, uint32_t kmax,
                                         bool bins, bool listing, float from) {
  decide<T, ONE, true>(r, a, row, kmax, bins, listing, from);
  return r.turn;
}

// (four CTAs of 256 threads on an SM, or one of 512; rest: the marked rows only)
template <typename T, int THREADS, bool ONE>
__global__ void __launch_bounds__(THREADS, THREADS == 256 ? 4 : 1)
    k_sample(const __grid_constant__ SampleArgs a, int slice_vecs, int resident, int rest) {
  extern __shared__ uint4 s_slice[];
  __shared__ Shared sh;
  constexpr int VE = Vec<T>::N;
  Row<T, ONE> r(sh);
  r.lane = threadIdx.x & 31;
  r.warp = threadIdx.x >> 5;
  r.nt = blockDim.x;
  r.nw = blockDim.x >> 5;
  r.C = ONE ? 1 : static_cast<int>(r.cl.num_blocks());
  r.rank = ONE ? 0 : static_cast<int>(r.cl.block_rank());
  r.V = a.V;
  if (slice_vecs * VE < 131072) r.hist_bits = 15.f;  // (of 2^13, kMaxFast stay below 2^32)
  r.parts = reinterpret_cast<Part*>(s_slice + (resident ? slice_vecs : 0));
  if (threadIdx.x < 32) sh.tab[threadIdx.x] = c_exp2_32[threadIdx.x];
  const int n_cl = gridDim.x / r.C;
  for (int64_t row = blockIdx.x / r.C; row < a.rows; row += n_cl) {
    const int32_t mark = rest ? a.tokens[row] : kUndecided;
    if (mark > kUndecided) continue;
    r.place(a, row, slice_vecs, resident ? s_slice : nullptr);
    const float prm_t = a.temperature ? __ldg(a.temperature + row) : 1.f;
    const float prm_p = a.top_p ? __ldg(a.top_p + row) : 1.f;
    const int prm_k = a.top_k ? __ldg(a.top_k + row) : 0;
    const float prm_q = a.min_p ? __ldg(a.min_p + row) : 0.f;
    const float prm_u = threadIdx.x == 0 ? a.u[row] : 0.f;

    const float mx = r.copy_in();
    // weights below 2^-40 are 0: a lower q keeps every token that counts
    const bool use_q = prm_q >= 9.094947e-13f && prm_t > 0.f;
    if (threadIdx.x == 0) {
      sh.ans[r.par].bad = 0;
      set_row(sh, prm_t, prm_k, prm_p, use_q, prm_u, a.V);
    }
    __syncwarp();
    // A list of candidates is made where few tokens can stay: the one of a greedy
    // row, top-k's, those from min-p's floor on, and with top-p alone a first guess.
    // The k largest of the warps' maxima, or with larger k the warps' own j-th largest
    // lane maxima, are k logits of the row at least: candidates lie from the smallest
    // of them on.
    const bool has_k = prm_k > 0 && prm_k < a.V, floored = use_q && !has_k;
    const int kk = !(prm_t > 0.f) ? 1 : has_k ? prm_k : prm_p < 1.f ? kGuess : 0;
    const int n_warps = r.C * r.nw, j = (kk + n_warps - 1) / n_warps;
    const bool listing = floored || (kk > 0 && kk <= kCap / 2 && j <= 32);
    Part p;
    p.hi = key_of(mx);
    if (!floored && j > 1 && j <= 32) {
      const uint32_t mine[1] = {p.hi};
      p.lo = kth_from_below<1>(mine, j);
    }
    const Part tops = r.template join<P_HI | P_LO>(p);
    const uint32_t kmax = tops.hi;
    float from = -INFINITY;
    if (kk > 0 && !floored && j <= 32) {
      uint32_t key = kk == 1 ? kmax : tops.lo;
      if (kk > 1 && j == 1) {
        const Part* slots = r.parts + (r.turn ^ 1) * r.C * r.nw;  // that join's
        uint32_t top[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) top[i] = r.lane + 32 * i < n_warps ? slots[r.lane + 32 * i].hi : 0;
        key = kth_from_below<4>(top, kk);
      }
      from = float_of(max(key, key_of(-INFINITY)));
    }
    const float zmax = float_of(kmax);
    if (zmax == -INFINITY) {  // nothing to choose from
      if (r.rank == 0 && threadIdx.x == 0) {
        a.tokens[row] = -1;
        a.logp[row] = -INFINITY;
      }
      continue;
    }
    if (threadIdx.x == 0) {  // (read behind the next join)
      sh.w.zmax = zmax;
      sh.floor_z = !use_q ? -INFINITY : prm_q >= 1.f ? zmax : min_logit(sh.w, sh.temp, prm_q);
    }
    if (floored) {
      __syncthreads();
      from = sh.floor_z;
    }
    // (a T near 0 or infinity is the exact way's)
    const bool fast = zmax < INFINITY && slice_vecs * VE <= kMaxFast && sh.w.c_hi > 1e-30f && sh.w.c_hi < 1e30f;
    if (mark == kClose || !fast || !decide<T, ONE, false>(r, a, row, kmax, true, listing, from)) {
      r.sync();  // (a row's CTAs leave it at the same point where it was not decided)
      r.turn = decide_exact<T, ONE>(r, a, row, kmax, fast, listing, from);
    }
    r.par ^= 1;
  }
  r.sync();  // no CTA leaves while another may read its shared memory
}

// Many rows: a CTA takes a row and reads it once for the maximum and the mass (each
// lane weighs against the largest logit it has seen, and scales its sum down when a
// larger one comes). On the way it notes the pieces that may hold candidates, from a
// bound that rises as the row is read; only the row's first steps are read again. Greedy,
// top-k, min-p and plain softmax rows end here, and top-p rows whose cut is within the
// list; what is left is marked for a second launch. 512 greedy rows of 201088 take 66 us,
// with a second pass for the candidates 85. The masses are of rough weights: with the
// fast ones, which leave fewer rows, that was 118, and as many plain rows took 163 for
// 133 (spread-out logits) and 244 for 238 (flat).
constexpr int kRowThreads = 256;
constexpr int kFirstSteps = 4;  // a power of two
template <typename T>
__global__ void __launch_bounds__(kRowThreads, 1024 / kRowThreads) k_sample_rows(const __grid_constant__ SampleArgs a) {
  __shared__ Shared sh;
  __shared__ Part s_parts[2 * (kRowThreads / 32)];
  __shared__ uint32_t s_hits;
  __shared__ int s_hit[kCap];
  __shared__ volatile uint32_t s_low[kRowThreads / 32];
  constexpr int VE = Vec<T>::N;
  Row<T, true> r(sh);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  r.lane = lane;
  r.warp = warp;
  r.nt = kRowThreads;
  r.nw = kRowThreads / 32;
  r.C = 1;
  r.rank = 0;
  r.V = a.V;
  r.parts = s_parts;
  r.slice = nullptr;
  const int64_t row = blockIdx.x;
  const T* z = static_cast<const T*>(a.logits) + row * a.ld;
  const int off = static_cast<int>((reinterpret_cast<uintptr_t>(z) & 15) / sizeof(T));
  r.n_vec = static_cast<int>((off + a.V + VE - 1) / VE);
  r.pos0 = -off;
  const int per = (r.n_vec + r.nw - 1) / r.nw;
  r.v0 = min(r.n_vec, warp * per);
  r.v1 = min(r.n_vec, r.v0 + per);
  r.full0 = off ? 1 : 0;
  r.full1 = static_cast<int>((a.V + off) / VE);
  r.row = z;
  r.global = reinterpret_cast<const uint4*>(z - off);

  const float prm_t = a.temperature ? __ldg(a.temperature + row) : 1.f;
  const float prm_p = a.top_p ? __ldg(a.top_p + row) : 1.f;
  const float prm_q = a.min_p ? __ldg(a.min_p + row) : 0.f;
  const int prm_k = a.top_k ? __ldg(a.top_k + row) : 0;
  const bool warm = prm_t > 0.f, use_q = prm_q >= 9.094947e-13f && warm, has_k = prm_k > 0 && prm_k < a.V;
  const bool floored = use_q && !has_k;
  const int kk = !warm ? 1 : has_k ? prm_k : prm_p < 1.f ? kGuess : 0;
  const int j = (kk + r.nw - 1) / r.nw;
  const bool listing = floored || (kk > 0 && kk <= kCap / 2 && j <= 32);
  if (kk > 0 && !listing) {  // too many candidates for a list
    if (threadIdx.x == 0) a.tokens[row] = kUndecided;
    return;
  }
  if (threadIdx.x < 32) sh.tab[threadIdx.x] = c_exp2_32[threadIdx.x];
  if (threadIdx.x == 0) s_hits = 0;
  if (threadIdx.x == 0) set_row(sh, prm_t, prm_k, prm_p, use_q, a.u[row], a.V);

  __syncthreads();
  // ---- the maximum and the mass
  Weigher w = sh.w;
  float mx = -INFINITY, err = 0.f;  // err: what the scalings rounded, in units of 2^-24
  PairSum all;
  // (what needs the better weights to end here: float32 rows without a cut-off)
  const bool rough = sizeof(T) == 2 || kk > 0;
  // What the list will be taken from is known at the end only, but a bound from below is
  // known on the way: of the pieces from the fifth step on, those that reach it are noted.
  float low = INFINITY;
  const float to_floor = floored ? fminf(log2f(prm_q), 0.f) * kLn2 * prm_t : 0.f;
  auto pass = [&](auto is_rough) {
    constexpr bool ROUGH = decltype(is_rough)::value;
    const uint64_t c_hi = pair_of(w.c_hi), c_lo = pair_of(w.c_lo);
    const int steps = (per + 127) / 128;  // the same for every warp
    for (int step = 0; step < steps; ++step) {
      const int vb = r.v0 + 128 * step + lane;
      if (listing && step >= kFirstSteps && (step & (step - 1)) == 0) {
        if (floored) {
          const float top = float_of(__reduce_max_sync(0xffffffffu, key_of(mx)));
          low = top + to_floor - (fabsf(top) + fabsf(to_floor)) * 1e-5f;
          if (!(low > -INFINITY)) low = -INFINITY;
        } else {
          const uint32_t mine[1] = {key_of(mx)};
          uint32_t key = kth_from_below<1>(mine, j);
          if (kk > 1) {  // the least of the warps' bounds (later, of what they had when this one looks)
            if (lane == 0) s_low[warp] = key;
            if (step == kFirstSteps) __syncthreads();
            key = __reduce_min_sync(0xffffffffu, s_low[lane % (kRowThreads / 32)]);
          }
          low = float_of(max(key, key_of(-INFINITY)));
        }
      }
      Vec<T> x[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) x[i].raw = make_uint4(0, 0, 0, 0);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (vb + 32 * i < r.v1) x[i] = r.fetch(vb + 32 * i);
      float m = -INFINITY;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (vb + 32 * i < r.v1) m = fmaxf(m, x[i].max());
      if (m >= low) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (vb + 32 * i < r.v1 && x[i].max() >= low) {
            const uint32_t at = atomicAdd(&s_hits, 1u);
            if (at < kCap) s_hit[at] = vb + 32 * i;
          }
      }
      if (m > mx) {
        w.zmax = m;
        const float f = mx > -INFINITY ? fast_weight(w, mx) : 0.f;
        err = (err + 4.f * all.hi) * f;
        all.hi *= f;
        all.lo *= f;
        mx = m;
      }
      const uint64_t top = pair_of(-mx);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (vb + 32 * i < r.v1 && mx > -INFINITY) {
          uint64_t s[VE / 2];
#pragma unroll
          for (int k = 0; k < VE / 2; ++k)
            s[k] = ROUGH ? rough_weight2(x[i].pair(k), top, c_hi) : fast_weight2(x[i].pair(k), top, w.d_min, c_hi, c_lo);
#pragma unroll
          for (int o = 1; o < VE / 2; o <<= 1)
#pragma unroll
            for (int k = 0; k + o < VE / 2; k += 2 * o) s[k] = add2(s[k], s[k + o]);
          const float2 u = of_pair(s[0]);
          all.add(u.x + u.y);
        }
      }
    }
  };
  if (rough) pass(std::true_type());
  else if constexpr (sizeof(T) == 4) pass(std::false_type());
  Part p;
  p.hi = key_of(mx);
  if (listing && !floored && j > 1) {
    const uint32_t mine[1] = {p.hi};
    p.lo = kth_from_below<1>(mine, j);
  }
  const Part tops = r.template join<P_HI | P_LO>(p);
  const uint32_t kmax = tops.hi;
  const float zmax = float_of(kmax);
  if (zmax == -INFINITY) {  // nothing to choose from
    if (threadIdx.x == 0) {
      a.tokens[row] = -1;
      a.logp[row] = -INFINITY;
    }
    return;
  }
  float from = INFINITY;
  if (listing && !floored) {
    uint32_t key = kk == 1 ? kmax : tops.lo;
    if (kk > 1 && j == 1) {
      const uint32_t top[1] = {lane < r.nw ? s_parts[(r.turn ^ 1) * r.nw + lane].hi : 0};
      key = kth_from_below<1>(top, kk);
    }
    from = float_of(max(key, key_of(-INFINITY)));
  }
  if (threadIdx.x == 0) {  // (read behind the next barrier)
    sh.w.zmax = zmax;
    sh.floor_z = !use_q ? -INFINITY : prm_q >= 1.f ? zmax : min_logit(sh.w, sh.temp, prm_q);
  }
  if (floored) {
    __syncthreads();
    from = sh.floor_z;
  }
  bool decided = false;
  w.zmax = zmax;
  uint64_t mass = 0;
  if (zmax < INFINITY && w.c_hi > 1e-30f && w.c_hi < 1e30f) {
    Part q;
    if (mx > -INFINITY) {  // from the lane's largest logit to the row's
      const float f = fast_weight(w, mx);
      q.sum = (err + 4.f * all.hi) * f;
      all.hi *= f;
      all.lo *= f;
      q.mass = all.fixed(w.one);
    }
    // ---- the list: the pieces that may hold candidates, their tokens below; if too many
    // were noted, those that do
    if (listing) {
      const bool again = s_hits > kCap;
      __syncthreads();
      if (again) {
        if (threadIdx.x == 0) s_hits = 0;
        __syncthreads();
      }
      const int v1 = again ? r.v1 : min(r.v1, r.v0 + 128 * kFirstSteps);
      for (int vb = r.v0 + lane; vb < v1; vb += 256) {
        Vec<T> x[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (vb + 32 * i < v1) x[i] = r.fetch(vb + 32 * i);
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (vb + 32 * i < v1 && x[i].max() >= from) {
            const uint32_t at = atomicAdd(&s_hits, 1u);
            if (at < kCap) s_hit[at] = vb + 32 * i;
          }
      }
    }
    Part mine, before;
    const Part S = r.template join<P_MASS | P_SUM>(q, &mine, &before);
    mass = S.mass;
    bool fits = false;
    if (listing) {
      fits = s_hits <= kCap;
      for (uint32_t i = threadIdx.x; fits && i < s_hits; i += kRowThreads) {
        const int v = s_hit[i];
        const Vec<T> x = r.load(v);
#pragma unroll
        for (int e = 0; e < VE; ++e) {
          const float f = x.get(e);
          if (f >= from && f > -INFINITY) r.list(f, v, e);
        }
      }
      __syncthreads();
      fits = fits && sh.n_cand <= kCap;
      if (fits && warm && !has_k && !floored) {  // the top-p cut may fall behind the list
        Part l;
        for (uint32_t i = threadIdx.x; i < sh.n_cand; i += kRowThreads)
          l.sum += ex2_approx(fast_y(w, float_of(static_cast<uint32_t>(sh.cand[i] >> 32))));
        const float s = r.template join<P_SUM>(l).sum;
        fits = s > 0.9999f * sh.top_p * (static_cast<float>(mass) / w.one);
      }
    }
    const uint64_t E =
        warm ? error_bound<T>(w, S.mass, a.V, rough) + static_cast<uint64_t>(__float2ll_ru(S.sum * 6.0e-8f * w.one)) : 0;
    if (listing) {
      if (fits) {
        draw_from_list<T, true>(r, sh.n_cand, warm, S.mass, 2 * E, floored, floored);
        __syncthreads();
        decided = sh.ans[0].bad == L_DONE;
      }
    } else if (kk == 0) {
      // ---- the draw from all tokens: the warp that holds u, then the chunk of it
      // (every warp takes one), then the piece and the token
      bool rest;
      const uint64_t target = mul_floor(sh.u, S.mass, rest);
      if (threadIdx.x == 0) sh.ans[0].bad = L_CLOSE;
      if (before.mass <= target && before.mass + mine.mass > target && lane == 0) {
        sh.b = warp;
        sh.base = before.mass;
      }
      __syncthreads();
      const int v0 = min(r.n_vec, sh.b * per), v1 = min(r.n_vec, v0 + per);
      const int chunk = (per + 32 * r.nw - 1) / (32 * r.nw) * 32;  // pieces of a chunk: whole steps
      const int c0 = min(v1, v0 + warp * chunk), c1 = min(v1, c0 + chunk);
      auto piece = [&](int v) {
        const Vec<T> x = r.load(v);
        float f = 0.f;
#pragma unroll
        for (int e = 0; e < VE; ++e) f += fast_weight(w, x.get(e));
        return static_cast<uint64_t>(__float2ll_rn(f * w.one));
      };
      uint64_t m = 0;
      for (int v = c0 + lane; v < c1; v += 32) m += piece(v);
      m = warp_sum(m);
      if (lane == 0) sh.chunk[warp] = m;
      __syncthreads();
      uint64_t ahead = sh.base;
      for (int i = 0; i < warp; ++i) ahead += sh.chunk[i];
      if (ahead <= target && ahead + m > target) {
        for (int vb = c0; vb < c1; vb += 32) {
          const int v = vb + lane;
          const uint64_t s = v < c1 ? piece(v) : 0;
          const uint64_t upto = ahead + warp_scan(s, lane);
          const uint32_t hit = __ballot_sync(0xffffffffu, upto > target);
          if (hit) {
            if (lane == __ffs(hit) - 1) {
              const Vec<T> x = r.load(v);
              uint64_t at = upto - s;
              for (int e = 0; e < VE; ++e) {
                const uint64_t was = at;
                at += weigh<false>(w, x.get(e));
                if (at > target) {  // a border within E of u is left to the exact weights
                  if (at - target > 2 * E && distance(target, was) > 2 * E) {
                    sh.ans[0].t = static_cast<uint32_t>(r.pos0 + static_cast<int64_t>(v) * VE + e);
                    sh.ans[0].bad = L_DONE;
                  }
                  break;
                }
              }
            }
            break;
          }
          ahead = __shfl_sync(0xffffffffu, upto, 31);
        }
      }
      __syncthreads();
      decided = sh.ans[0].bad == L_DONE;
    }
  }
  if (threadIdx.x == 0) {
    if (decided) write_row(a, row, z, sh, w, mass);
    else a.tokens[row] = kk == 0 ? kClose : kUndecided;
  }
}

// bf16 logits have few values: those of 30 binary orders below the largest magnitude
// that weighs are 7679, and a row is its counts of them. From the counts every sum
// is exact (a count times a weight), so that a cut-off is a search in them and no
// draw has to be done again. A cluster takes a row: each CTA counts its slice in
// shared memory, and adds up a share of the counters over the cluster. The draw
// weighs each token that stays by its counter's place in a table of exact weights.
// A row that does not fit the counters (nonzero values more than 30 binary orders
// below) and T near 0 or infinity go through decide().
//
// One row of 128256 on 8 CTAs takes 30,000 cycles: 2,000 until the loads are out, 4,000
// for the counts, 6,000 for the weights, 2,000 to 2,600 for each join, 5,000 for the cut,
// 8,000 for the draw. With one CTA a row the two passes are most of it, 7 and 10
// cycles for 32 logits: the banks of shared memory, on which 32 values fall in 3 or
// 4 turns. (The draw's pass with the fast weights took as long: their 12
// instructions a logit.) Against lists, histograms of masses and the two ways of
// weighing, as float32 rows have them, one row with top-p took 15 us for 61, 61 rows
// with all cut-offs 33 for 37, and the rows that 512 mixed ones leave 50 for 330.
constexpr int kSide = 3840;           // values of one sign, 128 a binary order
constexpr int kCounts = 2 * kSide;    // in the order of descending logits; the last is for what weighs nothing
constexpr int kMostCounted = 200 * 1024;  // dynamic shared memory
constexpr int kUsual = 0x4300 - kSide;  // m0 for magnitudes below 2^7

// Magnitudes up to m0 share the counter of 0.
__device__ __forceinline__ uint32_t count_at(uint32_t bits, int m0) {
  const int m = max(static_cast<int>(bits & 0x7FFFu) - m0, 0);
  return min(static_cast<uint32_t>(kSide - 1 + ((bits & 0x8000u) ? m : -m)), static_cast<uint32_t>(kCounts - 1));
}
__device__ __forceinline__ float count_value(int i, int m0) {
  const int s = i - (kSide - 1);
  const uint32_t bits = s > 0 ? 0x8000u | static_cast<uint32_t>(s + m0) : static_cast<uint32_t>(m0 - s);
  return i == kCounts - 1 ? -INFINITY : s == 0 ? 0.f : __uint_as_float(bits << 16);
}

// The weights of the slice's own values in the counters ahead of `end` (this CTA's
// share of the counters has them).
__device__ __forceinline__ void fill_table(const Row<__nv_bfloat16, false>& r, const Weigher& w, int m0, int end,
                                           const uint32_t* counts, uint64_t* table) {
  const int share = kCounts / r.C;
  for (int i = 2 * threadIdx.x; i < end; i += 2 * r.nt) {
    const uint2 c = *reinterpret_cast<const uint2*>(counts + i);
    if ((c.x | c.y) && (i < r.rank * share || i >= (r.rank + 1) * share)) {
      uint64_t w0, w1;
      weight2(w, pair_of(__float_as_uint(count_value(i, m0)), __float_as_uint(count_value(i + 1, m0))), w0, w1);
      table[i] = w0;
      table[i + 1] = w1;
    }
  }
}

// The token that u falls on, of the counters ahead of `cut` and `ties` of its own,
// which weigh `kept`.
template <int U>
__device__ __forceinline__ void draw_counted(Row<__nv_bfloat16, false>& r, const SampleArgs& a, int64_t row, const Weigher& w,
                             uint32_t cut, uint32_t ties, uint64_t kept, uint64_t mass, int m0,
                             const uint64_t* table) {
  using T = __nv_bfloat16;
  constexpr int VE = Vec<T>::N;
  Shared& sh = r.sh;
  const int lane = r.lane;
  const float z_cut = count_value(cut, m0);
  const uint64_t w_cut = ties ? weight(w, z_cut) : 0;
  auto piece = [&](const Vec<T>& x, uint64_t& s, uint32_t& eq) {
    if (!(x.max() >= z_cut)) return;
#pragma unroll
    for (uint32_t b : {x.raw.x, x.raw.y, x.raw.z, x.raw.w}) {
      const uint32_t i = count_at(b, m0), j = count_at(b >> 16, m0);
      if (i < cut) s += table[i];
      if (j < cut) s += table[j];
      eq += (i == cut) + (j == cut);
    }
  };
  if (threadIdx.x == 0) sh.b = -1;
  // the mass and ties ahead of each warp, then the warp that holds u
  Part q, mine, before;
  r.template pieces<U>([&](const Vec<T>& x, int) { piece(x, q.mass, q.count); });
  r.template join<P_MASS | P_COUNT>(q, &mine, &before);
  bool left;
  const uint64_t target = mul_floor(sh.u, kept, left);
  auto upto = [&](uint64_t m, uint32_t e) { return m + min(e, ties) * w_cut; };
  auto holds = [&](uint64_t m, uint32_t e, uint64_t dm, uint32_t de) {
    return upto(m, e) <= target && upto(m + dm, e + de) > target;
  };
  if (holds(before.mass, before.count, mine.mass, mine.count) && lane == 0) {
    sh.b = r.warp;
    sh.base = before.mass;
    sh.base_ties = before.count;
  }
  __syncthreads();
  if (sh.b < 0) return;
  // the chunk of its pieces (every warp takes one), the piece and the token
  const int per = (r.n_vec + r.nw - 1) / r.nw, v0 = min(r.n_vec, sh.b * per), v1 = min(r.n_vec, v0 + per);
  const int chunk = (per + r.nw - 1) / r.nw;
  const int c0 = min(v1, v0 + r.warp * chunk), c1 = min(v1, c0 + chunk);
  Part c;
#pragma unroll 1
  for (int v = c0 + lane; v < c1; v += 32) piece(r.load(v), c.mass, c.count);
  r.template lanes<P_MASS | P_COUNT>(c);
  const uint64_t s = c.mass;
  const uint32_t eq = c.count;
  if (lane == 0) {
    sh.chunk[r.warp] = s;
    sh.chunk_ties[r.warp] = eq;
  }
  __syncthreads();
  uint64_t m = sh.base;
  uint32_t e = sh.base_ties;
  for (int i = 0; i < r.warp; ++i) {
    m += sh.chunk[i];
    e += sh.chunk_ties[i];
  }
  if (holds(m, e, s, eq)) {
    for (int vb = c0; vb < c1; vb += 32) {
      const int v = vb + lane;
      uint64_t s1 = 0;
      uint32_t e1 = 0;
      if (v < c1) piece(r.load(v), s1, e1);
      const uint64_t s_in = m + warp_scan(s1, lane);
      uint32_t e_in = e1;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t y = __shfl_up_sync(0xffffffffu, e_in, o);
        if (lane >= o) e_in += y;
      }
      e_in += e;
      const uint32_t hit = __ballot_sync(0xffffffffu, upto(s_in, e_in) > target);
      if (hit) {
        if (lane == __ffs(hit) - 1) {
          const Vec<T> x = r.load(v);
          uint64_t sm = s_in - s1;
          uint32_t se = e_in - e1;
#pragma unroll 1
          for (int i = 0; i < VE; ++i) {
            const uint32_t at = count_at(__float_as_uint(x.get(i)) >> 16, m0);
            if (at < cut) sm += table[at];
            se += at == cut;
            if (upto(sm, se) > target) {
              sh.ans[0].t = static_cast<uint32_t>(r.pos0 + static_cast<int64_t>(v) * VE + i);
              break;
            }
          }
          write_row(a, row, r.row, sh, w, mass);
        }
        break;
      }
      m = __shfl_sync(0xffffffffu, s_in, 31);
      e = __shfl_sync(0xffffffffu, e_in, 31);
    }
  }
}

// (rest: the marked rows only)
template <int THREADS>
__global__ void __launch_bounds__(THREADS, 1)
    k_sample_counts(const __grid_constant__ SampleArgs a, int slice_vecs, int resident, int rest) {
  using T = __nv_bfloat16;
  extern __shared__ uint4 s_slice[];
  __shared__ Shared sh;
  Row<T, false> r(sh);
  r.lane = threadIdx.x & 31;
  r.warp = threadIdx.x >> 5;
  r.nt = THREADS;
  r.nw = THREADS / 32;
  r.C = static_cast<int>(r.cl.num_blocks());
  r.rank = static_cast<int>(r.cl.block_rank());
  uint32_t* counts = reinterpret_cast<uint32_t*>(s_slice + (resident ? slice_vecs : 0));
  uint64_t* table = reinterpret_cast<uint64_t*>(counts + kCounts);
  uint32_t* joined = r.C == 1 ? counts : reinterpret_cast<uint32_t*>(table + kCounts);
  r.parts = reinterpret_cast<Part*>(reinterpret_cast<uint32_t*>(table + kCounts) + (r.C == 1 ? 0 : kSide));
  const int64_t row = blockIdx.x / r.C;
  if (rest && a.tokens[row] > kUndecided) return;
  if (threadIdx.x < 32) sh.tab[threadIdx.x] = c_exp2_32[threadIdx.x];
  r.place(a, row, slice_vecs, resident ? s_slice : nullptr);
  const int lane = r.lane;

  if (threadIdx.x == 0) {
    const float t = a.temperature ? __ldg(a.temperature + row) : 1.f, q = a.min_p ? __ldg(a.min_p + row) : 0.f;
    // weights below 2^-40 are 0: a lower q keeps every token that counts
    set_row(sh, t, a.top_k ? __ldg(a.top_k + row) : 0, a.top_p ? __ldg(a.top_p + row) : 1.f,
            q >= 9.094947e-13f && t > 0.f, a.u[row], a.V);
    sh.floor_z = q;
    sh.ans[0].bad = 0;
  }
  // ---- the counts, with the maximum, while the slice comes in: for the magnitudes
  // that logits have as a rule, and where these do not fit, once more for the row's own
  Part p;
  Weigher w;
  int m0 = kUsual;
  uint32_t kmax;
  bool good;
  for (int again = 0;; ++again) {
    for (int i = threadIdx.x; i < kCounts / 4; i += THREADS) reinterpret_cast<uint4*>(counts)[i] = make_uint4(0, 0, 0, 0);
    __syncthreads();
    float mx = -INFINITY;
    for (int vb = r.v0 + lane; vb < r.v1; vb += 32 * 8) {
      Vec<T> x[8];
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (vb + 32 * i < r.v1) x[i] = r.fetch(vb + 32 * i);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if (vb + 32 * i >= r.v1) continue;
        if (resident) s_slice[vb + 32 * i] = x[i].raw;
        mx = fmaxf(mx, x[i].max());
#pragma unroll
        for (uint32_t b : {x[i].raw.x, x[i].raw.y, x[i].raw.z, x[i].raw.w}) {
          const uint32_t j = count_at(b, m0), k = count_at(b >> 16, m0);
          if (j < kCounts - 1) atomicAdd(counts + j, 1u);
          if (k < kCounts - 1) atomicAdd(counts + k, 1u);
        }
      }
    }
    __syncthreads();
    p = Part();
    p.hi = key_of(mx);
    p.lo = 1;
    if (m0 > 0 && counts[kSide - 1]) {  // zeros, or values too small for a counter of their own?
      r.pieces([&](const Vec<T>& x, int) {
#pragma unroll
        for (uint32_t b : {x.raw.x, x.raw.y, x.raw.z, x.raw.w})
          for (int m : {static_cast<int>(b & 0x7FFFu), static_cast<int>((b >> 16) & 0x7FFFu)})
            if (m > 0 && m <= m0) p.lo = 0;
      });
    }
    p = r.template join<P_HI | P_LO>(p);
    kmax = p.hi;
    const float zmax = float_of(kmax);
    if (zmax == -INFINITY) {  // nothing to choose from
      if (r.rank == 0 && threadIdx.x == 0) {
        a.tokens[row] = -1;
        a.logp[row] = -INFINITY;
      }
      return;
    }
    w = sh.w;
    w.zmax = zmax;
    // (a T near 0 or infinity, and an infinite logit, are the other way's)
    good = zmax < INFINITY && w.c_hi > 1e-30f && w.c_hi < 1e30f;
    if (!good) break;
    const float z_lo = zmax - 41.f / w.c_hi;  // what lies below weighs nothing
    const int most = max(__float_as_uint(fabsf(zmax)) >> 16, (__float_as_uint(fabsf(z_lo)) >> 16) + 1);
    good = p.lo == 1 && most < m0 + kSide;
    if (good || again) break;
    m0 = max(min(most, 0x7F7F) - (kSide - 1), 0);
  }
  if (threadIdx.x == 0) {  // (read behind the next barrier)
    sh.w.zmax = w.zmax;
    const float q = sh.floor_z;
    sh.floor_z = !sh.use_q ? -INFINITY : q >= 1.f ? w.zmax : min_logit(sh.w, sh.temp, q);
  }
  p = Part();
  Part S, mine, before;
  if (good) {
    // ---- this CTA's share of the counters over the cluster, a warp a run of them
    const int share = kCounts / r.C, run = share / r.nw, first = r.rank * share + r.warp * run;
    for (int i = 2 * lane; i < run; i += 64) {
      const int b = first + i;
      uint2 c = *reinterpret_cast<const uint2*>(counts + b), o[kMaxCluster];
#pragma unroll
      for (int k = 1; k < kMaxCluster; ++k)
        o[k] = k < r.C ? *reinterpret_cast<const uint2*>(r.of_rank(counts, r.rank ^ k) + b) : make_uint2(0, 0);
#pragma unroll
      for (int k = 1; k < kMaxCluster; ++k) {
        c.x += o[k].x;
        c.y += o[k].y;
      }
      if (r.C > 1) *reinterpret_cast<uint2*>(joined + r.warp * run + i) = c;
      if (c.x | c.y) {
        uint64_t w0, w1;
        weight2(w, pair_of(__float_as_uint(count_value(b, m0)), __float_as_uint(count_value(b + 1, m0))), w0, w1);
        table[b] = w0;
        table[b + 1] = w1;
        p.mass += c.x * w0 + c.y * w1;
        p.count += c.x + c.y;
      }
    }
    // with a narrow cut to come, few of the table's weights are needed
    const bool narrow = sh.warm == 0 || sh.top_k > 0 || sh.use_q;
    if (!narrow) fill_table(r, w, m0, kCounts, counts, table);
    S = r.template join<P_MASS | P_COUNT>(p, &mine, &before);
    {
      // f(counter, its count, its weight, tokens and mass ahead of it), for this warp's counters
      auto each = [&](auto f) {
        uint32_t n = before.count;
        uint64_t m = before.mass;
        for (int i0 = 0; i0 < run; i0 += 32) {
          const int b = first + i0 + lane;
          const bool in = i0 + lane < run;
          const uint32_t c = in ? joined[b - (r.C > 1 ? r.rank * share : 0)] : 0;
          const uint64_t wt = c ? table[b] : 0;
          if (!__any_sync(0xffffffffu, c != 0)) {
            if (in) f(b, c, wt, n, m);
            continue;
          }
          uint32_t n_in = c;
#pragma unroll
          for (int o = 1; o < 32; o <<= 1) {
            const uint32_t y = __shfl_up_sync(0xffffffffu, n_in, o);
            if (lane >= o) n_in += y;
          }
          const uint64_t m_in = warp_scan(c * wt, lane);
          if (in) f(b, c, wt, n + n_in - c, m + m_in - c * wt);
          n += __shfl_sync(0xffffffffu, n_in, 31);
          m += __shfl_sync(0xffffffffu, m_in, 31);
        }
      };
      // ---- what stays: the counters ahead of `cut` and `ties` of its own, `kept` in all
      const bool warm = sh.warm != 0;
      uint32_t cut = kCounts - 1, ties = 0;
      uint64_t kept = S.mass;
      uint32_t stay = S.count;
      if (warm && sh.use_q) {
        const float floor_z = sh.floor_z;
        Part q;
        each([&](int b, uint32_t, uint64_t, uint32_t n, uint64_t m) {
          if (count_value(b, m0) < floor_z && (b == 0 || count_value(b - 1, m0) >= floor_z)) {
            q.lo = b;
            q.count = n;
            q.mass = m;
          }
        });
        q = r.template join<P_MASS | P_COUNT | P_LO>(q);
        if (q.lo < cut) {
          cut = q.lo;
          stay = q.count;
          kept = q.mass;
        }
      }
      const uint32_t k = !warm ? 1 : sh.top_k > 0 ? sh.top_k : 0xFFFFFFFFu;
      if (k < stay) {
        Part q;
        if (before.count <= k && before.count + mine.count > k)
          each([&](int b, uint32_t c, uint64_t wt, uint32_t n, uint64_t m) {
            if (n <= k && n + c > k) {
              q.lo = b;
              q.count = k - n;
              q.mass = m + (k - n) * wt;
            }
          });
        q = r.template join<P_MASS | P_COUNT | P_LO>(q);
        cut = q.lo;
        ties = q.count;
        kept = q.mass;
      }
      if (warm && sh.use_p) {
        const uint64_t want = max(mul_ceil(sh.top_p, kept), static_cast<uint64_t>(1));
        Part q;
        if (before.mass < want && before.mass + mine.mass >= want)
          each([&](int b, uint32_t c, uint64_t wt, uint32_t, uint64_t m) {
            if (m < want && m + c * wt >= want) {
              const uint32_t n = static_cast<uint32_t>((want - m + wt - 1) / wt);
              q.lo = b;
              q.count = n;
              q.mass = m + n * wt;
            }
          });
        q = r.template join<P_MASS | P_COUNT | P_LO>(q);
        cut = q.lo;
        ties = q.count;
        kept = q.mass;
      }
      if (narrow) {
        fill_table(r, w, m0, cut, counts, table);
        __syncthreads();
      }
      draw_counted<THREADS == 512 ? 8 : 4>(r, a, row, w, cut, ties, kept, S.mass, m0, table);
      return;  // (none reads or writes another's shared memory any more)
    }
  }
  decide_exact<T, false>(r, a, row, kmax, false, false, -INFINITY);
  r.sync();  // no CTA leaves while another may read its shared memory
}

template <int THREADS>
cudaError_t launch_counts(const SampleArgs& a, int C, int rest, cudaStream_t s) {
  auto kernel = k_sample_counts<THREADS>;
  // counts, weights, joined counts, and what is joined
  const int words = kCounts * 12 + (C == 1 ? 0 : kSide * 4) + 2 * C * (THREADS / 32) * static_cast<int>(sizeof(Part));
  static std::atomic<uint64_t> configured{0};  // one bit a device
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = 1ull << (dev & 63);
  if (!(configured.load() & bit)) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMostCounted);
    if (e != cudaSuccess) return e;
    configured.fetch_or(bit);
  }
  const int64_t slice = ((a.V + 7) / 8 + 1 + C - 1) / C;  // a row may start inside its first piece
  if (slice > INT32_MAX / 8) return cudaErrorInvalidValue;
  const bool resident = C > 1 && slice * 16 + words <= kMostCounted;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(a.rows * C));
  cfg.blockDim = dim3(THREADS);
  cfg.dynamicSmemBytes = static_cast<size_t>((resident ? slice * 16 : 0) + words);
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = C;
  at[0].val.clusterDim.y = 1;
  at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, a, static_cast<int>(slice), resident ? 1 : 0, rest);
}

template <typename T, int THREADS, bool ONE>
cudaError_t launch_with(const SampleArgs& a, int C, int most_clusters, int rest, cudaStream_t s) {
  constexpr int VE = 16 / static_cast<int>(sizeof(T));
  auto kernel = k_sample<T, THREADS, ONE>;
  constexpr int parts = 2 * (ONE ? 1 : kMaxCluster) * (THREADS / 32) * static_cast<int>(sizeof(Part));
  static std::atomic<uint64_t> configured{0};  // one bit a device
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = 1ull << (dev & 63);
  if (!(configured.load() & bit)) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSliceBytes + parts);
    if (e != cudaSuccess) return e;
    configured.fetch_or(bit);
  }
  const int64_t pieces = (a.V + VE - 1) / VE + 1;  // a row may start inside its first piece
  const int64_t slice = (pieces + C - 1) / C;
  if (slice > INT32_MAX / VE) return cudaErrorInvalidValue;
  // A slice stays in shared memory where four CTAs of 256 threads, or one of 512,
  // have room for theirs; else it is read again from L2.
  const bool resident = !ONE && slice * 16 <= (THREADS == 512 ? kMaxSliceBytes : kSliceBytes);
  cudaLaunchConfig_t cfg = {};
  const int64_t clusters = a.rows < most_clusters ? a.rows : most_clusters;
  cfg.gridDim = dim3(static_cast<unsigned>(clusters * C));
  cfg.blockDim = dim3(THREADS);
  cfg.dynamicSmemBytes = static_cast<size_t>(resident ? slice * 16 : 0) + parts;
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = C;
  at[0].val.clusterDim.y = 1;
  at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = ONE ? 0 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, a, static_cast<int>(slice), resident ? 1 : 0, rest);
}

template <typename T>
cudaError_t launch(const SampleArgs& a, int sms, cudaStream_t s) {
  const int64_t bytes = a.V * static_cast<int64_t>(sizeof(T));
  // Short rows: a CTA a row, which needs no cluster's barriers.
  if (bytes <= 16 * 1024) return launch_with<T, 256, true>(a, 1, 1 << 30, 0, s);
  // Rows enough for every SM: one CTA a row as well, and what that leaves, as a rule
  // top-p rows whose cut is behind the list, a second launch does.
  const bool many = a.rows >= sms && a.V <= kMaxFast;
  if (many) {
    k_sample_rows<T><<<static_cast<unsigned>(a.rows), kRowThreads, 0, s>>>(a);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  // Else as many CTAs a row as there are SMs for, each with 16 KB of it at least.
  if constexpr (sizeof(T) == 2) {
    int C = 1;
    while (!many && C < kMaxCluster && a.rows * C * 2 <= sms && bytes / C > 16 * 1024) C *= 2;
    return C == 1 ? launch_counts<1024>(a, C, many, s) : launch_counts<512>(a, C, many, s);
  } else {
    if (many) return launch_with<T, 256, false>(a, kMaxCluster, 4 * sms / kMaxCluster, 1, s);
    int C = 2;
    while (C < kMaxCluster && a.rows * C < sms && bytes / C > 16 * 1024) C *= 2;
    if (a.rows * C <= sms) return launch_with<T, 512, false>(a, C, 65536, 0, s);
    return launch_with<T, 256, false>(a, C, 65536, 0, s);
  }
}

}  // namespace

cudaError_t launch_sample(const SampleArgs& a, int sms, cudaStream_t s) {
  return a.bf16 ? launch<__nv_bfloat16>(a, sms, s) : launch<float>(a, sms, s);
}

}  // namespace grpo
