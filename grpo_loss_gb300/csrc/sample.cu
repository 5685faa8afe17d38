// Token sampling with temperature, top-k, top-p and min-p from given uniforms.
//
// A row's weights w_i = exp((z_i - zmax) / T) are summed as integers of fixed
// point, W = w 2^B, so that sums do not depend on their order, and the token is
// the one that real numbers give: the draw compares u sum W with the running sum,
// and with 10^5 tokens of similar weight, sums of float32 weights (2^-22 off, or
// so) would pick a neighbour in one draw of ten. Two ways of weighing share one
// body. The fast one takes 2^y from the special-function unit and carries a bound
// E on the error of its sums; where the draw or the top-p cut falls within E of a
// border, the row is done again with weights from pairs of floats (2^-43), whose
// integer sums decide. A trained model's rows (a few likely tokens) seldom need
// that; flat rows always do.
//
// All three cut-offs keep a prefix of the order (logit descending, index
// ascending): what is kept is a threshold t on the logit's sort key and a number
// of ties at t, the first in index order.
//
// A cluster of CTAs takes a row, each CTA one slice of it that it copies into
// shared memory once (a row of 128K bf16 logits is 250 KB: more than one SM
// holds). Every later question (maximum, sums, histogram, draw) reads shared
// memory and is joined over the cluster through distributed shared memory, so
// the logits cross HBM once and a row needs one launch.
#include <cooperative_groups.h>
#include <cuda_bf16.h>

#include <atomic>

#include "internal.h"
#include "ptx.cuh"

namespace cg = cooperative_groups;

namespace grpo {

namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCluster = 8;                 // the portable cluster size
constexpr int kBins = 1280;                    // 1/32 of a binary order each, down to 2^-40
constexpr int kCap = 1024;                     // candidates that one CTA sorts
constexpr int kMaxSliceBytes = 184 * 1024;     // of a row's slice kept in shared memory
constexpr float kCut = -40.f;                  // binary orders below the top that weigh nothing

// 2^(j/32), j = 0..31, each as the sum of two floats.
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

// A 16-byte piece of a row.
template <typename T>
struct Vec {
  static constexpr int N = 16 / sizeof(T);
  uint4 raw;
  __device__ __forceinline__ float get(int e) const;
};
template <>
__device__ __forceinline__ float Vec<float>::get(int e) const {
  return clean(__uint_as_float(e == 0 ? raw.x : e == 1 ? raw.y : e == 2 ? raw.z : raw.w));
}
template <>
__device__ __forceinline__ float Vec<__nv_bfloat16>::get(int e) const {
  const uint32_t w = e < 2 ? raw.x : e < 4 ? raw.y : e < 6 ? raw.z : raw.w;
  return clean(__uint_as_float((e & 1) ? (w & 0xFFFF0000u) : (w << 16)));
}

// What turns a logit into its weight: y = (z - zmax) log2(e) / T as a pair of
// floats, scaled by 2^B.
struct Weigher {
  float zmax, c_hi, c_lo, one;  // one = 2^B
  const float2* tab;
};

// W = round(2^(y + B)), 0 below y = -40. The argument error is 2^-46 |y|.
__device__ __forceinline__ uint64_t weight(const Weigher& w, float z) {
  if (z == w.zmax) return static_cast<uint64_t>(__float2ll_rn(w.one));
  // z - zmax without loss: the difference and what its rounding left
  const float d = z - w.zmax;
  const float bb = d - z;
  const float dl = (z - (d - bb)) + (-w.zmax - bb);
  const float p = d * w.c_hi;
  if (!(p >= -40.5f)) return 0;
  const float pl = __fmaf_rn(d, w.c_hi, -p) + __fmaf_rn(d, w.c_lo, dl * w.c_hi);
  if (p + pl < -40.f || (p == -40.f && pl < 0.f)) return 0;
  // y = k / 32 + r, |r| <= 1/64
  const float kf = rintf(p * 32.f);
  const int k = static_cast<int>(kf);
  const float r0 = __fmaf_rn(kf, -0.03125f, p);
  const float r = r0 + pl, rl = pl - (r - r0);
  // s = 2^r - 1 = x + x^2/2 + x^3/6 + ..., x = r ln 2, the first two terms in pairs
  const float kLn2 = 0x1.62e4300000000p-1f, kLn2Lo = -0x1.05c6100000000p-29f;
  const float x = r * kLn2;
  const float xl = __fmaf_rn(r, kLn2, -x) + __fmaf_rn(r, kLn2Lo, rl * kLn2);
  const float xx = x * x;
  const float xxl = __fmaf_rn(x, x, -xx) + 2.f * x * xl;
  const float cubic =
      xx * x * __fmaf_rn(x, __fmaf_rn(x, __fmaf_rn(x, 1.f / 720.f, 1.f / 120.f), 1.f / 24.f), 1.f / 6.f);
  const float s = __fmaf_rn(xx, 0.5f, x);
  const float sl = __fmaf_rn(xx, 0.5f, x - s) + (xl + 0.5f * xxl + cubic);
  // 2^(k/32) (1 + s)
  const float2 t = w.tab[k & 31];
  const float q = t.x * s;
  const float ql = __fmaf_rn(t.x, s, -q) + __fmaf_rn(t.x, sl, t.y * s);
  const float h = t.x + q;
  const float hl = (q - (h - t.x)) + (ql + t.y);
  const float scale = w.one * __uint_as_float(static_cast<uint32_t>(127 + (k >> 5)) << 23);
  return static_cast<uint64_t>(__float2ll_rn(h * scale) +
                               static_cast<long long>(__float2int_rn(hl * scale)));
}


// The fast weight's y = (z - zmax) log2(e) / T (zmax finite). Its error is
// 3 * 2^-24 |y| (three roundings), that of 2^y 2^-22: together
// w (4 + 2.1 |y|) 2^-24.
__device__ __forceinline__ float fast_y(const Weigher& w, float z) { return (z - w.zmax) * w.c_hi; }
__device__ __forceinline__ float fast_weight(float y) { return y < kCut ? 0.f : ex2_approx(y); }

// Element weight as an integer.
template <bool EXACT>
__device__ __forceinline__ uint64_t weigh(const Weigher& w, float z) {
  if (EXACT) return weight(w, z);
  return static_cast<uint64_t>(__float2ll_rn(fast_weight(fast_y(w, z)) * w.one));
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

// What one warp tells the cluster.
struct Part {
  uint64_t mass;
  uint64_t mass2;
  uint32_t count;
  uint32_t lo, hi;
  float err;
};

struct Shared {
  float2 tab[32];
  Part part[2][kWarps];          // alternating between joins
  uint32_t cnt[kBins];
  uint32_t mass[kBins];
  uint64_t cand[kCap];
  uint64_t wts[kCap];
  uint32_t n_cand;
  // leader's answers to the cluster
  uint32_t t, ties;
  int again, bad;
  // this CTA's scratch
  float scan_f[kWarps];
  uint32_t scan_u[kWarps];
  int b1, b2;
  uint32_t upto;
  Weigher w;
  float floor_z, top_p, u;
  int top_k, warm, use_p, use_q;
  double temp;
};

// One row, seen from one CTA.
template <typename T>
struct Row {
  static constexpr int VE = Vec<T>::N;
  cg::cluster_group cl = cg::this_cluster();
  Shared& sh;
  const uint4* slice;  // this CTA's slice in shared memory, or null: the logits are read again
  const uint4* global; // its first piece among the logits
  const T* row;
  int n_vec;           // 16-byte pieces of the slice
  int64_t pos0;        // row index of the slice's first element (may be below 0)
  int64_t V;
  int lane, warp, C, rank, turn = 0;
  int v0, v1;          // this warp's pieces

  __device__ __forceinline__ Row(Shared& s) : sh(s) {}

  // Piece v from global memory. The pieces at the row's ends hold other rows'
  // elements, or none: these are read one by one, with -inf in their place.
  __device__ __forceinline__ Vec<T> fetch(int v) const {
    Vec<T> x;
    const int64_t i0 = pos0 + static_cast<int64_t>(v) * VE;
    if (i0 >= 0 && i0 + VE <= V) {
      x.raw = __ldg(global + v);
    } else {
      uint32_t w[4];
      T* e = reinterpret_cast<T*>(w);
#pragma unroll
      for (int i = 0; i < VE; ++i)
        e[i] = i0 + i >= 0 && i0 + i < V ? row[i0 + i] : static_cast<T>(-INFINITY);
      x.raw = make_uint4(w[0], w[1], w[2], w[3]);
    }
    return x;
  }
  __device__ __forceinline__ Vec<T> load(int v) const {
    if (slice == nullptr) return fetch(v);
    Vec<T> x;
    x.raw = slice[v];
    return x;
  }

  // f(z) for this warp's elements; (step, lane, e) is their index order.
  template <typename F>
  __device__ __forceinline__ void each(F f) const {
    for (int v = v0 + lane; v < v1; v += 32) {
      const Vec<T> x = load(v);
#pragma unroll
      for (int e = 0; e < VE; ++e) f(x.get(e));
    }
  }

  // Joins one Part of each warp over the cluster; every thread gets the whole.
  __device__ __forceinline__ Part join(Part p) {
    p.mass = warp_sum(p.mass);
    p.mass2 = warp_sum(p.mass2);
    p.count = __reduce_add_sync(0xffffffffu, p.count);
    p.lo = __reduce_min_sync(0xffffffffu, p.lo);
    p.hi = __reduce_max_sync(0xffffffffu, p.hi);
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) p.err += __shfl_xor_sync(0xffffffffu, p.err, o);
    Part* mine = sh.part[turn];
    if (lane == 0) mine[warp] = p;
    cl.sync();
    Part q = {0, 0, 0, 0xFFFFFFFFu, 0, 0.f};
    for (int i = lane; i < C * kWarps; i += 32) {
      const Part o = cl.map_shared_rank(mine, i / kWarps)[i % kWarps];
      q.mass += o.mass;
      q.mass2 += o.mass2;
      q.count += o.count;
      q.lo = min(q.lo, o.lo);
      q.hi = max(q.hi, o.hi);
      q.err += o.err;
    }
    q.mass = warp_sum(q.mass);
    q.mass2 = warp_sum(q.mass2);
    q.count = __reduce_add_sync(0xffffffffu, q.count);
    q.lo = __reduce_min_sync(0xffffffffu, q.lo);
    q.hi = __reduce_max_sync(0xffffffffu, q.hi);
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) q.err += __shfl_xor_sync(0xffffffffu, q.err, o);
    turn ^= 1;
    return q;
  }

  // Number of tokens with key above k, and their mass.
  template <bool MASS>
  __device__ Part above(const Weigher& w, uint32_t k) {
    Part p = {0, 0, 0, 0xFFFFFFFFu, 0, 0.f};
    each([&](float z) {
      if (key_of(z) > k) {
        ++p.count;
        if (MASS) p.mass += weight(w, z);
      }
    });
    return join(p);
  }

  // Bin of a logit in steps of 1/32 of a binary order below the top.
  __device__ __forceinline__ static int bin_of(float y) { return static_cast<int>(-32.f * y); }

  // Copies the elements f accepts to the leader's list; returns their number
  // over the cluster (the list is cut at kCap).
  template <typename F>
  __device__ uint32_t gather(F accept) {
    uint32_t* n = cl.map_shared_rank(&sh.n_cand, 0);
    uint64_t* to = cl.map_shared_rank(sh.cand, 0);
    for (int vb = v0; vb < v1; vb += 32) {
      const int v = vb + lane;
      Vec<T> x;
      uint32_t want = 0;
      if (v < v1) {
        x = load(v);
#pragma unroll
        for (int e = 0; e < VE; ++e) want |= accept(x.get(e)) ? (1u << e) : 0u;
      }
      if (!__any_sync(0xffffffffu, want != 0)) continue;
      const uint32_t mine = __popc(want);
      uint32_t at = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t y = __shfl_up_sync(0xffffffffu, at, o);
        if (lane >= o) at += y;
      }
      uint32_t base = 0;
      if (lane == 31) base = atomicAdd(n, at);
      base = __shfl_sync(0xffffffffu, base, 31) + at - mine;
#pragma unroll
      for (int e = 0; e < VE; ++e) {
        if (want >> e & 1) {
          const uint32_t idx = static_cast<uint32_t>(pos0 + static_cast<int64_t>(v) * VE + e);
          if (base < kCap) to[base] = (static_cast<uint64_t>(key_of(x.get(e))) << 32) | ~idx;
          ++base;
        }
      }
    }
    cl.sync();
    return *n;
  }

  // Sorts the first n of a list in shared memory, largest first (one CTA).
  __device__ void sort_desc(uint64_t* a, uint32_t n) {
    uint32_t n2 = 2;
    while (n2 < n) n2 <<= 1;
    for (uint32_t i = n + threadIdx.x; i < n2; i += kThreads) a[i] = 0;
    __syncthreads();
    for (uint32_t k = 2; k <= n2; k <<= 1)
      for (uint32_t j = k >> 1; j > 0; j >>= 1) {
        for (uint32_t i = threadIdx.x; i < n2 / 2; i += kThreads) {
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

// Threshold and ties that a cut keeps, or the token itself.
struct Kept {
  uint32_t t = 0, ties = 0xFFFFFFFFu;
};

// One row with one way of weighing. Returns whether the token is decided; with
// EXACT it always is. Every thread of the cluster returns the same.
template <typename T, bool EXACT>
__device__ bool decide(Row<T>& r, const SampleArgs& a, int64_t row, uint32_t kmax, float my_max,
                       bool hist) {
  constexpr int VE = Vec<T>::N;
  Shared& sh = r.sh;
  const Weigher w = sh.w;
  const int lane = r.lane, warp = r.warp;
  const float floor_z = sh.floor_z;  // min-p keeps logits from here on (-inf: off)
  const bool warm = sh.warm != 0, use_k = sh.top_k > 0, use_p = sh.use_p != 0;

  // ---- the mass of all tokens, and of those that min-p keeps
  Part p = {0, 0, 0, 0xFFFFFFFFu, 0, 0.f};
  if (EXACT) {
    r.each([&](float z) {
      const uint64_t x = weight(w, z);
      p.mass += x;
      if (z >= floor_z) p.mass2 += x;
    });
  } else {
    PairSum all, kept;
    float e = 0.f;
    for (int v = r.v0 + lane; v < r.v1; v += 32) {
      const Vec<T> x = r.load(v);
      float s[VE], k[VE];
#pragma unroll
      for (int i = 0; i < VE; ++i) {
        const float z = x.get(i), y = fast_y(w, z);
        s[i] = fast_weight(y);
        e = fmaf(s[i], -fmaxf(y, kCut), e);
        k[i] = z >= floor_z ? s[i] : 0.f;
      }
#pragma unroll
      for (int o = 1; o < VE; o <<= 1)
#pragma unroll
        for (int i = 0; i + o < VE; i += 2 * o) {
          s[i] += s[i + o];
          k[i] += k[i + o];
        }
      all.add(s[0]);
      if (sh.use_q) kept.add(k[0]);
    }
    p.mass = all.fixed(w.one);
    p.mass2 = sh.use_q ? kept.fixed(w.one) : p.mass;
    // w (4 + 2.1 |y|) 2^-24, three more roundings in the sum of a piece, and
    // the slack of this bound's own sums
    p.err = (7.5f * all.hi + 2.2f * e) * 5.9604645e-8f;
  }
  // the warps' masses stay where they are for a draw without cut-offs
  const uint64_t warp_all = warp_sum(p.mass);
  const Part S = r.join(p);
  // bound on the error of any sum of weights, in units of W
  const double E = EXACT || !warm ? 0.0
                                  : static_cast<double>(S.err) * w.one * 1.01 + static_cast<double>(r.V) + 1024.0;

  Kept keep;
  int token = -1;         // decided by the leader alone
  bool leader_draws = false;
  if (!warm) {
    keep.t = kmax;
    keep.ties = 1;
  } else if (use_k || use_p) {
    // ---- candidates: every token that can stay has a bin of at most b_cut
    int b_cut = kBins - 1;
    bool listed = false;
    if (hist) {
      for (int i = threadIdx.x; i < kBins; i += kThreads) sh.cnt[i] = sh.mass[i] = 0;
      if (threadIdx.x == 0) sh.n_cand = 0;
      __syncthreads();
      const bool fits = w.zmax < INFINITY;
      if (use_k) {
        // The k-th largest of the threads' maxima is at most the k-th largest
        // logit: bins up to its own hold at least k tokens, and few more.
        const float y = fast_y(w, my_max);
        if (fits && y >= kCut) atomicAdd(&sh.cnt[min(Row<T>::bin_of(y), kBins - 1)], 1u);
      } else {
        // Tokens lighter than (1 - p) mass / V sum to less than (1 - p) mass.
        const float y = log2f(fmaxf(0.5f * (1.f - sh.top_p) * (static_cast<float>(S.mass2) / w.one) /
                                        static_cast<float>(r.V), 1e-30f));
        b_cut = y > kCut ? max(0, Row<T>::bin_of(fminf(y, 0.f))) : kBins - 1;
        b_cut = min(b_cut + 1, kBins - 1);
        r.each([&](float z) {
          const float yy = fast_y(w, z);
          if (yy >= kCut && z >= floor_z) {
            const int b = min(Row<T>::bin_of(yy), kBins - 1);
            if (b <= b_cut) {
              atomicAdd(&sh.cnt[b], 1u);
              // the weight over the bin's own: 15 bits
              atomicAdd(&sh.mass[b], __float2uint_rn(32768.f * ex2_approx(yy + 0.03125f * b)));
            }
          }
        });
      }
      r.cl.sync();
      // running sums over the bins of all slices; each thread takes three bins
      uint32_t n[3];
      float m[3], n_m = 0.f;
      uint32_t n_c = 0;
#pragma unroll
      for (int i = 0; i < 3; ++i) {
        const int b = threadIdx.x * 3 + i;
        n[i] = 0;
        uint64_t mm = 0;
        if (b <= b_cut)
          for (int c = 0; c < r.C; ++c) {
            n[i] += r.cl.map_shared_rank(sh.cnt, c)[b];
            if (!use_k) mm += r.cl.map_shared_rank(sh.mass, c)[b];
          }
        m[i] = static_cast<float>(mm) * ex2_approx(-15.f - 0.03125f * b);
        n_c += n[i];
        n_m += m[i];
      }
      uint32_t n_in = n_c;
      float m_in = n_m;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t x = __shfl_up_sync(0xffffffffu, n_in, o);
        const float y = __shfl_up_sync(0xffffffffu, m_in, o);
        if (lane >= o) {
          n_in += x;
          m_in += y;
        }
      }
      if (lane == 31) {
        sh.scan_u[warp] = n_in;
        sh.scan_f[warp] = m_in;
      }
      if (threadIdx.x == 0) {
        sh.b1 = sh.b2 = kBins - 1;
        sh.upto = 0xFFFFFFFFu;
      }
      __syncthreads();
      uint32_t n_at = n_in - n_c;
      float m_at = m_in - n_m;
      for (int i = 0; i < warp; ++i) {
        n_at += sh.scan_u[i];
        m_at += sh.scan_f[i];
      }
      // the masses here are 2^-16 off for their 15 bits, and 2^-20 for the rest
      const float need = sh.top_p * (static_cast<float>(S.mass2) / w.one);
#pragma unroll
      for (int i = 0; i < 3; ++i) {
        const int b = threadIdx.x * 3 + i;
        n_at += n[i];
        m_at += m[i];
        if (b >= kBins) continue;
        if (use_k) {
          if (n_at >= static_cast<uint32_t>(sh.top_k)) atomicMin(&sh.b2, b);
        } else {
          if (m_at * (1.f + 6e-5f) >= need) atomicMin(&sh.b1, b);
          if (m_at * (1.f - 6e-5f) > need) {  // (running counts ascend with b)
            atomicMin(&sh.b2, b);
            atomicMin(&sh.upto, n_at);
          }
        }
      }
      __syncthreads();
      const int b1 = sh.b1, b2 = sh.b2;
      auto in_bins = [&](float z, int lo, int hi) {
        const float y = fast_y(w, z);
        if (!(y >= kCut) || !(z >= floor_z)) return false;
        const int b = min(Row<T>::bin_of(y), kBins - 1);
        return b >= lo && b <= hi;
      };
      if (fits && (use_k || sh.upto <= kCap)) {
        // ---- few candidates: the leader finishes the row with exact weights
        const uint32_t n_all = r.gather([&](float z) { return in_bins(z, 0, b2); });
        if (n_all <= kCap) {
          listed = leader_draws = true;
          if (r.rank == 0) {
            uint32_t n_l = n_all;
            r.sort_desc(sh.cand, n_l);
            for (uint32_t i = threadIdx.x; i < n_l; i += kThreads)
              sh.wts[i] = weight(w, float_of(static_cast<uint32_t>(sh.cand[i] >> 32)));
            __syncthreads();
            if (warp == 0) {
              if (use_k) n_l = min(n_l, static_cast<uint32_t>(sh.top_k));
              uint64_t total = 0;
              for (uint32_t i = lane; i < n_l; i += 32) total += sh.wts[i];
              total = warp_sum(total);
              bool bad = false;
              if (use_p) {
                // with top-k the mass is this list's; else everything's, within E
                const double base = static_cast<double>(use_k ? total : S.mass2);
                const double want = static_cast<double>(sh.top_p) * base;
                const double slack = use_k ? 0.0 : 2.0 * E;
                uint64_t run = 0;
                uint32_t stay = 0;
                for (uint32_t i0 = 0; i0 < n_l; i0 += 32) {
                  const uint32_t i = i0 + lane;
                  const uint64_t x = i < n_l ? sh.wts[i] : 0;
                  const uint64_t before = run + warp_scan(x, lane) - x;
                  const double off = static_cast<double>(before) - want;
                  stay += __popc(__ballot_sync(0xffffffffu, i < n_l && off < 0.0));
                  bad |= __any_sync(0xffffffffu, slack > 0.0 && i < n_l && i > 0 && fabs(off) <= slack);
                  run += warp_sum(x);
                }
                // the last one's far side, where the cut may fall behind the list
                bad |= slack > 0.0 && static_cast<double>(run) - want <= slack;
                n_l = max(1u, stay);
              }
              if (lane == 0) {
                sh.upto = n_l;
                sh.bad = bad ? 1 : 0;
              }
            }
            __syncthreads();
            n_l = sh.upto;
            // by index: the draw runs in the row's own order
            for (uint32_t i = threadIdx.x; i < n_l; i += kThreads)
              sh.cand[i] = (sh.cand[i] << 32) | i;  // ~index descends as the index ascends
            __syncthreads();
            r.sort_desc(sh.cand, n_l);
            if (warp == 0) {
              uint64_t total = 0;
              for (uint32_t i = lane; i < n_l; i += 32) total += sh.wts[i];
              total = warp_sum(total);
              const double target = static_cast<double>(sh.u) * static_cast<double>(total);
              uint64_t run = 0;
              for (uint32_t i0 = 0; i0 < n_l; i0 += 32) {
                const uint32_t i = i0 + lane;
                const uint64_t c = i < n_l ? sh.cand[i] : 0;
                const uint64_t x = i < n_l ? sh.wts[static_cast<uint32_t>(c)] : 0;
                const uint64_t upto = run + warp_scan(x, lane);
                const uint32_t hit = __ballot_sync(0xffffffffu, static_cast<double>(upto) > target);
                if (hit) {
                  token = static_cast<int>(~static_cast<uint32_t>(
                      __shfl_sync(0xffffffffu, c, __ffs(hit) - 1) >> 32));
                  break;
                }
                run += warp_sum(x);
              }
            }
          }
        }
      } else if (fits && !use_k) {
        // ---- many tokens stay: the cut falls in bins b1 to b2, whose tokens are
        // of one value (they tie) or few enough to be sorted
        Part q = {0, 0, 0, 0xFFFFFFFFu, 0, 0.f};
        r.each([&](float z) {
          const float y = fast_y(w, z);
          if (!(y >= kCut) || !(z >= floor_z)) return;
          const int b = min(Row<T>::bin_of(y), kBins - 1);
          if (b < b1) {
            q.mass += weigh<EXACT>(w, z);
          } else if (b <= b2) {
            const uint32_t key = key_of(z);
            ++q.count;
            q.lo = min(q.lo, key);
            q.hi = max(q.hi, key);
          }
        });
        q = r.join(q);
        const double want = static_cast<double>(sh.top_p) * static_cast<double>(S.mass2);
        const double rest = want - static_cast<double>(q.mass);
        if (q.count > 0 && q.lo == q.hi) {
          const double each = static_cast<double>(weight(w, float_of(q.lo)));
          const double m = rest / each, up = ceil(m);
          // the cut is the interval's own only if it falls inside it
          if (rest > 0.0 && up <= static_cast<double>(q.count)) {
            if (!EXACT && ((up - m) * each <= 2.0 * E || (m - (up - 1.0)) * each <= 2.0 * E)) return false;
            keep.t = q.lo;
            keep.ties = static_cast<uint32_t>(up);
            listed = true;
          }
        } else if (q.count > 0 && q.count <= kCap) {
          r.gather([&](float z) { return in_bins(z, b1, b2); });
          if (r.rank == 0) {
            r.sort_desc(sh.cand, q.count);
            for (uint32_t i = threadIdx.x; i < q.count; i += kThreads)
              sh.wts[i] = weight(w, float_of(static_cast<uint32_t>(sh.cand[i] >> 32)));
            __syncthreads();
            if (warp == 0) {
              uint64_t run = 0;
              uint32_t stay = 0;
              bool bad = false;
              for (uint32_t i0 = 0; i0 < q.count; i0 += 32) {
                const uint32_t i = i0 + lane;
                const uint64_t x = i < q.count ? sh.wts[i] : 0;
                const double off = static_cast<double>(run + warp_scan(x, lane) - x) - rest;
                stay += __popc(__ballot_sync(0xffffffffu, i < q.count && off < 0.0));
                bad |= !EXACT && __any_sync(0xffffffffu, i < q.count && fabs(off) <= 2.0 * E);
                run += warp_sum(x);
              }
              bad |= !EXACT && fabs(static_cast<double>(run) - rest) <= 2.0 * E;
              bad |= stay == 0 || (stay == q.count && static_cast<double>(run) < rest);
              const uint32_t t = stay ? static_cast<uint32_t>(sh.cand[stay - 1] >> 32) : 0;
              uint32_t ties = 0;
              for (uint32_t i = lane; i < stay; i += 32)
                ties += static_cast<uint32_t>(sh.cand[i] >> 32) == t;
              ties = __reduce_add_sync(0xffffffffu, ties);
              if (lane == 0) {
                sh.t = t;
                sh.ties = ties;
                sh.bad = bad ? 1 : 0;
              }
            }
          }
          r.cl.sync();
          const Shared& lead = *r.cl.map_shared_rank(&sh, 0);
          keep.t = lead.t;
          keep.ties = lead.ties;
          listed = lead.bad == 0;
        }
      }
    }
    if (!listed) {
      // ---- by halves of the key's range: any row, any number of ties
      if (!EXACT) return false;
      if (use_k) {  // smallest t with fewer than k keys above it
        const uint32_t k = static_cast<uint32_t>(sh.top_k);
        uint32_t lo = 0, hi = kmax;
        while (lo < hi) {
          const uint32_t mid = lo + (hi - lo) / 2;
          if (r.template above<false>(w, mid).count < k) hi = mid;
          else lo = mid + 1;
        }
        keep.t = lo;
        keep.ties = k - r.template above<false>(w, lo).count;
      }
      if (sh.use_q && key_of(floor_z) > keep.t) {
        keep.t = key_of(floor_z);
        keep.ties = 0xFFFFFFFFu;
      }
      if (use_p) {
        const uint32_t t = keep.t;
        const Part over = r.template above<true>(w, t);
        // t = 0 has no ties: no logit has key 0
        const uint32_t from = t == 0 ? over.count : r.template above<false>(w, t - 1).count;
        const uint64_t at = min(keep.ties, from - over.count);
        const uint64_t kept = over.mass + (t == 0 ? 0 : at * weight(w, float_of(t)));
        const double need = static_cast<double>(sh.top_p) * static_cast<double>(kept);
        uint32_t lo = t, hi = kmax;  // smallest key with less than `need` above it
        while (lo < hi) {
          const uint32_t mid = lo + (hi - lo) / 2;
          if (static_cast<double>(r.template above<true>(w, mid).mass) < need) hi = mid;
          else lo = mid + 1;
        }
        const double rest = need - static_cast<double>(r.template above<true>(w, lo).mass);
        const double each = static_cast<double>(weight(w, float_of(lo)));
        uint32_t more = 0xFFFFFFFFu;  // ties before which there is less than `need`
        if (rest <= 0.0) more = 1;    // p <= 0: the first token alone
        else if (each > 0.0 && rest / each < 4294967295.0)
          more = static_cast<uint32_t>(ceil(rest / each));
        keep.ties = lo > t ? more : min(keep.ties, more);
        keep.t = lo;
      }
    }
  } else if (sh.use_q) {
    keep.t = key_of(floor_z);
  }

  if (leader_draws) {
    if (threadIdx.x == 0 && r.rank == 0 && !sh.bad) sh.t = static_cast<uint32_t>(token);
  } else {
    // ---- the draw: the warps' masses and ties, then the one warp that holds u
    uint64_t my_mass = warp_all;
    uint32_t my_eq = 0;
    if (keep.t != 0) {
      uint64_t m = 0;
      PairSum f;
      uint32_t eq = 0;
      r.each([&](float z) {
        const uint32_t key = key_of(z);
        if (key > keep.t) {
          if (EXACT) m += weight(w, z);
          else f.add(fast_weight(fast_y(w, z)));
        }
        eq += key == keep.t;
      });
      my_mass = warp_sum(EXACT ? m : f.fixed(w.one));
      my_eq = __reduce_add_sync(0xffffffffu, eq);
    }
    Part* mine = sh.part[r.turn];
    if (lane == 0) {
      mine[warp].mass = my_mass;
      mine[warp].count = my_eq;
    }
    if (threadIdx.x == 0) sh.bad = 0;
    r.cl.sync();
    r.turn ^= 1;
    // before this warp, and in all: ranks and warps are in index order
    uint64_t m_before = 0, m_all = 0, e_before = 0, e_all = 0;
    for (int i = lane; i < r.C * kWarps; i += 32) {
      const Part& o = r.cl.map_shared_rank(mine, i / kWarps)[i % kWarps];
      const uint64_t m = o.mass, e = o.count;
      m_all += m;
      e_all += e;
      if (i < r.rank * kWarps + warp) {
        m_before += m;
        e_before += e;
      }
    }
    m_all = warp_sum(m_all);
    e_all = warp_sum(e_all);
    m_before = warp_sum(m_before);
    e_before = warp_sum(e_before);
    const uint64_t lim = keep.ties;
    const uint64_t wt = keep.t == 0 ? 0 : weigh<EXACT>(w, float_of(keep.t));
    const uint64_t total = m_all + min(e_all, lim) * wt;
    const double target = static_cast<double>(sh.u) * static_cast<double>(total);
    const uint64_t before = m_before + min(e_before, lim) * wt;
    const uint64_t after = m_before + my_mass + min(e_before + my_eq, lim) * wt;
    Shared* lead = r.cl.map_shared_rank(&sh, 0);
    if (static_cast<double>(before) <= target && static_cast<double>(after) > target) {
      uint64_t m = m_before, e = e_before;
      bool done = false;
      for (int vb = r.v0; vb < r.v1 && !done; vb += 32) {
        const int v = vb + lane;
        uint64_t s = 0, eq = 0;
        Vec<T> x;
        if (v < r.v1) {
          x = r.load(v);
#pragma unroll
          for (int i = 0; i < VE; ++i) {
            const float z = x.get(i);
            const uint32_t key = key_of(z);
            if (key > keep.t) s += weigh<EXACT>(w, z);
            eq += key == keep.t;
          }
        }
        const uint64_t s_in = m + warp_scan(s, lane), e_in = e + warp_scan(eq, lane);
        const uint32_t hit = __ballot_sync(
            0xffffffffu, static_cast<double>(s_in + min(e_in, lim) * wt) > target);
        if (hit) {
          done = true;
          if (lane == __ffs(hit) - 1) {
            uint64_t sm = s_in - s, se = e_in - eq;
            for (int i = 0; i < VE; ++i) {
              const float z = x.get(i);
              const uint32_t key = key_of(z);
              const double was = static_cast<double>(sm + min(se, lim) * wt);
              if (key > keep.t) sm += weigh<EXACT>(w, z);
              se += key == keep.t;
              const double now = static_cast<double>(sm + min(se, lim) * wt);
              if (now > target) {
                // a border within E of u: left to the exact weights
                if (!EXACT && (now - target <= 2.0 * E || target - was <= 2.0 * E)) lead->bad = 1;
                lead->t = static_cast<uint32_t>(r.pos0 + static_cast<int64_t>(v) * VE + i);
                break;
              }
            }
          }
        }
        m = __shfl_sync(0xffffffffu, s_in, 31);
        e = __shfl_sync(0xffffffffu, e_in, 31);
      }
      if (!EXACT && !done && lane == 0) lead->bad = 1;  // the float sums disagree by their rounding
    }
  }
  r.cl.sync();
  if (!EXACT && r.cl.map_shared_rank(&sh, 0)->bad) return false;
  if (r.rank == 0 && threadIdx.x == 0) {
    const int at = static_cast<int>(sh.t);
    const float z = clean(to_f(static_cast<const T*>(a.logits)[row * a.ld + at]));
    const double d = z == w.zmax ? 0.0 : (static_cast<double>(z) - w.zmax) / sh.temp;
    a.tokens[row] = at;
    a.logp[row] = static_cast<float>(d - log(static_cast<double>(S.mass) / w.one));
  }
  return true;
}

template <typename T>
__global__ void __launch_bounds__(kThreads, 2) k_sample(const SampleArgs a, int slice_vecs, int resident) {
  extern __shared__ uint4 s_slice[];
  __shared__ Shared sh;
  constexpr int VE = Vec<T>::N;
  Row<T> r(sh);
  r.lane = threadIdx.x & 31;
  r.warp = threadIdx.x >> 5;
  r.C = static_cast<int>(r.cl.num_blocks());
  r.rank = static_cast<int>(r.cl.block_rank());
  r.V = a.V;
  if (threadIdx.x < 32) sh.tab[threadIdx.x] = c_exp2_32[threadIdx.x];
  const int n_cl = gridDim.x / r.C;
  for (int64_t row = blockIdx.x / r.C; row < a.rows; row += n_cl) {
    const T* z = static_cast<const T*>(a.logits) + row * a.ld;
    // 16-byte pieces from the one that holds the row's first element
    const int off = static_cast<int>((reinterpret_cast<uintptr_t>(z) & 15) / sizeof(T));
    const int64_t pieces = (off + a.V + VE - 1) / VE;
    const int64_t p0 = static_cast<int64_t>(r.rank) * slice_vecs;
    r.n_vec = static_cast<int>(p0 >= pieces ? 0 : min(static_cast<int64_t>(slice_vecs), pieces - p0));
    r.pos0 = p0 * VE - off;
    const int per = (r.n_vec + kWarps - 1) / kWarps;
    r.v0 = min(r.n_vec, r.warp * per);
    r.v1 = min(r.n_vec, r.v0 + per);
    r.row = z;
    r.global = reinterpret_cast<const uint4*>(z - off) + p0;
    r.slice = resident ? s_slice : nullptr;

    // ---- copy the slice, taking the maximum on the way (a warp reads back its own)
    float mx = -INFINITY;
    for (int v = r.v0 + r.lane; v < r.v1; v += 32) {
      const Vec<T> x = r.fetch(v);
      if (resident) s_slice[v] = x.raw;
#pragma unroll
      for (int e = 0; e < VE; ++e) mx = fmaxf(mx, x.get(e));
    }
    __syncwarp();
    Part p = {0, 0, 0, 0xFFFFFFFFu, key_of(mx), 0.f};
    p = r.join(p);
    const uint32_t kmax = p.hi;
    const float zmax = float_of(kmax);
    if (zmax == -INFINITY) {  // nothing to choose from
      if (r.rank == 0 && threadIdx.x == 0) {
        a.tokens[row] = -1;
        a.logp[row] = -INFINITY;
      }
      continue;
    }
    if (threadIdx.x == 0) {
      const float T_in = a.temperature ? a.temperature[row] : 1.f;
      sh.warm = T_in > 0.f;
      const double temp = sh.warm ? static_cast<double>(T_in) : 1.0;
      sh.temp = temp;
      const double c = 1.4426950408889634074 / temp;
      sh.w.zmax = zmax;
      // within float range: a T of 0 or infinity up to rounding
      sh.w.c_hi = fminf(fmaxf(static_cast<float>(c), 1.4e-45f), 3.4e38f);
      sh.w.c_lo = c < 3.4e38 && c > 1e-30 ? static_cast<float>(c - static_cast<double>(sh.w.c_hi)) : 0.f;
      // V 2^B < 2^62
      const int bits = min(44, 62 - (32 - __clz(static_cast<int>(a.V))));
      sh.w.one = __uint_as_float(static_cast<uint32_t>(127 + bits) << 23);
      sh.w.tab = sh.tab;
      const int k = a.top_k ? a.top_k[row] : 0;
      sh.top_k = k > 0 && k < a.V ? k : 0;
      const float q = a.min_p ? a.min_p[row] : 0.f;
      sh.use_q = q > 0.f && sh.warm;
      // the smallest float z with exp((z - zmax) / T) >= q
      sh.floor_z = !sh.use_q ? -INFINITY
                   : q >= 1.f ? zmax
                              : fminf(zmax, __double2float_ru(zmax + temp * log(static_cast<double>(q))));
      sh.top_p = a.top_p ? a.top_p[row] : 1.f;
      sh.use_p = sh.top_p < 1.f;
      sh.top_p = fmaxf(sh.top_p, 0.f);
      sh.u = fminf(fmaxf(a.u[row], 0.f), 1.f - 5.9604645e-8f);
    }
    __syncthreads();
    if (!resident || zmax == INFINITY || !decide<T, false>(r, a, row, kmax, mx, true)) {
      // (the cluster's CTAs leave a row that was not decided at the same point)
      r.cl.sync();
      decide<T, true>(r, a, row, kmax, mx, resident && zmax < INFINITY);
    }
    r.cl.sync();
  }
}

template <typename T>
cudaError_t launch(const SampleArgs& a, int sms, cudaStream_t s) {
  constexpr int VE = 16 / static_cast<int>(sizeof(T));
  const int64_t bytes = a.V * static_cast<int64_t>(sizeof(T)) + 15;
  // The smallest cluster whose slices leave room for three CTAs on an SM, and
  // with few rows a larger one, down to 8 KB a CTA, until every SM has one.
  int C = 1;
  while (C < kMaxCluster && (bytes / C > 52 * 1024 || (a.rows * C < sms && bytes / C > 16 * 1024))) C *= 2;
  const int64_t pieces = (a.V + VE - 1) / VE + 1;  // a row may start inside its first piece
  const int64_t slice = (pieces + C - 1) / C;
  const bool resident = slice * 16 <= kMaxSliceBytes;
  if (slice > INT32_MAX / VE) return cudaErrorInvalidValue;
  const size_t smem = resident ? static_cast<size_t>(slice) * 16 : 0;
  static std::atomic<uint64_t> configured{0};  // one bit a device
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = 1ull << (dev & 63);
  if (!(configured.load() & bit)) {
    e = cudaFuncSetAttribute(k_sample<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSliceBytes);
    if (e != cudaSuccess) return e;
    configured.fetch_or(bit);
  }
  cudaLaunchConfig_t cfg = {};
  const int64_t clusters = a.rows < 65536 ? a.rows : 65536;
  cfg.gridDim = dim3(static_cast<unsigned>(clusters * C));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = C;
  at[0].val.clusterDim.y = 1;
  at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k_sample<T>, a, static_cast<int>(slice), resident ? 1 : 0);
}

}  // namespace

cudaError_t launch_sample(const SampleArgs& a, int sms, cudaStream_t s) {
  return a.bf16 ? launch<__nv_bfloat16>(a, sms, s) : launch<float>(a, sms, s);
}

}  // namespace grpo
