// Token sampling with temperature, top-k, top-p and min-p from given uniforms.
//
// A row's weights w_i = exp((z_i - zmax) / T) are formed as integers of fixed
// point, W_i = w_i 2^B, from 2^y evaluated in pairs of floats to about 2^-43:
// integer sums do not depend on their order, so the cut-offs and the token come
// out the same however a row is split, and they are the token of the real
// numbers unless u falls within about 2^-40 of a border. (Sums of float32
// weights would misplace borders by 2^-22 or so: with 10^5 tokens of similar
// weight one draw in ten would differ.)
//
// All three cut-offs keep a prefix of the order (logit descending, index
// ascending), so what is kept is a threshold t on the logit and a number of
// ties at t, the first in index order. A float's bits, mapped to an unsigned
// key that sorts like the float, make the threshold an integer to search for.
#include <cuda_bf16.h>

#include "internal.h"

namespace grpo {

namespace {

constexpr int kThreads = 1024;

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

__device__ __forceinline__ float load_logit(const float* p, int64_t i) { return p[i]; }
__device__ __forceinline__ float load_logit(const __nv_bfloat16* p, int64_t i) {
  return __bfloat162float(p[i]);
}
// NaN counts as -inf; -0 as +0, so that the two tie.
__device__ __forceinline__ float clean(float z) { return z != z ? -INFINITY : z + 0.f; }

__device__ __forceinline__ uint32_t key_of(float z) {
  const uint32_t b = __float_as_uint(z);
  return b ^ ((b >> 31) ? 0xFFFFFFFFu : 0x80000000u);
}
__device__ __forceinline__ float float_of(uint32_t key) {
  return __uint_as_float(key ^ ((key >> 31) ? 0x80000000u : 0xFFFFFFFFu));
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

__device__ __forceinline__ uint64_t warp_sum(uint64_t v) {
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// CTA-wide sums of a mass and a count.
struct Sum {
  uint64_t mass;
  uint32_t count;
};
__device__ __forceinline__ Sum block_sum(uint64_t mass, uint32_t count) {
  __shared__ uint64_t s_mass[32];
  __shared__ uint32_t s_count[32];
  mass = warp_sum(mass);
  count = __reduce_add_sync(0xffffffffu, count);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) {
    s_mass[threadIdx.x >> 5] = mass;
    s_count[threadIdx.x >> 5] = count;
  }
  __syncthreads();
  Sum r = {0, 0};
  for (int i = 0; i < kThreads / 32; ++i) {
    r.mass += s_mass[i];
    r.count += s_count[i];
  }
  return r;
}
__device__ __forceinline__ uint32_t block_max(uint32_t v) {
  __shared__ uint32_t s_max[32];
  v = __reduce_max_sync(0xffffffffu, v);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) s_max[threadIdx.x >> 5] = v;
  __syncthreads();
  for (int i = 0; i < kThreads / 32; ++i) v = max(v, s_max[i]);
  return v;
}

// One CTA a row; the row is read again for every question asked of it.
template <typename T>
__global__ void __launch_bounds__(kThreads) k_sample(SampleArgs a) {
  __shared__ float2 s_tab[32];
  __shared__ uint64_t s_scan[32], s_ties[32];
  __shared__ int s_token;
  const int64_t row = blockIdx.x;
  const T* z = static_cast<const T*>(a.logits) + row * a.ld;
  const int V = static_cast<int>(a.V);
  if (threadIdx.x < 32) s_tab[threadIdx.x] = c_exp2_32[threadIdx.x];
  if (threadIdx.x == 0) s_token = -1;

  uint32_t kmax = 0;
  for (int64_t i = threadIdx.x; i < V; i += kThreads) kmax = max(kmax, key_of(clean(load_logit(z, i))));
  kmax = block_max(kmax);
  const float zmax = float_of(kmax);
  if (zmax == -INFINITY) {  // nothing to choose from
    if (threadIdx.x == 0) {
      a.tokens[row] = -1;
      a.logp[row] = -INFINITY;
    }
    return;
  }
  const float T_in = a.temperature ? a.temperature[row] : 1.f;
  const bool warm = T_in > 0.f;
  const float temp = warm ? T_in : 1.f;
  const double c = 1.4426950408889634074 / static_cast<double>(temp);
  Weigher w;
  w.zmax = zmax;
  w.c_hi = static_cast<float>(c);
  w.c_lo = isinf(w.c_hi) ? 0.f : static_cast<float>(c - static_cast<double>(w.c_hi));
  // V 2^B < 2^62
  int bits = 62 - (32 - __clz(V));
  bits = min(bits, 44);
  w.one = __uint_as_float(static_cast<uint32_t>(127 + bits) << 23);
  w.tab = s_tab;

  // mass and number of the tokens with key > k
  auto above = [&](uint32_t k) {
    uint64_t mass = 0;
    uint32_t count = 0;
    for (int64_t i = threadIdx.x; i < V; i += kThreads) {
      const float v = clean(load_logit(z, i));
      if (key_of(v) > k) {
        mass += weight(w, v);
        ++count;
      }
    }
    return block_sum(mass, count);
  };

  const uint64_t all = above(0).mass;  // every key is above 0
  // kept: keys above t, and the first `ties` of those equal to t
  uint32_t t = 0;
  uint32_t ties = 0xFFFFFFFFu;
  if (!warm) {
    t = kmax;
    ties = 1;
  } else {
    const int k = a.top_k ? a.top_k[row] : 0;
    if (k > 0 && k < V) {  // smallest t with fewer than k keys above it
      uint32_t lo = 0, hi = kmax;
      while (lo < hi) {
        const uint32_t mid = lo + (hi - lo) / 2;
        if (above(mid).count < static_cast<uint32_t>(k)) hi = mid;
        else lo = mid + 1;
      }
      t = lo;
      ties = static_cast<uint32_t>(k) - above(t).count;
    }
    const float q = a.min_p ? a.min_p[row] : 0.f;
    if (q > 0.f) {  // smallest key of a weight of q or more
      const double least = fmin(static_cast<double>(q), 1.0) * static_cast<double>(w.one);
      uint32_t lo = t, hi = kmax;
      while (lo < hi) {
        const uint32_t mid = lo + (hi - lo) / 2;
        if (static_cast<double>(weight(w, float_of(mid))) >= least) hi = mid;
        else lo = mid + 1;
      }
      if (lo > t) {
        t = lo;
        ties = 0xFFFFFFFFu;
      }
    }
    const float p = a.top_p ? a.top_p[row] : 1.f;
    if (p < 1.f) {
      const Sum over = above(t), from = above(t - 1);  // t = 0 has no ties: no logit has key 0
      const uint32_t at = t == 0 ? 0 : min(ties, from.count - over.count);
      const uint64_t kept = over.mass + at * weight(w, float_of(t));
      const double need = static_cast<double>(p) * static_cast<double>(kept);
      // smallest key in [t, kmax] above which there is less than `need`
      uint32_t lo = t, hi = kmax;
      while (lo < hi) {
        const uint32_t mid = lo + (hi - lo) / 2;
        if (static_cast<double>(above(mid).mass) < need) hi = mid;
        else lo = mid + 1;
      }
      const double rest = need - static_cast<double>(above(lo).mass);
      const double each = static_cast<double>(weight(w, float_of(lo)));
      uint32_t more = 0xFFFFFFFFu;  // ties before which there is less than `need`
      if (rest <= 0.0) more = 1;    // p <= 0: the first token alone
      else if (each > 0.0 && rest / each < 4294967295.0) more = static_cast<uint32_t>(ceil(rest / each));
      ties = lo > t ? more : min(ties, more);
      t = lo;
    }
  }

  // the draw: threads own consecutive pieces of the row
  const int piece = (V + kThreads - 1) / kThreads;
  const int i0 = min(V, static_cast<int>(threadIdx.x) * piece), i1 = min(V, i0 + piece);
  uint64_t mass = 0, eq = 0;
  for (int i = i0; i < i1; ++i) {
    const float v = clean(load_logit(z, i));
    const uint32_t key = key_of(v);
    if (key > t) mass += weight(w, v);
    eq += key == t;
  }
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint64_t m_in = mass, e_in = eq;  // inclusive scans over the CTA
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint64_t m = __shfl_up_sync(0xffffffffu, m_in, o), e = __shfl_up_sync(0xffffffffu, e_in, o);
    if (lane >= o) {
      m_in += m;
      e_in += e;
    }
  }
  if (lane == 31) {
    s_scan[warp] = m_in;
    s_ties[warp] = e_in;
  }
  __syncthreads();
  uint64_t m_all = 0, e_all = 0, m_before = 0, e_before = 0;
  for (int i = 0; i < kThreads / 32; ++i) {
    if (i == warp) {
      m_before = m_all + m_in - mass;
      e_before = e_all + e_in - eq;
    }
    m_all += s_scan[i];
    e_all += s_ties[i];
  }
  const uint64_t wt = t == 0 ? 0 : weight(w, float_of(t));
  const uint64_t lim = ties;
  const uint64_t total = m_all + min(e_all, lim) * wt;
  const float u = fminf(fmaxf(a.u[row], 0.f), 1.f - 5.9604645e-8f);
  const double target = static_cast<double>(u) * static_cast<double>(total);
  const uint64_t before = m_before + min(e_before, lim) * wt;
  const uint64_t after = m_before + mass + min(e_before + eq, lim) * wt;
  if (static_cast<double>(before) <= target && static_cast<double>(after) > target) {
    uint64_t m = m_before, e = e_before;
    for (int i = i0; i < i1; ++i) {
      const float v = clean(load_logit(z, i));
      const uint32_t key = key_of(v);
      if (key > t) m += weight(w, v);
      e += key == t;
      if (static_cast<double>(m + min(e, lim) * wt) > target) {
        s_token = i;
        break;
      }
    }
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    const int token = s_token;
    const float v = clean(load_logit(z, token));
    const double d = v == zmax ? 0.0 : (static_cast<double>(v) - zmax) / temp;
    a.tokens[row] = token;
    a.logp[row] = static_cast<float>(d - log(static_cast<double>(all) / static_cast<double>(w.one)));
  }
}

}  // namespace

cudaError_t launch_sample(const SampleArgs& a, int, cudaStream_t s) {
  if (a.bf16)
    k_sample<__nv_bfloat16><<<static_cast<unsigned>(a.rows), kThreads, 0, s>>>(a);
  else
    k_sample<float><<<static_cast<unsigned>(a.rows), kThreads, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace grpo
