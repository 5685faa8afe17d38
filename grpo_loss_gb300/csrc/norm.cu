// Layer norm and RMS norm over rows, forward and backward.
//   y = (x - mean) r w + b,  r = 1 / sqrt(mean((x - mean)^2) + eps)
//   g = dy w, h = (x - mean) r:  dx = r (g - mean(g) - h mean(g h)),
//   dw = sum_rows dy h,  db = sum_rows dy            (RMS: mean = 0, no b)
// Bound by memory: the forward reads x and writes y, the backward reads x and
// dy and writes dx, each once; a row stays in registers between its sums and
// its output. The backward's CTAs walk over the rows and keep dw and db of
// their columns in registers, so that x and dy are not read again for the
// column sums: those leave one partial row pair a CTA, joined in a fixed order.
// 262144 rows of 2880 in bf16, RMS: forward 441 us (6.8 TB/s); 163840 of 4096: backward
// 671 us (6.0 TB/s; two rows' sums, barriers and column sums a turn beside the bytes),
// of the RMS form 637.
#include <cuda_bf16.h>

#include <atomic>

#include "f32x2.cuh"
#include "internal.h"
#include "pieces.cuh"

namespace grpo {

namespace {

// ---------------------------------------------------------------- forward
// A group of G threads takes a row, R rows a CTA; each thread holds NV pieces of
// N values of it (G N NV >= d).
template <typename T, int N, int NV, int G, int R>
__global__ void __launch_bounds__(G * R) k_norm_fwd(NormArgs a) {
  __shared__ float part[2 * 128];
  const int tid = threadIdx.x % G;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * R + threadIdx.x / G;
  const bool live = row < a.rows;  // every thread takes part in the barriers
  const int d = static_cast<int>(a.d);
  const T* x = static_cast<const T*>(a.x) + (live ? row : 0) * a.ld_x;
  Piece<T, N> v[NV];
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    const int i = (k * G + tid) * N;
    if (i < d) v[k] = load_piece<T, N>(x + i);
  }
  const float inv_d = 1.f / d;
  float mean = 0.f;
  if (!a.rms) {
    float s = 0.f;
#pragma unroll
    for (int k = 0; k < NV; ++k)
      if ((k * G + tid) * N < d)
#pragma unroll
        for (int e = 0; e < N; ++e) s += v[k].get(e);
    mean = group_sum<G>(s, part, 0) * inv_d;
  }
  float q = 0.f;
#pragma unroll
  for (int k = 0; k < NV; ++k)
    if ((k * G + tid) * N < d)
#pragma unroll
      for (int e = 0; e < N; ++e) {
        const float c = v[k].get(e) - mean;
        q = fmaf(c, c, q);
      }
  const float r = rsqrtf(group_sum<G>(q, part, 1) * inv_d + a.eps);
  if (!live) return;
  T* y = static_cast<T*>(a.y) + row * a.ld_y;
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    const int i = (k * G + tid) * N;
    if (i < d) {
      float o[N], w[N];
      load_params<N>(a.weight, a.param_bf16, i, w);
#pragma unroll
      for (int e = 0; e < N; ++e) o[e] = (v[k].get(e) - mean) * r * w[e];
      if (a.bias) {
        load_params<N>(a.bias, a.param_bf16, i, w);
#pragma unroll
        for (int e = 0; e < N; ++e) o[e] += w[e];
      }
      Piece<T, N> p;
      p.set(o);
      store_piece<T, N>(y + i, p);
    }
  }
  if (tid == 0) {
    if (a.mean) a.mean[row] = mean;
    if (a.rstd) a.rstd[row] = r;
  }
}

// Clears the first n elements of a 16-byte piece.
template <typename T, int N>
__device__ __forceinline__ void clear_first(Piece<T, N>& p, int n) {
  if constexpr (N * sizeof(T) == 16) {
    const int bits = n * 8 * static_cast<int>(sizeof(T));  // below 128
    auto keep = [&](int word) {
      const int b = min(max(bits - 32 * word, 0), 32);
      return b == 32 ? 0u : 0xFFFFFFFFu << b;
    };
    p.raw.x &= keep(0);
    p.raw.y &= keep(1);
    p.raw.z &= keep(2);
    p.raw.w &= keep(3);
  }
}

// Rows that are not on 16-byte boundaries, or not a multiple of 16 bytes long: a
// row's pieces are those of the 16-byte granules it lies in. A group walks over rows
// a multiple of 8 apart, which all start `off` elements inside a granule, so that the
// weights of its pieces stay the same; they are in shared memory, each thread's own in
// the order it reads them, and the next row is on its way there meanwhile. What a
// granule holds beside the row is cleared, and not written. (99900 rows of 1001 in
// bf16: 99 us; single elements 183, granules without the copies ahead 134.)
template <typename T, int NV, int G, int R>
__global__ void __launch_bounds__(G * R) k_norm_fwd_ragged(NormArgs a) {
  constexpr int N = 16 / static_cast<int>(sizeof(T)), THREADS = G * R;
  using V = Piece<T, N>;
  extern __shared__ __align__(16) unsigned char ring_raw[];
  __shared__ float part[2 * 128];
  V* const ring = reinterpret_cast<V*>(ring_raw) + threadIdx.x;  // [2 rows][NV][threads]
  // [w, b][NV][threads] pieces of bf16, or [w, b][NV][N / 4][threads] of four floats
  unsigned char* const params = ring_raw + 2 * NV * THREADS * 16;
  using P16 = Piece<__nv_bfloat16, N>;
  auto par16 = [&](int which, int k) -> P16& { return reinterpret_cast<P16*>(params)[(which * NV + k) * THREADS + threadIdx.x]; };
  auto par32 = [&](int which, int k, int f) -> float4& {
    return reinterpret_cast<float4*>(params)[((which * NV + k) * (N / 4) + f) * THREADS + threadIdx.x];
  };
  const int tid = threadIdx.x % G, d = static_cast<int>(a.d);
  const int64_t groups = static_cast<int64_t>(gridDim.x) * R, row0 = static_cast<int64_t>(blockIdx.x) * R + threadIdx.x / G;
  const int off = static_cast<int>((reinterpret_cast<uintptr_t>(static_cast<const T*>(a.x) + row0 * a.ld_x) & 15) / sizeof(T));
  auto column = [&](int k) { return (k * G + tid) * N - off; };  // of a piece's first element
  auto inside = [&](int i) { return i >= 0 && i < d; };
  for (int which = 0; which < (a.bias ? 2 : 1); ++which) {
    const void* const from = which ? a.bias : a.weight;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      float v[N];
#pragma unroll
      for (int e = 0; e < N; ++e) v[e] = inside(column(k) + e) ? param(from, a.param_bf16, column(k) + e) : 0.f;
      if (a.param_bf16) par16(which, k).set(v);  // (exact)
      else
#pragma unroll
        for (int f = 0; f < N / 4; ++f) par32(which, k, f) = make_float4(v[4 * f], v[4 * f + 1], v[4 * f + 2], v[4 * f + 3]);
    }
  }
  auto load_par = [&](int which, int k, float (&v)[N]) {
    if (a.param_bf16) {
      const P16 q = par16(which, k);
#pragma unroll
      for (int e = 0; e < N; ++e) v[e] = q.get(e);
    } else {
#pragma unroll
      for (int f = 0; f < N / 4; ++f) {
        const float4 q = par32(which, k, f);
        v[4 * f] = q.x, v[4 * f + 1] = q.y, v[4 * f + 2] = q.z, v[4 * f + 3] = q.w;
      }
    }
  };
  auto fetch = [&](int64_t row, int half) {
    if (row < a.rows) {
      const T* x = static_cast<const T*>(a.x) + row * a.ld_x;
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        const int i = column(k);
        V& to = ring[(half * NV + k) * THREADS];
        if (i < 0 && row < off) {  // the granule begins before the matrix (a row is an element long at least)
#pragma unroll
          for (int e = 0; e < N; ++e) reinterpret_cast<T*>(&to)[e] = inside(i + e) ? x[i + e] : static_cast<T>(0.f);
        } else if (i < d) {
          copy_async_zero(&to, x + i, min(N, d - i) * static_cast<int>(sizeof(T)));
        }
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  const float inv_d = 1.f / d;
  int slot = 1, half = 0;
  fetch(row0, 0);
  // every group of a CTA makes the same number of turns: barriers are the CTA's
  for (int64_t first = static_cast<int64_t>(blockIdx.x) * R; first < a.rows; first += groups, half ^= 1) {
    const int64_t row = first + threadIdx.x / G;
    const bool live = row < a.rows;
    fetch(row + groups, half ^ 1);
    asm volatile("cp.async.wait_group 1;" ::: "memory");
    V v[NV];
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      v[k].raw = make_uint4(0, 0, 0, 0);
      if (live && column(k) < d) v[k] = ring[(half * NV + k) * THREADS];
    }
    if (tid == 0 && off > 0) clear_first(v[0], off);
    float mean = 0.f;
    if (!a.rms) {
      float t = 0.f;
#pragma unroll
      for (int k = 0; k < NV; ++k)
#pragma unroll
        for (int e = 0; e < N; ++e) t += v[k].get(e);
      mean = group_sum<G>(t, part, 0) * inv_d;
    }
    float q = 0.f;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int i = column(k);
      if (i >= 0 && i + N <= d) {
#pragma unroll
        for (int e = 0; e < N; ++e) {
          const float c = v[k].get(e) - mean;
          q = fmaf(c, c, q);
        }
      } else if (i < d) {
#pragma unroll
        for (int e = 0; e < N; ++e) {
          const float c = inside(i + e) ? v[k].get(e) - mean : 0.f;
          q = fmaf(c, c, q);
        }
      }
    }
    const float r = rsqrtf(group_sum<G>(q, part, slot) * inv_d + a.eps);
    if (a.rms) slot ^= 1;  // (else the mean's sum has the other)
    if (!live) continue;
    T* y = static_cast<T*>(a.y) + row * a.ld_y;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int i = column(k);
      if (i >= d) continue;
      float o[N], w[N];
      load_par(0, k, w);
#pragma unroll
      for (int e = 0; e < N; ++e) o[e] = (v[k].get(e) - mean) * r * w[e];
      if (a.bias) {
        load_par(1, k, w);
#pragma unroll
        for (int e = 0; e < N; ++e) o[e] += w[e];
      }
      if (i >= 0 && i + N <= d && a.out16) {
        V p;
        p.set(o);
        store_piece<T, N>(y + i, p);
      } else {
#pragma unroll
        for (int e = 0; e < N; ++e)
          if (inside(i + e)) stf(y, i + e, o[e]);
      }
    }
    if (tid == 0) {
      if (a.mean) a.mean[row] = mean;
      if (a.rstd) a.rstd[row] = r;
    }
  }
}

// --------------------------------------------------------------- backward
// A group of G threads walks over the rows group, + groups, ... (R groups a CTA);
// each thread holds NV pieces of N columns: their values of a row and their column
// sums. It takes Q rows a turn, so that the joining of the row sums over the CTA
// (a barrier, and the shuffles before and behind it) is waited for once in Q rows;
// meanwhile its pieces of the next turn's rows are on their way into shared
// memory, whence they are read twice, for the sums and for dx. A thread reads back
// what it copied itself, so no barrier is needed for that. (163840 x 4096 bf16: 2
// rows ahead or 4 make no difference, one row a turn takes 936 us.)
// RAGGED: the pieces of a row are those of the 16-byte granules that it lies in, as in
// k_norm_fwd_ragged, `off` elements before its first. (99900 rows of 1001 in bf16: 150
// us, 60 % of the bytes' time; single elements 436.)
template <typename T, int N, int NV, int G, int R, int Q, bool RAGGED>
__global__ void __launch_bounds__(G * R) k_norm_bwd(NormArgs a) {
  constexpr int B = N * static_cast<int>(sizeof(T));
  using V = Piece<T, N>;
  extern __shared__ __align__(16) unsigned char ring_raw[];
  __shared__ float part[2 * 128];
  V* ring = reinterpret_cast<V*>(ring_raw) + threadIdx.x;  // [2 turns][Q][2][NV][threads]
  const int tid = threadIdx.x % G, d = static_cast<int>(a.d);
  const int64_t groups = static_cast<int64_t>(gridDim.x) * R;
  const int64_t row0 = static_cast<int64_t>(blockIdx.x) * R + threadIdx.x / G;
  const int off = RAGGED ? static_cast<int>((reinterpret_cast<uintptr_t>(static_cast<const T*>(a.x) + row0 * a.ld_x) & 15) / sizeof(T)) : 0;
  const int end = d + off;  // the pieces are those from 0 on that begin before it
  auto inside = [&](int i) { return i >= 0 && i < d; };
  auto whole = [&](int i) { return !RAGGED || (i >= 0 && i + N <= d && a.out16); };
  // columns in pairs (a column alone has a pair of its own)
  constexpr int H = (N + 1) / 2;
  uint64_t dw[NV][H], db[NV][H], w[NV][H];
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    const int i = (k * G + tid) * N - off;
    float ww[2 * H] = {};
    if constexpr (RAGGED) {
#pragma unroll
      for (int e = 0; e < N; ++e) ww[e] = inside(i + e) ? param(a.weight, a.param_bf16, i + e) : 0.f;
    } else if (i < d) {
      load_params<N>(a.weight, a.param_bf16, i, ww);
    }
#pragma unroll
    for (int e = 0; e < H; ++e) {
      dw[k][e] = db[k][e] = pair_of(0.f, 0.f);
      w[k][e] = pair_of(ww[2 * e], ww[2 * e + 1]);
    }
  }
  auto slot_of = [&](int s, int which, int k) -> V& {
    return ring[((s * 2 + which) * NV + k) * (G * R)];
  };
  // this thread's first piece of the row that is fetched next, and of the row that
  // is written; `left` rows of the group are still to be fetched
  const int64_t step = groups, mine = row0 < a.rows ? (a.rows - row0 + groups - 1) / groups : 0;
  const T* xp = static_cast<const T*>(a.x) + row0 * a.ld_x + tid * N - off;
  const T* gp = static_cast<const T*>(a.dy) + row0 * a.ld_dy + tid * N - off;
  T* dp = static_cast<T*>(a.dx) + row0 * a.ld_dx + tid * N - off;
  const float* mp = a.mean + (a.rms ? 0 : row0);
  const float* rp = a.rstd + row0;
  int left = static_cast<int>(mine);
  int64_t from = row0;  // the row that is fetched next (a row is an element long at least)
  auto fetch = [&](int half) {
#pragma unroll
    for (int q = 0; q < Q; ++q) {
      if (left > 0) {
        const int s = half * Q + q;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
          if ((k * G + tid) * N < end) {
            const int i = (k * G + tid) * N - off;
            if (RAGGED && i < 0 && from < off) {
              // the granule begins before the matrix
#pragma unroll
              for (int e = 0; e < N; ++e) {
                const bool in = inside(i + e);
                reinterpret_cast<T*>(&slot_of(s, 0, k))[e] = in ? xp[k * G * N + e] : static_cast<T>(0.f);
                reinterpret_cast<T*>(&slot_of(s, 1, k))[e] = in ? gp[k * G * N + e] : static_cast<T>(0.f);
              }
            } else if (RAGGED && i + N > d) {
              copy_async_zero(&slot_of(s, 0, k), xp + k * G * N, (d - i) * static_cast<int>(sizeof(T)));
              copy_async_zero(&slot_of(s, 1, k), gp + k * G * N, (d - i) * static_cast<int>(sizeof(T)));
            } else if constexpr (B >= 4) {
              copy_async<B>(&slot_of(s, 0, k), xp + k * G * N);
              copy_async<B>(&slot_of(s, 1, k), gp + k * G * N);
            } else {
              slot_of(s, 0, k) = load_piece<T, N>(xp + k * G * N);
              slot_of(s, 1, k) = load_piece<T, N>(gp + k * G * N);
            }
          }
        }
        xp += step * a.ld_x;
        gp += step * a.ld_dy;
        from += step;
        --left;
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  const float inv_d = 1.f / d;
  // every group of a CTA makes the same number of turns: barriers are the CTA's
  const int64_t first = static_cast<int64_t>(blockIdx.x) * R;
  const int rows = static_cast<int>(first < a.rows ? (a.rows - first + groups - 1) / groups : 0);
  float mean_next[Q], rstd_next[Q];
  auto fetch_stats = [&](int n) {  // of the group's rows from n on
#pragma unroll
    for (int q = 0; q < Q; ++q) {
      mean_next[q] = rstd_next[q] = 0.f;
      if (n + q < static_cast<int>(mine)) {
        if (!a.rms) {
          mean_next[q] = *mp;
          mp += step;
        }
        rstd_next[q] = *rp;
        rp += step;
      }
    }
  };
  fetch(0);
  fetch_stats(0);
  int half = 0;
  for (int n = 0; n < rows; n += Q, half ^= 1) {
    fetch(half ^ 1);
    asm volatile("cp.async.wait_group 1;" ::: "memory");
    float mean[Q], r[Q], sums[2 * Q];
#pragma unroll
    for (int q = 0; q < Q; ++q) {
      mean[q] = mean_next[q];
      r[q] = rstd_next[q];
    }
    fetch_stats(n + Q);
    // (x - mean) r, the difference first: x and mean may be large and close
    auto columns = [&](int q, int k, int e, const V& xv, const V& gv, uint64_t& g, uint64_t& h) {
      const bool two = 2 * e + 1 < N;
      g = pair_of(gv.get(2 * e), two ? gv.get(2 * e + 1) : 0.f);
      const uint64_t x2 = pair_of(xv.get(2 * e), two ? xv.get(2 * e + 1) : 0.f);
      h = mul2(add2(x2, pair_of(-mean[q], -mean[q])), pair_of(r[q], r[q]));
    };
#pragma unroll
    for (int q = 0; q < Q; ++q) {
      uint64_t sg = pair_of(0.f, 0.f), sgh = sg;
      if (n + q < static_cast<int>(mine)) {
#pragma unroll
        for (int k = 0; k < NV; ++k) {
          if ((k * G + tid) * N < end) {
            V xv = slot_of(half * Q + q, 0, k), gv = slot_of(half * Q + q, 1, k);
            if (RAGGED && k == 0 && tid == 0 && off > 0) {  // what is before the row counts for nothing
              clear_first(xv, off);
              clear_first(gv, off);
            }
#pragma unroll
            for (int e = 0; e < H; ++e) {
              uint64_t g, h;
              columns(q, k, e, xv, gv, g, h);
              dw[k][e] = fma2(g, h, dw[k][e]);
              db[k][e] = add2(db[k][e], g);
              const uint64_t gw = mul2(g, w[k][e]);
              sg = add2(sg, gw);
              sgh = fma2(gw, h, sgh);
            }
          }
        }
      }
      const float2 pg = of_pair(sg), ph = of_pair(sgh);
      sums[2 * q] = pg.x + pg.y;
      sums[2 * q + 1] = ph.x + ph.y;
    }
    group_sums<G, 2 * Q>(sums, part, half);
#pragma unroll
    for (int q = 0; q < Q; ++q) {
      if (n + q < static_cast<int>(mine)) {
        const float m1 = a.rms ? 0.f : -sums[2 * q] * inv_d, m2 = -sums[2 * q + 1] * inv_d;
        const uint64_t c1 = pair_of(m1, m1), c2 = pair_of(m2, m2), rr = pair_of(r[q], r[q]);
#pragma unroll
        for (int k = 0; k < NV; ++k) {
          if ((k * G + tid) * N < end) {
            const V xv = slot_of(half * Q + q, 0, k), gv = slot_of(half * Q + q, 1, k);
            float o[2 * H];
#pragma unroll
            for (int e = 0; e < H; ++e) {
              uint64_t g, h;
              columns(q, k, e, xv, gv, g, h);
              const float2 t = of_pair(mul2(fma2(h, c2, fma2(g, w[k][e], c1)), rr));
              o[2 * e] = t.x;
              o[2 * e + 1] = t.y;
            }
            const int i = (k * G + tid) * N - off;
            if (whole(i)) {
              V p;
              p.set(o);
              store_piece<T, N>(dp + k * G * N, p);
            } else {
#pragma unroll
              for (int e = 0; e < N; ++e)
                if (inside(i + e)) stf(dp, k * G * N + e, o[e]);
            }
          }
        }
        dp += step * a.ld_dx;
      }
    }
  }
  if (!a.partial) return;
  float* pw = a.partial + 2 * row0 * d;  // one pair of rows a group
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    const int i = (k * G + tid) * N - off;
    if (i < d) {
#pragma unroll
      for (int e = 0; e < H; ++e) {
        const float2 p = of_pair(dw[k][e]), q = of_pair(db[k][e]);
        if (!RAGGED || inside(i + 2 * e)) {
          pw[i + 2 * e] = p.x;
          pw[d + i + 2 * e] = q.x;
        }
        if (2 * e + 1 < N && (!RAGGED || inside(i + 2 * e + 1))) {
          pw[i + 2 * e + 1] = p.y;
          pw[d + i + 2 * e + 1] = q.y;
        }
      }
    }
  }
}

// Rows too long for registers: three passes, the later ones from cache.
constexpr int kLong = 1024;
template <typename T>
__global__ void __launch_bounds__(kLong) k_norm_fwd_long(NormArgs a) {
  __shared__ float part[2 * 128];
  const int64_t row = blockIdx.x;
  const T* x = static_cast<const T*>(a.x) + row * a.ld_x;
  T* y = static_cast<T*>(a.y) + row * a.ld_y;
  const int d = static_cast<int>(a.d);
  float mean = 0.f;
  if (!a.rms) {
    float s = 0.f;
    for (int i = threadIdx.x; i < d; i += kLong) s += ldf(x, i);
    mean = group_sum<kLong>(s, part, 0) / d;
  }
  float q = 0.f;
  for (int i = threadIdx.x; i < d; i += kLong) {
    const float c = ldf(x, i) - mean;
    q = fmaf(c, c, q);
  }
  const float r = rsqrtf(group_sum<kLong>(q, part, 1) / d + a.eps);
  for (int i = threadIdx.x; i < d; i += kLong) {
    float v = (ldf(x, i) - mean) * r * param(a.weight, a.param_bf16, i);
    if (a.bias) v += param(a.bias, a.param_bf16, i);
    stf(y, i, v);
  }
  if (threadIdx.x == 0) {
    if (a.mean) a.mean[row] = mean;
    if (a.rstd) a.rstd[row] = r;
  }
}

// The same for the backward; the column sums are in the partial rows of the CTA
// from its first row on. (4096 x 16384 float32: 494 us, 24 % of the bytes' rate; of
// 12288, which fits the ring, 112 us, 81 %.)
template <typename T>
__global__ void __launch_bounds__(kLong) k_norm_bwd_long(NormArgs a) {
  __shared__ float part[2 * 128];
  const int d = static_cast<int>(a.d);
  float* pw = a.partial ? a.partial + 2 * static_cast<int64_t>(blockIdx.x) * d : nullptr;
  int slot = 0;
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const T* x = static_cast<const T*>(a.x) + row * a.ld_x;
    const T* dy = static_cast<const T*>(a.dy) + row * a.ld_dy;
    T* dx = static_cast<T*>(a.dx) + row * a.ld_dx;
    const float mean = a.rms ? 0.f : a.mean[row], r = a.rstd[row];
    const bool first = row == blockIdx.x;
    float sg = 0.f, sgh = 0.f;
    for (int i = threadIdx.x; i < d; i += kLong) {
      const float g = ldf(dy, i), h = (ldf(x, i) - mean) * r, gw = g * param(a.weight, a.param_bf16, i);
      sg += gw;
      sgh = fmaf(gw, h, sgh);
      if (pw) {
        pw[i] = fmaf(g, h, first ? 0.f : pw[i]);
        pw[d + i] = g + (first ? 0.f : pw[d + i]);
      }
    }
    float sums[2] = {sg, sgh};
    group_sums<kLong, 2>(sums, part, slot);
    float2 s = make_float2(sums[0], sums[1]);
    slot ^= 1;
    s.x = a.rms ? 0.f : s.x / d;
    s.y /= d;
    for (int i = threadIdx.x; i < d; i += kLong) {
      const float gw = ldf(dy, i) * param(a.weight, a.param_bf16, i);
      stf(dx, i, r * (gw - s.x - (ldf(x, i) - mean) * r * s.y));
    }
  }
}

// Joins the partial column sums: 32 columns a CTA, each warp takes every 32nd
// part; added up in a fixed order.
__global__ void __launch_bounds__(1024) k_norm_colsum(NormArgs a, int parts) {
  __shared__ float2 s[32][33];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t col = static_cast<int64_t>(blockIdx.x) * 32 + lane;
  float sw = 0.f, sb = 0.f;
  if (col < a.d) {
#pragma unroll 8
    for (int p = warp; p < parts; p += 32) {
      const float* q = a.partial + 2 * static_cast<int64_t>(p) * a.d + col;
      sw += q[0];
      sb += q[a.d];
    }
  }
  s[warp][lane] = make_float2(sw, sb);
  __syncthreads();
  const float2 v = s[lane][warp];  // part `lane` of column `warp`
  sw = v.x;
  sb = v.y;
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) {
    sw += __shfl_xor_sync(0xffffffffu, sw, o);
    sb += __shfl_xor_sync(0xffffffffu, sb, o);
  }
  const int64_t to = static_cast<int64_t>(blockIdx.x) * 32 + warp;
  if (lane == 0 && to < a.d) {
    if (a.dweight) a.dweight[to] = sw;
    if (a.dbias) a.dbias[to] = sb;
  }
}

// How a call's rows are taken: in 16-byte pieces where every row of every operand,
// and the weights, are on 16-byte boundaries and d is whole pieces; else by 16-byte
// granules, where the rows of the inputs lie alike in these; else element by element.
// An output that lies otherwise is written element by element: the order of a row's
// sums, so y, dx and the statistics, do not depend on it, in rows of up to 2048 pieces
// (longer ones are taken element by element then).
enum : int { WHOLE, GRANULES, SINGLES };
int pieces_of(NormArgs& a, bool fwd) {
  const int es = a.bf16 ? 2 : 4;
  auto at = [&](const void* p, int64_t ld) {
    return static_cast<int>(reinterpret_cast<uintptr_t>(p) & 15) | static_cast<int>(ld * es & 15) << 4;
  };
  const int x = at(a.x, a.ld_x);
  a.out16 = x == (fwd ? at(a.y, a.ld_y) : at(a.dx, a.ld_dx));
  a.rows16 = x == 0;
  if (!fwd && x != at(a.dy, a.ld_dy)) return SINGLES;
  return a.rows16 && a.out16 && a.d * es % 16 == 0 && at(a.weight, 0) == 0 && (!fwd || at(a.bias, 0) == 0) ? WHOLE
                                                                                                           : GRANULES;
}
// 16-byte pieces of a row, at most.
template <int N>
int64_t granules(const NormArgs& a) {
  return (a.d + (a.rows16 ? 1 : 2) * (N - 1)) / N;
}
// CTAs whose groups, R a CTA, are a multiple of 8: rows so far apart lie alike in the
// granules. (No more than one row a group: any number.)
template <int R>
int64_t whole_eights(int64_t grid, int64_t rows) {
  constexpr int unit = R >= 8 ? 1 : 8 / R;
  return grid * R >= rows || grid < unit ? grid : grid / unit * unit;
}
// CTAs of a kernel that an SM holds, asked once a device; -1 where that fails. `most`:
// the largest shared memory that it is launched with.
template <typename K>
int ctas_of(K kernel, int threads, int smem, int most, std::atomic<uint64_t>& configured, std::atomic<int>& per_sm, cudaError_t* e) {
  int dev = 0;
  *e = cudaGetDevice(&dev);
  if (*e != cudaSuccess) return -1;
  const uint64_t bit = 1ull << (dev & 63);
  if (!(configured.load() & bit)) {
    *e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
    int n = 0;
    if (*e == cudaSuccess) *e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kernel, threads, smem);
    if (*e != cudaSuccess) return -1;
    per_sm.store(n < 1 ? 1 : n);
    configured.fetch_or(bit);
  }
  return per_sm.load();
}

template <typename T, int N, int NV, int G, int R>
cudaError_t fwd(const NormArgs& a, cudaStream_t s) {
  const unsigned grid = static_cast<unsigned>((a.rows + R - 1) / R);
  k_norm_fwd<T, N, NV, G, R><<<grid, G * R, 0, s>>>(a);
  return cudaGetLastError();
}
template <typename T, int NV, int G, int R>
cudaError_t fwd_ragged(const NormArgs& a, int sms, cudaStream_t s) {
  constexpr int N = 16 / static_cast<int>(sizeof(T)), ring = 2 * NV * 16 * G * R, par = NV * N * 4 * G * R;
  const int smem = ring + (a.bias ? 2 : 1) * (a.param_bf16 ? par / 2 : par);
  auto kernel = k_norm_fwd_ragged<T, NV, G, R>;
  static std::atomic<uint64_t> configured[4];
  static std::atomic<int> per_sm[4];
  cudaError_t e;
  const int which = (a.bias ? 2 : 0) + (a.param_bf16 ? 1 : 0);
  const int n = ctas_of(kernel, G * R, smem, ring + 2 * par, configured[which], per_sm[which], &e);
  if (n < 0) return e;
  const int64_t all = (a.rows + R - 1) / R, most = static_cast<int64_t>(n) * sms;
  const int64_t grid = whole_eights<R>(all < most ? all : most, a.rows);
  kernel<<<static_cast<unsigned>(grid), G * R, smem, s>>>(a);
  return cudaGetLastError();
}
template <typename T, int N>
cudaError_t fwd_n(const NormArgs& a, cudaStream_t s) {
  const int64_t pieces = (a.d + N - 1) / N;
  if (N > 1 && pieces <= 8) return fwd<T, N, 1, 8, 32>(a, s);
  if (N > 1 && pieces <= 16) return fwd<T, N, 1, 16, 16>(a, s);
  if (pieces <= 32) return fwd<T, N, 1, 32, 8>(a, s);
  if (pieces <= 64) return fwd<T, N, 2, 32, 4>(a, s);
  if (pieces <= 128) return fwd<T, N, 4, 32, 4>(a, s);
  if (pieces <= 256) return fwd<T, N, 2, 128, 1>(a, s);
  if (pieces <= 512) return fwd<T, N, 4, 128, 1>(a, s);
  if (pieces <= 1024) return fwd<T, N, 4, 256, 1>(a, s);
  if (pieces <= 2048) return fwd<T, N, 4, 512, 1>(a, s);
  if (pieces <= 4096) return fwd<T, N, 4, 1024, 1>(a, s);
  if (pieces <= 8192) return fwd<T, N, 8, 1024, 1>(a, s);
  k_norm_fwd_long<T><<<static_cast<unsigned>(a.rows), kLong, 0, s>>>(a);
  return cudaGetLastError();
}
template <typename T>
cudaError_t fwd_granules(const NormArgs& a, int sms, cudaStream_t s) {
  constexpr int N = 16 / static_cast<int>(sizeof(T));
  const int64_t pieces = granules<N>(a);
  if (pieces <= 8) return fwd_ragged<T, 1, 8, 32>(a, sms, s);
  if (pieces <= 16) return fwd_ragged<T, 1, 16, 16>(a, sms, s);
  if (pieces <= 32) return fwd_ragged<T, 1, 32, 8>(a, sms, s);
  if (pieces <= 64) return fwd_ragged<T, 2, 32, 4>(a, sms, s);
  if (pieces <= 128) return fwd_ragged<T, 4, 32, 4>(a, sms, s);
  if (pieces <= 256) return fwd_ragged<T, 2, 128, 1>(a, sms, s);
  if (pieces <= 512) return fwd_ragged<T, 4, 128, 1>(a, sms, s);
  if (pieces <= 768) return fwd_ragged<T, 3, 256, 1>(a, sms, s);
  if (pieces <= 1024) return fwd_ragged<T, 4, 256, 1>(a, sms, s);
  if (pieces <= 1536) return fwd_ragged<T, 3, 512, 1>(a, sms, s);
  if (pieces <= 2048) return fwd_ragged<T, 4, 512, 1>(a, sms, s);
  return fwd_n<T, 1>(a, s);
}

// One backward launch: as many CTAs as the SMs hold at a time, so that each walks
// over its share of the rows once. *groups: rows of partial sums it writes.
template <typename T, int N, int NV, int G, int R, bool RAGGED>
cudaError_t bwd(const NormArgs& a, int sms, int* groups, cudaStream_t s) {
  constexpr int slot = 2 * NV * N * static_cast<int>(sizeof(T)) * G * R;
  constexpr int Q = 4 * slot <= 200 * 1024 ? 2 : 1;
  constexpr int smem = 2 * Q * slot;
  auto kernel = k_norm_bwd<T, N, NV, G, R, Q, RAGGED>;
  static std::atomic<uint64_t> configured{0};
  static std::atomic<int> per_sm{0};
  cudaError_t e;
  const int n = ctas_of(kernel, G * R, smem, smem, configured, per_sm, &e);
  if (n < 0) return e;
  // four rows a group at least, where that leaves the SMs at work: a group's
  // partial sums are written and read again
  int64_t grid = (a.rows + R - 1) / R;
  if (grid > sms / 2) grid = grid / 4 > sms / 2 ? grid / 4 : sms / 2;
  const int64_t most = static_cast<int64_t>(n) * sms, room = norm_parts(a, sms) / R;
  grid = grid < most ? grid : most;
  grid = grid < room ? grid : room;
  if (RAGGED) grid = whole_eights<R>(grid, a.rows);
  *groups = static_cast<int>(grid) * R;
  kernel<<<static_cast<unsigned>(grid), G * R, smem, s>>>(a);
  return cudaGetLastError();
}

// A row is given to few threads with several pieces each: the fewer warps join
// their sums, the more rows an SM has under way (163840 x 4096 bf16: 512 threads
// a row 811 us, 256 with two pieces 679 us).
template <typename T, int N, bool RAGGED>
cudaError_t bwd_n(const NormArgs& a, int sms, int* groups, cudaStream_t s) {
  const int64_t pieces = RAGGED ? granules<N>(a) : (a.d + N - 1) / N;
  if (pieces <= 32) return bwd<T, N, 1, 32, 8, RAGGED>(a, sms, groups, s);
  if (pieces <= 64) return bwd<T, N, 2, 32, 8, RAGGED>(a, sms, groups, s);
  if (pieces <= 128) return bwd<T, N, 2, 64, 4, RAGGED>(a, sms, groups, s);
  if (pieces <= 256) return bwd<T, N, 2, 128, 1, RAGGED>(a, sms, groups, s);
  if (pieces <= 384) return bwd<T, N, 3, 128, 1, RAGGED>(a, sms, groups, s);
  if (pieces <= 512) return bwd<T, N, 2, 256, 1, RAGGED>(a, sms, groups, s);
  if (pieces <= 768) return bwd<T, N, 3, 256, 1, RAGGED>(a, sms, groups, s);
  if (pieces <= 1024) return bwd<T, N, 2, 512, 1, RAGGED>(a, sms, groups, s);
  if (pieces <= 1536) return bwd<T, N, 3, 512, 1, RAGGED>(a, sms, groups, s);
  if (pieces <= 2048) return bwd<T, N, 4, 512, 1, RAGGED>(a, sms, groups, s);
  if constexpr (N > 1) {
    if (pieces <= 3 * 1024) return bwd<T, N, 3, 1024, 1, RAGGED>(a, sms, groups, s);
  } else {
    if (pieces <= 4096) return bwd<T, N, 4, 1024, 1, RAGGED>(a, sms, groups, s);
  }
  const int64_t most = 2ll * sms;
  *groups = static_cast<int>(a.rows < most ? a.rows : most);
  k_norm_bwd_long<T><<<*groups, kLong, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace

// Rows of partial column sums that the workspace holds.
int norm_parts(const NormArgs& a, int sms) {
  // A bound that does not depend on addresses (the workspace is sized before they
  // are known): up to 8 groups a CTA, 32 an SM for short rows and 8 for others.
  const int64_t most = 8ll * sms * (a.d <= 512 ? 4 : 1), need = (a.rows + 7) / 8 * 8;
  return static_cast<int>(need < 8 ? 8 : need < most ? need : most);
}

cudaError_t launch_norm_fwd(const NormArgs& args, int sms, cudaStream_t s) {
  NormArgs a = args;
  const int how = pieces_of(a, true);
  if (a.bf16)
    return how == WHOLE      ? fwd_n<__nv_bfloat16, 8>(a, s)
           : how == GRANULES ? fwd_granules<__nv_bfloat16>(a, sms, s)
                             : fwd_n<__nv_bfloat16, 1>(a, s);
  return how == WHOLE ? fwd_n<float, 4>(a, s) : how == GRANULES ? fwd_granules<float>(a, sms, s) : fwd_n<float, 1>(a, s);
}

cudaError_t launch_norm_bwd(const NormArgs& args, int sms, int* groups, cudaStream_t s) {
  NormArgs a = args;
  const int how = pieces_of(a, false);
  if (a.bf16)
    return how == WHOLE      ? bwd_n<__nv_bfloat16, 8, false>(a, sms, groups, s)
           : how == GRANULES ? bwd_n<__nv_bfloat16, 8, true>(a, sms, groups, s)
                             : bwd_n<__nv_bfloat16, 1, false>(a, sms, groups, s);
  return how == WHOLE      ? bwd_n<float, 4, false>(a, sms, groups, s)
         : how == GRANULES ? bwd_n<float, 4, true>(a, sms, groups, s)
                           : bwd_n<float, 1, false>(a, sms, groups, s);
}

cudaError_t launch_norm_colsum(const NormArgs& a, int groups, cudaStream_t s) {
  k_norm_colsum<<<static_cast<unsigned>((a.d + 31) / 32), 1024, 0, s>>>(a, groups);
  return cudaGetLastError();
}

}  // namespace grpo
