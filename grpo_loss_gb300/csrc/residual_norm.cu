// The norms behind and before a block of a model, with the block's gate and residual
// scale:  p = post_norm(x) or x,  h = residual + scale gate p,  y = norm(h).
// Backward, of dy and dh:
//   g  = dh + norm'(dy)             the gradient of h, and of the residual
//   q  = scale gate g               that of p;  dgate = sum over its rows of scale g p
//   dx = post_norm'(q) or q
// with norm'(v) = r (v w - mean(v w) - k mean(v w k)), k = (h - m) r.
// Bound by memory: the forward reads x and the residual and writes h and y, the backward
// (residual_norm_bwd.cuh) reads dy, dh, h and x and writes both gradients, each once:
// 163840 x 4096 bf16, RMS with a post norm, 754 us forward (7.1 TB/s) and 1210 backward (6.7).
// Here stand the forward, the backward with gates of another type than the rows, and the join
// of the walkers' column sums. Four ways for a row: registers, in whole 16-byte pieces; pieces
// that are cut (ROWS_SHIFTED of the backward); staged and taken column by column; and, what is
// too long for these, a CTA a row with h in shared memory.
#include <cuda_bf16.h>

#include "residual_norm_bwd.cuh"

namespace grpo {

namespace {

__device__ __forceinline__ void put(void* p, int bf16, int64_t i, float v) {
  if (bf16) static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(v);
  else static_cast<float*>(p)[i] = v;
}

__device__ float gate_of(const ResNormArgs& a, int64_t row, int i) {
  return a.gate ? a.scale * param(a.gate, a.gate_bf16, row / a.gate_rows * a.ld_gate + i) : a.scale;
}

// A group of G threads takes a row, R rows a CTA; each thread holds NV pieces of N values
// of it, in registers from the loads to y.
template <typename T, int N, int NV, int G, int R, bool POST>
__global__ void __launch_bounds__(G * R) k_resnorm_fwd(ResNormArgs a) {
  __shared__ float part[2 * 128];
  const int tid = threadIdx.x % G, d = static_cast<int>(a.d);
  const int64_t row = static_cast<int64_t>(blockIdx.x) * R + threadIdx.x / G;
  const bool live = row < a.rows;  // every thread takes part in the barriers
  const int64_t from = live ? row : 0;
  const T* x = static_cast<const T*>(a.x) + from * a.ld_x;
  const T* res = static_cast<const T*>(a.residual) + from * a.ld_res;
  auto column = [&](int k) { return (k * G + tid) * N; };
  Piece<T, N> vx[NV], vr[NV];
#pragma unroll
  for (int k = 0; k < NV; ++k)
    if (column(k) < d) {
      vx[k] = load_piece<T, N>(x + column(k));
      vr[k] = load_piece<T, N>(res + column(k));
    }
  const float inv_d = 1.f / d;
  float pm = 0.f, pr = 1.f;
  if constexpr (POST) {
    if (!a.rms) {
      float s = 0.f;
#pragma unroll
      for (int k = 0; k < NV; ++k)
        if (column(k) < d)
#pragma unroll
          for (int e = 0; e < N; ++e) s += vx[k].get(e);
      pm = group_sum<G>(s, part, 0) * inv_d;
    }
    float q = 0.f;
#pragma unroll
    for (int k = 0; k < NV; ++k)
      if (column(k) < d)
#pragma unroll
        for (int e = 0; e < N; ++e) {
          const float c = vx[k].get(e) - pm;
          q = fmaf(c, c, q);
        }
    pr = rsqrtf(group_sum<G>(q, part, 1) * inv_d + a.eps);
  }
  float h[NV][N];
  float s = 0.f;
  const int64_t gate_at = a.gate ? from / a.gate_rows * a.ld_gate : 0;
#pragma unroll
  for (int k = 0; k < NV; ++k)
    if (column(k) < d) {
      float p[N], w[N];
#pragma unroll
      for (int e = 0; e < N; ++e) p[e] = vx[k].get(e);
      if constexpr (POST) {
        load_params<N>(a.post_weight, a.param_bf16, column(k), w);
#pragma unroll
        for (int e = 0; e < N; ++e) p[e] = (p[e] - pm) * pr * w[e];
        if (a.post_bias) {
          load_params<N>(a.post_bias, a.param_bf16, column(k), w);
#pragma unroll
          for (int e = 0; e < N; ++e) p[e] += w[e];
        }
      }
      if (a.gate) {
        const char* g = static_cast<const char*>(a.gate) + gate_at * (a.gate_bf16 ? 2 : 4);
        load_params<N>(g, a.gate_bf16, column(k), w);
#pragma unroll
        for (int e = 0; e < N; ++e) p[e] *= w[e];
      }
#pragma unroll
      for (int e = 0; e < N; ++e) {
        h[k][e] = fmaf(a.scale, p[e], vr[k].get(e));
        s += h[k][e];
      }
      Piece<T, N> out;
      out.set(h[k]);
      if (live) store_piece<T, N>(static_cast<T*>(a.h_out) + row * a.ld_h + column(k), out);
    }
  float m = 0.f;
  if (!a.rms) m = group_sum<G>(s, part, 0) * inv_d;
  float q = 0.f;
#pragma unroll
  for (int k = 0; k < NV; ++k)
    if (column(k) < d)
#pragma unroll
      for (int e = 0; e < N; ++e) {
        const float c = h[k][e] - m;
        q = fmaf(c, c, q);
      }
  // (a slot is written again behind another slot's barrier)
  const float r = rsqrtf(group_sum<G>(q, part, POST && a.rms ? 0 : 1) * inv_d + a.eps);
  if (!live) return;
#pragma unroll
  for (int k = 0; k < NV; ++k)
    if (column(k) < d) {
      float w[N];
      load_params<N>(a.weight, a.param_bf16, column(k), w);
#pragma unroll
      for (int e = 0; e < N; ++e) h[k][e] = (h[k][e] - m) * r * w[e];
      if (a.bias) {
        load_params<N>(a.bias, a.param_bf16, column(k), w);
#pragma unroll
        for (int e = 0; e < N; ++e) h[k][e] += w[e];
      }
      Piece<T, N> out;
      out.set(h[k]);
      store_piece<T, N>(static_cast<T*>(a.y) + row * a.ld_y + column(k), out);
    }
  if (tid == 0) {
    if (a.mean) a.mean[row] = m;
    if (a.rstd) a.rstd[row] = r;
    if (a.post_mean) a.post_mean[row] = pm;
    if (a.post_rstd) a.post_rstd[row] = pr;
  }
}

// Rows that do not come in whole pieces: a group of threads walks over rows, each staged by
// the granules it lies in while the one before is worked on; a thread's N columns are G
// apart. The weights of its columns stay in registers; the biases, and a gate as long as it
// is shared, in shared memory, each thread its own. (99900 x 1001 bf16, RMS with a post norm:
// 194 us; eight columns a thread, and what is there asked for column by column, 269; single
// elements from global memory 451.)
struct StridedLayout {
  int pitch, arrays;                     // staged rows: x, residual and a gate of the same type
  bool gate_staged;
  int gate, bias, post_bias, bytes;      // offsets of the vectors, -1 where there is none; a group's size
};
__host__ __device__ __forceinline__ StridedLayout strided_layout(const ResNormArgs& a) {
  StridedLayout l;
  const int d = static_cast<int>(a.d);
  l.pitch = staged_pitch(d, a.bf16 ? 2 : 4);
  l.gate_staged = a.gate && a.gate_rows == 1 && a.gate_bf16 == a.bf16;
  l.arrays = l.gate_staged ? 3 : 2;
  int at = 2 * l.arrays * l.pitch;
  auto take = [&](bool there) {
    const int from = there ? at : -1;
    if (there) at += (d * 4 + 15) / 16 * 16;
    return from;
  };
  l.gate = take(a.gate && !l.gate_staged);
  l.bias = take(a.bias != nullptr);
  l.post_bias = take(a.post_bias != nullptr);
  l.bytes = at;
  return l;
}
template <typename T, int N, int G, int R, bool POST>
__global__ void __launch_bounds__(G * R) k_resnorm_fwd_strided(ResNormArgs a, int walkers) {
  static_assert(R == 1 || G == 32, "");
  extern __shared__ __align__(16) unsigned char staged_raw[];
  __shared__ float part[2 * 128];
  const StridedLayout l = strided_layout(a);
  const int tid = threadIdx.x % G, d = static_cast<int>(a.d), pitch = l.pitch;
  unsigned char* const staged = staged_raw + threadIdx.x / G * l.bytes;  // the group's
  const int64_t walker = static_cast<int64_t>(blockIdx.x) * R + threadIdx.x / G;
  if (R > 1 && walker >= walkers) return;  // (no barrier but the warp's)
  const int64_t from = first_row(a.rows, walker, walkers), to = first_row(a.rows, walker + 1, walkers);
  const float inv_d = 1.f / d;
  auto column = [&](int i) { return i * G + tid; };
  float w[N], pw[N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    w[i] = column(i) < d ? param(a.weight, a.param_bf16, column(i)) : 0.f;
    if (POST) pw[i] = column(i) < d ? param(a.post_weight, a.param_bf16, column(i)) : 0.f;
  }
  auto vector = [&](int at) { return reinterpret_cast<float*>(staged + at); };
  auto keep = [&](int place, const void* p, int bf16, int64_t first) {
    for (int i = 0; i < N; ++i)
      if (column(i) < d) vector(place)[column(i)] = param(p, bf16, first + column(i));
  };
  if (l.bias >= 0) keep(l.bias, a.bias, a.param_bf16, 0);
  if (POST && l.post_bias >= 0) keep(l.post_bias, a.post_bias, a.param_bf16, 0);
  auto fetch = [&](int64_t row, int half) {
    if (row < to) {
      const T *x = static_cast<const T*>(a.x), *res = static_cast<const T*>(a.residual), *gate = static_cast<const T*>(a.gate);
      stage_row<T, G>(staged + l.arrays * half * pitch, x + row * a.ld_x, x, d, tid);
      stage_row<T, G>(staged + (l.arrays * half + 1) * pitch, res + row * a.ld_res, res, d, tid);
      if (l.gate_staged) stage_row<T, G>(staged + (l.arrays * half + 2) * pitch, gate + row * a.ld_gate, gate, d, tid);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  auto values = [&](int which, const void* base, int64_t first) {
    const int off = static_cast<int>(reinterpret_cast<uintptr_t>(static_cast<const T*>(base) + first) & 15);
    return reinterpret_cast<const T*>(staged + which * pitch + off);
  };
  fetch(from, 0);
  int half = 0, slot = 0;
  int64_t gate_to = from;  // the rows that the gate in shared memory is for end here
  auto sum = [&](float v) {
    slot ^= 1;
    return group_sum<G>(v, part, slot);
  };
  for (int64_t row = from; row < to; ++row, half ^= 1) {
    // this row is here, of every thread's copies, and the last one's place is free
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    if constexpr (G == 32) __syncwarp();
    else __syncthreads();
    fetch(row + 1, half ^ 1);
    if (l.gate >= 0 && row >= gate_to) {
      const int64_t q = row / a.gate_rows;
      gate_to = (q + 1) * a.gate_rows;
      keep(l.gate, a.gate, a.gate_bf16, q * a.ld_gate);
    }
    const T *x = values(l.arrays * half, a.x, row * a.ld_x), *res = values(l.arrays * half + 1, a.residual, row * a.ld_res);
    float h[N];
#pragma unroll
    for (int i = 0; i < N; ++i) h[i] = column(i) < d ? ldf(x, column(i)) : 0.f;
    // (0 beside the row; what is not there for any column is asked for once)
    auto centred = [&](float mean) {
      float q = 0.f;
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const float c = column(i) < d ? h[i] - mean : 0.f;
        q = fmaf(c, c, q);
      }
      return rsqrtf(sum(q) * inv_d + a.eps);
    };
    auto mean_of = [&] {
      float s = 0.f;
#pragma unroll
      for (int i = 0; i < N; ++i) s += h[i];
      return sum(s) * inv_d;
    };
    float pm = 0.f, pr = 1.f;
    if constexpr (POST) {
      if (!a.rms) pm = mean_of();
      pr = centred(pm);
#pragma unroll
      for (int i = 0; i < N; ++i) h[i] = (h[i] - pm) * pr * pw[i];  // (pw: 0 beside the row)
      if (l.post_bias >= 0)
#pragma unroll
        for (int i = 0; i < N; ++i)
          if (column(i) < d) h[i] += vector(l.post_bias)[column(i)];
    }
    if (l.gate >= 0) {
#pragma unroll
      for (int i = 0; i < N; ++i)
        if (column(i) < d) h[i] *= vector(l.gate)[column(i)];
    } else if (l.gate_staged) {
      const T* gate = values(l.arrays * half + 2, a.gate, row * a.ld_gate);
#pragma unroll
      for (int i = 0; i < N; ++i)
        if (column(i) < d) h[i] *= ldf(gate, column(i));
    }
    T* const to_h = static_cast<T*>(a.h_out) + row * a.ld_h;
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (column(i) < d) {
        h[i] = fmaf(a.scale, h[i], ldf(res, column(i)));
        stf(to_h, column(i), h[i]);
      }
    const float m = a.rms ? 0.f : mean_of(), r = centred(m);
    T* const to_y = static_cast<T*>(a.y) + row * a.ld_y;
#pragma unroll
    for (int i = 0; i < N; ++i) h[i] = (h[i] - m) * r * w[i];
    if (l.bias >= 0)
#pragma unroll
      for (int i = 0; i < N; ++i)
        if (column(i) < d) h[i] += vector(l.bias)[column(i)];
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (column(i) < d) stf(to_y, column(i), h[i]);
    if (tid == 0) {
      if (a.mean) a.mean[row] = m;
      if (a.rstd) a.rstd[row] = r;
      if (a.post_mean) a.post_mean[row] = pm;
      if (a.post_rstd) a.post_rstd[row] = pr;
    }
  }
}

// Rows that lie in their granules alike: a walker's threads have whole pieces that keep their
// columns (see the backward). The weights of these stay in registers; the biases, and a gate
// that all rows share, in shared memory, each thread its own. (30000 x 2881 bf16, RMS with a
// post norm: 173 us, as strided rows 277; with two pieces a thread 203.)
struct ShiftedLayout {
  bool gate_rows;
  int arrays, bias, post_bias, gate, vectors;  // staged rows; the vectors' places, and how many
};
__host__ __device__ __forceinline__ ShiftedLayout shifted_layout(const ResNormArgs& a) {
  ShiftedLayout l;
  l.gate_rows = a.gate && a.gate_rows == 1;
  l.arrays = l.gate_rows ? 3 : 2;
  l.bias = 0;
  l.post_bias = l.bias + (a.bias != nullptr);
  l.gate = l.post_bias + (a.post_bias != nullptr);
  l.vectors = l.gate + (a.gate && !l.gate_rows);
  return l;
}
template <typename T, int N, int NV, int G, int R, bool POST>
__global__ void __launch_bounds__(G * R) k_resnorm_fwd_shifted(ResNormArgs a, int walkers, int step) {
  extern __shared__ __align__(16) unsigned char ring_raw[];
  __shared__ float part[2 * 128];
  using V = Piece<T, N>;
  constexpr int es = static_cast<int>(sizeof(T)), THREADS = G * R;
  const int tid = threadIdx.x % G, d = static_cast<int>(a.d);
  const int64_t walker = static_cast<int64_t>(blockIdx.x) * R + threadIdx.x / G;
  const Walk walk = shifted_walk(a, a.ld_x, walker, walkers, step, es);
  const float inv_d = 1.f / d;
  const ShiftedLayout l = shifted_layout(a);
  const bool gate_rows = l.gate_rows;
  auto column = [&](int k) { return (k * G + tid) * N - walk.shift; };
  auto there = [&](int k) { return column(k) < d; };
  auto inside = [&](int k, int e) { return static_cast<unsigned>(column(k) + e) < static_cast<unsigned>(d); };
  auto inside_all = [&](int k) { return column(k) >= 0 && column(k) + N <= d; };
  V* const ring = reinterpret_cast<V*>(ring_raw) + threadIdx.x;  // [2][x, residual, a gate][NV][threads]
  auto slot_of = [&](int half, int which, int k) -> V& { return ring[((half * l.arrays + which) * NV + k) * THREADS]; };
  float* const vectors = reinterpret_cast<float*>(ring_raw + 2 * l.arrays * NV * 16 * THREADS) + threadIdx.x;  // [vectors][NV][N][threads]
  auto kept = [&](int which, int k, int e) -> float& { return vectors[((which * NV + k) * N + e) * THREADS]; };
  float w[NV][N], pw[NV][N];
#pragma unroll
  for (int k = 0; k < NV; ++k)
#pragma unroll
    for (int e = 0; e < N; ++e) {
      const bool in = inside(k, e);
      const int c = column(k) + e;
      w[k][e] = in ? param(a.weight, a.param_bf16, c) : 0.f;
      if (POST) pw[k][e] = in ? param(a.post_weight, a.param_bf16, c) : 0.f;
      if (a.bias) kept(l.bias, k, e) = in ? param(a.bias, a.param_bf16, c) : 0.f;
      if (POST && a.post_bias) kept(l.post_bias, k, e) = in ? param(a.post_bias, a.param_bf16, c) : 0.f;
      if (a.gate && !gate_rows) kept(l.gate, k, e) = in ? param(a.gate, a.gate_bf16, c) : 0.f;
    }
  auto row_at = [&](int n) { return walk.from + static_cast<int64_t>(n) * step; };
  auto fetch = [&](int n, int half) {
    if (n < walk.mine) {
      const int64_t row = row_at(n);
      auto copy = [&](int which, const void* p, int64_t ld) {
        const T* const q = static_cast<const T*>(p) + row * ld;
#pragma unroll
        for (int k = 0; k < NV; ++k)
          if (there(k)) copy_async_zero(&slot_of(half, which, k), q + column(k), min(16, (d - column(k)) * es));
      };
      copy(0, a.x, a.ld_x);
      copy(1, a.residual, a.ld_res);
      if (gate_rows) copy(2, a.gate, a.ld_gate);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  int slot = 0;
  auto sum = [&](float v) {
    slot ^= 1;
    return group_sum<G>(v, part, slot);
  };
  fetch(0, 0);
  int half = 0;
  for (int n = 0; n < walk.turns; ++n, half ^= 1) {
    fetch(n + 1, half ^ 1);
    asm volatile("cp.async.wait_group 1;" ::: "memory");
    const bool live = n < walk.mine;
    const int64_t row = row_at(n);
    if (live && column(0) < 0)  // the row before
      for (int which = 0; which < 2 + gate_rows; ++which)
        for (int i = 0; i < walk.shift; ++i) reinterpret_cast<T*>(&slot_of(half, which, 0))[i] = T(0.f);
    float h[NV][N];  // 0 beside the row
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      V v;
      if (live && there(k)) v = slot_of(half, 0, k);
#pragma unroll
      for (int e = 0; e < N; ++e) h[k][e] = live && there(k) ? v.get(e) : 0.f;
    }
    auto mean_of = [&] {
      float s = 0.f;
#pragma unroll
      for (int k = 0; k < NV; ++k)
#pragma unroll
        for (int e = 0; e < N; ++e) s += h[k][e];
      return sum(s) * inv_d;
    };
    auto rstd_of = [&](float mean) {
      float q = 0.f;
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        if (a.rms || inside_all(k)) {
#pragma unroll
          for (int e = 0; e < N; ++e) q = fmaf(h[k][e] - mean, h[k][e] - mean, q);
        } else {
#pragma unroll
          for (int e = 0; e < N; ++e)
            if (inside(k, e)) q = fmaf(h[k][e] - mean, h[k][e] - mean, q);
        }
      }
      return rsqrtf(sum(q) * inv_d + a.eps);
    };
    auto store = [&](void* p, int64_t ld, int k, const float* v) {
      T* const to = static_cast<T*>(p) + row * ld + column(k);
      if (inside_all(k)) {
        V o;
        o.set(v);
        store_piece(to, o);
      } else {
#pragma unroll
        for (int e = 0; e < N; ++e)
          if (inside(k, e)) stf(to, e, v[e]);
      }
    };
    float pm = 0.f, pr = 1.f;
    if constexpr (POST) {
      if (!a.rms) pm = mean_of();
      pr = rstd_of(pm);
#pragma unroll
      for (int k = 0; k < NV; ++k)
#pragma unroll
        for (int e = 0; e < N; ++e) {
          h[k][e] = (h[k][e] - pm) * pr * pw[k][e];
          if (a.post_bias) h[k][e] += kept(l.post_bias, k, e);
        }
    }
#pragma unroll
    for (int k = 0; k < NV; ++k)
      if (live && there(k)) {
        if (gate_rows) {
          const V g = slot_of(half, 2, k);
#pragma unroll
          for (int e = 0; e < N; ++e) h[k][e] *= g.get(e);
        } else if (a.gate) {
#pragma unroll
          for (int e = 0; e < N; ++e) h[k][e] *= kept(l.gate, k, e);
        }
        const V v = slot_of(half, 1, k);
#pragma unroll
        for (int e = 0; e < N; ++e) h[k][e] = fmaf(a.scale, h[k][e], v.get(e));
        store(a.h_out, a.ld_h, k, h[k]);
      }
    const float m = a.rms ? 0.f : mean_of(), r = rstd_of(m);
    if (!live) continue;
#pragma unroll
    for (int k = 0; k < NV; ++k)
      if (there(k)) {
#pragma unroll
        for (int e = 0; e < N; ++e) {
          h[k][e] = (h[k][e] - m) * r * w[k][e];
          if (a.bias) h[k][e] += kept(l.bias, k, e);
        }
        store(a.y, a.ld_y, k, h[k]);
      }
    if (tid == 0) {
      if (a.mean) a.mean[row] = m;
      if (a.rstd) a.rstd[row] = r;
      if (a.post_mean) a.post_mean[row] = pm;
      if (a.post_rstd) a.post_rstd[row] = pr;
    }
  }
}

// Rows too long for registers: h stands in shared memory, x is read again, mostly from L2;
// kMany columns of a thread at a time, so that their loads are in flight together. (9000 x
// 16383 bf16, RMS with a post norm, floor 176 us: 620: the loads of one batch are waited for
// before the next.)
constexpr int kLong = 512, kWide = 1024, kMany = 4;
// body(u, i) of a thread's kMany columns i from i0 on, of a CTA of THREADS.
template <int THREADS, typename F>
__device__ __forceinline__ void columns(int d, int i0, F body) {
#pragma unroll
  for (int u = 0; u < kMany; ++u) {
    const int i = i0 + u * THREADS;
    if (i < d) body(u, i);
  }
}
template <typename T>
__global__ void __launch_bounds__(kLong) k_resnorm_fwd_long(ResNormArgs a) {
  extern __shared__ float h[];
  __shared__ float part[2 * 128];
  const int d = static_cast<int>(a.d);
  const float inv_d = 1.f / d;
  const int64_t row = blockIdx.x;
  const T *x = static_cast<const T*>(a.x) + row * a.ld_x, *res = static_cast<const T*>(a.residual) + row * a.ld_res;
  int slot = 0;
  auto sum = [&](float v) {
    slot ^= 1;
    return group_sum<kLong>(v, part, slot);
  };
  float pm = 0.f, pr = 1.f;
  if (a.post_weight) {
    float s = 0.f;
    if (!a.rms) {
#pragma unroll 4
      for (int i = threadIdx.x; i < d; i += kLong) s += ldf(x, i);
      pm = sum(s) * inv_d;
    }
    s = 0.f;
#pragma unroll 4
    for (int i = threadIdx.x; i < d; i += kLong) {
      const float c = ldf(x, i) - pm;
      s = fmaf(c, c, s);
    }
    pr = rsqrtf(sum(s) * inv_d + a.eps);
  }
  T* const to_h = static_cast<T*>(a.h_out) + row * a.ld_h;
  float s = 0.f;
  for (int i0 = threadIdx.x; i0 < d; i0 += kLong * kMany) {
    float p[kMany], e[kMany], w[kMany], b[kMany], f[kMany];
    columns<kLong>(d, i0, [&](int u, int i) {
      p[u] = ldf(x, i), e[u] = ldf(res, i), f[u] = gate_of(a, row, i);
      w[u] = a.post_weight ? param(a.post_weight, a.param_bf16, i) : 1.f;
      b[u] = a.post_bias ? param(a.post_bias, a.param_bf16, i) : 0.f;
    });
    columns<kLong>(d, i0, [&](int u, int i) {
      h[i] = fmaf(f[u], (p[u] - pm) * pr * w[u] + b[u], e[u]);
      s += h[i];
      stf(to_h, i, h[i]);
    });
  }
  const float m = a.rms ? 0.f : sum(s) * inv_d;
  s = 0.f;
  for (int i = threadIdx.x; i < d; i += kLong) s = fmaf(h[i] - m, h[i] - m, s);
  const float r = rsqrtf(sum(s) * inv_d + a.eps);
  T* const to_y = static_cast<T*>(a.y) + row * a.ld_y;
  for (int i0 = threadIdx.x; i0 < d; i0 += kLong * kMany) {
    float w[kMany], b[kMany];
    columns<kLong>(d, i0, [&](int u, int i) { w[u] = param(a.weight, a.param_bf16, i), b[u] = a.bias ? param(a.bias, a.param_bf16, i) : 0.f; });
    columns<kLong>(d, i0, [&](int u, int i) { stf(to_y, i, (h[i] - m) * r * w[u] + b[u]); });
  }
  if (threadIdx.x == 0) {
    if (a.mean) a.mean[row] = m;
    if (a.rstd) a.rstd[row] = r;
    if (a.post_mean) a.post_mean[row] = pm;
    if (a.post_rstd) a.post_rstd[row] = pr;
  }
}

// The backward with a gate for each row that is of another type than these: a CTA a row, g in
// shared memory. `fit` column sums stand beside g, in the order of their first use; others are
// added up in their partial rows.
template <typename T>
__global__ void __launch_bounds__(kWide) k_resnorm_bwd_long(ResNormArgs a, int walkers, int fit) {
  extern __shared__ float g[];
  __shared__ float red[2 * 256];
  const int d = static_cast<int>(a.d);
  const float inv_d = 1.f / d;
  const int64_t from = first_row(a.rows, blockIdx.x, walkers), to = first_row(a.rows, blockIdx.x + 1, walkers);
  auto part = [&](int which) { return a.partial + (static_cast<int64_t>(which) * walkers + blockIdx.x) * d; };
  int used = 0;
  auto place = [&](bool there, float* global) {
    if (!there) return static_cast<float*>(nullptr);
    if (used == fit) return global;
    return g + static_cast<int64_t>(++used) * d;
  };
  float* const pw = place(a.dweight, part(a.at_dw));
  float* const ppw = place(a.dpost_weight, part(a.at_dpw));
  float* const pb = place(a.dbias, part(a.at_db));
  float* const ppb = place(a.dpost_bias, part(a.at_dpb));
  auto row_of = [](const void* p, int64_t ld, int64_t row) { return static_cast<const T*>(p) + row * ld; };
  int slot = 0;
  for (int64_t row = from; row < to; ++row) {
    const bool first = row == from;
    const float m = a.rms ? 0.f : a.mean[row], r = a.rstd[row];
    const T *dy = row_of(a.dy, a.ld_dy, row), *h = row_of(a.h, a.ld_h, row), *dh = a.dh ? row_of(a.dh, a.ld_dh, row) : nullptr;
    const T* x = row_of(a.x, a.ld_x, row);
    float s[2] = {0.f, 0.f};
    for (int i0 = threadIdx.x; i0 < d; i0 += kWide * kMany) {
      float v[kMany], k[kMany], w[kMany];
      columns<kWide>(d, i0, [&](int u, int i) { v[u] = ldf(dy, i), k[u] = ldf(h, i), w[u] = param(a.weight, a.param_bf16, i); });
      columns<kWide>(d, i0, [&](int u, int i) {
        const float hat = (k[u] - m) * r, vw = v[u] * w[u];
        s[0] += vw;
        s[1] = fmaf(vw, hat, s[1]);
        if (pw) pw[i] = fmaf(v[u], hat, first ? 0.f : pw[i]);
        if (pb) pb[i] = v[u] + (first ? 0.f : pb[i]);
      });
    }
    group_sums<kWide, 2>(s, red, slot);
    slot ^= 1;
    const float c1 = a.rms ? 0.f : s[0] * inv_d, c2 = s[1] * inv_d;
    T* const dres = static_cast<T*>(a.dres) + row * a.ld_dres;
    for (int i0 = threadIdx.x; i0 < d; i0 += kWide * kMany) {
      float v[kMany], k[kMany], w[kMany], e[kMany];
      columns<kWide>(d, i0, [&](int u, int i) {
        v[u] = ldf(dy, i), k[u] = ldf(h, i), w[u] = param(a.weight, a.param_bf16, i);
        e[u] = dh ? ldf(dh, i) : 0.f;
      });
      columns<kWide>(d, i0, [&](int u, int i) {
        g[i] = fmaf(r, v[u] * w[u] - c1 - (k[u] - m) * r * c2, e[u]);
        stf(dres, i, g[i]);
      });
    }
    if (!a.dx && !a.dgate && !a.dpost_weight && !a.dpost_bias) continue;
    const float pm = a.post_weight && !a.rms ? a.post_mean[row] : 0.f, pr = a.post_weight ? a.post_rstd[row] : 1.f;
    s[0] = s[1] = 0.f;
    for (int i0 = threadIdx.x; i0 < d; i0 += kWide * kMany) {
      float xs[kMany], w[kMany], gt[kMany], pb_[kMany];
      columns<kWide>(d, i0, [&](int u, int i) {
        xs[u] = ldf(x, i);
        w[u] = a.post_weight ? param(a.post_weight, a.param_bf16, i) : 1.f;
        gt[u] = gate_of(a, row, i);
        pb_[u] = a.post_bias && a.dgate ? param(a.post_bias, a.param_bf16, i) : 0.f;
      });
      columns<kWide>(d, i0, [&](int u, int i) {
        const float k = (xs[u] - pm) * pr;
        if (a.dgate) put(a.dgate, a.gate_bf16, row * a.ld_dgate + i, a.scale * g[i] * fmaf(k, w[u], pb_[u]));
        const float qv = g[i] * gt[u];
        g[i] = qv;
        if (a.post_weight) {
          s[0] = fmaf(qv, w[u], s[0]);
          s[1] = fmaf(qv * w[u], k, s[1]);
          if (ppw) ppw[i] = fmaf(qv, k, first ? 0.f : ppw[i]);
          if (ppb) ppb[i] = qv + (first ? 0.f : ppb[i]);
        }
      });
    }
    if (a.post_weight) {
      group_sums<kWide, 2>(s, red, slot);
      slot ^= 1;
      s[0] = a.rms ? 0.f : s[0] * inv_d;
      s[1] *= inv_d;
    }
    if (!a.dx) continue;
    T* const dx = static_cast<T*>(a.dx) + row * a.ld_dx;
    for (int i0 = threadIdx.x; i0 < d; i0 += kWide * kMany) {
      float xs[kMany], w[kMany];
      if (a.post_weight) columns<kWide>(d, i0, [&](int u, int i) { xs[u] = ldf(x, i), w[u] = param(a.post_weight, a.param_bf16, i); });
      columns<kWide>(d, i0, [&](int u, int i) {
        stf(dx, i, a.post_weight ? pr * (g[i] * w[u] - s[0] - (xs[u] - pm) * pr * s[1]) : g[i]);
      });
    }
  }
  // (each thread's own columns)
  auto leave = [&](const float* sums, bool there, int which) {
    if (!there || sums == part(which)) return;
    for (int i = threadIdx.x; i < d; i += kWide) part(which)[i] = sums[i];
  };
  leave(pw, a.dweight, a.at_dw);
  leave(ppw, a.dpost_weight, a.at_dpw);
  leave(pb, a.dbias, a.at_db);
  leave(ppb, a.dpost_bias, a.at_dpb);
}

// Joins the walkers' partial sums of a column: one after the other in a fixed order.
// blockIdx.y: the parameters' sums, then the gates that several walkers share.
__global__ void __launch_bounds__(1024) k_resnorm_join(ResNormArgs a, int walkers) {
  __shared__ float s[32][33];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t col = static_cast<int64_t>(blockIdx.x) * 32 + lane, d = a.d;
  int which = a.at_head, tail = -1;
  int64_t w0 = 0, w1 = walkers - 1;
  float* to;
  if (static_cast<int>(blockIdx.y) < a.at_head) {
    which = blockIdx.y;
    to = which == a.at_dw ? a.dweight : which == a.at_db ? a.dbias : which == a.at_dpw ? a.dpost_weight : a.dpost_bias;
  } else {
    const int64_t q = blockIdx.y - a.at_head, q0 = q * a.gate_rows;
    w0 = walker_of(a.rows, q0, walkers);
    w1 = walker_of(a.rows, q0 + a.gate_rows - 1, walkers);
    if (w0 == w1) return;  // written whole
    if (q0 > first_row(a.rows, w0, walkers)) tail = static_cast<int>(w0);
    to = static_cast<float*>(a.dgate) + q * d;
  }
  float sum = 0.f;
  if (col < d)
    for (int64_t w = w0 + warp; w <= w1; w += 32)
      sum += a.partial[(static_cast<int64_t>(w == tail ? a.at_tail : which) * walkers + w) * d + col];
  s[warp][lane] = sum;
  __syncthreads();
  sum = s[lane][warp];
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  const int64_t at = static_cast<int64_t>(blockIdx.x) * 32 + warp;
  if (lane == 0 && at < d) to[at] = sum;
}

// Whether every row of every operand, and the parameters, are on 16-byte boundaries and
// the rows whole pieces.
bool whole(const ResNormArgs& a, bool fwd) {
  const int64_t es = a.bf16 ? 2 : 4, gs = a.gate_bf16 ? 2 : 4;
  uintptr_t all = static_cast<uintptr_t>(a.d * es);
  auto rows = [&](const void* p, int64_t ld, int64_t size) {
    if (p) all |= reinterpret_cast<uintptr_t>(p) | static_cast<uintptr_t>(ld * size);
  };
  rows(a.x, a.ld_x, es);
  rows(a.gate, a.ld_gate, gs);
  if (fwd) {
    rows(a.residual, a.ld_res, es);
    rows(a.h_out, a.ld_h, es);
    rows(a.y, a.ld_y, es);
  } else {
    rows(a.h, a.ld_h, es);
    rows(a.dy, a.ld_dy, es);
    rows(a.dh, a.ld_dh, es);
    rows(a.dx, a.ld_dx, es);
    rows(a.dres, a.ld_dres, es);
    if (a.gate_rows == 1) rows(a.dgate, a.ld_dgate, gs);
  }
  for (const void* p : {a.weight, a.bias, a.post_weight, a.post_bias}) rows(p, 0, 0);
  return all % 16 == 0;
}

template <typename T, int N, int NV, int G, int R>
cudaError_t fwd(const ResNormArgs& a, cudaStream_t s) {
  const unsigned grid = static_cast<unsigned>((a.rows + R - 1) / R);
  if (a.post_weight) k_resnorm_fwd<T, N, NV, G, R, true><<<grid, G * R, 0, s>>>(a);
  else k_resnorm_fwd<T, N, NV, G, R, false><<<grid, G * R, 0, s>>>(a);
  return cudaGetLastError();
}
template <typename T, int N>
cudaError_t fwd_n(const ResNormArgs& a, cudaStream_t s) {
  const int64_t pieces = a.d / N;
  // Few threads with several pieces each, as far as their registers leave four rows an SM: the
  // fewer warps join their sums, the better (163840 x 4096 bf16, RMS with a post norm: 256
  // threads with two pieces 867 us, 128 with four 755, 64 with eight 796).
  if (pieces <= 8) return fwd<T, N, 1, 8, 32>(a, s);
  if (pieces <= 16) return fwd<T, N, 1, 16, 16>(a, s);
  if (pieces <= 32) return fwd<T, N, 1, 32, 8>(a, s);
  if (pieces <= 64) return fwd<T, N, 2, 32, 4>(a, s);
  if constexpr (N == 8) {
    if (pieces <= 128) return fwd<T, N, 4, 32, 4>(a, s);
    if (pieces <= 256) return fwd<T, N, 4, 64, 2>(a, s);
    if (pieces <= 384) return fwd<T, N, 3, 128, 1>(a, s);
    if (pieces <= 512) return fwd<T, N, 4, 128, 1>(a, s);
    if (pieces <= 768) return fwd<T, N, 3, 256, 1>(a, s);
    if (pieces <= 1024) return fwd<T, N, 4, 256, 1>(a, s);
    if (pieces <= 1536) return fwd<T, N, 6, 256, 1>(a, s);
    if (pieces <= 2048) return fwd<T, N, 8, 256, 1>(a, s);
    if (pieces <= 4096) return fwd<T, N, 8, 512, 1>(a, s);
  } else {
    if (pieces <= 128) return fwd<T, N, 2, 64, 2>(a, s);
    if (pieces <= 256) return fwd<T, N, 2, 128, 1>(a, s);
    if (pieces <= 512) return fwd<T, N, 2, 256, 1>(a, s);
    if (pieces <= 768) return fwd<T, N, 3, 256, 1>(a, s);
    if (pieces <= 1024) return fwd<T, N, 4, 256, 1>(a, s);
    if (pieces <= 2048) return fwd<T, N, 4, 512, 1>(a, s);
    if (pieces <= 4096) return fwd<T, N, 8, 512, 1>(a, s);
  }
  return cudaErrorNotSupported;  // longer rows
}

template <typename T, int N, int G, int R, bool POST>
cudaError_t fwd_strided(const ResNormArgs& a, int sms, cudaStream_t s) {
  auto kernel = k_resnorm_fwd_strided<T, N, G, R, POST>;
  static std::atomic<uint64_t> configured{0};
  static std::atomic<int> per_sm{0};
  cudaError_t e;
  const int smem = strided_layout(a).bytes * R;
  if (smem > kResNormRing) return cudaErrorNotSupported;
  // (as many as the registers leave: the shared memory, which differs from call to call, is
  // counted here)
  const int n = resident_ctas(reinterpret_cast<const void*>(kernel), G * R, 0, kResNormRing, configured, per_sm, &e);
  if (n < 0) return e;
  const int fit = 228 * 1024 / (smem + 3 * 1024), most = n < fit ? n : fit;
  const int64_t all = static_cast<int64_t>(most < 1 ? 1 : most) * sms, need = (a.rows + R - 1) / R;
  const int64_t grid = need < all ? need : all, walkers = grid * R < a.rows ? grid * R : a.rows;
  kernel<<<static_cast<unsigned>(grid), G * R, smem, s>>>(a, static_cast<int>(walkers));
  return cudaGetLastError();
}
template <typename T, int N, int NV, int G, int R, bool POST>
cudaError_t fwd_shifted(const ResNormArgs& a, int step, int sms, cudaStream_t s) {
  auto kernel = k_resnorm_fwd_shifted<T, N, NV, G, R, POST>;
  static std::atomic<uint64_t> configured{0};
  static std::atomic<int> per_sm{0};
  cudaError_t e;
  const ShiftedLayout l = shifted_layout(a);
  const int smem = (2 * l.arrays * 16 + l.vectors * N * 4) * NV * G * R;
  if (smem > kResNormRing) return cudaErrorNotSupported;  // a long row with biases and a gate
  // (as many as the registers leave, and this call's shared memory)
  const int n = resident_ctas(reinterpret_cast<const void*>(kernel), G * R, 0, kResNormRing, configured, per_sm, &e);
  if (n < 0) return e;
  const int fit = kResNormRing / (smem + 3 * 1024), most = n < fit ? n : fit;
  const int64_t need = (a.rows + R - 1) / R, all = static_cast<int64_t>(most < 1 ? 1 : most) * sms, grid = need < all ? need : all;
  const int64_t walkers = (grid * R < a.rows ? grid * R : a.rows) / step * step;
  kernel<<<static_cast<unsigned>(grid), G * R, smem, s>>>(a, static_cast<int>(walkers), step);
  return cudaGetLastError();
}
template <typename T, int N, bool POST>
cudaError_t fwd_shifted_n(const ResNormArgs& a, int step, int sms, cudaStream_t s) {
  const int64_t pieces = (a.d + 2 * N - 2) / N;  // a row begins up to N - 1 elements late
  if (pieces <= 32) return cudaErrorNotSupported;  // few columns: sooner done as strided rows
  if (pieces <= 64) return fwd_shifted<T, N, 2, 32, 4, POST>(a, step, sms, s);
  if (pieces <= 128) return fwd_shifted<T, N, 2, 64, 1, POST>(a, step, sms, s);
  if (pieces <= 256) return fwd_shifted<T, N, 2, 128, 1, POST>(a, step, sms, s);
  if (pieces <= 384) return fwd_shifted<T, N, 3, 128, 1, POST>(a, step, sms, s);
  if (pieces <= 512) return fwd_shifted<T, N, 2, 256, 1, POST>(a, step, sms, s);
  if (pieces <= 1024) return fwd_shifted<T, N, 2, 512, 1, POST>(a, step, sms, s);
  if (pieces <= 1536) return fwd_shifted<T, N, 3, 512, 1, POST>(a, step, sms, s);
  if constexpr (N == 4)
    if (pieces <= 2048) return fwd_shifted<T, N, 4, 512, 1, POST>(a, step, sms, s);
  return cudaErrorNotSupported;
}
template <typename T, bool POST>
cudaError_t fwd_any(const ResNormArgs& a, int sms, cudaStream_t s) {
  if (const int step = resnorm_step(a, true)) {
    const cudaError_t e = fwd_shifted_n<T, 16 / static_cast<int>(sizeof(T)), POST>(a, step, sms, s);
    if (e != cudaErrorNotSupported) return e;
  }
  if (a.d <= 256) return fwd_strided<T, 8, 32, 8, POST>(a, sms, s);
  if (a.d <= 512) return fwd_strided<T, 16, 32, 8, POST>(a, sms, s);
  if (a.d <= 1024) return fwd_strided<T, 16, 64, 1, POST>(a, sms, s);
  if (a.d <= 2048) return fwd_strided<T, 16, 128, 1, POST>(a, sms, s);
  if (a.d <= 4096) return fwd_strided<T, 16, 256, 1, POST>(a, sms, s);
  if (a.d <= 8192) return fwd_strided<T, 16, 512, 1, POST>(a, sms, s);
  return cudaErrorNotSupported;
}

// The same for gates of which there are many, each shared by few walkers: a thread a
// column, one CTA row for every border between walkers; the first border inside a gate's
// rows takes them.
__global__ void __launch_bounds__(256) k_resnorm_join_gates(ResNormArgs a, int walkers) {
  const int64_t border = first_row(a.rows, static_cast<int64_t>(blockIdx.y) + 1, walkers), q = border / a.gate_rows;
  const int64_t q0 = q * a.gate_rows, col = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (border == q0) return;  // no gate has rows on both sides
  const int64_t w0 = walker_of(a.rows, q0, walkers), w1 = walker_of(a.rows, q0 + a.gate_rows - 1, walkers);
  if (w0 != static_cast<int64_t>(blockIdx.y) || col >= a.d) return;
  float sum = 0.f;
  for (int64_t w = w0; w <= w1; ++w) {
    const int which = w == w0 && q0 > first_row(a.rows, w0, walkers) ? a.at_tail : a.at_head;
    sum += a.partial[(static_cast<int64_t>(which) * walkers + w) * a.d + col];
  }
  static_cast<float*>(a.dgate)[q * a.d + col] = sum;
}
constexpr int64_t kFewGates = 32;

}  // namespace

int resnorm_walkers(const ResNormArgs& a, int sms) {
  // A bound that does not depend on addresses (the workspace is sized before they are
  // known): up to 8 walkers a CTA, 32 an SM for short rows, 8 for others, and for long ones
  // no more than an SM holds of their CTAs: 4 of 256 threads, 2 of 512 or of 1024.
  const int64_t each = a.d <= 512 ? 32 : a.d <= 4096 ? 8 : a.d <= 8192 ? 4 : 2;
  const int64_t most = each * sms, need = (a.rows + 7) / 8 * 8;
  return static_cast<int>(need < most ? need : most);
}

cudaError_t launch_resnorm_fwd(const ResNormArgs& a, int sms, cudaStream_t s) {
  const bool pieces = whole(a, true);
  cudaError_t e;
  if (pieces) e = a.bf16 ? fwd_n<__nv_bfloat16, 8>(a, s) : fwd_n<float, 4>(a, s);
  else if (a.post_weight) e = a.bf16 ? fwd_any<__nv_bfloat16, true>(a, sms, s) : fwd_any<float, true>(a, sms, s);
  else e = a.bf16 ? fwd_any<__nv_bfloat16, false>(a, sms, s) : fwd_any<float, false>(a, sms, s);
  if (e != cudaErrorNotSupported) return e;
  auto kernel = a.bf16 ? k_resnorm_fwd_long<__nv_bfloat16> : k_resnorm_fwd_long<float>;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kMaxResNormDim * 4));
  if (e != cudaSuccess) return e;
  kernel<<<static_cast<unsigned>(a.rows), kLong, a.d * 4, s>>>(a);
  return cudaGetLastError();
}
cudaError_t launch_resnorm_bwd(const ResNormArgs& a, int sms, int* walkers, cudaStream_t s) {
  if (!(a.gate && a.gate_rows == 1 && a.gate_bf16 != a.bf16)) {
    const bool w = whole(a, false);
    if (a.bf16) return a.post_weight ? resnorm_bwd_bf16_post(a, w, sms, walkers, s) : resnorm_bwd_bf16(a, w, sms, walkers, s);
    return a.post_weight ? resnorm_bwd_f32_post(a, w, sms, walkers, s) : resnorm_bwd_f32(a, w, sms, walkers, s);
  }
  // every sum that fits beside the row, one CTA an SM then
  const int sums = (a.dweight != nullptr) + (a.dbias != nullptr) + (a.dpost_weight != nullptr) + (a.dpost_bias != nullptr);
  const int room = static_cast<int>(kResNormRing / (a.d * 4)) - 1, fit = sums < room ? sums : room;
  const int smem = static_cast<int>(a.d * 4) * (1 + fit);
  auto kernel = a.bf16 ? k_resnorm_bwd_long<__nv_bfloat16> : k_resnorm_bwd_long<float>;
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kResNormRing);
  if (e != cudaSuccess) return e;
  const int64_t most = sms;
  *walkers = static_cast<int>(a.rows < most ? a.rows : most);
  kernel<<<*walkers, kWide, smem, s>>>(a, *walkers, fit);
  return cudaGetLastError();
}
cudaError_t launch_resnorm_join(const ResNormArgs& a, int walkers, cudaStream_t s) {
  const int64_t gates = a.dgate && a.gate_rows > 1 ? a.rows / a.gate_rows : 0;
  const int64_t few = a.at_head + (gates <= kFewGates ? gates : 0);
  if (few > 0) k_resnorm_join<<<dim3(static_cast<unsigned>((a.d + 31) / 32), static_cast<unsigned>(few)), 1024, 0, s>>>(a, walkers);
  if (gates > kFewGates && walkers > 1)
    k_resnorm_join_gates<<<dim3(static_cast<unsigned>((a.d + 255) / 256), static_cast<unsigned>(walkers - 1)), 256, 0, s>>>(a, walkers);
  return cudaGetLastError();
}

}  // namespace grpo
