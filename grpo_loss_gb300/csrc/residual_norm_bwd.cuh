// Backward of the norms around a block, rows in whole pieces. With hat = (h - m) r,
// e = dh + r dy w, k = (x - pm) pr and a = scale gate pw,
//   g  = e - r (c1 + hat c2),   c1 = mean(dy w),  c2 = mean(dy w hat)
//   dx = pr (a g - mean(a g) - k mean(a g k)),
// where the two means over a g are sums over e less c1 and c2 times sums that need neither,
//   sum a g   = sum a e   - r c1 sum a   - r c2 sum a hat
//   sum a g k = sum a e k - r c1 sum a k - r c2 sum a hat k,
// so that all sums of a row (8, or 3 of RMS norms) are taken in one pass and joined once.
#pragma once

#include <cooperative_groups.h>

#include <atomic>

#include "f32x2.cuh"
#include "internal.h"
#include "pieces.cuh"

namespace grpo {

// The walker w of n takes rows [w rows / n, (w + 1) rows / n).
__device__ __forceinline__ int64_t first_row(int64_t rows, int64_t w, int64_t n) { return w * rows / n; }
__device__ __forceinline__ int64_t walker_of(int64_t rows, int64_t row, int64_t n) { return ((row + 1) * n - 1) / rows; }

enum : int { GATE_NONE, GATE_SHARED, GATE_ROWS };
enum : int { ROWS_WHOLE, ROWS_SHIFTED, ROWS_STRIDED };
constexpr int kResNormRing = 224 * 1024;  // of shared memory, beside the sums
constexpr int kResNormCluster = 8;        // CTAs that share a row, at most
// Rows that lie in their granules alike, in every operand: how many rows on they do so again. 0
// where the operands differ; where a gate has some of the rows, for what a walker takes is not
// contiguous; and where there are few rows of a step (8191 bf16 columns: 600 rows 72 us for 62 as
// strided ones, 20000 rows 646 for 723; 30000 x 2881 236 for 468).
constexpr int kShiftedRows = 256;
inline int resnorm_step(const ResNormArgs& a, bool fwd) {
  if (a.gate && a.gate_rows > 1 && a.gate_rows != a.rows) return 0;
  const int64_t es = a.bf16 ? 2 : 4, cut = (fwd ? a.ld_x : a.ld_h) * es % 16;
  bool alike = true;
  auto rows = [&](const void* p, int64_t ld) {
    if (p) alike = alike && reinterpret_cast<uintptr_t>(p) % 16 == 0 && ld * es % 16 == cut;
  };
  rows(a.x, a.ld_x);
  if (fwd) {
    rows(a.residual, a.ld_res);
    rows(a.h_out, a.ld_h);
    rows(a.y, a.ld_y);
  } else {
    rows(a.h, a.ld_h);
    rows(a.dy, a.ld_dy);
    rows(a.dh, a.ld_dh);
    rows(a.dx, a.ld_dx);
    rows(a.dres, a.ld_dres);
  }
  if (a.gate && a.gate_rows == 1) {
    if (a.gate_bf16 != a.bf16) return 0;
    rows(a.gate, a.ld_gate);
    rows(a.dgate, a.ld_dgate);
  }
  int step = 1;
  while (cut * step % 16) step *= 2;
  return alike && a.rows >= kShiftedRows * step ? step : 0;
}
// The rows that a walker has of those: from, from + step, ..., `mine` of them.
struct Walk {
  int64_t from;
  int mine, turns;  // turns: the most that a walker has
  int shift;        // elements of the first granule that are not the row's
};
__device__ __forceinline__ Walk shifted_walk(const ResNormArgs& a, int64_t ld, int64_t walker, int walkers, int step, int size) {
  const int64_t run = walker / step, runs = walkers / step;
  Walk w = {0, 0, static_cast<int>(((a.rows + runs - 1) / runs + step - 1) / step), 0};
  if (walker < walkers) {
    const int64_t to = first_row(a.rows, run + 1, runs);
    w.from = first_row(a.rows, run, runs);
    w.from += (walker % step + step - w.from % step) % step;
    w.mine = w.from < to ? static_cast<int>((to - w.from + step - 1) / step) : 0;
  }
  w.shift = static_cast<int>((w.from * ld * size) & 15) / size;
  return w;
}

// Columns of each CTA of a cluster, whole pieces of n; the last one's may be fewer. (Clustered
// rows have over a thousand pieces, so that it has some.)
__host__ __device__ __forceinline__ int resnorm_share(int d, int n, int ranks) { return (d / n + ranks - 1) / ranks * n; }

// CTAs of a kernel that an SM holds with `smem` bytes each, asked once a device; -1 where that
// fails. `most`: the largest shared memory that it is launched with.
inline int resident_ctas(const void* kernel, int threads, int smem, int most, std::atomic<uint64_t>& configured, std::atomic<int>& per_sm,
                         cudaError_t* e) {
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

// Whether layer norms' second sums are in shared memory (see the kernel).
template <int N, int G, int R, bool RMS, int MODE>
constexpr bool resnorm_stash() {
  return !RMS && MODE != ROWS_STRIDED && N == 8 && G * R <= 256;
}

// Copies a row of d elements by the 16-byte granules it lies in while the G threads go on;
// `to` has the place of the first granule.
template <typename T, int G>
__device__ __forceinline__ void stage_row(unsigned char* to, const T* row, const T* matrix, int d, int tid) {
  constexpr int es = static_cast<int>(sizeof(T));
  const int off = static_cast<int>(reinterpret_cast<uintptr_t>(row) & 15), bytes = off + d * es;
  const char* const from = reinterpret_cast<const char*>(row) - off;
  int i = tid * 16;
  if (tid == 0 && from < reinterpret_cast<const char*>(matrix)) {  // the granule begins before the matrix
    for (int e = 0; e < d && off + e * es < 16; ++e) reinterpret_cast<T*>(to + off)[e] = row[e];
    i = G * 16;
  }
#pragma unroll 2
  for (; i < bytes; i += G * 16) copy_async_zero(to + i, from + i, min(16, bytes - i));
}
constexpr int staged_pitch(int d, int size) { return (d * size + 31) / 16 * 16; }

// A group of G threads is a walker, R of them a CTA; each thread holds NV pieces of N
// columns: their values of a row, and their column sums. The next row's pieces are on
// their way into shared memory meanwhile, whence they are read twice, for the sums and for
// the outputs. A thread reads back what it copied itself.
// The gate's sums are e1 = sum scale g k and e0 = sum scale g over the rows that share it,
// of which dgate = pw e1 + pb e0, and gate e1 and gate e0 are these rows' parts of the post
// norm's dweight and dbias: taken when the gate changes, so that a row adds to two sums and
// not to three.
// ROWS_SHIFTED: rows that begin and end inside a 16-byte granule, at the same place in every
// operand. A walker takes every step-th row of a run, whose granules are cut alike, so that
// its threads' pieces are granules and keep their columns: the first one may have elements of
// the row before, which are cleared as they arrive.
// ROWS_STRIDED: others that do not come in whole pieces. A row is staged by the 16-byte granules it
// lies in, and a thread's N columns are G apart, so that a warp's accesses are to
// consecutive elements wherever the row begins; one more barrier a row lets the threads
// read what others copied.
// CLUSTER: rows too long for one CTA's shared memory. A cluster is a walker, each of its CTAs
// has an equal run of the columns, and a row's sums are exchanged by one cluster barrier
// while the next row is on its way. (40960 x 8192 float32, RMS with a post norm, floor 1204 us:
// 1501; a CTA a row that waits for its loads 5030. 40960 x 16384 bf16: 2106 for 11700.)
template <typename T, int N, int NV, int G, int R, bool RMS, bool POST, int GATE, int MODE, bool CLUSTER>
__global__ void __launch_bounds__(G * R) k_resnorm_bwd(ResNormArgs a, int walkers, int steps) {
  constexpr bool STRIDED = MODE == ROWS_STRIDED, SHIFTED = MODE == ROWS_SHIFTED;
  static_assert(!STRIDED || (NV == 1 && (R == 1 || G == 32)), "");
  static_assert(!CLUSTER || (R == 1 && !SHIFTED), "");
  constexpr int B = N * static_cast<int>(sizeof(T)), H = N / 2;
  static_assert(STRIDED || B == 16, "");
  constexpr bool INNER = POST || GATE != GATE_NONE;
  constexpr int ARRAYS = 3 + INNER + (GATE == GATE_ROWS);  // dy, h, dh, x, gate
  constexpr int SUMS = POST ? (RMS ? 4 : 8) : 2;
  using V = Piece<T, STRIDED ? 1 : N>;
  extern __shared__ __align__(16) unsigned char ring_raw[];
  __shared__ float part[2 * (SUMS < 4 ? 128 : 32 * SUMS)];
  V* const ring = reinterpret_cast<V*>(ring_raw) + threadIdx.x;  // [2][ARRAYS][NV][threads]
  __shared__ float rank_sums[2][CLUSTER ? kResNormCluster : 1][SUMS];  // of every CTA of the cluster
  const int tid = threadIdx.x % G, d = static_cast<int>(a.d);
  auto cluster = cooperative_groups::this_cluster();
  const int ranks = CLUSTER ? static_cast<int>(cluster.num_blocks()) : 1, rank = CLUSTER ? static_cast<int>(cluster.block_rank()) : 0;
  // the CTA's columns
  const int share = CLUSTER ? resnorm_share(d, STRIDED ? 1 : N, ranks) : d, first = rank * share;
  const int edge = !CLUSTER || d < first + share ? d : first + share;
  const int64_t walker = CLUSTER ? blockIdx.x / ranks : static_cast<int64_t>(blockIdx.x) * R + threadIdx.x / G;
  // its rows: from, from + step, ..., `mine` of them; every group of a CTA makes the same
  // number of turns: barriers are the CTA's
  int64_t from;
  int mine, turns, shift = 0;
  const int step = SHIFTED ? steps : 1;
  if constexpr (SHIFTED) {
    const Walk walk = shifted_walk(a, a.ld_h, walker, walkers, step, static_cast<int>(sizeof(T)));
    from = walk.from, mine = walk.mine, turns = walk.turns, shift = walk.shift;
  } else {
    from = walker < walkers ? first_row(a.rows, walker, walkers) : 0;
    mine = walker < walkers ? static_cast<int>(first_row(a.rows, walker + 1, walkers) - from) : 0;
    turns = static_cast<int>((a.rows + walkers - 1) / walkers);
  }

  uint64_t w[NV][H], f[NV][H], dw[NV][H], e1[NV][H];  // f: a; scale gate without a post norm; pw with a gate for each row
  // The sums of dy and of scale g, that layer norms have beside: in registers, or where these
  // would leave an SM one CTA in shared memory, each thread its own.
  constexpr bool STASH = resnorm_stash<N, G, R, RMS, MODE>();
  uint64_t db_reg[STASH ? 1 : NV][H], e0_reg[STASH ? 1 : NV][H];
  ulonglong2* const stash = reinterpret_cast<ulonglong2*>(ring_raw + 2 * ARRAYS * NV * B * G * R) + threadIdx.x;
  auto load_sums = [&](int which, int k, uint64_t (&v)[H]) {  // 0: of dy, 1: of scale g
    if constexpr (STASH) {
#pragma unroll
      for (int e = 0; e < H; e += 2) {
        const ulonglong2 u = stash[((which * NV + k) * (H / 2) + e / 2) * (G * R)];
        v[e] = u.x, v[e + 1] = u.y;
      }
    } else {
#pragma unroll
      for (int e = 0; e < H; ++e) v[e] = which ? e0_reg[k][e] : db_reg[k][e];
    }
  };
  auto keep_sums = [&](int which, int k, const uint64_t (&v)[H]) {
    if constexpr (STASH) {
#pragma unroll
      for (int e = 0; e < H; e += 2) stash[((which * NV + k) * (H / 2) + e / 2) * (G * R)] = make_ulonglong2(v[e], v[e + 1]);
    } else {
#pragma unroll
      for (int e = 0; e < H; ++e) (which ? e0_reg[k][e] : db_reg[k][e]) = v[e];
    }
  };
  // column i of the thread's piece k; a piece's columns are all in the CTA's, or each is looked at
  auto column = [&](int k, int i = 0) { return first + (STRIDED ? i * G + tid : (k * G + tid) * N + i - shift); };
  auto inside = [&](int k, int i) { return STRIDED ? column(0, i) < edge : !SHIFTED || static_cast<unsigned>(column(k, i)) < static_cast<unsigned>(d); };
  auto inside_all = [&](int k) { return !SHIFTED || (column(k) >= 0 && column(k) + N <= d); };
  // N parameters from element `at` of p on
  auto load_pairs = [&](const void* p, int bf16, int64_t at, int k, uint64_t (&v)[H]) {
    float u[N] = {};
    if constexpr (STRIDED || SHIFTED) {
#pragma unroll
      for (int i = 0; i < N; ++i)
        if (inside(k, i)) u[i] = bf16 ? ldf(static_cast<const __nv_bfloat16*>(p), at + column(k, i)) : ldf(static_cast<const float*>(p), at + column(k, i));
    } else {
      if (bf16) load_params<N>(static_cast<const __nv_bfloat16*>(p) + at, 1, column(k), u);
      else load_params<N>(static_cast<const float*>(p) + at, 0, column(k), u);
    }
#pragma unroll
    for (int e = 0; e < H; ++e) v[e] = pair_of(u[2 * e], u[2 * e + 1]);
  };
  const uint64_t zero = pair_of(0.f, 0.f), scale2 = pair_of(a.scale);
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    uint64_t none[H];
#pragma unroll
    for (int e = 0; e < H; ++e) {
      w[k][e] = dw[k][e] = e1[k][e] = none[e] = zero;
      f[k][e] = scale2;
    }
    keep_sums(0, k, none);
    if constexpr (POST) keep_sums(1, k, none);
    if (column(k) < edge) {
      load_pairs(a.weight, a.param_bf16, 0, k, w[k]);
      if constexpr (POST && GATE != GATE_SHARED) {
        uint64_t pw[H];
        load_pairs(a.post_weight, a.param_bf16, 0, k, pw);
#pragma unroll
        for (int e = 0; e < H; ++e) f[k][e] = GATE == GATE_ROWS ? pw[e] : mul2(pw[e], scale2);
      }
    }
  }

  auto slot_of = [&](int half, int which, int k) -> V& { return ring[((half * ARRAYS + which) * NV + k) * (G * R)]; };
  const int pitch = staged_pitch(share, sizeof(T));
  unsigned char* const staged = ring_raw + threadIdx.x / G * (2 * ARRAYS * pitch);  // the group's
  auto fetch = [&](int n, int half) {
    if (n < mine) {
      const int64_t row = from + static_cast<int64_t>(n) * step;
      auto copy = [&](int which, const void* p, int64_t ld) {
        const T* q = static_cast<const T*>(p) + row * ld;  // (with `shift` before it in its granule)
        if constexpr (STRIDED) {
          stage_row<T, G>(staged + (half * ARRAYS + which) * pitch, q + first, static_cast<const T*>(p), edge - first, tid);
        } else {
#pragma unroll
          for (int k = 0; k < NV; ++k)
            if (column(k) < edge) {
              if constexpr (SHIFTED) copy_async_zero(&slot_of(half, which, k), q + column(k), min(B, (d - column(k)) * static_cast<int>(sizeof(T))));
              else copy_async<B>(&slot_of(half, which, k), q + column(k));
            }
        }
      };
      copy(0, a.dy, a.ld_dy);
      copy(1, a.h, a.ld_h);
      if (a.dh) copy(2, a.dh, a.ld_dh);
      if constexpr (INNER) copy(3, a.x, a.ld_x);
      if constexpr (GATE == GATE_ROWS) copy(4, a.gate, a.ld_gate);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  // The values of a piece of a row that has arrived, by pairs.
  struct Values {
    V v;
    const T* p;
  };
  auto values = [&](int half, int which, int k, const void* base, int64_t ld, int64_t row) {
    Values u;
    if constexpr (STRIDED) {
      const int off = static_cast<int>(reinterpret_cast<uintptr_t>(static_cast<const T*>(base) + row * ld + first) & 15);
      u.p = reinterpret_cast<const T*>(staged + (half * ARRAYS + which) * pitch + off);
    } else {
      u.v = slot_of(half, which, k);
    }
    return u;
  };
  auto pair = [&](const Values& u, int e) {
    if constexpr (STRIDED)
      return pair_of(inside(0, 2 * e) ? ldf(u.p, column(0, 2 * e) - first) : 0.f, inside(0, 2 * e + 1) ? ldf(u.p, column(0, 2 * e + 1) - first) : 0.f);
    else
      return pair_of(u.v.get(2 * e), u.v.get(2 * e + 1));
  };
  auto store = [&](T* to, int k, const float* o) {
    if (!STRIDED && inside_all(k)) {
      V p;
      p.set(o);
      store_piece(to + column(k), p);
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i)
        if (inside(k, i)) stf(to, column(k, i), o[i]);
    }
  };
  auto store_sums = [&](float* to, int k, const uint64_t (&v)[H]) {
#pragma unroll
    for (int e = 0; e < H; ++e) {
      const float2 p = of_pair(v[e]);
      if (inside(k, 2 * e)) to[column(k, 2 * e)] = p.x;
      if (inside(k, 2 * e + 1)) to[column(k, 2 * e + 1)] = p.y;
    }
  };
  auto part_of = [&](int which) { return a.partial + (static_cast<int64_t>(which) * walkers + walker) * d; };

  // The rows of a gate that this walker has, from row `begin` on and before `end`, are done.
  int flushed = 0;
  auto flush = [&](int64_t begin, int64_t end) {
    const int64_t q = begin / a.gate_rows, q0 = q * a.gate_rows;
    // written whole, or left as a part: a gate's last rows, or its first ones
    // (shifted rows: one gate has all rows)
    float* const to = !a.dgate ? nullptr
                      : SHIFTED ? (walkers == 1 ? static_cast<float*>(a.dgate) : part_of(a.at_head))
                      : q0 == begin && q0 + a.gate_rows == end ? static_cast<float*>(a.dgate) + q * d
                      : begin == from ? part_of(a.at_head)
                                      : part_of(a.at_tail);
#pragma unroll
    for (int k = 0; k < NV; ++k)
      if (column(k) < edge) {
        uint64_t pw[H], g[H], v[H], e0[H];
        if constexpr (POST) {
          load_sums(1, k, e0);
          load_pairs(a.post_weight, a.param_bf16, 0, k, pw);
          load_pairs(a.gate, a.gate_bf16, q * a.ld_gate, k, g);
        }
        if (to) {
#pragma unroll
          for (int e = 0; e < H; ++e) v[e] = POST ? mul2(pw[e], e1[k][e]) : e1[k][e];
          if (POST && !RMS && a.post_bias) {
            uint64_t pb[H];
            load_pairs(a.post_bias, a.param_bf16, 0, k, pb);
#pragma unroll
            for (int e = 0; e < H; ++e) v[e] = fma2(pb[e], e0[e], v[e]);
          }
          store_sums(to, k, v);
        }
        if constexpr (POST) {
          auto add = [&](float* p, const uint64_t (&s)[H]) {
#pragma unroll
            for (int e = 0; e < H; ++e) {
              const uint64_t before = !flushed ? zero
                                               : pair_of(inside(k, 2 * e) ? p[column(k, 2 * e)] : 0.f,
                                                         inside(k, 2 * e + 1) ? p[column(k, 2 * e + 1)] : 0.f);
              v[e] = fma2(g[e], s[e], before);
            }
            store_sums(p, k, v);
          };
          if (a.dpost_weight) add(part_of(a.at_dpw), e1[k]);
          if (!RMS && a.dpost_bias) add(part_of(a.at_dpb), e0);
        }
#pragma unroll
        for (int e = 0; e < H; ++e) e1[k][e] = e0[e] = zero;
        if constexpr (POST) keep_sums(1, k, e0);
      }
    flushed = 1;
  };

  const float inv_d = 1.f / d;
  struct Stats {
    float m, r, pm, pr;
  };
  auto stats_of = [&](int n) {
    Stats s = {0.f, 0.f, 0.f, 1.f};
    if (n < mine) {
      const int64_t row = from + static_cast<int64_t>(n) * step;
      if (!RMS) s.m = a.mean[row];
      s.r = a.rstd[row];
      if (POST) {
        if (!RMS) s.pm = a.post_mean[row];
        s.pr = a.post_rstd[row];
      }
    }
    return s;
  };
  int64_t gate_from = from, gate_to = GATE == GATE_SHARED ? from : 0;  // the rows of the gate in f
  Stats next = stats_of(0);
  fetch(0, 0);
  if constexpr (CLUSTER) cluster.sync();  // every CTA runs: its shared memory may be written
  int half = 0;
  for (int n = 0; n < turns; ++n, half ^= 1) {
    if constexpr (STRIDED) {
      // this row is here, of every thread's copies, and the last one's place is free
      asm volatile("cp.async.wait_group 0;" ::: "memory");
      if constexpr (G == 32) __syncwarp();
      else __syncthreads();
      fetch(n + 1, half ^ 1);
    } else {
      fetch(n + 1, half ^ 1);
      asm volatile("cp.async.wait_group 1;" ::: "memory");
      if (SHIFTED && n < mine && column(0) < 0) {
        for (int which = 0; which < ARRAYS; ++which)
          for (int i = 0; i < shift; ++i) reinterpret_cast<T*>(&slot_of(half, which, 0))[i] = T(0.f);
      }
    }
    const Stats s = next;
    next = stats_of(n + 1);
    const bool live = n < mine;
    const int64_t row = from + static_cast<int64_t>(n) * step;
    if constexpr (GATE == GATE_SHARED) {
      if (live && row >= gate_to) {
        if (n > 0) flush(gate_from, gate_to);
        gate_from = row;
        gate_to = (row / a.gate_rows + 1) * a.gate_rows;
#pragma unroll
        for (int k = 0; k < NV; ++k)
          if (column(k) < edge) {
            load_pairs(a.gate, a.gate_bf16, row / a.gate_rows * a.ld_gate, k, f[k]);
            uint64_t pw[H];
            if constexpr (POST) load_pairs(a.post_weight, a.param_bf16, 0, k, pw);
#pragma unroll
            for (int e = 0; e < H; ++e) f[k][e] = POST ? mul2(mul2(pw[e], scale2), f[k][e]) : mul2(f[k][e], scale2);
          }
      }
    }
    const uint64_t r2 = pair_of(s.r), pr2 = pair_of(s.pr), m2 = pair_of(-s.m), pm2 = pair_of(-s.pm);
    // (x - mean) r, the difference first: x and mean may be large and close
    auto hat_of = [&](uint64_t v, uint64_t m, uint64_t r) { return mul2(RMS ? v : add2(v, m), r); };
    uint64_t t[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) t[i] = zero;
    if (live) {
#pragma unroll
      for (int k = 0; k < NV; ++k)
        if (column(k) < edge) {
          const Values vy = values(half, 0, k, a.dy, a.ld_dy, row), vh = values(half, 1, k, a.h, a.ld_h, row);
          Values vd, vx, vg;
          if constexpr (POST) {
            if (a.dh) vd = values(half, 2, k, a.dh, a.ld_dh, row);
            vx = values(half, 3, k, a.x, a.ld_x, row);
            if constexpr (GATE == GATE_ROWS) vg = values(half, 4, k, a.gate, a.ld_gate, row);
          }
          uint64_t db[H];
          if (!RMS) load_sums(0, k, db);
#pragma unroll
          for (int e = 0; e < H; ++e) {
            const uint64_t y = pair(vy, e), hat = hat_of(pair(vh, e), m2, r2), yw = mul2(y, w[k][e]);
            dw[k][e] = fma2(y, hat, dw[k][e]);
            if (!RMS) db[e] = add2(db[e], y);
            t[0] = fma2(yw, hat, t[0]);
            if (!RMS) t[1] = add2(t[1], yw);
            if constexpr (POST) {
              uint64_t av = f[k][e];
              if constexpr (GATE == GATE_ROWS) av = mul2(av, pair(vg, e));
              const uint64_t kx = hat_of(pair(vx, e), pm2, pr2);
              const uint64_t ae = mul2(av, a.dh ? fma2(r2, yw, pair(vd, e)) : mul2(r2, yw));
              const uint64_t ah = mul2(av, hat);
              t[2] = fma2(ae, kx, t[2]);
              t[3] = fma2(ah, kx, t[3]);
              if (!RMS) {
                t[4] = add2(t[4], ae);
                t[5] = add2(t[5], ah);
                t[6] = add2(t[6], av);
                t[7] = fma2(av, kx, t[7]);
              }
            }
          }
          if (!RMS) keep_sums(0, k, db);
        }
    }
    float sums[SUMS];
#pragma unroll
    for (int i = 0; i < SUMS; ++i) {
      const float2 p = of_pair(t[i]);
      sums[i] = p.x + p.y;
    }
    group_sums<G, SUMS>(sums, part, half);
    if constexpr (CLUSTER) {
      // (a half is written again two rows on, behind a barrier that its readers have reached)
      if (tid < ranks) {
        float* const to = cluster.map_shared_rank(&rank_sums[half][rank][0], tid);
#pragma unroll
        for (int i = 0; i < SUMS; ++i) to[i] = sums[i];
      }
      cluster.sync();
#pragma unroll
      for (int i = 0; i < SUMS; ++i) {
        sums[i] = rank_sums[half][0][i];
        for (int c = 1; c < ranks; ++c) sums[i] += rank_sums[half][c][i];
      }
    }
    if (!live) continue;
    if constexpr (POST && GATE == GATE_ROWS) {  // (of a over scale)
#pragma unroll
      for (int i = 2; i < SUMS; ++i) sums[i] *= a.scale;
    }
    // r c2, r c1
    const float c2 = s.r * sums[0] * inv_d, c1 = RMS ? 0.f : s.r * sums[1] * inv_d;
    float b1 = 0.f, b2 = 0.f;  // means of a g and of a g k
    if constexpr (POST) {
      b2 = fmaf(-c2, sums[3], sums[2]);
      if constexpr (!RMS) {
        b2 = fmaf(-c1, sums[7], b2) * inv_d;
        b1 = fmaf(-c1, sums[6], fmaf(-c2, sums[5], sums[4])) * inv_d;
      } else {
        b2 *= inv_d;
      }
    }
    const uint64_t n1 = pair_of(-c1), n2 = pair_of(-c2), o1 = pair_of(-b1), o2 = pair_of(-b2);
    T* const to_res = static_cast<T*>(a.dres) + row * a.ld_dres;
    T* const to_x = a.dx ? static_cast<T*>(a.dx) + row * a.ld_dx : nullptr;
#pragma unroll
    for (int k = 0; k < NV; ++k)
      if (column(k) < edge) {
        const Values vy = values(half, 0, k, a.dy, a.ld_dy, row), vh = values(half, 1, k, a.h, a.ld_h, row);
        Values vd, vx, vg;
        if (a.dh) vd = values(half, 2, k, a.dh, a.ld_dh, row);
        if constexpr (INNER) vx = values(half, 3, k, a.x, a.ld_x, row);
        if constexpr (GATE == GATE_ROWS) vg = values(half, 4, k, a.gate, a.ld_gate, row);
        float res[N], dx[N], dg[N];
        uint64_t e0[H];
        if constexpr (POST && !RMS) load_sums(1, k, e0);
        uint64_t pb[H];
#pragma unroll
        for (int e = 0; e < H; ++e) pb[e] = zero;
        if constexpr (GATE == GATE_ROWS && POST && !RMS)
          if (a.dgate && a.post_bias) load_pairs(a.post_bias, a.param_bf16, 0, k, pb);
#pragma unroll
        for (int e = 0; e < H; ++e) {
          const uint64_t hat = hat_of(pair(vh, e), m2, r2);
          uint64_t g = fma2(r2, mul2(pair(vy, e), w[k][e]), fma2(hat, n2, n1));
          if (a.dh) g = add2(g, pair(vd, e));
          const float2 gr = of_pair(g);
          res[2 * e] = gr.x, res[2 * e + 1] = gr.y;
          const uint64_t sg = mul2(g, scale2);
          uint64_t out = POST && GATE == GATE_ROWS ? mul2(sg, f[k][e]) : mul2(g, f[k][e]);  // a g, or scale gate g
          if constexpr (INNER) {
            const uint64_t kx = POST ? hat_of(pair(vx, e), pm2, pr2) : pair(vx, e);
            if constexpr (GATE == GATE_ROWS) {
              // dgate = scale g p; p = k pw + pb is rounded once, for its parts may cancel
              const float2 dv = of_pair(POST ? mul2(sg, RMS ? mul2(kx, f[k][e]) : fma2(kx, f[k][e], pb[e])) : mul2(out, kx));
              dg[2 * e] = dv.x, dg[2 * e + 1] = dv.y;
              out = mul2(out, pair(vg, e));
            }
            if constexpr (POST || GATE == GATE_SHARED) {
              const uint64_t part_g = GATE == GATE_ROWS ? mul2(sg, pair(vg, e)) : sg;  // with a gate for every row: of q
              e1[k][e] = fma2(part_g, kx, e1[k][e]);
              if (POST && !RMS) e0[e] = add2(e0[e], part_g);
            }
            if constexpr (POST) out = mul2(fma2(kx, o2, add2(out, o1)), pr2);
          }
          const float2 ov = of_pair(out);
          dx[2 * e] = ov.x, dx[2 * e + 1] = ov.y;
        }
        if constexpr (POST && !RMS) keep_sums(1, k, e0);
        store(to_res, k, res);
        if (to_x) store(to_x, k, dx);
        if constexpr (GATE == GATE_ROWS)
          if (a.dgate) store(static_cast<T*>(a.dgate) + row * a.ld_dgate, k, dg);
      }
  }
  if (mine == 0) return;
  if constexpr (GATE == GATE_SHARED) flush(gate_from, from + mine);
#pragma unroll
  for (int k = 0; k < NV; ++k)
    if (column(k) < edge) {
      if (a.dweight) store_sums(part_of(a.at_dw), k, dw[k]);
      uint64_t v[H];
      if (!RMS && a.dbias) {
        load_sums(0, k, v);
        store_sums(part_of(a.at_db), k, v);
      }
      if constexpr (POST && GATE != GATE_SHARED) {
        if (a.dpost_weight) store_sums(part_of(a.at_dpw), k, e1[k]);
        if (!RMS && a.dpost_bias) {
          load_sums(1, k, v);
          store_sums(part_of(a.at_dpb), k, v);
        }
      }
    }
}

// One launch: as many CTAs as the SMs hold at a time, so that each walks over its share of
// the rows once. *walkers: rows of partial sums it writes.
template <typename T, int N, int NV, int G, int R, bool RMS, bool POST, int GATE, int MODE>
cudaError_t resnorm_bwd(const ResNormArgs& a, int step, int sms, int* walkers, cudaStream_t s) {
  constexpr int arrays = 3 + (POST || GATE != GATE_NONE) + (GATE == GATE_ROWS);
  constexpr bool STRIDED = MODE == ROWS_STRIDED;
  constexpr int stash = resnorm_stash<N, G, R, RMS, MODE>() ? (POST ? 2 : 1) * NV * N * 4 * G * R : 0;
  constexpr int smem = 2 * arrays * (NV * N * static_cast<int>(sizeof(T)) * G + (STRIDED ? 32 : 0)) * R + stash;
  static_assert(smem <= kResNormRing, "shared memory");
  auto kernel = k_resnorm_bwd<T, N, NV, G, R, RMS, POST, GATE, MODE, false>;
  static std::atomic<uint64_t> configured{0};
  static std::atomic<int> per_sm{0};
  cudaError_t e;
  const int n = resident_ctas(reinterpret_cast<const void*>(kernel), G * R, smem, smem, configured, per_sm, &e);
  if (n < 0) return e;
  // four rows a walker at least, where that leaves the SMs at work: its partial sums are
  // written and read again
  int64_t grid = (a.rows + R - 1) / R;
  if (grid > sms / 2) grid = grid / 4 > sms / 2 ? grid / 4 : sms / 2;
  const int64_t most = static_cast<int64_t>(n) * sms, room = resnorm_walkers(a, sms) / R;
  grid = grid < most ? grid : most;
  grid = grid < room ? grid : room;
  const int64_t w = grid * R < a.rows ? grid * R : a.rows;
  *walkers = static_cast<int>(w / step * step);
  kernel<<<static_cast<unsigned>(grid), G * R, smem, s>>>(a, *walkers, step);
  return cudaGetLastError();
}

// The same with a cluster of 2, 4 or 8 CTAs for a row, as few as hold it.
template <typename T, int N, int NV, int G, bool RMS, bool POST, int GATE, int MODE>
cudaError_t resnorm_bwd_cluster(const ResNormArgs& a, int sms, int* walkers, cudaStream_t s) {
  constexpr int arrays = 3 + (POST || GATE != GATE_NONE) + (GATE == GATE_ROWS);
  constexpr bool STRIDED = MODE == ROWS_STRIDED;
  constexpr int smem = 2 * arrays * (NV * N * static_cast<int>(sizeof(T)) * G + (STRIDED ? 32 : 0));
  static_assert(smem <= kResNormRing && !resnorm_stash<N, G, 1, RMS, MODE>(), "shared memory");
  static_assert(kMaxResNormDim <= static_cast<int64_t>(kResNormCluster) * NV * N * G, "the longest rows");
  auto kernel = k_resnorm_bwd<T, N, NV, G, 1, RMS, POST, GATE, MODE, true>;
  int ranks = 2, log = 0;
  while (resnorm_share(static_cast<int>(a.d), STRIDED ? 1 : N, ranks) > NV * N * G) ranks *= 2, ++log;
  cudaLaunchConfig_t config = {};
  config.gridDim = dim3(static_cast<unsigned>(ranks));
  config.blockDim = dim3(G);
  config.dynamicSmemBytes = smem;
  config.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(ranks);
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  config.attrs = attr;
  config.numAttrs = 1;
  // clusters that the GPU holds at a time, asked once a device and size
  static std::atomic<uint64_t> configured[3];
  static std::atomic<int> clusters[3];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = 1ull << (dev & 63);
  if (!(configured[log].load() & bit)) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    int n = 0;
    if (e == cudaSuccess) e = cudaOccupancyMaxActiveClusters(&n, kernel, &config);
    if (e != cudaSuccess) return e;
    clusters[log].store(n < 1 ? 1 : n);
    configured[log].fetch_or(bit);
  }
  const int64_t most = clusters[log].load(), half = sms / ranks / 2;
  int64_t w = a.rows;  // (rows a walker as above)
  if (w > half) w = w / 4 > half ? w / 4 : half;
  const int64_t room = resnorm_walkers(a, sms);
  w = w < most ? w : most;
  w = w < room ? w : room;
  *walkers = static_cast<int>(w);
  config.gridDim = dim3(static_cast<unsigned>(w * ranks));
  return cudaLaunchKernelEx(&config, kernel, a, *walkers, 1);
}

// A row is given to few threads with several pieces each (see the norm's backward). Short rows
// to as many groups a CTA as make 256 threads, or 128 of bf16: most of their kernels have
// 130 to 170 registers, of which an SM holds one CTA of 256 or three of 128 (320000 x 1000 bf16
// with a post norm: layer norms 990 us with 256 threads, 717 with 128; RMS norms 649 and 674;
// 800000 x 512 float32 1500 and 1545).
template <int N>
constexpr int resnorm_few() {
  return N == 8 ? 4 : 8;
}
template <typename T, int N, bool RMS, bool POST, int GATE>
cudaError_t resnorm_bwd_n(const ResNormArgs& a, int sms, int* walkers, cudaStream_t s) {
  const int64_t pieces = a.d / N;
  constexpr int few = resnorm_few<N>();
#define RESNORM_CASE(most, NV, G, R) \
  if (pieces <= most) return resnorm_bwd<T, N, NV, G, R, RMS, POST, GATE, ROWS_WHOLE>(a, 1, sms, walkers, s);
  RESNORM_CASE(32, 1, 32, 8)
  RESNORM_CASE(64, 2, 32, few)
  RESNORM_CASE(128, 2, 64, few / 2)
  RESNORM_CASE(256, 2, 128, 1)
  RESNORM_CASE(384, 3, 128, 1)
  RESNORM_CASE(512, 2, 256, 1)
  RESNORM_CASE(768, 3, 256, 1)
  RESNORM_CASE(1024, 2, 512, 1)
  if constexpr (GATE != GATE_ROWS) RESNORM_CASE(1536, 3, 512, 1)
#undef RESNORM_CASE
  return resnorm_bwd_cluster<T, N, 2, 512, RMS, POST, GATE, ROWS_WHOLE>(a, sms, walkers, s);
}
template <typename T, int N, bool RMS, bool POST, int GATE>
cudaError_t resnorm_bwd_shifted(const ResNormArgs& a, int step, int sms, int* walkers, cudaStream_t s) {
  const int64_t pieces = (a.d + 2 * N - 2) / N;  // a row begins up to N - 1 elements late
  constexpr int few = resnorm_few<N>();
#define RESNORM_CASE(most, NV, G, R) \
  if (pieces <= most) return resnorm_bwd<T, N, NV, G, R, RMS, POST, GATE, ROWS_SHIFTED>(a, step, sms, walkers, s);
  RESNORM_CASE(32, 1, 32, 8)
  RESNORM_CASE(64, 2, 32, few)
  RESNORM_CASE(128, 2, 64, few / 2)
  RESNORM_CASE(256, 2, 128, 1)
  RESNORM_CASE(384, 3, 128, 1)
  RESNORM_CASE(512, 2, 256, 1)
  RESNORM_CASE(1024, 2, 512, 1)
  if constexpr (GATE != GATE_ROWS) RESNORM_CASE(1536, 3, 512, 1)
#undef RESNORM_CASE
  return cudaErrorNotSupported;
}
template <typename T, bool RMS, bool POST, int GATE>
cudaError_t resnorm_bwd_strided(const ResNormArgs& a, int sms, int* walkers, cudaStream_t s) {
  if (const int step = resnorm_step(a, false)) {
    const cudaError_t e = resnorm_bwd_shifted<T, 16 / static_cast<int>(sizeof(T)), RMS, POST, GATE>(a, step, sms, walkers, s);
    if (e != cudaErrorNotSupported) return e;  // (longer rows)
  }
  if (a.d <= 256) return resnorm_bwd<T, 8, 1, 32, 8, RMS, POST, GATE, ROWS_STRIDED>(a, 1, sms, walkers, s);
  if (a.d <= 1024) return resnorm_bwd<T, 8, 1, 128, 1, RMS, POST, GATE, ROWS_STRIDED>(a, 1, sms, walkers, s);
  if (a.d <= 2048) return resnorm_bwd<T, 8, 1, 256, 1, RMS, POST, GATE, ROWS_STRIDED>(a, 1, sms, walkers, s);
  if (a.d <= 4096) return resnorm_bwd<T, 8, 1, 512, 1, RMS, POST, GATE, ROWS_STRIDED>(a, 1, sms, walkers, s);
  if constexpr (sizeof(T) == 2)
    if (a.d <= 8192) return resnorm_bwd<T, 8, 1, 1024, 1, RMS, POST, GATE, ROWS_STRIDED>(a, 1, sms, walkers, s);
  return resnorm_bwd_cluster<T, 8, 1, sizeof(T) == 2 ? 1024 : 512, RMS, POST, GATE, ROWS_STRIDED>(a, sms, walkers, s);
}

template <typename T, bool POST>
cudaError_t resnorm_bwd_kind(const ResNormArgs& a, bool whole, int sms, int* walkers, cudaStream_t s) {
  constexpr int N = 16 / static_cast<int>(sizeof(T));
  const int gate = !a.gate ? GATE_NONE : a.gate_rows == 1 ? GATE_ROWS : GATE_SHARED;
  if (!whole) {
    if (a.rms)
      return gate == GATE_NONE     ? resnorm_bwd_strided<T, true, POST, GATE_NONE>(a, sms, walkers, s)
             : gate == GATE_SHARED ? resnorm_bwd_strided<T, true, POST, GATE_SHARED>(a, sms, walkers, s)
                                   : resnorm_bwd_strided<T, true, POST, GATE_ROWS>(a, sms, walkers, s);
    return gate == GATE_NONE     ? resnorm_bwd_strided<T, false, POST, GATE_NONE>(a, sms, walkers, s)
           : gate == GATE_SHARED ? resnorm_bwd_strided<T, false, POST, GATE_SHARED>(a, sms, walkers, s)
                                 : resnorm_bwd_strided<T, false, POST, GATE_ROWS>(a, sms, walkers, s);
  }
  if (a.rms)
    return gate == GATE_NONE     ? resnorm_bwd_n<T, N, true, POST, GATE_NONE>(a, sms, walkers, s)
           : gate == GATE_SHARED ? resnorm_bwd_n<T, N, true, POST, GATE_SHARED>(a, sms, walkers, s)
                                 : resnorm_bwd_n<T, N, true, POST, GATE_ROWS>(a, sms, walkers, s);
  return gate == GATE_NONE     ? resnorm_bwd_n<T, N, false, POST, GATE_NONE>(a, sms, walkers, s)
         : gate == GATE_SHARED ? resnorm_bwd_n<T, N, false, POST, GATE_SHARED>(a, sms, walkers, s)
                               : resnorm_bwd_n<T, N, false, POST, GATE_ROWS>(a, sms, walkers, s);
}

// Whole: rows in 16-byte pieces. (A translation unit each.)
cudaError_t resnorm_bwd_f32(const ResNormArgs& a, bool whole, int sms, int* walkers, cudaStream_t s);
cudaError_t resnorm_bwd_f32_post(const ResNormArgs& a, bool whole, int sms, int* walkers, cudaStream_t s);
cudaError_t resnorm_bwd_bf16(const ResNormArgs& a, bool whole, int sms, int* walkers, cudaStream_t s);
cudaError_t resnorm_bwd_bf16_post(const ResNormArgs& a, bool whole, int sms, int* walkers, cudaStream_t s);

}  // namespace grpo
