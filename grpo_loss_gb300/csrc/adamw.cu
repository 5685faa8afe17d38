// One AdamW step over many tensors at once:
//   m = b1 m + (1 - b1) g,  v = b2 v + (1 - b2) g^2,
//   x = x (1 - lr wd) - lr_t m / (sqrt(v) / sqrt(1 - b2^t) + eps)
// with float32 arithmetic and states in float32 or in e4m3 codes with one
// power of two a block of 32. Bound by memory: every buffer is read and written
// once (30 bytes an element with bf16 parameters, masters and float32
// gradients and states; 10 with bf16 gradients and 8-bit states). 233 M elements
// with masters: 992 us (7.1 TB/s); with 8-bit states and float32 gradients 467 us
// (6.1 TB/s) into other buffers: there some 60 instructions an element weigh as much as
// the bytes (with the update's arithmetic one element at a time, 71 of them, 557 us; with
// pairs 513; the rest is the second step's bytes asked for ahead). In place the latter
// takes 633 us. Buffers off a 16-byte boundary, element by element: 1739 and 3414 us.
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include "f32x2.cuh"
#include "internal.h"

namespace grpo {

namespace {

constexpr int kThreads = 256;
constexpr int kChunk = 4096;  // elements a CTA takes at a time (a multiple of 32: whole blocks)

// The table of one launch, a kernel parameter: no copy to the device goes before
// the launch, and a captured launch holds its own.
struct AdamTable {
  AdamConst c;
  int n;
  uint32_t chunks;
  AdamTensor t[kAdamMaxTensors];
};

// The dither of element i at step t: the high 16 bits of i * kDitherIndex + t *
// 0xC13FA9A9 + salt (see grpo_adamw_step in grpo.h).
constexpr uint32_t kDitherIndex = 0x91E10DA5u, kSaltV = 0x55555555u, kSaltP = 0xAAAAAAAAu;

// Smallest power-of-two byte E with amax * 2^(127 - E) <= 448 = 1.75 * 2^8:
// adding 0x1FFFFF to the bits carries into the exponent when the significand
// is above 1.75. 255 marks infinities and NaN.
__device__ __forceinline__ uint32_t block_scale(uint32_t b) {
  if (b >= 0x7F800000u) return 255u;
  const int e = static_cast<int>((b + 0x1FFFFFu) >> 23) - 8;
  return e < 0 ? 0u : static_cast<uint32_t>(e);
}
// 2^(E - 127); E = 0 is the subnormal 2^-127, 255 reads as NaN.
__device__ __forceinline__ float scale_value(uint32_t e) {
  return __uint_as_float(e == 0 ? 0x00400000u : e == 255 ? 0x7FC00000u : e << 23);
}
// 2^(127 - E)
__device__ __forceinline__ float inv_scale_value(uint32_t e) {
  return __uint_as_float(e == 255 ? 0x3F800000u : (254u - e) << 23);
}

// Magnitude y <= 448 to the e4m3 grid, rounded down after adding the dither d
// (2^-16 of a grid step). Above 2^-6 a step is the last of three significand
// bits, so the dither is added to the 20 bits below it; under 2^-6, where the
// step is 2^-9 throughout, y is first moved to [2^-6, 2^-5), whose significand
// step is the same.
__device__ __forceinline__ float dither_e4m3(float y, uint32_t d) {  // the dither: d's high 16 bits
  const float base = y < 0.015625f ? 0.015625f : 0.f;
  uint32_t high;  // (a shift that the compiler does not fold, to a shift and add in one)
  asm("shr.u32 %0, %1, 16;" : "=r"(high) : "r"(d));
  const uint32_t b = __float_as_uint(y + base) + (high << 4);
  return __uint_as_float(b & 0xFFF00000u) - base;
}

// The update of one element. Roundings are spelled out, so that every inlined
// copy gives the same bits and a tensor's result does not depend on its place
// in a table; those of the moments are the formula's own, operation by operation,
// so that 8-bit states are the same as those of any float32 code. The root and the quotient are the special-function unit's, some
// 2^-22 off together: of the update, not of the parameter.
__device__ __forceinline__ void update(const AdamConst& c, float gs, float keep, float g, float& x, float& m,
                                       float& v) {
  g = __fmul_rn(g, gs);
  m = __fadd_rn(__fmul_rn(c.beta1, m), __fmul_rn(c.one_m_beta1, g));
  v = __fadd_rn(__fmul_rn(c.beta2, v), __fmul_rn(__fmul_rn(c.one_m_beta2, g), g));
  float root;
  asm("sqrt.approx.f32 %0, %1;" : "=f"(root) : "f"(v));
  // (the root of a float is at least 2^-75: with eps = 0, too, den is normal or 0)
  const float den = __fmaf_rn(root, c.rsqrt_c2, c.eps);
  float inv;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(den));
  x = __fmaf_rn(-c.lr_t, __fmul_rn(m, inv), __fmul_rn(x, keep));
}

// The same of two elements, bit by bit. (The sums are one at a time: the assembler
// fuses a product and a sum of pairs into one rounding.)
__device__ __forceinline__ void update2(const AdamConst& c, float gs, float keep, float* g, float* x, float* m, float* v) {
  const uint64_t g2 = mul2(pair_of(g[0], g[1]), pair_of(gs));
  const float2 m0 = of_pair(mul2(pair_of(c.beta1), pair_of(m[0], m[1]))), m1 = of_pair(mul2(pair_of(c.one_m_beta1), g2));
  const float2 v0 = of_pair(mul2(pair_of(c.beta2), pair_of(v[0], v[1])));
  const float2 v1 = of_pair(mul2(mul2(pair_of(c.one_m_beta2), g2), g2));
  const float2 mm = make_float2(__fadd_rn(m0.x, m1.x), __fadd_rn(m0.y, m1.y));
  const float2 vv = make_float2(__fadd_rn(v0.x, v1.x), __fadd_rn(v0.y, v1.y));
  float2 root, inv;
  asm("sqrt.approx.f32 %0, %1;" : "=f"(root.x) : "f"(vv.x));
  asm("sqrt.approx.f32 %0, %1;" : "=f"(root.y) : "f"(vv.y));
  const float2 den = of_pair(fma2(pair_of(root.x, root.y), pair_of(c.rsqrt_c2), pair_of(c.eps)));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv.x) : "f"(den.x));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv.y) : "f"(den.y));
  const float2 xx = of_pair(fma2(pair_of(-c.lr_t), mul2(pair_of(mm.x, mm.y), pair_of(inv.x, inv.y)), mul2(pair_of(x[0], x[1]), pair_of(keep))));
  m[0] = mm.x, m[1] = mm.y, v[0] = vv.x, v[1] = vv.y, x[0] = xx.x, x[1] = xx.y;
}

// W consecutive elements of a buffer, W = 4 or 8. With float32 states a thread
// takes four: a warp's accesses are then whole 128-byte lines for every type.
// (Eight, as two 16-byte accesses, reach each line twice: 1179 instead of 998 us
// on 233 M elements with masters.) With 8-bit states, where the instructions of
// a piece weigh more than its bytes, it takes eight.
template <bool BF16, int W>
__device__ __forceinline__ void load(const void* p, int k, float (&v)[W]) {
  if constexpr (BF16) {
    uint32_t w[W / 2];
    const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(p) + k;
    if constexpr (W == 8) {
      const uint4 r = __ldcs(reinterpret_cast<const uint4*>(q));
      w[0] = r.x, w[1] = r.y, w[2] = r.z, w[3] = r.w;
    } else {
      const uint2 r = __ldcs(reinterpret_cast<const uint2*>(q));
      w[0] = r.x, w[1] = r.y;
    }
#pragma unroll
    for (int e = 0; e < W; ++e) v[e] = __uint_as_float((e & 1) ? (w[e / 2] & 0xFFFF0000u) : (w[e / 2] << 16));
  } else {
    const float4* q = reinterpret_cast<const float4*>(static_cast<const float*>(p) + k);
#pragma unroll
    for (int f = 0; f < W / 4; ++f) {
      const float4 a = W == 4 ? __ldcs(q) : q[f];  // (of eight, the second half is in the same line)
      v[4 * f] = a.x, v[4 * f + 1] = a.y, v[4 * f + 2] = a.z, v[4 * f + 3] = a.w;
    }
  }
}
template <int W>
__device__ __forceinline__ void store(void* p, int k, const float (&v)[W]) {
  float4* q = reinterpret_cast<float4*>(static_cast<float*>(p) + k);
#pragma unroll
  for (int f = 0; f < W / 4; ++f) __stcs(q + f, make_float4(v[4 * f], v[4 * f + 1], v[4 * f + 2], v[4 * f + 3]));
}
// Decodes or encodes a pair of e4m3 codes.
__device__ __forceinline__ float2 decode2(uint32_t c) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(c), __NV_E4M3);
  return __half22float2(__half2(h));
}
__device__ __forceinline__ uint32_t encode2(float lo, float hi) {
  return __nv_cvt_float2_to_fp8x2(make_float2(lo, hi), __NV_SATFINITE, __NV_E4M3);
}
// bf16 bits of x: to nearest beside a master, else dithered
template <bool NEAREST>
__device__ __forceinline__ uint32_t param_bits(float x, uint32_t d) {
  if (NEAREST || !(fabsf(x) < INFINITY)) return __bfloat16_as_ushort(__float2bfloat16_rn(x));
  return (__float_as_uint(x) + d) >> 16;
}
// Magnitude bits: they order like the magnitudes, infinities and NaN above all.
__device__ __forceinline__ uint32_t magnitude(float x) { return __float_as_uint(x) & 0x7FFFFFFFu; }

// Asks L2 for n elements from `from` on.
__device__ __forceinline__ void prefetch(const char* p, int size, int from, int n) {
  asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(p + from * size), "r"(n * size) : "memory");
}

// Whole pieces of W elements of a chunk that starts at element i0, `end` elements
// in all (a multiple of 32; every buffer on a 16-byte boundary). With 8-bit
// states four threads hold a block of 32.
template <int KIND>
__device__ __forceinline__ void pieces(const AdamConst& c, float gs, const AdamTensor& t, int64_t i0, int end) {
  constexpr bool kPBf16 = (KIND & ADAM_P_BF16) != 0, kGBf16 = (KIND & ADAM_G_BF16) != 0;
  constexpr bool kMaster = (KIND & ADAM_MASTER) != 0, k8 = (KIND & ADAM_BITS8) != 0;
  constexpr int W = k8 ? 8 : 4, U = k8 ? 1 : 2;  // U pieces' loads are in flight together
  // the chunk's own pointers: elements of it have 32-bit offsets
  auto at = [&](const void* p, int size) { return static_cast<const char*>(p) + i0 * size; };
  auto to = [&](void* p, int size) { return static_cast<char*>(p) + i0 * size; };
  constexpr int kSS = k8 ? 1 : 4;
  const char* const g_in = at(t.g, kGBf16 ? 2 : 4);
  const char* const x_in = kMaster ? at(t.w, 4) : at(t.p, kPBf16 ? 2 : 4);
  const char* const m_in = at(t.m, kSS);
  const char* const v_in = at(t.v, kSS);
  char* const m_to = to(t.m_out, kSS);
  char* const v_to = to(t.v_out, kSS);
  char* const p_to = to(t.p_out, kPBf16 ? 2 : 4);
  const float keep = t.keep;
  if (k8 && threadIdx.x == 0 && end > kThreads * W) {
    // the second step's bytes, asked for while the first's are waited for (registers for
    // them there are none: two steps' loads at a time spill, 647 us); with float32
    // states two steps' loads are in flight as it is
    const int from = kThreads * W, n = end - from;
    prefetch(g_in, kGBf16 ? 2 : 4, from, n);
    prefetch(x_in, kMaster || !kPBf16 ? 4 : 2, from, n);
    prefetch(m_in, 1, from, n);
    prefetch(v_in, 1, from, n);
  }
  for (int k0 = threadIdx.x * W; k0 < end; k0 += kThreads * W * U) {
    float g[U][W], x[U][W], m[U][W], v[U][W];
    uint2 cm, cv;
    uint32_t sm = 0, sv = 0;
#pragma unroll
    for (int j = 0; j < U; ++j) {
      const int k = k0 + j * kThreads * W;
      if (k < end) {
        load<kGBf16, W>(g_in, k, g[j]);
        load<kPBf16 && !kMaster, W>(x_in, k, x[j]);
        if constexpr (k8) {
          cm = __ldcs(reinterpret_cast<const uint2*>(m_in + k));
          cv = __ldcs(reinterpret_cast<const uint2*>(v_in + k));
          sm = t.ms[(i0 + k) >> 5];
          sv = t.vs[(i0 + k) >> 5];
        } else {
          load<false, W>(m_in, k, m[j]);
          load<false, W>(v_in, k, v[j]);
        }
      }
    }
#pragma unroll
    for (int j = 0; j < U; ++j) {
      const int k = k0 + j * kThreads * W;
      if (k >= end) break;  // (a block's threads are in or out together)
      if constexpr (k8) {
        const float a = scale_value(sm), b = scale_value(sv);
#pragma unroll
        for (int e = 0; e < W; e += 2) {
          const float2 p = decode2((e < 4 ? cm.x : cm.y) >> (8 * (e & 3)));
          const float2 q = decode2((e < 4 ? cv.x : cv.y) >> (8 * (e & 3)));
          const float2 m2 = of_pair(mul2(pair_of(p.x, p.y), pair_of(a))), v2 = of_pair(mul2(pair_of(q.x, q.y), pair_of(b)));
          m[j][e] = m2.x, m[j][e + 1] = m2.y;
          v[j][e] = v2.x, v[j][e + 1] = v2.y;
        }
      }
#pragma unroll
      for (int e = 0; e < W; e += 2) update2(c, gs, keep, g[j] + e, x[j] + e, m[j] + e, v[j] + e);
      const uint32_t d0 = static_cast<uint32_t>(i0 + k) * kDitherIndex + c.dither;  // of the first element
      if constexpr (k8) {
        uint32_t am = 0, av = 0;  // (v has no sign; a NaN's would leave it the largest)
#pragma unroll
        for (int e = 0; e < W; ++e) {
          am = max(am, magnitude(m[j][e]));
          av = max(av, __float_as_uint(v[j][e]));
        }
        const uint32_t who = 0xFu << (threadIdx.x & 28);
#pragma unroll
        for (int o = 1; o < 4; o <<= 1) {
          am = max(am, __shfl_xor_sync(who, am, o));
          av = max(av, __shfl_xor_sync(who, av, o));
        }
        const uint32_t em = block_scale(am), ev = block_scale(av);
        const float im = inv_scale_value(em), iv = inv_scale_value(ev);
        const float least = av == 0 ? 0.f : 0.001953125f;
        float ym[W], yv[W];
#pragma unroll
        for (int e = 0; e < W; ++e) {
          const uint32_t d = d0 + e * kDitherIndex;
          const uint64_t p = mul2(pair_of(m[j][e & ~1], m[j][e | 1]), pair_of(im)), q = mul2(pair_of(v[j][e & ~1], v[j][e | 1]), pair_of(iv));
          ym[e] = copysignf(dither_e4m3(fabsf((e & 1) ? of_pair(p).y : of_pair(p).x), d), m[j][e]);
          yv[e] = fmaxf(dither_e4m3((e & 1) ? of_pair(q).y : of_pair(q).x, d + kSaltV), least);
        }
        __stcs(reinterpret_cast<uint2*>(m_to + k), make_uint2(encode2(ym[0], ym[1]) | encode2(ym[2], ym[3]) << 16,
                                                              encode2(ym[4], ym[5]) | encode2(ym[6], ym[7]) << 16));
        __stcs(reinterpret_cast<uint2*>(v_to + k), make_uint2(encode2(yv[0], yv[1]) | encode2(yv[2], yv[3]) << 16,
                                                              encode2(yv[4], yv[5]) | encode2(yv[6], yv[7]) << 16));
        if ((k & 31) == 0) {
          t.ms_out[(i0 + k) >> 5] = static_cast<uint8_t>(em);
          t.vs_out[(i0 + k) >> 5] = static_cast<uint8_t>(ev);
        }
      } else {
        store<W>(m_to, k, m[j]);
        store<W>(v_to, k, v[j]);
      }
      if constexpr (kMaster) store<W>(to(t.w_out, 4), k, x[j]);
      if constexpr (kPBf16) {
        uint32_t b[W / 2];
#pragma unroll
        for (int e = 0; e < W; e += 2) {
          const uint32_t d = d0 + e * kDitherIndex + kSaltP;
          b[e / 2] = param_bits<kMaster>(x[j][e], d >> 16) |
                     param_bits<kMaster>(x[j][e + 1], (d + kDitherIndex) >> 16) << 16;
        }
        __nv_bfloat16* q = reinterpret_cast<__nv_bfloat16*>(p_to) + k;
        if constexpr (W == 8) __stcs(reinterpret_cast<uint4*>(q), make_uint4(b[0], b[1], b[2], b[3]));
        else __stcs(reinterpret_cast<uint2*>(q), make_uint2(b[0], b[1]));
      } else {
        store<W>(p_to, k, x[j]);
      }
    }
  }
}

// Elements first to end of a chunk one by one (a tensor's ragged end, buffers
// off a 16-byte boundary); with 8-bit states a warp holds a block of 32.
template <int KIND>
__device__ __forceinline__ void singles(const AdamConst& c, float gs, const AdamTensor& t, int64_t i0, int first,
                                        int end) {
  constexpr bool kPBf16 = (KIND & ADAM_P_BF16) != 0, kGBf16 = (KIND & ADAM_G_BF16) != 0;
  constexpr bool kMaster = (KIND & ADAM_MASTER) != 0, k8 = (KIND & ADAM_BITS8) != 0;
  for (int k = first + threadIdx.x; k < kChunk; k += kThreads) {  // (first is a multiple of 32)
    const bool in = k < end;
    if (!__any_sync(0xffffffffu, in)) break;
    const int64_t i = i0 + k, blk = i >> 5;
    float g = 0.f, x = 0.f, m = 0.f, v = 0.f;
    if (in) {
      g = kGBf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(t.g)[i])
                 : static_cast<const float*>(t.g)[i];
      x = kMaster ? t.w[i]
          : kPBf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(t.p)[i])
                   : static_cast<const float*>(t.p)[i];
      if (k8) {
        m = decode2(static_cast<const uint8_t*>(t.m)[i]).x * scale_value(t.ms[blk]);
        v = decode2(static_cast<const uint8_t*>(t.v)[i]).x * scale_value(t.vs[blk]);
      } else {
        m = static_cast<const float*>(t.m)[i];
        v = static_cast<const float*>(t.v)[i];
      }
      update(c, gs, t.keep, g, x, m, v);
    }
    const uint32_t d = static_cast<uint32_t>(i) * kDitherIndex + c.dither;
    if (k8) {
      const uint32_t av = __reduce_max_sync(0xffffffffu, magnitude(v));
      const uint32_t em = block_scale(__reduce_max_sync(0xffffffffu, magnitude(m))), ev = block_scale(av);
      const float ym = dither_e4m3(fabsf(m) * inv_scale_value(em), d);
      const float yv = fmaxf(dither_e4m3(v * inv_scale_value(ev), d + kSaltV), av == 0 ? 0.f : 0.001953125f);
      if (in) {
        static_cast<uint8_t*>(t.m_out)[i] = static_cast<uint8_t>(encode2(copysignf(ym, m), 0.f));
        static_cast<uint8_t*>(t.v_out)[i] = static_cast<uint8_t>(encode2(yv, 0.f));
        if ((k & 31) == 0) {
          t.ms_out[blk] = static_cast<uint8_t>(em);
          t.vs_out[blk] = static_cast<uint8_t>(ev);
        }
      }
    } else if (in) {
      static_cast<float*>(t.m_out)[i] = m;
      static_cast<float*>(t.v_out)[i] = v;
    }
    if (in) {
      if (kMaster) t.w_out[i] = x;
      if (kPBf16)
        static_cast<__nv_bfloat16*>(t.p_out)[i] =
            __ushort_as_bfloat16(static_cast<unsigned short>(param_bits<kMaster>(x, (d + kSaltP) >> 16)));
      else
        static_cast<float*>(t.p_out)[i] = x;
    }
  }
}

template <int KIND>
__global__ void __launch_bounds__(kThreads, (KIND & ADAM_BITS8) ? 4 : 3) k_adamw(const __grid_constant__ AdamTable tab) {
  // (a kernel of its own with the factor: without one the scale stays a constant)
  const float gs = (KIND & ADAM_FACTOR) ? __fmul_rn(tab.c.grad_scale, *tab.c.factor) : tab.c.grad_scale;
  for (uint32_t chunk = blockIdx.x; chunk < tab.chunks; chunk += gridDim.x) {
    int lo = 0, hi = tab.n - 1;  // the last tensor whose first chunk is not past this one
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (tab.t[mid].chunk0 <= chunk) lo = mid;
      else hi = mid - 1;
    }
    const AdamTensor& t = tab.t[lo];
    const int64_t i0 = static_cast<int64_t>(chunk - t.chunk0) * kChunk;
    const int end = static_cast<int>(t.n - i0 < kChunk ? t.n - i0 : kChunk);
    const int whole = t.on16 ? end & ~31 : 0;
    pieces<KIND>(tab.c, gs, t, i0, whole);
    if (whole < end) singles<KIND>(tab.c, gs, t, i0, whole, end);
  }
}

static_assert(sizeof(AdamTable) <= 32764, "kernel parameters");

template <int KIND>
cudaError_t launch_kind(const AdamTable& tab, int64_t grid, cudaStream_t s) {
  k_adamw<KIND><<<static_cast<unsigned>(grid), kThreads, 0, s>>>(tab);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_adamw(AdamTensor* t, int n, int kind, const AdamConst& c,
                         cudaStream_t s) {
  AdamTable tab;
  tab.c = c;
  tab.n = n;
  uint32_t chunks = 0;
  for (int i = 0; i < n; ++i) {
    tab.t[i] = t[i];
    tab.t[i].chunk0 = chunks;
    chunks += static_cast<uint32_t>((t[i].n + kChunk - 1) / kChunk);
    uintptr_t low = 0;  // (narrower types need less)
    for (const void* p : {t[i].g, t[i].p, static_cast<const void*>(t[i].w), t[i].m, t[i].v,
                          static_cast<const void*>(t[i].p_out), static_cast<const void*>(t[i].w_out),
                          static_cast<const void*>(t[i].m_out), static_cast<const void*>(t[i].v_out)})
      low |= reinterpret_cast<uintptr_t>(p);
    tab.t[i].on16 = low % 16 == 0;
  }
  tab.chunks = chunks;
  // a CTA a chunk: the SMs take the next as they come free (998 us on 233 M elements
  // with masters; CTAs that walk over the chunks, 4 to 16 an SM, 1047 to 1078)
  const int64_t grid = chunks < (1u << 30) ? chunks : 1 << 30;
  switch (kind) {
#define ADAM_CASE(k) \
  case k: return launch_kind<k>(tab, grid, s); \
  case (k) | ADAM_FACTOR: return launch_kind<(k) | ADAM_FACTOR>(tab, grid, s);
    ADAM_CASE(0)
    ADAM_CASE(ADAM_P_BF16)
    ADAM_CASE(ADAM_G_BF16)
    ADAM_CASE(ADAM_P_BF16 | ADAM_G_BF16)
    ADAM_CASE(ADAM_P_BF16 | ADAM_MASTER)
    ADAM_CASE(ADAM_P_BF16 | ADAM_G_BF16 | ADAM_MASTER)
    ADAM_CASE(ADAM_BITS8)
    ADAM_CASE(ADAM_BITS8 | ADAM_P_BF16)
    ADAM_CASE(ADAM_BITS8 | ADAM_G_BF16)
    ADAM_CASE(ADAM_BITS8 | ADAM_P_BF16 | ADAM_G_BF16)
    ADAM_CASE(ADAM_BITS8 | ADAM_P_BF16 | ADAM_MASTER)
    ADAM_CASE(ADAM_BITS8 | ADAM_P_BF16 | ADAM_G_BF16 | ADAM_MASTER)
#undef ADAM_CASE
  }
  return cudaErrorInvalidValue;
}

}  // namespace grpo
