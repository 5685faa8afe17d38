// One AdamW step over many tensors at once:
//   m = b1 m + (1 - b1) g,  v = b2 v + (1 - b2) g^2,
//   x = x (1 - lr wd) - lr_t m / (sqrt(v) / sqrt(1 - b2^t) + eps)
// with float32 arithmetic and states in float32 or in e4m3 codes with one
// power of two a block of 32. Bound by memory: every buffer is read and written
// once (30 bytes an element with bf16 parameters, masters and float32
// gradients and states; 10 with bf16 gradients and 8-bit states).
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include "internal.h"

namespace grpo {

namespace {

constexpr int kThreads = 256;
constexpr int kChunk = 4096;  // elements a CTA takes at a time (a multiple of 32: whole blocks)

struct AdamTable {
  AdamConst c;
  int n;
  uint32_t chunks;
  AdamTensor t[kAdamMaxTensors];
};

// The dither of element i: 16 bits (see grpo_adamw_step in grpo.h).
__device__ __forceinline__ uint32_t dither16(uint32_t i, uint32_t base) {
  return (i * 0x91E10DA5u + base) >> 16;
}

// Largest power-of-two byte E with amax * 2^(127 - E) <= 448 = 1.75 * 2^8:
// adding 0x1FFFFF to the bits carries into the exponent when the significand
// is above 1.75. 255 marks infinities and NaN.
__device__ __forceinline__ uint32_t block_scale(float amax) {
  const uint32_t b = __float_as_uint(amax);
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
__device__ __forceinline__ float dither_e4m3(float y, uint32_t d) {
  const float base = y < 0.015625f ? 0.015625f : 0.f;
  const uint32_t b = __float_as_uint(y + base) + (d << 4);
  return __uint_as_float(b & 0xFFF00000u) - base;
}

__device__ __forceinline__ float decode_e4m3(uint8_t c) {
  __nv_fp8_e4m3 q;
  q.__x = c;
  return static_cast<float>(q);
}
__device__ __forceinline__ uint8_t encode_e4m3(float y) {
  return __nv_cvt_float_to_fp8(y, __NV_SATFINITE, __NV_E4M3);
}

// Maximum over the warp that keeps a NaN.
__device__ __forceinline__ float warp_amax(float a) {
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) {
    const float b = __shfl_xor_sync(0xffffffffu, a, o);
    a = (a != a || a > b) ? a : b;
  }
  return a;
}

// The update of one element. Roundings are spelled out, so that every inlined
// copy gives the same bits and a tensor's result does not depend on its place
// in a table.
__device__ __forceinline__ void update(const AdamConst& c, float keep, float g, float& x, float& m,
                                       float& v) {
  g = __fmul_rn(g, c.grad_scale);
  m = __fmaf_rn(c.beta1, m, __fmul_rn(c.one_m_beta1, g));
  v = __fmaf_rn(c.beta2, v, __fmul_rn(__fmul_rn(c.one_m_beta2, g), g));
  const float den = __fmaf_rn(__fsqrt_rn(v), c.rsqrt_c2, c.eps);
  x = __fmaf_rn(-c.lr_t, __fdiv_rn(m, den), __fmul_rn(x, keep));
}

// A thread takes one element at a time; with 8-bit states a warp holds one
// block of 32.
template <int KIND>
__global__ void __launch_bounds__(kThreads) k_adamw(const __grid_constant__ AdamTable tab) {
  constexpr bool kPBf16 = (KIND & ADAM_P_BF16) != 0, kGBf16 = (KIND & ADAM_G_BF16) != 0;
  constexpr bool kMaster = (KIND & ADAM_MASTER) != 0, k8 = (KIND & ADAM_BITS8) != 0;
  const AdamConst& c = tab.c;
  for (uint32_t chunk = blockIdx.x; chunk < tab.chunks; chunk += gridDim.x) {
    int lo = 0, hi = tab.n - 1;  // the last tensor whose first chunk is not past this one
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (tab.t[mid].chunk0 <= chunk) lo = mid;
      else hi = mid - 1;
    }
    const AdamTensor& t = tab.t[lo];
    const int64_t i0 = static_cast<int64_t>(chunk - t.chunk0) * kChunk;
    const int64_t end = t.n - i0 < kChunk ? t.n - i0 : kChunk;
    for (int k = threadIdx.x; k < kChunk; k += kThreads) {
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
          m = decode_e4m3(static_cast<const uint8_t*>(t.m)[i]) * scale_value(t.ms[blk]);
          v = decode_e4m3(static_cast<const uint8_t*>(t.v)[i]) * scale_value(t.vs[blk]);
        } else {
          m = static_cast<const float*>(t.m)[i];
          v = static_cast<const float*>(t.v)[i];
        }
        update(c, t.keep, g, x, m, v);
      }
      const uint32_t i32 = static_cast<uint32_t>(i);
      if (k8) {
        const uint32_t em = block_scale(warp_amax(fabsf(m))), ev = block_scale(warp_amax(v));
        const float ym = dither_e4m3(fabsf(m) * inv_scale_value(em), dither16(i32, c.dither));
        float yv = dither_e4m3(v * inv_scale_value(ev), dither16(i32, c.dither + 0x55555555u));
        const bool zero = warp_amax(v) == 0.f;
        if (!zero) yv = fmaxf(yv, 0.001953125f);
        if (in) {
          static_cast<uint8_t*>(t.m_out)[i] = encode_e4m3(copysignf(ym, m));
          static_cast<uint8_t*>(t.v_out)[i] = encode_e4m3(yv);
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
        if (!kPBf16) {
          static_cast<float*>(t.p_out)[i] = x;
        } else if (kMaster || !(fabsf(x) < INFINITY)) {
          static_cast<__nv_bfloat16*>(t.p_out)[i] = __float2bfloat16_rn(x);
        } else {
          const uint32_t b = __float_as_uint(x) + dither16(i32, c.dither + 0xAAAAAAAAu);
          static_cast<__nv_bfloat16*>(t.p_out)[i] =
              __ushort_as_bfloat16(static_cast<unsigned short>(b >> 16));
        }
      }
    }
  }
}

template <int KIND>
cudaError_t launch_kind(const AdamTable& tab, int grid, cudaStream_t s) {
  k_adamw<KIND><<<grid, kThreads, 0, s>>>(tab);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_adamw(AdamTensor* t, int n, int kind, const AdamConst& c, int sms,
                         cudaStream_t s) {
  AdamTable tab;
  tab.c = c;
  tab.n = n;
  uint32_t chunks = 0;
  for (int i = 0; i < n; ++i) {
    tab.t[i] = t[i];
    tab.t[i].chunk0 = chunks;
    chunks += static_cast<uint32_t>((t[i].n + kChunk - 1) / kChunk);
  }
  tab.chunks = chunks;
  const int grid = static_cast<int>(chunks < 8u * sms ? chunks : 8u * sms);
  switch (kind) {
#define ADAM_CASE(k) case k: return launch_kind<k>(tab, grid, s);
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
