// C entry points of the operators around the loss head: token sampling, layer
// norm and AdamW. Argument checks and launches only; the mathematics and the
// layouts stand at the kernels (sample.cu, norm.cu, adamw.cu).
#include <float.h>
#include <math.h>

#include "../../include/grpo.h"
#include "api_common.h"
#include "internal.h"

using namespace grpo;

namespace {

constexpr int64_t kMaxRows = (static_cast<int64_t>(1) << 31) - 1;
constexpr int64_t kMaxNormDim = 65536;

bool is_f32_or_bf16(grpo_dtype t) { return t == GRPO_F32 || t == GRPO_BF16; }
size_t elem_size(grpo_dtype t) { return t == GRPO_F32 ? 4 : 2; }

// ------------------------------------------------------------- layer norm
grpo_status norm_args(const grpo_layernorm_problem* p, NormArgs* a) {
  if (!p || p->rows < 0 || p->d < 1) return GRPO_ERR_INVALID_ARG;
  if (!is_f32_or_bf16(p->dtype) || !is_f32_or_bf16(p->param_dtype)) return GRPO_ERR_INVALID_ARG;
  if (p->rms != 0 && p->rms != 1) return GRPO_ERR_INVALID_ARG;
  if (!isfinite(p->eps) || p->eps < 0.f) return GRPO_ERR_INVALID_ARG;
  for (int64_t ld : {p->ld_x, p->ld_y, p->ld_dy, p->ld_dx})
    if (ld != 0 && ld < p->d) return GRPO_ERR_INVALID_ARG;
  if (p->d > kMaxNormDim || p->rows > kMaxRows) return GRPO_ERR_UNSUPPORTED;
  *a = NormArgs();
  a->rows = p->rows;
  a->d = p->d;
  a->ld_x = p->ld_x ? p->ld_x : p->d;
  a->ld_y = p->ld_y ? p->ld_y : p->d;
  a->ld_dy = p->ld_dy ? p->ld_dy : p->d;
  a->ld_dx = p->ld_dx ? p->ld_dx : p->d;
  a->eps = p->eps;
  a->rms = p->rms;
  a->bf16 = p->dtype == GRPO_BF16 ? 1 : 0;
  a->param_bf16 = p->param_dtype == GRPO_BF16 ? 1 : 0;
  return GRPO_OK;
}

// The parameter and state buffers of one tensor.
grpo_status adamw_buffers(const grpo_adamw_tensor& t, bool eight) {
  if (!t.param || !t.m || !t.v) return GRPO_ERR_INVALID_ARG;
  if (eight != (t.m_scale != nullptr) || eight != (t.v_scale != nullptr))
    return GRPO_ERR_INVALID_ARG;
  const size_t ss = eight ? 1 : 4;
  if (!aligned_to(t.param, elem_size(t.param_dtype)) || !aligned_to(t.master, 4) ||
      !aligned_to(t.m, ss) || !aligned_to(t.v, ss))
    return GRPO_ERR_UNSUPPORTED;
  return GRPO_OK;
}

size_t norm_bwd_bytes(const NormArgs& a, int sms) {
  return sizeof(float) * 2 * static_cast<size_t>(norm_parts(a, sms)) * static_cast<size_t>(a.d);
}

}  // namespace

extern "C" {

grpo_status grpo_sample(const grpo_sample_problem* p, const void* logits, const float* u,
                        const float* temperature, const int32_t* top_k, const float* top_p,
                        const float* min_p, int32_t* tokens, float* logp, cudaStream_t stream) {
  NvtxRange nvtx_range("grpo_sample");
  if (!p || p->rows < 0 || p->V < 1) return GRPO_ERR_INVALID_ARG;
  if (!is_f32_or_bf16(p->dtype)) return GRPO_ERR_INVALID_ARG;
  if (p->ld != 0 && p->ld < p->V) return GRPO_ERR_INVALID_ARG;
  if (p->rows > kMaxRows || p->V > kMaxRows) return GRPO_ERR_UNSUPPORTED;
  if (p->rows == 0) return GRPO_OK;
  if (!logits || !u || !tokens || !logp) return GRPO_ERR_INVALID_ARG;
  if (!aligned_to(logits, elem_size(p->dtype)) || !aligned_to(u, 4) ||
      !aligned_to(temperature, 4) || !aligned_to(top_k, 4) || !aligned_to(top_p, 4) ||
      !aligned_to(min_p, 4) || !aligned_to(tokens, 4) || !aligned_to(logp, 4))
    return GRPO_ERR_UNSUPPORTED;
  int sms = 0;
  const grpo_status st = device_info(&sms);
  if (st != GRPO_OK) return st;
  SampleArgs a;
  a.logits = logits;
  a.rows = p->rows;
  a.V = p->V;
  a.ld = p->ld ? p->ld : p->V;
  a.bf16 = p->dtype == GRPO_BF16 ? 1 : 0;
  a.u = u;
  a.temperature = temperature;
  a.top_k = top_k;
  a.top_p = top_p;
  a.min_p = min_p;
  a.tokens = tokens;
  a.logp = logp;
  LAUNCH(K_SAMPLE, stream, launch_sample(a, sms, stream));
  return GRPO_OK;
}

grpo_status grpo_layernorm_workspace_size(const grpo_layernorm_problem* p, size_t* bwd_bytes) {
  NormArgs a;
  grpo_status st = norm_args(p, &a);
  if (st != GRPO_OK) return st;
  int sms = 0;
  if ((st = device_info(&sms)) != GRPO_OK) return st;
  if (bwd_bytes) *bwd_bytes = norm_bwd_bytes(a, sms);
  return GRPO_OK;
}

grpo_status grpo_layernorm_fwd(const grpo_layernorm_problem* p, const void* x,
                               const void* weight, const void* bias, void* y, float* mean,
                               float* rstd, cudaStream_t stream) {
  NvtxRange nvtx_range("grpo_layernorm_fwd");
  NormArgs a;
  grpo_status st = norm_args(p, &a);
  if (st != GRPO_OK) return st;
  if (a.rms && bias) return GRPO_ERR_INVALID_ARG;
  if (a.rows == 0) return GRPO_OK;
  if (!x || !weight || !y) return GRPO_ERR_INVALID_ARG;
  const size_t es = elem_size(p->dtype), ps = elem_size(p->param_dtype);
  if (!aligned_to(x, es) || !aligned_to(y, es) || !aligned_to(weight, ps) ||
      !aligned_to(bias, ps) || !aligned_to(mean, 4) || !aligned_to(rstd, 4))
    return GRPO_ERR_UNSUPPORTED;
  int sms = 0;
  if ((st = device_info(&sms)) != GRPO_OK) return st;
  a.x = x;
  a.weight = weight;
  a.bias = bias;
  a.y = y;
  a.mean = a.rms ? nullptr : mean;
  a.rstd = rstd;
  LAUNCH(K_NORM_FWD, stream, launch_norm_fwd(a, sms, stream));
  return GRPO_OK;
}

grpo_status grpo_layernorm_bwd(const grpo_layernorm_problem* p, const void* x,
                               const void* weight, const void* dy, const float* mean,
                               const float* rstd, void* dx, float* dweight, float* dbias,
                               void* workspace, size_t workspace_bytes, cudaStream_t stream) {
  NvtxRange nvtx_range("grpo_layernorm_bwd");
  NormArgs a;
  grpo_status st = norm_args(p, &a);
  if (st != GRPO_OK) return st;
  if (a.rms && dbias) return GRPO_ERR_INVALID_ARG;
  const size_t es = elem_size(p->dtype), ps = elem_size(p->param_dtype);
  if (!aligned_to(dweight, 4) || !aligned_to(dbias, 4)) return GRPO_ERR_UNSUPPORTED;
  if (a.rows == 0) {  // empty sums
    if (dweight && cudaMemsetAsync(dweight, 0, sizeof(float) * a.d, stream) != cudaSuccess)
      return GRPO_ERR_CUDA;
    if (dbias && cudaMemsetAsync(dbias, 0, sizeof(float) * a.d, stream) != cudaSuccess)
      return GRPO_ERR_CUDA;
    return GRPO_OK;
  }
  if (!x || !weight || !dy || !rstd || !dx || (!mean && !a.rms)) return GRPO_ERR_INVALID_ARG;
  if (!aligned_to(x, es) || !aligned_to(dy, es) || !aligned_to(dx, es) ||
      !aligned_to(weight, ps) || !aligned_to(mean, 4) || !aligned_to(rstd, 4))
    return GRPO_ERR_UNSUPPORTED;
  int sms = 0;
  if ((st = device_info(&sms)) != GRPO_OK) return st;
  const bool sums = dweight || dbias;
  if (sums && (!workspace || !aligned16(workspace) || workspace_bytes < norm_bwd_bytes(a, sms)))
    return GRPO_ERR_WORKSPACE;
  a.x = x;
  a.weight = weight;
  a.dy = dy;
  a.dx = dx;
  a.mean = a.rms ? nullptr : const_cast<float*>(mean);
  a.rstd = const_cast<float*>(rstd);
  a.dweight = dweight;
  a.dbias = dbias;
  a.partial = sums ? static_cast<float*>(workspace) : nullptr;
  int groups = 0;
  LAUNCH(K_NORM_BWD, stream, launch_norm_bwd(a, sms, &groups, stream));
  if (sums) LAUNCH(K_NORM_COLSUM, stream, launch_norm_colsum(a, groups, stream));
  return GRPO_OK;
}

grpo_status grpo_adamw_step(const grpo_adamw_config* c, const grpo_adamw_tensor* tensors,
                            const grpo_adamw_tensor* out, int32_t n_tensors,
                            cudaStream_t stream) {
  NvtxRange nvtx_range("grpo_adamw_step");
  if (!c || n_tensors < 0 || (n_tensors > 0 && !tensors) || c->step < 1)
    return GRPO_ERR_INVALID_ARG;
  for (double b : {c->beta1, c->beta2})
    if (!(b >= 0.0 && b < 1.0)) return GRPO_ERR_INVALID_ARG;
  for (double v : {c->lr, c->eps})
    if (!isfinite(v) || v < 0.0) return GRPO_ERR_INVALID_ARG;
  if (!isfinite(c->grad_scale)) return GRPO_ERR_INVALID_ARG;
  if (c->state_bits != 32 && c->state_bits != 8) return GRPO_ERR_INVALID_ARG;
  const bool eight = c->state_bits == 8;
  // every tensor is checked before the first launch
  for (int32_t i = 0; i < n_tensors; ++i) {
    const grpo_adamw_tensor& t = tensors[i];
    if (t.n < 0 || !isfinite(t.weight_decay) || t.weight_decay < 0.f) return GRPO_ERR_INVALID_ARG;
    if (!is_f32_or_bf16(t.param_dtype) || !is_f32_or_bf16(t.grad_dtype))
      return GRPO_ERR_INVALID_ARG;
    if (out && (out[i].n != t.n || out[i].param_dtype != t.param_dtype ||
                (out[i].master != nullptr) != (t.master != nullptr)))
      return GRPO_ERR_INVALID_ARG;
    if (t.n == 0) continue;
    if (!t.grad) return GRPO_ERR_INVALID_ARG;
    if (t.master && t.param_dtype == GRPO_F32) return GRPO_ERR_INVALID_ARG;
    for (const grpo_adamw_tensor* u : {&t, out ? out + i : &t}) {
      const grpo_status st = adamw_buffers(*u, eight);
      if (st != GRPO_OK) return st;
    }
    if (!aligned_to(t.grad, elem_size(t.grad_dtype)) || t.n > (static_cast<int64_t>(1) << 40))
      return GRPO_ERR_UNSUPPORTED;
  }
  // The scalars are formed in float64 and rounded once.
  AdamConst k;
  const double b1 = c->beta1, b2 = c->beta2, t = static_cast<double>(c->step);
  k.beta1 = static_cast<float>(b1);
  k.one_m_beta1 = static_cast<float>(1.0 - b1);
  k.beta2 = static_cast<float>(b2);
  k.one_m_beta2 = static_cast<float>(1.0 - b2);
  k.lr_t = static_cast<float>(c->lr / (1.0 - pow(b1, t)));
  k.rsqrt_c2 = static_cast<float>(1.0 / sqrt(1.0 - pow(b2, t)));
  // (the kernel's reciprocal takes a denominator below 2^-126 for 0, and 0 / eps is 0)
  k.eps = c->eps > 0.0 ? fmaxf(static_cast<float>(c->eps), FLT_MIN) : 0.f;
  k.grad_scale = c->grad_scale;
  k.dither = static_cast<uint32_t>(static_cast<uint64_t>(c->step) * 0xC13FA9A9ull);

  // One launch for each set of types that occurs (and each kAdamMaxTensors
  // tensors of it): the kernels are compiled for one set.
  AdamTensor table[kAdamMaxTensors];
  for (int kind = 0; kind < 8; ++kind) {
    int used = 0;
    for (int32_t i = 0; i <= n_tensors; ++i) {
      if (used == kAdamMaxTensors || (i == n_tensors && used > 0)) {
        LAUNCH(K_ADAMW, stream,
               launch_adamw(table, used, kind | (eight ? ADAM_BITS8 : 0), k, stream));
        used = 0;
      }
      if (i == n_tensors) break;
      const grpo_adamw_tensor& s = tensors[i];
      const int of = (s.param_dtype == GRPO_BF16 ? ADAM_P_BF16 : 0) |
                     (s.grad_dtype == GRPO_BF16 ? ADAM_G_BF16 : 0) |
                     (s.master ? ADAM_MASTER : 0);
      if (s.n == 0 || of != kind) continue;
      AdamTensor& d = table[used++];
      d.g = s.grad;
      d.p = s.param;
      d.w = s.master;
      d.m = s.m;
      d.v = s.v;
      d.ms = s.m_scale;
      d.vs = s.v_scale;
      const grpo_adamw_tensor& o = out ? out[i] : s;
      d.p_out = o.param;
      d.w_out = o.master;
      d.m_out = o.m;
      d.v_out = o.v;
      d.ms_out = o.m_scale;
      d.vs_out = o.v_scale;
      d.n = s.n;
      d.keep = static_cast<float>(1.0 - c->lr * s.weight_decay);
      d.chunk0 = 0;
    }
  }
  return GRPO_OK;
}

}  // extern "C"
