// C entry points of the operators of an update beyond a rollout's first: the clipped
// policy loss, the norms around a block, the norm of the gradients and clipping by it.
// Argument checks and launches only; the mathematics and the layouts stand at the kernels
// (policy.cu, residual_norm.cu, grad_norm.cu).
#include <math.h>

#include "../../include/grpo.h"
#include "api_common.h"
#include "internal.h"

using namespace grpo;

namespace {

constexpr int64_t kMaxRows = (static_cast<int64_t>(1) << 31) - 1;

bool is_f32_or_bf16(grpo_dtype t) { return t == GRPO_F32 || t == GRPO_BF16; }
size_t elem_size(grpo_dtype t) { return t == GRPO_F32 ? 4 : 2; }

// ------------------------------------------------------------ policy loss
// log of a bound in two floats; none: beyond every float.
void log_bound(double v, float* hi, float* lo) {
  const double l = log(v);
  *hi = static_cast<float>(l);
  *lo = isfinite(l) ? static_cast<float>(l - static_cast<double>(*hi)) : 0.f;
}

grpo_status policy_args(const grpo_policy_problem* p, PolicyArgs* a) {
  if (!p || p->num_seqs < 0 || p->seq_len < 0) return GRPO_ERR_INVALID_ARG;
  for (int64_t ld : {p->ld_logp, p->ld_old, p->ld_ref, p->ld_adv, p->ld_mask, p->ld_dlogp})
    if (ld != 0 && ld < p->seq_len) return GRPO_ERR_INVALID_ARG;
  for (double v : {p->clip_low, p->clip_high})
    if (!(v >= 0.0)) return GRPO_ERR_INVALID_ARG;
  if (!(p->dual_clip == 0.0 || p->dual_clip >= 1.0)) return GRPO_ERR_INVALID_ARG;
  if (!isfinite(p->beta)) return GRPO_ERR_INVALID_ARG;
  if (p->ratio != 0 && p->ratio != 1) return GRPO_ERR_INVALID_ARG;
  if (p->reduce < 0 || p->reduce > 2) return GRPO_ERR_INVALID_ARG;
  if (p->token_adv != 0 && p->token_adv != 1) return GRPO_ERR_INVALID_ARG;
  if (p->reduce == 2 && !(p->divisor > 0.0 && isfinite(p->divisor))) return GRPO_ERR_INVALID_ARG;
  if (p->num_seqs > kMaxRows || p->seq_len > kMaxRows - 4095 ||
      p->num_seqs * p->seq_len > static_cast<int64_t>(1) << 40)
    return GRPO_ERR_UNSUPPORTED;
  *a = PolicyArgs();
  a->B = p->num_seqs;
  a->T = p->seq_len;
  auto ld = [&](int64_t v) { return v ? v : p->seq_len; };
  a->ld_logp = ld(p->ld_logp);
  a->ld_old = ld(p->ld_old);
  a->ld_ref = ld(p->ld_ref);
  a->ld_adv = ld(p->ld_adv);
  a->ld_mask = ld(p->ld_mask);
  a->ld_dlogp = ld(p->ld_dlogp);
  a->token_adv = p->token_adv;
  a->sequence_ratio = p->ratio;
  a->reduce = p->reduce;
  a->inv_divisor = p->reduce == 2 ? static_cast<float>(1.0 / p->divisor) : 0.f;
  a->beta = static_cast<float>(p->beta);
  const double up = 1.0 + p->clip_high, down = p->clip_low < 1.0 ? 1.0 - p->clip_low : 0.0;
  const double far = p->dual_clip > 0.0 ? p->dual_clip : INFINITY;
  a->e_up = static_cast<float>(p->clip_high);
  a->e_down = static_cast<float>(down - 1.0);
  a->e_far = static_cast<float>(far - 1.0);
  log_bound(up, &a->up_hi, &a->up_lo);
  log_bound(down, &a->down_hi, &a->down_lo);
  log_bound(far, &a->far_hi, &a->far_lo);
  return GRPO_OK;
}

// --------------------------------------------------- norms around a block
grpo_status resnorm_args(const grpo_residual_norm_problem* p, ResNormArgs* a) {
  if (!p || p->rows < 0 || p->d < 1) return GRPO_ERR_INVALID_ARG;
  for (grpo_dtype t : {p->dtype, p->param_dtype, p->gate_dtype})
    if (!is_f32_or_bf16(t)) return GRPO_ERR_INVALID_ARG;
  if (p->rms != 0 && p->rms != 1) return GRPO_ERR_INVALID_ARG;
  if (!isfinite(p->eps) || p->eps < 0.f || !isfinite(p->scale)) return GRPO_ERR_INVALID_ARG;
  for (int64_t ld : {p->ld_x, p->ld_residual, p->ld_h, p->ld_y, p->ld_gate, p->ld_dy, p->ld_dh,
                     p->ld_dx, p->ld_dresidual, p->ld_dgate})
    if (ld != 0 && ld < p->d) return GRPO_ERR_INVALID_ARG;
  if (p->gate_rows < 0) return GRPO_ERR_INVALID_ARG;
  if (p->d > kMaxResNormDim || p->rows > kMaxRows) return GRPO_ERR_UNSUPPORTED;
  *a = ResNormArgs();
  a->rows = p->rows;
  a->d = p->d;
  auto ld = [&](int64_t v) { return v ? v : p->d; };
  a->ld_x = ld(p->ld_x);
  a->ld_res = ld(p->ld_residual);
  a->ld_h = ld(p->ld_h);
  a->ld_y = ld(p->ld_y);
  a->ld_gate = ld(p->ld_gate);
  a->ld_dy = ld(p->ld_dy);
  a->ld_dh = ld(p->ld_dh);
  a->ld_dx = ld(p->ld_dx);
  a->ld_dres = ld(p->ld_dresidual);
  a->ld_dgate = ld(p->ld_dgate);
  a->eps = p->eps;
  a->scale = p->scale;
  a->rms = p->rms;
  a->bf16 = p->dtype == GRPO_BF16 ? 1 : 0;
  a->param_bf16 = p->param_dtype == GRPO_BF16 ? 1 : 0;
  a->gate_bf16 = p->gate_dtype == GRPO_BF16 ? 1 : 0;
  a->gate_rows = p->gate_rows;
  return GRPO_OK;
}

// Whether gate_rows divides the rows, where there is a gate.
bool gate_fits(const ResNormArgs& a, const void* gate) {
  return !gate || a.rows == 0 || (a.gate_rows >= 1 && a.rows % a.gate_rows == 0);
}

// Bytes for the most arrays of partial sums that a call can have: the parameters', and a
// shared gate's two.
size_t resnorm_bytes(const ResNormArgs& a, int sms) {
  const size_t arrays = (a.rms ? 2 : 4) + (a.gate_rows > 1 ? 2 : 0);
  return sizeof(float) * arrays * static_cast<size_t>(resnorm_walkers(a, sms)) * static_cast<size_t>(a.d);
}

// -------------------------------------------------------------- gradients
size_t grad_bytes(int sms, int launches) { return sizeof(double) * grad_parts(sms) * launches; }
// Launches whose partial norms the workspace holds; more tensors than these have are
// taken in turns, each joined to what the former left.
constexpr int kGradLaunches = 16;
// Of a list, so that its chunks' numbers are 32 bits.
constexpr int64_t kMaxGradElements = static_cast<int64_t>(1) << 40;

grpo_status clip_grads(const grpo_grad_tensor* tensors, int32_t n_tensors, int32_t norm_type,
                       double max_norm, double eps, float* norm, float* factor, bool scale,
                       void* workspace, size_t workspace_bytes, cudaStream_t stream) {
  if (n_tensors < 0 || (n_tensors > 0 && !tensors) || !norm || (scale && !factor))
    return GRPO_ERR_INVALID_ARG;
  if (norm_type != 2 && norm_type != 0) return GRPO_ERR_INVALID_ARG;
  if (!(max_norm >= 0.0) || !(eps >= 0.0) || !isfinite(eps)) return GRPO_ERR_INVALID_ARG;
  if (!aligned_to(norm, 4) || !aligned_to(factor, 4)) return GRPO_ERR_UNSUPPORTED;
  int64_t all = 0;
  for (int32_t i = 0; i < n_tensors; ++i) {
    const grpo_grad_tensor& t = tensors[i];
    if (t.n < 0 || !is_f32_or_bf16(t.dtype)) return GRPO_ERR_INVALID_ARG;
    if (t.n == 0) continue;
    if (!t.grad || (scale && !t.out)) return GRPO_ERR_INVALID_ARG;
    if (!aligned_to(t.grad, elem_size(t.dtype)) || (scale && !aligned_to(t.out, elem_size(t.dtype))) ||
        t.n > kMaxGradElements - all)
      return GRPO_ERR_UNSUPPORTED;
    all += t.n;
  }
  int sms = 0;
  const grpo_status st = device_info(&sms);
  if (st != GRPO_OK) return st;
  const bool room = workspace && aligned16(workspace) && workspace_bytes >= grad_bytes(sms, kGradLaunches);
  GradJoin join = {static_cast<double*>(workspace), 0, norm_type == 0 ? 1 : 0, max_norm, eps, norm, factor};
  GradTensor table[kGradMaxTensors];
  int launches = 0;
  for (int pass = 0; pass < (scale ? 2 : 1); ++pass) {
    int used = 0;
    for (int32_t i = 0; i <= n_tensors; ++i) {
      if (used == kGradMaxTensors || (i == n_tensors && used > 0)) {
        if (pass == 0 && launches == 0 && i == n_tensors && grad_small(table, used)) {
          LAUNCH(K_GRAD_NORM, stream, launch_grad_small(table, used, join, scale ? 1 : 0, stream));
          return GRPO_OK;
        }
        if (!room) return GRPO_ERR_WORKSPACE;
        if (pass == 0) {
          if (launches == kGradLaunches) {
            LAUNCH(K_GRAD_JOIN, stream, launch_grad_fold(join.partial, join.parts, join.inf, stream));
            join.parts = launches = 1;
          }
          int more = 0;
          LAUNCH(K_GRAD_NORM, stream,
                 launch_grad_norm(table, used, join.inf, sms, join.partial + join.parts, &more, stream));
          join.parts += more;
          ++launches;
        } else {
          LAUNCH(K_GRAD_SCALE, stream, launch_grad_scale(table, used, join, sms, stream));
          join.norm = nullptr;
        }
        used = 0;
      }
      if (i == n_tensors) break;
      if (tensors[i].n == 0) continue;
      GradTensor& d = table[used++];
      d.grad = tensors[i].grad;
      d.out = tensors[i].out;
      d.n = tensors[i].n;
      d.chunk0 = 0;
      d.bf16 = tensors[i].dtype == GRPO_BF16 ? 1 : 0;
    }
    // (what scales joins the parts by itself; without a tensor there is nothing to scale)
    if (pass == 0 && launches == 0 && !room) return GRPO_ERR_WORKSPACE;
    if (pass == 0 && (!scale || launches == 0)) LAUNCH(K_GRAD_JOIN, stream, launch_grad_join(join, stream));
  }
  return GRPO_OK;
}

}  // namespace

extern "C" {

grpo_status grpo_policy_loss_workspace_size(const grpo_policy_problem* p, size_t* bytes) {
  PolicyArgs a;
  grpo_status st = policy_args(p, &a);
  if (st != GRPO_OK) return st;
  int sms = 0;
  if ((st = device_info(&sms)) != GRPO_OK) return st;
  const size_t n = policy_plan(a, sms, nullptr);
  if (bytes) *bytes = n;
  return GRPO_OK;
}

grpo_status grpo_policy_loss(const grpo_policy_problem* p, const float* logp, const float* logp_old,
                             const float* logp_ref, const float* adv, const uint8_t* mask,
                             float* loss, float* stats, float* dlogp, void* workspace,
                             size_t workspace_bytes, cudaStream_t stream) {
  NvtxRange nvtx_range("grpo_policy_loss");
  PolicyArgs a;
  grpo_status st = policy_args(p, &a);
  if (st != GRPO_OK) return st;
  if (!loss) return GRPO_ERR_INVALID_ARG;
  if (!aligned_to(loss, 4) || !aligned_to(stats, 4)) return GRPO_ERR_UNSUPPORTED;
  if (a.B == 0 || a.T == 0) {  // empty sums
    if (cudaMemsetAsync(loss, 0, sizeof(float), stream) != cudaSuccess) return GRPO_ERR_CUDA;
    if (stats && cudaMemsetAsync(stats, 0, 4 * sizeof(float), stream) != cudaSuccess)
      return GRPO_ERR_CUDA;
    return GRPO_OK;
  }
  if (!logp || !adv || !mask) return GRPO_ERR_INVALID_ARG;
  if (!aligned_to(logp, 4) || !aligned_to(logp_old, 4) || !aligned_to(logp_ref, 4) ||
      !aligned_to(adv, 4) || !aligned_to(dlogp, 4))
    return GRPO_ERR_UNSUPPORTED;
  int sms = 0;
  if ((st = device_info(&sms)) != GRPO_OK) return st;
  if (!logp_old) a.sequence_ratio = 0;
  const size_t need = policy_plan(a, sms, workspace);
  if (need && (!workspace || !aligned16(workspace) || workspace_bytes < need))
    return GRPO_ERR_WORKSPACE;
  a.logp = logp;
  a.old = logp_old;
  a.ref = logp_ref;
  a.adv = adv;
  a.mask = mask;
  a.loss = loss;
  a.stats = stats;
  a.dlogp = dlogp;
  if (policy_counts_first(a)) LAUNCH(K_POLICY_COUNT, stream, launch_policy_count(a, stream));
  LAUNCH(K_POLICY_LOSS, stream, launch_policy_loss(a, stream));
  return GRPO_OK;
}

grpo_status grpo_residual_norm_workspace_size(const grpo_residual_norm_problem* p,
                                              size_t* bwd_bytes) {
  ResNormArgs a;
  grpo_status st = resnorm_args(p, &a);
  if (st != GRPO_OK) return st;
  int sms = 0;
  if ((st = device_info(&sms)) != GRPO_OK) return st;
  if (bwd_bytes) *bwd_bytes = resnorm_bytes(a, sms);
  return GRPO_OK;
}

grpo_status grpo_residual_norm_fwd(const grpo_residual_norm_problem* p, const void* x,
                                   const void* residual, const void* weight, const void* bias,
                                   const void* post_weight, const void* post_bias,
                                   const void* gate, void* h, void* y, float* mean, float* rstd,
                                   float* post_mean, float* post_rstd, cudaStream_t stream) {
  NvtxRange nvtx_range("grpo_residual_norm_fwd");
  ResNormArgs a;
  grpo_status st = resnorm_args(p, &a);
  if (st != GRPO_OK) return st;
  if ((a.rms && (bias || post_bias)) || (post_bias && !post_weight) || !gate_fits(a, gate))
    return GRPO_ERR_INVALID_ARG;
  if (a.rows == 0) return GRPO_OK;
  if (!x || !residual || !weight || !h || !y || h == y) return GRPO_ERR_INVALID_ARG;
  const size_t es = elem_size(p->dtype), ps = elem_size(p->param_dtype);
  for (const void* q : {x, residual, static_cast<const void*>(h), static_cast<const void*>(y)})
    if (!aligned_to(q, es)) return GRPO_ERR_UNSUPPORTED;
  for (const void* q : {weight, bias, post_weight, post_bias})
    if (!aligned_to(q, ps)) return GRPO_ERR_UNSUPPORTED;
  for (const float* q : {mean, rstd, post_mean, post_rstd})
    if (!aligned_to(q, 4)) return GRPO_ERR_UNSUPPORTED;
  if (!aligned_to(gate, elem_size(p->gate_dtype))) return GRPO_ERR_UNSUPPORTED;
  int sms = 0;
  if ((st = device_info(&sms)) != GRPO_OK) return st;
  a.x = x;
  a.residual = residual;
  a.weight = weight;
  a.bias = bias;
  a.post_weight = post_weight;
  a.post_bias = post_bias;
  a.gate = gate;
  a.h_out = h;
  a.y = y;
  a.mean = a.rms ? nullptr : mean;
  a.rstd = rstd;
  a.post_mean = post_weight && !a.rms ? post_mean : nullptr;
  a.post_rstd = post_weight ? post_rstd : nullptr;
  LAUNCH(K_RESNORM_FWD, stream, launch_resnorm_fwd(a, sms, stream));
  return GRPO_OK;
}

grpo_status grpo_residual_norm_bwd(const grpo_residual_norm_problem* p, const void* dy,
                                   const void* dh, const void* h, const void* weight,
                                   const float* mean, const float* rstd, const void* x,
                                   const void* post_weight, const void* post_bias,
                                   const float* post_mean, const float* post_rstd,
                                   const void* gate, void* dx, void* dresidual, float* dweight,
                                   float* dbias, float* dpost_weight, float* dpost_bias,
                                   void* dgate, void* workspace, size_t workspace_bytes,
                                   cudaStream_t stream) {
  NvtxRange nvtx_range("grpo_residual_norm_bwd");
  ResNormArgs a;
  grpo_status st = resnorm_args(p, &a);
  if (st != GRPO_OK) return st;
  if ((a.rms && (dbias || dpost_bias || post_bias)) || (!post_weight && (post_bias || dpost_weight || dpost_bias)) ||
      (dgate && !gate) || !gate_fits(a, gate))
    return GRPO_ERR_INVALID_ARG;
  const bool shared = dgate && a.gate_rows > 1;
  float* const vectors[] = {dweight, dbias, dpost_weight, dpost_bias};
  for (const float* q : vectors)
    if (!aligned_to(q, 4)) return GRPO_ERR_UNSUPPORTED;
  if (!aligned_to(dgate, shared ? 4 : elem_size(p->gate_dtype))) return GRPO_ERR_UNSUPPORTED;
  if (a.rows == 0) {  // empty sums
    for (float* q : vectors)
      if (q && cudaMemsetAsync(q, 0, sizeof(float) * a.d, stream) != cudaSuccess) return GRPO_ERR_CUDA;
    return GRPO_OK;
  }
  if (!dy || !h || !weight || !rstd || !dresidual || dx == dresidual || (!mean && !a.rms))
    return GRPO_ERR_INVALID_ARG;
  if (post_weight && (!post_rstd || (!post_mean && !a.rms))) return GRPO_ERR_INVALID_ARG;
  if ((post_weight || gate) && !x) return GRPO_ERR_INVALID_ARG;
  const size_t es = elem_size(p->dtype), ps = elem_size(p->param_dtype);
  for (const void* q : {dy, dh, h, x, static_cast<const void*>(dx), static_cast<const void*>(dresidual)})
    if (!aligned_to(q, es)) return GRPO_ERR_UNSUPPORTED;
  for (const void* q : {weight, post_weight, post_bias})
    if (!aligned_to(q, ps)) return GRPO_ERR_UNSUPPORTED;
  for (const float* q : {mean, rstd, post_mean, post_rstd})
    if (!aligned_to(q, 4)) return GRPO_ERR_UNSUPPORTED;
  if (!aligned_to(gate, elem_size(p->gate_dtype))) return GRPO_ERR_UNSUPPORTED;
  int sms = 0;
  if ((st = device_info(&sms)) != GRPO_OK) return st;
  // the arrays of partial sums that this call has
  int arrays = 0;
  a.at_dw = dweight ? arrays++ : -1;
  a.at_db = dbias ? arrays++ : -1;
  a.at_dpw = dpost_weight ? arrays++ : -1;
  a.at_dpb = dpost_bias ? arrays++ : -1;
  a.at_head = arrays;
  a.at_tail = arrays + 1;
  if (shared) arrays += 2;
  if (arrays && (!workspace || !aligned16(workspace) || workspace_bytes < resnorm_bytes(a, sms)))
    return GRPO_ERR_WORKSPACE;
  a.dy = dy;
  a.dh = dh;
  a.h = h;
  a.weight = weight;
  a.mean = a.rms ? nullptr : const_cast<float*>(mean);
  a.rstd = const_cast<float*>(rstd);
  a.x = post_weight || gate ? x : nullptr;
  a.post_weight = post_weight;
  a.post_bias = post_bias;
  a.post_mean = a.rms ? nullptr : const_cast<float*>(post_mean);
  a.post_rstd = const_cast<float*>(post_rstd);
  a.gate = gate;
  a.dx = dx;
  a.dres = dresidual;
  a.dweight = dweight;
  a.dbias = dbias;
  a.dpost_weight = dpost_weight;
  a.dpost_bias = dpost_bias;
  a.dgate = dgate;
  a.partial = static_cast<float*>(workspace);
  int walkers = 0;
  LAUNCH(K_RESNORM_BWD, stream, launch_resnorm_bwd(a, sms, &walkers, stream));
  if (arrays) LAUNCH(K_RESNORM_JOIN, stream, launch_resnorm_join(a, walkers, stream));
  return GRPO_OK;
}

grpo_status grpo_grad_norm_workspace_size(size_t* bytes) {
  int sms = 0;
  const grpo_status st = device_info(&sms);
  if (st != GRPO_OK) return st;
  if (bytes) *bytes = grad_bytes(sms, kGradLaunches);
  return GRPO_OK;
}

grpo_status grpo_grad_norm(const grpo_grad_tensor* tensors, int32_t n_tensors, int32_t norm_type,
                           double max_norm, double eps, float* norm, float* factor,
                           void* workspace, size_t workspace_bytes, cudaStream_t stream) {
  NvtxRange nvtx_range("grpo_grad_norm");
  return clip_grads(tensors, n_tensors, norm_type, max_norm, eps, norm, factor, false, workspace,
                    workspace_bytes, stream);
}

grpo_status grpo_clip_grad_norm(const grpo_grad_tensor* tensors, int32_t n_tensors,
                                int32_t norm_type, double max_norm, double eps, float* norm,
                                float* factor, void* workspace, size_t workspace_bytes,
                                cudaStream_t stream) {
  NvtxRange nvtx_range("grpo_clip_grad_norm");
  return clip_grads(tensors, n_tensors, norm_type, max_norm, eps, norm, factor, true, workspace,
                    workspace_bytes, stream);
}

}  // extern "C"
