"""GB300-native memory-efficient GRPO loss.

The fused lm_head projection, log-softmax and GRPO objective (reverse-KL
estimator plus the exp(q - q.detach()) * A advantage term) over the
flattened token axis, in hand-written sm_103a CUDA kernels behind the C ABI
of include/grpo.h; and the operators around that loss in a GRPO iteration: the
draw of completion tokens (``sample``), the norm before the head with its
gradients (``layer_norm``) and the optimizer step (``AdamW``). Importing the
package does not load the library; the first call does, and raises if it has
not been built.
"""
from __future__ import annotations

import copy
import operator
from typing import Optional, Sequence

import numpy as np
import torch

from . import _lib
from ._lib import (GrpoError, Problem, advantages, device_status, layernorm_bwd, layernorm_fwd,
                   loss_bwd, loss_bwd_e4m3, loss_fwd, loss_fwd_e4m3, make_problem,
                   profile_collect, profile_enable, quantize_e4m3_rows, sample, workspace_size)

__all__ = ["GrpoError", "Problem", "advantages", "device_status", "layernorm_bwd",
           "layernorm_fwd", "loss_bwd", "loss_bwd_e4m3", "loss_fwd", "loss_fwd_e4m3",
           "make_problem", "profile_collect", "profile_enable", "quantize_e4m3_rows", "sample",
           "workspace_size", "GRPOLoss", "grpo_loss", "layer_norm", "AdamW"]


_CTRL_BYTES = 256  # control block at the start of every workspace (error word, counts)


class GRPOLoss:
    """Owns the workspaces of one problem shape and runs the library calls.

    ``forward`` returns (loss, kl_mean, logp_pol, logp_ref) as CUDA tensors;
    ``backward`` returns dH_pol (and fills ``self.dW``, float32 [V, d], when
    built with ``compute_dW``). Buffers are allocated once with torch and
    reused across calls.

    With ``dtype=torch.float8_e4m3fn`` the engine takes float32 or bf16 H_pol,
    H_ref and W, quantizes them row-wise to e4m3 with the library's quantizer
    and runs the e4m3 problem; dH is then bf16. The backward reuses the
    forward's quantized H_pol and W while those tensors are unchanged (same
    storage and version counter).
    """

    def __init__(self, num_seqs: int, seq_len: int, d: int, V: int, group_size: int,
                 beta: float = 0.04, eps: float = 1e-4, std_unbiased: int = 1,
                 chunk_rows: int = 0, dtype=torch.bfloat16, device="cuda",
                 compute_dW: bool = False, token_level: bool = False,
                 logit_multiply: float = 0.0, logit_divide: float = 0.0, softcap: float = 0.0,
                 temperature: float = 0.0, ref_logp_given: bool = False, kl_mode: int = 0,
                 cluster_mode: int = 0):
        self.problem = make_problem(num_seqs, seq_len, d, V, group_size, beta, eps,
                                    std_unbiased, chunk_rows, dtype, compute_dW, token_level,
                                    logit_multiply, logit_divide, softcap, temperature,
                                    ref_logp_given, kl_mode, cluster_mode)
        fwd_b, bwd_b = workspace_size(self.problem)
        dev = torch.device(device)
        self.ws_fwd = torch.empty(fwd_b, dtype=torch.uint8, device=dev)
        self.ws_bwd = torch.empty(bwd_b, dtype=torch.uint8, device=dev)
        # every call clears its workspace's control block (the device error
        # word) first; clear both now, so check() before a backward has run
        # does not read stale bytes from the allocator's cache
        self.ws_fwd[:_CTRL_BYTES].zero_()
        self.ws_bwd[:_CTRL_BYTES].zero_()
        N = num_seqs * seq_len
        self.adv = torch.empty(num_seqs, dtype=torch.float32, device=dev)
        self.logp_pol = torch.empty(N, dtype=torch.float32, device=dev)
        self.logp_ref = torch.empty(N, dtype=torch.float32, device=dev)
        self.lse_pol = torch.empty(N, dtype=torch.float32, device=dev)
        self.loss = torch.empty(1, dtype=torch.float32, device=dev)
        self.kl_mean = torch.empty(1, dtype=torch.float32, device=dev)
        self.dtype = dtype
        self.dH = None
        self.dW = (torch.empty(V, d, dtype=torch.float32, device=dev) if compute_dW else None)
        self.e4m3 = dtype == torch.float8_e4m3fn
        if self.e4m3:
            u8, f32 = torch.uint8, torch.float32
            self.q_pol = torch.empty(N, d, dtype=u8, device=dev)
            self.s_pol = torch.empty(N, dtype=f32, device=dev)
            self.q_ref = None if ref_logp_given else torch.empty(N, d, dtype=u8, device=dev)
            self.s_ref = None if ref_logp_given else torch.empty(N, dtype=f32, device=dev)
            self.q_W = torch.empty(V, d, dtype=u8, device=dev)
            self.s_W = torch.empty(V, dtype=f32, device=dev)
            self._quantized = None  # (H_pol, W) identities the codes were made from

    @staticmethod
    def _ident(t):
        return (t.data_ptr(), t._version, tuple(t.shape), t.dtype)

    def _quantize(self, H_pol, W):
        quantize_e4m3_rows(H_pol, self.q_pol, self.s_pol)
        quantize_e4m3_rows(W, self.q_W, self.s_W)
        self._quantized = (self._ident(H_pol), self._ident(W))

    def advantages(self, rewards: torch.Tensor) -> torch.Tensor:
        p = self.problem
        return advantages(rewards, p.group_size, p.eps, p.std_unbiased, self.adv)

    def forward(self, H_pol, H_ref, W, ids, mask, adv, logp_ref=None):
        """With ``ref_logp_given`` pass H_ref=None and the reference log-probs
        as ``logp_ref`` (float32 [N]); they are copied into the engine."""
        if self.problem.ref_logp_given:
            if logp_ref is None:
                raise ValueError("ref_logp_given needs logp_ref")
            self.logp_ref.copy_(logp_ref)
        if self.e4m3:
            self._quantize(H_pol, W)
            if H_ref is not None and self.q_ref is not None:
                quantize_e4m3_rows(H_ref, self.q_ref, self.s_ref)
            loss_fwd_e4m3(self.problem, self.q_pol, self.s_pol, self.q_ref, self.s_ref, self.q_W,
                          self.s_W, ids, mask, adv, self.logp_pol, self.logp_ref, self.lse_pol,
                          self.loss, self.kl_mean, self.ws_fwd)
        else:
            loss_fwd(self.problem, H_pol, H_ref, W, ids, mask, adv, self.logp_pol, self.logp_ref,
                     self.lse_pol, self.loss, self.kl_mean, self.ws_fwd)
        return self.loss, self.kl_mean, self.logp_pol, self.logp_ref

    def backward(self, H_pol, W, ids, mask, adv, grad_loss: float = 1.0, dH=None):
        if dH is None:
            if self.dH is None:
                self.dH = (torch.empty(H_pol.shape, dtype=torch.bfloat16, device=H_pol.device)
                           if self.e4m3 else torch.empty_like(H_pol))
            dH = self.dH
        if self.e4m3:
            if self._quantized != (self._ident(H_pol), self._ident(W)):
                self._quantize(H_pol, W)
            loss_bwd_e4m3(self.problem, self.q_pol, self.s_pol, self.q_W, self.s_W, ids, mask,
                          adv, self.logp_pol, self.logp_ref, self.lse_pol, grad_loss, dH,
                          self.ws_bwd, dW=self.dW)
        else:
            loss_bwd(self.problem, H_pol, W, ids, mask, adv, self.logp_pol, self.logp_ref,
                     self.lse_pol, grad_loss, dH, self.ws_bwd, dW=self.dW)
        return dH

    def check(self) -> None:
        """Raise if a kernel of the last calls recorded a device error."""
        for ws in (self.ws_fwd, self.ws_bwd):
            st = device_status(ws)
            if st != 0:
                raise GrpoError(st, "device")


class _GRPOLossFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, H_pol, H_ref, W, ids, mask, adv, engine):
        loss, kl_mean, _, _ = engine.forward(H_pol, H_ref, W, ids, mask, adv)
        ctx.engine = engine
        ctx.save_for_backward(H_pol, W, ids, mask, adv)
        return loss.clone().reshape(()), kl_mean.clone().reshape(())

    @staticmethod
    def backward(ctx, g_loss, g_kl):
        # with a graph to be made of it, the gradient is a node that refuses its own
        grads = _GRPOLossGradFn.apply if torch.is_grad_enabled() else _grpo_loss_grads
        dH, dW = grads(g_loss, *ctx.saved_tensors, ctx.engine)
        return dH, None, dW, None, None, None, None


def _grpo_loss_grads(g_loss, H_pol, W, ids, mask, adv, eng):
    # the upstream gradient is read on the host: one scalar per backward
    dH = eng.backward(H_pol, W, ids, mask, adv, g_loss.item(),
                      dH=torch.empty(H_pol.shape, dtype=torch.bfloat16, device=H_pol.device)
                      if eng.e4m3 else torch.empty_like(H_pol))
    return dH.to(H_pol.dtype), eng.dW.detach().to(W.dtype) if eng.dW is not None else None


class _GRPOLossGradFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, *args):
        return _grpo_loss_grads(*args)

    @staticmethod
    def backward(ctx, *grads):
        raise RuntimeError("grpo_loss is once differentiable: its gradients have no gradients of their own")


def grpo_loss(H_pol, H_ref, W, ids, mask, adv, engine: GRPOLoss):
    """Autograd entry: returns (loss, kl_mean); backward gives the gradient
    of the loss with respect to H_pol, and with respect to W when the engine
    was built with ``compute_dW`` (the reference model is frozen; kl_mean is a
    metric and carries no gradient). The gradients have none of their own: asking
    for them is an error."""
    return _GRPOLossFn.apply(H_pol, H_ref, W, ids, mask, adv, engine)


class _LayerNormFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, eps, rms):
        y, mean, rstd = layernorm_fwd(x, weight, bias, eps=eps, rms=rms)
        ctx.save_for_backward(x, weight, mean, rstd)
        ctx.rms, ctx.bias_dtype = rms, None if bias is None else bias.dtype
        return y

    @staticmethod
    def backward(ctx, dy):
        x, weight, mean, rstd = ctx.saved_tensors
        need_x, need_w, need_b = ctx.needs_input_grad[:3]
        # with a graph to be made of it, the gradient is a node that refuses its own
        grads = _LayerNormGradFn.apply if torch.is_grad_enabled() else _layer_norm_grads
        dx, dw, db = grads(dy, x, weight, mean, rstd, ctx.rms, need_w, need_b, ctx.bias_dtype)
        return dx if need_x else None, dw, db, None, None, None


def _layer_norm_grads(dy, x, weight, mean, rstd, rms, need_w, need_b, bias_dtype):
    if dy.stride(-1) != 1 or (dy.shape[0] > 1 and dy.stride(0) < dy.shape[1]):
        dy = dy.contiguous()        # a broadcast gradient, as of a sum
    dx, dw, db = layernorm_bwd(x, weight, dy.to(x.dtype), mean, rstd, rms=rms, bias=need_b, need_dweight=need_w)
    return dx, dw.to(weight.dtype) if need_w else None, db.to(bias_dtype) if need_b else None


class _LayerNormGradFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, *args):
        return _layer_norm_grads(*args)

    @staticmethod
    def backward(ctx, *grads):
        raise RuntimeError("layer_norm is once differentiable: its gradients have no gradients of their own")


def layer_norm(x: torch.Tensor, weight: torch.Tensor, bias: Optional[torch.Tensor] = None,
               eps: float = 1e-5, rms: bool = False) -> torch.Tensor:
    """Autograd entry of the norm over the last dimension of ``x`` (RMS norm
    with ``rms``, which takes no bias): gradients for x, weight and bias, which have
    none of their own (asking for them is an error). Capture ``layernorm_fwd`` and
    ``layernorm_bwd`` into a CUDA graph rather than this."""
    return _LayerNormFn.apply(x.reshape(-1, x.shape[-1]), weight, bias, eps, rms).view(x.shape)


_DATA_PTR, _CONTIGUOUS, _GET_DEVICE = torch.Tensor.data_ptr, torch.Tensor.is_contiguous, torch.Tensor.get_device
_NBYTES, _DTYPE, _SHAPE = operator.attrgetter("nbytes"), operator.attrgetter("dtype"), operator.attrgetter("shape")
_LISTS = ("params", "masters", "exp_avg", "exp_avg_sq", "exp_avg_scale", "exp_avg_sq_scale")
_PLAIN_CODES = {torch.float32: _lib.GRPO_F32, torch.bfloat16: _lib.GRPO_BF16}


class AdamW:
    """AdamW over a list of CUDA tensors (float32 or bf16, contiguous), one call
    for all of them; the arithmetic and the state formats are those of
    grpo_adamw_step.

    ``state_bits`` 32 keeps the two moments in float32, 8 as e4m3 codes with a
    power of two for each 32 values. ``master=True`` keeps float32 masters of the
    bf16 parameters; without one a bf16 parameter is rounded with the step's
    dither, so that updates below half a bf16 step still count. ``weight_decay``
    is one number or one for each tensor. ``lr``, ``betas``, ``eps`` and
    ``weight_decay`` are read at every step.

    ``step(grads)`` applies the gradients (float32 or bf16, of the parameters'
    shapes). With ``out``, an AdamW over other tensors of the same shapes and
    types, the new parameters and states are written there and this object's stay
    as they are. A step that is captured into a CUDA graph holds its number, rates and
    dither: each replay is that same step, and 8-bit states replayed many times stall.

    The state of a run is ``step_count`` and the lists ``masters``, ``exp_avg``,
    ``exp_avg_sq``, ``exp_avg_scale`` and ``exp_avg_sq_scale``, beside the parameters:
    save those, and copy into or replace their tensors to restore it.
    """

    def __init__(self, params: Sequence[torch.Tensor], lr: float = 1e-3, betas=(0.9, 0.999),
                 eps: float = 1e-8, weight_decay=0.01, state_bits: int = 32, master: bool = False):
        if state_bits not in (8, 32):
            raise ValueError("state_bits must be 8 or 32, got %r" % (state_bits,))
        self.params = list(params)
        self.lr, self.betas, self.eps, self.state_bits = lr, tuple(betas), eps, state_bits
        n = len(self.params)
        self.weight_decay = list(weight_decay) if isinstance(weight_decay, (list, tuple)) else [weight_decay] * n
        self._check_decays(n)
        self.step_count = 0
        self.device = self.params[0].device if n else None
        self.masters, self.exp_avg, self.exp_avg_sq = [], [], []
        self.exp_avg_scale, self.exp_avg_sq_scale = [], []
        eight = state_bits == 8
        for i, p in enumerate(self.params):
            _lib._plain_code(p.dtype, "params[%d]" % i)
            _lib._ptr(p, "params[%d]" % i)
            self.masters.append(p.detach().float() if master and p.dtype == torch.bfloat16 else None)
            st = dict(dtype=torch.uint8 if eight else torch.float32, device=p.device)
            self.exp_avg.append(torch.zeros(p.shape, **st))
            self.exp_avg_sq.append(torch.zeros(p.shape, **st))
            for scales in (self.exp_avg_scale, self.exp_avg_sq_scale):
                scales.append(torch.zeros((p.numel() + 31) // 32, **st) if eight else None)
        self._none, self._mastered = [None] * n, any(m is not None for m in self.masters)
        self._bind(self._key())

    def _check_decays(self, n: int) -> None:
        if isinstance(self.weight_decay, (list, tuple)) and len(self.weight_decay) != n:
            raise ValueError("weight_decay must be one number or %d, got %d" % (n, len(self.weight_decay)))

    def _key(self, *others):
        """What the tables were made of (this object's, and others' behind it): the place
        of every tensor, the bytes of the states and masters, and of the parameters,
        which are the caller's, type, shape and layout. (Methods of the class, mapped: a
        step's host time is these walks.)"""
        params, states, some = [], [], []
        for o in (self, *others):
            none = o._none
            params += o.params
            states += o.exp_avg
            states += o.exp_avg_sq
            if o.state_bits == 8 or o.exp_avg_scale != none or o.exp_avg_sq_scale != none:
                states += [t for ts in (o.exp_avg_scale, o.exp_avg_sq_scale) for t in ts if t is not None]
            if o._mastered or o.masters != none:
                states += [t for t in o.masters if t is not None]
                some += [t is None for t in o.masters]
        return (list(map(_DATA_PTR, params + states)), list(map(_NBYTES, states)), list(map(_DTYPE, params)),
                list(map(_SHAPE, params)), all(map(_CONTIGUOUS, params)), self.state_bits, some)

    def _check_tables(self, out) -> None:
        """Make the tables of this object, and of ``out`` if it is given, again where they
        are not those of its tensors any more."""
        of = (self,) if out is None else (self, out)
        for o in of:
            key = o._key()
            if key != o._bound:
                o._bind(key)
        if out is not None:
            if out is self or out._bound[1:] != self._bound[1:] or out._at != self._at:
                raise ValueError("out must be another AdamW of the same shapes, types and states")
            self._pair = self._bound, out._bound, self._key(out)

    def _bind(self, key) -> None:
        """Make the table of the tensors that a step is given (again, when a tensor of
        the lists was replaced, moved or resized). A refusal leaves the old one."""
        n, state = len(self.params), torch.uint8 if self.state_bits == 8 else torch.float32
        table = (_lib.AdamwTensor * max(n, 1))()
        for i, p in enumerate(self.params):
            t, dev, many = table[i], self.device, p.numel()
            t.n = many
            t.param_dtype = _lib._plain_code(p.dtype, "params[%d]" % i)
            t.param = _lib._vec_ptr(p, "params[%d]" % i, p.dtype, many, dev)
            t.master = _lib._vec_ptr(self.masters[i], "masters[%d]" % i, torch.float32, many, dev)
            t.m = _lib._vec_ptr(self.exp_avg[i], "exp_avg[%d]" % i, state, many, dev)
            t.v = _lib._vec_ptr(self.exp_avg_sq[i], "exp_avg_sq[%d]" % i, state, many, dev)
            scales = (many + 31) // 32
            t.m_scale = _lib._vec_ptr(self.exp_avg_scale[i], "exp_avg_scale[%d]" % i, state, scales, dev)
            t.v_scale = _lib._vec_ptr(self.exp_avg_sq_scale[i], "exp_avg_sq_scale[%d]" % i, state, scales, dev)
        spans = sorted((t.data_ptr(), t.nbytes, "%s[%d]" % (name, i)) for name in _LISTS
                       for i, t in enumerate(getattr(self, name)) if t is not None and t.nbytes)
        for (at, size, one), (after, _, other) in zip(spans, spans[1:]):
            if at + size > after:
                raise ValueError("%s overlaps %s: every buffer is one tensor's own" % (one, other))
        self._table = table
        self._columns = np.frombuffer(table, dtype=_lib.ADAMW_COLUMNS)[:n]   # the same memory
        self._at = self.params[0].get_device() if n else -1
        self._mastered = bool(key[-1])
        self._filled, self._pair = None, (None, None, None)
        self._bound = key

    def step(self, grads: Sequence[torch.Tensor], grad_scale: float = 1.0, lr: Optional[float] = None,
             step: Optional[int] = None, out: Optional["AdamW"] = None, stream=None) -> None:
        """``step`` overrides the count of steps taken (1 for the first), ``lr``
        this step's rate; ``grad_scale`` multiplies every gradient."""
        n = len(self.params)
        if len(grads) != n:
            raise ValueError("expected %d gradients, got %d" % (n, len(grads)))
        if out is None:
            to, good = self, self._key() == self._bound
        else:
            mine, its, both = self._pair
            to, good = out, mine is self._bound and its is out._bound and self._key(out) == both
        if not good:
            self._check_tables(out)
        if not n:
            return
        dev, table = self.device, self._columns
        try:
            dtypes = list(map(_DTYPE, grads))
            good = list(map(_SHAPE, grads)) == self._bound[3] and all(map(_CONTIGUOUS, grads)) and \
                not any(map(self._at.__ne__, map(_GET_DEVICE, grads))) and not set(dtypes) - _PLAIN_CODES.keys()
        except (AttributeError, TypeError):     # not tensors
            good = False
        if not good:
            self._refuse(grads)
        table["grad"] = list(map(_DATA_PTR, grads))
        filled = dtypes, self.weight_decay
        if filled != self._filled:
            self._check_decays(n)
            table["grad_dtype"] = list(map(_PLAIN_CODES.get, dtypes))
            table["weight_decay"] = self.weight_decay
            self._filled = dtypes, copy.copy(self.weight_decay)
        count = self.step_count + 1 if step is None else step
        config = _lib.AdamwConfig(self.lr if lr is None else lr, self.betas[0], self.betas[1],
                                  self.eps, grad_scale, self.state_bits, count)
        _lib.adamw_step(config, self._table, None if out is None else out._table, n, dev, stream)
        if to._mastered:
            _lib._written(to.params, to.masters)
        else:
            torch.autograd.graph.increment_version(to.params)
        to.step_count = count

    def _refuse(self, grads) -> None:
        for i, (g, p) in enumerate(zip(grads, self.params)):
            if not torch.is_tensor(g):
                raise ValueError("grads[%d] must be a tensor, got %r (give a parameter without a gradient zeros, "
                                 "or leave it out of the optimizer)" % (i, type(g)))
            if g.shape != p.shape:
                raise ValueError("grads[%d] must have shape %s, got %s" % (i, tuple(p.shape), tuple(g.shape)))
            if g.device != self.device or not g.is_contiguous():
                raise ValueError("grads[%d] must be contiguous and on %s" % (i, self.device))
            _lib._plain_code(g.dtype, "grads[%d]" % i)
