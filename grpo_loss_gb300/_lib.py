"""ctypes binding of the C ABI declared in include/grpo.h.

Argument marshalling only: every step of the loss runs in the library's CUDA
kernels. There is no CPU fallback; if the shared library has not been built
the first call raises.
"""
from __future__ import annotations

import ctypes
import math
import operator
import os
import struct
import threading
from typing import Optional

import numpy as np
import torch

# The in-tree build; GRPO_GB300_LIB may name another build of the same library.
LIB_PATH = os.environ.get("GRPO_GB300_LIB") or os.path.join(
    os.path.dirname(os.path.abspath(__file__)), "libgrpo_gb300.so")

GRPO_OK = 0
STATUS_NAMES = {0: "GRPO_OK", 1: "GRPO_ERR_INVALID_ARG", 2: "GRPO_ERR_UNSUPPORTED",
                3: "GRPO_ERR_WORKSPACE", 4: "GRPO_ERR_CUDA", 5: "GRPO_ERR_TIMEOUT",
                6: "GRPO_ERR_BAD_TOKEN"}
GRPO_F32, GRPO_BF16, GRPO_E4M3 = 0, 1, 2


class GrpoError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__("%s failed: %s (%s)" % (where, STATUS_NAMES.get(status, status),
                                                  status_string(status)))


class Problem(ctypes.Structure):
    """Mirror of ``grpo_problem``."""
    _fields_ = [("N", ctypes.c_int64), ("d", ctypes.c_int64), ("V", ctypes.c_int64),
                ("num_seqs", ctypes.c_int32), ("seq_len", ctypes.c_int32),
                ("group_size", ctypes.c_int32), ("beta", ctypes.c_float),
                ("eps", ctypes.c_float), ("std_unbiased", ctypes.c_int32),
                ("chunk_rows", ctypes.c_int64), ("compute_dW", ctypes.c_int32),
                ("dtype", ctypes.c_int32), ("token_level", ctypes.c_int32),
                ("logit_multiply", ctypes.c_float), ("logit_divide", ctypes.c_float),
                ("softcap", ctypes.c_float), ("temperature", ctypes.c_float),
                ("ref_logp_given", ctypes.c_int32), ("kl_mode", ctypes.c_int32),
                ("cluster_mode", ctypes.c_int32)]


class SampleProblem(ctypes.Structure):
    """Mirror of ``grpo_sample_problem``."""
    _fields_ = [("rows", ctypes.c_int64), ("V", ctypes.c_int64), ("ld", ctypes.c_int64),
                ("dtype", ctypes.c_int32)]


class LayernormProblem(ctypes.Structure):
    """Mirror of ``grpo_layernorm_problem``."""
    _fields_ = [("rows", ctypes.c_int64), ("d", ctypes.c_int64), ("ld_x", ctypes.c_int64),
                ("ld_y", ctypes.c_int64), ("ld_dy", ctypes.c_int64), ("ld_dx", ctypes.c_int64),
                ("eps", ctypes.c_float), ("rms", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("param_dtype", ctypes.c_int32)]


class AdamwTensor(ctypes.Structure):
    """Mirror of ``grpo_adamw_tensor``."""
    _fields_ = [("n", ctypes.c_int64)] + \
        [(k, ctypes.c_void_p) for k in ("grad", "param", "master", "m", "v", "m_scale", "v_scale")] + \
        [("weight_decay", ctypes.c_float), ("param_dtype", ctypes.c_int32),
         ("grad_dtype", ctypes.c_int32)]


# The fields of AdamwTensor that a step fills, as columns of an array of them.
ADAMW_COLUMNS = np.dtype({"names": ["grad", "grad_dtype", "weight_decay"], "formats": [np.uint64, np.int32, np.float32],
                          "offsets": [AdamwTensor.grad.offset, AdamwTensor.grad_dtype.offset,
                                      AdamwTensor.weight_decay.offset],
                          "itemsize": ctypes.sizeof(AdamwTensor)})


class AdamwConfig(ctypes.Structure):
    """Mirror of ``grpo_adamw_config``."""
    _fields_ = [("lr", ctypes.c_double), ("beta1", ctypes.c_double), ("beta2", ctypes.c_double),
                ("eps", ctypes.c_double), ("grad_scale", ctypes.c_float),
                ("state_bits", ctypes.c_int32), ("step", ctypes.c_int64), ("factor", ctypes.c_void_p)]


class PolicyProblem(ctypes.Structure):
    """Mirror of ``grpo_policy_problem``."""
    _fields_ = [(k, ctypes.c_int64) for k in ("num_seqs", "seq_len", "ld_logp", "ld_old", "ld_ref", "ld_adv",
                                              "ld_mask", "ld_dlogp")] + \
        [(k, ctypes.c_double) for k in ("clip_low", "clip_high", "dual_clip", "beta", "divisor")] + \
        [(k, ctypes.c_int32) for k in ("ratio", "reduce", "token_adv")]


class ResidualNormProblem(ctypes.Structure):
    """Mirror of ``grpo_residual_norm_problem``."""
    _fields_ = [(k, ctypes.c_int64) for k in ("rows", "d", "ld_x", "ld_residual", "ld_h", "ld_y", "ld_gate", "ld_dy",
                                              "ld_dh", "ld_dx", "ld_dresidual", "ld_dgate", "gate_rows")] + \
        [("eps", ctypes.c_float), ("scale", ctypes.c_float)] + \
        [(k, ctypes.c_int32) for k in ("rms", "dtype", "param_dtype", "gate_dtype")]


class GradTensor(ctypes.Structure):
    """Mirror of ``grpo_grad_tensor``."""
    _fields_ = [("n", ctypes.c_int64), ("grad", ctypes.c_void_p), ("out", ctypes.c_void_p), ("dtype", ctypes.c_int32)]


def make_problem(num_seqs: int, seq_len: int, d: int, V: int, group_size: int,
                 beta: float = 0.04, eps: float = 1e-4, std_unbiased: int = 1,
                 chunk_rows: int = 0, dtype=torch.bfloat16, compute_dW: int = 0,
                 token_level: bool = False, logit_multiply: float = 0.0,
                 logit_divide: float = 0.0, softcap: float = 0.0, temperature: float = 0.0,
                 ref_logp_given: bool = False, kl_mode: int = 0,
                 cluster_mode: int = 0) -> Problem:
    return Problem(N=num_seqs * seq_len, d=d, V=V, num_seqs=num_seqs, seq_len=seq_len,
                   group_size=group_size, beta=beta, eps=eps, std_unbiased=std_unbiased,
                   chunk_rows=chunk_rows, compute_dW=1 if compute_dW else 0,
                   dtype=dtype_code(dtype),
                   token_level=1 if token_level else 0, logit_multiply=logit_multiply,
                   logit_divide=logit_divide, softcap=softcap, temperature=temperature,
                   ref_logp_given=1 if ref_logp_given else 0, kl_mode=kl_mode,
                   cluster_mode=cluster_mode)


def dtype_code(dtype) -> int:
    """grpo_dtype of a torch dtype: float32, bfloat16, or float8_e4m3fn for an
    e4m3 problem (operands as codes with row scales)."""
    if dtype == torch.float32:
        return GRPO_F32
    if dtype == torch.float8_e4m3fn:
        return GRPO_E4M3
    if dtype == torch.bfloat16:
        return GRPO_BF16
    raise ValueError("unsupported dtype %s" % (dtype,))


_lib = None
_lock = threading.Lock()

_VP = ctypes.c_void_p
_SIGNATURES = {
    "grpo_workspace_size": (ctypes.c_int, [ctypes.POINTER(Problem), ctypes.POINTER(ctypes.c_size_t),
                                           ctypes.POINTER(ctypes.c_size_t)]),
    "grpo_chunk_plan": (ctypes.c_int, [ctypes.POINTER(Problem), ctypes.POINTER(ctypes.c_int64),
                                       ctypes.POINTER(ctypes.c_int32),
                                       ctypes.POINTER(ctypes.c_size_t)]),
    "grpo_advantages": (ctypes.c_int, [_VP, ctypes.c_int32, ctypes.c_int32, ctypes.c_float,
                                       ctypes.c_int32, _VP, _VP]),
    "grpo_loss_fwd": (ctypes.c_int, [ctypes.POINTER(Problem)] + [_VP] * 11 +
                      [_VP, ctypes.c_size_t, _VP]),
    "grpo_loss_bwd": (ctypes.c_int, [ctypes.POINTER(Problem)] + [_VP] * 8 +
                      [ctypes.c_float, _VP, _VP, _VP, ctypes.c_size_t, _VP]),
    "grpo_loss_fwd_e4m3": (ctypes.c_int, [ctypes.POINTER(Problem)] + [_VP] * 14 +
                           [_VP, ctypes.c_size_t, _VP]),
    "grpo_loss_bwd_e4m3": (ctypes.c_int, [ctypes.POINTER(Problem)] + [_VP] * 10 +
                           [ctypes.c_float, _VP, _VP, _VP, ctypes.c_size_t, _VP]),
    "grpo_quantize_e4m3_rows": (ctypes.c_int, [_VP, ctypes.c_int, ctypes.c_int64, ctypes.c_int64,
                                               _VP, _VP, _VP]),
    "grpo_sample": (ctypes.c_int, [ctypes.POINTER(SampleProblem)] + [_VP] * 9),
    "grpo_layernorm_workspace_size": (ctypes.c_int, [ctypes.POINTER(LayernormProblem),
                                                     ctypes.POINTER(ctypes.c_size_t)]),
    "grpo_layernorm_fwd": (ctypes.c_int, [ctypes.POINTER(LayernormProblem)] + [_VP] * 7),
    "grpo_layernorm_bwd": (ctypes.c_int, [ctypes.POINTER(LayernormProblem)] + [_VP] * 9 +
                           [ctypes.c_size_t, _VP]),
    "grpo_adamw_step": (ctypes.c_int, [ctypes.POINTER(AdamwConfig), ctypes.POINTER(AdamwTensor),
                                       ctypes.POINTER(AdamwTensor), ctypes.c_int32, _VP]),
    "grpo_policy_loss_workspace_size": (ctypes.c_int, [ctypes.POINTER(PolicyProblem),
                                                       ctypes.POINTER(ctypes.c_size_t)]),
    "grpo_policy_loss": (ctypes.c_int, [ctypes.POINTER(PolicyProblem)] + [_VP] * 9 + [ctypes.c_size_t, _VP]),
    "grpo_loss_bwd_dlogp": (ctypes.c_int, [ctypes.POINTER(Problem)] + [_VP] * 6 +
                            [ctypes.c_float, _VP, _VP, _VP, ctypes.c_size_t, _VP]),
    "grpo_loss_bwd_dlogp_e4m3": (ctypes.c_int, [ctypes.POINTER(Problem)] + [_VP] * 8 +
                                 [ctypes.c_float, _VP, _VP, _VP, ctypes.c_size_t, _VP]),
    "grpo_residual_norm_workspace_size": (ctypes.c_int, [ctypes.POINTER(ResidualNormProblem),
                                                         ctypes.POINTER(ctypes.c_size_t)]),
    "grpo_residual_norm_fwd": (ctypes.c_int, [ctypes.POINTER(ResidualNormProblem)] + [_VP] * 14),
    "grpo_residual_norm_bwd": (ctypes.c_int, [ctypes.POINTER(ResidualNormProblem)] + [_VP] * 20 +
                               [ctypes.c_size_t, _VP]),
    "grpo_grad_norm_workspace_size": (ctypes.c_int, [ctypes.POINTER(ctypes.c_size_t)]),
    "grpo_grad_norm": (ctypes.c_int, [_VP, ctypes.c_int32, ctypes.c_int32, ctypes.c_double, ctypes.c_double] +
                       [_VP] * 3 + [ctypes.c_size_t, _VP]),
    "grpo_clip_grad_norm": (ctypes.c_int, [_VP, ctypes.c_int32, ctypes.c_int32, ctypes.c_double, ctypes.c_double] +
                            [_VP] * 3 + [ctypes.c_size_t, _VP]),
    "grpo_get_device_status": (ctypes.c_int, [_VP, _VP]),
    "grpo_status_string": (ctypes.c_char_p, [ctypes.c_int]),
    "grpo_profile_enable": (ctypes.c_int, [ctypes.c_int32]),
    "grpo_profile_collect": (ctypes.c_int, [ctypes.POINTER(ctypes.c_double),
                                            ctypes.POINTER(ctypes.c_int64), ctypes.c_int32]),
    "grpo_profile_kind_count": (ctypes.c_int32, []),
    "grpo_test_pipeline_stall": (ctypes.c_int, [ctypes.c_int32, ctypes.c_uint32]),
    "grpo_profile_kind_name": (ctypes.c_char_p, [ctypes.c_int32]),
}


def lib() -> ctypes.CDLL:
    """Load the in-tree shared library (raises if it has not been built)."""
    global _lib
    if _lib is None:
        with _lock:
            if _lib is None:
                if not os.path.exists(LIB_PATH):
                    raise RuntimeError(
                        "libgrpo_gb300.so is missing: build it with "
                        "`python -m grpo_loss_gb300.build` (needs nvcc); there is no CPU fallback")
                handle = ctypes.CDLL(LIB_PATH)
                for name, (res, args) in _SIGNATURES.items():
                    fn = getattr(handle, name)
                    fn.restype = res
                    fn.argtypes = args
                _lib = handle
    return _lib


def status_string(status: int) -> str:
    return lib().grpo_status_string(status).decode()


def _check(status: int, where: str) -> None:
    if status != GRPO_OK:
        raise GrpoError(status, where)


def _ptr(t: Optional[torch.Tensor], name: str, dtype=None, numel: Optional[int] = None):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("%s must be a CUDA tensor" % name)
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    if dtype is not None and t.dtype != dtype:
        raise ValueError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if numel is not None and t.numel() != numel:
        raise ValueError("%s must have %d elements, got %d" % (name, numel, t.numel()))
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream=None):
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def workspace_size(problem: Problem):
    f, b = ctypes.c_size_t(0), ctypes.c_size_t(0)
    _check(lib().grpo_workspace_size(ctypes.byref(problem), ctypes.byref(f), ctypes.byref(b)),
           "grpo_workspace_size")
    return f.value, b.value


def chunk_plan(problem: Problem):
    """(chunk_rows, n_chunks, dz_chunk_bytes) of the backward's chunk plan."""
    r, n, b = ctypes.c_int64(0), ctypes.c_int32(0), ctypes.c_size_t(0)
    _check(lib().grpo_chunk_plan(ctypes.byref(problem), ctypes.byref(r), ctypes.byref(n),
                                 ctypes.byref(b)), "grpo_chunk_plan")
    return r.value, n.value, b.value


def advantages(rewards: torch.Tensor, group_size: int, eps: float, std_unbiased: int,
               adv: torch.Tensor, stream=None) -> torch.Tensor:
    B = rewards.numel()
    _check(lib().grpo_advantages(_ptr(rewards, "rewards", torch.float32), B, group_size, eps,
                                 std_unbiased, _ptr(adv, "adv", torch.float32, B), _stream(stream)),
           "grpo_advantages")
    return adv


def loss_fwd(problem: Problem, H_pol, H_ref, W, ids, mask, adv, logp_pol, logp_ref, lse_pol,
             loss, kl_mean, workspace: torch.Tensor, stream=None) -> None:
    N = problem.N
    _check(lib().grpo_loss_fwd(
        ctypes.byref(problem), _ptr(H_pol, "H_pol"),
        None if H_ref is None else _ptr(H_ref, "H_ref"), _ptr(W, "W"),
        _ptr(ids, "ids", torch.int32, N), _ptr(mask, "mask", torch.uint8, N),
        _ptr(adv, "adv", torch.float32, problem.num_seqs),
        _ptr(logp_pol, "logp_pol", torch.float32, N), _ptr(logp_ref, "logp_ref", torch.float32, N),
        _ptr(lse_pol, "lse_pol", torch.float32, N), _ptr(loss, "loss", torch.float32, 1),
        _ptr(kl_mean, "kl_mean", torch.float32, 1), _ptr(workspace, "workspace"),
        workspace.numel() * workspace.element_size(), _stream(stream)), "grpo_loss_fwd")


def loss_bwd(problem: Problem, H_pol, W, ids, mask, adv, logp_pol, logp_ref, lse_pol,
             grad_loss: float, dH, workspace: torch.Tensor, stream=None, dW=None) -> None:
    N = problem.N
    _check(lib().grpo_loss_bwd(
        ctypes.byref(problem), _ptr(H_pol, "H_pol"), _ptr(W, "W"),
        _ptr(ids, "ids", torch.int32, N), _ptr(mask, "mask", torch.uint8, N),
        _ptr(adv, "adv", torch.float32, problem.num_seqs),
        _ptr(logp_pol, "logp_pol", torch.float32, N), _ptr(logp_ref, "logp_ref", torch.float32, N),
        _ptr(lse_pol, "lse_pol", torch.float32, N), float(grad_loss), _ptr(dH, "dH"),
        _ptr(dW, "dW", torch.float32, problem.V * problem.d),
        _ptr(workspace, "workspace"), workspace.numel() * workspace.element_size(),
        _stream(stream)), "grpo_loss_bwd")


def _codes(t, name: str, numel: int):
    """Pointer to e4m3 codes held as uint8 or float8_e4m3fn."""
    if t is None:
        return None
    if t.dtype not in (torch.uint8, torch.float8_e4m3fn):
        raise ValueError("%s must hold e4m3 codes (uint8 or float8_e4m3fn), got %s" % (name, t.dtype))
    return _ptr(t, name, None, numel)


def quantize_e4m3_rows(x: torch.Tensor, q=None, scale=None, stream=None):
    """Row-wise e4m3 codes (uint8 [rows, cols]) and scales (float32 [rows]) of
    a float32 or bf16 CUDA matrix; see grpo_quantize_e4m3_rows."""
    if x.dim() != 2:
        raise ValueError("x must be 2-D")
    rows, cols = x.shape
    if x.dtype == torch.float32:
        code = GRPO_F32
    elif x.dtype == torch.bfloat16:
        code = GRPO_BF16
    else:
        raise ValueError("x must be float32 or bfloat16")
    if q is None:
        q = torch.empty(rows, cols, dtype=torch.uint8, device=x.device)
    if scale is None:
        scale = torch.empty(rows, dtype=torch.float32, device=x.device)
    _check(lib().grpo_quantize_e4m3_rows(_ptr(x, "x"), code, rows, cols,
                                         _codes(q, "q", rows * cols),
                                         _ptr(scale, "scale", torch.float32, rows),
                                         _stream(stream)), "grpo_quantize_e4m3_rows")
    return q, scale


def loss_fwd_e4m3(problem: Problem, H_pol, s_pol, H_ref, s_ref, W, s_W, ids, mask, adv,
                  logp_pol, logp_ref, lse_pol, loss, kl_mean, workspace: torch.Tensor,
                  stream=None) -> None:
    N, Nd, Vd = problem.N, problem.N * problem.d, problem.V * problem.d
    _check(lib().grpo_loss_fwd_e4m3(
        ctypes.byref(problem), _codes(H_pol, "H_pol", Nd), _ptr(s_pol, "s_pol", torch.float32, N),
        _codes(H_ref, "H_ref", Nd), _ptr(s_ref, "s_ref", torch.float32, N),
        _codes(W, "W", Vd), _ptr(s_W, "s_W", torch.float32, problem.V),
        _ptr(ids, "ids", torch.int32, N), _ptr(mask, "mask", torch.uint8, N),
        _ptr(adv, "adv", torch.float32, problem.num_seqs),
        _ptr(logp_pol, "logp_pol", torch.float32, N), _ptr(logp_ref, "logp_ref", torch.float32, N),
        _ptr(lse_pol, "lse_pol", torch.float32, N), _ptr(loss, "loss", torch.float32, 1),
        _ptr(kl_mean, "kl_mean", torch.float32, 1), _ptr(workspace, "workspace"),
        workspace.numel() * workspace.element_size(), _stream(stream)), "grpo_loss_fwd_e4m3")


def loss_bwd_e4m3(problem: Problem, H_pol, s_pol, W, s_W, ids, mask, adv, logp_pol, logp_ref,
                  lse_pol, grad_loss: float, dH, workspace: torch.Tensor, stream=None,
                  dW=None) -> None:
    N, Nd, Vd = problem.N, problem.N * problem.d, problem.V * problem.d
    _check(lib().grpo_loss_bwd_e4m3(
        ctypes.byref(problem), _codes(H_pol, "H_pol", Nd), _ptr(s_pol, "s_pol", torch.float32, N),
        _codes(W, "W", Vd), _ptr(s_W, "s_W", torch.float32, problem.V),
        _ptr(ids, "ids", torch.int32, N), _ptr(mask, "mask", torch.uint8, N),
        _ptr(adv, "adv", torch.float32, problem.num_seqs),
        _ptr(logp_pol, "logp_pol", torch.float32, N), _ptr(logp_ref, "logp_ref", torch.float32, N),
        _ptr(lse_pol, "lse_pol", torch.float32, N), float(grad_loss),
        _ptr(dH, "dH", torch.bfloat16, Nd),
        _ptr(dW, "dW", torch.float32, Vd),
        _ptr(workspace, "workspace"), workspace.numel() * workspace.element_size(),
        _stream(stream)), "grpo_loss_bwd_e4m3")


def _plain_code(dtype, name: str) -> int:
    """grpo_dtype of float32 or bfloat16."""
    if dtype == torch.float32:
        return GRPO_F32
    if dtype == torch.bfloat16:
        return GRPO_BF16
    raise ValueError("%s must be float32 or bfloat16, got %s" % (name, dtype))


def _device_of(t: torch.Tensor, name: str):
    if not t.is_cuda:
        raise ValueError("%s must be a CUDA tensor" % name)
    return t.device


def _rows_ptr(t: torch.Tensor, name: str, dtype, rows: int, cols: int, device):
    """(pointer, row stride) of a [rows, cols] matrix on ``device`` whose columns
    are contiguous; the rows may be strided."""
    if t.dtype != dtype:
        raise ValueError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if t.device != device:
        raise ValueError("%s must be on %s, got %s" % (name, device, t.device))
    if t.shape != (rows, cols):
        raise ValueError("%s must have shape (%d, %d), got %s" % (name, rows, cols, tuple(t.shape)))
    ld, inner = t.stride()
    if inner != 1 and cols > 1:
        raise ValueError("%s must be contiguous along its last dimension" % name)
    if rows <= 1:
        ld = cols
    elif ld < cols:
        raise ValueError("%s must have a row stride of at least %d, got %d" % (name, cols, ld))
    return t.data_ptr(), ld


def _vec_ptr(t, name: str, dtype, numel: int, device):
    """Pointer of an optional contiguous tensor of ``numel`` elements on ``device``."""
    if t is None:
        return None
    if t.dtype != dtype:
        raise ValueError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if t.device != device:
        raise ValueError("%s must be on %s, got %s" % (name, device, t.device))
    if t.numel() != numel:
        raise ValueError("%s must have %d elements, got %d" % (name, numel, t.numel()))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    return t.data_ptr()


def _rows_out(t, name: str, dtype, rows: int, cols: int, device):
    """(tensor, pointer, row stride) of an output that is given or made."""
    if t is None:
        t = torch.empty(rows, cols, dtype=dtype, device=device)
        return t, t.data_ptr(), cols
    return (t,) + _rows_ptr(t, name, dtype, rows, cols, device)


def _vec_out(t, name: str, dtype, numel: int, device):
    """(tensor, pointer) of an output that is given or made."""
    if t is None:
        t = torch.empty(numel, dtype=dtype, device=device)
        return t, t.data_ptr()
    return t, _vec_ptr(t, name, dtype, numel, device)


def _vec_outs(given, numel: int, device):
    """[(tensor, pointer)] of float32 outputs that are given, made, or not there: given has
    (tensor or None, name, whether it is made). Three and more are made at once."""
    if sum(t is None and made for t, _, made in given) >= 3:
        rows = iter(torch.empty(len(given), numel, dtype=torch.float32, device=device).unbind(0))
        given = [(next(rows) if t is None and made else t, name, made) for t, name, made in given]
    return [(None, None) if t is None and not made else _vec_out(t, name, torch.float32, numel, device)
            for t, name, made in given]


def _call(fn, where: str, device, stream, *args) -> None:
    """fn(*args, stream) with ``device`` current, on ``stream`` or the device's
    current one. The launches of small operators are bound by the host: torch's
    own stream and device objects are not made where their numbers will do (nor is
    new_empty used for outputs: torch.empty takes 2 us less of a tensor)."""
    at = device.index
    raw = stream.cuda_stream if stream is not None else torch._C._cuda_getCurrentRawStream(at)
    if torch._C._cuda_getDevice() == at:
        status = fn(*args, raw)
    else:
        with torch.cuda.device(device):
            status = fn(*args, raw)
    if status != GRPO_OK:
        raise GrpoError(status, where)


def _written(*lists) -> None:
    """Autograd learns that a call wrote the tensors of these (None for one that was not
    given): what it saved of them is gone."""
    given = [t for ts in lists for t in ts if t is not None]
    if given:
        torch.autograd.graph.increment_version(given)


def sample(logits: torch.Tensor, u: torch.Tensor, temperature=None, top_k=None, top_p=None,
           min_p=None, tokens=None, logp=None, stream=None):
    """One token a row of ``logits`` (float32 or bf16 [rows, V], rows may be
    strided) from the uniforms ``u`` (float32 [rows]): (tokens int32 [rows],
    logp float32 [rows]). ``temperature``, ``top_p``, ``min_p`` (float32 [rows])
    and ``top_k`` (int32 [rows]) are optional; see grpo_sample for the
    definition. logp is the token's log-probability under the full softmax at
    its temperature, what a GRPOLoss with that temperature calls logp_pol.
    Outputs that are not given belong to ``stream``."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return sample(logits, u, temperature, top_k, top_p, min_p, tokens, logp)
    if logits.dim() != 2:
        raise ValueError("logits must be 2-D")
    rows, V = logits.shape
    i32, f32 = torch.int32, torch.float32
    code = _plain_code(logits.dtype, "logits")
    dev = _device_of(logits, "logits")
    ptr, ld = _rows_ptr(logits, "logits", logits.dtype, rows, V, dev)
    given = tokens, logp
    tokens, tp = _vec_out(tokens, "tokens", i32, rows, dev)
    logp, lp = _vec_out(logp, "logp", f32, rows, dev)
    _call(lib().grpo_sample, "grpo_sample", dev, None, SampleProblem(rows, V, ld, code), ptr,
          _vec_ptr(u, "u", f32, rows, dev), _vec_ptr(temperature, "temperature", f32, rows, dev),
          _vec_ptr(top_k, "top_k", i32, rows, dev), _vec_ptr(top_p, "top_p", f32, rows, dev),
          _vec_ptr(min_p, "min_p", f32, rows, dev), tp, lp)
    _written(given)
    return tokens, logp


def layernorm_workspace_size(problem: LayernormProblem) -> int:
    """Bytes of grpo_layernorm_bwd's workspace on the current device."""
    b = ctypes.c_size_t(0)
    _check(lib().grpo_layernorm_workspace_size(ctypes.byref(problem), ctypes.byref(b)),
           "grpo_layernorm_workspace_size")
    return b.value


def layernorm_fwd(x: torch.Tensor, weight: torch.Tensor, bias=None, eps: float = 1e-5,
                  rms: bool = False, y=None, mean=None, rstd=None, stream=None):
    """Layer norm (RMS norm with ``rms``) of the rows of ``x`` (float32 or bf16
    [rows, d], rows may be strided): (y, mean, rstd), mean None with ``rms``.
    ``weight`` and ``bias`` are float32 or bf16 [d], of one type. Outputs that are
    not given belong to ``stream``."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return layernorm_fwd(x, weight, bias, eps, rms, y, mean, rstd)
    if x.dim() != 2:
        raise ValueError("x must be 2-D")
    rows, d = x.shape
    f32, dt, pt = torch.float32, x.dtype, weight.dtype
    code, pcode = _plain_code(dt, "x"), _plain_code(pt, "weight")
    dev = _device_of(x, "x")
    xp, ld_x = _rows_ptr(x, "x", dt, rows, d, dev)
    given = y, None if rms else mean, rstd
    y, yp, ld_y = _rows_out(y, "y", dt, rows, d, dev)
    mean, mp = (None, None) if rms else _vec_out(mean, "mean", f32, rows, dev)
    rstd, rp = _vec_out(rstd, "rstd", f32, rows, dev)
    problem = LayernormProblem(rows, d, ld_x, ld_y, 0, 0, eps, 1 if rms else 0, code, pcode)
    _call(lib().grpo_layernorm_fwd, "grpo_layernorm_fwd", dev, None, problem, xp,
          _vec_ptr(weight, "weight", pt, d, dev), _vec_ptr(bias, "bias", pt, d, dev), yp, mp, rp)
    _written(given)
    return y, mean, rstd


def layernorm_bwd(x: torch.Tensor, weight: torch.Tensor, dy: torch.Tensor, mean, rstd,
                  rms: bool = False, bias: bool = True, dx=None, dweight=None, dbias=None,
                  need_dweight: bool = True, workspace=None, stream=None):
    """Gradients of ``layernorm_fwd`` from its inputs and statistics: (dx,
    dweight, dbias), dx of x's type, the column sums float32 [d]; dweight is None
    without ``need_dweight``, dbias without ``bias`` or with ``rms``. Outputs and a
    workspace that are not given belong to ``stream``."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return layernorm_bwd(x, weight, dy, mean, rstd, rms, bias, dx, dweight, dbias,
                                 need_dweight, workspace)
    if x.dim() != 2:
        raise ValueError("x must be 2-D")
    rows, d = x.shape
    f32, dt, pt = torch.float32, x.dtype, weight.dtype
    code, pcode = _plain_code(dt, "x"), _plain_code(pt, "weight")
    dev = _device_of(x, "x")
    if mean is None and not rms:
        raise ValueError("mean is needed unless rms")
    xp, ld_x = _rows_ptr(x, "x", dt, rows, d, dev)
    gp, ld_dy = _rows_ptr(dy, "dy", dt, rows, d, dev)
    given = dx, dweight, dbias
    dx, dxp, ld_dx = _rows_out(dx, "dx", dt, rows, d, dev)
    wp = bp = None
    if dweight is not None or need_dweight:
        dweight, wp = _vec_out(dweight, "dweight", f32, d, dev)
    if dbias is not None or (bias and not rms):
        dbias, bp = _vec_out(dbias, "dbias", f32, d, dev)
    problem = LayernormProblem(rows, d, ld_x, 0, ld_dy, ld_dx, 0.0, 1 if rms else 0, code, pcode)
    size = 0
    if workspace is None and (dweight is not None or dbias is not None):
        if torch._C._cuda_getDevice() == dev.index:
            size = layernorm_workspace_size(problem)
        else:
            with torch.cuda.device(dev):
                size = layernorm_workspace_size(problem)
        workspace = torch.empty(size, dtype=torch.uint8, device=dev)
    elif workspace is not None:
        size = workspace.numel() * workspace.element_size()
    _call(lib().grpo_layernorm_bwd, "grpo_layernorm_bwd", dev, None, problem, xp,
          _vec_ptr(weight, "weight", pt, d, dev), gp,
          None if rms else _vec_ptr(mean, "mean", f32, rows, dev),
          _vec_ptr(rstd, "rstd", f32, rows, dev), dxp, wp, bp,
          None if workspace is None else _vec_ptr(workspace, "workspace", workspace.dtype,
                                                  workspace.numel(), dev), size)
    _written(given)
    return dx, dweight, dbias


def adamw_step(config: AdamwConfig, tensors, out, n: int, device, stream=None) -> None:
    """One grpo_adamw_step over ctypes arrays of AdamwTensor (``out`` may be None);
    the AdamW class checks the tensors and fills the arrays."""
    _call(lib().grpo_adamw_step, "grpo_adamw_step", device, stream, config, tensors, out, n)


_sizes = {}


def _bytes(key, fn, where: str, dev, *args) -> int:
    """A workspace's size, asked with ``dev`` current, once for each ``key`` (what it depends
    on) and device."""
    key = key, dev.index
    size = _sizes.get(key)
    if size is not None:
        return size
    b = ctypes.c_size_t(0)
    if torch._C._cuda_getDevice() == dev.index:
        status = fn(*args, ctypes.byref(b))
    else:
        with torch.cuda.device(dev):
            status = fn(*args, ctypes.byref(b))
    if status != GRPO_OK:
        raise GrpoError(status, where)
    if len(_sizes) >= 4096:
        _sizes.clear()
    _sizes[key] = b.value
    return b.value


def _workspace(workspace, size: int, dev):
    """(tensor, pointer, bytes) of a workspace that is given or made of ``size`` bytes."""
    if workspace is None:
        if not size:
            return None, None, 0
        workspace = torch.empty(size, dtype=torch.uint8, device=dev)
        return workspace, workspace.data_ptr(), size
    return workspace, _vec_ptr(workspace, "workspace", workspace.dtype, workspace.numel(), dev), workspace.nbytes


_RATIOS = {"token": 0, "sequence": 1, "sequence_token": 1}
_REDUCES = {"sequence": 0, "token": 1, "constant": 2}


def policy_workspace_size(problem: PolicyProblem) -> int:
    """Bytes of grpo_policy_loss's workspace on the current device."""
    b = ctypes.c_size_t(0)
    _check(lib().grpo_policy_loss_workspace_size(ctypes.byref(problem), ctypes.byref(b)),
           "grpo_policy_loss_workspace_size")
    return b.value


def policy_loss(logp: torch.Tensor, advantages: torch.Tensor, mask: torch.Tensor, logp_old=None, logp_ref=None,
                clip=(0.2, 0.2), dual_clip: Optional[float] = None, beta: float = 0.0, ratio: str = "token",
                reduce: str = "sequence", divisor: Optional[float] = None, need_dlogp: bool = True, loss=None,
                dlogp=None, stats=None, workspace=None, stream=None):
    """The clipped policy loss with its KL term over ``logp`` (float32 [B, T], rows may
    be strided, as those of every [B, T] here): (loss float32 [1], dlogp float32 [B, T],
    stats float32 [4]); see grpo_policy_loss for the definition. ``advantages`` is float32
    [B] or [B, T]; ``mask`` bool or uint8 [B, T]; ``logp_old`` and ``logp_ref`` float32
    [B, T], optional: ratio 1, and no KL term. ``clip`` is (low, high); ``ratio`` "token",
    "sequence" or "sequence_token". The last two have the ratio of the mean over a sequence,
    with the same loss; dlogp is the loss's gradient where the advantages are [B], and where
    they are [B, T] that of the surrogate in which each token has the sequence's ratio times
    its own probability over itself held constant (its name is "sequence_token"; "sequence"
    is taken for it here). ``reduce`` "sequence" (the mean over each sequence's tokens, then over
    sequences), "token" (over all tokens) or "constant" (the sum over ``divisor``).
    ``stats`` are means over valid tokens: the KL estimate, the shares of tokens whose
    gradient the lower and the upper bound took away, the ratio. dlogp is None without
    ``need_dlogp``. Outputs and a workspace that are not given belong to ``stream``."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return policy_loss(logp, advantages, mask, logp_old, logp_ref, clip, dual_clip, beta, ratio, reduce,
                               divisor, need_dlogp, loss, dlogp, stats, workspace)
    if logp.dim() != 2:
        raise ValueError("logp must be 2-D")
    try:
        clip_low, clip_high = clip
    except (TypeError, ValueError):
        raise ValueError("clip must be two numbers, (low, high), got %r" % (clip,)) from None
    if ratio not in _RATIOS:
        raise ValueError("ratio must be one of %s, got %r" % (sorted(_RATIOS), ratio))
    if reduce not in _REDUCES:
        raise ValueError("reduce must be one of %s, got %r" % (sorted(_REDUCES), reduce))
    if (reduce == "constant") != (divisor is not None):
        raise ValueError("divisor is needed with reduce=\"constant\", and only there")
    B, T = logp.shape
    f32 = torch.float32
    dev = _device_of(logp, "logp")
    lp, ld = _rows_ptr(logp, "logp", f32, B, T, dev)
    if mask.dtype != torch.bool and mask.dtype != torch.uint8:
        raise ValueError("mask must be bool or uint8, got %s" % (mask.dtype,))
    mp, ld_mask = _rows_ptr(mask, "mask", mask.dtype, B, T, dev)
    op, ld_old = (None, 0) if logp_old is None else _rows_ptr(logp_old, "logp_old", f32, B, T, dev)
    rp, ld_ref = (None, 0) if logp_ref is None else _rows_ptr(logp_ref, "logp_ref", f32, B, T, dev)
    per_token = advantages.dim() == 2
    if per_token:
        ap, ld_adv = _rows_ptr(advantages, "advantages", f32, B, T, dev)
    else:
        ap, ld_adv = _vec_ptr(advantages, "advantages", f32, B, dev), 0
    given = loss, dlogp, stats
    loss, out = _vec_out(loss, "loss", f32, 1, dev)
    stats, sp = _vec_out(stats, "stats", f32, 4, dev)
    dp, ld_d = None, 0
    if dlogp is not None or need_dlogp:
        dlogp, dp, ld_d = _rows_out(dlogp, "dlogp", f32, B, T, dev)
    problem = PolicyProblem(B, T, ld, ld_old, ld_ref, ld_adv, ld_mask, ld_d, clip_low, clip_high, dual_clip or 0.0, beta,
                            divisor or 0.0, _RATIOS[ratio], _REDUCES[reduce], 1 if per_token else 0)
    L = lib()
    size = 0 if workspace is not None else _bytes(("policy", B, T, ratio), L.grpo_policy_loss_workspace_size,
                                                  "grpo_policy_loss_workspace_size", dev, problem)
    workspace, wp, size = _workspace(workspace, size, dev)
    _call(L.grpo_policy_loss, "grpo_policy_loss", dev, None, problem, lp, op, rp, ap, mp, out, sp, dp, wp, size)
    _written(given)
    return loss, dlogp, stats


def loss_bwd_dlogp(problem: Problem, H_pol, W, ids, mask, dlogp, lse_pol, grad_loss: float, dH,
                   workspace: torch.Tensor, stream=None, dW=None) -> None:
    N = problem.N
    _check(lib().grpo_loss_bwd_dlogp(
        ctypes.byref(problem), _ptr(H_pol, "H_pol"), _ptr(W, "W"), _ptr(ids, "ids", torch.int32, N),
        _ptr(mask, "mask", torch.uint8, N), _ptr(dlogp, "dlogp", torch.float32, N),
        _ptr(lse_pol, "lse_pol", torch.float32, N), float(grad_loss), _ptr(dH, "dH"),
        _ptr(dW, "dW", torch.float32, problem.V * problem.d), _ptr(workspace, "workspace"),
        workspace.numel() * workspace.element_size(), _stream(stream)), "grpo_loss_bwd_dlogp")


def loss_bwd_dlogp_e4m3(problem: Problem, H_pol, s_pol, W, s_W, ids, mask, dlogp, lse_pol, grad_loss: float, dH,
                        workspace: torch.Tensor, stream=None, dW=None) -> None:
    N, Nd, Vd = problem.N, problem.N * problem.d, problem.V * problem.d
    _check(lib().grpo_loss_bwd_dlogp_e4m3(
        ctypes.byref(problem), _codes(H_pol, "H_pol", Nd), _ptr(s_pol, "s_pol", torch.float32, N),
        _codes(W, "W", Vd), _ptr(s_W, "s_W", torch.float32, problem.V), _ptr(ids, "ids", torch.int32, N),
        _ptr(mask, "mask", torch.uint8, N), _ptr(dlogp, "dlogp", torch.float32, N),
        _ptr(lse_pol, "lse_pol", torch.float32, N), float(grad_loss), _ptr(dH, "dH", torch.bfloat16, Nd),
        _ptr(dW, "dW", torch.float32, Vd), _ptr(workspace, "workspace"),
        workspace.numel() * workspace.element_size(), _stream(stream)), "grpo_loss_bwd_dlogp_e4m3")


def residual_norm_workspace_size(problem: ResidualNormProblem) -> int:
    """Bytes of grpo_residual_norm_bwd's workspace on the current device."""
    b = ctypes.c_size_t(0)
    _check(lib().grpo_residual_norm_workspace_size(ctypes.byref(problem), ctypes.byref(b)),
           "grpo_residual_norm_workspace_size")
    return b.value


def _gate_ptr(gate, rows: int, d: int, device):
    """(pointer, row stride, rows that share a gate's row, type) of an optional gate."""
    if gate is None:
        return None, 0, 0, GRPO_F32
    if gate.dim() != 2:
        raise ValueError("gate must be 2-D")
    n = gate.shape[0]
    if n < 1 and rows > 0 or n > 0 and rows % n != 0:
        raise ValueError("gate must have a number of rows that divides %d, got %d" % (rows, n))
    code = _plain_code(gate.dtype, "gate")
    gp, ld = _rows_ptr(gate, "gate", gate.dtype, n, d, device)
    return gp, ld, rows // n if n else 1, code


def residual_norm_fwd(x: torch.Tensor, residual: torch.Tensor, weight: torch.Tensor, bias=None, post_weight=None,
                      post_bias=None, gate=None, scale: float = 1.0, eps: float = 1e-5, rms: bool = False, h=None,
                      y=None, mean=None, rstd=None, post_mean=None, post_rstd=None, stream=None):
    """h = residual + scale * gate * post_norm(x) and y = norm(h) over the rows of ``x``
    and ``residual`` (float32 or bf16 [rows, d], rows may be strided): (h, y, mean, rstd,
    post_mean, post_rstd). Without ``post_weight`` x is taken as it is, and the post_*
    statistics are None; the means are with ``rms``. ``gate`` (float32 or bf16, rows may be
    strided) has one row, or one for every row or for as many rows as divide them; the
    parameters are float32 or bf16 [d], of one type. Outputs that are not given belong to
    ``stream``."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return residual_norm_fwd(x, residual, weight, bias, post_weight, post_bias, gate, scale, eps, rms, h, y,
                                     mean, rstd, post_mean, post_rstd)
    if x.dim() != 2:
        raise ValueError("x must be 2-D")
    rows, d = x.shape
    f32, dt, pt, post = torch.float32, x.dtype, weight.dtype, post_weight is not None
    code, pcode = _plain_code(dt, "x"), _plain_code(pt, "weight")
    dev = _device_of(x, "x")
    xp, ld_x = _rows_ptr(x, "x", dt, rows, d, dev)
    sp, ld_res = _rows_ptr(residual, "residual", dt, rows, d, dev)
    gp, ld_gate, gate_rows, gcode = _gate_ptr(gate, rows, d, dev)
    given = h, y, None if rms else mean, rstd, post_mean if post and not rms else None, post_rstd if post else None
    h, hp, ld_h = _rows_out(h, "h", dt, rows, d, dev)
    y, yp, ld_y = _rows_out(y, "y", dt, rows, d, dev)
    layer = not rms
    (mean, mp), (rstd, rp), (post_mean, pmp), (post_rstd, prp) = _vec_outs(
        ((mean if layer else None, "mean", layer), (rstd, "rstd", True),
         (post_mean if layer and post else None, "post_mean", layer and post),
         (post_rstd if post else None, "post_rstd", post)), rows, dev)
    problem = ResidualNormProblem(rows, d, ld_x, ld_res, ld_h, ld_y, ld_gate, 0, 0, 0, 0, 0, gate_rows, eps, scale,
                                  1 if rms else 0, code, pcode, gcode)
    _call(lib().grpo_residual_norm_fwd, "grpo_residual_norm_fwd", dev, None, problem, xp, sp,
          _vec_ptr(weight, "weight", pt, d, dev), _vec_ptr(bias, "bias", pt, d, dev),
          _vec_ptr(post_weight, "post_weight", pt, d, dev), _vec_ptr(post_bias, "post_bias", pt, d, dev), gp, hp, yp,
          mp, rp, pmp, prp)
    _written(given)
    return h, y, mean, rstd, post_mean, post_rstd


def residual_norm_bwd(dy: torch.Tensor, dh, h: torch.Tensor, weight: torch.Tensor, mean, rstd, x=None,
                      post_weight=None, post_bias=None, post_mean=None, post_rstd=None, gate=None, scale: float = 1.0,
                      rms: bool = False, bias: bool = True, dx=None, dresidual=None, dweight=None, dbias=None,
                      dpost_weight=None, dpost_bias=None, dgate=None, need_params: bool = True,
                      need_dgate: bool = True, workspace=None, stream=None):
    """Gradients of ``residual_norm_fwd`` from its inputs, statistics and h, from ``dy``
    and ``dh`` (None: zero): (dx, dresidual, dweight, dbias, dpost_weight, dpost_bias,
    dgate). dx and dresidual have h's type; where there is neither a gate nor a post norm
    and ``scale`` is 1, dx is dresidual, the same tensor unless one is given. The column
    sums are float32 [d]: None without ``need_params``, dbias also without ``bias`` or with
    ``rms``, dpost_bias without ``post_bias``. dgate is float32 of the gate's shape, or of
    its type where the gate has a row for every row (a single row's gate too). ``x`` is needed for a gate or a post norm. Outputs and a workspace that
    are not given belong to ``stream``."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return residual_norm_bwd(dy, dh, h, weight, mean, rstd, x, post_weight, post_bias, post_mean, post_rstd,
                                     gate, scale, rms, bias, dx, dresidual, dweight, dbias, dpost_weight, dpost_bias,
                                     dgate, need_params, need_dgate, workspace)
    if h.dim() != 2:
        raise ValueError("h must be 2-D")
    rows, d = h.shape
    f32, dt, pt, post = torch.float32, h.dtype, weight.dtype, post_weight is not None
    code, pcode = _plain_code(dt, "h"), _plain_code(pt, "weight")
    dev = _device_of(h, "h")
    if mean is None and not rms:
        raise ValueError("mean is needed unless rms")
    if post and (post_rstd is None or (post_mean is None and not rms)):
        raise ValueError("the post norm's statistics are needed")
    inner = post or gate is not None
    if inner and x is None:
        raise ValueError("x is needed with a gate or a post norm")
    yp, ld_dy = _rows_ptr(dy, "dy", dt, rows, d, dev)
    zp, ld_dh = (None, 0) if dh is None else _rows_ptr(dh, "dh", dt, rows, d, dev)
    hp, ld_h = _rows_ptr(h, "h", dt, rows, d, dev)
    xp, ld_x = _rows_ptr(x, "x", dt, rows, d, dev) if inner else (None, 0)
    gp, ld_gate, gate_rows, gcode = _gate_ptr(gate, rows, d, dev)
    given = dx, dresidual, dweight, dbias, dpost_weight, dpost_bias, dgate
    dresidual, sp, ld_s = _rows_out(dresidual, "dresidual", dt, rows, d, dev)
    dxp, ld_dx, same = None, 0, not inner and scale == 1.0 and dx is None
    if not same:
        dx, dxp, ld_dx = _rows_out(dx, "dx", dt, rows, d, dev)
    (dweight, wp), (dbias, bp), (dpost_weight, pwp), (dpost_bias, pbp) = _vec_outs(
        ((dweight, "dweight", need_params), (dbias, "dbias", need_params and bias and not rms),
         (dpost_weight, "dpost_weight", need_params and post),
         (dpost_bias, "dpost_bias", need_params and post_bias is not None)), d, dev)
    dgp, ld_dg = None, 0
    if dgate is not None or (gate is not None and need_dgate):
        if gate is None:
            raise ValueError("dgate needs a gate")
        n = gate.shape[0]
        if gate_rows == 1:
            dgate, dgp, ld_dg = _rows_out(dgate, "dgate", gate.dtype, n, d, dev)
        else:
            if dgate is None:
                dgate = torch.empty(n, d, dtype=f32, device=dev)
            dgp = _vec_ptr(dgate, "dgate", f32, n * d, dev)
        if rows == 0:       # sums of none (the library cannot tell how many rows the gate has)
            dgate.zero_()
    problem = ResidualNormProblem(rows, d, ld_x, 0, ld_h, 0, ld_gate, ld_dy, ld_dh, ld_dx, ld_s, ld_dg, gate_rows, 0.0,
                                  scale, 1 if rms else 0, code, pcode, gcode)
    L = lib()
    wsp, size = None, 0
    if wp or bp or pwp or pbp or (dgp and gate_rows > 1):
        if workspace is None:
            size = _bytes(("residual_norm", rows, d, rms, gate_rows > 1), L.grpo_residual_norm_workspace_size,
                          "grpo_residual_norm_workspace_size", dev, problem)
        workspace, wsp, size = _workspace(workspace, size, dev)
    _call(L.grpo_residual_norm_bwd, "grpo_residual_norm_bwd", dev, None, problem, yp, zp, hp,
          _vec_ptr(weight, "weight", pt, d, dev), None if rms else _vec_ptr(mean, "mean", f32, rows, dev),
          _vec_ptr(rstd, "rstd", f32, rows, dev), xp, _vec_ptr(post_weight, "post_weight", pt, d, dev),
          _vec_ptr(post_bias, "post_bias", pt, d, dev),
          _vec_ptr(post_mean, "post_mean", f32, rows, dev) if post and not rms else None,
          _vec_ptr(post_rstd, "post_rstd", f32, rows, dev) if post else None, gp, dxp, sp, wp, bp, pwp, pbp, dgp, wsp,
          size)
    _written(given)
    return dresidual if same else dx, dresidual, dweight, dbias, dpost_weight, dpost_bias, dgate


_PLAIN = {torch.float32: GRPO_F32, torch.bfloat16: GRPO_BF16}
_NORM_TYPES = {2: 2, float("inf"): 0}
_TENSOR = torch.Tensor
_DTYPE_OF, _SHAPE_OF = operator.attrgetter("dtype"), operator.attrgetter("shape")
_GRAD_PACKS = {}


def _refuse_grads(grads, out, name: str) -> None:
    """The error of a list that is not contiguous float32 or bf16 CUDA tensors of one device,
    or of an ``out`` that is not alike."""
    for i, t in enumerate(grads):
        if not torch.is_tensor(t):
            raise ValueError("%s[%d] must be a tensor, got %r" % (name, i, type(t)))
        _plain_code(t.dtype, "%s[%d]" % (name, i))
        _device_of(t, "%s[%d]" % (name, i))
        _vec_ptr(t, "%s[%d]" % (name, i), t.dtype, t.numel(), grads[0].device)
    for i, (t, g) in enumerate(zip(out or (), grads)):
        if not torch.is_tensor(t) or t.dtype != g.dtype or t.shape != g.shape or t.device != g.device or \
                not t.is_contiguous():
            raise ValueError("out[%d] must be contiguous, of %s[%d]'s shape %s and type %s, on %s" % (
                i, name, i, tuple(g.shape), g.dtype, g.device))


def _grad_table(grads, out, name: str):
    """(an array of GradTensor, sizes, gradients' and outs' addresses, types, device)."""
    n = len(grads)
    if out is not None and len(out) != n:
        raise ValueError("expected %d tensors in out, got %d" % (n, len(out)))
    if not n:
        return b"", [], [], [], [], None
    try:
        at, types = grads[0].get_device(), list(map(_DTYPE_OF, grads))
        codes = list(map(_PLAIN.__getitem__, types))
        good = at >= 0 and all(map(_TENSOR.is_contiguous, grads)) and \
            not any(map(at.__ne__, map(_TENSOR.get_device, grads)))
        if out is not None:
            good = good and list(map(_DTYPE_OF, out)) == types and list(map(_SHAPE_OF, out)) == \
                list(map(_SHAPE_OF, grads)) and all(map(_TENSOR.is_contiguous, out)) and \
                not any(map(at.__ne__, map(_TENSOR.get_device, out)))
    except (AttributeError, TypeError, KeyError):       # not tensors, or of other types
        good = False
    if not good:
        _refuse_grads(grads, out, name)
    sizes, places = list(map(_TENSOR.numel, grads)), list(map(_TENSOR.data_ptr, grads))
    outs = places if out is None else list(map(_TENSOR.data_ptr, out))
    pack = _GRAD_PACKS.get(n)
    if pack is None:
        pack = _GRAD_PACKS[n] = struct.Struct("@" + "qQQi4x" * n)
    flat = [0] * (4 * n)
    flat[0::4], flat[1::4], flat[2::4], flat[3::4] = sizes, places, outs, codes
    return pack.pack(*flat), sizes, places, outs, codes, grads[0].device


def _no_overlap(sizes, places, outs, codes) -> None:
    """A clipped tensor is written: no other may share its bytes (two gradients that are only
    read may share theirs)."""
    ends = [o + (n << 2 if c == GRPO_F32 else n << 1) for n, o, c in zip(sizes, outs, codes)]
    starts, read = outs, []
    if outs is not places:
        read = [(p, p + e - o) for p, o, e in zip(places, outs, ends) if p != o]
        starts, ends = starts + [p for p, _ in read], ends + [e for _, e in read]
    # (spans are apart where, in order, each begins behind the end before; one of no bytes
    # may lie anywhere, and only seem not to)
    if not any(map(operator.lt, sorted(starts)[1:], sorted(ends))):
        return
    spans = sorted([(o, o + (n << 2 if c == GRPO_F32 else n << 1), True, i)
                    for i, (n, o, c) in enumerate(zip(sizes, outs, codes)) if n] +
                   [(p, e, False, -1) for p, e in read if e > p])
    last = last_written = 0
    for start, end, written, i in spans:
        if start < last and (written or start < last_written):
            raise ValueError("the gradients or out overlap%s: what is written is one tensor's own" %
                             (" at number %d" % i if written else ""))
        last = max(last, end)
        if written:
            last_written = max(last_written, end)


def _grad_call(grads, clip: bool, max_norm, norm_type, eps, out, norm, factor, workspace):
    grads = list(grads)
    if norm_type not in _NORM_TYPES:
        raise ValueError("norm_type must be 2 or inf, got %r" % (norm_type,))
    if max_norm is not None and not max_norm >= 0.0:
        raise ValueError("max_norm must not be negative, got %r" % (max_norm,))
    table, sizes, places, outs, codes, dev = _grad_table(grads, out, "grads")
    if dev is None:
        given, which = (norm, "norm") if norm is not None else (factor, "factor")
        dev = _device_of(given, which) if given is not None else torch.device("cuda", torch.cuda.current_device())
    given = norm, factor
    norm, at_norm = _vec_out(norm, "norm", torch.float32, 1, dev)
    at_factor = None
    if clip or factor is not None or max_norm is not None:
        factor, at_factor = _vec_out(factor, "factor", torch.float32, 1, dev)
    if clip:
        _no_overlap(sizes, places, outs, codes)
    L, size, n = lib(), 0, len(sizes)
    # (one launch takes a short list, with no workspace)
    if workspace is None and not (0 < n <= 8 and sum(sizes) <= 65536 and all(sizes)):
        size = _bytes("grad_norm", L.grpo_grad_norm_workspace_size, "grpo_grad_norm_workspace_size", dev)
    workspace, wp, size = _workspace(workspace, size, dev)
    name = "grpo_clip_grad_norm" if clip else "grpo_grad_norm"
    _call(L.grpo_clip_grad_norm if clip else L.grpo_grad_norm, name, dev, None, table, n, _NORM_TYPES[norm_type],
          math.inf if max_norm is None else max_norm, eps, at_norm, at_factor, wp, size)
    _written(given, (grads if out is None else out) if clip else ())
    return norm, factor


def grad_norm(grads, norm_type: float = 2.0, max_norm: Optional[float] = None, eps: float = 1e-6, norm=None,
              factor=None, workspace=None, stream=None):
    """The norm (float32 [1]) of ``grads`` (contiguous float32 or bf16 CUDA tensors) taken
    as one vector, ``norm_type`` 2 or inf; see grpo_grad_norm. With ``max_norm``, (norm,
    factor): factor = min(1, max_norm / (norm + eps)) stays on the device, where
    ``AdamW.step(factor=...)`` takes it. Outputs and a workspace that are not given belong
    to ``stream``."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return grad_norm(grads, norm_type, max_norm, eps, norm, factor, workspace)
    norm, factor = _grad_call(grads, False, max_norm, norm_type, eps, None, norm, factor, workspace)
    return norm if max_norm is None else (norm, factor)


def clip_grad_norm(grads, max_norm: float, norm_type: float = 2.0, eps: float = 1e-6, out=None, norm=None, factor=None,
                   workspace=None, stream=None):
    """Scales ``grads`` by min(1, max_norm / (norm + eps)), in place or into the tensors of
    ``out`` (of the same shapes and types), and returns their norm before that (float32
    [1]). Tensors that overlap are refused. Outputs and a workspace that are not given
    belong to ``stream``."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return clip_grad_norm(grads, max_norm, norm_type, eps, out, norm, factor, workspace)
    return _grad_call(grads, True, max_norm, norm_type, eps, None if out is None else list(out), norm, factor,
                      workspace)[0]


def device_status(workspace: torch.Tensor, stream=None) -> int:
    """Synchronise and return (and clear) the workspace's device error status."""
    return lib().grpo_get_device_status(_ptr(workspace, "workspace"), _stream(stream))


def profile_enable(on: bool) -> None:
    _check(lib().grpo_profile_enable(1 if on else 0), "grpo_profile_enable")


def profile_collect():
    """{kernel name: (milliseconds, launches)} since the last collect."""
    n = lib().grpo_profile_kind_count()
    ms = (ctypes.c_double * n)()
    cnt = (ctypes.c_int64 * n)()
    _check(lib().grpo_profile_collect(ms, cnt, n), "grpo_profile_collect")
    return {lib().grpo_profile_kind_name(k).decode(): (ms[k], cnt[k]) for k in range(n)}
