"""ctypes binding of the C ABI declared in include/grpo.h.

Argument marshalling only: every step of the loss runs in the library's CUDA
kernels. There is no CPU fallback; if the shared library has not been built
the first call raises.
"""
from __future__ import annotations

import ctypes
import os
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
                ("state_bits", ctypes.c_int32), ("step", ctypes.c_int64)]


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
