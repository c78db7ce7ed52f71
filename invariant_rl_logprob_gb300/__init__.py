"""Batch-invariant selected-token logprob on GB300 (sm_103a).

Thin Python binding over the C-ABI library ``librk.so`` (see ``include/rk.h``).
This module only marshals arguments -- device pointers, sizes and the current
CUDA stream -- and allocates outputs and workspace with PyTorch; every step of
the computation runs in the library's CUDA kernels.  There is no CPU path: if
``librk.so`` is missing or no GPU is present the calls raise.

Operators (RL-Kernel issue #101, maintainer comment, P0 operator list):

* :func:`linear_logp`      -- ``logp[t] = z[t, target_t] - logsumexp_v z[t, v]``, ``z = h W^T``
* :func:`logp_from_logits` -- the same from materialised bf16 logits
* :func:`linear_logp_bwd`  -- ``dh[t] = g[t] (W[target_t] - softmax(z[t]) W)``
* :func:`logits_rules_apply`, :func:`logp_from_logits_rules`,
  :func:`logp_from_logits_rules_bwd` -- logits under sampling rules
  (:class:`LogitsRules`: penalties, biases, grammar masks, temperature), the
  selected logprob under them and its gradient
* :func:`embedding`, :func:`embedding_bwd` -- the scaled token embedding and
  its gradient, summed per token in canonical order

Each is bitwise invariant for a given logical row under changes of batch
size, row position, neighbour content, padding and varlen packing.
"""
from __future__ import annotations

import ctypes
import os

import torch

__all__ = [
    "RkError", "library_path", "load_library",
    "linear_logp", "linear_logp_workspace_size",
    "logp_from_logits",
    "linear_logp_bwd", "linear_logp_bwd_workspace_size", "linear_logp_bwd_min_workspace_size",
    "lm_head", "logp_from_logits_bwd", "grpo_token_loss", "linear_logp_grpo", "linear_greedy",
    "linear_logp_fwd_saved", "linear_logp_bwd_saved", "linear_logp_saved_size",
    "linear_logp_bwd_saved_workspace_size", "linear_logp_bwd_full_saved",
    "linear_greedy_workspace_size", "linear_logp_dw", "linear_logp_dw_workspace_size",
    "linear_logp_bwd_full", "linear_logp_bwd_full_workspace_size", "lm_head_workspace_size",
    "LogitsRules", "logits_rules_apply", "logp_from_logits_rules",
    "logp_from_logits_rules_workspace_size", "logp_from_logits_rules_bwd",
    "embedding", "embedding_bwd", "embedding_bwd_workspace_size",
    "get_device_error", "selftest_wait_timeout", "set_row_blocks", "last_row_blocks", "DEVERR_TARGET_RANGE", "DEVERR_TIMEOUT", "DEVERR_LSE",
    "DEVERR_RULES",
]

_PKG = os.path.dirname(os.path.abspath(__file__))
_LIB_PATH = os.path.join(_PKG, "librk.so")
_lib = None

RK_OK, RK_ERR_INVALID_ARG, RK_ERR_UNSUPPORTED, RK_ERR_WORKSPACE, RK_ERR_CUDA = range(5)
DEVERR_TARGET_RANGE = 0x1
DEVERR_TIMEOUT = 0x2
DEVERR_LSE = 0x4
DEVERR_RULES = 0x8


class RkError(RuntimeError):
    def __init__(self, what: str, status: int, cuda_error: int = 0):
        self.status = status
        self.cuda_error = cuda_error
        name = _lib.rk_status_string(status).decode() if _lib is not None else str(status)
        msg = f"{what} failed: {name}"
        if status == RK_ERR_CUDA:
            msg += f" (cudaError {cuda_error})"
        super().__init__(msg)


def library_path() -> str:
    return _LIB_PATH


def load_library() -> ctypes.CDLL:
    """Load librk.so (built by ``invariant_rl_logprob_gb300.build``); raises if absent."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(_LIB_PATH):
        raise RuntimeError(
            f"{_LIB_PATH} is missing: build it with `python -m invariant_rl_logprob_gb300.build` "
            "(there is no CPU fallback)")
    lib = ctypes.CDLL(_LIB_PATH)
    vp, i64, i32, sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_size_t
    lib.rk_linear_logp_workspace_size.argtypes = [i64, i64, i64]
    lib.rk_linear_logp_workspace_size.restype = sz
    lib.rk_linear_logp.argtypes = [vp, vp, vp, vp, i32, i64, i64, i64, vp, vp, vp, sz, vp]
    lib.rk_linear_logp.restype = ctypes.c_int
    lib.rk_logp_from_logits.argtypes = [vp, vp, vp, i32, i64, i64, vp, vp, vp]
    lib.rk_logp_from_logits.restype = ctypes.c_int
    lib.rk_linear_logp_bwd_workspace_size.argtypes = [i64, i64, i64]
    lib.rk_linear_logp_bwd_workspace_size.restype = sz
    lib.rk_linear_logp_bwd_min_workspace_size.argtypes = [i64, i64]
    lib.rk_linear_logp_bwd_min_workspace_size.restype = sz
    lib.rk_linear_logp_bwd.argtypes = [vp, vp, vp, vp, i32, i64, i64, i64, vp, vp, vp, vp, sz, vp]
    lib.rk_linear_logp_bwd.restype = ctypes.c_int
    lib.rk_lm_head.argtypes = [vp, vp, i64, i64, i64, vp, i64, vp, sz, vp]
    lib.rk_lm_head_workspace_size.argtypes = []
    lib.rk_lm_head_workspace_size.restype = sz
    lib.rk_lm_head.restype = ctypes.c_int
    lib.rk_logp_from_logits_bwd.argtypes = [vp, vp, vp, i32, i64, i64, vp, vp, vp, vp]
    lib.rk_logp_from_logits_bwd.restype = ctypes.c_int
    f32 = ctypes.c_float
    lib.rk_grpo_token_loss.argtypes = [vp, vp, vp, vp, vp, vp, i32, i64, f32, f32, f32, f32,
                                       vp, vp, vp, vp, vp]
    lib.rk_grpo_token_loss.restype = ctypes.c_int
    lib.rk_linear_greedy_workspace_size.argtypes = [i64, i64, i64]
    lib.rk_linear_greedy_workspace_size.restype = sz
    lib.rk_linear_greedy.argtypes = [vp, vp, vp, i32, i64, i64, i64, vp, vp, vp, vp, sz, vp]
    lib.rk_linear_greedy.restype = ctypes.c_int
    lib.rk_linear_logp_dw_workspace_size.argtypes = [i64, i64, i64]
    lib.rk_linear_logp_dw_workspace_size.restype = sz
    lib.rk_linear_logp_dw.argtypes = [vp, vp, vp, vp, i32, i64, i64, i64, vp, vp, vp, i64, vp, vp,
                                      sz, vp]
    lib.rk_linear_logp_dw.restype = ctypes.c_int
    lib.rk_linear_logp_bwd_full_workspace_size.argtypes = [i64, i64, i64]
    lib.rk_linear_logp_bwd_full_workspace_size.restype = sz
    lib.rk_linear_logp_bwd_full.argtypes = [vp, vp, vp, vp, i32, i64, i64, i64, vp, vp, vp, i64,
                                            vp, vp, vp, sz, vp]
    lib.rk_linear_logp_bwd_full.restype = ctypes.c_int
    lib.rk_selftest_wait_timeout.argtypes = [i64, vp]
    lib.rk_selftest_wait_timeout.restype = ctypes.c_int
    lib.rk_get_device_error.argtypes = [vp, ctypes.POINTER(i32)]
    lib.rk_get_device_error.restype = ctypes.c_int
    lib.rk_status_string.argtypes = [ctypes.c_int]
    lib.rk_status_string.restype = ctypes.c_char_p
    lib.rk_last_cuda_error.argtypes = []
    lib.rk_last_cuda_error.restype = ctypes.c_int
    lib.rk_version.argtypes = []
    lib.rk_version.restype = ctypes.c_char_p
    f32 = ctypes.c_float
    lib.rk_linear_logp_grpo.argtypes = [vp, vp, vp, vp, i32, i64, i64, i64, vp, vp, vp, f32, f32,
                                        f32, f32, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    lib.rk_linear_logp_grpo.restype = ctypes.c_int
    lib.rk_linear_logp_saved_size.argtypes = [i64, i64, i64]
    lib.rk_linear_logp_saved_size.restype = sz
    lib.rk_linear_logp_fwd_saved.argtypes = [vp, vp, vp, vp, i32, i64, i64, i64, vp, vp, vp, sz, vp]
    lib.rk_linear_logp_fwd_saved.restype = ctypes.c_int
    lib.rk_linear_logp_bwd_saved_workspace_size.argtypes = [i64, i64, i64]
    lib.rk_linear_logp_bwd_saved_workspace_size.restype = sz
    lib.rk_linear_logp_bwd_saved.argtypes = [vp, vp, vp, vp, i32, i64, i64, i64, vp, vp, vp, sz, vp,
                                             vp, sz, vp]
    lib.rk_linear_logp_bwd_saved.restype = ctypes.c_int
    lib.rk_linear_logp_bwd_full_saved.argtypes = [vp, vp, vp, vp, i32, i64, i64, i64, vp, vp, vp,
                                                  sz, vp, i64, vp, vp, vp, sz, vp]
    lib.rk_linear_logp_bwd_full_saved.restype = ctypes.c_int
    lib.rk_set_row_blocks.argtypes = [i32]
    lib.rk_set_row_blocks.restype = ctypes.c_int
    lib.rk_last_row_blocks.argtypes = [i32]
    lib.rk_last_row_blocks.restype = i32
    lib.rk_last_tile_order.argtypes = [i32]
    lib.rk_last_tile_order.restype = i32
    rp = ctypes.c_void_p  # a _RulesStruct, passed by address
    lib.rk_logits_rules_apply.argtypes = [vp, i32, i64, rp, i64, i64, vp, i32, i64, vp]
    lib.rk_logits_rules_apply.restype = ctypes.c_int
    lib.rk_logp_from_logits_rules_workspace_size.argtypes = [i64, i64]
    lib.rk_logp_from_logits_rules_workspace_size.restype = sz
    lib.rk_logp_from_logits_rules.argtypes = [vp, i32, i64, vp, vp, i32, rp, i64, i64, vp, vp, vp, sz,
                                              vp]
    lib.rk_logp_from_logits_rules.restype = ctypes.c_int
    lib.rk_logp_from_logits_rules_lse64.argtypes = lib.rk_logp_from_logits_rules.argtypes
    lib.rk_logp_from_logits_rules_lse64.restype = ctypes.c_int
    lib.rk_logp_from_logits_rules_bwd.argtypes = [vp, i32, i64, vp, vp, i32, rp, i64, i64, vp, vp, vp,
                                                  i32, i64, vp]
    lib.rk_logp_from_logits_rules_bwd.restype = ctypes.c_int
    lib.rk_logp_from_logits_rules_bwd_lse64.argtypes = lib.rk_logp_from_logits_rules_bwd.argtypes
    lib.rk_logp_from_logits_rules_bwd_lse64.restype = ctypes.c_int
    lib.rk_embedding.argtypes = [vp, vp, i32, vp, i32, i64, i64, i64, f32, vp, i32, vp]
    lib.rk_embedding.restype = ctypes.c_int
    lib.rk_embedding_bwd_workspace_size.argtypes = [i64, i64, i64]
    lib.rk_embedding_bwd_workspace_size.restype = sz
    lib.rk_embedding_bwd.argtypes = [vp, i32, vp, vp, i32, i64, i64, i64, f32, vp, i64, vp, i32, vp,
                                     sz, vp]
    lib.rk_embedding_bwd.restype = ctypes.c_int
    _lib = lib
    return lib


def _check(status: int, what: str) -> None:
    if status != RK_OK:
        raise RkError(what, status, _lib.rk_last_cuda_error() if status == RK_ERR_CUDA else 0)


def _ptr(t: torch.Tensor | None):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream_handle(stream, device) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream(device)
    return ctypes.c_void_p(stream.cuda_stream)


def _need(t: torch.Tensor, name: str, dtype: torch.dtype, ndim: int) -> None:
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device.type != "cuda":
        raise ValueError(f"{name} must be a CUDA tensor (no CPU path), got {t.device}")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dims, got shape {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _rows(targets, cu_seqlens, T, device, name="targets"):
    _need(targets, name, torch.int64, 1)
    if targets.shape[0] != T or targets.device != device:
        raise ValueError(f"{name} must be [T] on the same device")
    if cu_seqlens is None:
        return None, 0
    _need(cu_seqlens, "cu_seqlens", torch.int32, 1)
    if cu_seqlens.device != device or cu_seqlens.numel() < 1:
        raise ValueError("cu_seqlens must be a non-empty int32 tensor on the same device")
    return cu_seqlens, cu_seqlens.numel() - 1


def linear_logp_workspace_size(T: int, H: int, V: int) -> int:
    return int(load_library().rk_linear_logp_workspace_size(T, H, V))


def linear_logp(h: torch.Tensor, W: torch.Tensor, targets: torch.Tensor,
                cu_seqlens: torch.Tensor | None = None, *, out: torch.Tensor | None = None,
                lse: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                stream: torch.cuda.Stream | None = None):
    """Selected-token logprob of ``h W^T``: returns ``(logp, lse)``, fp32 ``[T]``."""
    lib = load_library()
    _need(h, "h", torch.bfloat16, 2)
    _need(W, "W", torch.bfloat16, 2)
    T, H = h.shape
    V = W.shape[0]
    if W.shape[1] != H or W.device != h.device:
        raise ValueError("W must be [V, H] on h's device")
    cu, ns = _rows(targets, cu_seqlens, T, h.device)
    if out is None:
        out = torch.empty(T, dtype=torch.float32, device=h.device)
    if lse is None:
        lse = torch.empty(T, dtype=torch.float32, device=h.device)
    need = int(lib.rk_linear_logp_workspace_size(T, H, V))
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=h.device)
    st = lib.rk_linear_logp(_ptr(h), _ptr(W), _ptr(targets), _ptr(cu), ns, T, H, V,
                            _ptr(out), _ptr(lse), _ptr(workspace), workspace.numel(),
                            _stream_handle(stream, h.device))
    _check(st, "rk_linear_logp")
    return out, lse


def logp_from_logits(logits: torch.Tensor, targets: torch.Tensor,
                     cu_seqlens: torch.Tensor | None = None, *, out: torch.Tensor | None = None,
                     lse: torch.Tensor | None = None, stream: torch.cuda.Stream | None = None):
    """Selected-token logprob from bf16 logits ``[T, V]``: returns ``(logp, lse)``."""
    lib = load_library()
    _need(logits, "logits", torch.bfloat16, 2)
    T, V = logits.shape
    cu, ns = _rows(targets, cu_seqlens, T, logits.device)
    if out is None:
        out = torch.empty(T, dtype=torch.float32, device=logits.device)
    if lse is None:
        lse = torch.empty(T, dtype=torch.float32, device=logits.device)
    st = lib.rk_logp_from_logits(_ptr(logits), _ptr(targets), _ptr(cu), ns, T, V, _ptr(out),
                                 _ptr(lse), _stream_handle(stream, logits.device))
    _check(st, "rk_logp_from_logits")
    return out, lse


def linear_logp_bwd_workspace_size(T: int, H: int, V: int) -> int:
    return int(load_library().rk_linear_logp_bwd_workspace_size(T, H, V))


def linear_logp_bwd_min_workspace_size(H: int, V: int) -> int:
    return int(load_library().rk_linear_logp_bwd_min_workspace_size(H, V))


def linear_logp_bwd(h: torch.Tensor, W: torch.Tensor, targets: torch.Tensor, lse: torch.Tensor,
                    grad_logp: torch.Tensor, cu_seqlens: torch.Tensor | None = None, *,
                    dh: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                    stream: torch.cuda.Stream | None = None) -> torch.Tensor:
    """dh = g (W[target] - softmax(h W^T) W) in fp32 ``[T, H]``."""
    lib = load_library()
    _need(h, "h", torch.bfloat16, 2)
    _need(W, "W", torch.bfloat16, 2)
    T, H = h.shape
    V = W.shape[0]
    if W.shape[1] != H or W.device != h.device:
        raise ValueError("W must be [V, H] on h's device")
    cu, ns = _rows(targets, cu_seqlens, T, h.device)
    _need(lse, "lse", torch.float32, 1)
    _need(grad_logp, "grad_logp", torch.float32, 1)
    if dh is None:
        dh = torch.empty((T, H), dtype=torch.float32, device=h.device)
    if workspace is None:
        need = int(lib.rk_linear_logp_bwd_workspace_size(T, H, V))
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=h.device)
    st = lib.rk_linear_logp_bwd(_ptr(h), _ptr(W), _ptr(targets), _ptr(cu), ns, T, H, V,
                                _ptr(lse), _ptr(grad_logp), _ptr(dh), _ptr(workspace),
                                workspace.numel(), _stream_handle(stream, h.device))
    _check(st, "rk_linear_logp_bwd")
    return dh


def lm_head_workspace_size() -> int:
    return int(load_library().rk_lm_head_workspace_size())


def lm_head(h: torch.Tensor, W: torch.Tensor, *, out: torch.Tensor | None = None,
            workspace: torch.Tensor | None = None,
            stream: torch.cuda.Stream | None = None) -> torch.Tensor:
    """Dense path: bf16 logits ``[T, V]`` = bf16(h W^T) (fp32 accumulation).

    ``workspace`` (uint8, >= ``rk_lm_head_workspace_size()`` bytes) holds the
    tile counter; one is allocated when it is None."""
    lib = load_library()
    _need(h, "h", torch.bfloat16, 2)
    _need(W, "W", torch.bfloat16, 2)
    T, H = h.shape
    V = W.shape[0]
    if W.shape[1] != H or W.device != h.device:
        raise ValueError("W must be [V, H] on h's device")
    ld = (V + 7) // 8 * 8
    if out is None:
        buf = torch.empty((T, ld), dtype=torch.bfloat16, device=h.device)
        out = buf[:, :V]
    else:
        if out.dtype != torch.bfloat16 or out.dim() != 2 or out.stride(1) != 1:
            raise ValueError("out must be a bf16 [T, V] view with unit column stride")
        ld = out.stride(0)
    if workspace is None:
        workspace = torch.empty(int(lib.rk_lm_head_workspace_size()), dtype=torch.uint8,
                                device=h.device)
    st = lib.rk_lm_head(_ptr(h), _ptr(W), T, H, V, _ptr(out), ld, _ptr(workspace),
                        workspace.numel(), _stream_handle(stream, h.device))
    _check(st, "rk_lm_head")
    return out


def logp_from_logits_bwd(logits: torch.Tensor, targets: torch.Tensor, lse: torch.Tensor,
                         grad_logp: torch.Tensor, cu_seqlens: torch.Tensor | None = None, *,
                         out: torch.Tensor | None = None,
                         stream: torch.cuda.Stream | None = None) -> torch.Tensor:
    """dlogits = g (onehot - softmax(logits)) in fp32 ``[T, V]``."""
    lib = load_library()
    _need(logits, "logits", torch.bfloat16, 2)
    T, V = logits.shape
    cu, ns = _rows(targets, cu_seqlens, T, logits.device)
    _need(lse, "lse", torch.float32, 1)
    _need(grad_logp, "grad_logp", torch.float32, 1)
    if out is None:
        out = torch.empty((T, V), dtype=torch.float32, device=logits.device)
    st = lib.rk_logp_from_logits_bwd(_ptr(logits), _ptr(targets), _ptr(cu), ns, T, V, _ptr(lse),
                                     _ptr(grad_logp), _ptr(out),
                                     _stream_handle(stream, logits.device))
    _check(st, "rk_logp_from_logits_bwd")
    return out


def grpo_token_loss(logp: torch.Tensor, logp_old: torch.Tensor, advantages: torch.Tensor,
                    targets: torch.Tensor, cu_seqlens: torch.Tensor | None = None, *,
                    logp_ref: torch.Tensor | None = None, eps_low: float = 0.2,
                    eps_high: float = 0.2, beta: float = 0.0, scale: float = 1.0,
                    stream: torch.cuda.Stream | None = None) -> dict:
    """Per-token GRPO loss: dict with fp32 ``loss``, ``grad`` (d loss/d logp),
    ``ratio`` and ``kl``, each ``[T]``."""
    lib = load_library()
    for name, t in (("logp", logp), ("logp_old", logp_old), ("advantages", advantages)):
        _need(t, name, torch.float32, 1)
    T = logp.shape[0]
    if logp_ref is not None:
        _need(logp_ref, "logp_ref", torch.float32, 1)
    cu, ns = _rows(targets, cu_seqlens, T, logp.device)
    out = {k: torch.empty(T, dtype=torch.float32, device=logp.device)
           for k in ("loss", "grad", "ratio", "kl")}
    st = lib.rk_grpo_token_loss(_ptr(logp), _ptr(logp_old), _ptr(logp_ref), _ptr(advantages),
                                _ptr(targets), _ptr(cu), ns, T, eps_low, eps_high, beta, scale,
                                _ptr(out["loss"]), _ptr(out["grad"]), _ptr(out["ratio"]),
                                _ptr(out["kl"]), _stream_handle(stream, logp.device))
    _check(st, "rk_grpo_token_loss")
    return out


def linear_logp_grpo(h: torch.Tensor, W: torch.Tensor, targets: torch.Tensor,
                     logp_old: torch.Tensor, advantages: torch.Tensor,
                     cu_seqlens: torch.Tensor | None = None, *,
                     logp_ref: torch.Tensor | None = None, eps_low: float = 0.2,
                     eps_high: float = 0.2, beta: float = 0.0, scale: float = 1.0,
                     workspace: torch.Tensor | None = None,
                     stream: torch.cuda.Stream | None = None) -> dict:
    """linear_logp with the per-token GRPO loss applied in its merge: dict of
    fp32 ``[T]`` tensors ``logp``, ``lse``, ``loss``, ``grad``, ``ratio``,
    ``kl`` (the same bits as linear_logp followed by grpo_token_loss)."""
    lib = load_library()
    _need(h, "h", torch.bfloat16, 2)
    _need(W, "W", torch.bfloat16, 2)
    T, H = h.shape
    V = W.shape[0]
    if W.shape[1] != H or W.device != h.device:
        raise ValueError("W must be [V, H] on h's device")
    for name, t in (("logp_old", logp_old), ("advantages", advantages)):
        _need(t, name, torch.float32, 1)
    if logp_ref is not None:
        _need(logp_ref, "logp_ref", torch.float32, 1)
    cu, ns = _rows(targets, cu_seqlens, T, h.device)
    out = {k: torch.empty(T, dtype=torch.float32, device=h.device)
           for k in ("logp", "lse", "loss", "grad", "ratio", "kl")}
    need = int(lib.rk_linear_logp_workspace_size(T, H, V))
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=h.device)
    st = lib.rk_linear_logp_grpo(_ptr(h), _ptr(W), _ptr(targets), _ptr(cu), ns, T, H, V,
                                 _ptr(logp_old), _ptr(logp_ref), _ptr(advantages), eps_low,
                                 eps_high, beta, scale, _ptr(out["logp"]), _ptr(out["lse"]),
                                 _ptr(out["loss"]), _ptr(out["grad"]), _ptr(out["ratio"]),
                                 _ptr(out["kl"]), _ptr(workspace), workspace.numel(),
                                 _stream_handle(stream, h.device))
    _check(st, "rk_linear_logp_grpo")
    return out


def linear_logp_saved_size(T: int, H: int, V: int) -> int:
    return int(load_library().rk_linear_logp_saved_size(T, H, V))


def linear_logp_bwd_saved_workspace_size(T: int, H: int, V: int) -> int:
    return int(load_library().rk_linear_logp_bwd_saved_workspace_size(T, H, V))


def linear_logp_fwd_saved(h: torch.Tensor, W: torch.Tensor, targets: torch.Tensor,
                          cu_seqlens: torch.Tensor | None = None, *,
                          out: torch.Tensor | None = None, lse: torch.Tensor | None = None,
                          saved: torch.Tensor | None = None,
                          stream: torch.cuda.Stream | None = None):
    """linear_logp that also keeps its softmax terms for
    :func:`linear_logp_bwd_saved`: returns ``(logp, lse, saved)``."""
    lib = load_library()
    _need(h, "h", torch.bfloat16, 2)
    _need(W, "W", torch.bfloat16, 2)
    T, H = h.shape
    V = W.shape[0]
    if W.shape[1] != H or W.device != h.device:
        raise ValueError("W must be [V, H] on h's device")
    cu, ns = _rows(targets, cu_seqlens, T, h.device)
    if out is None:
        out = torch.empty(T, dtype=torch.float32, device=h.device)
    if lse is None:
        lse = torch.empty(T, dtype=torch.float32, device=h.device)
    if saved is None:
        saved = torch.empty(max(int(lib.rk_linear_logp_saved_size(T, H, V)), 1), dtype=torch.uint8,
                            device=h.device)
    st = lib.rk_linear_logp_fwd_saved(_ptr(h), _ptr(W), _ptr(targets), _ptr(cu), ns, T, H, V,
                                      _ptr(out), _ptr(lse), _ptr(saved), saved.numel(),
                                      _stream_handle(stream, h.device))
    _check(st, "rk_linear_logp_fwd_saved")
    return out, lse, saved


def linear_logp_bwd_saved(h: torch.Tensor, W: torch.Tensor, targets: torch.Tensor,
                          lse: torch.Tensor, grad_logp: torch.Tensor, saved: torch.Tensor,
                          cu_seqlens: torch.Tensor | None = None, *,
                          dh: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                          stream: torch.cuda.Stream | None = None) -> torch.Tensor:
    """dh fp32 ``[T, H]`` from the state :func:`linear_logp_fwd_saved` kept
    (which this call consumes)."""
    lib = load_library()
    _need(h, "h", torch.bfloat16, 2)
    _need(W, "W", torch.bfloat16, 2)
    _need(lse, "lse", torch.float32, 1)
    _need(grad_logp, "grad_logp", torch.float32, 1)
    T, H = h.shape
    V = W.shape[0]
    cu, ns = _rows(targets, cu_seqlens, T, h.device)
    if dh is None:
        dh = torch.empty((T, H), dtype=torch.float32, device=h.device)
    if workspace is None:
        need = int(lib.rk_linear_logp_bwd_saved_workspace_size(T, H, V))
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=h.device)
    st = lib.rk_linear_logp_bwd_saved(_ptr(h), _ptr(W), _ptr(targets), _ptr(cu), ns, T, H, V,
                                      _ptr(lse), _ptr(grad_logp), _ptr(saved), saved.numel(),
                                      _ptr(dh), _ptr(workspace), workspace.numel(),
                                      _stream_handle(stream, h.device))
    _check(st, "rk_linear_logp_bwd_saved")
    return dh


def linear_logp_bwd_full_saved(h: torch.Tensor, W: torch.Tensor, targets: torch.Tensor,
                               lse: torch.Tensor, grad_logp: torch.Tensor, saved: torch.Tensor,
                               cu_seqlens: torch.Tensor | None = None, *,
                               row_order: torch.Tensor | None = None,
                               dh: torch.Tensor | None = None, dW: torch.Tensor | None = None,
                               workspace: torch.Tensor | None = None,
                               stream: torch.cuda.Stream | None = None):
    """(dh fp32 [T, H], dW fp32 [V, H]) from the state :func:`linear_logp_fwd_saved`
    kept (read only)."""
    lib = load_library()
    _need(h, "h", torch.bfloat16, 2)
    _need(W, "W", torch.bfloat16, 2)
    T, H = h.shape
    V = W.shape[0]
    cu, ns = _rows(targets, cu_seqlens, T, h.device)
    if row_order is not None:
        _need(row_order, "row_order", torch.int64, 1)
        n = row_order.shape[0]
    else:
        n = T
    if dh is None:
        dh = torch.empty((T, H), dtype=torch.float32, device=h.device)
    if dW is None:
        dW = torch.empty((V, H), dtype=torch.float32, device=h.device)
    if workspace is None:
        need = int(lib.rk_linear_logp_bwd_full_workspace_size(n, H, V))
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=h.device)
    st = lib.rk_linear_logp_bwd_full_saved(_ptr(h), _ptr(W), _ptr(targets), _ptr(cu), ns, T, H, V,
                                           _ptr(lse), _ptr(grad_logp), _ptr(saved), saved.numel(),
                                           _ptr(row_order), n, _ptr(dh), _ptr(dW),
                                           _ptr(workspace), workspace.numel(),
                                           _stream_handle(stream, h.device))
    _check(st, "rk_linear_logp_bwd_full_saved")
    return dh, dW


def linear_greedy_workspace_size(T: int, H: int, V: int) -> int:
    return int(load_library().rk_linear_greedy_workspace_size(T, H, V))


def linear_greedy(h: torch.Tensor, W: torch.Tensor, cu_seqlens: torch.Tensor | None = None, *,
                  workspace: torch.Tensor | None = None,
                  stream: torch.cuda.Stream | None = None):
    """Greedy step: ``(token int64 [T], logp fp32 [T], lse fp32 [T])``."""
    lib = load_library()
    _need(h, "h", torch.bfloat16, 2)
    _need(W, "W", torch.bfloat16, 2)
    T, H = h.shape
    V = W.shape[0]
    if W.shape[1] != H or W.device != h.device:
        raise ValueError("W must be [V, H] on h's device")
    cu, ns = (None, 0)
    if cu_seqlens is not None:
        _need(cu_seqlens, "cu_seqlens", torch.int32, 1)
        cu, ns = cu_seqlens, cu_seqlens.numel() - 1
    token = torch.empty(T, dtype=torch.int64, device=h.device)
    logp = torch.empty(T, dtype=torch.float32, device=h.device)
    lse = torch.empty(T, dtype=torch.float32, device=h.device)
    if workspace is None:
        need = int(lib.rk_linear_greedy_workspace_size(T, H, V))
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=h.device)
    st = lib.rk_linear_greedy(_ptr(h), _ptr(W), _ptr(cu), ns, T, H, V, _ptr(token), _ptr(logp),
                              _ptr(lse), _ptr(workspace), workspace.numel(),
                              _stream_handle(stream, h.device))
    _check(st, "rk_linear_greedy")
    return token, logp, lse


def linear_logp_dw_workspace_size(n: int, H: int, V: int) -> int:
    return int(load_library().rk_linear_logp_dw_workspace_size(n, H, V))


def linear_logp_dw(h: torch.Tensor, W: torch.Tensor, targets: torch.Tensor, lse: torch.Tensor,
                   grad_logp: torch.Tensor, cu_seqlens: torch.Tensor | None = None, *,
                   row_order: torch.Tensor | None = None, dW: torch.Tensor | None = None,
                   workspace: torch.Tensor | None = None,
                   stream: torch.cuda.Stream | None = None) -> torch.Tensor:
    """dW fp32 ``[V, H]`` summed over the active rows in canonical order
    (``row_order``, int64 physical row indices; ascending rows by default)."""
    lib = load_library()
    _need(h, "h", torch.bfloat16, 2)
    _need(W, "W", torch.bfloat16, 2)
    T, H = h.shape
    V = W.shape[0]
    if W.shape[1] != H or W.device != h.device:
        raise ValueError("W must be [V, H] on h's device")
    cu, ns = _rows(targets, cu_seqlens, T, h.device)
    _need(lse, "lse", torch.float32, 1)
    _need(grad_logp, "grad_logp", torch.float32, 1)
    n = T
    if row_order is not None:
        _need(row_order, "row_order", torch.int64, 1)
        n = row_order.numel()
    if dW is None:
        dW = torch.empty((V, H), dtype=torch.float32, device=h.device)
    if workspace is None:
        need = int(lib.rk_linear_logp_dw_workspace_size(n, H, V))
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=h.device)
    st = lib.rk_linear_logp_dw(_ptr(h), _ptr(W), _ptr(targets), _ptr(cu), ns, T, H, V, _ptr(lse),
                               _ptr(grad_logp), _ptr(row_order), n, _ptr(dW), _ptr(workspace),
                               workspace.numel(), _stream_handle(stream, h.device))
    _check(st, "rk_linear_logp_dw")
    return dW


def linear_logp_bwd_full_workspace_size(n: int, H: int, V: int) -> int:
    return int(load_library().rk_linear_logp_bwd_full_workspace_size(n, H, V))


def linear_logp_bwd_full(h: torch.Tensor, W: torch.Tensor, targets: torch.Tensor,
                         lse: torch.Tensor, grad_logp: torch.Tensor,
                         cu_seqlens: torch.Tensor | None = None, *,
                         row_order: torch.Tensor | None = None, dh: torch.Tensor | None = None,
                         dW: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                         stream: torch.cuda.Stream | None = None):
    """(dh fp32 [T, H], dW fp32 [V, H]) from one shared softmax pass."""
    lib = load_library()
    _need(h, "h", torch.bfloat16, 2)
    _need(W, "W", torch.bfloat16, 2)
    T, H = h.shape
    V = W.shape[0]
    if W.shape[1] != H or W.device != h.device:
        raise ValueError("W must be [V, H] on h's device")
    cu, ns = _rows(targets, cu_seqlens, T, h.device)
    _need(lse, "lse", torch.float32, 1)
    _need(grad_logp, "grad_logp", torch.float32, 1)
    n = T
    if row_order is not None:
        _need(row_order, "row_order", torch.int64, 1)
        n = row_order.numel()
    if dh is None:
        dh = torch.empty((T, H), dtype=torch.float32, device=h.device)
    if dW is None:
        dW = torch.empty((V, H), dtype=torch.float32, device=h.device)
    if workspace is None:
        need = int(lib.rk_linear_logp_bwd_full_workspace_size(n, H, V))
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=h.device)
    st = lib.rk_linear_logp_bwd_full(_ptr(h), _ptr(W), _ptr(targets), _ptr(cu), ns, T, H, V,
                                     _ptr(lse), _ptr(grad_logp), _ptr(row_order), n, _ptr(dh),
                                     _ptr(dW), _ptr(workspace), workspace.numel(),
                                     _stream_handle(stream, h.device))
    _check(st, "rk_linear_logp_bwd_full")
    return dh, dW


class _RulesStruct(ctypes.Structure):
    """rk_logits_rules of include/rk.h."""
    _fields_ = [("num_requests", ctypes.c_int64)] + \
        [(n, ctypes.c_void_p) for n in ("temperature", "repetition", "frequency", "presence",
                                        "tokens")] + \
        [("num_tokens", ctypes.c_int64), ("token_offsets", ctypes.c_void_p),
         ("prompt_lengths", ctypes.c_void_p), ("bias_ids", ctypes.c_void_p),
         ("bias_values", ctypes.c_void_p), ("num_bias", ctypes.c_int64),
         ("bias_offsets", ctypes.c_void_p), ("mask", ctypes.c_void_p),
         ("mask_rows", ctypes.c_int64)] + \
        [(n, ctypes.c_void_p) for n in ("row_request", "row_length", "row_mask")]


class LogitsRules:
    """What a decoding loop does to the logits before it draws a token.

    Row ``t`` belongs to request ``r = row_request[t]`` (default ``t``) and has
    seen the first ``row_length[t]`` (default: all) of that request's tokens,
    ``tokens[token_offsets[r] : token_offsets[r + 1]]``, of which the first
    ``prompt_lengths[r]`` (default 0) are the prompt and the others were
    produced.  With ``n[v]`` how often ``v`` was produced::

        y = z;  where v was seen at all:  z / repetition  (z > 0),  z * repetition  (z <= 0)
        y = y - frequency * n - presence * (n > 0) + bias
        x = y / temperature,  -inf where the row's mask has a 0 bit

    Per request: ``temperature``, ``repetition``, ``frequency``, ``presence``
    (fp32 ``[R]``), ``prompt_lengths`` (int32 ``[R]``), ``token_offsets`` and
    ``bias_offsets`` (int64 ``[R + 1]``) into ``tokens`` (int64) and into
    ``bias_ids`` (int64) / ``bias_values`` (fp32).  ``mask`` is int32
    ``[M, ceil(V / 32)]``, bit ``v % 32`` of word ``v // 32`` set where token ``v``
    is allowed.  Per row, int32 ``[T]``: ``row_request`` (-1: padding),
    ``row_length``, ``row_mask`` (default ``t``; negative: no mask).  All are
    contiguous CUDA tensors, kept by the object; whatever is left out does not
    apply.  The tensors are read when an operator runs, so their contents may
    change between calls (a replayed CUDA graph reads the new ones, and needs the
    object alive).
    """

    __slots__ = ("device", "struct", "address", "rows", "mask_words", "_kept")

    def __init__(self, *, temperature: torch.Tensor | None = None,
                 repetition: torch.Tensor | None = None, frequency: torch.Tensor | None = None,
                 presence: torch.Tensor | None = None, tokens: torch.Tensor | None = None,
                 token_offsets: torch.Tensor | None = None,
                 prompt_lengths: torch.Tensor | None = None, bias_ids: torch.Tensor | None = None,
                 bias_values: torch.Tensor | None = None, bias_offsets: torch.Tensor | None = None,
                 mask: torch.Tensor | None = None, row_request: torch.Tensor | None = None,
                 row_length: torch.Tensor | None = None, row_mask: torch.Tensor | None = None):
        kept = (temperature, repetition, frequency, presence, tokens, token_offsets, prompt_lengths,
                bias_ids, bias_values, bias_offsets, mask, row_request, row_length, row_mask)
        address = []
        device = index = requests = rows = None
        for t, (name, dtype, ndim, extra) in zip(kept, _RULES):
            if t is None:
                address.append(None)
                continue
            if not (isinstance(t, torch.Tensor) and t.is_cuda and t.dtype is dtype
                    and t.is_contiguous()) or t.dim() != ndim:
                _need(t, name, dtype, ndim)
            if index is None:
                device, index = t.device, t.get_device()
            elif t.get_device() != index:
                raise ValueError(f"{name} is on {t.device}, not on {device}")
            if extra is not None:
                n = t.numel()  # one dimension
                if extra < 0:  # per row
                    if n != rows:
                        if rows is not None:
                            raise ValueError(f"{name} does not fit {rows} rows")
                        rows = n
                elif n - extra != requests:
                    if requests is not None or n < extra:
                        raise ValueError(f"{name} does not fit {'any' if requests is None else requests} requests")
                    requests = n - extra
            # an empty list still has to be told from a missing one
            address.append(t.data_ptr() or _EMPTY)
        if (tokens is None) != (token_offsets is None):
            raise ValueError("tokens and token_offsets go together")
        if tokens is None and (prompt_lengths is not None or row_length is not None):
            raise ValueError("prompt_lengths and row_length need tokens")
        if not ((bias_ids is None) == (bias_values is None) == (bias_offsets is None)):
            raise ValueError("bias_ids, bias_values and bias_offsets go together")
        if row_mask is not None and mask is None:
            raise ValueError("row_mask needs mask")
        num_bias = 0 if bias_ids is None else bias_ids.size(0)
        if num_bias and num_bias != bias_values.size(0):
            raise ValueError("bias_ids and bias_values differ in length")
        if requests == 0 and rows:
            raise ValueError(f"no requests for {rows} rows")
        if requests is not None and row_request is None:
            if rows is not None and rows != requests:
                raise ValueError(f"{requests} requests for {rows} rows: row_request is missing")
            rows = requests
        mask_rows, self.mask_words = (0, None) if mask is None else mask.shape
        if mask is not None and row_mask is None:
            if rows is not None and rows != mask_rows:
                raise ValueError(f"{mask_rows} masks for {rows} rows: row_mask is missing")
            rows = mask_rows
        self.struct = s = _RulesStruct(
            requests or 0, *address[:5], 0 if tokens is None else tokens.size(0), *address[5:9],
            num_bias, address[9], address[10], mask_rows, *address[11:])
        self.device, self.rows = device, rows
        self.address, self._kept = ctypes.addressof(s), kept


_EMPTY = 256  # an address that an empty list never reads
# name, type, dimensions, and entries beyond one per request (-1: one per row, None: neither)
_RULES = (("temperature", torch.float32, 1, 0), ("repetition", torch.float32, 1, 0),
          ("frequency", torch.float32, 1, 0), ("presence", torch.float32, 1, 0),
          ("tokens", torch.int64, 1, None), ("token_offsets", torch.int64, 1, 1),
          ("prompt_lengths", torch.int32, 1, 0), ("bias_ids", torch.int64, 1, None),
          ("bias_values", torch.float32, 1, None), ("bias_offsets", torch.int64, 1, 1),
          ("mask", torch.int32, 2, None), ("row_request", torch.int32, 1, -1),
          ("row_length", torch.int32, 1, -1), ("row_mask", torch.int32, 1, -1))
_TYPE_CODES = {torch.bfloat16: 0, torch.float32: 1}


def _matrix(t: torch.Tensor, name: str, shape=None, device=None):
    """(type code, row stride) of a bf16 or fp32 [T, V] matrix with unit column stride."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor (no CPU path), got {t.device}")
    code = _TYPE_CODES.get(t.dtype)
    if code is None:
        raise TypeError(f"{name} must be bfloat16 or float32, got {t.dtype}")
    if t.dim() != 2 or (shape is not None and t.shape != shape):
        raise ValueError(f"{name} must be {list(shape) if shape else '[T, V]'}, "
                         f"got shape {tuple(t.shape)}")
    if device is not None and t.device != device:
        raise ValueError(f"{name} must be on {device}, got {t.device}")
    T, V = t.shape
    ld, unit = t.stride()
    if V > 1 and unit != 1:
        raise ValueError(f"{name} must have unit column stride")
    if T <= 1:
        ld = max(V, 1)
    if ld < V:
        raise ValueError(f"{name}'s rows overlap")
    return code, ld


def _empty(shape, dtype, device, stream) -> torch.Tensor:
    """New memory of the stream that the operator runs on: another stream's may still be
    in use there, and would be handed out again while this one works on it."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _result(out, dtype, shape, device, stream):
    """(matrix, type code, row stride) of a result: ``out`` if it is given, or a new one."""
    if out is not None:
        return out, *_matrix(out, "out", shape, device)
    code = _TYPE_CODES.get(dtype)
    if code is None:
        raise TypeError(f"out must be bfloat16 or float32, got {dtype}")
    return _empty(shape, dtype, device, stream), code, shape[1]


def _rules_for(rules: LogitsRules, T: int, V: int, device) -> None:
    if not isinstance(rules, LogitsRules):
        raise TypeError("rules must be a LogitsRules")
    if rules.device is not None and rules.device != device:
        raise ValueError(f"the rules are on {rules.device}, the logits on {device}")
    if rules.rows is not None and rules.rows != T:
        raise ValueError(f"the rules are for {rules.rows} rows, the logits have {T}")
    if rules.mask_words is not None and rules.mask_words != (V + 31) // 32:
        raise ValueError(f"mask must have ceil(V / 32) = {(V + 31) // 32} words a row, "
                         f"got {rules.mask_words}")


def _vector(t: torch.Tensor, name: str, T: int, device) -> None:
    _need(t, name, torch.float32, 1)
    if t.shape[0] != T or t.device != device:
        raise ValueError(f"{name} must be [T] on {device}")


def _is_lse64(lse: torch.Tensor, T: int, device) -> bool:
    """Whether a log-sum-exp, fp32 or fp64 [T], is the latter."""
    if not isinstance(lse, torch.Tensor) or lse.dtype is not torch.float64:
        _vector(lse, "lse", T, device)
        return False
    _need(lse, "lse", torch.float64, 1)
    if lse.shape[0] != T or lse.device != device:
        raise ValueError(f"lse must be [T] on {device}")
    return True


def _run(what: str, fn, device, stream, *args) -> None:
    """Calls the library on ``device``, with the stream's handle behind ``args``."""
    if stream is None:
        handle = torch._C._cuda_getCurrentRawStream(device.index)
    elif stream.device != device:
        raise ValueError(f"the stream is on {stream.device}, the tensors on {device}")
    else:
        handle = stream.cuda_stream
    if torch._C._cuda_getDevice() == device.index:
        st = fn(*args, handle)
    else:
        with torch.cuda.device(device):
            st = fn(*args, handle)
    if st != RK_OK:
        _check(st, what)


def _scratch(workspace, need: int, device, stream) -> torch.Tensor:
    if workspace is None:
        return _empty(max(need, 1), torch.uint8, device, stream)
    _need(workspace, "workspace", torch.uint8, 1)
    if workspace.device != device:
        raise ValueError(f"workspace must be on {device}")
    return workspace


def logits_rules_apply(logits: torch.Tensor, rules: LogitsRules, *,
                       out: torch.Tensor | None = None, out_dtype: torch.dtype = torch.float32,
                       stream: torch.cuda.Stream | None = None) -> torch.Tensor:
    """The logits under ``rules``, ``[T, V]`` in ``out_dtype`` (bf16 or fp32).

    ``logits`` is bf16 or fp32 ``[T, V]`` with any row stride (the output of
    :func:`lm_head` as it is); ``out`` may be ``logits`` itself, or a matrix whose rows
    have no byte in common with those of ``logits``.  Rows with ``row_request`` -1 are
    left as they are in ``out`` (undefined in a new one)."""
    lib = _lib or load_library()
    code, ld = _matrix(logits, "logits")
    T, V = logits.shape
    device = logits.device
    _rules_for(rules, T, V, device)
    out, out_code, out_ld = _result(out, out_dtype, (T, V), device, stream)
    _run("rk_logits_rules_apply", lib.rk_logits_rules_apply, device, stream, logits.data_ptr(), code,
         ld, rules.address, T, V, out.data_ptr(), out_code, out_ld)
    return out


def logp_from_logits_rules_workspace_size(T: int, V: int) -> int:
    return int(load_library().rk_logp_from_logits_rules_workspace_size(T, V))


def logp_from_logits_rules(logits: torch.Tensor, targets: torch.Tensor, rules: LogitsRules,
                           cu_seqlens: torch.Tensor | None = None, *,
                           out: torch.Tensor | None = None, lse: torch.Tensor | None = None,
                           lse_dtype: torch.dtype = torch.float32,
                           workspace: torch.Tensor | None = None,
                           stream: torch.cuda.Stream | None = None):
    """Selected-token logprob of the distribution that ``rules`` leave: returns
    ``(logp, lse)``, fp32 ``[T]``.  Both are -inf on a row of which the rules
    leave nothing, logp where the target is masked.  With ``lse_dtype``
    (or an ``lse``) of float64 the log-sum-exp is not rounded to fp32, which
    :func:`logp_from_logits_rules_bwd` needs at low temperatures."""
    lib = _lib or load_library()
    code, ld = _matrix(logits, "logits")
    T, V = logits.shape
    device = logits.device
    cu, ns = _rows(targets, cu_seqlens, T, device)
    _rules_for(rules, T, V, device)
    if out is None:
        out = _empty(T, torch.float32, device, stream)
    else:
        _vector(out, "out", T, device)
    if lse is None:
        if lse_dtype is not torch.float32 and lse_dtype is not torch.float64:
            raise TypeError(f"lse must be float32 or float64, got {lse_dtype}")
        lse = _empty(T, lse_dtype, device, stream)
        wide = lse_dtype is torch.float64
    else:
        wide = _is_lse64(lse, T, device)
    workspace = _scratch(workspace, lib.rk_logp_from_logits_rules_workspace_size(T, V), device,
                         stream)
    _run("rk_logp_from_logits_rules",
         lib.rk_logp_from_logits_rules_lse64 if wide else lib.rk_logp_from_logits_rules, device, stream,
         logits.data_ptr(), code, ld, targets.data_ptr(), _ptr(cu), ns, rules.address, T, V,
         out.data_ptr(), lse.data_ptr(), workspace.data_ptr(), workspace.numel())
    return out, lse


def logp_from_logits_rules_bwd(logits: torch.Tensor, targets: torch.Tensor, rules: LogitsRules,
                               lse: torch.Tensor, grad_logp: torch.Tensor,
                               cu_seqlens: torch.Tensor | None = None, *,
                               out: torch.Tensor | None = None,
                               out_dtype: torch.dtype = torch.float32,
                               stream: torch.cuda.Stream | None = None) -> torch.Tensor:
    """The gradient of :func:`logp_from_logits_rules` with respect to the logits,
    ``[T, V]`` in ``out_dtype`` (bf16 or fp32); ``out`` as for :func:`logits_rules_apply`.

    An fp32 ``lse`` leaves every probability a relative error of up to 2**-23 * |lse|, and
    the gradient grows with 1 / temperature: below a temperature of some 0.1 use a float64
    ``lse`` (``lse_dtype`` of :func:`logp_from_logits_rules`)."""
    lib = _lib or load_library()
    code, ld = _matrix(logits, "logits")
    T, V = logits.shape
    device = logits.device
    cu, ns = _rows(targets, cu_seqlens, T, device)
    _rules_for(rules, T, V, device)
    wide = _is_lse64(lse, T, device)
    _vector(grad_logp, "grad_logp", T, device)
    out, out_code, out_ld = _result(out, out_dtype, (T, V), device, stream)
    _run("rk_logp_from_logits_rules_bwd",
         lib.rk_logp_from_logits_rules_bwd_lse64 if wide else lib.rk_logp_from_logits_rules_bwd, device, stream,
         logits.data_ptr(), code, ld, targets.data_ptr(), _ptr(cu), ns, rules.address, T, V,
         lse.data_ptr(), grad_logp.data_ptr(), out.data_ptr(), out_code, out_ld)
    return out


def _dense(t: torch.Tensor, name: str, shape, device) -> int:
    """Type code of a contiguous bf16 or fp32 matrix."""
    code, _ = _matrix(t, name, shape, device)
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return code


def embedding(ids: torch.Tensor, E: torch.Tensor, cu_seqlens: torch.Tensor | None = None, *,
              scale: float = 1.0, out: torch.Tensor | None = None,
              out_dtype: torch.dtype | None = None,
              stream: torch.cuda.Stream | None = None) -> torch.Tensor:
    """``scale * E[ids]``, ``[T, H]`` in ``out_dtype`` (default: E's), 0 in rows with a
    negative id or outside ``cu_seqlens``; E is bf16 or fp32 ``[V, H]``."""
    lib = _lib or load_library()
    code = _dense(E, "E", None, None)
    V, H = E.shape
    device = E.device
    T = ids.shape[0] if isinstance(ids, torch.Tensor) and ids.dim() == 1 else 0
    cu, ns = _rows(ids, cu_seqlens, T, device, "ids")
    if out is not None and not out.is_contiguous():
        raise ValueError("out must be contiguous")
    out, out_code, _ = _result(out, out_dtype or E.dtype, (T, H), device, stream)
    _run("rk_embedding", lib.rk_embedding, device, stream, ids.data_ptr(), _ptr(cu), ns, E.data_ptr(),
         code, T, H, V, scale, out.data_ptr(), out_code)
    return out


def embedding_bwd_workspace_size(n: int, H: int, V: int) -> int:
    return int(load_library().rk_embedding_bwd_workspace_size(n, H, V))


def embedding_bwd(grad_out: torch.Tensor, ids: torch.Tensor, V: int,
                  cu_seqlens: torch.Tensor | None = None, *, scale: float = 1.0,
                  row_order: torch.Tensor | None = None, dE: torch.Tensor | None = None,
                  accumulate: bool = False, workspace: torch.Tensor | None = None,
                  stream: torch.cuda.Stream | None = None) -> torch.Tensor:
    """dE fp32 ``[V, H]``: ``scale *`` the sum of ``grad_out``'s rows (bf16 or fp32
    ``[T, H]``) of each id over the active rows in canonical order (``row_order``, int64
    physical row indices; ascending rows by default).  With ``accumulate`` it is added
    to what ``dE`` holds (a weight tied to the lm_head's: ``dE`` from
    :func:`linear_logp_dw`)."""
    lib = _lib or load_library()
    code = _dense(grad_out, "grad_out", None, None)
    T, H = grad_out.shape
    device = grad_out.device
    cu, ns = _rows(ids, cu_seqlens, T, device, "ids")
    n, order = T, None
    if row_order is not None:
        _need(row_order, "row_order", torch.int64, 1)
        if row_order.device != device:
            raise ValueError(f"row_order must be on {device}")
        n = row_order.shape[0]
        order = row_order.data_ptr() or _EMPTY
    if dE is None:
        if accumulate:
            raise ValueError("accumulate needs a dE to add to")
        dE = _empty((V, H), torch.float32, device, stream)
    elif _dense(dE, "dE", (V, H), device) != 1:
        raise TypeError("dE must be float32")
    workspace = _scratch(workspace, lib.rk_embedding_bwd_workspace_size(n, H, V), device, stream)
    _run("rk_embedding_bwd", lib.rk_embedding_bwd, device, stream, grad_out.data_ptr(), code,
         ids.data_ptr(), _ptr(cu), ns, T, H, V, scale, order, n, dE.data_ptr(), int(accumulate),
         workspace.data_ptr(), workspace.numel())
    return dE


def selftest_wait_timeout(limit_ns: int, stream: torch.cuda.Stream | None = None) -> None:
    """Launch a kernel whose bounded wait must time out after ``limit_ns``."""
    lib = load_library()
    _check(lib.rk_selftest_wait_timeout(int(limit_ns), _stream_handle(stream, None)),
           "rk_selftest_wait_timeout")


def set_row_blocks(n: int) -> None:
    """Row blocks per tile of the dh and dW GEMMs: 0 automatic (default), or
    1 / 2 forced for every later launch in the process (bits are unchanged)."""
    _check(load_library().rk_set_row_blocks(int(n)), "rk_set_row_blocks")


def last_row_blocks(gemm: str) -> int:
    """Row blocks per tile of the last ``"dh"`` or ``"dw"`` GEMM launched on
    this thread (0 before the first)."""
    return int(load_library().rk_last_row_blocks({"dh": 0, "dw": 1}[gemm]))


def last_tile_order(gemm: str) -> int:
    """Tile order of the last ``"dh"`` or ``"dw"`` GEMM launched on this
    thread: 2 rounds started together, 1 tiles from a counter, 0 before the
    first."""
    return int(load_library().rk_last_tile_order({"dh": 0, "dw": 1}[gemm]))


def get_device_error(stream: torch.cuda.Stream | None = None) -> int:
    """Read and clear the device error word (synchronises the stream)."""
    lib = load_library()
    v = ctypes.c_int32(0)
    _check(lib.rk_get_device_error(_stream_handle(stream, None), ctypes.byref(v)),
           "rk_get_device_error")
    return int(v.value)
