"""Python binding of libslr: the 2:4-sparse + low-rank linear layer on B200.

Argument marshalling only.  Every step of the computation runs in the CUDA
kernels of ``libslr.so`` (built in-tree by ``python
sparse_rank_linear_02_b200/build.py``); there is no fallback of any kind, and the
import fails if the library is missing.

Functions mirror the C ABI in ``include/slr.h``:

* ``pack_2to4(W) -> (vals, meta)``  -- ``slr_pack_2to4``
* ``pack_2to4_scaled(W, scale) -> (vals, meta)``  -- ``slr_pack_2to4_scaled``
* ``column_norms(X, sumsq=None) -> (norms, sumsq)``  -- ``slr_column_norms``
* ``pack_2to8(W, dense=True, as_2to4=True)``  -- ``slr_pack_2to8``
* ``forward_2to8(X, vals8, meta8, U, V) -> Y``  -- ``slr_forward_2to8``
* ``lora_backward(X, dY, U, V, T=None) -> (dU, dV)``  -- ``slr_lora_backward``
* ``decompose_datafree(W, r, iters, ...) -> (vals, meta, U, V, objective)``  --
  ``slr_decompose_datafree``
* ``forward(X, vals, meta, U, V) -> Y``  -- ``slr_forward`` /
  ``slr_forward_with_path`` / ``slr_forward_ex``
* ``forward_epilogue(X, vals, meta, U, V, bias, act, residual) -> Y``  --
  ``slr_forward_epilogue``
* ``epilogue_backward(dY, Z, act) -> (dZ, dbias)``  -- ``slr_epilogue_backward``
* ``input_backward(dY, vals, meta, U, V) -> dX``  -- ``slr_input_backward``
* ``distill_forward(logits, idx, teacher) -> (loss, lse)``, ``distill_backward(...) -> dlogits``,
  ``distill_loss_grad(...) -> (loss, dlogits)``  -- ``slr_distill_*``
* ``workspace_size``, ``select_path``, ``check_kernel_error``

Tensors are torch CUDA tensors (torch only provides memory and the current
stream): bf16 for W, X, U, V, vals and Y, uint8 for meta.
"""
from __future__ import annotations

import ctypes
import os

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libslr.so")

SLR_OK = 0
STATUS_NAMES = {0: "SLR_OK", 1: "SLR_ERR_NULL", 2: "SLR_ERR_SHAPE", 3: "SLR_ERR_ALIGN",
                4: "SLR_ERR_WORKSPACE", 5: "SLR_ERR_DEVICE", 6: "SLR_ERR_CUDA",
                7: "SLR_ERR_TIMEOUT", 8: "SLR_ERR_ARG"}
PATHS = {"auto": 0, "decode": 1, "tensor": 2}
PATH_NAMES = {v: k for k, v in PATHS.items()}
ACTS = {"none": 0, "relu": 1, "gelu": 2, "gelu_tanh": 3, "silu": 4}


class SlrError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {STATUS_NAMES.get(status, status)} "
                         f"({_lib.slr_status_string(status).decode()})")


def _load() -> ctypes.CDLL:
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is missing; build it with "
                          f"`python sparse_rank_linear_02_b200/build.py`")
    lib = ctypes.CDLL(LIB_PATH)
    i64, p, sz, st = ctypes.c_int64, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int
    lib.slr_status_string.restype = ctypes.c_char_p
    lib.slr_status_string.argtypes = [st]
    lib.slr_version.restype = ctypes.c_int
    lib.slr_pack_2to4.restype = st
    lib.slr_pack_2to4.argtypes = [p, i64, i64, i64, p, p, p]
    lib.slr_meta_row_bytes.restype = i64
    lib.slr_meta_row_bytes.argtypes = [i64]
    lib.slr_pack_2to4_scaled.restype = st
    lib.slr_pack_2to4_scaled.argtypes = [p, i64, i64, i64, p, p, p, p]
    lib.slr_pack_2to8.restype = st
    lib.slr_pack_2to8.argtypes = [p, i64, i64, i64, p, p, p, p, p]
    lib.slr_forward_2to8.restype = st
    lib.slr_forward_2to8.argtypes = [p, i64, p, p, i64, i64, p, p, i64, p, p, sz, p]
    lib.slr_decompose_datafree.restype = st
    lib.slr_decompose_datafree.argtypes = [p, i64, i64, i64, ctypes.c_int, ctypes.c_int, ctypes.c_int, p, p, p, p,
                                           p, p, p, sz, p]
    lib.slr_decompose_factors_f32.restype = st
    lib.slr_decompose_factors_f32.argtypes = [p, sz, i64, i64, i64, p, p, p]
    lib.slr_decompose_workspace_size.restype = sz
    lib.slr_decompose_workspace_size.argtypes = [i64, i64, i64]
    lib.slr_lora_backward.restype = st
    lib.slr_lora_backward.argtypes = [p, i64, p, i64, i64, p, p, i64, p, p, p, p, sz, p]
    lib.slr_lora_backward_workspace_size.restype = sz
    lib.slr_lora_backward_workspace_size.argtypes = [i64, i64]
    lib.slr_column_norms.restype = st
    lib.slr_column_norms.argtypes = [p, i64, i64, i64, p, p, p, sz, p]
    lib.slr_column_norms_workspace_size.restype = sz
    lib.slr_column_norms_workspace_size.argtypes = [i64, i64]
    lib.slr_forward.restype = st
    lib.slr_forward.argtypes = [p, i64, p, p, i64, i64, p, p, i64, p, p, sz, p]
    lib.slr_forward_with_path.restype = st
    lib.slr_forward_with_path.argtypes = [p, i64, p, p, i64, i64, p, p, i64, p, p, sz, st, p]
    lib.slr_forward_ex.restype = st
    lib.slr_forward_ex.argtypes = [p, i64, p, p, i64, i64, p, p, i64, p, p, sz, st, ctypes.c_uint32, p]
    lib.slr_forward_epilogue.restype = st
    lib.slr_forward_epilogue.argtypes = [p, i64, p, p, i64, i64, p, p, i64, p, st, p, i64, p, p, p, sz, st,
                                         ctypes.c_uint32, p]
    lib.slr_epilogue_backward.restype = st
    lib.slr_epilogue_backward.argtypes = [p, p, i64, i64, st, p, p, p]
    lib.slr_input_backward.restype = st
    lib.slr_input_backward.argtypes = [p, i64, p, p, i64, i64, p, p, i64, p, p, sz, p]
    lib.slr_input_backward_workspace_size.restype = sz
    lib.slr_input_backward_workspace_size.argtypes = [i64, i64, i64, i64]
    f32 = ctypes.c_float
    lib.slr_distill_forward.restype = st
    lib.slr_distill_forward.argtypes = [p, i64, i64, i64, p, p, i64, f32, p, p, p]
    lib.slr_distill_backward.restype = st
    lib.slr_distill_backward.argtypes = [p, i64, i64, i64, p, p, i64, f32, p, p, p, i64, p]
    lib.slr_distill_loss_grad.restype = st
    lib.slr_distill_loss_grad.argtypes = [p, i64, i64, i64, p, p, i64, f32, p, p, p, i64, p]
    lib.slr_forward_workspace_size.restype = sz
    lib.slr_forward_workspace_size.argtypes = [i64, i64, i64, i64]
    lib.slr_forward_select_path.restype = st
    lib.slr_forward_select_path.argtypes = [i64, i64, i64, i64]
    lib.slr_check_kernel_error.restype = st
    lib.slr_check_kernel_error.argtypes = []
    lib.slr_forward_project.restype = st
    lib.slr_forward_project.argtypes = [p, i64, p, i64, i64, i64, p, sz, st, p]
    lib.slr_forward_combine.restype = st
    lib.slr_forward_combine.argtypes = [p, i64, p, p, i64, i64, p, i64, p, p, sz, st, p]
    lib.slr_forward_decode_noalloc.restype = st
    lib.slr_forward_decode_noalloc.argtypes = [p, i64, p, p, i64, i64, p, p, i64, p, p]
    lib.slr_selftest_wait_timeout.restype = st
    lib.slr_selftest_wait_timeout.argtypes = [i64, p]
    i32 = ctypes.c_int32
    lib.slr_plan_check.restype = i64
    lib.slr_plan_check.argtypes = [i64, i64, i64, i64, i32, i32, i32, i32]
    return lib


_lib = _load()


PLAN_KERNELS = {"2sm128": 0, "2sm240": 1, "2smtall": 2, "2sm256": 3}
PLAN_TAILS = {"whole": 0, "tokens": 1, "k": 2}


def plan_check(M: int, d_out: int, d_in: int, r: int, kernel: str, tail: str, max_pairs: int,
               chunk_units: int = 0) -> int:
    """``slr_plan_check``: the number of violations in the pair kernels' work
    plan for this shape (0 = sound; host only, no device needed)."""
    return int(_lib.slr_plan_check(M, d_out, d_in, r, PLAN_KERNELS[kernel], PLAN_TAILS[tail], max_pairs,
                                   chunk_units))


def lib() -> ctypes.CDLL:
    """The loaded ``libslr.so`` (for direct C-ABI calls)."""
    return _lib


def _stream() -> int:
    return torch.cuda.current_stream().cuda_stream


def _ptr(t: torch.Tensor | None):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _check(status: int, what: str):
    if status != SLR_OK:
        raise SlrError(status, what)


def _expect(name: str, t: torch.Tensor, dtype: torch.dtype, shape: tuple, device: torch.device):
    """Refuse an operand whose type, shape, layout or device is not what the call reads."""
    if t.dtype is not dtype or t.shape != shape or not t.is_contiguous() or t.device != device:
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {tuple(shape)} on {device}, not "
                         f"{t.dtype} {tuple(t.shape)} with strides {t.stride()} on {t.device}")


def _current(t: torch.Tensor) -> tuple[torch.device, int]:
    """The operand's device, which has to be the current one, and its current stream."""
    device = t.device
    if device.type != "cuda" or device.index != torch.cuda.current_device():
        raise ValueError(f"the operands are on {device}, not on the current CUDA device")
    return device, torch._C._cuda_getCurrentRawStream(device.index)


def _addr(t: torch.Tensor | None) -> int | None:
    return None if t is None else t.data_ptr()


def _expect_layer(vals: torch.Tensor, meta: torch.Tensor, U: torch.Tensor | None, V: torch.Tensor | None,
                  device: torch.device) -> tuple[int, int, int]:
    """(d_out, d_in, r) of a packed layer, its operands checked."""
    if vals.dim() != 2 or (U is None) != (V is None):
        raise ValueError("vals must be 2-D, and U and V come together")
    d_out, half = vals.shape
    _expect("vals", vals, torch.bfloat16, (d_out, half), device)
    _expect("meta", meta, torch.uint8, (d_out, (half + 3) // 4), device)
    if U is None:
        return d_out, 2 * half, 0
    r = V.shape[0]
    _expect("U", U, torch.bfloat16, (d_out, r), device)
    _expect("V", V, torch.bfloat16, (r, 2 * half), device)
    return d_out, 2 * half, r


def _scratch(workspace: torch.Tensor | None, need: int, device: torch.device) -> tuple[torch.Tensor | None, int]:
    """The caller's workspace, or a new one of `need` bytes, and its bytes."""
    if workspace is None:
        return (torch.empty(need, dtype=torch.uint8, device=device), need) if need else (None, 0)
    if not workspace.is_contiguous() or workspace.device != device:
        raise ValueError(f"workspace must be a contiguous tensor on {device}")
    return workspace, workspace.nbytes


def meta_row_bytes(d_in: int) -> int:
    return int(_lib.slr_meta_row_bytes(d_in))


def pack_2to4(W: torch.Tensor) -> tuple[torch.Tensor, torch.Tensor]:
    """2:4 projection by magnitude and packing of bf16 ``W`` [d_out, d_in]."""
    if W.dtype != torch.bfloat16 or W.dim() != 2 or not W.is_cuda or W.stride(1) != 1:
        raise ValueError("W must be a 2-D CUDA bf16 tensor with unit column stride")
    d_out, d_in = W.shape
    vals = torch.empty((d_out, d_in // 2), dtype=torch.bfloat16, device=W.device)
    meta = torch.empty((d_out, meta_row_bytes(d_in)), dtype=torch.uint8, device=W.device)
    _check(_lib.slr_pack_2to4(_ptr(W), d_out, d_in, W.stride(0), _ptr(vals), _ptr(meta), _stream()),
           "slr_pack_2to4")
    return vals, meta


def pack_2to4_scaled(W: torch.Tensor, scale: torch.Tensor) -> tuple[torch.Tensor, torch.Tensor]:
    """Activation-aware 2:4 projection of bf16 ``W`` [d_out, d_in]: weights of
    column j ranked by |w| * |scale[j]| (fp32 ``scale`` [d_in])."""
    if W.dtype != torch.bfloat16 or W.dim() != 2 or not W.is_cuda or W.stride(1) != 1:
        raise ValueError("W must be a 2-D CUDA bf16 tensor with unit column stride")
    d_out, d_in = W.shape
    if scale.dtype != torch.float32 or scale.shape != (d_in,) or not scale.is_contiguous() or \
            scale.device != W.device:
        raise ValueError("scale must be a contiguous fp32 tensor of d_in elements on W's device")
    vals = torch.empty((d_out, d_in // 2), dtype=torch.bfloat16, device=W.device)
    meta = torch.empty((d_out, meta_row_bytes(d_in)), dtype=torch.uint8, device=W.device)
    _check(_lib.slr_pack_2to4_scaled(_ptr(W), d_out, d_in, W.stride(0), _ptr(scale), _ptr(vals), _ptr(meta),
                                     _stream()), "slr_pack_2to4_scaled")
    return vals, meta


def column_norms_workspace_size(M: int, d_in: int) -> int:
    return int(_lib.slr_column_norms_workspace_size(M, d_in))


def column_norms(X: torch.Tensor, sumsq: torch.Tensor | None = None, *, want_norms: bool = True,
                 workspace: torch.Tensor | None = None) -> tuple[torch.Tensor | None, torch.Tensor]:
    """Add the column sums of squares of bf16 ``X`` [M, d_in] to the fp64
    running sum ``sumsq`` (a new zero sum when None) and return
    ``(norms, sumsq)``, norms = fp32 sqrt(sumsq) (None unless ``want_norms``)."""
    if X.dtype != torch.bfloat16 or X.dim() != 2 or not X.is_cuda or (X.numel() > 0 and X.stride(1) != 1):
        raise ValueError("X must be a 2-D CUDA bf16 tensor with unit column stride")
    M, d_in = X.shape
    ldx = X.stride(0) if X.numel() > 0 else d_in
    if sumsq is None:
        sumsq = torch.zeros(d_in, dtype=torch.float64, device=X.device)
    elif sumsq.dtype != torch.float64 or sumsq.shape != (d_in,) or not sumsq.is_contiguous():
        raise ValueError("sumsq must be a contiguous fp64 tensor of d_in elements")
    norms = torch.empty(d_in, dtype=torch.float32, device=X.device) if want_norms else None
    need = column_norms_workspace_size(M, d_in)
    if workspace is None:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=X.device)
    _check(_lib.slr_column_norms(_ptr(X), M, d_in, ldx, _ptr(sumsq), _ptr(norms), _ptr(workspace),
                                 workspace.numel(), _stream()), "slr_column_norms")
    return norms, sumsq


def pack_2to8(W: torch.Tensor, *, dense: bool = True, as_2to4: bool = True):
    """2:8 projection of bf16 ``W`` [d_out, d_in]: returns ``(vals8, meta8,
    vals4, meta4)``, the dense 2:8 packing and the 2:4 packing of the same
    projected matrix (an unrequested pair is ``None``)."""
    if W.dtype != torch.bfloat16 or W.dim() != 2 or not W.is_cuda or W.stride(1) != 1:
        raise ValueError("W must be a 2-D CUDA bf16 tensor with unit column stride")
    d_out, d_in = W.shape
    dev = W.device
    vals8 = torch.empty((d_out, d_in // 4), dtype=torch.bfloat16, device=dev) if dense else None
    meta8 = torch.empty((d_out, d_in // 8), dtype=torch.uint8, device=dev) if dense else None
    vals4 = torch.empty((d_out, d_in // 2), dtype=torch.bfloat16, device=dev) if as_2to4 else None
    meta4 = torch.empty((d_out, meta_row_bytes(d_in)), dtype=torch.uint8, device=dev) if as_2to4 else None
    _check(_lib.slr_pack_2to8(_ptr(W), d_out, d_in, W.stride(0), _ptr(vals8), _ptr(meta8), _ptr(vals4),
                              _ptr(meta4), _stream()), "slr_pack_2to8")
    return vals8, meta8, vals4, meta4


def forward_2to8(X: torch.Tensor, vals8: torch.Tensor, meta8: torch.Tensor, U: torch.Tensor | None,
                 V: torch.Tensor | None, *, out: torch.Tensor | None = None,
                 workspace: torch.Tensor | None = None, vals4: torch.Tensor | None = None,
                 meta4: torch.Tensor | None = None) -> torch.Tensor:
    """``Y = X @ S.T + (X @ V.T) @ U.T`` with S in the dense 2:8 packing.

    The 2:8 streaming kernel is issue-bound and only pays at one token; given
    the 2:4 packing of the same matrix (``vals4``, ``meta4`` from
    :func:`pack_2to8`), calls with more than one token run ``slr_forward`` on
    it instead (the same product: a 2:8 pattern is a 2:4 pattern)."""
    M, d_in = X.shape
    d_out = vals8.shape[0]
    r = 0 if U is None else U.shape[1]
    if M > 1 and vals4 is not None and meta4 is not None:
        return forward(X, vals4, meta4, U, V, out=out, workspace=workspace)
    if out is None:
        out = torch.empty((M, d_out), dtype=torch.bfloat16, device=X.device)
    need = workspace_size(M, d_out, d_in, r)
    if workspace is None and need > 0:
        workspace = torch.empty(need, dtype=torch.uint8, device=X.device)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(_lib.slr_forward_2to8(_ptr(X), M, _ptr(vals8), _ptr(meta8), d_out, d_in, _ptr(U), _ptr(V), r,
                                 _ptr(out), _ptr(workspace), ws_bytes, _stream()), "slr_forward_2to8")
    return out


def lora_backward(X: torch.Tensor, dY: torch.Tensor, U: torch.Tensor, V: torch.Tensor,
                  T: torch.Tensor | None = None) -> tuple[torch.Tensor, torch.Tensor]:
    """Gradients of the layer w.r.t. U and V for upstream ``dY`` [M, d_out]:
    ``dU = dY^T (X V^T)`` (fp32 [d_out, r]), ``dV = (dY U)^T X`` (fp32 [r, d_in]).
    ``T`` is the forward's ``X V^T`` (bf16 [M, r]) if kept."""
    M, d_in = X.shape
    d_out = dY.shape[1]
    r = U.shape[1]
    dU = torch.empty((d_out, r), dtype=torch.float32, device=X.device)
    dV = torch.empty((r, d_in), dtype=torch.float32, device=X.device)
    need = int(_lib.slr_lora_backward_workspace_size(M, r))
    ws = torch.empty(max(need, 256), dtype=torch.uint8, device=X.device)
    _check(_lib.slr_lora_backward(_ptr(X), M, _ptr(dY), d_out, d_in, _ptr(U), _ptr(V), r, _ptr(T), _ptr(dU),
                                  _ptr(dV), _ptr(ws), ws.numel(), _stream()), "slr_lora_backward")
    return dU, dV


def decompose_datafree(W: torch.Tensor, r: int, iters: int, *, power_first: int = 8, power: int = 2,
                       Q0: torch.Tensor | None = None, seed: int = 0, factors_f32: bool = False):
    """Data-free alternating minimisation W ~ S + U V (S 2:4, rank r): returns
    ``(vals, meta, U, V, objective)`` with ``objective`` an fp64 CUDA tensor of
    ``iters + 1`` values.  ``Q0`` (fp32 [d_in, r]) is the random start of the
    subspace iteration; by default a standard normal one from ``seed``.  With
    ``factors_f32`` the fp32 factors before their rounding to bf16
    (``slr_decompose_factors_f32``) are appended: ``(..., U32, V32)``."""
    if W.dtype != torch.bfloat16 or W.dim() != 2 or not W.is_cuda or not W.is_contiguous():
        raise ValueError("W must be a contiguous 2-D CUDA bf16 tensor")
    d_out, d_in = W.shape
    dev = W.device
    if Q0 is None:
        g = torch.Generator(device=dev)
        g.manual_seed(seed)
        Q0 = torch.randn((d_in, r), generator=g, device=dev, dtype=torch.float32)
    vals = torch.empty((d_out, d_in // 2), dtype=torch.bfloat16, device=dev)
    meta = torch.empty((d_out, meta_row_bytes(d_in)), dtype=torch.uint8, device=dev)
    U = torch.empty((d_out, r), dtype=torch.bfloat16, device=dev)
    V = torch.empty((r, d_in), dtype=torch.bfloat16, device=dev)
    obj = torch.empty(iters + 1, dtype=torch.float64, device=dev)
    need = int(_lib.slr_decompose_workspace_size(d_out, d_in, r))
    ws = torch.empty(max(need, 256), dtype=torch.uint8, device=dev)
    _check(_lib.slr_decompose_datafree(_ptr(W), d_out, d_in, r, iters, power_first, power, _ptr(Q0), _ptr(vals),
                                       _ptr(meta), _ptr(U), _ptr(V), _ptr(obj), _ptr(ws), ws.numel(), _stream()),
           "slr_decompose_datafree")
    if not factors_f32:
        return vals, meta, U, V, obj
    U32 = torch.empty((d_out, r), dtype=torch.float32, device=dev)
    V32 = torch.empty((r, d_in), dtype=torch.float32, device=dev)
    _check(_lib.slr_decompose_factors_f32(_ptr(ws), ws.numel(), d_out, d_in, r, _ptr(U32), _ptr(V32), _stream()),
           "slr_decompose_factors_f32")
    return vals, meta, U, V, obj, U32, V32


def workspace_size(M: int, d_out: int, d_in: int, r: int) -> int:
    return int(_lib.slr_forward_workspace_size(M, d_out, d_in, r))


def select_path(M: int, d_out: int, d_in: int, r: int) -> str:
    return PATH_NAMES[int(_lib.slr_forward_select_path(M, d_out, d_in, r))]


FWD_OVERLAP_PRECEDING = 1


def forward(X: torch.Tensor, vals: torch.Tensor, meta: torch.Tensor, U: torch.Tensor | None,
            V: torch.Tensor | None, *, path: str = "auto", out: torch.Tensor | None = None,
            workspace: torch.Tensor | None = None, overlap_preceding: bool = False) -> torch.Tensor:
    """``Y = X @ S.T + (X @ V.T) @ U.T`` with S given packed by ``pack_2to4``.

    ``overlap_preceding`` sets ``SLR_FWD_OVERLAP_PRECEDING`` (``slr_forward_ex``):
    the call may start reading its weights while the kernel queued just before
    it is still running, which that kernel must not write."""
    M, d_in = X.shape
    d_out = vals.shape[0]
    r = 0 if U is None else U.shape[1]
    if out is None:
        out = torch.empty((M, d_out), dtype=torch.bfloat16, device=X.device)
    need = workspace_size(M, d_out, d_in, r)
    if workspace is None and need > 0:
        workspace = torch.empty(need, dtype=torch.uint8, device=X.device)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    flags = FWD_OVERLAP_PRECEDING if overlap_preceding else 0
    _check(_lib.slr_forward_ex(_ptr(X), M, _ptr(vals), _ptr(meta), d_out, d_in, _ptr(U), _ptr(V), r,
                               _ptr(out), _ptr(workspace), ws_bytes, PATHS[path], flags, _stream()),
           "slr_forward")
    return out


def forward_epilogue(X: torch.Tensor, vals: torch.Tensor, meta: torch.Tensor, U: torch.Tensor | None,
                     V: torch.Tensor | None, *, bias: torch.Tensor | None = None, act: str = "none",
                     residual: torch.Tensor | None = None, preact: torch.Tensor | None = None, path: str = "auto",
                     out: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                     overlap_preceding: bool = False) -> torch.Tensor:
    """``Y = act(X @ S.T + (X @ V.T) @ U.T + bias) + residual`` in the kernels of
    :func:`forward` (``slr_forward_epilogue``).

    ``bias`` is bf16 [d_out], ``act`` one of :data:`ACTS`, ``residual`` bf16
    [M, d_out] with unit column stride (its rows may be a slice of wider ones;
    ``out`` itself updates it in place).  ``preact`` (bf16 [M, d_out]) receives
    the pre-activation for :func:`epilogue_backward`.  The workspace is
    :func:`forward`'s (:func:`workspace_size`)."""
    if X.dim() != 2 or act not in ACTS:
        raise ValueError(f"X must be 2-D and act one of {', '.join(ACTS)}")
    device, stream = _current(X)
    M = X.shape[0]
    d_out, d_in, r = _expect_layer(vals, meta, U, V, device)
    _expect("X", X, torch.bfloat16, (M, d_in), device)
    if out is None:
        out = torch.empty((M, d_out), dtype=torch.bfloat16, device=device)
    else:
        _expect("out", out, torch.bfloat16, (M, d_out), device)
    if bias is not None:
        _expect("bias", bias, torch.bfloat16, (d_out,), device)
    if preact is not None:
        _expect("preact", preact, torch.bfloat16, (M, d_out), device)
    ldr = d_out
    if residual is not None:
        if residual.dtype is not torch.bfloat16 or residual.shape != (M, d_out) or residual.device != device or \
                (d_out > 1 and residual.stride(1) != 1):
            raise ValueError(f"residual must be a bf16 tensor of shape {(M, d_out)} on {device} with unit column stride")
        if M > 1:
            ldr = residual.stride(0)
    # The library checks a given workspace's size; only a new one needs to know it here.
    workspace, ws_bytes = _scratch(workspace, 0 if workspace is not None else workspace_size(M, d_out, d_in, r), device)
    _check(_lib.slr_forward_epilogue(X.data_ptr(), M, vals.data_ptr(), meta.data_ptr(), d_out, d_in, _addr(U), _addr(V),
                                     r, _addr(bias), ACTS[act], _addr(residual), ldr, _addr(preact), out.data_ptr(),
                                     _addr(workspace), ws_bytes, PATHS[path],
                                     FWD_OVERLAP_PRECEDING if overlap_preceding else 0, stream),
           "slr_forward_epilogue")
    return out


def epilogue_backward(dY: torch.Tensor, Z: torch.Tensor | None, act: str, *, want_dbias: bool = True,
                      out: torch.Tensor | None = None) -> tuple[torch.Tensor, torch.Tensor | None]:
    """``(dZ, dbias)`` of :func:`forward_epilogue` for upstream ``dY`` [M, d_out]
    (``slr_epilogue_backward``): ``dZ = dY * act'(Z)`` (bf16) and its column
    sums (fp32 [d_out]; None unless ``want_dbias``).  ``out`` receives dZ and
    may be ``dY`` or ``Z``.  Without an activation the gradient passes
    unchanged: ``dY`` itself is returned when no ``out`` is given."""
    if dY.dim() != 2 or act not in ACTS:
        raise ValueError(f"dY must be 2-D and act one of {', '.join(ACTS)}")
    device, stream = _current(dY)
    shape = dY.shape
    _expect("dY", dY, torch.bfloat16, shape, device)
    if act != "none":
        if Z is None:
            raise ValueError("an activation's gradient needs the pre-activation Z")
        _expect("Z", Z, torch.bfloat16, shape, device)
    if out is not None:
        _expect("out", out, torch.bfloat16, shape, device)
    elif act != "none":
        out = torch.empty_like(dY)
    elif not want_dbias:
        return dY, None
    dbias = torch.empty(shape[1], dtype=torch.float32, device=device) if want_dbias else None
    _check(_lib.slr_epilogue_backward(dY.data_ptr(), _addr(Z) if act != "none" else None, shape[0], shape[1], ACTS[act],
                                      _addr(out), _addr(dbias), stream), "slr_epilogue_backward")
    return (dY if out is None else out), dbias


def input_backward_workspace_size(M: int, d_out: int, d_in: int, r: int) -> int:
    return int(_lib.slr_input_backward_workspace_size(M, d_out, d_in, r))


def input_backward(dY: torch.Tensor, vals: torch.Tensor, meta: torch.Tensor, U: torch.Tensor | None,
                   V: torch.Tensor | None, *, out: torch.Tensor | None = None,
                   workspace: torch.Tensor | None = None) -> torch.Tensor:
    """Gradient of the layer's input for upstream ``dY`` [M, d_out]:
    ``dX = dY @ S + (dY @ U) @ V`` (bf16 [M, d_in]; ``slr_input_backward``)."""
    if dY.dim() != 2:
        raise ValueError("dY must be 2-D")
    device, stream = _current(dY)
    M = dY.shape[0]
    d_out, d_in, r = _expect_layer(vals, meta, U, V, device)
    _expect("dY", dY, torch.bfloat16, (M, d_out), device)
    if out is None:
        out = torch.empty((M, d_in), dtype=torch.bfloat16, device=device)
    else:
        _expect("out", out, torch.bfloat16, (M, d_in), device)
    workspace, ws_bytes = _scratch(
        workspace, 0 if workspace is not None else input_backward_workspace_size(M, d_out, d_in, r), device)
    _check(_lib.slr_input_backward(dY.data_ptr(), M, vals.data_ptr(), meta.data_ptr(), d_out, d_in, _addr(U), _addr(V), r,
                                   out.data_ptr(), _addr(workspace), ws_bytes, stream), "slr_input_backward")
    return out


def _expect_logits(name: str, t: torch.Tensor, shape: tuple, device: torch.device) -> int:
    """Leading dimension of bf16 logits, whose rows may be a slice of wider (padded) ones."""
    if t.dtype is not torch.bfloat16 or t.shape != shape or t.device != device or (shape[1] > 1 and t.stride(1) != 1):
        raise ValueError(f"{name} must be a bf16 tensor of shape {tuple(shape)} on {device} with unit column stride")
    return t.stride(0) if shape[0] > 1 else shape[1]


def _distill_operands(logits: torch.Tensor, idx: torch.Tensor, teacher: torch.Tensor):
    if logits.dim() != 2 or idx.dim() != 2:
        raise ValueError("logits and idx must be 2-D")
    device, stream = _current(logits)
    (M, n), k = logits.shape, idx.shape[1]
    ldz = _expect_logits("logits", logits, (M, n), device)
    _expect("idx", idx, torch.int32, (M, k), device)
    _expect("teacher", teacher, torch.float32, (M, k), device)
    return device, stream, M, n, k, ldz


def distill_forward(logits: torch.Tensor, idx: torch.Tensor, teacher: torch.Tensor, *,
                    tau: float = 1.0) -> tuple[torch.Tensor, torch.Tensor]:
    """``(loss, lse)`` per token (fp32 [M]) of bf16 student ``logits`` [M, n_vocab]
    against a teacher's top logits: columns ``idx`` (int32 [M, k], -1 where there
    is none) and values ``teacher`` (fp32 [M, k]) at temperature ``tau``
    (``slr_distill_forward``): tau^2 KL(p || softmax(logits / tau)), p the softmax
    of the listed teacher logits."""
    device, stream, M, n, k, ldz = _distill_operands(logits, idx, teacher)
    loss = torch.empty(M, dtype=torch.float32, device=device)
    lse = torch.empty(M, dtype=torch.float32, device=device)
    _check(_lib.slr_distill_forward(logits.data_ptr(), M, n, ldz, idx.data_ptr(), teacher.data_ptr(), k, tau,
                                    loss.data_ptr(), lse.data_ptr(), stream), "slr_distill_forward")
    return loss, lse


def distill_backward(logits: torch.Tensor, idx: torch.Tensor, teacher: torch.Tensor, lse: torch.Tensor,
                     dloss: torch.Tensor, *, tau: float = 1.0, out: torch.Tensor | None = None) -> torch.Tensor:
    """Gradient of :func:`distill_forward`'s losses with respect to the logits
    (bf16) for the upstream ``dloss`` (fp32 [M]), from the forward's ``lse``
    (``slr_distill_backward``; where ``|lse|`` exceeds 64 the row's statistics are
    formed again from its logits).  ``out`` may be ``logits`` itself."""
    device, stream, M, n, k, ldz = _distill_operands(logits, idx, teacher)
    _expect("lse", lse, torch.float32, (M,), device)
    _expect("dloss", dloss, torch.float32, (M,), device)
    if out is None:
        out = torch.empty((M, n), dtype=torch.bfloat16, device=device)
    lddz = _expect_logits("out", out, (M, n), device)
    _check(_lib.slr_distill_backward(logits.data_ptr(), M, n, ldz, idx.data_ptr(), teacher.data_ptr(), k, tau,
                                     lse.data_ptr(), dloss.data_ptr(), out.data_ptr(), lddz, stream),
           "slr_distill_backward")
    return out


def distill_loss_grad(logits: torch.Tensor, idx: torch.Tensor, teacher: torch.Tensor, dloss: torch.Tensor, *,
                      tau: float = 1.0, out: torch.Tensor | None = None) -> tuple[torch.Tensor, torch.Tensor]:
    """``(loss, dlogits)`` of :func:`distill_forward` and :func:`distill_backward`
    in one call, for weights ``dloss`` known beforehand
    (``slr_distill_loss_grad``).  ``out`` may be ``logits`` itself."""
    device, stream, M, n, k, ldz = _distill_operands(logits, idx, teacher)
    _expect("dloss", dloss, torch.float32, (M,), device)
    loss = torch.empty(M, dtype=torch.float32, device=device)
    if out is None:
        out = torch.empty((M, n), dtype=torch.bfloat16, device=device)
    lddz = _expect_logits("out", out, (M, n), device)
    _check(_lib.slr_distill_loss_grad(logits.data_ptr(), M, n, ldz, idx.data_ptr(), teacher.data_ptr(), k, tau,
                                      dloss.data_ptr(), loss.data_ptr(), out.data_ptr(), lddz, stream),
           "slr_distill_loss_grad")
    return loss, out


def forward_project(X: torch.Tensor, V: torch.Tensor | None, d_out: int, workspace: torch.Tensor, *,
                    path: str = "auto") -> None:
    """Stage 1 of ``forward``: T = X V^T into ``workspace`` (``slr_forward_project``)."""
    M, d_in = X.shape
    r = 0 if V is None else V.shape[0]
    _check(_lib.slr_forward_project(_ptr(X), M, _ptr(V), d_out, d_in, r, _ptr(workspace),
                                    workspace.numel() * workspace.element_size(), PATHS[path], _stream()),
           "slr_forward_project")


def forward_combine(X: torch.Tensor, vals: torch.Tensor, meta: torch.Tensor, U: torch.Tensor | None,
                    out: torch.Tensor, workspace: torch.Tensor | None, *, path: str = "auto") -> torch.Tensor:
    """Stage 2 of ``forward``: Y = X S^T + T U^T with T from ``workspace``."""
    M, d_in = X.shape
    d_out = vals.shape[0]
    r = 0 if U is None else U.shape[1]
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(_lib.slr_forward_combine(_ptr(X), M, _ptr(vals), _ptr(meta), d_out, d_in, _ptr(U), r, _ptr(out),
                                    _ptr(workspace), ws_bytes, PATHS[path], _stream()),
           "slr_forward_combine")
    return out


NOALLOC_MAX_T_ELEMS = 16384


def forward_decode_noalloc(X: torch.Tensor, vals: torch.Tensor, meta: torch.Tensor, U: torch.Tensor | None,
                           V: torch.Tensor | None, out: torch.Tensor) -> torch.Tensor:
    """Small-M forward for callers that cannot allocate device memory
    (``slr_forward_decode_noalloc``): no workspace; the rank projection lives in
    a fixed array inside the library (M * r <= NOALLOC_MAX_T_ELEMS).  ``out``
    must be provided."""
    M, d_in = X.shape
    d_out = vals.shape[0]
    r = 0 if U is None else U.shape[1]
    _check(_lib.slr_forward_decode_noalloc(_ptr(X), M, _ptr(vals), _ptr(meta), d_out, d_in, _ptr(U), _ptr(V), r,
                                           _ptr(out), _stream()),
           "slr_forward_decode_noalloc")
    return out


def check_kernel_error() -> None:
    """Synchronise and raise if a tensor-core kernel reported a bounded-wait timeout."""
    _check(_lib.slr_check_kernel_error(), "slr_check_kernel_error")


def selftest_wait_timeout(limit_cycles: int = 2_000_000) -> None:
    """Launch the failure-detection self-test (``slr_selftest_wait_timeout``): a
    bounded wait that expires after ``limit_cycles`` SM cycles and records a
    timeout that the next :func:`check_kernel_error` raises."""
    _check(_lib.slr_selftest_wait_timeout(int(limit_cycles), _stream()), "slr_selftest_wait_timeout")
