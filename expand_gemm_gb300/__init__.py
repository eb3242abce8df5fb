"""GB300 (sm_103a) multi-LoRA shrink/expand: thin PyTorch binding.

Every step runs in the CUDA kernels of ``liblora_punica.so`` (C ABI in
``include/lora_punica.h``); this module only checks tensor dtypes and
layouts, collects device pointers and the current CUDA stream, and calls the
library.  PyTorch provides device memory and streams, nothing else.  There
is no CPU fallback: without the built library every call raises.

Names follow vLLM's API pages:

* :class:`LoRAKernelMeta` -- page ``vllm.lora.ops.triton_ops.lora_kernel_metadata``
  (``make``, ``prepare_tensors``, ``meta_args``; ``no_lora`` is the host copy of
  the flag, the page's ``no_lora_flag_cpu``).
* :func:`lora_shrink`, :func:`lora_expand`, :func:`add_lora_linear`,
  :func:`add_lora_embedding`, :func:`add_lora_logits` -- page
  ``vllm.lora.punica_wrapper.punica_gpu`` (``PunicaWrapperGPU.add_shrink``,
  ``add_expand``, ``add_lora_linear``, ``add_lora_embedding``,
  ``add_lora_logits``).
"""
from __future__ import annotations

import ctypes
import math
from typing import Optional, Sequence

import torch

from . import _lib
from ._lib import (LoraError, LORA_MAX_LORAS, LORA_MAX_RANK, LORA_MAX_SLICES,  # noqa: F401
                   LORA_NOALLOC_MAX_FLOATS)

__all__ = ["LoRAKernelMeta", "lora_meta_prepare", "lora_shrink", "lora_expand",
           "lora_linear", "lora_linear_noalloc", "add_lora_linear", "add_lora_embedding",
           "add_lora_logits", "lora_cross_entropy", "lora_cross_entropy_workspace",
           "lora_linear_backward", "lora_linear_backward_workspace",
           "lora_orthogonalize", "lora_orthogonalize_workspace",
           "lora_expert_linear", "lora_expert_linear_workspace",
           "lora_expert_linear_backward", "lora_expert_linear_backward_workspace",
           "lora_quantize_mxfp4", "lora_dequantize_mxfp4", "LoRAGradients", "lora_clip_gradients",
           "reload_options", "LoraError", "library", "build"]


def library():
    """The loaded ctypes library (raises if it is not built)."""
    return _lib.load()


def build(force: bool = False) -> str:
    from .build import build as _build
    return _build(force=force)


def reload_options() -> None:
    """Re-read the LORA_PUNICA_* tuning variables (the library reads them
    once, at its first call): ``lora_reload_options``."""
    _lib.load().lora_reload_options()


def _stream_handle(device: torch.device) -> int:
    return torch.cuda.current_stream(device).cuda_stream


def _need(t: torch.Tensor, name: str, dtype: torch.dtype) -> None:
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    if not t.is_cuda:
        raise ValueError("%s must be a CUDA tensor (no CPU path exists)" % name)
    if t.dtype != dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))


def _same_device(meta: "LoRAKernelMeta", named) -> None:
    """Every tensor of ``named`` ((name, tensor or None) pairs) must be on
    the GPU that holds the metadata: the kernels take raw pointers, so a
    tensor on another device would be read through the wrong address space."""
    dev = meta.no_lora_flag.get_device()
    for name, t in named:
        if t is not None and t.get_device() != dev:
            raise ValueError("%s is on cuda:%d, the metadata on cuda:%d"
                             % (name, t.get_device(), dev))


def _call(fn: str, device: torch.device, *args) -> None:
    """Calls library entry point `fn` with `device` current (the library
    looks up per-device state for the current device), then raises on a
    non-zero status."""
    f = getattr(_lib.load(), fn)
    if device.index is None or device.index == torch.cuda.current_device():
        st = f(*args)
    else:
        with torch.cuda.device(device):
            st = f(*args)
    if st:
        _lib.check(fn, st)


def _ptr_array(tensors) -> ctypes.Array:
    arr = (ctypes.c_void_p * len(tensors))()
    for i, t in enumerate(tensors):
        arr[i] = None if t is None else t.data_ptr()
    return arr


class LoRAKernelMeta:
    """Per-forward metadata buffers (LoRAKernelMeta of the metadata page).

    Buffers are int32 device tensors allocated once by :meth:`make`; the
    no-LoRA flag lives on the device (the kernels read it there, so no host
    sync is needed; :meth:`no_lora` copies it to the host on request);
    ``error_word`` counts ids outside ``[-1, max_loras)`` seen by the last
    :meth:`prepare_tensors`.
    """

    def __init__(self, max_loras: int, max_num_tokens: int, device):
        if not 1 <= max_loras <= LORA_MAX_LORAS:
            raise ValueError("max_loras must be in [1, %d]" % LORA_MAX_LORAS)
        if max_num_tokens < 0:
            raise ValueError("max_num_tokens must be >= 0")
        dev = torch.device(device)
        i32 = dict(dtype=torch.int32, device=dev)
        self.max_loras = int(max_loras)
        self.max_num_tokens = int(max_num_tokens)
        self.token_lora_mapping = torch.empty(max(max_num_tokens, 1), **i32)
        self.token_indices_sorted_by_lora_ids = torch.empty(max(max_num_tokens, 1), **i32)
        self.active_lora_ids = torch.full((max_loras + 1,), -1, **i32)
        self.num_tokens_per_lora = torch.zeros(max_loras + 1, **i32)
        self.lora_token_start_loc = torch.zeros(max_loras + 2, **i32)
        self.no_lora_flag = torch.ones(1, **i32)
        self.error_word = torch.zeros(1, **i32)
        # grid barrier of lora_linear's single-kernel path (left zero by every call)
        self.grid_sync = torch.zeros(2, **i32)
        self.c = _lib.LoraMetaC(
            self.token_lora_mapping.data_ptr(),
            self.token_indices_sorted_by_lora_ids.data_ptr(),
            self.num_tokens_per_lora.data_ptr(),
            self.lora_token_start_loc.data_ptr(),
            self.active_lora_ids.data_ptr(),
            self.no_lora_flag.data_ptr(),
            self.error_word.data_ptr(),
            self.max_loras, self.max_num_tokens,
            self.grid_sync.data_ptr())
        self.device = dev

    @staticmethod
    def make(max_loras: int, max_num_tokens: int, device) -> "LoRAKernelMeta":
        return LoRAKernelMeta(max_loras, max_num_tokens, device)

    def prepare_tensors(self, token_lora_mapping: torch.Tensor) -> None:
        lora_meta_prepare(token_lora_mapping, self)

    def meta_args(self, token_nums: int):
        """The six metadata tensors in the order the kernels take them."""
        return (self.token_lora_mapping[:token_nums],
                self.token_indices_sorted_by_lora_ids[:token_nums],
                self.num_tokens_per_lora, self.lora_token_start_loc,
                self.active_lora_ids, self.no_lora_flag)

    def no_lora(self) -> bool:
        """Host read of the flag through ``lora_meta_read_no_lora``
        (synchronises the current stream; the kernels never need it)."""
        out = ctypes.c_int32(-1)
        _call("lora_meta_read_no_lora", self.device, ctypes.byref(self.c),
              _stream_handle(self.device), ctypes.byref(out))
        return bool(out.value)


def lora_meta_prepare(token_lora_mapping: torch.Tensor, meta: LoRAKernelMeta) -> None:
    m = token_lora_mapping
    _need(m, "token_lora_mapping", torch.int32)
    if m.dim() != 1 or not m.is_contiguous():
        raise ValueError("token_lora_mapping must be a contiguous 1-D tensor")
    _same_device(meta, [("token_lora_mapping", m)])
    _call("lora_meta_prepare", meta.device, m.data_ptr() if m.numel() else None, m.numel(),
          ctypes.byref(meta.c), _stream_handle(meta.device))


def _weights(ws: Sequence[torch.Tensor], name: str):
    if isinstance(ws, torch.Tensor):
        ws = (ws,)
    out = []
    for i, w in enumerate(ws):
        _need(w, "%s[%d]" % (name, i), torch.bfloat16)
        if not w.is_contiguous():
            raise ValueError("%s[%d] must be contiguous" % (name, i))
        if w.dim() == 4 and w.size(1) == 1:          # [L, 1, rows, cols] layer dim
            w = w.view(w.size(0), w.size(2), w.size(3))
        if w.dim() != 3:
            raise ValueError("%s[%d] must be [max_loras, rows, cols]" % (name, i))
        out.append(w)
    return out


def lora_shrink(x: torch.Tensor, lora_a_stacked, y: torch.Tensor,
                meta: LoRAKernelMeta, scale: float) -> None:
    """y[s] += scale * x @ lora_a_stacked[s][id]^T for tokens with a LoRA."""
    _need(x, "x", torch.bfloat16)
    _need(y, "y", torch.float32)
    x2 = x.view(-1, x.shape[-1]) if x.dim() != 2 else x
    if x2.stride(1) != 1:
        raise ValueError("x rows must be contiguous")
    A = _weights(lora_a_stacked, "lora_a_stacked")
    T, H = x2.shape
    L, r, Ha = A[0].shape
    if Ha != H or any(a.shape != A[0].shape for a in A):
        raise ValueError("lora_a_stacked shapes must all be [L, r, %d]" % H)
    if L < meta.max_loras:
        raise ValueError("lora_a_stacked has %d LoRAs, metadata expects %d" % (L, meta.max_loras))
    if tuple(y.shape) != (len(A), T, r) or not y.is_contiguous():
        raise ValueError("y must be a contiguous fp32 [%d, %d, %d] tensor" % (len(A), T, r))
    _same_device(meta, [("x", x), ("y", y)] +
                 [("lora_a_stacked[%d]" % i, a) for i, a in enumerate(A)])
    _call("lora_shrink", x.device, x2.data_ptr(), T, H, x2.stride(0), _ptr_array(A), len(A), r,
          y.data_ptr(), ctypes.byref(meta.c), float(scale), _stream_handle(x.device))


def lora_expand(x: torch.Tensor, lora_b_stacked, y: torch.Tensor,
                meta: LoRAKernelMeta, offset_start: int = 0, add_inputs: bool = True,
                lora_bias_stacked: Optional[Sequence[Optional[torch.Tensor]]] = None) -> None:
    """y[:, off_s:off_s+n_s] (+)= x[s] @ lora_b_stacked[s][id]^T (+ bias).

    x is fp32 (the shrink's buffer; rounded to bf16 for the tensor cores) or
    bf16 (taken as it is: lora_expand_bf16)."""
    if not isinstance(x, torch.Tensor) or x.dtype not in (torch.float32, torch.bfloat16):
        raise TypeError("x must be a float32 or bfloat16 torch.Tensor")
    _need(x, "x", x.dtype)
    _need(y, "y", torch.bfloat16)
    B = _weights(lora_b_stacked, "lora_b_stacked")
    if x.dim() != 3 or not x.is_contiguous() or x.size(0) != len(B):
        raise ValueError("x must be a contiguous [num_slices, T, r] tensor")
    S, T, r = x.shape
    L = B[0].size(0)
    if L < meta.max_loras:
        raise ValueError("lora_b_stacked has %d LoRAs, metadata expects %d" % (L, meta.max_loras))
    for i, b in enumerate(B):
        if b.size(0) != L or b.size(2) != r:
            raise ValueError("lora_b_stacked[%d] must be [%d, n, %d]" % (i, L, r))
    sizes = [b.size(1) for b in B]
    y2 = y.view(-1, y.shape[-1]) if y.dim() != 2 else y
    if y2.stride(1) != 1 or y2.size(0) != T:
        raise ValueError("y must be [T, width] with contiguous rows")
    bias_arr = None
    if lora_bias_stacked is not None:
        if len(lora_bias_stacked) != S:
            raise ValueError("lora_bias_stacked needs one entry per slice")
        bl = []
        for i, (bb, n) in enumerate(zip(lora_bias_stacked, sizes)):
            if bb is None:
                bl.append(None)
                continue
            _need(bb, "lora_bias_stacked[%d]" % i, torch.bfloat16)
            if not bb.is_contiguous() or bb.numel() != L * n:
                raise ValueError("lora_bias_stacked[%d] must be [%d, %d]" % (i, L, n))
            bl.append(bb)
        bias_arr = _ptr_array(bl)
    biases = () if lora_bias_stacked is None else lora_bias_stacked
    _same_device(meta, [("x", x), ("y", y)] +
                 [("lora_b_stacked[%d]" % i, b) for i, b in enumerate(B)] +
                 [("lora_bias_stacked[%d]" % i, b) for i, b in enumerate(biases)])
    size_arr = (ctypes.c_int32 * S)(*sizes)
    fn = "lora_expand_bf16" if x.dtype == torch.bfloat16 else "lora_expand"
    _call(fn, x.device, x.data_ptr(), _ptr_array(B), bias_arr, size_arr, S, r,
          y2.data_ptr(), y2.stride(0), T, int(offset_start), 1 if add_inputs else 0,
          ctypes.byref(meta.c), _stream_handle(x.device))


def add_lora_embedding(y: torch.Tensor, x: torch.Tensor, lora_b_stacked,
                       meta: LoRAKernelMeta, add_inputs: bool = True) -> None:
    """PunicaWrapperGPU.add_lora_embedding: y (+)= x @ lora_b_stacked[id]^T,
    where x is bf16 [T, r] (the embedding LoRA's A rows looked up per
    token) and add_inputs is passed through."""
    _need(x, "x", torch.bfloat16)
    x2 = x.view(-1, x.shape[-1])
    lora_expand(x2.unsqueeze(0), lora_b_stacked, y, meta, 0, add_inputs)


def add_lora_logits(y: torch.Tensor, x: torch.Tensor, lora_a_stacked, lora_b_stacked,
                    scale: float, meta: LoRAKernelMeta, *,
                    buffer: Optional[torch.Tensor] = None) -> None:
    """PunicaWrapperGPU.add_lora_logits: buffer = scale * x @ A[id]^T, then
    y += buffer @ B[id]^T, both driven by ``meta`` (the prompt/sampler
    metadata instance, one id per logits row)."""
    y2 = y.view(-1, y.shape[-1])
    x2 = x.view(-1, x.shape[-1])
    B = _weights(lora_b_stacked, "lora_b_stacked")
    if len(B) != 1:
        raise ValueError("add_lora_logits takes one lora_b tensor")
    r = B[0].size(-1)
    if buffer is None:
        buffer = torch.zeros((x2.size(0), r), dtype=torch.float32, device=x.device)
    lora_shrink(x2, lora_a_stacked, buffer.unsqueeze(0), meta, scale)
    lora_expand(buffer.unsqueeze(0), B, y2, meta, 0, True)


def add_lora_linear(y: torch.Tensor, x: torch.Tensor, lora_a_stacked, lora_b_stacked,
                    lora_bias_stacked, scale: float, output_slices, meta: LoRAKernelMeta,
                    *, buffer: Optional[torch.Tensor] = None) -> None:
    """PunicaWrapperGPU.add_lora_linear: shrink into an fp32 buffer, then
    expand into y with the bias fused into the expand kernel."""
    A = _weights(lora_a_stacked, "lora_a_stacked")
    B = _weights(lora_b_stacked, "lora_b_stacked")
    if not len(A) == len(B) == len(output_slices):
        raise ValueError("lora_a_stacked, lora_b_stacked and output_slices differ in length")
    if lora_bias_stacked is not None and len(lora_bias_stacked) != len(output_slices):
        raise ValueError("lora_bias_stacked needs one entry per slice")
    for b, n in zip(B, output_slices):
        if b.size(1) != n:
            raise ValueError("lora_b_stacked widths must match output_slices")
    x2 = x.view(-1, x.shape[-1])
    r = B[0].size(-1)
    if buffer is None:
        buffer = torch.zeros((len(output_slices), x2.size(0), r), dtype=torch.float32,
                             device=x.device)
    lora_shrink(x2, A, buffer, meta, scale)
    lora_expand(buffer, B, y, meta, 0, True, lora_bias_stacked)


def _linear_args(token_lora_mapping, x, lora_a_stacked, lora_b_stacked, lora_bias_stacked,
                 buffer, y):
    """Checks shared by lora_linear and lora_linear_noalloc; returns the
    marshalled C arguments in lora_linear's order (buffer pointer None when
    no buffer is given)."""
    m = token_lora_mapping
    _need(m, "token_lora_mapping", torch.int32)
    _need(x, "x", torch.bfloat16)
    _need(y, "y", torch.bfloat16)
    x2 = x.view(-1, x.shape[-1]) if x.dim() != 2 else x
    y2 = y.view(-1, y.shape[-1]) if y.dim() != 2 else y
    A = _weights(lora_a_stacked, "lora_a_stacked")
    B = _weights(lora_b_stacked, "lora_b_stacked")
    T, H = x2.shape
    if m.dim() != 1 or m.numel() != T or not m.is_contiguous():
        raise ValueError("token_lora_mapping must be a contiguous [T] tensor")
    if x2.stride(1) != 1 or y2.stride(1) != 1 or y2.size(0) != T:
        raise ValueError("x and y need contiguous rows and T rows")
    if len(A) != len(B):
        raise ValueError("lora_a_stacked and lora_b_stacked differ in length")
    L, r, Ha = A[0].shape
    if Ha != H or any(a.shape != A[0].shape for a in A):
        raise ValueError("lora_a_stacked shapes must all be [L, r, %d]" % H)
    for i, b in enumerate(B):
        if b.size(0) != B[0].size(0) or b.size(2) != r:
            raise ValueError("lora_b_stacked[%d] must be [%d, n, %d]" % (i, B[0].size(0), r))
    if buffer is not None:
        _need(buffer, "buffer", torch.float32)
        if tuple(buffer.shape) != (len(A), T, r) or not buffer.is_contiguous():
            raise ValueError("buffer must be a contiguous fp32 [%d, %d, %d] tensor"
                             % (len(A), T, r))
    sizes = [b.size(1) for b in B]
    bias_arr = None
    if lora_bias_stacked is not None:
        if len(lora_bias_stacked) != len(B):
            raise ValueError("lora_bias_stacked needs one entry per slice")
        for i, (bb, n) in enumerate(zip(lora_bias_stacked, sizes)):
            if bb is not None:
                _need(bb, "lora_bias_stacked[%d]" % i, torch.bfloat16)
                if not bb.is_contiguous() or bb.numel() != B[0].size(0) * n:
                    raise ValueError("lora_bias_stacked[%d] must be [L, %d]" % (i, n))
        bias_arr = _ptr_array(list(lora_bias_stacked))
    size_arr = (ctypes.c_int32 * len(B))(*sizes)
    named = ([("token_lora_mapping", m), ("x", x), ("y", y), ("buffer", buffer)] +
             [("lora_a_stacked[%d]" % i, a) for i, a in enumerate(A)] +
             [("lora_b_stacked[%d]" % i, b) for i, b in enumerate(B)] +
             [("lora_bias_stacked[%d]" % i, b)
              for i, b in enumerate(() if lora_bias_stacked is None else lora_bias_stacked)])
    return dict(L=L, nb=B[0].size(0), named=named,
                head=(m.data_ptr(), T, x2.data_ptr(), H, x2.stride(0), _ptr_array(A),
                      _ptr_array(B), bias_arr, size_arr, len(B), r),
                buf=None if buffer is None else buffer.data_ptr(),
                tail=(y2.data_ptr(), y2.stride(0)))


def lora_linear(token_lora_mapping: torch.Tensor, x: torch.Tensor, lora_a_stacked,
                lora_b_stacked, lora_bias_stacked, scale: float, buffer: torch.Tensor,
                y: torch.Tensor, meta: LoRAKernelMeta) -> None:
    """Metadata + shrink + expand of one LoRA layer in one library call
    (PunicaWrapperGPU.update_metadata followed by add_lora_linear).  Small
    batches run as one kernel, larger ones as three overlapping launches;
    see include/lora_punica.h."""
    if not isinstance(buffer, torch.Tensor):
        raise TypeError("buffer must be a torch.Tensor (lora_linear_noalloc needs none)")
    a = _linear_args(token_lora_mapping, x, lora_a_stacked, lora_b_stacked, lora_bias_stacked,
                     buffer, y)
    if a["L"] < meta.max_loras or a["nb"] < meta.max_loras:
        raise ValueError("weights hold fewer LoRAs than the metadata expects")
    _same_device(meta, a["named"])
    _call("lora_linear", x.device, *a["head"], float(scale), a["buf"], *a["tail"],
          ctypes.byref(meta.c), _stream_handle(x.device))


def lora_linear_noalloc(token_lora_mapping: torch.Tensor, x: torch.Tensor, lora_a_stacked,
                        lora_b_stacked, lora_bias_stacked, scale: float, y: torch.Tensor,
                        meta: LoRAKernelMeta) -> None:
    """lora_linear without a caller buffer: the fp32 intermediate lives in a
    fixed array the library owns on each device (at most
    LORA_NOALLOC_MAX_FLOATS = slices x tokens x rank floats), cleared by each
    call, so no device memory is allocated.  Calls on one device share that
    array and must not overlap; see include/lora_punica.h."""
    a = _linear_args(token_lora_mapping, x, lora_a_stacked, lora_b_stacked, lora_bias_stacked,
                     None, y)
    if a["L"] < meta.max_loras or a["nb"] < meta.max_loras:
        raise ValueError("weights hold fewer LoRAs than the metadata expects")
    _same_device(meta, a["named"])
    _call("lora_linear_noalloc", x.device, *a["head"], float(scale), *a["tail"],
          ctypes.byref(meta.c), _stream_handle(x.device))


# ------------------------------------------------------------ training the adapters
#
# In a small batch the checks cost more than the kernels (64 tokens: 23 us
# of Python for 8 us of launches), so each call tests its tensors in one
# expression and looks for the culprit, to word the error, only when that
# fails.

_BF16, _F32, _I32, _U8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8
_F32_MAX = torch.finfo(torch.float32).max
_PTRS = [ctypes.c_void_p * n for n in range(LORA_MAX_SLICES + 1)]
_SIZES = [ctypes.c_int32 * n for n in range(LORA_MAX_SLICES + 1)]
try:
    _raw_stream = torch._C._cuda_getCurrentRawStream      # what current_stream() wraps, without the object
except AttributeError:
    def _raw_stream(index: int) -> int:
        return torch.cuda.current_stream(index).cuda_stream


def _all(index: int, *named) -> None:
    """Each (tensor or None, dtype, name) is a CUDA tensor of that type on GPU `index`."""
    for t, dtype, name in named:
        if t is None:
            continue
        if not isinstance(t, torch.Tensor) or t.dtype is not dtype or t.get_device() != index:
            _need(t, name, dtype)
            raise ValueError("%s is on cuda:%d, expected cuda:%d" % (name, t.get_device(), index))


def _is(t: Optional[torch.Tensor], dtype, index: int) -> bool:
    return t is None or (t.dtype is dtype and t.get_device() == index)


def _gpu(t: torch.Tensor, name: str) -> int:
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    if not t.is_cuda:
        raise ValueError("%s must be a CUDA tensor (no CPU path exists)" % name)
    return t.get_device()


def _workspace_bytes(fn: str, device, *args) -> int:
    with torch.cuda.device(device):
        n = getattr(_lib.load(), fn)(*args)
    if n < 0:
        _lib.check(fn, int(n))
    return int(n)


def _call_with(fn: str, workspace: Optional[torch.Tensor], device, size_args, *args) -> None:
    """Calls fn(*args, workspace, its bytes, the current stream); the
    workspace is allocated when None."""
    if workspace is None:
        workspace = torch.empty(_workspace_bytes(fn + "_workspace", device, *size_args), dtype=_U8,
                                device=device)
    elif not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    try:
        _call(fn, device, *args, workspace.data_ptr(), workspace.numel(), _raw_stream(device.index))
    except LoraError as e:
        if e.status == _lib.LORA_ERR_WORKSPACE:
            raise ValueError("workspace must have at least %d bytes"
                             % _workspace_bytes(fn + "_workspace", device, *size_args)) from e
        raise


def _rows(t: torch.Tensor, name: str):
    """(rows, columns, row stride) of t as a matrix whose rows are contiguous."""
    if t.dim() != 2:
        t = t.view(-1, t.shape[-1])
    n, c = t.shape
    ld, unit = t.stride()
    if unit == 1 and ld >= c:
        return n, c, ld
    if (c > 1 and unit != 1) or (n > 1 and ld < c):
        raise ValueError("%s needs contiguous rows that do not overlap" % name)
    return n, c, max(ld, c)


def _vector(t: Optional[torch.Tensor], name: str, n: int) -> Optional[int]:
    if t is None:
        return None
    if t.numel() != n or not t.is_contiguous():
        raise ValueError("%s must be contiguous with %d elements" % (name, n))
    return t.data_ptr()


def lora_cross_entropy_workspace(num_tokens: int, hidden: int, vocab: int, *,
                                 hidden_grad: bool = True, weight_grad: bool = False,
                                 device="cuda") -> int:
    """Bytes of workspace of :func:`lora_cross_entropy` at these sizes."""
    return _workspace_bytes("lora_cross_entropy_workspace", device, num_tokens, hidden, vocab,
                            int(hidden_grad), int(weight_grad))


def lora_cross_entropy(hidden: torch.Tensor, weight: torch.Tensor, targets: torch.Tensor,
                       loss: torch.Tensor, *, token_weight: Optional[torch.Tensor] = None,
                       logsumexp: Optional[torch.Tensor] = None,
                       hidden_grad: Optional[torch.Tensor] = None,
                       weight_grad: Optional[torch.Tensor] = None,
                       error_word: Optional[torch.Tensor] = None,
                       workspace: Optional[torch.Tensor] = None) -> None:
    """Cross entropy of the logits hidden @ weight^T against targets, and its
    gradients, without keeping the logits.

    loss[t] (fp32) = w_t (logsumexp_t - logit of targets[t]), w_t =
    token_weight[t] (fp32; 1 when None).  A target outside [0, vocab) (-100,
    say) means none: zero loss and gradient.  hidden_grad (bf16, like hidden,
    or hidden itself) and weight_grad (bf16, like weight) are overwritten when given;
    error_word (int32 [1]) receives the count of targets >= vocab.  A
    workspace (uint8) is allocated when none is given."""
    try:
        i = hidden.get_device()
        ok = (i >= 0 and hidden.dtype is _BF16 and weight.dtype is _BF16 and targets.dtype is _I32
              and loss.dtype is _F32 and weight.get_device() == i and targets.get_device() == i
              and loss.get_device() == i and _is(token_weight, _F32, i) and _is(logsumexp, _F32, i)
              and _is(hidden_grad, _BF16, i) and _is(weight_grad, _BF16, i)
              and _is(error_word, _I32, i) and _is(workspace, _U8, i))
    except AttributeError:
        ok = False
    if not ok:
        _all(_gpu(hidden, "hidden"), (hidden, _BF16, "hidden"), (weight, _BF16, "weight"),
             (targets, _I32, "targets"), (loss, _F32, "loss"), (token_weight, _F32, "token_weight"),
             (logsumexp, _F32, "logsumexp"), (hidden_grad, _BF16, "hidden_grad"),
             (weight_grad, _BF16, "weight_grad"), (error_word, _I32, "error_word"),
             (workspace, _U8, "workspace"))
        raise TypeError("weight, targets and loss must be tensors")
    T, H, ld = _rows(hidden, "hidden")
    if weight.dim() != 2 or weight.shape[1] != H or not weight.is_contiguous():
        raise ValueError("weight must be a contiguous [vocab, %d] tensor" % H)
    V = weight.shape[0]
    dh, dh_ld, dw = None, H, None
    if hidden_grad is not None:
        rows, cols, dh_ld = _rows(hidden_grad, "hidden_grad")
        if (rows, cols) != (T, H):
            raise ValueError("hidden_grad must be [%d, %d]" % (T, H))
        dh = hidden_grad.data_ptr()
    if weight_grad is not None:
        if weight_grad.shape != weight.shape or not weight_grad.is_contiguous():
            raise ValueError("weight_grad must be contiguous like weight")
        dw = weight_grad.data_ptr()
    _call_with("lora_cross_entropy", workspace, hidden.device,
               (T, H, V, int(dh is not None), int(dw is not None)),
               hidden.data_ptr(), T, H, ld, weight.data_ptr(), V, _vector(targets, "targets", T),
               _vector(token_weight, "token_weight", T), _vector(loss, "loss", T),
               _vector(logsumexp, "logsumexp", T), dh, dh_ld, dw, _vector(error_word, "error_word", 1))


def lora_linear_backward_workspace(num_tokens: int, hidden: int, output_slices, rank: int,
                                   max_loras: int, *, device="cuda") -> int:
    """Bytes of workspace of :func:`lora_linear_backward` at these sizes."""
    sizes = (ctypes.c_int32 * len(output_slices))(*output_slices)
    return _workspace_bytes("lora_linear_backward_workspace", device, num_tokens, hidden, sizes,
                            len(output_slices), rank, max_loras)


def _stacks(ws, name: str, index: int):
    """The slices' bf16 [max_loras, rows, cols] stacks on GPU `index` (a
    singleton layer dimension, [L, 1, rows, cols], is taken out), their
    shapes, and the array of their pointers."""
    if isinstance(ws, torch.Tensor):
        ws = (ws,)
    shapes, ptrs = [], []
    try:
        for w in ws:
            if w.dtype is not _BF16 or w.get_device() != index or w.dim() != 3 or not w.is_contiguous():
                break
            shapes.append(w.shape)
            ptrs.append(w.data_ptr())
        ok = len(ptrs) == len(ws)
    except AttributeError:
        ok = False
    if not ok:
        ws = _weights(ws, name)
        _all(index, *((w, _BF16, "%s[%d]" % (name, i)) for i, w in enumerate(ws)))
        shapes, ptrs = [w.shape for w in ws], [w.data_ptr() for w in ws]
    if not 1 <= len(ptrs) <= LORA_MAX_SLICES:
        raise ValueError("%s must hold 1 to %d tensors" % (name, LORA_MAX_SLICES))
    return shapes, _PTRS[len(ptrs)](*ptrs)


def _grads(grads, name: str, like, index: int):
    """Pointer array of the gradients (None, or a tensor or None per slice),
    each with the elements and outer sizes of the shape in `like`."""
    if grads is None:
        return None
    if isinstance(grads, torch.Tensor):
        grads = (grads,)
    if len(grads) != len(like):
        raise ValueError("%s needs one entry per slice" % name)
    ptrs = []
    for g, shape in zip(grads, like):
        if g is None:
            ptrs.append(None)
            continue
        try:
            ok = g.dtype is _BF16 and g.get_device() == index and g.shape == shape and g.is_contiguous()
        except AttributeError:
            ok = False
        if not ok:
            _all(index, (g, _BF16, "%s[%d]" % (name, len(ptrs))))
            s = g.shape
            if g.numel() != math.prod(shape) or s[0] != shape[0] or s[-1] != shape[-1] or not g.is_contiguous():
                raise ValueError("%s[%d] must be a contiguous %s tensor" % (name, len(ptrs), list(shape)))
        ptrs.append(g.data_ptr())
    return _PTRS[len(ptrs)](*ptrs)


def _clear_behind(named: int, *grads) -> None:
    """Zeros in the gradients of the adapters that the metadata does not name."""
    for of_slices in grads:
        for g in (of_slices,) if isinstance(of_slices, torch.Tensor) else of_slices or ():
            if g is not None:
                g.detach()[named:].zero_()


def lora_linear_backward(dy: torch.Tensor, x: torch.Tensor, buffer: torch.Tensor, lora_a_stacked,
                         lora_b_stacked, scale: float, meta: LoRAKernelMeta, *,
                         dx: Optional[torch.Tensor] = None, add_inputs: bool = True,
                         d_lora_a=None, d_lora_b=None, d_lora_bias=None,
                         workspace: Optional[torch.Tensor] = None) -> None:
    """Gradients of one layer that add_lora_linear (or lora_linear) ran:
    dy is the gradient of its output [T, sum of the slices], x its input,
    buffer the fp32 buffer it left, meta the batch's metadata.

    Each output is optional and bf16.  dx [T, H]: the adapters' part is added
    to it, or with add_inputs=False it is overwritten; it may be dy or x
    itself (all of them are read before it is written).  d_lora_a, d_lora_b,
    d_lora_bias: one tensor (or None) per slice, shaped as the weights and
    biases, overwritten; adapters without tokens get zeros, and so do those
    that the weights hold beyond the metadata's."""
    index = meta.no_lora_flag.get_device()
    try:
        ok = (index >= 0 and dy.dtype is _BF16 and x.dtype is _BF16 and buffer.dtype is _F32 and dy.get_device() == index
              and x.get_device() == index and buffer.get_device() == index and _is(dx, _BF16, index)
              and _is(workspace, _U8, index))
    except AttributeError:
        ok = False
    if not ok:
        _gpu(dy, "dy")
        _all(index, (dy, _BF16, "dy"), (x, _BF16, "x"), (buffer, _F32, "buffer"), (dx, _BF16, "dx"),
             (workspace, _U8, "workspace"))
        raise TypeError("x and buffer must be tensors")
    a_shapes, a_ptrs = _stacks(lora_a_stacked, "lora_a_stacked", index)
    b_shapes, b_ptrs = _stacks(lora_b_stacked, "lora_b_stacked", index)
    S = len(a_shapes)
    if S != len(b_shapes):
        raise ValueError("lora_a_stacked and lora_b_stacked differ in length")
    T, H, x_ld = _rows(x, "x")
    L, r, _ = a_shapes[0]
    for s in a_shapes:
        if s != (L, r, H):
            raise ValueError("lora_a_stacked shapes must all be [%d, %d, %d]" % (L, r, H))
    Lb = b_shapes[0][0]
    for s in b_shapes:
        if s[0] != Lb or s[2] != r:
            raise ValueError("lora_b_stacked shapes must all be [%d, n, %d]" % (Lb, r))
    named = meta.max_loras
    if L < named or Lb < named:
        raise ValueError("the weights hold %d LoRAs, metadata expects %d" % (min(L, Lb), named))
    sizes = [s[1] for s in b_shapes]
    rows, cols, dy_ld = _rows(dy, "dy")
    if rows != T or cols != sum(sizes):
        raise ValueError("dy must be [%d, %d]" % (T, sum(sizes)))
    if buffer.shape != (S, T, r) or not buffer.is_contiguous():
        raise ValueError("buffer must be a contiguous fp32 [%d, %d, %d] tensor" % (S, T, r))
    dx_ptr, dx_ld = None, H
    if dx is not None:
        rows, cols, dx_ld = _rows(dx, "dx")
        if rows != T or cols != H:
            raise ValueError("dx must be [%d, %d]" % (T, H))
        dx_ptr = dx.data_ptr()
    c_sizes = _SIZES[S](*sizes)
    _call_with("lora_linear_backward", workspace, x.device, (T, H, c_sizes, S, r, named),
               dy.data_ptr(), dy_ld, T, x.data_ptr(), H, x_ld, buffer.data_ptr(), a_ptrs,
               b_ptrs, c_sizes, S, r, float(scale), dx_ptr, dx_ld, 1 if add_inputs else 0,
               _grads(d_lora_a, "d_lora_a", a_shapes, index),
               _grads(d_lora_b, "d_lora_b", b_shapes, index),
               None if d_lora_bias is None else
               _grads(d_lora_bias, "d_lora_bias", [(Lb, n) for n in sizes], index),
               ctypes.byref(meta.c))
    if L > named or Lb > named:
        _clear_behind(named, d_lora_a, d_lora_b, d_lora_bias)


def lora_orthogonalize_workspace(count: int, rows: int, cols: int, *, device="cuda") -> int:
    """Bytes of workspace of :func:`lora_orthogonalize` at these sizes."""
    return _workspace_bytes("lora_orthogonalize_workspace", device, count, rows, cols)


_LONG_RUN = math.log(512.0)         # steps x log |a| above which a run is long


def lora_orthogonalize(update: torch.Tensor, out: torch.Tensor, *, steps: int = 5,
                       scale: float = 1.0, eps: float = 1e-7,
                       coefficients: Sequence[float] = (3.4445, -4.7750, 2.0315),
                       error_word: Optional[torch.Tensor] = None,
                       workspace: Optional[torch.Tensor] = None) -> None:
    """Newton-Schulz orthogonalisation of stacked updates, as the Muon
    optimiser takes them: every matrix of update [..., rows, cols] (bf16 or
    fp32; the shorter side, an adapter's rank, at most 128) divided by its
    norm and taken through ``steps`` of X <- a X + (b G + c G^2) X, G = X X^T;
    out (bf16, like update, or update itself) receives scale * X.  Bit 30 of
    error_word (int32 [1]) is set if a bounded wait on the GPU ran out.  Runs
    of steps with |a|^steps above 512 (six of the default ones) are many times
    slower: they form X and its products afresh every few steps, a group of
    matrices at a time (larger groups with a larger workspace)."""
    index = _gpu(update, "update")
    f32 = update.dtype is _F32
    if not f32 and update.dtype is not _BF16:
        raise TypeError("update must be bfloat16 or float32, got %s" % update.dtype)
    if not (isinstance(out, torch.Tensor) and _is(out, _BF16, index) and _is(error_word, _I32, index)
            and _is(workspace, _U8, index)):
        _all(index, (out, _BF16, "out"), (error_word, _I32, "error_word"), (workspace, _U8, "workspace"))
    if out is None or out.shape != update.shape or not out.is_contiguous():
        raise ValueError("out must be contiguous like update")
    if update.dim() < 2 or not update.is_contiguous():
        raise ValueError("update must be contiguous [..., rows, cols]")
    if len(coefficients) != 3:
        raise ValueError("coefficients must be three numbers")
    rows, cols = update.shape[-2:]
    count = update.numel() // max(1, rows * cols)
    a, b, c = coefficients
    if workspace is None and count > 1 and abs(a) > 1.0 and steps * math.log(abs(a)) > _LONG_RUN:
        # matrices of a long run are taken by groups: all at once, up to 1 GB
        one = lora_orthogonalize_workspace(1, rows, cols, device=update.device)
        need = lora_orthogonalize_workspace(count, rows, cols, device=update.device)
        workspace = torch.empty(max(need, min(count * one, 1 << 30)), dtype=_U8, device=update.device)
    _call_with("lora_orthogonalize", workspace, update.device, (count, rows, cols), update.data_ptr(),
               int(f32), count, rows, cols, int(steps), float(a), float(b), float(c), float(eps),
               float(scale), out.data_ptr(), _vector(error_word, "error_word", 1))


# ------------------------------------------------------------ the layers under the adapters

def _expert_weight(weight, scale, meta, k: int):
    """(experts, rows) of the bf16 or MXFP4 stack, checked against hidden size k."""
    if scale is None:
        if weight.dim() != 3 or weight.shape[2] != k or not weight.is_contiguous():
            raise ValueError("weight must be a contiguous [max_loras, n, %d] tensor" % k)
    else:
        if k % 32:
            raise ValueError("4-bit weights need a hidden size that is a multiple of 32, got %d" % k)
        if weight.dim() != 3 or weight.shape[2] * 2 != k or not weight.is_contiguous():
            raise ValueError("weight must be contiguous codes [max_loras, n, %d]" % (k // 2))
        if tuple(scale.shape) != (*weight.shape[:2], k // 32) or not scale.is_contiguous():
            raise ValueError("weight_scale must be a contiguous %s tensor" % [*weight.shape[:2], k // 32])
    if weight.shape[0] < meta.max_loras:
        raise ValueError("weight holds %d experts, metadata expects %d" % (weight.shape[0], meta.max_loras))
    return weight.shape[0], weight.shape[1]


def _expert_types(first, first_name, meta, named, weight, scale, workspace) -> None:
    """Checks the types and devices of an expert call's tensors."""
    index = meta.no_lora_flag.get_device()
    try:
        ok = (index >= 0 and all(_is(t, _BF16, index) for t, _ in named) and _is(workspace, _U8, index)
              and weight.get_device() == index and weight.dtype is (_BF16 if scale is None else _U8)
              and _is(scale, _U8, index))
    except AttributeError:
        ok = False
    if not ok:
        _gpu(first, first_name)
        _all(index, *((t, _BF16, name) for t, name in named),
             (weight, _BF16 if scale is None else _U8, "weight"), (scale, _U8, "weight_scale"),
             (workspace, _U8, "workspace"))
        raise TypeError("weight must be a tensor")


def _fan_out(rows: int, tokens: int) -> int:
    if rows == 0 and tokens == 0:
        return 1
    if tokens == 0 or rows % tokens or rows == 0:
        raise ValueError("%d rows cannot be shared evenly by %d tokens" % (rows, tokens))
    return rows // tokens


def lora_expert_linear_workspace(num_rows: int, hidden: int, out_features: int, max_loras: int, *,
                                 quantized: bool = False, device="cuda") -> int:
    """Bytes of workspace of :func:`lora_expert_linear` at these sizes."""
    return _workspace_bytes("lora_expert_linear_workspace", device, num_rows, hidden, out_features,
                            max_loras, int(quantized))


def lora_expert_linear(x: torch.Tensor, weight: torch.Tensor, y: torch.Tensor, meta: LoRAKernelMeta, *,
                       weight_scale: Optional[torch.Tensor] = None, add_inputs: bool = False,
                       workspace: Optional[torch.Tensor] = None) -> None:
    """y[i] (+)= weight[id(i)] @ x[i // k]: the product of a mixture of
    experts, which adapters are then added to (add_lora_linear); with one
    expert, of one frozen layer.

    meta was prepared for one expert id per row of y (-1: none, the row is left
    as it is); x has a k-th of the rows, k of them in a row for each token (k =
    1: as many).  weight is bf16 [max_loras, n, hidden], or the uint8 codes
    [max_loras, n, hidden / 2] of :func:`lora_quantize_mxfp4` with their
    weight_scale [max_loras, n, hidden / 32].  y overlaps nothing that is read.
    A workspace (uint8) is allocated when none is given."""
    _expert_types(x, "x", meta, ((x, "x"), (y, "y")), weight, weight_scale, workspace)
    if x is None or y is None:
        raise TypeError("x and y must be tensors")
    T, K, x_ld = _rows(x, "x")
    R, cols, y_ld = _rows(y, "y")
    E, N = _expert_weight(weight, weight_scale, meta, K)
    if cols != N:
        raise ValueError("y must have %d columns" % N)
    k = _fan_out(R, T)
    if y.data_ptr() == x.data_ptr() and R > 0:
        raise ValueError("y must not be x")
    _call_with("lora_expert_linear", workspace, x.device, (R, K, N, meta.max_loras, int(weight_scale is not None)),
               x.data_ptr(), x_ld, R, k, K, weight.data_ptr(),
               None if weight_scale is None else weight_scale.data_ptr(), N, y.data_ptr(), y_ld,
               1 if add_inputs else 0, ctypes.byref(meta.c))


def lora_expert_linear_backward_workspace(num_rows: int, hidden: int, out_features: int, max_loras: int, *,
                                          fan_out: int = 1, hidden_grad: bool = True, weight_grad: bool = False,
                                          quantized: bool = False, device="cuda") -> int:
    """Bytes of workspace of :func:`lora_expert_linear_backward` at these sizes."""
    return _workspace_bytes("lora_expert_linear_backward_workspace", device, num_rows, fan_out, hidden,
                            out_features, max_loras, int(hidden_grad), int(weight_grad), int(quantized))


def lora_expert_linear_backward(dy: torch.Tensor, x: torch.Tensor, weight: torch.Tensor, meta: LoRAKernelMeta, *,
                                weight_scale: Optional[torch.Tensor] = None, dx: Optional[torch.Tensor] = None,
                                add_inputs: bool = False, d_weight: Optional[torch.Tensor] = None,
                                workspace: Optional[torch.Tensor] = None) -> None:
    """Gradients of :func:`lora_expert_linear`: dy is the gradient of its
    output, the rest what it was given.

    dx (bf16, like x): the sum over each token's rows, written, or with
    add_inputs added to what is there; tokens without an expert get zeros, or
    are left as they are.  d_weight (bf16 [max_loras, n, hidden], also for
    4-bit weights) is overwritten; experts without rows get zeros, and so do
    those that the weights hold beyond the metadata's.  Neither output overlaps
    an input or the other."""
    _expert_types(dy, "dy", meta, ((dy, "dy"), (x, "x"), (dx, "dx"), (d_weight, "d_weight")), weight,
                  weight_scale, workspace)
    if dy is None or x is None:
        raise TypeError("dy and x must be tensors")
    T, K, x_ld = _rows(x, "x")
    R, cols, dy_ld = _rows(dy, "dy")
    E, N = _expert_weight(weight, weight_scale, meta, K)
    if cols != N:
        raise ValueError("dy must have %d columns" % N)
    k = _fan_out(R, T)
    dx_ptr, dx_ld, dw_ptr = None, K, None
    if dx is not None:
        rows, cols, dx_ld = _rows(dx, "dx")
        if (rows, cols) != (T, K):
            raise ValueError("dx must be [%d, %d]" % (T, K))
        dx_ptr = dx.data_ptr()
        if R > 0 and (dx_ptr == x.data_ptr() or dx_ptr == dy.data_ptr()):
            raise ValueError("dx must be neither x nor dy")
    if d_weight is not None:
        if tuple(d_weight.shape) != (E, N, K) or not d_weight.is_contiguous():
            raise ValueError("d_weight must be a contiguous %s tensor" % [E, N, K])
        dw_ptr = d_weight.data_ptr()
    _call_with("lora_expert_linear_backward", workspace, x.device,
               (R, k, K, N, meta.max_loras, int(dx_ptr is not None), int(dw_ptr is not None),
                int(weight_scale is not None)),
               dy.data_ptr(), dy_ld, R, k, x.data_ptr(), x_ld, K, weight.data_ptr(),
               None if weight_scale is None else weight_scale.data_ptr(), N, dx_ptr, dx_ld,
               1 if add_inputs else 0, dw_ptr, ctypes.byref(meta.c))
    if d_weight is not None and E > meta.max_loras:
        _clear_behind(meta.max_loras, d_weight)


def _mx_tensors(values: torch.Tensor, name: str, codes: torch.Tensor, scales: torch.Tensor) -> int:
    try:
        index, (*lead, n) = values.get_device(), values.shape
        if (index >= 0 and (values.dtype is _BF16 or values.dtype is _F32) and codes.dtype is _U8 and scales.dtype is _U8
                and codes.get_device() == index and scales.get_device() == index and n % 32 == 0
                and codes.shape == (*lead, n // 2) and scales.shape == (*lead, n // 32) and values.is_contiguous()
                and codes.is_contiguous() and scales.is_contiguous()):
            return index
    except (AttributeError, ValueError):
        pass
    index = _gpu(values, name)
    if values.dtype is not _BF16 and values.dtype is not _F32:
        raise TypeError("%s must be bfloat16 or float32, got %s" % (name, values.dtype))
    if not (isinstance(codes, torch.Tensor) and isinstance(scales, torch.Tensor)):
        raise TypeError("codes and scales must be tensors")
    _all(index, (codes, _U8, "codes"), (scales, _U8, "scales"))
    if values.dim() < 1 or values.shape[-1] % 32 or not values.is_contiguous():
        raise ValueError("%s must be contiguous [..., a multiple of 32]" % name)
    for t, what, part in ((codes, "codes", 2), (scales, "scales", 32)):
        if tuple(t.shape) != (*values.shape[:-1], values.shape[-1] // part) or not t.is_contiguous():
            raise ValueError("%s must be a contiguous %s tensor"
                             % (what, [*values.shape[:-1], values.shape[-1] // part]))
    return index


def lora_quantize_mxfp4(weight: torch.Tensor, codes: torch.Tensor, scales: torch.Tensor) -> None:
    """weight (bf16 or fp32 [..., n], n a multiple of 32) to microscaled 4 bits:
    codes (uint8 [..., n / 2]) and a scale for every 32 elements (uint8 [..., n
    / 32]), as :func:`lora_expert_linear` takes them.  A block with a NaN or an
    infinity becomes NaN as a whole."""
    index = _mx_tensors(weight, "weight", codes, scales)
    _call("lora_quantize_mxfp4", weight.device, weight.data_ptr(), int(weight.dtype is _F32), weight.numel(),
          codes.data_ptr(), scales.data_ptr(), _raw_stream(index))


def lora_dequantize_mxfp4(codes: torch.Tensor, scales: torch.Tensor, out: torch.Tensor) -> None:
    """The values that 4-bit codes stand for (bf16 or fp32 [..., n]), exactly."""
    index = _mx_tensors(out, "out", codes, scales)
    _call("lora_dequantize_mxfp4", out.device, codes.data_ptr(), scales.data_ptr(), out.numel(), out.data_ptr(),
          int(out.dtype is _F32), _raw_stream(index))


def _capturing(index: int) -> bool:
    """Whether the current stream of GPU `index` is being captured into a graph."""
    if torch.cuda.current_device() == index:
        return torch.cuda.is_current_stream_capturing()
    with torch.cuda.device(index):
        return torch.cuda.is_current_stream_capturing()


def _refuse_overlaps(grads, out) -> None:
    """Each tensor is read and written as a whole, in no order: no two of the written ones may share
    memory, nor may one share another's gradient (its own: only as a whole)."""
    spans = []
    for i, g in enumerate(grads):
        w = g if out is None else out[i]
        spans.append((w.data_ptr(), w.data_ptr() + w.numel() * w.element_size(), i, True))
        if w.data_ptr() != g.data_ptr():
            spans.append((g.data_ptr(), g.data_ptr() + g.numel() * g.element_size(), i, False))
    end = written = 0                       # of all spans so far, and of those that are written
    for first, last, i, write in sorted(spans):
        if first < last:
            if first < (end if write else written):
                raise ValueError("grads[%d] or its output overlaps another tensor" % i)
            end = max(end, last)
            written = max(written, last) if write else written


class LoRAGradients:
    """The gradients of many layers, checked once, for
    :func:`lora_clip_gradients` to be called on them every step.

    grads: bf16 or fp32 tensors (None is skipped), contiguous, on one GPU.
    groups: how many adapters their first dimension stacks (1: any shape).
    out: None (they are scaled in place), or tensors like them that receive the
    scaled gradients.  No two may share memory.  The tensors are kept; their
    storage must stay where it is.  Workspaces are kept for each stream, and a
    captured call has one of its own, so an object may be used on any stream,
    captured, and dropped while its calls run or graphs hold them (the tensors
    themselves are the caller's to keep until then)."""

    def __init__(self, grads, groups: int = 1, out=None):
        if isinstance(grads, torch.Tensor):
            grads = (grads,)
        if isinstance(out, torch.Tensor):
            out = (out,)
        if groups < 1:
            raise ValueError("groups must be at least 1")
        if out is not None and len(out) != len(grads):
            raise ValueError("out needs one entry per gradient")
        pairs = [(i, g, None if out is None else out[i]) for i, g in enumerate(grads) if g is not None]
        if not pairs:
            raise ValueError("there are no gradients")
        self.index = index = _gpu(pairs[0][1], "grads[%d]" % pairs[0][0])
        for i, g, o in pairs:
            _gpu(g, "grads[%d]" % i)
            if g.dtype is not _BF16 and g.dtype is not _F32:
                raise TypeError("grads[%d] must be bfloat16 or float32, got %s" % (i, g.dtype))
            _all(index, (g, g.dtype, "grads[%d]" % i), (o, g.dtype, "out[%d]" % i))
            if not g.is_contiguous():
                raise ValueError("grads[%d] must be contiguous" % i)
            if groups > 1 and (g.dim() < 1 or g.shape[0] != groups):
                raise ValueError("grads[%d] must stack %d adapters in its first dimension" % (i, groups))
            if out is not None and (o is None or o.shape != g.shape or not o.is_contiguous()):
                raise ValueError("out[%d] must be contiguous like its gradient" % i)
        n = len(pairs)
        _refuse_overlaps([p[1] for p in pairs], None if out is None else [p[2] for p in pairs])
        self.grads, self.out, self.groups, self.count = [p[1] for p in pairs], [p[2] for p in pairs], groups, n
        self.device = self.grads[0].device
        self.c_grads = (ctypes.c_void_p * n)(*[g.data_ptr() for g in self.grads])
        self.c_out = None if out is None else (ctypes.c_void_p * n)(*[o.data_ptr() for o in self.out])
        self.c_sizes = (ctypes.c_int64 * n)(*[g.numel() // groups for g in self.grads])
        self.c_f32 = (ctypes.c_int32 * n)(*[int(g.dtype is _F32) for g in self.grads])
        self.workspace_bytes = _workspace_bytes("lora_clip_gradients_workspace", self.device, groups)
        self.workspaces = {}

    @staticmethod
    def make(grads, groups: int = 1, *, out=None) -> "LoRAGradients":
        return LoRAGradients(grads, groups, out)

    def workspace(self, stream: int) -> torch.Tensor:
        """The workspace of a call on the current stream, whose handle is `stream`.

        Memory belongs to the stream that it was allocated on: given back while
        calls on another stream run, it would be handed out again under them.
        A captured call's belongs to its graph, which may outlive the object and
        be replayed beside another one."""
        if _capturing(self.index):
            return torch.empty(self.workspace_bytes, dtype=_U8, device=self.device)
        kept = self.workspaces.get(stream)
        if kept is None:
            kept = self.workspaces[stream] = torch.empty(self.workspace_bytes, dtype=_U8, device=self.device)
        return kept


def lora_clip_gradients(grads, max_norm: Optional[float], norms: torch.Tensor, *, eps: float = 1e-6) -> None:
    """Scales gradients down to a largest norm: norms (fp32 [groups]) receives
    the root of the sum of squares over all tensors, for each adapter of their
    stacks (groups of them) or, with one element, over everything; gradients
    are multiplied by min(1, max_norm / (norm + eps)).

    grads is a :class:`LoRAGradients` (for every step), or the tensors
    themselves, which are then scaled in place and stack norms.numel() adapters.
    max_norm None (or infinite) computes the norms alone; other values of it
    and of eps fit into 32 bits.  Nothing is read back
    to the host: a NaN norm makes its adapter's gradients NaN, and leaves the
    others'."""
    if not isinstance(norms, torch.Tensor):
        raise TypeError("norms must be a torch.Tensor")
    if not isinstance(grads, LoRAGradients):
        grads = LoRAGradients(grads, norms.numel())
    _all(grads.index, (norms, _F32, "norms"))
    limit, eps = math.inf if max_norm is None else float(max_norm), float(eps)
    if not limit >= 0.0 or not eps >= 0.0:
        raise ValueError("max_norm and eps must not be negative")
    # the library takes them in 32 bits, where larger ones would be infinite
    if _F32_MAX < limit < math.inf or eps > _F32_MAX:
        raise ValueError("max_norm must be None, infinite or at most %g, eps at most that" % _F32_MAX)
    norms_ptr, stream = _vector(norms, "norms", grads.groups), _raw_stream(grads.index)
    workspace = grads.workspace(stream)
    _call("lora_clip_gradients", grads.device, grads.c_grads, grads.c_out, grads.c_sizes, grads.c_f32, grads.count,
          grads.groups, limit, eps, norms_ptr, workspace.data_ptr(), grads.workspace_bytes, stream)
