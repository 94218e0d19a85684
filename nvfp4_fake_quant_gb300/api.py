"""PyTorch-facing binding of the C ABI (argument marshalling only).

Every function takes CUDA tensors, checks dtype/layout/device, allocates the
outputs and the workspace the caller did not pass, and calls the entry point
of the same name on the current CUDA stream.  All computation happens in the
library's kernels; there is no CPU or PyTorch fallback.

``AttnQAT`` mirrors the pages' ``AttentionImpl(num_heads, head_size,
softmax_scale, causal).forward(q, k, v)`` ("attn_qat_train" API page,
``AttnQatTrainImpl``): q, k, v in [B, L, H, D] layout, dropout rejected,
softmax_scale None meaning 1/sqrt(D).
"""
from __future__ import annotations

import functools
import math
import typing

import torch

from . import _lib

BF16 = torch.bfloat16


def _stream_ptr(t: torch.Tensor):
    return torch.cuda.current_stream(t.device).cuda_stream


def _ptr(t):
    return None if t is None else t.data_ptr()


def _check(t: torch.Tensor, name: str, dtype=BF16):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")


def _check_bnhd(t, name, shape=None):
    _check(t, name)
    if t.dim() != 4 or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous [B, N, H, D] tensor")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")


def _rows_ld(x: torch.Tensor):
    if x.dim() != 2 or x.stride(1) != 1:
        raise ValueError("x must be a 2-D tensor with unit column stride")
    return x.shape[0], x.shape[1], x.stride(0)


# ------------------------------------------------------------------ quantizer

def nvfp4_global_sf(x: torch.Tensor, out: torch.Tensor | None = None) -> torch.Tensor:
    """fp32 scalar tensor 448*6/max(amax(|x|), 1e-12) computed on the device."""
    _check(x, "x")
    rows, cols, ld = _rows_ld(x)
    if out is None:
        out = torch.empty((), dtype=torch.float32, device=x.device)
    _lib.call("nvfp4_global_sf", _ptr(x), rows, cols, ld, _ptr(out), _stream_ptr(x))
    return out


def nvfp4_fake_quant(x: torch.Tensor, global_sf: torch.Tensor | None = None,
                     out: torch.Tensor | None = None, scales: torch.Tensor | None = None,
                     want_scales: bool = True):
    """NVFP4 fake quantization of a bf16 [rows, cols] matrix, cols % 16 == 0.

    Returns (out bf16 [rows, cols], scales uint8 [rows, cols/16] E4M3FN bytes or
    None).  ``global_sf`` is a device fp32 scalar or None (unit scale).
    """
    _check(x, "x")
    rows, cols, ld = _rows_ld(x)
    if out is None:
        out = torch.empty((rows, cols), dtype=BF16, device=x.device)
    _check(out, "out")
    if scales is None and want_scales:
        scales = torch.empty((rows, cols // 16), dtype=torch.uint8, device=x.device)
    if global_sf is not None:
        _check(global_sf, "global_sf", torch.float32)
    _lib.call("nvfp4_fake_quant", _ptr(x), rows, cols, ld, _ptr(global_sf), _ptr(out),
              out.stride(0), _ptr(scales), 0 if scales is None else scales.stride(0),
              _stream_ptr(x))
    return out, scales


def nvfp4_quantize_codes(x: torch.Tensor, global_sf: torch.Tensor | None = None,
                         codes: torch.Tensor | None = None, scales: torch.Tensor | None = None):
    """Packed NVFP4 codes (uint8 [rows, cols/2], element 2i in the low nibble) and
    E4M3FN scale bytes (uint8 [rows, cols/16])."""
    _check(x, "x")
    rows, cols, ld = _rows_ld(x)
    if codes is None:
        codes = torch.empty((rows, cols // 2), dtype=torch.uint8, device=x.device)
    if scales is None:
        scales = torch.empty((rows, cols // 16), dtype=torch.uint8, device=x.device)
    if global_sf is not None:
        _check(global_sf, "global_sf", torch.float32)
    _lib.call("nvfp4_quantize_codes", _ptr(x), rows, cols, ld, _ptr(global_sf), _ptr(codes),
              codes.stride(0), _ptr(scales), scales.stride(0), _stream_ptr(x))
    return codes, scales


# ------------------------------------------------------------------ attention

def default_scale(d: int) -> float:
    """sm_scale default of attn_qat_train(): 1/sqrt(D)."""
    return 1.0 / math.sqrt(d)


def _scale(scale, d: int) -> float:
    """The softmax scale to pass: None or NaN mean the default 1/sqrt(D)."""
    if scale is None or math.isnan(float(scale)):
        return default_scale(d)
    return float(scale)


def attn_qat_fwd_workspace(b, nq, nkv, h, d) -> int:
    return int(_lib.load().attn_qat_fwd_workspace(b, nq, nkv, h, d))


def attn_qat_bwd_workspace(b, nq, nkv, h, d) -> int:
    return int(_lib.load().attn_qat_bwd_workspace(b, nq, nkv, h, d))


NO_REGION = 2 ** 64 - 1  # SIZE_MAX: the workspace has no such region


def attn_qat_layout(b, nq, nkv, h, d, which: str = "fwd") -> dict:
    """Byte offsets of the regions of the forward ("fwd") or backward ("bwd")
    workspace (nvq_attn_layout); absent regions are left out."""
    import ctypes
    lay = _lib.AttnLayout()
    _lib.call(f"attn_qat_{which}_layout", b, nq, nkv, h, d, ctypes.addressof(lay))
    return {name: getattr(lay, name) for name, _ in lay._fields_
            if getattr(lay, name) != NO_REGION}


def _workspace(nbytes: int, device, ws: torch.Tensor | None) -> torch.Tensor:
    if ws is None or ws.numel() * ws.element_size() < nbytes:
        ws = torch.empty(max(nbytes, 256), dtype=torch.uint8, device=device)
    return ws


def _fwd_args(q, k, v, scale, o, stats, workspace):
    _check_bnhd(q, "q")
    b, nq, h, d = q.shape
    nkv = k.shape[1]
    _check_bnhd(k, "k", (b, nkv, h, d))
    _check_bnhd(v, "v", (b, nkv, h, d))
    scale = _scale(scale, d)
    if o is None:
        o = torch.empty_like(q)
    if stats is None:
        stats = torch.empty((b, h, 2, nq), dtype=torch.float32, device=q.device)
    ws = _workspace(attn_qat_fwd_workspace(b, nq, nkv, h, d), q.device, workspace)
    return (b, nq, nkv, h, d), scale, o, stats, ws


def attn_qat_fwd(q, k, v, scale=None, causal=False, o=None, stats=None, workspace=None):
    """Forward: returns (o bf16 [B, Nq, H, D], stats fp32 [B, H, 2, Nq] = (LSE, m))."""
    dims, scale, o, stats, ws = _fwd_args(q, k, v, scale, o, stats, workspace)
    _lib.call("attn_qat_fwd", _ptr(q), _ptr(k), _ptr(v), *dims, scale,
              int(bool(causal)), _ptr(o), _ptr(stats), _ptr(ws), ws.numel() * ws.element_size(),
              _stream_ptr(q))
    return o, stats


def attn_qat_fwd_hp(q, k, v, scale=None, causal=False, o=None, o_hp=None, stats=None,
                    workspace=None):
    """Forward with the auxiliary high-precision output: returns (o, o_hp, stats),
    o_hp = P V~ / l with P unquantized (bf16 [B, Nq, H, D]); o and stats as in
    attn_qat_fwd.  Passing o_hp as ``o`` to attn_qat_bwd takes delta from it."""
    dims, scale, o, stats, ws = _fwd_args(q, k, v, scale, o, stats, workspace)
    if o_hp is None:
        o_hp = torch.empty_like(q)
    _check_bnhd(o_hp, "o_hp", q.shape)
    _lib.call("attn_qat_fwd_hp", _ptr(q), _ptr(k), _ptr(v), *dims, scale,
              int(bool(causal)), _ptr(o), _ptr(o_hp), _ptr(stats), _ptr(ws),
              ws.numel() * ws.element_size(), _stream_ptr(q))
    return o, o_hp, stats


def attn_qat_bwd(q, k, v, o, stats, do, scale=None, causal=False, dq=None, dk=None, dv=None,
                 workspace=None):
    """Straight-through backward: returns (dq, dk, dv), bf16, shaped like q, k, v."""
    _check_bnhd(q, "q")
    b, nq, h, d = q.shape
    nkv = k.shape[1]
    _check_bnhd(k, "k", (b, nkv, h, d))
    _check_bnhd(v, "v", (b, nkv, h, d))
    _check_bnhd(o, "o", q.shape)
    _check_bnhd(do, "do", q.shape)
    _check(stats, "stats", torch.float32)
    scale = _scale(scale, d)
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    ws = _workspace(attn_qat_bwd_workspace(b, nq, nkv, h, d), q.device, workspace)
    _lib.call("attn_qat_bwd", _ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(stats), _ptr(do),
              _ptr(dq), _ptr(dk), _ptr(dv), b, nq, nkv, h, d, scale, int(bool(causal)),
              _ptr(ws), ws.numel() * ws.element_size(), _stream_ptr(q))
    return dq, dk, dv


def attn_qat_bwd_saved(saved, o, stats, do, scale=None, causal=False, nkv=None, dq=None,
                       dk=None, dv=None, workspace=None):
    """Straight-through backward from the quantized operands a forward left in its
    workspace ``saved`` (the ``workspace`` tensor passed to attn_qat_fwd or
    attn_qat_fwd_hp on the same q, k, v): returns (dq, dk, dv), equal to
    attn_qat_bwd's bit for bit.  ``nkv`` is the key count (default Nq)."""
    _check_bnhd(o, "o")
    b, nq, h, d = o.shape
    nkv = nq if nkv is None else int(nkv)
    _check_bnhd(do, "do", o.shape)
    _check(stats, "stats", torch.float32)
    _check(saved, "saved", torch.uint8)
    scale = _scale(scale, d)
    dq = torch.empty_like(o) if dq is None else dq
    dk = torch.empty((b, nkv, h, d), dtype=BF16, device=o.device) if dk is None else dk
    dv = torch.empty((b, nkv, h, d), dtype=BF16, device=o.device) if dv is None else dv
    need = int(_lib.load().attn_qat_bwd_saved_workspace(b, nq, nkv, h, d))
    ws = _workspace(need, o.device, workspace)
    _lib.call("attn_qat_bwd_saved", _ptr(saved), saved.numel(), _ptr(o), _ptr(stats), _ptr(do),
              _ptr(dq), _ptr(dk), _ptr(dv), b, nq, nkv, h, d, scale, int(bool(causal)), _ptr(ws),
              ws.numel() * ws.element_size(), _stream_ptr(o))
    return dq, dk, dv


# ------------------------------------------------------------------ NVFP4 linear
def nvfp4_tiled_scale_bytes(rows: int, cols: int) -> int:
    return int(_lib.load().nvfp4_tiled_scale_bytes(rows, cols))


def nvfp4_quantize_tiled(x: torch.Tensor, global_sf: torch.Tensor | None = None,
                         codes: torch.Tensor | None = None, scales: torch.Tensor | None = None):
    """Packed E2M1 codes (uint8 [rows, cols/2]) and E4M3 scales in the 128x4 tiled
    layout of block-scaled FP4 GEMMs (uint8, nvfp4_tiled_scale_bytes) of a bf16
    matrix x [rows, cols]."""
    _check(x, "x")
    rows, cols, ld = _rows_ld(x)
    if codes is None:
        codes = torch.empty((rows, cols // 2), dtype=torch.uint8, device=x.device)
    if scales is None:
        scales = torch.empty(nvfp4_tiled_scale_bytes(rows, cols), dtype=torch.uint8,
                             device=x.device)
    _lib.call("nvfp4_quantize_tiled", _ptr(x), rows, cols, ld, _opt_ptr(global_sf),
              _ptr(codes), _ptr(scales), _stream_ptr(x))
    return codes, scales


def _opt_ptr(t):
    if t is None:
        return None
    _check(t, "global_sf", torch.float32)
    return _ptr(t)


def _linear_dims(x, w):
    _check(x, "x")
    _check(w, "w")
    if x.dim() != 2 or w.dim() != 2 or x.shape[1] != w.shape[1]:
        raise ValueError(f"x [M, K] and w [N, K] expected, got {tuple(x.shape)}, {tuple(w.shape)}")
    if not (x.is_contiguous() and w.is_contiguous()):
        raise ValueError("x and w must be contiguous")
    return x.shape[0], w.shape[0], x.shape[1]


def nvfp4_linear_fwd(x, w, bias=None, x_global_sf=None, w_global_sf=None, out=None,
                     workspace=None):
    """out [M, N] bf16 = x~ w~^T (+ bias): both operands NVFP4-quantized under
    their global scales (None: 448*6/amax of the operand), FP4 block-scaled GEMM."""
    m, n, k = _linear_dims(x, w)
    if bias is not None:
        _check(bias, "bias")
    if out is None:
        out = torch.empty((m, n), dtype=BF16, device=x.device)
    ws = _workspace(int(_lib.load().nvfp4_linear_workspace(m, n, k)), x.device, workspace)
    _lib.call("nvfp4_linear_fwd", _ptr(x), _ptr(w), None if bias is None else _ptr(bias), m, n, k,
              _opt_ptr(x_global_sf), _opt_ptr(w_global_sf), _ptr(out), _ptr(ws),
              ws.numel() * ws.element_size(), _stream_ptr(x))
    return out


def nvfp4_linear_bwd(grad, x, w, need_bias=True, workspace=None):
    """Straight-through gradients (grad_x [M, K], grad_w [N, K], grad_b [N] or None), bf16."""
    m, n, k = _linear_dims(x, w)
    _check(grad, "grad")
    if tuple(grad.shape) != (m, n) or not grad.is_contiguous():
        raise ValueError("grad must be a contiguous [M, N] tensor")
    gx = torch.empty_like(x)
    gw = torch.empty_like(w)
    gb = torch.empty((n,), dtype=BF16, device=x.device) if need_bias else None
    ws = _workspace(int(_lib.load().nvfp4_linear_bwd_workspace(m, n, k)), x.device, workspace)
    _lib.call("nvfp4_linear_bwd", _ptr(grad), _ptr(x), _ptr(w), m, n, k, _ptr(gx), _ptr(gw),
              None if gb is None else _ptr(gb), _ptr(ws), ws.numel() * ws.element_size(),
              _stream_ptr(x))
    return gx, gw, gb


class NVFP4LinearFunction(torch.autograd.Function):
    """Forward: the NVFP4 linear (both operands quantized, FP4 GEMM); backward: the
    full-precision linear gradients (straight-through)."""

    @staticmethod
    def forward(ctx, x, w, bias, x_global_sf):
        shape = x.shape
        x2 = x.reshape(-1, shape[-1]).contiguous()
        out = nvfp4_linear_fwd(x2, w.contiguous(), bias, x_global_sf)
        ctx.save_for_backward(x2, w)
        ctx.has_bias, ctx.shape = bias is not None, shape
        return out.view(*shape[:-1], w.shape[0])

    @staticmethod
    def backward(ctx, grad):
        x2, w = ctx.saved_tensors
        g2 = grad.reshape(-1, grad.shape[-1]).contiguous()
        gx, gw, gb = nvfp4_linear_bwd(g2, x2, w.contiguous(), ctx.has_bias)
        return gx.view(ctx.shape), gw, gb, None


class NVFP4Linear(torch.nn.Module):
    """A bf16 linear layer whose forward runs as the NVFP4 GEMM (weight quantized
    under 448*6/amax(w) at every call, input under ``input_global_sf`` or its own
    amax) and whose backward is straight-through."""

    def __init__(self, in_features: int, out_features: int, bias: bool = True,
                 input_global_sf: torch.Tensor | None = None, device=None):
        super().__init__()
        self.weight = torch.nn.Parameter(torch.empty(out_features, in_features, dtype=BF16,
                                                     device=device))
        self.bias = torch.nn.Parameter(torch.zeros(out_features, dtype=BF16, device=device)) \
            if bias else None
        self.input_global_sf = input_global_sf
        torch.nn.init.normal_(self.weight, std=in_features ** -0.5)

    def forward(self, x):
        return NVFP4LinearFunction.apply(x, self.weight, self.bias, self.input_global_sf)

    def pack(self) -> "NVFP4PackedLinear":
        """The layer for serving: its weight quantized once, under the same scale."""
        return NVFP4PackedLinear(self.weight, self.bias, self.input_global_sf)


# ------------------------------------------------- single tokens: shared helpers
#
# These calls take microseconds on the device, so their checks are written for the
# valid call: one pass over plain attributes, with the explanation left to the path
# that raises.

_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                      lambda index: torch.cuda.current_stream(index).cuda_stream)
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _launch(index: int, name: str, *args) -> None:
    """The entry point on the current stream of device ``index``, with that device
    current (the library works on the current device)."""
    if index == _current_device():
        st = getattr(_lib._lib or _lib.load(), name)(*args, _raw_stream(index))
        if st:
            _lib.fail(name, st)
    else:
        with torch.cuda.device(index):
            _lib.call(name, *args, _raw_stream(index))


def _on(index: int, name: str, *args) -> int:
    """A size query with device ``index`` current (sizes follow its SM count)."""
    f = getattr(_lib.load(), name)
    if index == _current_device():
        return int(f(*args))
    with torch.cuda.device(index):
        return int(f(*args))


def _device_of(first, *others) -> int:
    """The device index that all tensors (None entries left out) share."""
    index = first.get_device()
    for t in others:
        if t is not None and t.get_device() != index:
            raise ValueError(f"tensors on {first.device} and {t.device}: one device expected")
    return index


def _rows_nd(x: torch.Tensor, name: str):
    """(rows, heads, D, row stride) of a bf16 [rows, heads, D] tensor whose rows are
    contiguous inside."""
    if not (isinstance(x, torch.Tensor) and x.dtype is BF16 and x.is_cuda):
        _check(x, name)
    shape = x.shape
    if len(shape) == 3:
        t, h, d = shape
        row, s1, s2 = x.stride()
        if (s2 == 1 or d == 1) and (s1 == d or h == 1) or t * h * d == 0:
            return t, h, d, row if t > 1 else h * d
    raise ValueError(f"{name} must be [tokens, heads, D] with contiguous heads")


def _int32(t, name, dim):
    """(shape, strides) of an int32 tensor of ``dim`` dimensions with unit last stride
    (its device is looked at with the others', by _device_of)."""
    if not (isinstance(t, torch.Tensor) and t.dtype is torch.int32):
        _check(t, name, torch.int32)
    shape, strides = t.shape, t.stride()
    if len(shape) != dim or (strides[-1] != 1 and t.numel() > 1):
        raise ValueError(f"{name} must be a {dim}-dimensional int32 tensor with unit last stride")
    return shape, strides


def _check_out(t, name, shape, dtype, like):
    """An output to write: the caller's, checked, or a new contiguous one."""
    if t is None:
        return torch.empty(shape, dtype=dtype, device=like.device)
    _check(t, name, dtype)
    if tuple(t.shape) != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous, of shape {shape}")
    return t


def _count(n) -> int:
    """A number of tokens as a C int, which ctypes would cut to its low 32 bits: those past
    any length are as good as the largest, those below 0 are refused by the call."""
    return max(-1, min(int(n), 0x7FFFFFFF))


def _check_workspace(ws):
    """A caller's workspace: the kernels take all of its bytes as lying one after another (a
    broadcast view has fewer)."""
    if ws is not None and not ws.is_contiguous():
        raise ValueError("workspace must be contiguous")


def _overwritten(*outs):
    """Tells autograd that the caller's tensors have been written, as torch's own in-place
    operations do: a graph that saved one of them refuses its backward."""
    for t in outs:
        if t is not None:
            torch.autograd.graph.increment_version(t)


def _loadable(x: torch.Tensor):
    """x [rows, ...] itself where the kernels read its layout (contiguous rows with a
    stride of whole 16-byte units), else a contiguous copy: heads or features of another
    order, rows that are broadcast, a start between the units."""
    inner = 1
    for size, stride in zip(reversed(x.shape[1:]), reversed(x.stride()[1:])):
        if size > 1 and stride != inner:
            return x.contiguous()
        inner *= size
    if x.shape[0] > 1 and (x.stride(0) < inner or x.stride(0) % 8) or x.data_ptr() % 16:
        return x.clone(memory_format=torch.contiguous_format)
    return x


def _moved_only(module, apply, fn, recurse):
    """Module._apply for buffers whose types are part of their meaning: they follow the
    module to a device, not to another type (model.to(bfloat16), model.half())."""
    kept = dict(module._buffers)
    apply(fn, recurse)
    for name, t in kept.items():
        if t is not None and module._buffers[name].dtype != t.dtype:
            module._buffers[name] = t.to(module._buffers[name].device)
    return module


# ------------------------------------------------------- NVFP4 linear, packed weight

def nvfp4_linear_packed_workspace(m: int, n: int, k: int) -> int:
    return int(_lib.load().nvfp4_linear_packed_workspace(m, n, k))


def nvfp4_linear_packed_fwd(x, w_codes, w_scales, w_global_sf=None, bias=None, x_global_sf=None,
                            out=None, workspace=None):
    """out [M, N] bf16 = x~ w~^T (+ bias) for a weight packed by nvfp4_quantize_tiled
    (codes uint8 [N, K/2], tiled scales) under ``w_global_sf`` (None: 1).  x bf16
    [M, K], rows may be strided, not under ``out``; ``x_global_sf`` None: 448*6/amax(x).
    No rows (M = 0) is a valid call that launches nothing."""
    if not (isinstance(x, torch.Tensor) and x.dtype is BF16 and x.is_cuda):
        _check(x, "x")
    m, k, ld = _rows_ld(x)
    for t, name in ((w_codes, "w_codes"), (w_scales, "w_scales")):
        if not (isinstance(t, torch.Tensor) and t.dtype is torch.uint8):
            _check(t, name, torch.uint8)
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
    shape = w_codes.shape
    if len(shape) != 2 or shape[1] * 2 != k:
        raise ValueError(f"w_codes must be [N, {k // 2}], got {tuple(shape)}")
    n = shape[0]
    # the 128x4 tiles of nvfp4_tiled_scale_bytes (k % 16 != 0 is refused below)
    if w_scales.numel() != -(-n // 128) * -(-(k // 16) // 4) * 512:
        raise ValueError("w_scales must be the tiled scales of w_codes")
    if bias is not None:
        _check(bias, "bias")
        if bias.dim() != 1 or bias.shape[0] != n or not bias.is_contiguous():
            raise ValueError(f"bias must be contiguous [{n}]")
    index = _device_of(x, w_codes, w_scales, w_global_sf, bias, x_global_sf, out, workspace)
    _check_workspace(workspace)
    given, out = out, _check_out(out, "out", (m, n), BF16, x)
    if m == 0 and nvfp4_linear_packed_workspace(1, n, k):  # no rows of a layer that is served
        return out
    ws = workspace
    if ws is None:
        ws = _workspace(nvfp4_linear_packed_workspace(m, n, k), x.device, None)
    args = (x.data_ptr(), ld if m > 1 else k, w_codes.data_ptr(), w_scales.data_ptr(),
            _opt_ptr(w_global_sf), None if bias is None else bias.data_ptr(), m, n, k,
            _opt_ptr(x_global_sf), out.data_ptr())
    try:
        _launch(index, "nvfp4_linear_packed_fwd", *args, ws.data_ptr(),
                ws.numel() * ws.element_size())
    except _lib.NvqError as e:
        if e.status != 3 or workspace is None:
            raise
        # the caller's workspace is too small (or misaligned): one of our own, as elsewhere
        ws = _workspace(nvfp4_linear_packed_workspace(m, n, k), x.device, None)
        _launch(index, "nvfp4_linear_packed_fwd", *args, ws.data_ptr(), ws.numel())
    _overwritten(given)
    return out


class NVFP4PackedLinear(torch.nn.Module):
    """The serving form of NVFP4Linear: the weight's codes, tiled scales and global
    scale, packed once; the forward of the layer it was packed from."""

    def __init__(self, weight, bias=None, input_global_sf=None):
        super().__init__()
        w = weight.detach().contiguous()
        self.register_buffer("weight_global_sf", nvfp4_global_sf(w))
        codes, scales = nvfp4_quantize_tiled(w, self.weight_global_sf)
        self.register_buffer("codes", codes)
        self.register_buffer("scales", scales)
        self.register_buffer("bias", None if bias is None else bias.detach().clone())
        self.register_buffer("input_global_sf", input_global_sf)

    def _apply(self, fn, recurse=True):
        return _moved_only(self, super()._apply, fn, recurse)

    @torch.no_grad()
    def forward(self, x):
        out = nvfp4_linear_packed_fwd(_loadable(x.reshape(-1, x.shape[-1])), self.codes,
                                      self.scales, self.weight_global_sf, self.bias, self.input_global_sf)
        return out.view(*x.shape[:-1], self.codes.shape[0])


# ----------------------------------------------------------------- rotary positions

def rope_inv_freq(rot_dim: int, theta: float = 10000.0, scaling: str | None = None,
                  factor: float = 1.0, original_len: int = 8192, beta_fast: float = 32.0,
                  beta_slow: float = 1.0, device=None):
    """(inv_freq f64 [rot_dim/2], mscale) for rope_apply.

    inv_freq[p] = theta^(-2p/rot_dim).  For contexts ``factor`` times longer than the
    ``original_len`` trained on, ``scaling`` is
      "linear"    every frequency divided by factor (positions interpolated);
      "theta"     theta raised to theta * factor^(rot_dim/(rot_dim - 2)), which divides
                  the lowest frequency by factor and leaves the highest;
      "by_parts"  pairs that turn fewer than beta_slow times in original_len positions
                  divided by factor, those over beta_fast kept, a linear blend between;
                  rotated elements multiplied by mscale = 0.1 ln(factor) + 1.
    """
    if rot_dim < 2 or rot_dim % 2 or not theta > 0 or not factor >= 1:
        raise ValueError("rot_dim must be even and >= 2, theta > 0, factor >= 1")
    if scaling not in (None, "linear", "theta", "by_parts"):
        raise ValueError(f"unknown scaling {scaling!r}")
    mscale = 1.0
    if scaling == "theta" and rot_dim > 2:
        theta = theta * factor ** (rot_dim / (rot_dim - 2))
    f = float(theta) ** (-torch.arange(0, rot_dim, 2, dtype=torch.float64) / rot_dim)
    if scaling == "linear":
        f = f / factor
    elif scaling == "by_parts" and factor > 1:
        if not beta_fast > beta_slow:
            raise ValueError("beta_fast must be over beta_slow")
        turns = original_len * f / (2 * math.pi)
        keep = ((turns - beta_slow) / (beta_fast - beta_slow)).clamp(0, 1)
        f = f / factor * (1 - keep) + f * keep
        mscale = 0.1 * math.log(factor) + 1
    return f.to(device), mscale


@functools.lru_cache(maxsize=256)
def _host_ints(values: tuple):
    """A C array of the ints (read by the entry point before it returns)."""
    return (_lib.c_int * len(values))(*values)


def rope_apply(q, k, positions, inv_freq, interleaved=False, axis_pairs=None, mscale=1.0,
               inverse=False, q_out=None, k_out=None):
    """Rotary positions of q [T, Hq, D] and k [T, Hk, D] (bf16, token rows may be
    strided; k may be None): returns (q_out, k_out).  ``positions`` int32 [T] or
    [T, axes]; ``axis_pairs`` the number of pairs that turn by each axis (default:
    all by the first); ``inv_freq`` f64 [rot_dim/2].  q_out / k_out may be q / k: the raw
    call is outside autograd (Rotary is inside), whose graphs that saved them then refuse
    their backward."""
    t, hq, d, ld_q = _rows_nd(q, "q")
    if not (isinstance(inv_freq, torch.Tensor) and inv_freq.dtype is torch.float64):
        _check(inv_freq, "inv_freq", torch.float64)
    shape = inv_freq.shape
    if len(shape) != 1 or not inv_freq.is_contiguous():
        raise ValueError("inv_freq must be a contiguous vector")
    rot = 2 * shape[0]
    if not (isinstance(positions, torch.Tensor) and positions.dtype is torch.int32):
        _check(positions, "positions", torch.int32)
    shape = positions.shape
    axes = 1 if len(shape) == 1 else shape[1] if len(shape) == 2 else 0
    if axes == 0 or shape[0] != t or not positions.is_contiguous():
        raise ValueError(f"positions must be contiguous [{t}] or [{t}, axes]")
    given = (q_out, k_out)
    pairs = (rot // 2,) + (0,) * (axes - 1) if axis_pairs is None else tuple(axis_pairs)
    if len(pairs) != axes or axes > 3:
        raise ValueError(f"axis_pairs must give one count for each of 1..3 axes, got {pairs}")
    if q_out is None:
        q_out, ld_qo = torch.empty((t, hq, d), dtype=BF16, device=q.device), hq * d
    else:
        *shape, ld_qo = _rows_nd(q_out, "q_out")
        if shape != [t, hq, d]:
            raise ValueError(f"q_out must be {(t, hq, d)}, got {tuple(shape)}")
    hk = ld_k = ld_ko = 0
    if k is None:
        k_out = None
    else:
        tk, hk, dk, ld_k = _rows_nd(k, "k")
        if tk != t or dk != d:
            raise ValueError(f"k must be [{t}, heads, {d}], got {tuple(k.shape)}")
        if k_out is None:
            k_out, ld_ko = torch.empty((t, hk, d), dtype=BF16, device=q.device), hk * d
        else:
            *shape, ld_ko = _rows_nd(k_out, "k_out")
            if shape != [t, hk, d]:
                raise ValueError(f"k_out must be {(t, hk, d)}, got {tuple(shape)}")
    index = _device_of(q, k, positions, inv_freq, q_out, k_out)
    _launch(index, "rope_apply", q.data_ptr(), ld_q, q_out.data_ptr(), ld_qo, hq, _ptr(k), ld_k,
            _ptr(k_out), ld_ko, hk, t, d, rot, int(bool(interleaved)), positions.data_ptr(), axes,
            _host_ints(pairs), inv_freq.data_ptr(), float(mscale), int(bool(inverse)))
    _overwritten(*given)
    return q_out, k_out


class RotaryFunction(torch.autograd.Function):
    """rope_apply with its gradient (the rotation back, scaled alike), of any order: the
    backward is this function with the direction turned."""

    @staticmethod
    def forward(ctx, q, k, positions, inv_freq, interleaved, axis_pairs, mscale, inverse=False):
        ctx.save_for_backward(positions, inv_freq)
        ctx.args = (interleaved, axis_pairs, mscale, inverse)
        return rope_apply(q, k, positions, inv_freq, *ctx.args)

    @staticmethod
    def backward(ctx, gq, gk):
        positions, inv_freq = ctx.saved_tensors
        *args, inverse = ctx.args
        turn = RotaryFunction.apply if torch.is_grad_enabled() else rope_apply
        gq, gk = turn(_loadable(gq), _loadable(gk), positions, inv_freq, *args, not inverse)
        return gq, gk, None, None, None, None, None, None


class Rotary(torch.nn.Module):
    """Rotary positions of q and k before AttnQAT: forward(q, k, positions) with q, k
    bf16 [B, N, H, D] (or [T, H, D]; a layout the kernel does not read is copied) and
    positions int32 of N (shared by the batch) or B*N rows, [rows] or [rows, axes].
    ``scaling`` and the rest as in rope_inv_freq: ONE ladder of frequencies through the pairs
    of all axes, in order.  A model whose ladder restarts with each axis gives
    inv_freq=torch.cat([rope_inv_freq(2 * n)[0] for n in axis_pairs]).
    Differentiable any number of times.  Forward and backward may be captured into one CUDA
    graph; as for every autograd function, no graph of the same leaves that was recorded
    outside the capture may be alive then."""

    def __init__(self, rot_dim: int, interleaved: bool = False, axis_pairs=None, device=None,
                 inv_freq: torch.Tensor | None = None, **frequencies):
        super().__init__()
        self.mscale = 1.0
        if inv_freq is None:
            inv_freq, self.mscale = rope_inv_freq(rot_dim, device=device, **frequencies)
        elif frequencies:
            raise ValueError(f"inv_freq is given: {', '.join(frequencies)} would not be looked at")
        if inv_freq.numel() * 2 != rot_dim:
            raise ValueError(f"inv_freq must have {rot_dim // 2} entries")
        self.register_buffer("inv_freq", inv_freq.to(device), persistent=False)
        self.interleaved, self.axis_pairs = interleaved, axis_pairs

    def _apply(self, fn, recurse=True):
        return _moved_only(self, super()._apply, fn, recurse)

    def forward(self, q, k, positions):
        t = q.shape[:-2].numel()
        if positions.shape[0] != t and q.dim() == 4 and positions.shape[0] == q.shape[1]:
            positions = positions.repeat(q.shape[0], *(1,) * (positions.dim() - 1))
        q3, k3 = (_loadable(x.reshape(t, *x.shape[-2:])) for x in (q, k))
        qo, ko = RotaryFunction.apply(q3, k3, positions, self.inv_freq, self.interleaved,
                                      self.axis_pairs, self.mscale)
        return qo.view(q.shape), ko.view(k.shape)


# ------------------------------------------------------------- paged NVFP4 KV cache

KV_PAGE = 128  # tokens per page (NVQ_KV_PAGE)


def nvfp4_kv_page_bytes(hkv: int, d: int) -> int:
    return int(_lib.load().nvfp4_kv_page_bytes(hkv, d))


def nvfp4_kv_pool(num_pages: int, hkv: int, d: int, device="cuda") -> torch.Tensor:
    """A zeroed pool of pages: uint8 [num_pages, Hkv, record bytes]."""
    record = nvfp4_kv_page_bytes(1, d)
    if num_pages < 1 or hkv < 1 or record == 0:
        raise ValueError(f"bad pool sizes: {num_pages} pages, {hkv} heads of {d}")
    return torch.zeros((num_pages, hkv, record), dtype=torch.uint8, device=device)


def _check_pool(pool, d):
    """(pages, Hkv)."""
    if not (isinstance(pool, torch.Tensor) and pool.dtype is torch.uint8):
        _check(pool, "pool", torch.uint8)
    shape = pool.shape
    if len(shape) != 3 or shape[2] != 144 * d or not pool.is_contiguous():
        raise ValueError(f"pool must be contiguous uint8 [pages, Hkv, {144 * d}], "
                         f"got {tuple(shape)}")
    return shape[0], shape[1]


def _check_cache(pool, page_table, seq_lens, d):
    """(pages, Hkv, B, max_pages, row stride of the table)."""
    pages, hkv = _check_pool(pool, d)
    (b, max_pages), (ld, _) = _int32(page_table, "page_table", 2)
    (n,), _ = _int32(seq_lens, "seq_lens", 1)
    if n != b:
        raise ValueError(f"page_table has {b} rows, seq_lens {n}")
    return pages, hkv, b, max_pages, ld if b > 1 else max_pages


def nvfp4_kv_append(k, v, seq_lens, page_table, pool, cu_tokens=None) -> None:
    """Quantizes new tokens' k, v (bf16 [T, Hkv, D], token rows may be strided) into the
    pages of ``pool``.  seq_lens int32 [B]: lengths after the append; page_table int32
    [B, max_pages]; cu_tokens int32 [B + 1] (None: one token per sequence).  No tokens, or
    no sequences, is a valid call that does nothing."""
    t, hkv, d, ld_k = _rows_nd(k, "k")
    tv, hv, dv, ld_v = _rows_nd(v, "v")
    if (tv, hv, dv) != (t, hkv, d):
        raise ValueError(f"v must be {(t, hkv, d)}, got {(tv, hv, dv)}")
    pages, heads, b, max_pages, ld_t = _check_cache(pool, page_table, seq_lens, d)
    if heads != hkv:
        raise ValueError(f"pool has {heads} heads, k {hkv}")
    if cu_tokens is not None:
        if _int32(cu_tokens, "cu_tokens", 1)[0][0] != b + 1:
            raise ValueError(f"cu_tokens must have {b + 1} entries")
    elif t != b:
        raise ValueError(f"without cu_tokens one token per sequence is expected: {t} tokens, "
                         f"{b} sequences")
    index = _device_of(k, v, seq_lens, page_table, pool, cu_tokens)
    if b == 0 and t == 0 and nvfp4_kv_page_bytes(hkv, d):  # no sequences
        return
    _launch(index, "nvfp4_kv_append", k.data_ptr(), ld_k, v.data_ptr(), ld_v, t, b, hkv, d,
            _ptr(cu_tokens), seq_lens.data_ptr(), page_table.data_ptr(), ld_t, max_pages,
            pool.data_ptr(), pages)
    _overwritten(pool)


def nvfp4_kv_append_slots(k, v, slots, pool) -> None:
    """nvfp4_kv_append with each token's place given: slots int64 [T] (nvfp4_kv_extend's), 128 *
    page + row, each once; a token of a negative slot is not written."""
    t, hkv, d, ld_k = _rows_nd(k, "k")
    tv, hv, dv, ld_v = _rows_nd(v, "v")
    if (tv, hv, dv) != (t, hkv, d):
        raise ValueError(f"v must be {(t, hkv, d)}, got {(tv, hv, dv)}")
    pages, heads = _check_pool(pool, d)
    if heads != hkv:
        raise ValueError(f"pool has {heads} heads, k {hkv}")
    _check(slots, "slots", torch.int64)
    if slots.dim() != 1 or slots.shape[0] != t or not slots.is_contiguous():
        raise ValueError(f"slots must be contiguous [{t}]")
    index = _device_of(k, v, slots, pool)
    _launch(index, "nvfp4_kv_append_slots", k.data_ptr(), ld_k, v.data_ptr(), ld_v, t, hkv, d,
            slots.data_ptr(), pool.data_ptr(), pages)
    _overwritten(pool)


class KvStep(typing.NamedTuple):
    """What nvfp4_kv_extend tells of a step."""
    seq_lens: torch.Tensor    # int32 [B], after the step
    free_count: torch.Tensor  # int32 [1], after the step
    cu_tokens: torch.Tensor   # int32 [B + 1]: offsets of the sequences' new tokens
    positions: torch.Tensor   # int32 [tokens], for rope_apply; -1 behind the last token
    slots: torch.Tensor       # int64 [tokens], for nvfp4_kv_append_slots; -1 behind the last


def _check_free(page_table, seq_lens, free_pages, free_count):
    """(B, max_pages, row stride of the table, pages)."""
    (b, max_pages), (ld, _) = _int32(page_table, "page_table", 2)
    if _int32(seq_lens, "seq_lens", 1)[0][0] != b:
        raise ValueError(f"page_table has {b} rows, seq_lens {seq_lens.shape[0]}")
    (pages,), _ = _int32(free_pages, "free_pages", 1)
    if not (isinstance(free_count, torch.Tensor) and free_count.dtype is torch.int32 and
            free_count.numel() == 1):
        raise ValueError("free_count must be an int32 tensor of one number")
    return b, max_pages, ld if b > 1 else max_pages, pages


def nvfp4_kv_extend(new_tokens, seq_lens, page_table, free_pages, free_count, tokens=None,
                    start=None, seq_lens_out=None, free_count_out=None, cu_tokens=None,
                    positions=None, slots=None) -> KvStep:
    """Pages and places for new tokens, found on the device: new_tokens and seq_lens int32 [B],
    page_table int32 [B, max_pages] (entries of new pages are written), free_pages int32
    [pages] of which the first free_count (int32 [1]) are free and the last of those are taken.
    ``tokens``: rows of positions and slots (default: one per sequence).  ``start`` int32 [B]:
    added to the positions.  seq_lens_out and free_count_out may be seq_lens and free_count (no
    other output may lie over an argument): a captured step then advances them in place.  A call
    that does not fit (pages, rows, the table's width) changes nothing, gives no tokens and is
    reported by device_status()."""
    b, max_pages, ld, pages = _check_free(page_table, seq_lens, free_pages, free_count)
    if _int32(new_tokens, "new_tokens", 1)[0][0] != b:
        raise ValueError(f"new_tokens must be [{b}], got {tuple(new_tokens.shape)}")
    if start is not None and _int32(start, "start", 1)[0][0] != b:
        raise ValueError(f"start must be [{b}], got {tuple(start.shape)}")
    t = b if tokens is None else int(tokens)
    if t < 0:
        raise ValueError(f"tokens must be >= 0, got {t}")
    given = (seq_lens_out, free_count_out, cu_tokens, positions, slots)
    out = KvStep(_check_out(seq_lens_out, "seq_lens_out", (b,), torch.int32, seq_lens),
                 _check_out(free_count_out, "free_count_out", (1,), torch.int32, seq_lens),
                 _check_out(cu_tokens, "cu_tokens", (b + 1,), torch.int32, seq_lens),
                 _check_out(positions, "positions", (t,), torch.int32, seq_lens),
                 _check_out(slots, "slots", (t,), torch.int64, seq_lens))
    index = _device_of(seq_lens, new_tokens, page_table, free_pages, free_count, start, *out)
    if index < 0:
        _check(seq_lens, "seq_lens", torch.int32)
    if b == 0:  # no sequences
        out.free_count.copy_(free_count.view(1))
        for o, v in ((out.cu_tokens, 0), (out.positions, -1), (out.slots, -1)):
            o.fill_(v)
        return out
    _launch(index, "nvfp4_kv_extend", new_tokens.data_ptr(), seq_lens.data_ptr(), _ptr(start), b,
            page_table.data_ptr(), ld, max_pages, free_pages.data_ptr(), free_count.data_ptr(),
            pages, t, *(o.data_ptr() for o in out))
    _overwritten(page_table, *given)
    return out


def nvfp4_kv_release(done, seq_lens, page_table, free_pages, free_count, seq_lens_out=None,
                     free_count_out=None):
    """The pages of the sequences with done[b] (bool [B]) back to the free ones: returns
    (seq_lens, free_count) after it, the lengths of those sequences 0; free_pages is written
    behind its first free_count entries.  seq_lens_out and free_count_out may be seq_lens and
    free_count."""
    b, max_pages, ld, pages = _check_free(page_table, seq_lens, free_pages, free_count)
    _check(done, "done", torch.bool)
    if done.dim() != 1 or done.shape[0] != b or not done.is_contiguous():
        raise ValueError(f"done must be contiguous [{b}]")
    given = (seq_lens_out, free_count_out)
    lens = _check_out(seq_lens_out, "seq_lens_out", (b,), torch.int32, seq_lens)
    count = _check_out(free_count_out, "free_count_out", (1,), torch.int32, seq_lens)
    index = _device_of(seq_lens, done, page_table, free_pages, free_count, lens, count)
    if b == 0:  # no sequences
        count.copy_(free_count.view(1))
        return lens, count
    _launch(index, "nvfp4_kv_release", done.data_ptr(), seq_lens.data_ptr(), b,
            page_table.data_ptr(), ld, max_pages, free_pages.data_ptr(), free_count.data_ptr(),
            pages, lens.data_ptr(), count.data_ptr())
    _overwritten(free_pages, *given)
    return lens, count


def attn_qat_decode_workspace(b, h, hkv, d, max_pages) -> int:
    return int(_lib.load().attn_qat_decode_workspace(b, h, hkv, d, max_pages))


def attn_qat_decode(q, pool, page_table, seq_lens, scale=None, window=0, sinks=0, o=None, lse=None,
                    workspace=None):
    """Attention of one new token per sequence over the paged cache: q bf16 [B, H, D]
    (rows may be strided), returns (o bf16 [B, H, D], lse f32 [B, H]).  ``window`` > 0:
    only the last ``window`` keys and the first ``sinks`` are visible (numbers past any
    length: all of them).  No sequences (B = 0) is a valid call that launches nothing."""
    b, h, d, ld_q = _rows_nd(q, "q")
    pages, hkv, bt, max_pages, ld_t = _check_cache(pool, page_table, seq_lens, d)
    if bt != b:
        raise ValueError(f"q has {b} rows, page_table {bt}")
    scale = _scale(scale, d)
    _check_workspace(workspace)
    given = (o, lse)
    o = _check_out(o, "o", (b, h, d), BF16, q)
    lse = _check_out(lse, "lse", (b, h), torch.float32, q)
    index = _device_of(q, pool, page_table, seq_lens, o, lse, workspace)
    if b == 0 and attn_qat_decode_workspace(1, h, hkv, d, max(max_pages, 1)):  # no sequences
        return o, lse
    ws = workspace
    if ws is None:
        ws = _workspace(_on(index, "attn_qat_decode_workspace", b, h, hkv, d, max_pages),
                        q.device, None)
    args = (q.data_ptr(), ld_q, pool.data_ptr(), pages, page_table.data_ptr(), ld_t,
            max_pages, seq_lens.data_ptr(), b, h, hkv, d, scale, _count(window), _count(sinks),
            o.data_ptr(), lse.data_ptr())
    try:
        _launch(index, "attn_qat_decode", *args, ws.data_ptr(), ws.numel() * ws.element_size())
    except _lib.NvqError as e:
        if e.status != 3 or workspace is None:
            raise
        # the caller's workspace is too small (or misaligned): one of our own, as elsewhere
        ws = _workspace(_on(index, "attn_qat_decode_workspace", b, h, hkv, d, max_pages),
                        q.device, None)
        _launch(index, "attn_qat_decode", *args, ws.data_ptr(), ws.numel())
    _overwritten(*given)
    return o, lse


def _with_workspace(index, name, args, workspace, size, like):
    """The entry point with the caller's workspace, or with one of our own where none is given
    or it is too small (or misaligned)."""
    if workspace is not None:
        try:
            return _launch(index, name, *args, workspace.data_ptr(),
                           workspace.numel() * workspace.element_size())
        except _lib.NvqError as e:
            if e.status != 3:
                raise
    ws = _workspace(_on(index, name + "_workspace", *size), like.device, None)
    _launch(index, name, *args, ws.data_ptr(), ws.numel())


def _check_offsets(cu, name, groups, rows):
    """A device list of offsets, or None for equal groups."""
    if cu is not None:
        if _int32(cu, name, 1)[0][0] != groups + 1:
            raise ValueError(f"{name} must have {groups + 1} entries")
    elif groups == 0 or rows % groups:
        raise ValueError(f"without {name} equal groups are expected: {rows} rows, {groups} groups")


def attn_qat_cross_workspace(t, b, h, hkv, d, max_pages) -> int:
    return int(_lib.load().attn_qat_cross_workspace(t, b, h, hkv, d, max_pages))


def attn_qat_cross(q, pool, page_table, kv_lens, cu_tokens=None, scale=None, o=None, lse=None,
                   workspace=None):
    """Attention of every token of a sequence to all of the sequence's cached keys (an encoder's
    states): q bf16 [T, H, D] (rows may be strided), page_table int32 [B, max_pages], kv_lens
    int32 [B]; cu_tokens int32 [B + 1] offsets of the sequences' tokens (None: T / B each).
    Returns (o bf16 [T, H, D], lse f32 [T, H]); rows without keys or outside all sequences are
    0 and -inf.  No tokens is a valid call that launches nothing."""
    t, h, d, ld_q = _rows_nd(q, "q")
    pages, hkv, b, max_pages, ld_t = _check_cache(pool, page_table, kv_lens, d)
    if t > 0 or cu_tokens is not None:
        _check_offsets(cu_tokens, "cu_tokens", b, t)
    scale = _scale(scale, d)
    _check_workspace(workspace)
    given = (o, lse)
    o = _check_out(o, "o", (t, h, d), BF16, q)
    lse = _check_out(lse, "lse", (t, h), torch.float32, q)
    index = _device_of(q, pool, page_table, kv_lens, cu_tokens, o, lse, workspace)
    if t == 0 and attn_qat_cross_workspace(1, max(b, 1), h, hkv, d, max(max_pages, 1)):
        return o, lse  # no tokens
    if b == 0 and attn_qat_cross_workspace(t, 1, h, hkv, d, 1):  # no sequences: rows outside all
        o.zero_()
        lse.fill_(-math.inf)
        return o, lse
    _with_workspace(index, "attn_qat_cross",
                    (q.data_ptr(), ld_q, t, pool.data_ptr(), pages, page_table.data_ptr(), ld_t,
                     max_pages, kv_lens.data_ptr(), _ptr(cu_tokens), b, h, hkv, d, scale,
                     o.data_ptr(), lse.data_ptr()),
                    workspace, (t, b, h, hkv, d, max_pages), q)
    _overwritten(*given)
    return o, lse


def attn_qat_decode_prefix_workspace(b, groups, h, hkv, d, max_pages, prefix_pages) -> int:
    return int(_lib.load().attn_qat_decode_prefix_workspace(b, groups, h, hkv, d, max_pages,
                                                            prefix_pages))


def attn_qat_decode_prefix(q, pool, page_table, seq_lens, prefix_table, prefix_lens, cu_seqs=None,
                           scale=None, o=None, lse=None, workspace=None):
    """attn_qat_decode where groups of sequences share cached prefixes, each read once:
    page_table and seq_lens tell of the sequences' own keys, prefix_table int32 [S, pages] and
    prefix_lens int32 [S] of the shared ones, cu_seqs int32 [S + 1] which sequences share them
    (None: B / S consecutive ones each).  Returns (o bf16 [B, H, D], lse f32 [B, H]) over both
    together.  No sequences is a valid call that launches nothing."""
    b, h, d, ld_q = _rows_nd(q, "q")
    pages, hkv, bt, max_pages, ld_t = _check_cache(pool, page_table, seq_lens, d)
    if bt != b:
        raise ValueError(f"q has {b} rows, page_table {bt}")
    _, _, s, prefix_pages, ld_p = _check_cache(pool, prefix_table, prefix_lens, d)
    if b > 0 or cu_seqs is not None:
        _check_offsets(cu_seqs, "cu_seqs", s, b)
    if s == 0:  # no prefixes (offsets of no groups)
        return attn_qat_decode(q, pool, page_table, seq_lens, scale, 0, 0, o, lse, workspace)
    scale = _scale(scale, d)
    _check_workspace(workspace)
    given = (o, lse)
    o = _check_out(o, "o", (b, h, d), BF16, q)
    lse = _check_out(lse, "lse", (b, h), torch.float32, q)
    index = _device_of(q, pool, page_table, seq_lens, prefix_table, prefix_lens, cu_seqs, o, lse,
                       workspace)
    if b == 0 and attn_qat_decode_prefix_workspace(1, s, h, hkv, d, max(max_pages, 1),
                                                   max(prefix_pages, 1)):
        return o, lse  # no sequences
    _with_workspace(index, "attn_qat_decode_prefix",
                    (q.data_ptr(), ld_q, pool.data_ptr(), pages, page_table.data_ptr(), ld_t,
                     max_pages, seq_lens.data_ptr(), prefix_table.data_ptr(), ld_p, prefix_pages,
                     prefix_lens.data_ptr(), _ptr(cu_seqs), s, b, h, hkv, d, scale, o.data_ptr(),
                     lse.data_ptr()),
                    workspace, (b, s, h, hkv, d, max_pages, prefix_pages), q)
    _overwritten(*given)
    return o, lse


# Kernel kinds of nvq_timing_read (include/nvfp4attn.h, NVQ_KERNEL_*)
KERNEL_KINDS = {"quantize": 0, "attn_fwd": 1, "bwd_delta": 2, "bwd_dkdv": 3, "bwd_dq": 4,
                "global_sf": 5, "vsa": 6, "linear": 7}
SERVING_KINDS = {"rope": 16, "kv_append": 17, "decode": 18, "kv_tables": 19, "cross": 20}


def timing_enable(on: bool = True) -> None:
    """Start (discarding earlier records) or stop per-kernel event timing."""
    _lib.call("nvq_timing_enable", int(bool(on)))


def timing_read() -> dict:
    """{kind: (launches, total_ms)} for the launches recorded since timing_enable(True):
    every kind of KERNEL_KINDS, and those of SERVING_KINDS that were launched."""
    import ctypes
    out = {}
    for name, kind in (KERNEL_KINDS | SERVING_KINDS).items():
        n, ms = ctypes.c_int64(0), ctypes.c_double(0.0)
        _lib.call("nvq_timing_read", kind, ctypes.addressof(n), ctypes.addressof(ms))
        if n.value or name in KERNEL_KINDS:
            out[name] = (int(n.value), float(ms.value))
    return out


# ------------------------------------------------------- block-sparse (VSA)

VSA_TILE = 128  # tokens per tile: one 4x4x8 cube


def _check_tiles(kv_tiles, b, h, n):
    _check(kv_tiles, "kv_tiles", torch.int32)
    if kv_tiles.dim() != 4 or tuple(kv_tiles.shape[:3]) != (b, h, n // VSA_TILE) or \
            not kv_tiles.is_contiguous():
        raise ValueError(f"kv_tiles must be contiguous int32 [B, H, N/128, topk] = "
                         f"[{b}, {h}, {n // VSA_TILE}, topk], got {tuple(kv_tiles.shape)}")


def vsa_effective_topk(sparsity: float, num_blocks: int) -> int:
    """max(1, min(ceil((1 - sparsity) * num_blocks), num_blocks)) (the VSA metadata's formula)."""
    return max(1, min(math.ceil((1.0 - sparsity) * num_blocks), num_blocks))


def vsa_reorder(x, grid, cube=(4, 4, 8), to_cubes=True, out=None):
    """Token rows of bf16 [B, T*Hh*W, H, D] between raster and cube order."""
    _check(x, "x", torch.bfloat16)
    b, n, h, d = x.shape
    t, hh, w = grid
    if n != t * hh * w:
        raise ValueError(f"x has {n} tokens, the grid {t}x{hh}x{w}")
    out = torch.empty_like(x) if out is None else out
    _lib.call("vsa_reorder", _ptr(x), b, t, hh, w, h, d, cube[0], cube[1], cube[2],
              int(bool(to_cubes)), _ptr(out), _stream_ptr(x))
    return out


def vsa_select_tiles(q, k, topk, workspace=None):
    """int32 [B, H, N/128, topk]: per query tile the topk key tiles by cube-mean score."""
    _check_bnhd(q, "q")
    _check_bnhd(k, "k", q.shape)
    b, n, h, d = q.shape
    out = torch.empty((b, h, n // VSA_TILE, topk), dtype=torch.int32, device=q.device)
    need = vsa_select_workspace(b, n, h, d)
    ws = _workspace(need, q.device, workspace)
    _lib.call("vsa_select_tiles", _ptr(q), _ptr(k), b, n, h, d, int(topk), _ptr(out), _ptr(ws),
              ws.numel() * ws.element_size(), _stream_ptr(q))
    return out


def attn_qat_fwd_sparse(q, k, v, kv_tiles, scale=None, o=None, stats=None, workspace=None):
    """Block-sparse forward (tokens in cube order): (o, stats)."""
    _check_bnhd(q, "q")
    b, n, h, d = q.shape
    _check_bnhd(k, "k", q.shape)
    _check_bnhd(v, "v", q.shape)
    _check_tiles(kv_tiles, b, h, n)
    topk = kv_tiles.shape[-1]
    scale = _scale(scale, d)
    o = torch.empty_like(q) if o is None else o
    if stats is None:
        stats = torch.empty((b, h, 2, n), dtype=torch.float32, device=q.device)
    ws = _workspace(attn_qat_fwd_workspace(b, n, n, h, d), q.device, workspace)
    _lib.call("attn_qat_fwd_sparse", _ptr(q), _ptr(k), _ptr(v), b, n, h, d, scale, _ptr(kv_tiles),
              topk, _ptr(o), _ptr(stats), _ptr(ws), ws.numel() * ws.element_size(),
              _stream_ptr(q))
    return o, stats


def attn_qat_bwd_sparse_workspace(b, n, h, d, topk) -> int:
    return int(_lib.load().attn_qat_bwd_sparse_workspace(b, n, h, d, topk))


def vsa_select_workspace(b, n, h, d) -> int:
    return int(_lib.load().vsa_select_workspace(b, n, h, d))


def attn_qat_bwd_sparse(q, k, v, o, stats, do, kv_tiles, scale=None, dq=None, dk=None, dv=None,
                        workspace=None):
    """Block-sparse straight-through backward: (dq, dk, dv)."""
    _check_bnhd(q, "q")
    b, n, h, d = q.shape
    for t_, name in ((k, "k"), (v, "v"), (o, "o"), (do, "do")):
        _check_bnhd(t_, name, q.shape)
    _check(stats, "stats", torch.float32)
    _check_tiles(kv_tiles, b, h, n)
    topk = kv_tiles.shape[-1]
    scale = _scale(scale, d)
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    need = attn_qat_bwd_sparse_workspace(b, n, h, d, topk)
    ws = _workspace(need, q.device, workspace)
    _lib.call("attn_qat_bwd_sparse", _ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(stats), _ptr(do),
              _ptr(kv_tiles), topk, _ptr(dq), _ptr(dk), _ptr(dv), b, n, h, d, scale, _ptr(ws),
              ws.numel() * ws.element_size(), _stream_ptr(q))
    return dq, dk, dv


def attn_qat_bwd_sparse_saved_workspace(b, n, h, d, topk) -> int:
    return int(_lib.load().attn_qat_bwd_sparse_saved_workspace(b, n, h, d, topk))


def attn_qat_bwd_sparse_saved(saved, o, stats, do, kv_tiles, scale=None, dq=None, dk=None,
                              dv=None, workspace=None):
    """Block-sparse backward from the quantized operands attn_qat_fwd_sparse left in
    its workspace ``saved`` (same q, k, v and kv_tiles): (dq, dk, dv), equal to
    attn_qat_bwd_sparse's bit for bit, without its quantizer pass."""
    _check_bnhd(o, "o")
    b, n, h, d = o.shape
    _check_bnhd(do, "do", o.shape)
    _check(stats, "stats", torch.float32)
    _check(saved, "saved", torch.uint8)
    _check_tiles(kv_tiles, b, h, n)
    topk = kv_tiles.shape[-1]
    scale = _scale(scale, d)
    dq = torch.empty_like(o) if dq is None else dq
    dk = torch.empty_like(o) if dk is None else dk
    dv = torch.empty_like(o) if dv is None else dv
    ws = _workspace(attn_qat_bwd_sparse_saved_workspace(b, n, h, d, topk), o.device, workspace)
    _lib.call("attn_qat_bwd_sparse_saved", _ptr(saved), saved.numel(), _ptr(o), _ptr(stats),
              _ptr(do), _ptr(kv_tiles), topk, _ptr(dq), _ptr(dk), _ptr(dv), b, n, h, d, scale,
              _ptr(ws), ws.numel() * ws.element_size(), _stream_ptr(o))
    return dq, dk, dv


def device_status(device=None) -> int:
    """Synchronize the current stream and return (and clear) the device error word."""
    s = torch.cuda.current_stream(device).cuda_stream
    return int(_lib.load().nvq_device_status(s))


DELTA_MODES = ("o", "hp")


class AttnQATFunction(torch.autograd.Function):
    """O = attention with NVFP4 fake-quantized Q, K, V, P; straight-through backward.
    ``delta_mode`` "o": the backward's delta = rowsum(dO * O); "hp": from the
    auxiliary high-precision output P V~ / l, which the forward then also computes."""

    @staticmethod
    def forward(ctx, q, k, v, scale, causal, delta_mode="o"):
        b, nq, h, d = q.shape
        # the forward's workspace keeps Q~, K~, V~ in every form the backward
        # reads: it is saved instead of q, k, v, and the backward quantizes nothing
        saved = torch.empty(attn_qat_fwd_workspace(b, nq, k.shape[1], h, d), dtype=torch.uint8,
                            device=q.device)
        if delta_mode == "hp":
            o, o_d, stats = attn_qat_fwd_hp(q, k, v, scale, causal, workspace=saved)
        elif delta_mode == "o":
            o, stats = attn_qat_fwd(q, k, v, scale, causal, workspace=saved)
            o_d = o
        else:
            raise ValueError(f"delta_mode must be one of {DELTA_MODES}, got {delta_mode!r}")
        ctx.save_for_backward(saved, o_d, stats)
        ctx.scale, ctx.causal, ctx.nkv = scale, causal, k.shape[1]
        return o

    @staticmethod
    def backward(ctx, do):
        saved, o_d, stats = ctx.saved_tensors
        dq, dk, dv = attn_qat_bwd_saved(saved, o_d, stats, do.contiguous(), ctx.scale,
                                        ctx.causal, nkv=ctx.nkv)
        return dq, dk, dv, None, None, None


class AttnQAT(torch.nn.Module):
    """``AttentionImpl(num_heads, head_size, softmax_scale, causal)`` with ``forward(q, k, v)``.

    ``delta_mode`` chooses where the backward's delta comes from.  The default
    "o" takes it from the returned output O (the exact straight-through
    derivative of the forward, the reading the parity tests use).  This differs
    from the pages: ``attn_qat_train()`` ("attn_qat_train" API page) hard-codes
    ``use_high_prec_o = True``, i.e. delta from the auxiliary high-precision
    output P V~ / l, which ``delta_mode="hp"`` selects.
    """

    def __init__(self, num_heads: int, head_size: int, softmax_scale: float | None = None,
                 causal: bool = False, dropout_p: float = 0.0, delta_mode: str = "o"):
        super().__init__()
        if delta_mode not in DELTA_MODES:
            raise ValueError(f"delta_mode must be one of {DELTA_MODES}, got {delta_mode!r}")
        if dropout_p > 0:
            raise NotImplementedError(
                f"NVFP4 Attn-QAT attention applies no dropout (got dropout_p={dropout_p})")
        if head_size not in (64, 128):
            raise ValueError(f"head_size must be 64 or 128, got {head_size}")
        self.num_heads, self.head_size = num_heads, head_size
        self.softmax_scale = default_scale(head_size) if softmax_scale is None else softmax_scale
        self.causal = causal
        self.delta_mode = delta_mode

    def forward(self, q, k, v):
        return AttnQATFunction.apply(q, k, v, self.softmax_scale, self.causal, self.delta_mode)
