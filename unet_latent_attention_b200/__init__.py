"""Python binding of the sm_100a latent-diffusion hot-path library (``libsdk.so``).

Argument marshalling only: every step runs in the CUDA kernels behind the C ABI declared in
``include/sd_kernels.h``. PyTorch supplies device memory and the current CUDA stream. There is no
CPU fallback: if the library is missing or the tensors are not on a CUDA device, the calls raise.

    sd_group_norm(x, gamma, beta, groups=32, eps=1e-5, out=None)
    sd_group_norm_silu(x, gamma, beta, groups=32, eps=1e-5, out=None, out_dtype=None)
    sd_attention(q, k, v, scale=None, out=None)          (bf16 or fp16)
    sd_cfg_ddim_step(x, eps_u, eps_c, w, alpha_t, alpha_prev, out=None)
    sd_cfg_ddim_step_from_noise_pred(x, noise_pred, w, alpha_t, alpha_prev, out=None)
    sd_cfg_dpmpp_2m_step(x, eps_u, eps_c, d_prev, w, alpha_prev, alpha_t, alpha_next, order, out=None, d_out=None)

and, for transformer blocks, in the order in which a block calls them:

    sd_rms_norm(x, weight, eps=1e-6, residual=None)                  -> y or (y, residual)
    sd_rms_norm_fp8(x, weight, eps=1e-6, residual=None, block=0)     -> (y, scales) or (y, scales, residual)
    sd_rope_axes(q, k, positions, freqs, axis_dims, ...)             -> (q, k)     (freqs: rope_frequencies)
    sd_attention_masked(q, k, v, causal=, cap=, bias=, kv_lens=, q_offsets=, ...)
"""
from __future__ import annotations

import ctypes
import math
import os
import re
import struct

from .rope import rope_frequencies  # noqa: F401
from .schedule import (ddim_schedule, dpmpp_2m_schedule, dpmpp_3m_schedule, karras_alpha_bars,  # noqa: F401
                       scaled_linear_alphas_cumprod)

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libsdk.so")
HEADER_PATH = os.path.join(os.path.dirname(_HERE), "include", "sd_kernels.h")

SD_OK = 0
STATUS_NAMES = {0: "SD_OK", 1: "SD_ERR_INVALID_ARG", 2: "SD_ERR_UNSUPPORTED", 3: "SD_ERR_MISALIGNED",
                4: "SD_ERR_CUDA", 5: "SD_ERR_TIMEOUT"}


class SDError(RuntimeError):
    """A non-zero sd_status from the library."""

    def __init__(self, func: str, status: int, detail: str):
        self.status = status
        super().__init__(f"{func}: {STATUS_NAMES.get(status, status)}: {detail}")


# Layouts of the argument structs of include/sd_kernels.h (packed bytes cost a call far less than
# filling a ctypes.Structure field by field).
# sd_rope_args: 8 pointers, B .. dh, 4 x 3 strides, positions_batch_stride, axis_dims[4], axes, pairs, dtype, eps
_ROPE_ARGS = struct.Struct("@8P5q12qq4i3if")
# sd_attention_masked_args: 10 pointers, B .. dh, 4 x 3 strides, bias_radius, docs, causal, dtype, scale, cap
_ATTENTION_MASKED_ARGS = struct.Struct("@10P6q12q2q2i2f")


_lib = None


def lib() -> ctypes.CDLL:
    """Load libsdk.so once (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with `python -m unet_latent_attention_b200.build`")
        L = ctypes.CDLL(LIB_PATH)
        i64, f32, f64, vp, c_int = ctypes.c_int64, ctypes.c_float, ctypes.c_double, ctypes.c_void_p, ctypes.c_int
        L.sd_group_norm.argtypes = [vp, vp, vp, vp, i64, i64, i64, i64, i64, f32, vp]
        L.sd_group_norm_silu.argtypes = [vp, vp, vp, vp, i64, i64, i64, i64, i64, f32, c_int, vp]
        L.sd_attention.argtypes = [vp, vp, vp, vp, i64, i64, i64, i64, i64, f32, vp]
        L.sd_attention_noalloc.argtypes = [vp, vp, vp, vp, i64, i64, i64, i64, i64, f32, vp]
        L.sd_attention_f16.argtypes = [vp, vp, vp, vp, i64, i64, i64, i64, i64, f32, vp]
        L.sd_attention_layout.argtypes = [vp, vp, vp, vp, i64, i64, i64, i64, i64, f32, c_int, c_int, vp]
        L.sd_cfg_ddim_step.argtypes = [vp, vp, vp, vp, i64, f32, f64, f64, vp]
        L.sd_cfg_dpmpp_2m_step.argtypes = [vp, vp, vp, vp, vp, vp, i64, f32, f64, f64, f64, c_int, vp]
        L.sd_cfg_dpmpp_3m_step.argtypes = [vp, vp, vp, vp, vp, vp, vp, i64, f32, f64, f64, f64, f64, vp]
        L.sd_rms_norm.argtypes = [vp] * 5 + [i64] * 6 + [f32, c_int, c_int, vp]
        L.sd_rms_norm_fp8.argtypes = [vp] * 6 + [i64] * 6 + [f32, c_int, c_int, c_int, vp]
        L.sd_rope_axes.argtypes = [ctypes.c_char_p, vp]
        L.sd_attention_masked.argtypes = [ctypes.c_char_p, vp]
        L.sd_device_status.argtypes = [vp, c_int]
        L.sd_debug_set_fault.argtypes = [c_int]
        L.sd_debug_set_fault.restype = None
        for f in ("sd_group_norm", "sd_group_norm_silu", "sd_attention", "sd_attention_noalloc", "sd_attention_f16",
                  "sd_attention_layout", "sd_rms_norm", "sd_rms_norm_fp8", "sd_rope_axes", "sd_attention_masked",
                  "sd_cfg_ddim_step",
                  "sd_cfg_dpmpp_2m_step", "sd_cfg_dpmpp_3m_step", "sd_device_status"):
            getattr(L, f).restype = c_int
        L.sd_status_string.argtypes = [c_int]
        L.sd_status_string.restype = ctypes.c_char_p
        L.sd_last_error.argtypes = []
        L.sd_last_error.restype = ctypes.c_char_p
        L.sd_version.restype = c_int
        _lib = L
    return _lib


def header_functions() -> list[str]:
    """Names of the functions that include/sd_kernels.h declares."""
    text = open(HEADER_PATH).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return sorted(set(re.findall(r"\b(sd_[a-z_0-9]+)\s*\(", text)))


def _check(func: str, status: int) -> None:
    if status != SD_OK:
        raise SDError(func, status, lib().sd_last_error().decode(errors="replace"))


def _stream(t) -> int:
    import torch
    return torch.cuda.current_stream(t.device).cuda_stream


def _require_cuda(*ts) -> None:
    for t in ts:
        if not t.is_cuda:
            raise ValueError("sd kernels run on CUDA tensors only (no CPU fallback)")
        if not t.is_contiguous():
            raise ValueError("sd kernels take contiguous tensors")


def sd_group_norm(x, gamma, beta, groups: int = 32, eps: float = 1e-5, out=None):
    """GroupNorm of fp32 NCHW ``x`` with per-channel ``gamma``/``beta``; ``out`` may be ``x``."""
    import torch
    if x.dtype != torch.float32 or gamma.dtype != torch.float32 or beta.dtype != torch.float32:
        raise ValueError("sd_group_norm takes fp32 tensors")
    if x.dim() != 4:
        raise ValueError("x must be [B, C, H, W]")
    if out is None:
        out = torch.empty_like(x)
    _require_cuda(x, gamma, beta, out)
    B, C, H, W = x.shape
    if gamma.numel() != C or beta.numel() != C or out.shape != x.shape:
        raise ValueError("gamma/beta must have C elements and out the shape of x")
    _check("sd_group_norm", lib().sd_group_norm(x.data_ptr(), gamma.data_ptr(), beta.data_ptr(), out.data_ptr(),
                                                B, C, H, W, groups, eps, _stream(x)))
    return out


def sd_group_norm_silu(x, gamma, beta, groups: int = 32, eps: float = 1e-5, out=None, out_dtype=None):
    """SiLU(GroupNorm(x)) of fp32 NCHW ``x`` in one launch; the output is fp32 (``out`` may be ``x``)
    or bf16 (``out_dtype=torch.bfloat16``)."""
    import torch
    if x.dtype != torch.float32 or gamma.dtype != torch.float32 or beta.dtype != torch.float32:
        raise ValueError("sd_group_norm_silu takes fp32 x, gamma, beta")
    if x.dim() != 4:
        raise ValueError("x must be [B, C, H, W]")
    if out is None:
        out = torch.empty(x.shape, dtype=out_dtype or torch.float32, device=x.device)
    if out.dtype not in (torch.float32, torch.bfloat16) or out.shape != x.shape:
        raise ValueError("out must be fp32 or bf16 with the shape of x")
    _require_cuda(x, gamma, beta, out)
    B, C, H, W = x.shape
    if gamma.numel() != C or beta.numel() != C:
        raise ValueError("gamma/beta must have C elements")
    _check("sd_group_norm_silu", lib().sd_group_norm_silu(x.data_ptr(), gamma.data_ptr(), beta.data_ptr(),
                                                          out.data_ptr(), B, C, H, W, groups, eps,
                                                          1 if out.dtype == torch.bfloat16 else 0, _stream(x)))
    return out


def sd_attention(q, k, v, scale: float | None = None, out=None, layout: str = "bhld"):
    """softmax(q k^T * scale) v for q [B,h,Lq,dh], k/v [B,h,Lk,dh] (layout "bhld") or q [B,Lq,h,dh],
    k/v [B,Lk,h,dh] (layout "blhd"), all bf16 or all fp16 (the output has the type and layout of q);
    scale defaults to 1/sqrt(dh)."""
    import torch
    if q.dtype not in (torch.bfloat16, torch.float16) or k.dtype != q.dtype or v.dtype != q.dtype:
        raise ValueError("sd_attention takes q, k, v all bf16 or all fp16")
    if q.dim() != 4 or k.dim() != 4 or v.dim() != 4:
        raise ValueError("q, k, v must be 4-D")
    if layout not in ("bhld", "blhd"):
        raise ValueError("layout must be 'bhld' or 'blhd'")
    if layout == "blhd":
        B, Lq, Hh, dh = q.shape
        Lk = k.shape[1]
        if k.shape != (B, Lk, Hh, dh) or v.shape != k.shape:
            raise ValueError("k and v must be [B, Lk, heads, dh] matching q")
    else:
        B, Hh, Lq, dh = q.shape
        Lk = k.shape[2]
        if k.shape[:2] != (B, Hh) or v.shape != k.shape or k.shape[3] != dh:
            raise ValueError("k and v must be [B, heads, Lk, dh] matching q")
    if out is None:
        out = torch.empty_like(q)
    _require_cuda(q, k, v, out)
    if out.shape != q.shape or out.dtype != q.dtype:
        raise ValueError("out must have the shape and type of q")
    if scale is None:
        scale = 1.0 / math.sqrt(dh)
    f16, blhd = q.dtype == torch.float16, layout == "blhd"
    if not f16 and not blhd:
        st = lib().sd_attention(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), B, Hh, Lq, Lk, dh, scale,
                                _stream(q))
    else:
        st = lib().sd_attention_layout(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), B, Hh, Lq, Lk, dh,
                                       scale, int(f16), int(blhd), _stream(q))
    _check("sd_attention", st)
    return out


def sd_attention_noalloc(q, k, v, scale: float | None = None, out=None):
    """sd_attention (bf16, [B, heads, L, dh]) without any device allocation by the library: its
    split-item scratch is a fixed 16 MiB device array instead of a cudaMalloc'd workspace.

    For callers that cannot let a library call cudaMalloc: inside CUDA-graph capture, under a
    framework that owns all device memory, or in loops that cannot absorb cudaMalloc's implicit
    synchronisation. Pass ``out`` to avoid the allocation of the output tensor as well. Calls that
    overlap on the GPU race on the shared scratch.
    """
    import torch
    if q.dtype != torch.bfloat16 or k.dtype != torch.bfloat16 or v.dtype != torch.bfloat16:
        raise ValueError("sd_attention_noalloc takes bf16 q, k, v")
    if q.dim() != 4 or k.dim() != 4 or v.dim() != 4:
        raise ValueError("q, k, v must be 4-D [B, heads, L, dh]")
    B, Hh, Lq, dh = q.shape
    Lk = k.shape[2]
    if k.shape != (B, Hh, Lk, dh) or v.shape != k.shape:
        raise ValueError("k and v must be [B, heads, Lk, dh] matching q")
    if out is None:
        out = torch.empty_like(q)
    if out.shape != q.shape or out.dtype != q.dtype:
        raise ValueError("out must have the shape and type of q")
    _require_cuda(q, k, v, out)
    if scale is None:
        scale = 1.0 / math.sqrt(dh)
    _check("sd_attention_noalloc", lib().sd_attention_noalloc(q.data_ptr(), k.data_ptr(), v.data_ptr(),
                                                              out.data_ptr(), B, Hh, Lq, Lk, dh, scale,
                                                              _stream(q)))
    return out


def sd_cfg_ddim_step(x, eps_u, eps_c, w: float, alpha_t: float, alpha_prev: float, out=None):
    """x' = DDIM(eta=0) step of fp32 latent x with guided noise eps_u + w (eps_c - eps_u); out may be x."""
    import torch
    for t in (x, eps_u, eps_c):
        if t.dtype != torch.float32:
            raise ValueError("sd_cfg_ddim_step takes fp32 tensors")
    if eps_u.shape != x.shape or eps_c.shape != x.shape:
        raise ValueError("eps_u and eps_c must have the shape of x")
    if out is None:
        out = torch.empty_like(x)
    _require_cuda(x, eps_u, eps_c, out)
    _check("sd_cfg_ddim_step", lib().sd_cfg_ddim_step(x.data_ptr(), eps_u.data_ptr(), eps_c.data_ptr(),
                                                      out.data_ptr(), x.numel(), w, alpha_t, alpha_prev,
                                                      _stream(x)))
    return out


def sd_cfg_ddim_step_from_noise_pred(x, noise_pred, w: float, alpha_t: float, alpha_prev: float, out=None):
    """Same step taking the UNet output for the batch [uncond, cond] (uncond half first)."""
    eps_u, eps_c = noise_pred.chunk(2, dim=0)
    return sd_cfg_ddim_step(x, eps_u, eps_c, w, alpha_t, alpha_prev, out=out)


def sd_cfg_dpmpp_2m_step(x, eps_u, eps_c, d_prev, w: float, alpha_prev: float, alpha_t: float, alpha_next: float,
                         order: int, out=None, d_out=None):
    """Guided DPM-Solver++(2M) step; returns (x_next, d) where d is this step's data prediction (the
    history for the next step). ``d_prev`` is the previous step's d (unused, may be None, for order 1);
    ``out`` may be ``x`` and ``d_out`` may be ``d_prev``."""
    import torch
    for t in (x, eps_u, eps_c) + ((d_prev,) if d_prev is not None else ()):
        if t.dtype != torch.float32 or t.shape != x.shape:
            raise ValueError("sd_cfg_dpmpp_2m_step takes fp32 tensors of one shape")
    if order == 2 and d_prev is None:
        raise ValueError("order 2 needs d_prev")
    out = torch.empty_like(x) if out is None else out
    d_out = torch.empty_like(x) if d_out is None else d_out
    _require_cuda(x, eps_u, eps_c, out, d_out, *((d_prev,) if d_prev is not None else ()))
    _check("sd_cfg_dpmpp_2m_step", lib().sd_cfg_dpmpp_2m_step(
        x.data_ptr(), eps_u.data_ptr(), eps_c.data_ptr(), d_prev.data_ptr() if d_prev is not None else None,
        out.data_ptr(), d_out.data_ptr(), x.numel(), w, alpha_prev, alpha_t, alpha_next, int(order), _stream(x)))
    return out, d_out


def sd_cfg_dpmpp_3m_step(x, eps_u, eps_c, d_prev, d_prev2, w: float, alpha_prev2: float, alpha_prev: float,
                         alpha_t: float, alpha_next: float, out=None, d_out=None):
    """Guided third-order multistep DPM-Solver++ step; returns (x_next, d). ``out`` may be ``x``;
    ``d_out`` may be ``d_prev`` or ``d_prev2``."""
    import torch
    for t in (x, eps_u, eps_c, d_prev, d_prev2):
        if t.dtype != torch.float32 or t.shape != x.shape:
            raise ValueError("sd_cfg_dpmpp_3m_step takes fp32 tensors of one shape")
    out = torch.empty_like(x) if out is None else out
    d_out = torch.empty_like(x) if d_out is None else d_out
    _require_cuda(x, eps_u, eps_c, d_prev, d_prev2, out, d_out)
    _check("sd_cfg_dpmpp_3m_step", lib().sd_cfg_dpmpp_3m_step(
        x.data_ptr(), eps_u.data_ptr(), eps_c.data_ptr(), d_prev.data_ptr(), d_prev2.data_ptr(), out.data_ptr(),
        d_out.data_ptr(), x.numel(), w, alpha_prev2, alpha_prev, alpha_t, alpha_next, _stream(x)))
    return out, d_out


def _device_index(first, others) -> int:
    """The index of the CUDA device that holds all the tensors (None entries are skipped; views may be strided)."""
    dev = first.get_device()
    if dev < 0 or not first.is_cuda:
        raise ValueError("sd kernels run on CUDA tensors only (no CPU fallback)")
    for t in others:
        if t is not None and t.get_device() != dev:
            raise ValueError("sd kernels run on CUDA tensors only (no CPU fallback)" if t.get_device() < 0
                             else "all tensors must be on one CUDA device")
    return dev


_torch_c = None


def _call(name, dev: int, *args) -> None:
    """One library call on the current stream of device ``dev``, with ``dev`` as the current device."""
    global _torch_c
    if _torch_c is None:
        import torch
        _torch_c = torch._C
    f = getattr(_lib or lib(), name)
    if _torch_c._cuda_getDevice() == dev:
        st = f(*args, _torch_c._cuda_getCurrentRawStream(dev))
    else:
        import torch
        with torch.cuda.device(dev):
            st = f(*args, _torch_c._cuda_getCurrentRawStream(dev))
    if st != SD_OK:
        _check(name, st)


def _ptr(t) -> int:
    return 0 if t is None else t.data_ptr()


def _row_stride(t, name):
    """Elements between the rows of a tensor whose last dimension is contiguous."""
    C = t.shape[-1]
    if C > 1 and t.stride(-1) != 1:
        raise ValueError(f"the last dimension of {name} must be contiguous")
    n, step = 1, None
    for size, stride in zip(reversed(t.shape[:-1]), reversed(t.stride()[:-1])):
        if size == 1:
            continue
        if step is None:
            step = stride
        elif stride != step * n:
            raise ValueError(f"the rows of {name} must be equally far apart")
        n *= size
    return C if step is None else step


_DTYPE_CODES = {}


def _dtype_code(t, func):
    if not _DTYPE_CODES:
        import torch
        _DTYPE_CODES.update({torch.bfloat16: 0, torch.float16: 1, torch.float32: 2})
    code = _DTYPE_CODES.get(t.dtype)
    if code is None:
        raise ValueError(f"{func} takes bf16, fp16 or fp32 tensors")
    return code


def _rms(func, x, weight, eps, residual, out, residual_out, scales, block):
    import torch
    code = _dtype_code(x, func)
    shape, dtype = x.shape, x.dtype
    C = shape[-1]
    if residual is not None:
        if residual.shape != shape or residual.dtype != dtype:
            raise ValueError("residual must have the shape and type of x")
        if residual_out is None:
            residual_out = torch.empty_like(residual) if residual.is_contiguous() else torch.empty(shape, dtype=dtype, device=x.device)
        elif residual_out.shape != shape or residual_out.dtype != dtype:
            raise ValueError("residual_out must have the shape and type of x")
    elif residual_out is not None:
        raise ValueError("residual_out needs residual")
    wf32 = 1
    if weight is not None:
        wf32 = int(weight.dtype == torch.float32)
        if weight.shape != (C,) or not (wf32 or weight.dtype == dtype) or not weight.is_contiguous():
            raise ValueError("weight must be [C], contiguous, fp32 or of the type of x")
    dev = _device_index(x, (weight, residual, out, residual_out, scales))
    rows = x.numel() // C if C else 0
    xs = C if x.is_contiguous() else _row_stride(x, "x")
    ys = C if out.is_contiguous() else _row_stride(out, "out")
    rs = ros = C
    rp = rop = 0
    if residual is not None:
        rp, rop = residual.data_ptr(), residual_out.data_ptr()
        if not residual.is_contiguous():
            rs = _row_stride(residual, "residual")
        if not residual_out.is_contiguous():
            ros = _row_stride(residual_out, "residual_out")
    wp = 0 if weight is None else weight.data_ptr()
    if scales is None:
        _call(func, dev, x.data_ptr(), rp, wp, out.data_ptr(), rop, rows, C, xs, rs, ys, ros, eps, code, wf32)
    else:
        _call(func, dev, x.data_ptr(), rp, wp, out.data_ptr(), scales.data_ptr(), rop, rows, C, xs, rs, ys, ros, eps, code,
              wf32, block)
    return residual_out


def sd_rms_norm(x, weight=None, eps: float = 1e-6, residual=None, out=None, residual_out=None):
    """RMS norm over the last dimension of ``x`` (bf16, fp16 or fp32), or of ``x + residual``.

    ``weight`` is [C] in fp32 or the type of x (None: ones). Returns y, or (y, residual_out) with
    residual_out = x + residual where a residual is given. ``out`` and ``residual_out`` may be ``x`` or
    ``residual`` (in place); rows may be strided, columns are contiguous."""
    import torch
    if x.dim() < 1:
        raise ValueError("x must have at least one dimension")
    if out is None:
        out = torch.empty_like(x) if x.is_contiguous() else torch.empty(x.shape, dtype=x.dtype, device=x.device)
    elif out.shape != x.shape or out.dtype != x.dtype:
        raise ValueError("out must have the shape and type of x")
    ro = _rms("sd_rms_norm", x, weight, float(eps), residual, out, residual_out, None, 0)
    return out if ro is None else (out, ro)


def sd_rms_norm_fp8(x, weight=None, eps: float = 1e-6, residual=None, block: int = 0, out=None, scales=None,
                    residual_out=None):
    """sd_rms_norm with an e4m3 output: y = out * scale, a scale for each ``block`` columns of a row (32, 64
    or 128; 0: one a row). Returns (out, scales) or (out, scales, residual_out); scales is fp32
    [..., ceil(C / block)] ([..., 1] for block 0)."""
    import torch
    if block not in (0, 32, 64, 128):
        raise ValueError("block must be 0, 32, 64 or 128")
    if x.dim() < 1:
        raise ValueError("x must have at least one dimension")
    C = x.shape[-1]
    shape = (*x.shape[:-1], -(-C // block) if block else 1)
    if out is None:
        out = (torch.empty_like(x, dtype=torch.float8_e4m3fn) if x.is_contiguous()
               else x.new_empty(x.shape, dtype=torch.float8_e4m3fn))
    elif out.shape != x.shape or out.dtype != torch.float8_e4m3fn:
        raise ValueError("out must have the shape of x and type float8_e4m3fn")
    if scales is None:
        scales = x.new_empty(shape, dtype=torch.float32)
    elif scales.shape != shape or scales.dtype != torch.float32 or not scales.is_contiguous():
        raise ValueError(f"scales must be contiguous fp32 {list(shape)}")
    ro = _rms("sd_rms_norm_fp8", x, weight, float(eps), residual, out, residual_out, scales, block)
    return (out, scales) if ro is None else (out, scales, ro)


def _strides(t, blhd, name):
    """{batch, token, head} strides of a 4-D view with contiguous columns."""
    b, m, n, c = t.stride()
    if c != 1 and t.shape[3] > 1:
        raise ValueError(f"the last dimension of {name} must be contiguous")
    return (b, m, n) if blhd else (b, n, m)


def sd_rope_axes(q, k, positions, freqs, axis_dims, pairs: str = "interleaved", layout: str = "blhd", q_weight=None,
                 k_weight=None, eps: float = 1e-6, q_out=None, k_out=None):
    """Rotary positions with several axes for ``q`` and ``k`` (or None), after the RMS norm of each head where
    ``q_weight`` / ``k_weight`` (fp32 [dh]) is given; returns (q_out, k_out).

    q and k are [B, L, heads, dh] (layout "blhd") or [B, heads, L, dh] ("bhld"), bf16, fp16 or fp32, and may
    be strided views (a fused projection's rows). ``positions`` is int32 [B, L, axes] or [L, axes],
    ``axis_dims`` the columns of each axis and ``freqs`` the table of ``rope_frequencies``. ``pairs`` is
    "interleaved" (columns 2m, 2m + 1) or "half" (m, m + rot / 2). ``q_out`` may be ``q``, ``k_out`` ``k``."""
    import torch
    if pairs not in ("interleaved", "half"):
        raise ValueError("pairs must be 'interleaved' or 'half'")
    if layout not in ("bhld", "blhd"):
        raise ValueError("layout must be 'bhld' or 'blhd'")
    code = _dtype_code(q, "sd_rope_axes")
    blhd = layout == "blhd"
    if q.dim() != 4:
        raise ValueError("q must be 4-D")
    if blhd:
        B, L, H, dh = q.shape
    else:
        B, H, L, dh = q.shape
    axes = len(axis_dims)
    if not 1 <= axes <= 4:
        raise ValueError("1 to 4 axes")
    KV = 0
    if k is not None:
        if k.dim() != 4 or k.dtype != q.dtype:
            raise ValueError("k must match q in type, batch, length and head dim")
        Bk, m, n, dhk = k.shape
        Lk, KV = (m, n) if blhd else (n, m)
        if Bk != B or Lk != L or dhk != dh:
            raise ValueError("k must match q in type, batch, length and head dim")
    if positions.dtype != torch.int32 or positions.shape not in ((B, L, axes), (L, axes)) or not positions.is_contiguous():
        raise ValueError("positions must be contiguous int32 [B, L, axes] or [L, axes]")
    if freqs.dtype != torch.int64 or freqs.shape != (sum(axis_dims) // 2,) or not freqs.is_contiguous():
        raise ValueError("freqs must be int64 [sum(axis_dims) / 2]")
    for w in (q_weight, k_weight):
        if w is not None and (w.dtype != torch.float32 or w.shape != (dh,) or not w.is_contiguous()):
            raise ValueError("q_weight and k_weight must be contiguous fp32 [dh]")
    if q_out is None:
        q_out = torch.empty_like(q)
    elif q_out.shape != q.shape or q_out.dtype != q.dtype:
        raise ValueError("q_out must have the shape and type of q")
    if k is None:
        if k_out is not None:
            raise ValueError("k_out needs k")
    elif k_out is None:
        k_out = torch.empty_like(k)
    elif k_out.shape != k.shape or k_out.dtype != k.dtype:
        raise ValueError("k_out must have the shape and type of k")
    dev = _device_index(q, (k, positions, freqs, q_weight, k_weight, q_out, k_out))
    k_there = k is not None
    dims = tuple(axis_dims)
    a = _ROPE_ARGS.pack(
        q.data_ptr(), k.data_ptr() if k_there else 0, q_out.data_ptr(), k_out.data_ptr() if k_there else 0, _ptr(q_weight),
        _ptr(k_weight), positions.data_ptr(), freqs.data_ptr(), B, L, H, KV, dh,
        *_strides(q, blhd, "q"), *(_strides(k, blhd, "k") if k_there else (0, 0, 0)), *_strides(q_out, blhd, "q_out"),
        *(_strides(k_out, blhd, "k_out") if k_there else (0, 0, 0)), L * axes if positions.dim() == 3 else 0,
        *dims, *(0, 0, 0)[axes - 1:], axes, pairs == "half", code, eps)
    _call("sd_rope_axes", dev, a)
    return q_out, k_out


def _check_ints(name, t, n) -> None:
    import torch
    if t.dtype != torch.int32 or t.shape != (n,) or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous int32 [{n}]")


def sd_attention_masked(q, k, v, scale: float | None = None, layout: str = "bhld", causal: bool = False, cap: float | None = None,
                        bias=None, kv_lens=None, q_starts=None, prefix_lens=None, q_offsets=None, k_offsets=None,
                        out=None):
    """Attention with masks, a tanh cap of the scores and a bias by distance.

    q [B, heads, Lq, dh] and k, v [B, kv_heads, Lk, dh] (layout "bhld") or [B, L, heads, dh] ("blhd"), all
    bf16 or all fp16, possibly strided views; kv_heads divides heads; dh is a multiple of 8 up to 160; scale
    defaults to 1/sqrt(dh). Query i of a sequence stands at key position start + i.

    causal      a query sees keys up to its own position (and the first ``prefix_lens`` keys)
    cap         > 0: scores become cap * tanh(score / cap)
    bias        fp32 [heads, 2 R + 1]: score += bias[h, clamp(j - position, -R, R) + R]
    kv_lens     int32 [B]: keys behind a sequence's length are not seen (default Lk)
    q_starts    int32 [B or docs]: position of the first query (default Lk - Lq, or a document's keys - queries)
    q_offsets, k_offsets   int32 [docs + 1]: B = 1 holds packed documents; each sees only itself, and rows of
                ``out`` in no document are left as they were (0 where out is not given)

    A query that sees no key gets 0. Values of keys it does not see never reach it, NaN included."""
    import torch
    code = _dtype_code(q, "sd_attention_masked")
    if code == 2 or k.dtype != q.dtype or v.dtype != q.dtype:
        raise ValueError("sd_attention_masked takes q, k, v all bf16 or all fp16")
    if q.dim() != 4 or k.dim() != 4 or v.dim() != 4:
        raise ValueError("q, k, v must be 4-D")
    if layout not in ("bhld", "blhd"):
        raise ValueError("layout must be 'bhld' or 'blhd'")
    blhd = layout == "blhd"
    if blhd:
        (B, Lq, H, dh), (Bk, Lk, KV, dhk) = q.shape, k.shape
    else:
        (B, H, Lq, dh), (Bk, KV, Lk, dhk) = q.shape, k.shape
    if Bk != B or dhk != dh or v.shape != k.shape:
        raise ValueError("k and v must match each other, and q in batch and head dim")
    if (q_offsets is None) != (k_offsets is None):
        raise ValueError("q_offsets and k_offsets go together")
    docs = 0
    if q_offsets is not None:
        if kv_lens is not None:
            raise ValueError("packed documents have their lengths from k_offsets: kv_lens must be None")
        if B != 1:
            raise ValueError("packed documents need a batch of 1")
        docs = q_offsets.numel() - 1
        if docs < 1 or k_offsets.numel() != docs + 1:
            raise ValueError("q_offsets and k_offsets must both be [docs + 1], docs >= 1")
        _check_ints("q_offsets", q_offsets, docs + 1)
        _check_ints("k_offsets", k_offsets, docs + 1)
    if kv_lens is not None:
        _check_ints("kv_lens", kv_lens, B)
    if q_starts is not None:
        _check_ints("q_starts", q_starts, docs or B)
    if prefix_lens is not None:
        _check_ints("prefix_lens", prefix_lens, docs or B)
    if prefix_lens is not None and not causal:
        raise ValueError("prefix_lens needs causal")
    radius = 0
    if bias is not None:
        if (bias.dtype != torch.float32 or bias.dim() != 2 or bias.shape[0] != H or bias.shape[1] % 2 != 1
                or not bias.is_contiguous()):
            raise ValueError("bias must be contiguous fp32 [heads, 2 R + 1]")
        radius = bias.shape[1] // 2
    if out is None:
        out = torch.zeros_like(q) if docs else torch.empty_like(q)
    elif out.shape != q.shape or out.dtype != q.dtype:
        raise ValueError("out must have the shape and type of q")
    dev = _device_index(q, (k, v, out, bias, kv_lens, q_starts, prefix_lens, q_offsets, k_offsets))
    cap = 0.0 if cap is None else cap
    a = _ATTENTION_MASKED_ARGS.pack(
        q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), _ptr(bias), _ptr(kv_lens), _ptr(q_starts), _ptr(prefix_lens),
        _ptr(q_offsets), _ptr(k_offsets), B, H, KV, Lq, Lk, dh, *_strides(q, blhd, "q"), *_strides(k, blhd, "k"),
        *_strides(v, blhd, "v"), *_strides(out, blhd, "out"), radius, docs, bool(causal), code,
        1.0 / math.sqrt(dh) if scale is None else scale, cap)
    _call("sd_attention_masked", dev, a)
    return out


def sd_device_status(stream=None, reset: bool = True) -> int:
    """Synchronise and read the device status word; raises SDError on a recorded device failure."""
    s = stream.cuda_stream if stream is not None else 0
    st = lib().sd_device_status(s, 1 if reset else 0)
    _check("sd_device_status", st)
    return st


def sd_debug_set_fault(flags: int) -> None:
    """Test hook: bit 0 makes attention launches skip their first V tile (the bounded wait expires)."""
    lib().sd_debug_set_fault(int(flags))
