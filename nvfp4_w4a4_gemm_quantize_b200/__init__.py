"""NVFP4 two-level quantization and block-scaled FP4 GEMMs for B200 (sm_100a).

Python binding of the C ABI in include/nvfp4.h.  Every function below only
marshals torch tensors into pointers and sizes and calls the library of the
same name; all arithmetic runs in the CUDA kernels.  torch supplies device
memory and streams.  Every tensor must live on the current CUDA device (the
library launches there; nothing here switches devices), and the default stream
argument is that device's current torch stream.  On another stream the caller
sees to it that inputs are ready there and that results are waited for.

Low-level (same names and argument order as the C calls):
    nvfp4_sf_bytes, nvfp4_quantize_workspace_bytes, nvfp4_quantize,
    nvfp4_quantize_noalloc, nvfp4_layernorm_quantize, nvfp4_quantize_block, nvfp4_block_size_errors, nvfp4_select_block_size,
    nvfp4_dequantize, nvfp4_fake_quantize, nvfp4_ste_backward,
    nvfp4_gemm_w4a4, nvfp4_gemm_w4a4_grouped, nvfp4_gemm_w4a16, nvfp4_mx_sf_bytes, nvfp4_mx_quantize,
    nvfp4_mx_dequantize, nvfp4_mx_gemm, nvfp4_attention, nvfp4_attention_workspace_bytes, nvfp4_launch_count,
    nvfp4_gemv_w4a16, nvfp4_rotary, nvfp4_cross_attention, nvfp4_cross_attention_backward,
    nvfp4_cross_attention_backward_workspace_bytes (include/nvfp4_dit.h)
Convenience (allocate outputs with torch, then call the above):
    NVFP4Tensor, quantize, layernorm_quantize, dequantize, gemm_w4a4, gemm_w4a4_nvfp4_out, gemm_w4a4_grouped,
    gemm_w4a16,
    fake_quantize, ste_backward, FakeQuantizeSTE (autograd: the two kernels),
    MXTensor, mx_quantize, mx_dequantize, mx_gemm, quantize_block, block_size_errors, select_block_size,
    attention, gemv_w4a16,
    rotary, RotaryEmbedding (autograd), cross_attention, cross_attention_backward, CrossAttention (autograd)
"""
from __future__ import annotations

import ctypes
import functools
import struct
from dataclasses import dataclass

import torch

from ._lib import MAX_GROUP, NVFP4Error, NVFP4GemmProblem, check, lib  # noqa: F401

NVFP4_DTYPE_BF16 = 0
NVFP4_DTYPE_F32 = 1
NVFP4_SCALE_GIVEN = 1
NVFP4_ACT_NONE = 0
NVFP4_ACT_GELU_TANH = 1
NVFP4_WEIGHTS_NVFP4 = 0
NVFP4_WEIGHTS_MX = 1
NVFP4_GEMV_MAX_ROWS = 16
NVFP4_POSITION_I32 = 0
NVFP4_POSITION_F32 = 1
NVFP4_ROTARY_INTERLEAVED = 1
NVFP4_ROTARY_INVERSE = 2

_DT = {torch.bfloat16: NVFP4_DTYPE_BF16, torch.float32: NVFP4_DTYPE_F32}


def _ptr(t) -> int | None:
    if t is None:
        return None
    if not isinstance(t, torch.Tensor):
        raise TypeError("expected a torch.Tensor")
    if not t.is_cuda:
        raise ValueError("tensor must live on a CUDA device")
    return t.data_ptr()


def _stream(stream) -> int | None:
    if stream is None:
        # the current stream's handle without building a Stream object (3 us of host time a call)
        return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


# ----------------------------------------------------------------- C ABI
def nvfp4_sf_bytes(rows: int, k: int) -> int:
    return int(lib().nvfp4_sf_bytes(rows, k))


def nvfp4_quantize_workspace_bytes(rows: int, k: int) -> int:
    return int(lib().nvfp4_quantize_workspace_bytes(rows, k))


def nvfp4_launch_count() -> int:
    return int(lib().nvfp4_launch_count())


def nvfp4_shutdown() -> None:
    lib().nvfp4_shutdown()


def nvfp4_debug_wait_timeout(dev_status, limit_us: int, stream=None) -> None:
    """Check of the failure detection: one warp waits, with the library's
    bounded wait, on a barrier nothing arrives at, gives up after limit_us and
    writes NVFP4_ERR_TIMEOUT to dev_status (a zeroed device int32)."""
    st = lib().nvfp4_debug_wait_timeout(_ptr(dev_status), limit_us, _stream(stream))
    check(st, "nvfp4_debug_wait_timeout")


def nvfp4_quantize(x, rows, k, ld_x, codes, sf, tensor_scale, flags=0, workspace=None,
                   workspace_bytes=0, dev_status=None, stream=None) -> None:
    st = lib().nvfp4_quantize(_ptr(x), rows, k, ld_x, _ptr(codes), _ptr(sf), _ptr(tensor_scale),
                              flags, _ptr(workspace), workspace_bytes, _ptr(dev_status), _stream(stream))
    check(st, "nvfp4_quantize")


def nvfp4_layernorm_quantize(x, rows, k, ld_x, gamma, beta, rows_per_group, eps, codes, sf, tensor_scale, flags=0,
                             workspace=None, workspace_bytes=0, dev_status=None, stream=None) -> None:
    st = lib().nvfp4_layernorm_quantize(_ptr(x), rows, k, ld_x, _ptr(gamma), _ptr(beta), rows_per_group, float(eps),
                                        _ptr(codes), _ptr(sf), _ptr(tensor_scale), flags, _ptr(workspace),
                                        workspace_bytes, _ptr(dev_status), _stream(stream))
    check(st, "nvfp4_layernorm_quantize")


def nvfp4_quantize_noalloc(x, rows, k, ld_x, codes, sf, tensor_scale, flags=0, dev_status=None,
                           stream=None) -> None:
    """nvfp4_quantize without a workspace argument, for callers that cannot
    allocate device memory (the amax scratch is a fixed device array inside the
    library; overlapping calls race, see include/nvfp4.h)."""
    st = lib().nvfp4_quantize_noalloc(_ptr(x), rows, k, ld_x, _ptr(codes), _ptr(sf), _ptr(tensor_scale), flags,
                                      _ptr(dev_status), _stream(stream))
    check(st, "nvfp4_quantize_noalloc")


def nvfp4_quantize_block(x, rows, k, ld_x, block, codes, sf, tensor_scale, flags=0, workspace=None,
                         workspace_bytes=0, dev_status=None, stream=None) -> None:
    st = lib().nvfp4_quantize_block(_ptr(x), rows, k, ld_x, block, _ptr(codes), _ptr(sf), _ptr(tensor_scale), flags,
                                    _ptr(workspace), workspace_bytes, _ptr(dev_status), _stream(stream))
    check(st, "nvfp4_quantize_block")


def nvfp4_block_size_errors(x, rows, k, ld_x, tensor_scale, errors, stream=None) -> None:
    check(lib().nvfp4_block_size_errors(_ptr(x), rows, k, ld_x, _ptr(tensor_scale), _ptr(errors), _stream(stream)),
          "nvfp4_block_size_errors")


def nvfp4_select_block_size(errors_host, lam: float) -> int:
    """Eq. 9 on a host sequence of 8 doubles (the device errors copied back)."""
    arr = (ctypes.c_double * 8)(*[float(v) for v in errors_host])
    return int(lib().nvfp4_select_block_size(ctypes.addressof(arr), float(lam)))


def nvfp4_dequantize(codes, sf, tensor_scale, rows, k, out, out_dtype, stream=None) -> None:
    st = lib().nvfp4_dequantize(_ptr(codes), _ptr(sf), _ptr(tensor_scale), rows, k, _ptr(out),
                                out_dtype, _stream(stream))
    check(st, "nvfp4_dequantize")


def nvfp4_fake_quantize(x, rows, k, ld_x, y, y_dtype, clip_mask, tensor_scale, flags=0, workspace=None,
                        workspace_bytes=0, dev_status=None, stream=None) -> None:
    st = lib().nvfp4_fake_quantize(_ptr(x), rows, k, ld_x, _ptr(y), y_dtype, _ptr(clip_mask), _ptr(tensor_scale),
                                   flags, _ptr(workspace), workspace_bytes, _ptr(dev_status), _stream(stream))
    check(st, "nvfp4_fake_quantize")


def nvfp4_ste_backward(grad_y, clip_mask, rows, k, dtype, grad_x, stream=None) -> None:
    st = lib().nvfp4_ste_backward(_ptr(grad_y), _ptr(clip_mask), rows, k, dtype, _ptr(grad_x), _stream(stream))
    check(st, "nvfp4_ste_backward")


def nvfp4_gemm_w4a4(a_codes, a_sf, a_scale, b_codes, b_sf, b_scale, M, N, K, y=None,
                    y_dtype=NVFP4_DTYPE_BF16, y_codes=None, y_sf=None, y_scale=None, y_amax=None,
                    act=0, dev_status=None, stream=None) -> None:
    st = lib().nvfp4_gemm_w4a4(_ptr(a_codes), _ptr(a_sf), _ptr(a_scale), _ptr(b_codes), _ptr(b_sf),
                               _ptr(b_scale), M, N, K, _ptr(y), y_dtype, _ptr(y_codes), _ptr(y_sf),
                               _ptr(y_scale), _ptr(y_amax), act, _ptr(dev_status), _stream(stream))
    check(st, "nvfp4_gemm_w4a4")


def nvfp4_gemm_w4a4_grouped(problems, y_dtype=NVFP4_DTYPE_BF16, dev_status=None, stream=None) -> None:
    """``problems``: a list of dicts with the fields of nvfp4_gemm_problem
    (tensors or None for the pointers, ints for M, N, K)."""
    arr = (NVFP4GemmProblem * len(problems))()
    for i, d in enumerate(problems):
        for name, _ in NVFP4GemmProblem._fields_:
            v = d.get(name)
            setattr(arr[i], name, int(v or 0) if name in ("M", "N", "K", "act") else _ptr(v))
    st = lib().nvfp4_gemm_w4a4_grouped(ctypes.addressof(arr), len(problems), y_dtype, _ptr(dev_status),
                                       _stream(stream))
    check(st, "nvfp4_gemm_w4a4_grouped")


def nvfp4_mx_sf_bytes(rows: int, k: int) -> int:
    return int(lib().nvfp4_mx_sf_bytes(rows, k))


def nvfp4_mx_quantize(x, rows, k, ld_x, codes, sf, stream=None) -> None:
    check(lib().nvfp4_mx_quantize(_ptr(x), rows, k, ld_x, _ptr(codes), _ptr(sf), _stream(stream)),
          "nvfp4_mx_quantize")


def nvfp4_mx_dequantize(codes, sf, rows, k, out, out_dtype, stream=None) -> None:
    check(lib().nvfp4_mx_dequantize(_ptr(codes), _ptr(sf), rows, k, _ptr(out), out_dtype, _stream(stream)),
          "nvfp4_mx_dequantize")


def nvfp4_mx_gemm(a_codes, a_sf, b_codes, b_sf, M, N, K, y, y_dtype=NVFP4_DTYPE_BF16, act=0, dev_status=None,
                  stream=None) -> None:
    check(lib().nvfp4_mx_gemm(_ptr(a_codes), _ptr(a_sf), _ptr(b_codes), _ptr(b_sf), M, N, K, _ptr(y), y_dtype, act,
                              _ptr(dev_status), _stream(stream)), "nvfp4_mx_gemm")


def nvfp4_attention_workspace_bytes(H: int, Lk: int, d: int) -> int:
    return int(lib().nvfp4_attention_workspace_bytes(H, Lk, d))


def nvfp4_attention(q_codes, q_sf, q_scale, k_codes, k_sf, k_scale, v_codes, v_sf, v_scale, s_head, H, Lq, Lk, d,
                    out, workspace, workspace_bytes, dev_status=None, stream=None) -> None:
    check(lib().nvfp4_attention(_ptr(q_codes), _ptr(q_sf), _ptr(q_scale), _ptr(k_codes), _ptr(k_sf), _ptr(k_scale),
                                _ptr(v_codes), _ptr(v_sf), _ptr(v_scale), _ptr(s_head), H, Lq, Lk, d, _ptr(out),
                                _ptr(workspace), workspace_bytes, _ptr(dev_status), _stream(stream)),
          "nvfp4_attention")


def nvfp4_gemm_w4a16(x, w_codes, w_sf, w_scale, M, N, K, y, y_dtype=NVFP4_DTYPE_BF16,
                     dev_status=None, stream=None) -> None:
    st = lib().nvfp4_gemm_w4a16(_ptr(x), _ptr(w_codes), _ptr(w_sf), _ptr(w_scale), M, N, K, _ptr(y),
                                y_dtype, _ptr(dev_status), _stream(stream))
    check(st, "nvfp4_gemm_w4a16")


_PACK_HEADS = struct.Struct("Pqqq").pack


def _heads(t) -> bytes:
    """A [batch, tokens, heads, d] CUDA tensor (d contiguous) as nvfp4_heads."""
    if t.get_device() < 0:
        raise ValueError("tensor must live on a CUDA device")
    sb, sl, sh, _ = t.stride()
    return _PACK_HEADS(t.data_ptr(), sb, sl, sh)


def _new_heads(t, L, H, d) -> bytes:
    """The same of a contiguous tensor that the call allocated."""
    return _PACK_HEADS(t.data_ptr(), L * H * d, H * d, d)


@functools.lru_cache(maxsize=64)
def _ints(values: tuple) -> bytes:
    return struct.pack(f"{len(values)}i", *values)


def nvfp4_gemv_w4a16(x, ld_x, w_codes, w_sf, w_scale, w_format, bias, M, N, K, y, y_dtype=NVFP4_DTYPE_BF16,
                     stream=None) -> None:
    check(lib().nvfp4_gemv_w4a16(_ptr(x), ld_x, _ptr(w_codes), _ptr(w_sf), _ptr(w_scale), w_format, _ptr(bias), M, N,
                                 K, _ptr(y), y_dtype, _stream(stream)), "nvfp4_gemv_w4a16")


def nvfp4_rotary(x, positions, pos_dtype, pos_batch_stride, pos_token_stride, axis_dims, theta, B, L, H, d, dtype,
                 flags, out, stream=None) -> None:
    """``x`` and ``out``: [B, L, H, d] tensors; ``axis_dims``: a sequence of ints."""
    check(lib().nvfp4_rotary(_heads(x), _ptr(positions), pos_dtype, pos_batch_stride, pos_token_stride,
                             _ints(tuple(axis_dims)), len(axis_dims), theta, B, L, H, d, dtype, flags, _heads(out),
                             _stream(stream)), "nvfp4_rotary")


def nvfp4_cross_attention(q, k, v, kv_lens, scale, B, H, Hkv, Lq, Lk, d, out, lse, dev_status=None,
                          stream=None) -> None:
    """``q``, ``k``, ``v``, ``out``: [batch, tokens, heads, d] tensors."""
    check(lib().nvfp4_cross_attention(_heads(q), _heads(k), _heads(v), _ptr(kv_lens), scale, B, H, Hkv, Lq, Lk, d,
                                      _heads(out), _ptr(lse), _ptr(dev_status), _stream(stream)),
          "nvfp4_cross_attention")


@functools.lru_cache(maxsize=256)                      # of its sizes alone
def nvfp4_cross_attention_backward_workspace_bytes(B: int, H: int, Hkv: int, Lq: int, Lk: int, d: int) -> int:
    return int(lib().nvfp4_cross_attention_backward_workspace_bytes(B, H, Hkv, Lq, Lk, d))


def nvfp4_cross_attention_backward(grad_out, q, k, v, out, lse, kv_lens, scale, B, H, Hkv, Lq, Lk, d, dq, dk, dv,
                                   workspace, workspace_bytes, dev_status=None, stream=None) -> None:
    check(lib().nvfp4_cross_attention_backward(
        _heads(grad_out), _heads(q), _heads(k), _heads(v), _heads(out), _ptr(lse), _ptr(kv_lens), scale, B, H, Hkv,
        Lq, Lk, d, _heads(dq), _heads(dk), _heads(dv), _ptr(workspace), workspace_bytes, _ptr(dev_status),
        _stream(stream)), "nvfp4_cross_attention_backward")


# ----------------------------------------------------------------- convenience
@dataclass
class NVFP4Tensor:
    """codes [rows, k/2] uint8, sf [sf_bytes] uint8 (tensor-core layout),
    scale [1] float32 -- all on one CUDA device."""
    codes: torch.Tensor
    sf: torch.Tensor
    scale: torch.Tensor
    rows: int
    k: int

    @staticmethod
    def empty(rows: int, k: int, device) -> "NVFP4Tensor":
        return NVFP4Tensor(torch.empty(rows, k // 2, dtype=torch.uint8, device=device),
                           torch.empty(max(nvfp4_sf_bytes(rows, k), 16), dtype=torch.uint8, device=device),
                           torch.zeros(1, dtype=torch.float32, device=device), rows, k)


def quantize(x: torch.Tensor, scale: torch.Tensor | float | None = None, out: NVFP4Tensor | None = None,
             workspace: torch.Tensor | None = None, dev_status=None, stream=None) -> NVFP4Tensor:
    """Quantize a bf16 [rows, k] CUDA tensor.  ``scale`` given -> used as the
    tensor scale g; otherwise g = amax / 2688 is computed on the device."""
    assert x.dtype == torch.bfloat16 and x.dim() == 2 and x.stride(1) == 1
    rows, k = x.shape
    q = out if out is not None else NVFP4Tensor.empty(rows, k, x.device)
    flags = 0
    if scale is not None:
        if isinstance(scale, torch.Tensor):
            q.scale.copy_(scale.reshape(1).to(torch.float32))
        else:
            q.scale.fill_(float(scale))
        flags = NVFP4_SCALE_GIVEN
    wsb = nvfp4_quantize_workspace_bytes(rows, k)
    if flags == 0 and workspace is None:
        workspace = torch.empty(wsb, dtype=torch.uint8, device=x.device)
    nvfp4_quantize(x, rows, k, x.stride(0), q.codes, q.sf, q.scale, flags,
                   workspace if flags == 0 else None, wsb if flags == 0 else 0, dev_status, stream)
    return q


def layernorm_quantize(x: torch.Tensor, gamma: torch.Tensor | None = None, beta: torch.Tensor | None = None,
                       rows_per_group: int = 0, eps: float = 1e-6, scale: torch.Tensor | float | None = None,
                       out: NVFP4Tensor | None = None, workspace: torch.Tensor | None = None, dev_status=None,
                       stream=None) -> NVFP4Tensor:
    """LayerNorm of a bf16 [rows, k] CUDA tensor (optional FP32 affine per
    group of rows_per_group rows: gamma / beta [groups, k]) emitted directly as
    NVFP4.  ``scale`` given -> the tensor scale; otherwise the largest |y| / 2688."""
    assert x.dtype == torch.bfloat16 and x.dim() == 2 and x.stride(1) == 1
    rows, k = x.shape
    for t in (gamma, beta):
        assert t is None or (t.dtype == torch.float32 and t.is_contiguous() and t.shape[-1] == k)
    q = out if out is not None else NVFP4Tensor.empty(rows, k, x.device)
    flags = 0
    if scale is not None:
        if isinstance(scale, torch.Tensor):
            q.scale.copy_(scale.reshape(1).to(torch.float32))
        else:
            q.scale.fill_(float(scale))
        flags = NVFP4_SCALE_GIVEN
    wsb = nvfp4_quantize_workspace_bytes(rows, k)
    if flags == 0 and workspace is None:
        workspace = torch.empty(wsb, dtype=torch.uint8, device=x.device)
    nvfp4_layernorm_quantize(x, rows, k, x.stride(0), gamma, beta, rows_per_group, eps, q.codes, q.sf, q.scale, flags,
                             workspace if flags == 0 else None, wsb if flags == 0 else 0, dev_status, stream)
    return q


def dequantize(q: NVFP4Tensor, dtype=torch.bfloat16, stream=None) -> torch.Tensor:
    out = torch.empty(q.rows, q.k, dtype=dtype, device=q.codes.device)
    nvfp4_dequantize(q.codes, q.sf, q.scale, q.rows, q.k, out, _DT[dtype], stream)
    return out


def gemm_w4a4(a: NVFP4Tensor, b: NVFP4Tensor, out_dtype=torch.bfloat16, out: torch.Tensor | None = None,
              act=NVFP4_ACT_NONE, dev_status=None, stream=None) -> torch.Tensor:
    """Y = act(A B^T), A [M,K] activations, B [N,K] weights, both NVFP4."""
    assert a.k == b.k
    y = out if out is not None else torch.empty(a.rows, b.rows, dtype=out_dtype, device=a.codes.device)
    nvfp4_gemm_w4a4(a.codes, a.sf, a.scale, b.codes, b.sf, b.scale, a.rows, b.rows, a.k, y=y,
                    y_dtype=_DT[y.dtype], act=act, dev_status=dev_status, stream=stream)
    return y


def gemm_w4a4_nvfp4_out(a: NVFP4Tensor, b: NVFP4Tensor, y_scale: torch.Tensor, y_amax: torch.Tensor | None = None,
                        out: NVFP4Tensor | None = None, act=NVFP4_ACT_NONE, dev_status=None,
                        stream=None) -> NVFP4Tensor:
    """act(Y = A B^T) emitted directly as NVFP4 with the caller's tensor scale."""
    q = out if out is not None else NVFP4Tensor.empty(a.rows, b.rows, a.codes.device)
    q.scale.copy_(y_scale.reshape(1))
    nvfp4_gemm_w4a4(a.codes, a.sf, a.scale, b.codes, b.sf, b.scale, a.rows, b.rows, a.k,
                    y_codes=q.codes, y_sf=q.sf, y_scale=q.scale, y_amax=y_amax, act=act, dev_status=dev_status,
                    stream=stream)
    return q


def gemm_w4a4_grouped(pairs, out_dtype=torch.bfloat16, act=NVFP4_ACT_NONE, dev_status=None, stream=None) -> list:
    """Y_i = A_i B_i^T for up to MAX_GROUP independent (A_i, B_i) NVFP4 pairs in
    one launch; returns the outputs in order."""
    ys, probs = [], []
    for a, b in pairs:
        assert a.k == b.k
        y = torch.empty(a.rows, b.rows, dtype=out_dtype, device=a.codes.device)
        ys.append(y)
        probs.append(dict(a_codes=a.codes, a_sf=a.sf, a_scale=a.scale, b_codes=b.codes, b_sf=b.sf,
                          b_scale=b.scale, M=a.rows, N=b.rows, K=a.k, y=y, act=act))
    nvfp4_gemm_w4a4_grouped(probs, _DT[out_dtype], dev_status, stream)
    return ys


def gemm_w4a16(x: torch.Tensor, w: NVFP4Tensor, out_dtype=torch.bfloat16, out: torch.Tensor | None = None,
               dev_status=None, stream=None) -> torch.Tensor:
    """Y = X W^T, X bf16 [M,K], W NVFP4 [N,K]."""
    assert x.dtype == torch.bfloat16 and x.is_contiguous() and x.shape[1] == w.k
    y = out if out is not None else torch.empty(x.shape[0], w.rows, dtype=out_dtype, device=x.device)
    nvfp4_gemm_w4a16(x, w.codes, w.sf, w.scale, x.shape[0], w.rows, w.k, y, _DT[y.dtype], dev_status, stream)
    return y


# ----------------------------------------------------------------- QAT
def fake_quantize(x: torch.Tensor, scale: torch.Tensor | float | None = None, out_dtype=torch.bfloat16,
                  clip_mask: bool = True, workspace: torch.Tensor | None = None, dev_status=None, stream=None):
    """Fake-quantize a bf16 [rows, k] CUDA tensor: returns (y, mask, scale) with
    y = the NVFP4 value of each element (bf16 or f32), mask the packed clip
    bits ([rows, k/8] uint8, None unless ``clip_mask``) and scale the tensor
    scale used (computed on the device unless given)."""
    assert x.dtype == torch.bfloat16 and x.dim() == 2 and x.stride(1) == 1
    rows, k = x.shape
    y = torch.empty(rows, k, dtype=out_dtype, device=x.device)
    m = torch.empty(rows, k // 8, dtype=torch.uint8, device=x.device) if clip_mask else None
    g = torch.zeros(1, dtype=torch.float32, device=x.device)
    flags = 0
    if scale is not None:
        if isinstance(scale, torch.Tensor):
            g.copy_(scale.reshape(1).to(torch.float32))
        else:
            g.fill_(float(scale))
        flags = NVFP4_SCALE_GIVEN
    wsb = nvfp4_quantize_workspace_bytes(rows, k)
    if flags == 0 and workspace is None:
        workspace = torch.empty(wsb, dtype=torch.uint8, device=x.device)
    nvfp4_fake_quantize(x, rows, k, x.stride(0), y, _DT[out_dtype], m, g, flags,
                        workspace if flags == 0 else None, wsb if flags == 0 else 0, dev_status, stream)
    return y, m, g


def ste_backward(grad_y: torch.Tensor, clip_mask: torch.Tensor, out: torch.Tensor | None = None,
                 stream=None) -> torch.Tensor:
    """grad_y where the clip mask is clear, +0 where set (``out`` may be grad_y)."""
    assert grad_y.dim() == 2 and grad_y.is_contiguous() and grad_y.dtype in _DT
    rows, k = grad_y.shape
    gx = out if out is not None else torch.empty_like(grad_y)
    nvfp4_ste_backward(grad_y, clip_mask, rows, k, _DT[grad_y.dtype], gx, stream)
    return gx


class FakeQuantizeSTE(torch.autograd.Function):
    """Autograd wrapper of the two kernels: forward = nvfp4_fake_quantize,
    backward = nvfp4_ste_backward with the forward's clip mask (masked=True)
    or the identity (masked=False, the plain straight-through estimator)."""

    @staticmethod
    def forward(ctx, x, scale=None, masked=True):
        y, m, _ = fake_quantize(x, scale, clip_mask=masked)
        ctx.save_for_backward(*([m] if masked else []))
        ctx.masked = masked
        return y

    @staticmethod
    def backward(ctx, grad_y):
        if not ctx.masked:
            return grad_y, None, None
        (m,) = ctx.saved_tensors
        return ste_backward(grad_y.contiguous(), m), None, None


# ----------------------------------------------------------------- MX variant
@dataclass
class MXTensor:
    """codes [rows, k/2] uint8, sf [mx_sf_bytes] uint8 (E8M0, block 32)."""
    codes: torch.Tensor
    sf: torch.Tensor
    rows: int
    k: int

    @staticmethod
    def empty(rows: int, k: int, device) -> "MXTensor":
        return MXTensor(torch.empty(rows, k // 2, dtype=torch.uint8, device=device),
                        torch.empty(max(nvfp4_mx_sf_bytes(rows, k), 16), dtype=torch.uint8, device=device), rows, k)


def mx_quantize(x: torch.Tensor, out: MXTensor | None = None, stream=None) -> MXTensor:
    assert x.dtype == torch.bfloat16 and x.dim() == 2 and x.stride(1) == 1
    rows, k = x.shape
    q = out if out is not None else MXTensor.empty(rows, k, x.device)
    nvfp4_mx_quantize(x, rows, k, x.stride(0), q.codes, q.sf, stream)
    return q


def mx_dequantize(q: MXTensor, dtype=torch.bfloat16, stream=None) -> torch.Tensor:
    out = torch.empty(q.rows, q.k, dtype=dtype, device=q.codes.device)
    nvfp4_mx_dequantize(q.codes, q.sf, q.rows, q.k, out, _DT[dtype], stream)
    return out


def mx_gemm(a: MXTensor, b: MXTensor, out_dtype=torch.bfloat16, out: torch.Tensor | None = None,
            act=NVFP4_ACT_NONE, dev_status=None, stream=None) -> torch.Tensor:
    assert a.k == b.k
    y = out if out is not None else torch.empty(a.rows, b.rows, dtype=out_dtype, device=a.codes.device)
    nvfp4_mx_gemm(a.codes, a.sf, b.codes, b.sf, a.rows, b.rows, a.k, y, _DT[y.dtype], act, dev_status, stream)
    return y


# ----------------------------------------------------------------- block size (Algorithm 1 / Eq. 9)
def quantize_block(x: torch.Tensor, block: int, scale: torch.Tensor | float | None = None,
                   out: NVFP4Tensor | None = None, workspace: torch.Tensor | None = None, dev_status=None,
                   stream=None) -> NVFP4Tensor:
    """quantize() with `block` (16, 32, 64) values per scale; scales repeated in
    the block-16 layout, so gemm_w4a4 takes the result as it is."""
    assert x.dtype == torch.bfloat16 and x.dim() == 2 and x.stride(1) == 1
    rows, k = x.shape
    q = out if out is not None else NVFP4Tensor.empty(rows, k, x.device)
    flags = 0
    if scale is not None:
        if isinstance(scale, torch.Tensor):
            q.scale.copy_(scale.reshape(1).to(torch.float32))
        else:
            q.scale.fill_(float(scale))
        flags = NVFP4_SCALE_GIVEN
    wsb = nvfp4_quantize_workspace_bytes(rows, k)
    if flags == 0 and workspace is None:
        workspace = torch.empty(wsb, dtype=torch.uint8, device=x.device)
    nvfp4_quantize_block(x, rows, k, x.stride(0), block, q.codes, q.sf, q.scale, flags,
                         workspace if flags == 0 else None, wsb if flags == 0 else 0, dev_status, stream)
    return q


def block_size_errors(x: torch.Tensor, tensor_scale: torch.Tensor, stream=None) -> torch.Tensor:
    """Device float64 [8]: squared errors for b = 1, 2, ..., 64 and sum x^2."""
    assert x.dtype == torch.bfloat16 and x.dim() == 2 and x.stride(1) == 1
    errors = torch.empty(8, dtype=torch.float64, device=x.device)
    nvfp4_block_size_errors(x, x.shape[0], x.shape[1], x.stride(0), tensor_scale, errors, stream)
    return errors


def select_block_size(x: torch.Tensor, lam: float, tensor_scale: torch.Tensor | None = None) -> int:
    """Algorithm 1 / Eq. 9 for one tensor: errors on the device, the argmin on
    the host (one 64-byte copy)."""
    if tensor_scale is None:
        tensor_scale = quantize(x).scale
    return nvfp4_select_block_size(block_size_errors(x, tensor_scale).cpu().tolist(), lam)


# ----------------------------------------------------------------- attention (Eq. 10)
def attention(q: NVFP4Tensor, k: NVFP4Tensor, v: NVFP4Tensor, H: int, s_head: torch.Tensor | None = None,
              out: torch.Tensor | None = None, workspace: torch.Tensor | None = None, dev_status=None,
              stream=None) -> torch.Tensor:
    """softmax(Q K^T / sqrt(d) + log s_head) V per head over NVFP4 Q [H*Lq, d],
    K and V [H*Lk, d] (d = 128); returns bf16 [H*Lq, d]."""
    d = q.k
    Lq, Lk = q.rows // H, k.rows // H
    o = out if out is not None else torch.empty(q.rows, d, dtype=torch.bfloat16, device=q.codes.device)
    wsb = nvfp4_attention_workspace_bytes(H, Lk, d)
    if workspace is None:
        workspace = torch.empty(wsb, dtype=torch.uint8, device=q.codes.device)
    nvfp4_attention(q.codes, q.sf, q.scale, k.codes, k.sf, k.scale, v.codes, v.sf, v.scale, s_head, H, Lq, Lk, d, o,
                    workspace, wsb, dev_status, stream)
    return o


# ----------------------------------------------------------------- around the linear layers
def _require(ok: bool, what: str) -> None:
    if not ok:
        raise ValueError(what)


def _on_device(*tensors) -> None:
    """Every given tensor lives on the current CUDA device, where the kernels run."""
    here = None
    for t in tensors:
        if t is None:
            continue
        at = t.get_device()                            # -1 on the CPU
        if here is None and at >= 0:
            here = torch._C._cuda_getDevice()
        if at != here:
            raise ValueError(f"tensor on {t.device}: the call runs on the current CUDA device")


def _empty_on(stream, dtype, device, *shape, returned=True) -> torch.Tensor:
    """A tensor that a call writes on ``stream``, from that stream's own memory:
    memory that the current stream has freed may still be in use there.  What
    is ``returned`` may be used on the current stream (once that has waited for
    the call) and is not recycled before it has passed."""
    here = torch.cuda.current_stream()
    s = stream if isinstance(stream, torch.cuda.Stream) else torch.cuda.ExternalStream(int(stream))
    with torch.cuda.stream(s):
        t = torch.empty(*shape, dtype=dtype, device=device)
    if returned and s != here:
        t.record_stream(here)
    return t


def _empty(stream, dtype, device, *shape) -> torch.Tensor:
    if stream is None:
        return torch.empty(*shape, dtype=dtype, device=device)         # 0.7 us less than from a tuple
    return _empty_on(stream, dtype, device, *shape)


def gemv_w4a16(x: torch.Tensor, w: NVFP4Tensor | MXTensor, bias: torch.Tensor | None = None,
               out_dtype=torch.bfloat16, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Y = X W^T (+ bias) for at most NVFP4_GEMV_MAX_ROWS rows: X bf16 [M, K]
    (rows may be strided, or one row expanded to M), W NVFP4 or MX [N, K], bias
    FP32 [N], Y bf16 or FP32."""
    mx = isinstance(w, MXTensor)
    codes, sf, scale, N, K = w.codes, w.sf, None if mx else w.scale, w.rows, w.k
    if x.dtype is not torch.bfloat16 or x.dim() != 2 or x.shape[1] != K:
        raise ValueError("x must be bf16 [M, w.k]")
    M = x.shape[0]
    ld, step = x.stride()
    if M > NVFP4_GEMV_MAX_ROWS:
        raise ValueError("at most NVFP4_GEMV_MAX_ROWS rows: gemm_w4a16 takes more")
    if step != 1:
        raise ValueError("x must be contiguous along k")
    if M <= 1:
        ld = K                                         # never used
    elif 0 < ld < K:
        raise ValueError("rows of x must not overlap: their stride is at least w.k, or 0 for one row expanded")
    if bias is not None and (bias.dtype is not torch.float32 or bias.shape != (N,) or not bias.is_contiguous()):
        raise ValueError("bias must be a contiguous FP32 [N]")
    y_dtype = _DT.get(out_dtype if out is None else out.dtype)
    if y_dtype is None:
        raise ValueError("out must be a contiguous bf16 or FP32 [M, N]")
    _on_device(x, codes, sf, scale, bias, out)
    if out is None:
        y = _empty(stream, out_dtype, x.device, M, N)
    else:
        y = out
        _require(y.shape == (M, N) and y.is_contiguous(), "out must be a contiguous bf16 or FP32 [M, N]")
    check(lib().nvfp4_gemv_w4a16(x.data_ptr(), ld, codes.data_ptr(), sf.data_ptr(),
                                 None if mx else scale.data_ptr(), NVFP4_WEIGHTS_MX if mx else NVFP4_WEIGHTS_NVFP4,
                                 None if bias is None else bias.data_ptr(), M, N, K, y.data_ptr(), y_dtype,
                                 _stream(stream)), "nvfp4_gemv_w4a16")
    return y


def _rows16(t: torch.Tensor) -> torch.Tensor:
    """t with its last axis contiguous and 16-byte steps (a copy where it has not)."""
    if t.is_contiguous() and t.data_ptr() % 16 == 0 and t.shape[-1] * t.element_size() % 16 == 0:
        return t
    n = 16 // t.element_size()
    if t.stride(-1) == 1 and t.data_ptr() % 16 == 0 and all(
            s % n == 0 and (s >= t.shape[-1] or (s == 0 and i != 1)) for i, (s, size) in
            enumerate(zip(t.stride()[:-1], t.shape)) if size > 1):
        return t
    return t.clone(memory_format=torch.contiguous_format)      # contiguous() keeps a contiguous tensor where it is


def rotary(x: torch.Tensor, positions: torch.Tensor, axes, theta: float = 10000.0, interleaved: bool = True,
           inverse: bool = False, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Rotary positions with several axes: x [B, L, H, d] (bf16 or FP32, strided
    views such as a part of a fused projection included), positions int32 or
    FP32 [L, n_axes] or [B, L, n_axes], ``axes`` the values of a head each axis
    turns (even, together at most d; the rest is copied).  Pairs are neighbours
    (``interleaved``) or halves of the turned part; ``inverse`` turns back.
    ``out``: any [B, L, H, d] view (for instance of a [B, H, L, d] buffer, whose
    rows quantize() takes), or x itself."""
    dt, xs, st = x.dtype, x.shape, x.stride()
    dtype = _DT.get(dt)
    if dtype is None or len(xs) != 4 or st[3] != 1:
        raise ValueError("x must be bf16 or FP32 [B, L, H, d], d contiguous")
    B, L, H, d = xs
    axes = tuple(axes)
    ps, pt, pd = positions.shape, positions.stride(), positions.dtype
    n = len(ps)
    per_sample = n == 3 and ps[0] > 1
    if ((pd is not torch.int32 and pd is not torch.float32) or (n != 2 and n != 3) or ps[-2] != L or ps[-1] != len(axes)
            or (per_sample and ps[0] != B) or (n == 3 and ps[0] == 0 != B)):
        raise ValueError("positions must be int32 or FP32 [L, n_axes] or [B, L, n_axes]")
    if pt[-1] != 1 and len(axes) != 1:
        raise ValueError("positions must be contiguous along the axes")
    if out is None:
        _on_device(x, positions)
        y = _empty(stream, dt, x.device, B, L, H, d)
        to = _new_heads(y, L, H, d)
    else:
        y = out
        _require(y.dtype == dt and y.shape == xs and y.stride(3) == 1, "out must match x, d contiguous")
        _on_device(x, positions, y)
        to = _heads(y)
    flags = (NVFP4_ROTARY_INTERLEAVED if interleaved else 0) | (NVFP4_ROTARY_INVERSE if inverse else 0)
    check(lib().nvfp4_rotary(_PACK_HEADS(x.data_ptr(), st[0], st[1], st[2]), positions.data_ptr(),
                             NVFP4_POSITION_I32 if pd is torch.int32 else NVFP4_POSITION_F32, pt[0] if per_sample else 0,
                             pt[-2], _ints(axes), len(axes), float(theta), B, L, H, d, dtype, flags, to, _stream(stream)),
          "nvfp4_rotary")
    return y


class RotaryEmbedding(torch.autograd.Function):
    """Autograd wrapper of rotary(): the backward pass turns the gradient back,
    and can be differentiated again (the map is linear).  Positions get no
    gradient.  As for any torch operator, a backward pass is captured into a
    CUDA graph from leaves of the capture's own (x.detach().requires_grad_()):
    an eager graph of the same leaves invalidates it."""

    @staticmethod
    def forward(ctx, x, positions, axes, theta=10000.0, interleaved=True, inverse=False):
        ctx.save_for_backward(positions)
        ctx.how = (axes, theta, interleaved, not inverse)
        return rotary(x, positions, axes, theta, interleaved, inverse)

    @staticmethod
    def backward(ctx, grad):
        (positions,) = ctx.saved_tensors
        turn = RotaryEmbedding.apply if torch.is_grad_enabled() else rotary          # create_graph
        return turn(_rows16(grad), positions, *ctx.how), None, None, None, None, None


def _attention_operands(q, k, v, kv_lens):
    """(B, H, Hkv, Lq, Lk, d) and q, k, v as nvfp4_heads."""
    qs, ks, qt, kt, vt, bf16 = q.shape, k.shape, q.stride(), k.stride(), v.stride(), torch.bfloat16
    if len(qs) != 4 or len(ks) != 4 or v.shape != ks or ks[0] != qs[0] or ks[3] != qs[3]:
        raise ValueError("q must be [B, Lq, H, d], k and v [B, Lk, Hkv, d]")
    if (q.dtype is not bf16 or k.dtype is not bf16 or v.dtype is not bf16 or qt[3] != 1 or kt[3] != 1 or vt[3] != 1):
        raise ValueError("q, k and v must be bf16, d contiguous")
    B, Lq, H, d = qs
    if kv_lens is not None and (kv_lens.dtype is not torch.int32 or kv_lens.shape != (B,) or not kv_lens.is_contiguous()):
        raise ValueError("kv_lens must be a contiguous int32 [B]")
    return ((B, H, ks[2], Lq, ks[1], d), _PACK_HEADS(q.data_ptr(), qt[0], qt[1], qt[2]),
            _PACK_HEADS(k.data_ptr(), kt[0], kt[1], kt[2]), _PACK_HEADS(v.data_ptr(), vt[0], vt[1], vt[2]))


def cross_attention(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, kv_lens: torch.Tensor | None = None,
                    scale: float | None = None, out: torch.Tensor | None = None, return_lse: bool = False,
                    dev_status=None, stream=None):
    """softmax(scale q k^T) v: q [B, Lq, H, d], k and v [B, Lk, Hkv, d] (bf16,
    strided views included, d % 8 == 0 up to 128, Hkv divides H), over the first
    kv_lens[b] keys of sample b (all of them without kv_lens).  scale defaults
    to 1 / sqrt(d).  Returns bf16 [B, Lq, H, d], and with ``return_lse`` the FP32
    [B, H, Lq] log-sum-exp that cross_attention_backward() takes."""
    (B, H, Hkv, Lq, Lk, d), hq, hk, hv = _attention_operands(q, k, v, kv_lens)
    if out is None:
        _on_device(q, k, v, kv_lens, dev_status)
        o = _empty(stream, torch.bfloat16, q.device, B, Lq, H, d)
        to = _new_heads(o, Lq, H, d)
    else:
        o = out
        _require(o.dtype == torch.bfloat16 and o.shape == q.shape and o.stride(3) == 1, "out must be a bf16 tensor of q's shape")
        _on_device(q, k, v, kv_lens, o, dev_status)
        to = _heads(o)
    lse = _empty(stream, torch.float32, q.device, B, H, Lq) if return_lse else None
    check(lib().nvfp4_cross_attention(hq, hk, hv, None if kv_lens is None else kv_lens.data_ptr(),
                                      d ** -0.5 if scale is None else float(scale), B, H, Hkv, Lq, Lk, d, to,
                                      None if lse is None else lse.data_ptr(), _ptr(dev_status), _stream(stream)),
          "nvfp4_cross_attention")
    return (o, lse) if return_lse else o


def cross_attention_backward(grad_out: torch.Tensor, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                             out: torch.Tensor, lse: torch.Tensor, kv_lens: torch.Tensor | None = None,
                             scale: float | None = None, workspace: torch.Tensor | None = None, dev_status=None,
                             stream=None):
    """(dq, dk, dv) of cross_attention() from its ``out`` and ``lse``."""
    sizes, hq, hk, hv = _attention_operands(q, k, v, kv_lens)
    B, H, Hkv, Lq, Lk, d = sizes
    shape, bf16, device = q.shape, torch.bfloat16, q.device
    gt, ot = grad_out.stride(), out.stride()
    if (grad_out.dtype is not bf16 or out.dtype is not bf16 or grad_out.shape != shape or out.shape != shape or
            gt[3] != 1 or ot[3] != 1):
        raise ValueError("grad_out and out must be bf16 tensors of q's shape, d contiguous")
    if lse.dtype is not torch.float32 or lse.shape != (B, H, Lq) or not lse.is_contiguous():
        raise ValueError("lse must be a contiguous FP32 [B, H, Lq]")
    _on_device(grad_out, q, k, v, out, lse, kv_lens, workspace, dev_status)
    if workspace is None:
        bytes_ = nvfp4_cross_attention_backward_workspace_bytes(*sizes)
        ws = (torch.empty(bytes_, dtype=torch.uint8, device=device) if stream is None else
              _empty_on(stream, torch.uint8, device, bytes_, returned=False))
    else:
        ws = workspace
        _require(ws.is_contiguous(), "workspace must be contiguous")
        bytes_ = ws.numel() * ws.element_size()
    dq = _empty(stream, bf16, device, B, Lq, H, d)
    dk = _empty(stream, bf16, device, B, Lk, Hkv, d)
    dv = _empty(stream, bf16, device, B, Lk, Hkv, d)
    check(lib().nvfp4_cross_attention_backward(
        _PACK_HEADS(grad_out.data_ptr(), gt[0], gt[1], gt[2]), hq, hk, hv, _PACK_HEADS(out.data_ptr(), ot[0], ot[1], ot[2]),
        lse.data_ptr(),
        None if kv_lens is None else kv_lens.data_ptr(), d ** -0.5 if scale is None else float(scale), B, H, Hkv, Lq, Lk, d,
        _new_heads(dq, Lq, H, d), _new_heads(dk, Lk, Hkv, d), _new_heads(dv, Lk, Hkv, d), ws.data_ptr(), bytes_,
        _ptr(dev_status), _stream(stream)), "nvfp4_cross_attention_backward")
    return dq, dk, dv


class _CrossAttentionGradients(torch.autograd.Function):
    """The backward pass of CrossAttention under create_graph: its gradients
    depend on its inputs, but how is not known here."""

    @staticmethod
    def forward(ctx, dev_status, *args):
        return cross_attention_backward(*args, dev_status=dev_status)

    @staticmethod
    def backward(ctx, *grads):
        raise RuntimeError("CrossAttention has no second derivative")


class CrossAttention(torch.autograd.Function):
    """Autograd wrapper of cross_attention() and cross_attention_backward():
    gradients of q, k and v; a second derivative through it is refused.
    ``dev_status`` (a zeroed device int32, as for the two calls) is how a pass,
    forward or backward, tells that a wait in a kernel ran out and its results
    are incomplete: a training loop that can act on it passes one and looks at it
    where it looks at its loss.  Captured into a CUDA graph as RotaryEmbedding is."""

    @staticmethod
    def forward(ctx, q, k, v, kv_lens=None, scale=None, dev_status=None):
        out, lse = cross_attention(q, k, v, kv_lens, scale, return_lse=True, dev_status=dev_status)
        ctx.save_for_backward(q, k, v, out, lse, kv_lens)
        ctx.scale, ctx.dev_status = scale, dev_status
        return out

    @staticmethod
    def backward(ctx, grad):
        q, k, v, out, lse, kv_lens = ctx.saved_tensors
        args = (_rows16(grad), q, k, v, out, lse, kv_lens, ctx.scale)
        if torch.is_grad_enabled():                            # create_graph
            return (*_CrossAttentionGradients.apply(ctx.dev_status, *args), None, None, None)
        return (*cross_attention_backward(*args, dev_status=ctx.dev_status), None, None, None)
