"""Tensor-level wrappers over the C ABI (same names as include/w4a4.h).

Each wrapper checks dtypes/devices, allocates outputs with torch on the input's
device and calls the library on torch's current stream. Nothing is computed
here.
"""
from __future__ import annotations

import functools

import torch

from ._lib import Y_BF16, Y_F16, Y_F32, call, workspace_bytes


def _stream(t: torch.Tensor) -> int:
    return torch.cuda.current_stream(t.device).cuda_stream


def _need(t: torch.Tensor, dtype, name: str) -> None:
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA (HIP) tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")


def _ydtype(dtype) -> int:
    if dtype == torch.float32:
        return Y_F32
    if dtype == torch.float16:
        return Y_F16
    raise TypeError("output dtype must be torch.float32 or torch.float16")


def _check_out(t, name: str, shape, dtype, device, row_stride_ok: bool = False) -> None:
    """A caller-supplied output buffer must have exactly the shape, dtype and
    device the kernel writes (the C ABI cannot see buffer sizes: an undersized
    or foreign buffer would be written past its end). ``row_stride_ok``: a 2-D
    output may have a row stride above its width (unit column stride)."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a tensor")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if row_stride_ok and t.dim() == 2:
        if t.numel() and (t.stride(1) != 1 or t.stride(0) < t.shape[1]):
            raise ValueError(f"{name} must have unit column stride and row stride >= its width")
    elif not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _y_out(out, M: int, N: int, out_dtype, device) -> torch.Tensor:
    """The GEMM output: a new [M, N] tensor, or the caller's, checked (fp32 or
    fp16, [M, N] on the inputs' device, unit column stride, row stride >= N)."""
    if out is None:
        return torch.empty((M, N), dtype=out_dtype, device=device)
    _ydtype(out.dtype)
    _check_out(out, "out", (M, N), out.dtype, device, row_stride_ok=True)
    return out


def _need_scales(s: torch.Tensor, K: int, group: int, rows: int, name: str) -> None:
    """Group-major INT4 scales: contiguous, K/group x rows floats."""
    if group > 0 and K % group == 0 and (not s.is_contiguous() or s.numel() != (K // group) * rows):
        raise ValueError(f"{name} must be contiguous group-major scales [K/group, rows]")


def w4a4_quantize_act(x: torch.Tensor, group: int = 128, out=None):
    """INT4 group quantization of fp16 X[M, K] (row stride may exceed K).

    Returns ``(xq uint8 [M, K/2], xs float32 [K/group, M])``: the scales are
    group-major (``xs[c, m]`` is the scale of row m, group c).
    """
    _need(x, torch.float16, "x")
    if x.dim() != 2 or x.stride(1) != 1:
        raise ValueError("x must be 2-D with unit column stride")
    M, K = x.shape
    if out is None:
        xq = torch.empty((M, K // 2), dtype=torch.uint8, device=x.device)
        xs = torch.empty((max(K // max(group, 1), 0), M), dtype=torch.float32, device=x.device)
    else:
        xq, xs = out
        _check_out(xq, "xq", (M, K // 2), torch.uint8, x.device)
        _check_out(xs, "xs", (K // max(group, 1), M), torch.float32, x.device)
    call("w4a4_quantize_act", x.data_ptr(), M, K, x.stride(0), group,
         xq.data_ptr(), xs.data_ptr(), _stream(x))
    return xq, xs


def w4a4_pack_weight(w: torch.Tensor, group: int = 128, out=None):
    """Offline INT4 group quantization of fp16 W[N, K] (contiguous):
    ``(wq uint8 [N, K/2], ws float32 [K/group, N])``, scales group-major."""
    _need(w, torch.float16, "w")
    if w.dim() != 2 or not w.is_contiguous():
        raise ValueError("w must be a contiguous 2-D tensor")
    N, K = w.shape
    if out is None:
        wq = torch.empty((N, K // 2), dtype=torch.uint8, device=w.device)
        ws = torch.empty((max(K // max(group, 1), 0), N), dtype=torch.float32, device=w.device)
    else:
        wq, ws = out
        _check_out(wq, "wq", (N, K // 2), torch.uint8, w.device)
        _check_out(ws, "ws", (K // max(group, 1), N), torch.float32, w.device)
    call("w4a4_pack_weight", w.data_ptr(), N, K, group, wq.data_ptr(), ws.data_ptr(), _stream(w))
    return wq, ws


def w4a4_gemm(xq, xs, group_a: int, wq, ws, group_w: int, out_dtype=torch.float32, out=None):
    """Y[M, N] = group-dequantized INT4 GEMM of packed X and W."""
    for t, dt, n in ((xq, torch.uint8, "xq"), (wq, torch.uint8, "wq"),
                     (xs, torch.float32, "xs"), (ws, torch.float32, "ws")):
        _need(t, dt, n)
    M, K = xq.shape[0], xq.shape[1] * 2
    N = wq.shape[0]
    if wq.shape[1] * 2 != K:
        raise ValueError("K of xq and wq differ")
    _need_scales(xs, K, group_a, M, "xs")
    _need_scales(ws, K, group_w, N, "ws")
    y = _y_out(out, M, N, out_dtype, xq.device)
    call("w4a4_gemm", xq.data_ptr(), xs.data_ptr(), group_a, wq.data_ptr(), ws.data_ptr(), group_w,
         M, N, K, y.data_ptr(), _ydtype(y.dtype), y.stride(0), _stream(xq))
    return y


def w4a4_gemm_splitk(xq, xs, group_a: int, wq, ws, group_w: int, splits: int = 0,
                     out_dtype=torch.float32, out=None, workspace=None):
    """w4a4_gemm with K split across workgroups (``splits=0``: the library
    picks). The fp32 workspace is allocated here with torch unless given."""
    from ._lib import splitk_workspace_bytes
    for t, n in ((xq, "xq"), (wq, "wq")):
        _need(t, torch.uint8, n)
    _need(xs, torch.float32, "xs")
    _need(ws, torch.float32, "ws")
    M, K = xq.shape[0], xq.shape[1] * 2
    N = wq.shape[0]
    if wq.shape[1] * 2 != K:
        raise ValueError("K of xq and wq differ")
    _need_scales(xs, K, group_a, M, "xs")
    _need_scales(ws, K, group_w, N, "ws")
    nbytes = splitk_workspace_bytes(M, N, K, group_a, group_w, splits)
    if workspace is None:
        workspace = torch.empty((max(nbytes, 16) // 4,), dtype=torch.float32, device=xq.device)
    else:
        if not isinstance(workspace, torch.Tensor) or workspace.device != xq.device:
            raise ValueError("workspace must be a tensor on the inputs' device")
        if not workspace.is_contiguous():
            raise ValueError("workspace must be contiguous")
        if workspace.numel() * workspace.element_size() < nbytes:
            raise ValueError(f"workspace must hold {nbytes} bytes")
    y = _y_out(out, M, N, out_dtype, xq.device)
    call("w4a4_gemm_splitk", xq.data_ptr(), xs.data_ptr(), group_a, wq.data_ptr(), ws.data_ptr(), group_w,
         M, N, K, splits, workspace.data_ptr(), workspace.numel() * workspace.element_size(),
         y.data_ptr(), _ydtype(y.dtype), y.stride(0), _stream(xq))
    return y


# When w4a4_linear picks the fused launch by itself. The fused launch saves the
# activation quantizer's launch (about 5 us per linear at decode), but each of
# its workgroups re-reads and re-quantizes all of X: on 16-column tiles that
# is M/4 of the weight bytes again through L2, so its cost grows as M times the
# GEMM's own time. Measured FFN decode steps, fused against quantize + GEMM:
# LLaMA-2-70B (112 MiB of weights per linear) faster fused up to M = 3, slower
# at M = 4; LLaMA-2-7B (21.5 MiB) faster up to M = 4, even at M = 6, slower at
# M = 8. The rule M x (weight bytes + FUSED_FIXED_BYTES) <= FUSED_BUDGET_BYTES
# (the fixed term stands for the GEMM's latency, which does not shrink with
# the weights) takes M <= 3 and M <= 5 there; the kernel's own LDS limit
# (w4a4_linear_fused_supported) applies on top.
FUSED_FIXED_BYTES = 96 << 20
FUSED_BUDGET_BYTES = 640 << 20


def use_fused(M: int, N: int, K: int, group_a: int, group_w: int) -> bool:
    """Whether w4a4_linear takes the fused launch for this shape by default."""
    from ._lib import load_library
    return (M > 0 and N > 0 and M * (N * K // 2 + FUSED_FIXED_BYTES) <= FUSED_BUDGET_BYTES and
            bool(load_library().w4a4_linear_fused_supported(M, N, K, group_a, group_w)))


def w4a4_linear(x: torch.Tensor, wq, ws, group_a: int = 128, group_w: int = 128, out_dtype=torch.float32,
                out=None, fused: bool | None = None):
    """A W4A4 linear layer on fp16 activations: Y = Q(X) Q(W)^T with X quantized
    per group of ``group_a`` here. For few tokens (tiny M x K) one fused launch
    quantizes and multiplies (``w4a4_linear_fused``); otherwise the activation
    quantizer runs first and the GEMM (with its automatic K split) after it.
    ``fused``: None picks (:func:`use_fused`), True requires the fused path,
    False forbids it."""
    from ._lib import load_library
    _need(x, torch.float16, "x")
    _need(wq, torch.uint8, "wq")
    _need(ws, torch.float32, "ws")
    if x.dim() != 2 or x.stride(1) != 1:
        raise ValueError("x must be 2-D with unit column stride")
    M, K = x.shape
    N = wq.shape[0]
    if wq.shape[1] * 2 != K:
        raise ValueError("K of x and wq differ")
    _need_scales(ws, K, group_w, N, "ws")
    ok = M > 0 and N > 0 and bool(load_library().w4a4_linear_fused_supported(M, N, K, group_a, group_w))
    if fused and not ok:
        raise ValueError(f"the fused path does not take M={M} N={N} K={K} group_a={group_a}")
    if fused is None:
        fused = use_fused(M, N, K, group_a, group_w)
    if fused:
        y = _y_out(out, M, N, out_dtype, x.device)
        call("w4a4_linear_fused", x.data_ptr(), M, K, x.stride(0), group_a, wq.data_ptr(), ws.data_ptr(),
             group_w, N, y.data_ptr(), _ydtype(y.dtype), y.stride(0), _stream(x))
        return y
    xq, xs = w4a4_quantize_act(x, group_a)
    return w4a4_gemm_splitk(xq, xs, group_a, wq, ws, group_w, out_dtype=out_dtype, out=out)


def w4a4_gemm_debug_partials(xq, xs, group_a: int, wq, ws, group_w: int, m0: int, mc: int, n0: int, nc: int):
    """Exact int32 group partials P_b for the window; shape [K/g, mc, nc]."""
    for t, dt, n in ((xq, torch.uint8, "xq"), (wq, torch.uint8, "wq"),
                     (xs, torch.float32, "xs"), (ws, torch.float32, "ws")):
        _need(t, dt, n)
    M, K = xq.shape[0], xq.shape[1] * 2
    N = wq.shape[0]
    if wq.shape[1] * 2 != K:
        raise ValueError("K of xq and wq differ")
    _need_scales(xs, K, group_a, M, "xs")
    _need_scales(ws, K, group_w, N, "ws")
    g = min(group_a, group_w)
    if g <= 0 or K % g:
        raise ValueError("the finer group must divide K")
    part = torch.empty((K // g, mc, nc), dtype=torch.int32, device=xq.device)
    call("w4a4_gemm_debug_partials", xq.data_ptr(), xs.data_ptr(), group_a, wq.data_ptr(), ws.data_ptr(),
         group_w, M, N, K, m0, mc, n0, nc, part.data_ptr(), _stream(xq))
    return part


def mxfp4_quantize(x: torch.Tensor, out=None):
    """MXFP4 quantization of fp16 X[rows, K]: ``(codes uint8 [rows, K/2],
    e8m0 uint8 [rows*K/32] in the 256-k panel layout)``; see
    :func:`mxfp4_scales_to_rows` for the row-major form."""
    _need(x, torch.float16, "x")
    if x.dim() != 2 or x.stride(1) != 1:
        raise ValueError("x must be 2-D with unit column stride")
    R, K = x.shape
    if out is None:
        q = torch.empty((R, K // 2), dtype=torch.uint8, device=x.device)
        e = torch.empty((R * (K // 32),), dtype=torch.uint8, device=x.device)
    else:
        q, e = out
        _check_out(q, "codes", (R, K // 2), torch.uint8, x.device)
        _check_out(e, "e8m0", (R * (K // 32),), torch.uint8, x.device)
    call("mxfp4_quantize", x.data_ptr(), R, K, x.stride(0), q.data_ptr(), e.data_ptr(), _stream(x))
    return q, e


def _mxfp4_quantize_wide(fn: str, x: torch.Tensor, out):
    _need(x, torch.float16, "x")
    if x.dim() != 2 or x.stride(1) != 1:
        raise ValueError("x must be 2-D with unit column stride")
    R, K = x.shape
    if out is None:
        q = torch.empty((R, K), dtype=torch.uint8, device=x.device)
        e = torch.empty((R * (2 * K // 32),), dtype=torch.uint8, device=x.device)
    else:
        q, e = out
        _check_out(q, "codes", (R, K), torch.uint8, x.device)
        _check_out(e, "e8m0", (R * (2 * K // 32),), torch.uint8, x.device)
    call(fn, x.data_ptr(), R, K, x.stride(0), q.data_ptr(), e.data_ptr(), _stream(x))
    return q, e


def mxfp4_quantize_residual(x: torch.Tensor, out=None):
    """Two-pass MXFP4 with the residual appended along K: ``(codes uint8
    [rows, K] (2K codes: Q(x) then Q(x - deq Q(x))), e8m0 uint8 [rows*2K/32]
    in the panel layout of a 2K-wide matrix)``."""
    return _mxfp4_quantize_wide("mxfp4_quantize_residual", x, out)


def mxfp4_quantize_residual_tied(x: torch.Tensor, out=None):
    """Two-pass MXFP4 with the second scale tied to the first (no clipping in
    either pass; per-element error <= 2^(E1 + 3) / 64): shapes and layouts as
    :func:`mxfp4_quantize_residual`."""
    return _mxfp4_quantize_wide("mxfp4_quantize_residual_tied", x, out)


def mxfp4_quantize_append_copy(w: torch.Tensor, out=None):
    """``[Q(w) | Q(w)]`` along K (shapes as :func:`mxfp4_quantize_residual`):
    the weight side of the appended-residual GEMM."""
    return _mxfp4_quantize_wide("mxfp4_quantize_append_copy", w, out)


def _mx_shapes(xq, xe, wq, we):
    for t, n in ((xq, "xq"), (xe, "xe"), (wq, "wq"), (we, "we")):
        _need(t, torch.uint8, n)
    M, K = xq.shape[0], xq.shape[1] * 2
    N = wq.shape[0]
    if wq.shape[1] * 2 != K:
        raise ValueError("K of xq and wq differ")
    if xe.numel() != M * (K // 32) or we.numel() != N * (K // 32):
        raise ValueError("scale tensors must hold rows*K/32 bytes (panel layout)")
    return M, N, K


def mxfp4_gemm(xq, xe, wq, we, out_dtype=torch.float32, out=None):
    """Y[M, N] = block-scaled FP4 GEMM of MXFP4 X and W."""
    M, N, K = _mx_shapes(xq, xe, wq, we)
    y = _y_out(out, M, N, out_dtype, xq.device)
    call("mxfp4_gemm", xq.data_ptr(), xe.data_ptr(), wq.data_ptr(), we.data_ptr(), M, N, K,
         y.data_ptr(), _ydtype(y.dtype), y.stride(0), _stream(xq))
    return y


def mxfp4_gemm_debug_partials(xq, xe, wq, we, m0: int, mc: int, n0: int, nc: int):
    """Exact int32 block integers I_b = sum (2va)(2vw) for the window; [K/32, mc, nc]."""
    M, N, K = _mx_shapes(xq, xe, wq, we)
    part = torch.empty((K // 32, mc, nc), dtype=torch.int32, device=xq.device)
    call("mxfp4_gemm_debug_partials", xq.data_ptr(), xe.data_ptr(), wq.data_ptr(), we.data_ptr(),
         M, N, K, m0, mc, n0, nc, part.data_ptr(), _stream(xq))
    return part


# ------------------------------------------------------------------- NVFP4

def _need_scalar(t, name: str) -> None:
    _need(t, torch.float32, name)
    if t.numel() != 1:
        raise ValueError(f"{name} must hold one float")


def nvfp4_global_scale(x: torch.Tensor, out=None):
    """``fl32(max|x| / 2688)`` of fp16 X[rows, K] as a one-element float32
    tensor on the device (computed there, no host sync)."""
    _need(x, torch.float16, "x")
    if x.dim() != 2 or (x.shape[0] > 0 and x.stride(1) != 1):
        raise ValueError("x must be 2-D with unit column stride")
    g = torch.empty((1,), dtype=torch.float32, device=x.device) if out is None else out
    _check_out(g, "out", (1,), torch.float32, x.device)
    ldx = x.stride(0) if x.shape[0] > 0 else x.shape[1]
    call("nvfp4_global_scale", x.data_ptr(), x.shape[0], x.shape[1], ldx, g.data_ptr(), _stream(x))
    return g


def nvfp4_quantize(x: torch.Tensor, global_scale: torch.Tensor, out=None):
    """NVFP4 quantization of fp16 X[rows, K] with a device global scale:
    ``(codes uint8 [rows, K/2], E4M3 scales uint8 [rows*K/16] in the 256-k
    panel layout)``; see :func:`nvfp4_scales_to_rows`."""
    _need(x, torch.float16, "x")
    _need_scalar(global_scale, "global_scale")
    if x.dim() != 2 or x.stride(1) != 1:
        raise ValueError("x must be 2-D with unit column stride")
    R, K = x.shape
    if out is None:
        q = torch.empty((R, K // 2), dtype=torch.uint8, device=x.device)
        s = torch.empty((R * (K // 16),), dtype=torch.uint8, device=x.device)
    else:
        q, s = out
        _check_out(q, "codes", (R, K // 2), torch.uint8, x.device)
        _check_out(s, "scales", (R * (K // 16),), torch.uint8, x.device)
    call("nvfp4_quantize", x.data_ptr(), R, K, x.stride(0), global_scale.data_ptr(),
         q.data_ptr(), s.data_ptr(), _stream(x))
    return q, s


def _nv_shapes(xq, xs, wq, ws):
    for t, n in ((xq, "xq"), (xs, "xs"), (wq, "wq"), (ws, "ws")):
        _need(t, torch.uint8, n)
    M, K = xq.shape[0], xq.shape[1] * 2
    N = wq.shape[0]
    if wq.shape[1] * 2 != K:
        raise ValueError("K of xq and wq differ")
    if xs.numel() != M * (K // 16) or ws.numel() != N * (K // 16):
        raise ValueError("scale tensors must hold rows*K/16 bytes (panel layout)")
    return M, N, K


def nvfp4_gemm(xq, xs, x_global, wq, ws, w_global, out_dtype=torch.float32, out=None):
    """Y[M, N] = NVFP4 GEMM of X and W (fp16 matrix cores, fp32 accumulation)."""
    M, N, K = _nv_shapes(xq, xs, wq, ws)
    _need_scalar(x_global, "x_global")
    _need_scalar(w_global, "w_global")
    y = _y_out(out, M, N, out_dtype, xq.device)
    call("nvfp4_gemm", xq.data_ptr(), xs.data_ptr(), x_global.data_ptr(), wq.data_ptr(), ws.data_ptr(),
         w_global.data_ptr(), M, N, K, y.data_ptr(), _ydtype(y.dtype), y.stride(0), _stream(xq))
    return y


def nvfp4_gemm_debug_partials(xq, xs, wq, ws, m0: int, mc: int, n0: int, nc: int):
    """Exact int32 block integers I_b = sum (2vx)(2vw) over 16-blocks; [K/16, mc, nc]."""
    M, N, K = _nv_shapes(xq, xs, wq, ws)
    part = torch.empty((K // 16, mc, nc), dtype=torch.int32, device=xq.device)
    call("nvfp4_gemm_debug_partials", xq.data_ptr(), xs.data_ptr(), wq.data_ptr(), ws.data_ptr(),
         M, N, K, m0, mc, n0, nc, part.data_ptr(), _stream(xq))
    return part


# -------------------------------------------------------- storage conversions
# Canonical storage (two's-complement INT4 nibbles, row-major scales) <-> the
# layouts the GEMMs read; every conversion runs in the library's kernels.

def w4a4_repack_int4(nibbles: torch.Tensor, check: bool = True):
    """Canonical INT4 codes (uint8 [rows, K/2], two's-complement nibbles, even
    k low) -> the GEMM's INT4 layout. Returns ``(packed, minus8_count)``, the
    count a one-element int32 device tensor. With ``check`` (default) the call
    synchronizes and raises if any code is -8 (no sign-magnitude form)."""
    _need(nibbles, torch.uint8, "nibbles")
    if nibbles.dim() != 2 or not nibbles.is_contiguous():
        raise ValueError("nibbles must be a contiguous 2-D tensor")
    rows, K = nibbles.shape[0], nibbles.shape[1] * 2
    packed = torch.empty_like(nibbles)
    count = torch.empty((1,), dtype=torch.int32, device=nibbles.device)
    call("w4a4_repack_int4", nibbles.data_ptr(), rows, K, packed.data_ptr(), count.data_ptr(), _stream(nibbles))
    if check and int(count.item()) != 0:
        raise ValueError(f"{int(count.item())} INT4 codes are -8: the GEMM layout holds [-7, 7] only")
    return packed, count


def w4a4_unpack_int4(packed: torch.Tensor):
    """The GEMM's INT4 layout -> canonical two's-complement nibbles (-0 -> 0)."""
    _need(packed, torch.uint8, "packed")
    if packed.dim() != 2 or not packed.is_contiguous():
        raise ValueError("packed must be a contiguous 2-D tensor")
    out = torch.empty_like(packed)
    call("w4a4_unpack_int4", packed.data_ptr(), packed.shape[0], packed.shape[1] * 2, out.data_ptr(),
         _stream(packed))
    return out


def w4a4_scales_to_group_major(scales_rows: torch.Tensor):
    """Row-major INT4 scales float32 [rows, groups] -> group-major [groups, rows]."""
    _need(scales_rows, torch.float32, "scales_rows")
    if scales_rows.dim() != 2 or not scales_rows.is_contiguous():
        raise ValueError("scales_rows must be a contiguous 2-D tensor")
    rows, groups = scales_rows.shape
    out = torch.empty((groups, rows), dtype=torch.float32, device=scales_rows.device)
    call("w4a4_scales_to_group_major", scales_rows.data_ptr(), rows, groups, out.data_ptr(), _stream(scales_rows))
    return out


def w4a4_scales_to_row_major(scales_gm: torch.Tensor):
    """Group-major INT4 scales float32 [groups, rows] -> row-major [rows, groups]."""
    _need(scales_gm, torch.float32, "scales_gm")
    if scales_gm.dim() != 2 or not scales_gm.is_contiguous():
        raise ValueError("scales_gm must be a contiguous 2-D tensor")
    groups, rows = scales_gm.shape
    out = torch.empty((rows, groups), dtype=torch.float32, device=scales_gm.device)
    call("w4a4_scales_to_row_major", scales_gm.data_ptr(), rows, groups, out.data_ptr(), _stream(scales_gm))
    return out


def _panels(fn: str, src: torch.Tensor, rows: int, K: int, block: int, to_panels: bool):
    _need(src, torch.uint8, "scales")
    if not src.is_contiguous() or src.numel() != rows * (K // block):
        raise ValueError(f"scales must be contiguous with rows*K/{block} bytes")
    shape = (rows * (K // block),) if to_panels else (rows, K // block)
    out = torch.empty(shape, dtype=torch.uint8, device=src.device)
    call(fn, src.data_ptr(), rows, K, out.data_ptr(), _stream(src))
    return out


def mxfp4_scales_to_panels(e_rows: torch.Tensor):
    """Row-major E8M0 bytes [rows, K/32] -> the flat 256-k panel layout."""
    rows, nb = e_rows.shape
    return _panels("mxfp4_scales_to_panels", e_rows, rows, 32 * nb, 32, True)


def mxfp4_scales_to_rows(e: torch.Tensor, rows: int, K: int):
    """Panel-layout E8M0 bytes (flat, rows*K/32) -> row-major [rows, K/32]."""
    return _panels("mxfp4_scales_to_rows", e, rows, K, 32, False)


def nvfp4_scales_to_panels(s_rows: torch.Tensor):
    """Row-major E4M3 bytes [rows, K/16] -> the flat 256-k panel layout (K % 256 == 0)."""
    rows, nb = s_rows.shape
    return _panels("nvfp4_scales_to_panels", s_rows, rows, 16 * nb, 16, True)


def nvfp4_scales_to_rows(s: torch.Tensor, rows: int, K: int):
    """Panel-layout E4M3 bytes (flat, rows*K/16) -> row-major [rows, K/16]."""
    return _panels("nvfp4_scales_to_rows", s, rows, K, 16, False)


# ------------------------------------------------------- 8-bit linear layers

_DTYPE8 = {torch.float32: Y_F32, torch.float16: Y_F16, torch.bfloat16: Y_BF16}
_I8, _F32, _I32 = torch.int8, torch.float32, torch.int32


def _x_dtype8(t, name: str) -> int:
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA (HIP) tensor")
    if t.dtype not in (torch.float16, torch.bfloat16):
        raise TypeError(f"{name} must be torch.float16 or torch.bfloat16, got {t.dtype}")
    return _DTYPE8[t.dtype]


def _y_dtype8(dtype) -> int:
    if dtype not in _DTYPE8:
        raise TypeError("output dtype must be torch.float32, torch.float16 or torch.bfloat16")
    return _DTYPE8[dtype]


def _same_device(first, **others) -> None:
    for name, t in others.items():
        if t is not None and t.device != first.device:
            raise ValueError(f"{name} is on {t.device}, expected {first.device}")


def _call8(name: str, device, *args) -> None:
    """Calls an ABI entry point on ``device``'s current stream (passed last), with
    that device current for the launches."""
    index = device.index
    if index == torch._C._cuda_getDevice():
        call(name, *args, torch._C._cuda_getCurrentRawStream(index))
    else:
        with torch.cuda.device(device):
            call(name, *args, torch._C._cuda_getCurrentRawStream(index))


@functools.lru_cache(maxsize=4096)
def _workspace_size(name: str, *args) -> int:
    """A host-only workspace query (a function of its integer arguments alone)."""
    return workspace_bytes(name, *args)


def _rows_stride(x, name: str) -> int:
    """Row stride of a 2-D tensor of contiguous rows (any stride for one row)."""
    if x.dim() != 2 or (x.shape[1] > 1 and x.stride(1) != 1):
        raise ValueError(f"{name} must be 2-D with unit column stride")
    return x.stride(0) if x.shape[0] > 1 else max(x.shape[1], 1)


def _workspace8(workspace, nbytes: int, device):
    """(tensor or None, pointer, bytes): the caller's workspace, checked, or a new one."""
    if workspace is None:
        if nbytes == 0:
            return None, 0, 0
        workspace = torch.empty((nbytes,), dtype=torch.uint8, device=device)
    else:
        if not isinstance(workspace, torch.Tensor) or workspace.device != device:
            raise ValueError("workspace must be a tensor on the inputs' device")
        if not workspace.is_contiguous():
            raise ValueError("workspace must be contiguous")
        if workspace.numel() * workspace.element_size() < nbytes:
            raise ValueError(f"workspace must hold {nbytes} bytes")
    return workspace, workspace.data_ptr(), workspace.numel() * workspace.element_size()


def _w8_quantize(x, out, names):
    dt = _x_dtype8(x, names[0])
    ld = _rows_stride(x, names[0])
    M, K = x.shape
    if out is None:
        q = torch.empty((M, K), dtype=torch.int8, device=x.device)
        s = torch.empty((M,), dtype=torch.float32, device=x.device)
    else:
        q, s = out
        _check_out(q, names[1], (M, K), torch.int8, x.device)
        _check_out(s, names[2], (M,), torch.float32, x.device)
    _call8("w8a8_quantize_act", x.device, x.data_ptr(), dt, M, K, ld, q.data_ptr(), s.data_ptr())
    return q, s


def w8a8_quantize_act(x: torch.Tensor, out=None):
    """Symmetric INT8 quantization per token of fp16 or bf16 X[M, K] (row stride
    may exceed K): ``(xq int8 [M, K], xs float32 [M])``, ``x ~ xq * xs``; NaN scales
    for rows that are not finite."""
    return _w8_quantize(x, out, ("x", "xq", "xs"))


def w8a8_pack_weight(w: torch.Tensor, out=None):
    """Offline INT8 quantization per output channel of fp16 or bf16 W[N, K]:
    ``(wq int8 [N, K], ws float32 [N])``."""
    return _w8_quantize(w, out, ("w", "wq", "ws"))


def _w8_weights(wq, ws, bias, device):
    """Checks the weight side of a W8A8 product; returns (N, K)."""
    _need(wq, torch.int8, "wq")
    _need(ws, torch.float32, "ws")
    if wq.dim() != 2 or not wq.is_contiguous() or not ws.is_contiguous():
        raise ValueError("wq must be a contiguous 2-D tensor and ws contiguous")
    N, K = wq.shape
    if ws.shape != (N,):
        raise ValueError("ws must hold one scale per output channel: shape (N,)")
    if bias is not None:
        _need(bias, torch.float32, "bias")
        if bias.shape != (N,) or not bias.is_contiguous():
            raise ValueError("bias must be a contiguous [N] tensor")
        if bias.device != device:
            raise ValueError(f"bias is on {bias.device}, expected {device}")
    if wq.device != device or ws.device != device:
        raise ValueError(f"wq is on {wq.device} and ws on {ws.device}, expected {device}")
    return N, K


def _y_out8(out, shape, out_dtype, device, row_stride_ok=True):
    """The output of an 8-bit call (new, or the caller's, checked) and its dtype code."""
    if out is None:
        return torch.empty(shape, dtype=out_dtype, device=device), _y_dtype8(out_dtype)
    dt = _y_dtype8(out.dtype) if isinstance(out, torch.Tensor) else 0
    _check_out(out, "out", shape, getattr(out, "dtype", None), device, row_stride_ok=row_stride_ok)
    return out, dt


def w8a8_gemm(xq, xs, wq, ws, bias=None, out_dtype=torch.float32, out=None, workspace=None):
    """Y[M, N] = (xq @ wq^T) scaled by xs[m] * ws[n], plus ``bias`` float32 [N].
    The INT8 products are summed exactly. Y is fp32, fp16 or bf16; the
    workspace (K split across workgroups for small outputs) is allocated here
    with torch unless given."""
    _need(xq, torch.int8, "xq")
    _need(xs, torch.float32, "xs")
    if xq.dim() != 2 or not xq.is_contiguous() or not xs.is_contiguous():
        raise ValueError("xq must be a contiguous 2-D tensor and xs contiguous")
    M = xq.shape[0]
    N, K = _w8_weights(wq, ws, bias, xq.device)
    if xq.shape[1] != K:
        raise ValueError("K of xq and wq differ")
    if xs.shape != (M,):
        raise ValueError("xs must hold one scale per row: shape (M,)")
    _same_device(xq, xs=xs)
    y, dt = _y_out8(out, (M, N), out_dtype, xq.device)
    held, wptr, wbytes = _workspace8(workspace, _workspace_size("w8a8_gemm_workspace", M, N, K), xq.device)
    _call8("w8a8_gemm", xq.device, xq.data_ptr(), xs.data_ptr(), wq.data_ptr(), ws.data_ptr(),
           0 if bias is None else bias.data_ptr(), M, N, K, wptr, wbytes, y.data_ptr(), dt,
           y.stride(0) if M > 1 else max(N, 1))
    return y


def w8a8_linear(x: torch.Tensor, wq, ws, bias=None, out_dtype=torch.float32, out=None, workspace=None):
    """A W8A8 linear layer on fp16 or bf16 activations [M, K] (row stride may
    exceed K): X quantized per token, then the product of :func:`w8a8_gemm`, in one
    call. The workspace (codes, scales, partial sums) is allocated here with
    torch unless given."""
    xdt = _x_dtype8(x, "x")
    ld = _rows_stride(x, "x")
    M = x.shape[0]
    N, K = _w8_weights(wq, ws, bias, x.device)
    if x.shape[1] != K:
        raise ValueError("K of x and wq differ")
    y, dt = _y_out8(out, (M, N), out_dtype, x.device)
    held, wptr, wbytes = _workspace8(workspace, _workspace_size("w8a8_linear_workspace", M, N, K), x.device)
    _call8("w8a8_linear", x.device, x.data_ptr(), xdt, M, K, ld, wq.data_ptr(), ws.data_ptr(),
           0 if bias is None else bias.data_ptr(), N, wptr, wbytes, y.data_ptr(), dt,
           y.stride(0) if M > 1 else max(N, 1))
    return y


# ------------------------------------- around the W8A8 products: include/ffn8.h

_ACTIVATIONS = {None: 0, "relu": 1, "silu": 2, "gelu": 3, "gelu_tanh": 4}


def _activation(name) -> int:
    if name not in _ACTIVATIONS:
        raise ValueError(f"activation must be None, 'relu', 'silu', 'gelu' or 'gelu_tanh', got {name!r}")
    return _ACTIVATIONS[name]


def _need_rows(t, name: str, shape, dtype, device) -> int:
    """Row stride of a checked 2-D operand of contiguous rows."""
    try:                                               # the checks of _check_out, at a third of its time
        rows, one = t.stride()
        if t.dtype is dtype and t.shape == shape and one == 1 and rows >= shape[1] and t.device == device:
            return rows if shape[0] > 1 else max(shape[1], 1)
    except (AttributeError, TypeError, ValueError):    # not a 2-D tensor
        pass
    _check_out(t, name, shape, dtype, device, row_stride_ok=True)
    return t.stride(0) if shape[0] > 1 else max(shape[1], 1)


def _overlap(a, b) -> bool:
    """Whether two 2-D tensors of contiguous rows share memory (columns apart in rows of
    one stride do not)."""
    def span(t):
        rows, cols = t.shape
        start = t.data_ptr()
        return start, start + t.element_size() * ((rows - 1) * t.stride(0) + cols) if rows and cols else start
    (a0, a1), (b0, b1) = span(a), span(b)
    if a0 >= b1 or b0 >= a1:
        return False
    size, pitch = a.element_size(), a.stride(0)
    if a.shape[0] > 1 and b.shape[0] > 1 and size == b.element_size() and pitch == b.stride(0) and (b0 - a0) % size == 0:
        apart = (b0 - a0) // size % pitch
        return apart < a.shape[1] or apart + b.shape[1] > pitch
    return True


def _in_place_or_apart(out, t, names: str) -> None:
    """An output may be the input ``t`` itself, or must not meet it."""
    same = out.data_ptr() == t.data_ptr() and (out.shape[0] == 1 or out.stride(0) == t.stride(0))
    if not same and _overlap(out, t):
        raise ValueError(f"{names} overlap without being the same tensor")


def w8a8_rmsnorm_quantize(x: torch.Tensor, weight, eps: float = 1e-6, residual=None, return_normed: bool = False,
                          out=None):
    """RMS norm of fp16 or bf16 X[M, K] (row stride may exceed K) to INT8 codes and one
    scale per row, the input of :func:`w8a8_gemm` and :func:`w8a8_moe`: ``(xq int8
    [M, K], xs float32 [M])``, where ``xq * xs ~ h * weight / sqrt(mean(h^2) + eps)``.

    With ``residual`` (X's shape and type) h is x + residual, rounded to X's type, and
    comes third; with ``return_normed`` the normed rows in X's type come last. ``weight``:
    [K], float32 or X's type. ``out``: the tuple of outputs to fill instead; its h may
    be ``x`` or ``residual`` itself (in place), else the outputs lie apart from one another
    and from the inputs. ``eps``: at least 2^-126. Rows that are not finite have NaN scales."""
    dt = _x_dtype8(x, "x")
    ldx = _rows_stride(x, "x")
    shape, device, dtype = x.shape, x.device, x.dtype
    M, K = shape
    if not isinstance(weight, torch.Tensor) or (weight.dtype is not torch.float32 and weight.dtype is not dtype):
        raise TypeError(f"weight must be a torch.float32 or {dtype} tensor")
    if weight.shape != (K,) or not weight.is_contiguous() or weight.device != device:
        raise ValueError(f"weight must be a contiguous [{K}] tensor on {device}")
    if not 2.0 ** -126 <= eps < 2.0 ** 128:
        raise ValueError("eps must be at least 2^-126 and finite as a float32")
    r = ldr = h = ldh = y = ldy = 0
    if residual is not None:
        ldr = _need_rows(residual, "residual", shape, dtype, device)
        r = residual.data_ptr()
    if out is None:
        new = x.new_empty
        xq, xs = new(shape, dtype=_I8), new(M, dtype=_F32)
        out = xq, xs
        if residual is not None:
            ldh = K
            out += (new(shape),)
            h = out[2].data_ptr()
        if return_normed:
            ldy = K
            out += (new(shape),)
            y = out[-1].data_ptr()
    else:
        out = tuple(out)
        if len(out) != 2 + (residual is not None) + bool(return_normed):
            raise ValueError(f"out must hold {2 + (residual is not None) + bool(return_normed)} tensors")
        xq, xs = out[:2]
        _check_out(xq, "xq", shape, torch.int8, device)
        _check_out(xs, "xs", (M,), torch.float32, device)
        if residual is not None:
            ldh = _need_rows(out[2], "h", shape, dtype, device)
            h = out[2].data_ptr()
            _in_place_or_apart(out[2], x, "h and x")
            _in_place_or_apart(out[2], residual, "h and residual")
        if return_normed:
            ldy = _need_rows(out[-1], "normed", shape, dtype, device)
            y = out[-1].data_ptr()
            for t in (x, *((residual, out[2]) if residual is not None else ())):
                if _overlap(out[-1], t):
                    raise ValueError("normed overlaps x, residual or h")
    _call8("w8a8_rmsnorm_quantize", device, x.data_ptr(), dt, ldx, r, ldr, weight.data_ptr(), _DTYPE8[weight.dtype], eps,
           M, K, xq.data_ptr(), xs.data_ptr(), h, ldh, y, ldy)
    return out


def w8a8_pack_gated(w_gate: torch.Tensor, w_up: torch.Tensor):
    """Offline INT8 quantization of a gated layer's two weights (fp16 or bf16, both
    [N, K], or [E, N, K] for experts), channels interleaved: rows 2n and 2n + 1 of the
    result are the gate's and the other's row n. ``(wq int8 [2 N, K], ws float32
    [2 N])``, with a leading E for experts."""
    if w_gate.shape != w_up.shape or w_gate.dtype != w_up.dtype or w_gate.dim() not in (2, 3):
        raise ValueError("w_gate and w_up must be alike, [N, K] or [E, N, K]")
    w = torch.stack((w_gate, w_up), dim=-2).flatten(-3, -2)
    wq, ws = w8a8_pack_weight(w.reshape(-1, w.shape[-1]))
    return wq.view(w.shape), ws.view(w.shape[:-1])


def _act_operands(device, M, wq, ws, bias, gated, residual, out_dtype, out):
    """Checked weights and output of a product with an epilogue:
    (N, K, residual stride, y, dtype code, y's stride, wide)."""
    C, K = _w8_weights(wq, ws, bias, device)
    if gated and C % 2:
        raise ValueError("gated weights hold two channels an output: an even number of rows")
    N = C // 2 if gated else C
    if out is None:
        y = torch.empty((M, N), dtype=out_dtype, device=device)
    else:
        y = out
        _check_out(y, "out", (M, N), getattr(y, "dtype", None), device, row_stride_ok=True)
    if y.dtype is not torch.float16 and y.dtype is not torch.bfloat16:
        raise TypeError("output dtype must be torch.float16 or torch.bfloat16")
    ldy = y.stride(0) if M > 1 else max(N, 1)
    wide = N % 8 == 0 and ldy % 8 == 0 and ldy < 1 << 22 and y.data_ptr() % 16 == 0
    ldr = 0
    if residual is not None:
        ldr = _need_rows(residual, "residual", (M, N), y.dtype, device)
        wide = wide and ldr % 8 == 0 and ldr < 1 << 22 and residual.data_ptr() % 16 == 0
        if out is not None:
            _in_place_or_apart(out, residual, "out and residual")
    return N, K, ldr, y, _DTYPE8[y.dtype], ldy, int(wide)


def w8a8_gemm_act(xq, xs, wq, ws, bias=None, activation=None, gated: bool = False, residual=None,
                  out_dtype=torch.float16, out=None, workspace=None):
    """:func:`w8a8_gemm` with an epilogue: Y = act(v) + residual with v = (xq @ wq^T)
    scaled + ``bias``, in fp32, rounded once to fp16 or bf16.

    ``activation``: None, "relu", "silu", "gelu" or "gelu_tanh". ``gated``: ``wq`` [2 N, K] as
    :func:`w8a8_pack_gated` lays it out, and Y[m, n] = act(v[m, 2n]) * v[m, 2n + 1] +
    residual; ``bias`` is interleaved alike. ``residual``: [M, N] of Y's type; ``out`` may be
    it, and lies apart from every other input."""
    _need(xq, torch.int8, "xq")
    _need(xs, torch.float32, "xs")
    if xq.dim() != 2 or not xq.is_contiguous() or not xs.is_contiguous():
        raise ValueError("xq must be a contiguous 2-D tensor and xs contiguous")
    M = xq.shape[0]
    device = xq.device
    if xs.shape != (M,):
        raise ValueError("xs must hold one scale per row: shape (M,)")
    _same_device(xq, xs=xs)
    act, gated = _activation(activation), int(bool(gated))
    N, K, ldr, y, dt, ldy, wide = _act_operands(device, M, wq, ws, bias, gated, residual, out_dtype, out)
    if xq.shape[1] != K:
        raise ValueError("K of xq and wq differ")
    held, wptr, wbytes = _workspace8(workspace, _workspace_size("w8a8_gemm_act_workspace", M, N, K, gated, wide), device)
    _call8("w8a8_gemm_act", device, xq.data_ptr(), xs.data_ptr(), wq.data_ptr(), ws.data_ptr(),
           0 if bias is None else bias.data_ptr(), act, gated, 0 if residual is None else residual.data_ptr(), ldr,
           M, N, K, wptr, wbytes, y.data_ptr(), dt, ldy)
    return y


def w8a8_linear_act(x: torch.Tensor, wq, ws, bias=None, activation=None, gated: bool = False, residual=None,
                    out_dtype=torch.float16, out=None, workspace=None):
    """:func:`w8a8_linear` with the epilogue of :func:`w8a8_gemm_act`: fp16 or bf16
    activations [M, K] quantized per token, the product, bias, activation or gate, and
    residual, in one call. ``out`` may be ``residual`` but not overlap ``x``, which every
    workgroup reads, or another input."""
    xdt = _x_dtype8(x, "x")
    ld = _rows_stride(x, "x")
    M = x.shape[0]
    device = x.device
    act, gated = _activation(activation), int(bool(gated))
    N, K, ldr, y, dt, ldy, wide = _act_operands(device, M, wq, ws, bias, gated, residual, out_dtype, out)
    if x.shape[1] != K:
        raise ValueError("K of x and wq differ")
    if out is not None and _overlap(x, out):
        raise ValueError("out overlaps x")
    held, wptr, wbytes = _workspace8(workspace, _workspace_size("w8a8_linear_act_workspace", M, N, K, gated, wide), device)
    _call8("w8a8_linear_act", device, x.data_ptr(), xdt, M, K, ld, wq.data_ptr(), ws.data_ptr(),
           0 if bias is None else bias.data_ptr(), act, gated, 0 if residual is None else residual.data_ptr(), ldr,
           N, wptr, wbytes, y.data_ptr(), dt, ldy)
    return y


def moe_route(logits: torch.Tensor, top_k: int, renormalize: bool = True, out=None):
    """The ``top_k`` largest router logits of every token: ``(ids int32 [T, top_k], weights
    float32 [T, top_k])``, largest first, the lower id first among equals; the weights
    are a softmax over all experts, or with ``renormalize`` over the chosen ones.
    ``logits``: [T, E] fp32, fp16 or bf16 (row stride may exceed E). Minus infinity and NaN are
    never chosen: where fewer are left, ids are -1 and weights 0."""
    if not isinstance(logits, torch.Tensor) or not logits.is_cuda:
        raise TypeError("logits must be a CUDA (HIP) tensor")
    dt = _y_dtype8(logits.dtype)
    ld = _rows_stride(logits, "logits")
    T, E = logits.shape
    k = _need_max(top_k, "top_k")
    if out is None:
        ids = logits.new_empty((T, k), dtype=_I32)
        weights = logits.new_empty((T, k), dtype=_F32)
    else:
        ids, weights = out
        _check_out(ids, "ids", (T, k), torch.int32, logits.device)
        _check_out(weights, "weights", (T, k), torch.float32, logits.device)
    _call8("moe_route", logits.device, logits.data_ptr(), dt, T, E, ld, k, int(bool(renormalize)), ids.data_ptr(),
           weights.data_ptr())
    return ids, weights


_MOE_TENSORS = (("xq", torch.int8, 2), ("xs", torch.float32, 1), ("ids", torch.int32, 2), ("weights", torch.float32, 2),
                ("w13", torch.int8, 3), ("s13", torch.float32, 2), ("w2", torch.int8, 3), ("s2", torch.float32, 2))


def _moe_refuse(tensors):
    """Raises for the first of w8a8_moe's operands that a kernel cannot take."""
    device = next((t.device for t in tensors if isinstance(t, torch.Tensor)), None)
    for t, (name, dtype, dims) in zip(tensors, _MOE_TENSORS):
        _need(t, dtype, name)
        if t.dim() != dims or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous {dims}-D tensor")
        if t.device != device:
            raise ValueError(f"{name} is on {t.device}, expected {device}")


def w8a8_moe(xq, xs, ids, weights, w13, s13, w2, s2, activation="silu", out_dtype=torch.float16, out=None,
             workspace=None):
    """A mixture-of-experts layer of few tokens (T * k <= 512) on INT8 experts, in two
    launches (up to four for many pairs): Y[T, H] = sum over a token's choices of weight *
    (w2[e] @ quantized(act(gate) * up)), gate and up the interleaved channels of
    w13[e] @ x.

    ``xq`` int8 [T, H], ``xs`` float32 [T]: tokens as :func:`w8a8_rmsnorm_quantize` or
    :func:`w8a8_quantize_act` give them. ``ids`` int32, ``weights`` float32 [T, k]: from
    :func:`moe_route`; ids that are no expert add nothing. ``w13`` int8 [E, 2 I, H], ``s13``
    float32 [E, 2 I]: from :func:`w8a8_pack_gated`; ``w2`` int8 [E, H, I], ``s2`` [E, H]: from
    :func:`w8a8_pack_weight`. Longer batches go in slices of tokens. Y is fp16 or bf16."""
    try:                                               # the checks of _moe_refuse, at a third of its time
        at = xq.get_device()
        fine = (at >= 0 and xq.dtype is _I8 and xs.dtype is _F32 and ids.dtype is _I32 and weights.dtype is _F32 and
                w13.dtype is _I8 and s13.dtype is _F32 and w2.dtype is _I8 and s2.dtype is _F32 and
                at == xs.get_device() == ids.get_device() == weights.get_device() == w13.get_device() ==
                s13.get_device() == w2.get_device() == s2.get_device() and
                xq.is_contiguous() and xs.is_contiguous() and ids.is_contiguous() and weights.is_contiguous() and
                w13.is_contiguous() and s13.is_contiguous() and w2.is_contiguous() and s2.is_contiguous() and
                xq.dim() == ids.dim() == 2 and w13.dim() == 3)
    except AttributeError:                             # not a tensor
        fine = False
    if not fine:
        _moe_refuse((xq, xs, ids, weights, w13, s13, w2, s2))
    device = xq.device
    (T, H), (E, two_i, _), k = xq.shape, w13.shape, ids.shape[1]
    I = two_i // 2
    if xs.shape != (T,) or ids.shape != (T, k) or weights.shape != (T, k):
        raise ValueError("xs must be [T], ids and weights [T, k]")
    if two_i % 2 or w13.shape != (E, 2 * I, H) or s13.shape != (E, 2 * I) or w2.shape != (E, H, I) or s2.shape != (E, H):
        raise ValueError("w13 must be [E, 2 I, H], s13 [E, 2 I], w2 [E, H, I] and s2 [E, H]")
    act = _activation(activation)
    if out_dtype is not torch.float16 and out_dtype is not torch.bfloat16:
        raise TypeError("out_dtype must be torch.float16 or torch.bfloat16")
    if out is None:
        y = torch.empty((T, H), dtype=out_dtype, device=device)
    else:
        y = out
        _check_out(y, "out", (T, H), getattr(y, "dtype", None), device, row_stride_ok=True)
    dt = _x_dtype8(y, "out")
    held, wptr, wbytes = _workspace8(workspace, _workspace_size("w8a8_moe_workspace", T, k, E, H, I), device)
    _call8("w8a8_moe", device, xq.data_ptr(), xs.data_ptr(), ids.data_ptr(), weights.data_ptr(), T, k, w13.data_ptr(),
           s13.data_ptr(), w2.data_ptr(), s2.data_ptr(), E, H, I, act, wptr, wbytes, y.data_ptr(), dt,
           y.stride(0) if T > 1 else max(H, 1))
    return y


# ------------------------------------------------------ INT8 key/value cache

def kv8_new_cache(num_pages: int, heads: int, page: int, dim: int, device="cuda"):
    """An empty pool for :func:`kv8_append`: ``(k_cache int8 [num_pages, heads,
    page, dim], v_cache int8 [num_pages, heads, dim, page], k_scale, v_scale
    float32 [num_pages, heads])``, all zero. ``page``: positions per page (16,
    32, 64, 128 or 256); ``dim``: 64, 128, 192 or 256."""
    if page not in (16, 32, 64, 128, 256) or dim not in (64, 128, 192, 256):
        raise ValueError("page must be 16, 32, 64, 128 or 256 and dim 64, 128, 192 or 256")
    return (torch.zeros((num_pages, heads, page, dim), dtype=torch.int8, device=device),
            torch.zeros((num_pages, heads, dim, page), dtype=torch.int8, device=device),
            torch.zeros((num_pages, heads), dtype=torch.float32, device=device),
            torch.zeros((num_pages, heads), dtype=torch.float32, device=device))


_KV_TENSORS = (("k_cache", torch.int8), ("v_cache", torch.int8), ("k_scale", torch.float32),
               ("v_scale", torch.float32), ("block_table", torch.int32), ("cu_seqlens", torch.int32),
               ("seq_lens", torch.int32))


def _kv_refuse(tensors):
    """Raises for the first tensor of a pool or batch that a kernel cannot take."""
    device = next((t.device for t in tensors if isinstance(t, torch.Tensor)), None)
    for t, (name, dtype) in zip(tensors, _KV_TENSORS):
        _need(t, dtype, name)
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
        if t.device != device:
            raise ValueError(f"{name} is on {t.device}, expected {device}")


def _kv_pool(*tensors):
    """Checked pool and batch: (pool pointers, pool extents, batch pointers, B)."""
    k_cache, v_cache, k_scale, v_scale, block_table, cu_seqlens, seq_lens = tensors
    try:                                               # the checks of _kv_refuse, at a third of its time
        at = k_cache.get_device()
        fine = (at >= 0 and k_cache.dtype is _I8 and v_cache.dtype is _I8 and k_scale.dtype is _F32 and
                v_scale.dtype is _F32 and block_table.dtype is _I32 and cu_seqlens.dtype is _I32 and
                seq_lens.dtype is _I32 and
                at == v_cache.get_device() == k_scale.get_device() == v_scale.get_device() ==
                block_table.get_device() == cu_seqlens.get_device() == seq_lens.get_device() and
                k_cache.is_contiguous() and v_cache.is_contiguous() and k_scale.is_contiguous() and
                v_scale.is_contiguous() and block_table.is_contiguous() and cu_seqlens.is_contiguous() and
                seq_lens.is_contiguous())
    except AttributeError:                             # not a tensor
        fine = False
    if not fine:
        _kv_refuse(tensors)
    if k_cache.dim() != 4:
        raise ValueError("k_cache must be [num_pages, heads, page, dim]")
    extents = pages, heads, page, dim = k_cache.shape
    if v_cache.shape != (pages, heads, dim, page):
        raise ValueError("v_cache must be [num_pages, heads, dim, page]")
    if k_scale.shape != (pages, heads) or v_scale.shape != (pages, heads):
        raise ValueError("k_scale and v_scale must be [num_pages, heads]")
    lens, table = seq_lens.shape, block_table.shape
    if len(lens) != 1 or cu_seqlens.shape != (lens[0] + 1,):
        raise ValueError("cu_seqlens must be [B + 1] for seq_lens [B]")
    if len(table) != 2 or table[0] != lens[0]:
        raise ValueError("block_table must be [B, pages per sequence]")
    return (k_cache.data_ptr(), v_cache.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr()), extents, \
        (block_table.data_ptr(), table[1], cu_seqlens.data_ptr(), seq_lens.data_ptr()), lens[0]


def _need_max(value, name: str) -> int:
    if isinstance(value, bool) or not isinstance(value, int) or value < 0:
        raise ValueError(f"{name} must be a non-negative int")
    return value


def _heads_strides(t, name: str, heads: int, dim: int):
    """(token stride, head stride) of a [T, heads, dim] tensor of contiguous rows."""
    shape = t.shape
    if len(shape) != 3 or shape[1] != heads or shape[2] != dim:
        raise ValueError(f"{name} must be [T, {heads}, {dim}]")
    tok, head, one = t.stride()
    if one != 1 and t.numel():
        raise ValueError(f"{name} must have a unit stride along its last dimension")
    return (tok if shape[0] > 1 else heads * dim), (head if heads > 1 else dim)


def kv8_append(k, v, k_cache, v_cache, k_scale, v_scale, block_table, cu_seqlens, seq_lens, max_new: int):
    """Quantize the new keys and values (fp16 or bf16 [T, heads, dim], strided
    views allowed) into the pages of the cache, in place.

    Sequence b's new tokens are rows ``cu_seqlens[b] .. cu_seqlens[b+1] - 1``, and
    the last positions of its ``seq_lens[b]`` (new tokens included). A page keeps
    one scale per head: it grows when a new token needs it, and the codes
    already there are rescaled (each time off by half a step more, at most). NaN or
    infinite values make it NaN. Everything but ``max_new`` (at least the largest
    number of new tokens of a sequence) is read on the device."""
    ptrs, (pages, heads, page, dim), batch, B = _kv_pool(k_cache, v_cache, k_scale, v_scale, block_table,
                                                         cu_seqlens, seq_lens)
    dt = _x_dtype8(k, "k")
    _need(v, k.dtype, "v")
    _same_device(k_cache, k=k, v=v)
    kt, kh = _heads_strides(k, "k", heads, dim)
    vt, vh = _heads_strides(v, "v", heads, dim)
    if v.shape[0] != k.shape[0]:
        raise ValueError("k and v hold different numbers of tokens")
    _call8("kv8_append", k_cache.device, k.data_ptr(), v.data_ptr(), dt, kt, kh, vt, vh, *ptrs, pages, heads, page,
           dim, *batch, B, k.shape[0], _need_max(max_new, "max_new"), batch[1] * page)


def kv8_gather(k_cache, v_cache, k_scale, v_scale, block_table, cu_seqlens, seq_lens, total: int, max_new: int,
               out_dtype=torch.float16, out=None):
    """The cached keys and values as numbers: ``(k, v)`` of ``out_dtype``, each
    [total, heads, dim], rows ``cu_seqlens[b] .. cu_seqlens[b+1] - 1`` holding the last
    positions of sequence b (the mirror of :func:`kv8_append`). ``out``: a pair
    of contiguous tensors to fill instead; rows of no sequence are left alone."""
    ptrs, (pages, heads, page, dim), batch, B = _kv_pool(k_cache, v_cache, k_scale, v_scale, block_table,
                                                         cu_seqlens, seq_lens)
    shape = (_need_max(total, "total"), heads, dim)
    if out is None:
        _y_dtype8(out_dtype)
        k = torch.empty(shape, dtype=out_dtype, device=k_cache.device)
        v = torch.empty_like(k)
    else:
        k, v = out
        if isinstance(k, torch.Tensor):
            _y_dtype8(k.dtype)
        _check_out(k, "k", shape, getattr(k, "dtype", None), k_cache.device)
        _check_out(v, "v", shape, k.dtype, k_cache.device)
    _call8("kv8_gather", k_cache.device, *ptrs, pages, heads, page, dim, *batch, B, total,
           _need_max(max_new, "max_new"), batch[1] * page, k.data_ptr(), v.data_ptr(), _DTYPE8[k.dtype])
    return k, v


def kv8_attention(q, k_cache, v_cache, k_scale, v_scale, block_table, cu_seqlens, seq_lens, max_new: int,
                  max_len: int, scale: float | None = None, causal: bool = True, window: int = 0, out_dtype=None,
                  out=None, return_lse: bool = False, workspace=None):
    """Attention of the new tokens' queries (fp16 or bf16 [T, q_heads, dim],
    strided views allowed) over the cache that already holds their keys and
    values: one new token per sequence (decoding), a few (drafts) or many
    (prefill), in any mix.

    ``max_new`` / ``max_len``: at least every sequence's new tokens / cached
    positions (host numbers that size the launch; the true ones are read on the
    device). ``scale`` defaults to dim ** -0.5; ``window`` w > 0 hides the keys w
    and more positions back. Returns [T, q_heads, dim] of ``out_dtype`` (default:
    q's), with ``return_lse`` also float32 [T, q_heads] (natural log). A query that
    sees no key gives zeros and -inf; rows of no sequence are left alone. One
    kernel, chosen by ``max_new``, serves the call: many single tokens beside a long
    chunk are faster in a call of their own with the same ``out``. The
    workspace is allocated here with torch unless given."""
    ptrs, (pages, heads, page, dim), batch, B = _kv_pool(k_cache, v_cache, k_scale, v_scale, block_table,
                                                         cu_seqlens, seq_lens)
    dt = _x_dtype8(q, "q")
    _same_device(k_cache, q=q)
    if q.dim() != 3 or q.shape[1] == 0 or q.shape[1] % heads:
        raise ValueError(f"q must be [T, q_heads, {dim}] with q_heads a multiple of {heads}")
    T, hq = q.shape[:2]
    qt, qh = _heads_strides(q, "q", hq, dim)
    if isinstance(window, bool) or not isinstance(window, int) or window < 0:
        raise ValueError("window must be a non-negative int (0: none)")
    _need_max(max_new, "max_new")
    if _need_max(max_len, "max_len") > batch[1] * page:
        raise ValueError(f"max_len {max_len} is past the block table's {batch[1]} pages of {page}")
    device = q.device
    y, ydt = _y_out8(out, (T, hq, dim), out_dtype or q.dtype, device, row_stride_ok=False)
    lse = torch.empty((T, hq), dtype=torch.float32, device=device) if return_lse else None
    causal = int(causal)
    held, wptr, wbytes = _workspace8(workspace, _workspace_size(
        "kv8_attention_workspace", hq, heads, page, dim, B, T, max_new, max_len, causal, window), device)
    _call8("kv8_attention", device, q.data_ptr(), dt, qt, qh, hq, *ptrs, pages, heads, page, dim, *batch, B, T,
           max_new, max_len, dim ** -0.5 if scale is None else scale, causal, window, wptr, wbytes, y.data_ptr(),
           ydt, 0 if lse is None else lse.data_ptr())
    return (y, lse) if return_lse else y
