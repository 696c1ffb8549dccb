"""Python binding of libdynconv over torch tensors (argument marshalling only).

Every function has the name of the C entry point it calls; all compute runs in the HIP
kernels. Tensors must live on a ROCm device; PyTorch provides device memory and the
current stream, nothing else.
"""
from __future__ import annotations

import ctypes
from typing import NamedTuple

import torch

from . import _lib

_DTYPE = {torch.float32: _lib.DYNCONV_F32, torch.bfloat16: _lib.DYNCONV_BF16, torch.float16: _lib.DYNCONV_F16}


def _ptr(t):
    return ctypes.c_void_p(t.data_ptr()) if t is not None else ctypes.c_void_p(0)


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype not in _DTYPE:
        raise TypeError(f"unsupported dtype {t.dtype}; use float32, bfloat16 or float16")
    return _DTYPE[t.dtype]


def _require_device(*ts):
    dev = None
    for t in ts:
        if t is None:
            continue
        i = t.get_device()  # -1 on the CPU; half the time of comparing device objects
        if i < 0:
            raise RuntimeError("libdynconv runs on the GPU only: got a CPU tensor")
        if dev is None:
            dev, first = t.device, i
        elif i != first:
            raise RuntimeError("all tensors must be on the same device")
    return dev


def _stream(dev) -> ctypes.c_void_p:
    return ctypes.c_void_p(torch.cuda.current_stream(dev).cuda_stream)


def filter_strides(w: torch.Tensor):
    """Strides of a filter tensor: [B,T,G,W] as is; a static [G,W] filter gets zero b,t strides."""
    if w.dim() == 2:
        return [0, 0, w.stride(0), w.stride(1)]
    if w.dim() != 4:
        raise ValueError("filters are [B, T, D/H, W] or a static [D/H, W]")
    return list(w.stride())


def _seg_args(seq_idx, B: int, T: int):
    """(pointer, strides) of packed-sequence segment ids: int32 [B, T] (any strides)."""
    if seq_idx.dtype != torch.int32 or tuple(seq_idx.shape) != (B, T):
        raise ValueError(f"seq_idx must be int32 [B, T] = [{B}, {T}]; got {seq_idx.dtype} {tuple(seq_idx.shape)}")
    return _ptr(seq_idx), _lib.strides(seq_idx.stride())


def _conv_bias_arg(conv_bias, x):
    if conv_bias is None:
        return None
    D = x.shape[-1]
    if conv_bias.dim() != 1 or conv_bias.numel() != D or conv_bias.stride(0) != 1 or conv_bias.dtype != x.dtype:
        raise ValueError(f"conv_bias must be a contiguous [{D}] vector of dtype {x.dtype}")
    return conv_bias


def _expect(name: str, t, shape, dtype) -> None:
    """Raises unless t (if given) has exactly this shape and dtype: the C ABI receives
    strides, not extents, so a tensor of the wrong size would be read or written out of
    bounds instead of being refused."""
    if t is None:
        return
    if t.shape != shape and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {list(shape)}; got {list(t.shape)}")
    if t.dtype != dtype:
        raise TypeError(f"{name} is {t.dtype} but must be {dtype}")


def _groups(D: int, H: int) -> int:
    if H < 1 or D % H != 0:
        raise ValueError(f"H = {H} must be a positive divisor of D = {D}")
    return D // H


def _check_act3(x: torch.Tensor) -> tuple:
    if x.dim() != 3:
        raise ValueError(f"x must be [B, T, D]; got shape {list(x.shape)}")
    return tuple(x.shape)


def _check_filter(w: torch.Tensor, x: torch.Tensor, H: int) -> int:
    """w is per-token [B, T, D/H, W] or static [D/H, W], of x's dtype; returns W."""
    B, T, D = x.shape
    G = _groups(D, H)
    W = w.shape[-1]
    _expect("w", w, (G, W) if w.dim() == 2 else (B, T, G, W), x.dtype)
    return W


def dynconv_fwd(x: torch.Tensor, w: torch.Tensor, H: int = 1, out: torch.Tensor | None = None,
                seq_idx: torch.Tensor | None = None, conv_bias: torch.Tensor | None = None) -> torch.Tensor:
    """y = x + causal depthwise conv of x with per-token (or static) filters w (+ conv_bias
    [D] on every token). With seq_idx (int32 [B, T] segment ids of packed sequences) no tap
    crosses into another segment."""
    B, T, D = _check_act3(x)
    W = _check_filter(w, x, H)
    conv_bias = _conv_bias_arg(conv_bias, x)
    _expect("out", out, (B, T, D), x.dtype)
    y = torch.empty_like(x) if out is None else out
    dev = _require_device(x, w, y, seq_idx, conv_bias)
    lib = _lib.load()
    head = (_ptr(x), _lib.strides(x.stride()), _ptr(w), _lib.strides(filter_strides(w)))
    tail = (_ptr(y), _lib.strides(y.stride()), B, T, D, W, H, _dtype_code(x), _stream(dev))
    if conv_bias is not None:
        seg = _seg_args(seq_idx, B, T) if seq_idx is not None else (None, None)
        st = lib.dynconv_fwd_ex(*head, *seg, _ptr(conv_bias), *tail)
    elif seq_idx is None:
        st = lib.dynconv_fwd(*head, *tail)
    else:
        st = lib.dynconv_fwd_varlen(*head, *_seg_args(seq_idx, B, T), *tail)
    _lib.check("dynconv_fwd", st)
    return y


def dynconv_bwd_workspace_size(B, T, D, W, H, is_static, dtype) -> int:
    return int(_lib.load().dynconv_bwd_workspace_size(B, T, D, W, H, int(bool(is_static)), _DTYPE[dtype]))


def dynconv_bwd(x, w, dy, H: int = 1, need_dx: bool = True, need_dw: bool = True, dx=None, dw=None, seq_idx=None,
                want_dconv_bias: bool = False):
    """(dx, dw) of <dy, dynconv_fwd(x, w, H, seq_idx=seq_idx)>; dw of a static filter is
    float32 [D/H, W]. With want_dconv_bias, (dx, dw, dconv_bias) where dconv_bias is the
    float32 [D] gradient of a convolution bias (the sum of dy over every token)."""
    B, T, D = _check_act3(x)
    W = _check_filter(w, x, H)
    is_static = w.dim() == 2
    _expect("dy", dy, (B, T, D), x.dtype)
    _expect("dx", dx, (B, T, D), x.dtype)
    _expect("dw", dw, (D // H, W) if is_static else (B, T, D // H, W), torch.float32 if is_static else x.dtype)
    if need_dx and dx is None:
        dx = torch.empty_like(x)
    if need_dw and dw is None:
        dw = (torch.empty((D // H, W), dtype=torch.float32, device=x.device) if is_static
              else torch.empty((B, T, D // H, W), dtype=x.dtype, device=x.device))
    dev = _require_device(x, w, dy, dx, dw, seq_idx)
    lib = _lib.load()
    if want_dconv_bias:
        dcb = torch.empty((D,), dtype=torch.float32, device=x.device)
        ws_bytes = int(lib.dynconv_bwd_ex_workspace_size(B, T, D, W, H, int(is_static and need_dw), 1,
                                                         _DTYPE[x.dtype]))
    else:
        ws_bytes = dynconv_bwd_workspace_size(B, T, D, W, H, is_static and need_dw, x.dtype)
    work = torch.empty(max(ws_bytes, 1), dtype=torch.uint8, device=x.device) if ws_bytes else None
    head = (_ptr(x), _lib.strides(x.stride()), _ptr(w), _lib.strides(filter_strides(w)))
    tail = (
        _ptr(dy), _lib.strides(dy.stride()),
        _ptr(dx if need_dx else None), _lib.strides(dx.stride()) if need_dx else None,
        _ptr(dw if need_dw else None), _lib.strides(dw.stride()) if (need_dw and not is_static) else None,
        B, T, D, W, H, _dtype_code(x), _ptr(work), ws_bytes, _stream(dev),
    )
    if want_dconv_bias:
        seg = _seg_args(seq_idx, B, T) if seq_idx is not None else (None, None)
        st = lib.dynconv_bwd_ex(*head, *seg, *tail[:6], _ptr(dcb), *tail[6:])
        _lib.check("dynconv_bwd", st)
        return (dx if need_dx else None), (dw if need_dw else None), dcb
    if seq_idx is None:
        st = lib.dynconv_bwd(*head, *tail)
    else:
        st = lib.dynconv_bwd_varlen(*head, *_seg_args(seq_idx, B, T), *tail)
    _lib.check("dynconv_bwd", st)
    return (dx if need_dx else None), (dw if need_dw else None)


def dynconv_bwd_ex_noalloc(x, w, dy, H: int = 1, dx=None, dw=None, dconv_bias=None, seq_idx=None):
    """The allocation-free backward: (dx, dw, dconv_bias) as dynconv_bwd(..., want_dconv_bias=
    dconv_bias is not None) computes them, with the partial sums in the library's per-GPU
    scratch array instead of a workspace. The caller passes every output it wants (dx
    [B,T,D], dw per-token [B,T,D/H,W] or float32 [D/H,W] for a static w, dconv_bias float32
    [D]); this binding allocates nothing either. Calls that overlap on one GPU race."""
    B, T, D = _check_act3(x)
    W = _check_filter(w, x, H)
    is_static = w.dim() == 2
    _expect("dy", dy, (B, T, D), x.dtype)
    _expect("dx", dx, (B, T, D), x.dtype)
    _expect("dw", dw, (D // H, W) if is_static else (B, T, D // H, W), torch.float32 if is_static else x.dtype)
    _expect("dconv_bias", dconv_bias, (D,), torch.float32)
    dev = _require_device(x, w, dy, dx, dw, dconv_bias, seq_idx)
    seg = _seg_args(seq_idx, B, T) if seq_idx is not None else (None, None)
    st = _lib.load().dynconv_bwd_ex_noalloc(
        _ptr(x), _lib.strides(x.stride()), _ptr(w), _lib.strides(filter_strides(w)), *seg,
        _ptr(dy), _lib.strides(dy.stride()), _ptr(dx), _lib.strides(dx.stride()) if dx is not None else None,
        _ptr(dw), _lib.strides(dw.stride()) if (dw is not None and not is_static) else None, _ptr(dconv_bias),
        B, T, D, W, H, _dtype_code(x), _stream(dev))
    _lib.check("dynconv_bwd_ex_noalloc", st)
    return dx, dw, dconv_bias


def _check_lowrank_operands(x, z, U, bias, J: int):
    """z is [B, T, R] (or [B, R] for a decoding step, x [B, D]), U is [R, J] with unit
    column stride (rows ldu = U.stride(0) apart), bias a contiguous [J] vector or None, and
    every operand has the dtype of x."""
    R = z.shape[-1]
    if z.dim() != x.dim() or tuple(z.shape[:-1]) != tuple(x.shape[:-1]):
        raise ValueError(f"z must be {list(x.shape[:-1]) + ['R']}; got shape {list(z.shape)}")
    if U.dim() != 2 or tuple(U.shape) != (R, J) or (J > 1 and U.stride(1) != 1):
        raise ValueError(f"U must be [R, J] = [{R}, {J}] with unit column stride; got shape "
                         f"{tuple(U.shape)} strides {tuple(U.stride())}")
    if bias is not None and (bias.dim() != 1 or bias.numel() != J or (J > 1 and bias.stride(0) != 1)):
        raise ValueError(f"bias must be a contiguous [{J}] vector")
    for name, t in (("z", z), ("U", U), ("bias", bias)):
        if t is not None and t.dtype != x.dtype:
            raise TypeError(f"{name} is {t.dtype} but x is {x.dtype}")


def dynconv_lowrank_fwd(x, z, U, bias, W: int, H: int = 1, out=None, seq_idx=None, conv_bias=None):
    """y = x + conv(x) with filters z U + bias generated on the GPU (never stored), plus
    conv_bias [D] on every token if given; with seq_idx (int32 [B, T]) no tap crosses into
    another segment."""
    B, T, D = _check_act3(x)
    R = z.shape[-1]
    _check_lowrank_operands(x, z, U, bias, _groups(D, H) * W)
    conv_bias = _conv_bias_arg(conv_bias, x)
    _expect("out", out, (B, T, D), x.dtype)
    y = torch.empty_like(x) if out is None else out
    dev = _require_device(x, z, U, bias, y, seq_idx, conv_bias)
    lib = _lib.load()
    head = (_ptr(x), _lib.strides(x.stride()), _ptr(z), _lib.strides(z.stride()), _ptr(U), U.stride(0), _ptr(bias))
    tail = (_ptr(y), _lib.strides(y.stride()), B, T, D, W, H, R, _dtype_code(x), _stream(dev))
    if conv_bias is not None:
        seg = _seg_args(seq_idx, B, T) if seq_idx is not None else (None, None)
        st = lib.dynconv_lowrank_fwd_ex(*head, *seg, _ptr(conv_bias), *tail)
    elif seq_idx is None:
        st = lib.dynconv_lowrank_fwd(*head, *tail)
    else:
        st = lib.dynconv_lowrank_fwd_varlen(*head, *_seg_args(seq_idx, B, T), *tail)
    _lib.check("dynconv_lowrank_fwd", st)
    return y


def dynconv_lowrank_bwd_workspace_size(B, T, D, W, H, R, dtype, want_dconv_bias: bool = False) -> int:
    return int(_lib.load().dynconv_lowrank_bwd_ex_workspace_size(B, T, D, W, H, R, int(bool(want_dconv_bias)),
                                                                 _DTYPE[dtype]))


def dynconv_lowrank_bwd(x, z, U, bias, dy, W: int, H: int = 1, need_db: bool = True, workspace=None,
                        seq_idx=None, want_dconv_bias: bool = False):
    """(dx, dz, dU, db) of <dy, dynconv_lowrank_fwd(...)>; dU and db are float32. With
    want_dconv_bias, (dx, dz, dU, db, dconv_bias): the float32 [D] gradient of a convolution
    bias (the sum of dy over every token). A caller's workspace must be a contiguous tensor
    on x's device of at least dynconv_lowrank_bwd_workspace_size(..., want_dconv_bias)
    bytes (the library checks the size)."""
    B, T, D = _check_act3(x)
    R = z.shape[-1]
    J = _groups(D, H) * W
    _check_lowrank_operands(x, z, U, bias, J)
    _expect("dy", dy, (B, T, D), x.dtype)
    if workspace is not None and not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    dev = _require_device(x, z, U, bias, dy, seq_idx, workspace)
    dx = torch.empty_like(x)
    dz = torch.empty_like(z)
    dU = torch.empty((R, J), dtype=torch.float32, device=x.device)
    db = torch.empty((J,), dtype=torch.float32, device=x.device) if need_db else None
    dcb = torch.empty((D,), dtype=torch.float32, device=x.device) if want_dconv_bias else None
    lib = _lib.load()
    if workspace is None:
        ws_bytes = dynconv_lowrank_bwd_workspace_size(B, T, D, W, H, R, x.dtype, want_dconv_bias)
        workspace = torch.empty(max(ws_bytes, 1), dtype=torch.uint8, device=x.device)
    else:
        ws_bytes = workspace.numel() * workspace.element_size()
    head = (_ptr(x), _lib.strides(x.stride()), _ptr(z), _lib.strides(z.stride()), _ptr(U), U.stride(0), _ptr(bias))
    tail = (
        _ptr(dy), _lib.strides(dy.stride()), _ptr(dx), _lib.strides(dx.stride()), _ptr(dz), _lib.strides(dz.stride()),
        _ptr(dU), _ptr(db), B, T, D, W, H, R, _dtype_code(x), _ptr(workspace), ws_bytes, _stream(dev),
    )
    if want_dconv_bias:
        seg = _seg_args(seq_idx, B, T) if seq_idx is not None else (None, None)
        st = lib.dynconv_lowrank_bwd_ex(*head, *seg, *tail[:8], _ptr(dcb), *tail[8:])
        _lib.check("dynconv_lowrank_bwd", st)
        return dx, dz, dU, db, dcb
    if seq_idx is None:
        st = lib.dynconv_lowrank_bwd(*head, *tail)
    else:
        st = lib.dynconv_lowrank_bwd_varlen(*head, *_seg_args(seq_idx, B, T), *tail)
    _lib.check("dynconv_lowrank_bwd", st)
    return dx, dz, dU, db


# ----------------------------------------------------------------------------------
# The convolution in the epilogue of the producing projection: X = A Wp^T is formed in
# the same kernel and never stored
# ----------------------------------------------------------------------------------


def _check_projection(A, Wp, H: int):
    B, T, K = _check_act3(A)
    if Wp.dim() != 2 or Wp.shape[1] != K or (K > 1 and Wp.stride(1) != 1):
        raise ValueError(f"Wp must be [N, K={K}] with unit column stride; got shape {list(Wp.shape)} "
                         f"strides {list(Wp.stride())}")
    if Wp.dtype != A.dtype:
        raise TypeError(f"Wp is {Wp.dtype} but A is {A.dtype}")
    N = Wp.shape[0]
    return B, T, K, N, _groups(N, H)


def dynconv_gemm_fwd(A, Wp, w, H: int = 1, out=None):
    """y = X + conv(X) with X = A Wp^T (A [B,T,K], Wp [N,K]) computed in the same kernel;
    w: per-token filters [B,T,N/H,W] or a static [N/H,W]."""
    B, T, K, N, G = _check_projection(A, Wp, H)
    W = w.shape[-1]
    _expect("w", w, (G, W) if w.dim() == 2 else (B, T, G, W), A.dtype)
    _expect("out", out, (B, T, N), A.dtype)
    dev = _require_device(A, Wp, w, out)
    y = torch.empty((B, T, N), dtype=A.dtype, device=A.device) if out is None else out
    st = _lib.load().dynconv_gemm_fwd(_ptr(A), _lib.strides(A.stride()), _ptr(Wp), Wp.stride(0), _ptr(w),
                                      _lib.strides(filter_strides(w)), _ptr(y), _lib.strides(y.stride()), B, T, N, K,
                                      W, H, _dtype_code(A), _stream(dev))
    _lib.check("dynconv_gemm_fwd", st)
    return y


def dynconv_gemm_lowrank_fwd(A, Wp, z, U, bias, W: int, H: int = 1, out=None):
    """y = X + conv(X) with X = A Wp^T and filters z U + bias, both formed in the same kernel
    (neither X nor the filters are stored). z [B,T,R], U [R,(N/H)*W], bias [(N/H)*W] or None."""
    B, T, K, N, G = _check_projection(A, Wp, H)
    R = z.shape[-1]
    _check_lowrank_operands(A, z, U, bias, G * W)  # z [B, T, R] like A's leading dims, A's dtype
    _expect("out", out, (B, T, N), A.dtype)
    dev = _require_device(A, Wp, z, U, bias, out)
    y = torch.empty((B, T, N), dtype=A.dtype, device=A.device) if out is None else out
    st = _lib.load().dynconv_gemm_lowrank_fwd(
        _ptr(A), _lib.strides(A.stride()), _ptr(Wp), Wp.stride(0), _ptr(z), _lib.strides(z.stride()), _ptr(U),
        U.stride(0), _ptr(bias), _ptr(y), _lib.strides(y.stride()), B, T, N, K, W, H, R, _dtype_code(A), _stream(dev))
    _lib.check("dynconv_gemm_lowrank_fwd", st)
    return y


# ----------------------------------------------------------------------------------
# Inference: rolling cache of the last W-1 inputs, single-token decoding steps
# ----------------------------------------------------------------------------------


def new_cache(B: int, D: int, W: int, dtype, device) -> torch.Tensor | None:
    """A zeroed [B, W-1, D] cache (None for W == 1)."""
    if W == 1:
        return None
    return torch.zeros((B, W - 1, D), dtype=dtype, device=device)


def dynconv_cache_fill(x, W: int, cache=None, seq_idx=None):
    """Fills the cache with the last W-1 tokens of a prompt x [B,T,D] (zeros before t = 0).
    With seq_idx (int32 [B, T]) of a packed prompt, only the tokens of the last document
    (the segment of token T-1) are kept."""
    B, T, D = _check_act3(x)
    if W < 1:
        raise ValueError(f"W = {W} must be positive")
    _expect("cache", cache, (B, W - 1, D), x.dtype)
    if cache is None:
        cache = new_cache(B, D, W, x.dtype, x.device)
    if cache is None:
        return None
    dev = _require_device(x, cache, seq_idx)
    lib = _lib.load()
    if seq_idx is None:
        st = lib.dynconv_cache_fill(_ptr(x), _lib.strides(x.stride()), _ptr(cache), _lib.strides(cache.stride()),
                                    B, T, D, W, _dtype_code(x), _stream(dev))
    else:
        st = lib.dynconv_cache_fill_varlen(_ptr(x), _lib.strides(x.stride()), *_seg_args(seq_idx, B, T), _ptr(cache),
                                           _lib.strides(cache.stride()), B, T, D, W, _dtype_code(x), _stream(dev))
    _lib.check("dynconv_cache_fill", st)
    return cache


def dynconv_decode_step(x, w, cache, t: int, H: int = 1, out=None, conv_bias=None):
    """y [B,D] of token t from x [B,D], its filters w [B,D/H,W] (or a static [D/H,W]) and
    the cache of the previous W-1 inputs, which is updated in place (+ conv_bias [D])."""
    if x.dim() != 2:
        raise ValueError(f"x must be [B, D]; got shape {list(x.shape)}")
    B, D = x.shape
    G = _groups(D, H)
    W = w.shape[-1]
    _expect("w", w, (G, W) if w.dim() == 2 else (B, G, W), x.dtype)
    _expect("cache", cache, (B, W - 1, D), x.dtype)
    if cache is None and W > 1:
        raise ValueError("a cache [B, W-1, D] is required for W > 1")
    _expect("out", out, (B, D), x.dtype)
    ws = [0, w.stride(0), w.stride(1)] if w.dim() == 2 else list(w.stride())
    y = torch.empty_like(x) if out is None else out
    conv_bias = _conv_bias_arg(conv_bias, x)
    dev = _require_device(x, w, y, cache, conv_bias)
    cs = _lib.strides(cache.stride()) if cache is not None else None
    st = _lib.load().dynconv_decode_step_ex(_ptr(x), _lib.strides(x.stride()), _ptr(w), _lib.strides(ws),
                                            _ptr(conv_bias), _ptr(cache), cs, _ptr(y), _lib.strides(y.stride()),
                                            int(t), B, D, W, H, _dtype_code(x), _stream(dev))
    _lib.check("dynconv_decode_step", st)
    return y


def dynconv_lowrank_decode_step(x, z, U, bias, cache, t: int, W: int, out=None, H: int = 1, conv_bias=None):
    """y [B,D] of token t with filters z [B,R] U + bias generated on the GPU (U: [R, (D/H)*W]),
    plus conv_bias [D] if given; the cache is updated in place."""
    if x.dim() != 2:
        raise ValueError(f"x must be [B, D]; got shape {list(x.shape)}")
    B, D = x.shape
    R = z.shape[-1]
    _check_lowrank_operands(x, z, U, bias, _groups(D, H) * W)
    _expect("cache", cache, (B, W - 1, D), x.dtype)
    if cache is None and W > 1:
        raise ValueError("a cache [B, W-1, D] is required for W > 1")
    _expect("out", out, (B, D), x.dtype)
    y = torch.empty_like(x) if out is None else out
    conv_bias = _conv_bias_arg(conv_bias, x)
    dev = _require_device(x, z, U, bias, y, cache, conv_bias)
    cs = _lib.strides(cache.stride()) if cache is not None else None
    st = _lib.load().dynconv_lowrank_decode_step_ex(
        _ptr(x), _lib.strides(x.stride()), _ptr(z), _lib.strides(z.stride()), _ptr(U), U.stride(0), _ptr(bias),
        _ptr(conv_bias), _ptr(cache), cs, _ptr(y), _lib.strides(y.stride()), int(t), B, D, W, H, R, _dtype_code(x),
        _stream(dev))
    _lib.check("dynconv_lowrank_decode_step", st)
    return y


# ----------------------------------------------------------------------------------
# Gated delta rule: the recurrence behind the convolved q, k, v
# ----------------------------------------------------------------------------------


def _launch(fn: str, dev, *args) -> None:
    """Calls a C entry point on dev's current stream, with dev as the current device."""
    call = getattr(_lib.load(), fn)
    stream = torch._C._cuda_getCurrentRawStream(dev.index)  # current_stream() builds an object: 2 us
    if torch._C._cuda_getDevice() == dev.index:
        st = call(*args, stream)
    else:
        with torch.cuda.device(dev):
            st = call(*args, stream)
    if st != 0:
        _lib.check(fn, st)


def _sp(t):
    """(pointer, strides) of a tensor, or two NULLs."""
    return (t.data_ptr(), _lib.const_strides(t.stride())) if t is not None else (None, None)


def _dp(t):
    return t.data_ptr() if t is not None else None


def _delta_shapes(q, k, v, g, beta, token: bool):
    """Checks the operands of a gated delta rule call; returns (lead, Hk, Hv, dk, dv) with
    lead = (B, T), or (B,) for one token."""
    n = 3 if token else 4
    lead_name = "[B, Hk, dk]" if token else "[B, T, Hk, dk]"
    if q.dim() != n:
        raise ValueError(f"q must be {lead_name}; got shape {list(q.shape)}")
    if v.dim() != n:
        raise ValueError(f"v must be {lead_name.replace('k', 'v')}; got shape {list(v.shape)}")
    (*lead, Hk, dk), (Hv, dv) = q.shape, v.shape[-2:]
    if Hk < 1 or Hv < 1 or Hv % Hk != 0:
        raise ValueError(f"the {Hv} value heads must be a multiple of the {Hk} key heads")
    if dk < 1 or dv < 1:
        raise ValueError(f"heads need at least one channel; got {dk} of q and k, {dv} of v")
    _dtype_code(q)
    heads = (*lead, Hv)
    _expect("k", k, q.shape, q.dtype)
    _expect("v", v, (*heads, dv), q.dtype)
    _expect("g", g, heads, torch.float32)
    _expect("beta", beta, heads, q.dtype)
    return lead, Hk, Hv, dk, dv


def _delta_consts(scale, qk_norm_eps, dk: int):
    if qk_norm_eps is not None and not qk_norm_eps >= 0.0:
        raise ValueError(f"qk_norm_eps = {qk_norm_eps} must be at least 0, or None")
    return (float(dk) ** -0.5 if scale is None else float(scale)), -1.0 if qk_norm_eps is None else float(qk_norm_eps)


def new_delta_state(B: int, Hv: int, dk: int, dv: int, device) -> torch.Tensor:
    """A zeroed float32 [B, Hv, dk, dv] state of the gated delta rule."""
    return torch.zeros((B, Hv, dk, dv), dtype=torch.float32, device=device)


def dynconv_delta_fwd(q, k, v, g, beta, scale: float | None = None, qk_norm_eps: float | None = None, seq_idx=None,
                      state=None, want_state: bool = False, out=None, state_out=None):
    """o [B,T,Hv,dv] of the gated delta rule on q, k [B,T,Hk,dk], v [B,T,Hv,dv], log decays g
    (float32 [B,T,Hv]) and write strengths beta [B,T,Hv]:

        S_t = e^{g_t} S_{t-1} + k_t (beta_t (v_t - e^{g_t} S_{t-1}^T k_t))^T,  o_t = scale S_t^T q_t,

    scale = dk^-0.5 by default, key head h // (Hv // Hk) for value head h. With qk_norm_eps,
    q and k are divided by sqrt(|.|^2 + qk_norm_eps) first. With seq_idx (int32 [B,T]) the
    state restarts from zero at every document start. state: the float32 [B,Hv,dk,dv] state
    before token 0 (default zero). With want_state, or a state_out to write (which may be
    state itself), returns (o, state after token T-1)."""
    (B, T), Hk, Hv, dk, dv = _delta_shapes(q, k, v, g, beta, False)
    scale, eps = _delta_consts(scale, qk_norm_eps, dk)
    _expect("state", state, (B, Hv, dk, dv), torch.float32)
    _expect("state_out", state_out, (B, Hv, dk, dv), torch.float32)
    _expect("out", out, (B, T, Hv, dv), q.dtype)
    dev = _require_device(q, k, v, g, beta, seq_idx, state, out, state_out)
    seg = _seg_args(seq_idx, B, T) if seq_idx is not None else (None, None)
    o = torch.empty((B, T, Hv, dv), dtype=q.dtype, device=dev) if out is None else out
    if want_state and state_out is None:
        state_out = torch.empty((B, Hv, dk, dv), dtype=torch.float32, device=dev)
    code = _dtype_code(q)
    ws_bytes = int(_lib.load().dynconv_delta_fwd_workspace_size(B, T, Hk, Hv, dk, dv, code))
    work = torch.empty(ws_bytes, dtype=torch.uint8, device=dev) if ws_bytes else None
    _launch("dynconv_delta_fwd", dev, *_sp(q), *_sp(k), *_sp(v), *_sp(g), *_sp(beta), *seg, *_sp(state), *_sp(o),
            *_sp(state_out), B, T, Hk, Hv, dk, dv, scale, eps, code, _dp(work), ws_bytes)
    return o if state_out is None else (o, state_out)


def dynconv_delta_bwd(q, k, v, g, beta, do, scale: float | None = None, qk_norm_eps: float | None = None, seq_idx=None,
                      state=None, dstate_out=None, need_dstate: bool = False):
    """(dq, dk, dv, dg, dbeta, dstate) of <do, o> (+ <dstate_out, final state> with the float32
    [B,Hv,dk,dv] gradient of the state after the last token) for dynconv_delta_fwd with the
    same arguments; dg is float32, dstate (float32, the gradient of `state`) None unless
    need_dstate. The states are recomputed, nothing is kept from the forward."""
    (B, T), Hk, Hv, dk, dv = _delta_shapes(q, k, v, g, beta, False)
    scale, eps = _delta_consts(scale, qk_norm_eps, dk)
    _expect("do", do, (B, T, Hv, dv), q.dtype)
    _expect("state", state, (B, Hv, dk, dv), torch.float32)
    _expect("dstate_out", dstate_out, (B, Hv, dk, dv), torch.float32)
    dev = _require_device(q, k, v, g, beta, do, seq_idx, state, dstate_out)
    seg = _seg_args(seq_idx, B, T) if seq_idx is not None else (None, None)

    def new(shape, dtype):
        return torch.empty(shape, dtype=dtype, device=dev)

    dq, dk_ = new((B, T, Hk, dk), q.dtype), new((B, T, Hk, dk), q.dtype)
    dv_, dg, dbeta = new((B, T, Hv, dv), q.dtype), new((B, T, Hv), torch.float32), new((B, T, Hv), q.dtype)
    dstate = None
    if need_dstate:  # without tokens the state's gradient passes through
        dstate = new((B, Hv, dk, dv), torch.float32) if T else (
            torch.zeros((B, Hv, dk, dv), dtype=torch.float32, device=dev) if dstate_out is None else dstate_out.clone())
    code = _dtype_code(q)
    ws_bytes = int(_lib.load().dynconv_delta_bwd_workspace_size(B, T, Hk, Hv, dk, dv, code))
    work = torch.empty(ws_bytes, dtype=torch.uint8, device=dev) if ws_bytes else None
    _launch("dynconv_delta_bwd", dev, *_sp(q), *_sp(k), *_sp(v), *_sp(g), *_sp(beta), *seg, *_sp(state), *_sp(do),
            *_sp(dstate_out), *_sp(dq), *_sp(dk_), *_sp(dv_), *_sp(dg), *_sp(dbeta), *_sp(dstate), B, T, Hk, Hv, dk,
            dv, scale, eps, code, _dp(work), ws_bytes)
    return dq, dk_, dv_, dg, dbeta, dstate


def dynconv_delta_step(q, k, v, g, beta, state, scale: float | None = None, qk_norm_eps: float | None = None, out=None):
    """o [B,Hv,dv] of one token of every sequence (q, k [B,Hk,dk], v [B,Hv,dv], g float32 and
    beta [B,Hv]); state (float32 [B,Hv,dk,dv]) is updated in place."""
    (B,), Hk, Hv, dk, dv = _delta_shapes(q, k, v, g, beta, True)
    scale, eps = _delta_consts(scale, qk_norm_eps, dk)
    if state is None:
        raise ValueError("a state [B, Hv, dk, dv] is required")
    _expect("state", state, (B, Hv, dk, dv), torch.float32)
    _expect("out", out, (B, Hv, dv), q.dtype)
    dev = _require_device(q, k, v, g, beta, state, out)
    o = torch.empty((B, Hv, dv), dtype=q.dtype, device=dev) if out is None else out
    _launch("dynconv_delta_step", dev, *_sp(q), *_sp(k), *_sp(v), *_sp(g), *_sp(beta), *_sp(state), *_sp(o), B, Hk, Hv,
            dk, dv, scale, eps, _dtype_code(q))
    return o


# ----------------------------------------------------------------------------------
# RMS norm with a weight, a SiLU gate and a scaled residual
# ----------------------------------------------------------------------------------

_NORM_RESIDUAL = {None: 0, "before": 1, "after": 2}


def _norm_shape(x):
    if not 1 <= x.dim() <= 4:
        raise ValueError(f"x must have 1 to 4 dimensions; got shape {list(x.shape)}")
    return (1,) * (4 - x.dim()) + x.shape


def _sp4(t):
    """(pointer, four strides) of a tensor of up to 4 dimensions, or two NULLs."""
    return (t.data_ptr(), _lib.const_strides((0,) * (4 - t.dim()) + t.stride())) if t is not None else (None, None)


def _norm_weight(weight, x):
    if weight is None:
        return
    _expect("weight", weight, (x.shape[-1],), x.dtype)
    if weight.numel() > 1 and weight.stride(0) != 1:
        raise ValueError("weight must be contiguous")


def dynconv_norm_fwd(x, weight=None, gate=None, residual=None, residual_scale: float = 1.0, residual_at: str = "before",
                     eps: float = 1e-6, out=None, out_h=None):
    """y = x / sqrt(mean(x^2) + eps) * weight * silu(gate) over the last dimension of x (1 to 4
    dimensions; weight [D] and gate, of x's shape, are optional).

    With a residual (x's shape) and residual_at="before", h = residual + residual_scale * x
    takes x's place, and (y, h) is returned; with "after", y = residual + residual_scale * (...)."""
    shape = _norm_shape(x)
    code = _dtype_code(x)
    if residual_at not in ("before", "after"):
        raise ValueError(f"residual_at is 'before' or 'after'; got {residual_at!r}")
    before = residual is not None and residual_at == "before"
    _norm_weight(weight, x)
    for name, t in (("gate", gate), ("residual", residual), ("out", out), ("out_h", out_h)):
        _expect(name, t, x.shape, x.dtype)
    if out_h is not None and not before:
        raise ValueError("out_h goes with a residual before the norm")
    dev = _require_device(x, weight, gate, residual, out, out_h)
    y = torch.empty(x.shape, dtype=x.dtype, device=dev) if out is None else out
    h = (torch.empty(x.shape, dtype=x.dtype, device=dev) if out_h is None else out_h) if before else None
    _launch("dynconv_norm_fwd", dev, *_sp4(x), _dp(weight), *_sp4(gate), *_sp4(residual), int(residual_at == "after"),
            float(residual_scale), *_sp4(y), *_sp4(h), *shape, float(eps), code)
    return (y, h) if before else y


def dynconv_norm_bwd(x, weight, dy, gate=None, dh=None, residual_scale: float = 1.0, residual_at: str | None = None,
                     eps: float = 1e-6):
    """(dx, dresidual, dweight, dgate) of <dy, y> for dynconv_norm_fwd, None where there is no
    such input. x is what was normalised: the forward's x or, with residual_at="before", its h
    (dh is then the gradient of h from its other uses). residual_at=None: no residual; with
    "after" the residual's gradient is dy itself and None is returned in its place. dweight is
    float32 [D]."""
    shape = _norm_shape(x)
    code = _dtype_code(x)
    if residual_at not in _NORM_RESIDUAL:
        raise ValueError(f"residual_at is 'before', 'after' or None; got {residual_at!r}")
    if dh is not None and residual_at != "before":
        raise ValueError("dh goes with a residual before the norm")
    _norm_weight(weight, x)
    for name, t in (("dy", dy), ("gate", gate), ("dh", dh)):
        _expect(name, t, x.shape, x.dtype)
    dev = _require_device(x, weight, dy, gate, dh)

    def new():
        return torch.empty(x.shape, dtype=x.dtype, device=dev)

    dx, dres, dgate = new(), new() if residual_at == "before" else None, new() if gate is not None else None
    dw = torch.empty((x.shape[-1],), dtype=torch.float32, device=dev) if weight is not None else None
    ws_bytes = int(_lib.load().dynconv_norm_bwd_workspace_size(*shape, code)) if dw is not None else 0
    work = torch.empty(ws_bytes, dtype=torch.uint8, device=dev) if ws_bytes else None
    _launch("dynconv_norm_bwd", dev, *_sp4(x), _dp(weight), *_sp4(gate), *_sp4(dy), *_sp4(dh),
            _NORM_RESIDUAL[residual_at], float(residual_scale), *_sp4(dx), *_sp4(dres), _dp(dw), *_sp4(dgate), *shape,
            float(eps), code, _dp(work), ws_bytes)
    return dx, dres, dw, dgate


# ----------------------------------------------------------------------------------
# Plans: what a call needs besides pointers
# ----------------------------------------------------------------------------------

_PLANS: dict = {}


def _plan(make, extra: tuple, *tensors):
    """make(*extra, *tensors) checks a call's arguments and returns its sizes and stride arrays (not to be
    written): once for all calls whose tensors have these shapes, strides and types, which takes 5 to 8 us
    less than every time."""
    key = (make, extra, *[None if t is None else (t.shape, t.stride(), t.dtype) for t in tensors])
    plan = _PLANS.get(key)
    if plan is None:
        plan = make(*extra, *tensors)
        if len(_PLANS) >= 4096:
            _PLANS.clear()
        _PLANS[key] = plan
    return plan


def _st(t, n: int | None = None):
    """Stride array of a tensor (of n dimensions, leading ones of stride 0 added), or NULL."""
    return None if t is None else _lib.const_strides((0,) * (0 if n is None else n - t.dim()) + t.stride())


def _dense(shape, n: int | None = None):
    """Stride array of a new tensor of this shape."""
    strides, step = [], 1
    for size in reversed(shape):
        strides.append(step)
        step *= max(size, 1)
    return _lib.const_strides((0,) * (0 if n is None else n - len(shape)) + tuple(reversed(strides)))


def _workspace(fn: str, *sizes) -> int:
    return int(getattr(_lib.load(), fn)(*sizes))


def _seq_strides(seq_idx, B: int, T: int):
    return None if seq_idx is None else _seg_args(seq_idx, B, T)[1]


# ----------------------------------------------------------------------------------
# Activations in 8 bits, for backward passes
# ----------------------------------------------------------------------------------

PACK8_GROUP = 64  # channels that share a scale


class Packed8(NamedTuple):
    """A tensor in 8 bits: int8 codes of its shape, and uint8 scales [..., ceil(D/64)] (the float32
    exponent field of the step that 64 channels share). What dynconv_pack8 returns, and what the
    backward calls that say so take in place of the tensor."""

    codes: torch.Tensor
    scales: torch.Tensor


def _scales_shape(shape):
    return (*shape[:-1], -(-shape[-1] // PACK8_GROUP))


def _check_packed(name, codes, scales, shape):
    _expect(f"{name}.codes", codes, shape, torch.int8)
    _expect(f"{name}.scales", scales, _scales_shape(shape), torch.uint8)


def _pack_plan(x, codes, scales):
    sizes, code = _norm_shape(x), _dtype_code(x)
    if codes is not None:
        _check_packed("out", codes, scales, x.shape)
    shape = _scales_shape(x.shape)
    return (shape, _st(x, 4), _dense(x.shape, 4) if codes is None else _st(codes, 4),
            _dense(shape, 4) if scales is None else _st(scales, 4), (*sizes, code))


def dynconv_pack8(x, out: Packed8 | None = None) -> Packed8:
    """x (1 to 4 dimensions) in 8 bits: per row, every 64 channels are integers of -127 to 127 times
    the power of two 2^(floor(log2 max|x|) - 6) that they share. Half the memory of 16-bit
    activations (a quarter of float32) for what a training step keeps for its backward pass."""
    codes, scales = (None, None) if out is None else out
    shape, xs, cs, ss, sizes = _plan(_pack_plan, (), x, codes, scales)
    dev = _require_device(x, codes, scales)
    if out is None:
        out = Packed8(x.new_empty(x.shape, dtype=torch.int8), x.new_empty(shape, dtype=torch.uint8))
        codes, scales = out
    _launch("dynconv_pack", dev, x.data_ptr(), xs, codes.data_ptr(), cs, scales.data_ptr(), ss, *sizes)
    return out


def _unpack_plan(dtype, codes, scales, out):
    sizes = _norm_shape(codes)
    _check_packed("packed", codes, scales, codes.shape)
    _expect("out", out, codes.shape, dtype)
    if dtype not in _DTYPE:
        raise TypeError(f"unsupported dtype {dtype}; use float32, bfloat16 or float16")
    return _st(codes, 4), _st(scales, 4), _dense(codes.shape, 4) if out is None else _st(out, 4), (*sizes, _DTYPE[dtype])


def dynconv_unpack8(packed: Packed8, dtype=torch.bfloat16, out=None):
    """The values that a Packed8 stands for, as `dtype` (exact in the type that was packed)."""
    codes, scales = packed
    cs, ss, ys, sizes = _plan(_unpack_plan, (dtype,), codes, scales, out)
    dev = _require_device(codes, scales, out)
    y = codes.new_empty(codes.shape, dtype=dtype) if out is None else out
    _launch("dynconv_unpack", dev, codes.data_ptr(), cs, scales.data_ptr(), ss, y.data_ptr(), ys, *sizes)
    return y


# ----------------------------------------------------------------------------------
# Gated linear scan
# ----------------------------------------------------------------------------------

SCAN_CHUNK = 128  # tokens between the states that dynconv_scan_fwd keeps for the backward


def new_scan_state(B: int, D: int, device) -> torch.Tensor:
    """A zeroed float32 [B, D] state of the gated linear scan."""
    return torch.zeros((B, D), dtype=torch.float32, device=device)


def _check_rate(rate, D: int):
    _expect("rate", rate, (D,), torch.float32)
    if rate is None:
        raise ValueError("a rate [D] is required")
    if D > 1 and rate.stride(0) != 1:
        raise ValueError("rate must be contiguous")


def _scan_shape(x, decay, gate, rate, n: int):
    names = "[B, D]" if n == 2 else "[B, T, D]"
    if x.dim() != n:
        raise ValueError(f"x must be {names}; got shape {list(x.shape)}")
    _dtype_code(x)
    if decay is None:
        raise ValueError(f"a decay {names} is required")
    _expect("decay", decay, x.shape, x.dtype)
    _expect("gate", gate, x.shape, x.dtype)
    _check_rate(rate, x.shape[-1])
    return tuple(x.shape)


def _chunks_shape(B: int, T: int, D: int):
    return (B, -(-T // SCAN_CHUNK), D)


def _scan_fwd_plan(x, decay, rate, gate, seq_idx, state, state_out, out):
    B, T, D = _scan_shape(x, decay, gate, rate, 3)
    _expect("state", state, (B, D), torch.float32)
    _expect("state_out", state_out, (B, D), torch.float32)
    _expect("out", out, (B, T, D), x.dtype)
    code = _dtype_code(x)
    return ((B, T, D), _chunks_shape(B, T, D), code, _workspace("dynconv_scan_fwd_workspace_size", B, T, D, code), _st(x),
            _st(decay), _st(gate), _seq_strides(seq_idx, B, T), _st(state), _dense((B, T, D)) if out is None else _st(out),
            _dense((B, D)) if state_out is None else _st(state_out))


def dynconv_scan_fwd(x, decay, rate, gate=None, seq_idx=None, state=None, want_state: bool = False,
                     want_chunks: bool = False, out=None, state_out=None):
    """y = h [B,T,D] of the gated linear scan of x [B,T,D]:

        a_t = exp(-rate sigmoid(decay_t)),  h_t = a_t h_{t-1} + sqrt(1 - a_t^2) sigmoid(gate_t) x_t

    with decay and gate (optional) of x's shape and a float32 rate [D] >= 0. With seq_idx (int32
    [B,T]) the state restarts from zero at every document start. state: the float32 [B,D] state before
    token 0 (default zero). Returns y; with want_state, or a state_out to write (which may be state
    itself), (y, state after token T-1); want_chunks adds, last, the float32 states before every 128th
    token that dynconv_scan_bwd would else recompute."""
    shape, kept, code, ws_bytes, xs, as_, gs, ss, sis, ys, sos = _plan(_scan_fwd_plan, (), x, decay, rate, gate, seq_idx,
                                                                       state, state_out, out)
    dev = _require_device(x, decay, gate, rate, seq_idx, state, out, state_out)
    y = x.new_empty(shape) if out is None else out
    if want_state and state_out is None:
        state_out = rate.new_empty((shape[0], shape[2]))
    chunks = rate.new_empty(kept) if want_chunks else None
    work = x.new_empty(ws_bytes, dtype=torch.uint8) if ws_bytes else None
    _launch("dynconv_scan_fwd", dev, x.data_ptr(), xs, decay.data_ptr(), as_, _dp(gate), gs, rate.data_ptr(), _dp(seq_idx),
            ss, _dp(state), sis, y.data_ptr(), ys, _dp(state_out), sos, _dp(chunks), *shape, code, _dp(work), ws_bytes)
    if state_out is None and chunks is None:
        return y
    return (y,) + ((state_out,) if state_out is not None else ()) + ((chunks,) if chunks is not None else ())


def _scan_bwd_plan(packed, x, x_scales, decay, decay_scales, gate, gate_scales, rate, dy, seq_idx, state, chunks, dstate_out):
    if dy.dim() != 3:
        raise ValueError(f"dy must be [B, T, D]; got shape {list(dy.shape)}")
    B, T, D = dy.shape
    code = _dtype_code(dy)
    if packed:
        _check_packed("x", x, x_scales, dy.shape)
        _check_packed("decay", decay, decay_scales, dy.shape)
        if gate is not None:
            _check_packed("gate", gate, gate_scales, dy.shape)
        _check_rate(rate, D)
        if chunks is not None:
            raise ValueError("chunks do not go with Packed8 inputs: they are the states of the unpacked ones")
    else:
        _scan_shape(x, decay, gate, rate, 3)
        _expect("dy", dy, x.shape, x.dtype)
    _expect("state", state, (B, D), torch.float32)
    _expect("dstate_out", dstate_out, (B, D), torch.float32)
    _expect("chunks", chunks, _chunks_shape(B, T, D), torch.float32)
    if chunks is not None and not chunks.is_contiguous():
        raise ValueError("chunks must be contiguous")
    ws_bytes = _workspace("dynconv_scan_bwd_workspace_size", B, T, D, int(chunks is not None), code)
    return ((B, T, D), code, ws_bytes, _st(x), _st(decay), _st(gate), _st(x_scales), _st(decay_scales), _st(gate_scales),
            _seq_strides(seq_idx, B, T), _st(state), _st(dy), _st(dstate_out), _dense((B, T, D)), _dense((B, D)))


def dynconv_scan_bwd(x, decay, rate, dy, gate=None, seq_idx=None, state=None, chunks=None, dstate_out=None,
                     need_dstate: bool = False):
    """(dx, ddecay, drate, dgate, dstate) of <dy, y> (+ <dstate_out, final state>) for dynconv_scan_fwd
    with the same arguments; drate and dstate (the gradient of `state`, None unless need_dstate) are
    float32, dgate None without a gate. chunks: what the forward returned with want_chunks; without, the states
    are recomputed. x, decay and gate may all be Packed8: the gradients are then those at the values
    that the codes stand for, and no chunks are taken."""
    packed = isinstance(x, Packed8)
    if packed != isinstance(decay, Packed8) or (gate is not None and packed != isinstance(gate, Packed8)):
        raise ValueError("x, decay and gate are all Packed8 or none is")
    (x, xc), (decay, ac) = (x, decay) if packed else ((x, None), (decay, None))
    gate, gc = gate if packed and gate is not None else (gate, None)
    shape, code, ws_bytes, xs, as_, gs, xcs, acs, gcs, ss, sis, dys, dsos, new, newst = _plan(
        _scan_bwd_plan, (packed,), x, xc, decay, ac, gate, gc, rate, dy, seq_idx, state, chunks, dstate_out)
    dev = _require_device(x, xc, decay, ac, gate, gc, rate, dy, seq_idx, state, chunks, dstate_out)
    dx, da, dgate = dy.new_empty(shape), dy.new_empty(shape), dy.new_empty(shape) if gate is not None else None
    drate = rate.new_empty(shape[2:])
    dstate = rate.new_empty((shape[0], shape[2])) if need_dstate else None
    work = dy.new_empty(ws_bytes, dtype=torch.uint8) if ws_bytes else None
    _launch("dynconv_scan_bwd", dev, x.data_ptr(), xs, decay.data_ptr(), as_, _dp(gate), gs, _dp(xc), xcs, _dp(ac), acs,
            _dp(gc), gcs, rate.data_ptr(), _dp(seq_idx), ss, _dp(state), sis, _dp(chunks), dy.data_ptr(), dys, _dp(dstate_out),
            dsos, dx.data_ptr(), new, da.data_ptr(), new, drate.data_ptr(), _dp(dgate), new, _dp(dstate), newst, *shape, code,
            _dp(work), ws_bytes)
    return dx, da, drate, dgate, dstate


def _scan_step_plan(x, decay, rate, state, gate, out):
    B, D = _scan_shape(x, decay, gate, rate, 2)
    if state is None:
        raise ValueError("a state [B, D] is required")
    _expect("state", state, (B, D), torch.float32)
    _expect("out", out, (B, D), x.dtype)
    return _st(x), _st(decay), _st(gate), _st(state), _dense((B, D)) if out is None else _st(out), (B, D, _dtype_code(x))


def dynconv_scan_step(x, decay, rate, state, gate=None, out=None):
    """y [B,D] of one token of every sequence (x, decay, gate [B,D], float32 rate [D]); state (float32
    [B,D]) is updated in place."""
    xs, as_, gs, sts, ys, sizes = _plan(_scan_step_plan, (), x, decay, rate, state, gate, out)
    dev = _require_device(x, decay, gate, rate, state, out)
    y = x.new_empty(x.shape) if out is None else out
    _launch("dynconv_scan_step", dev, x.data_ptr(), xs, decay.data_ptr(), as_, _dp(gate), gs, rate.data_ptr(),
            state.data_ptr(), sts, y.data_ptr(), ys, *sizes)
    return y


# ----------------------------------------------------------------------------------
# Group norm, channels last
# ----------------------------------------------------------------------------------


def _group_args(shape, dtype, groups, weight, bias, gate, activation, over, lengths, stats):
    """Checks what both directions share; returns ((B, T, C), over sequences, SiLU)."""
    if over not in ("token", "sequence"):
        raise ValueError(f"over is 'token' or 'sequence'; got {over!r}")
    sequence = over == "sequence"
    if len(shape) != 3 and (sequence or len(shape) != 2):
        raise ValueError(f"x must be [B, T, C]{'' if sequence else ' or [tokens, C]'}; got shape {list(shape)}")
    if activation not in (None, "silu"):
        raise ValueError(f"activation is 'silu' or None; got {activation!r}")
    B, T, C = (1,) * (3 - len(shape)) + tuple(shape)
    if groups < 1 or C % groups != 0:
        raise ValueError(f"groups = {groups} must be a positive divisor of C = {C}")
    for name, t in (("weight", weight), ("bias", bias)):
        _expect(name, t, (C,), dtype)
        if t is not None and C > 1 and t.stride(0) != 1:
            raise ValueError(f"{name} must be contiguous")
    _expect("gate", gate, shape, dtype)
    if not sequence and (lengths is not None or stats is not None):
        raise ValueError("lengths and stats go with over='sequence'")
    _expect("lengths", lengths, (B,), torch.int32)
    _expect("stats", stats, (B, groups, 2), torch.float32)
    for name, t in (("lengths", lengths), ("stats", stats)):
        if t is not None and not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
    return (B, T, C), int(sequence), int(activation == "silu")


def _group_fwd_plan(groups, activation, over, eps, want_stats, x, weight, bias, gate, lengths, out):
    code = _dtype_code(x)
    (B, T, C), seq, silu = _group_args(x.shape, x.dtype, groups, weight, bias, gate, activation, over, lengths, None)
    _expect("out", out, x.shape, x.dtype)
    ws_bytes = _workspace("dynconv_groupnorm_fwd_workspace_size", B, T, C, groups, seq, int(want_stats), code)
    return ((B, groups, 2) if want_stats and seq else None, ws_bytes, _st(x, 3), _st(gate, 3),
            _dense(x.shape, 3) if out is None else _st(out, 3), (B, T, C, groups, seq, silu, float(eps), code))


def dynconv_groupnorm_fwd(x, groups: int, weight=None, bias=None, gate=None, activation: str | None = None,
                          over: str = "token", lengths=None, eps: float = 1e-5, want_stats: bool = False, out=None):
    """y = act(n * weight + bias) * silu(gate) with n = (x - mean) / sqrt(var + eps) over the C / groups
    neighbouring channels of each group of x [B,T,C] (or [tokens,C]): of each token (over="token"), or of all
    tokens of a sequence (over="sequence"). weight, bias [C] and gate (x's shape) are optional; act is
    SiLU with activation="silu", else nothing. Over sequences, lengths (int32 [B], 0 to T) says how many tokens
    of each count; y is 0 behind them. With want_stats returns (y, stats) for dynconv_groupnorm_bwd: float32
    [B,groups,2] over sequences, None per token (there the backward has the group in registers)."""
    kept, ws_bytes, xs, gs, ys, sizes = _plan(_group_fwd_plan, (groups, activation, over, eps, want_stats), x, weight, bias,
                                              gate, lengths, out)
    dev = _require_device(x, weight, bias, gate, lengths, out)
    y = x.new_empty(x.shape) if out is None else out
    stats = torch.empty(kept, dtype=torch.float32, device=dev) if kept is not None else None
    work = x.new_empty(ws_bytes, dtype=torch.uint8) if ws_bytes else None
    _launch("dynconv_groupnorm_fwd", dev, x.data_ptr(), xs, _dp(weight), _dp(bias), _dp(gate), gs, _dp(lengths), y.data_ptr(),
            ys, _dp(stats), *sizes, _dp(work), ws_bytes)
    return (y, stats) if want_stats else y


def _group_bwd_plan(groups, activation, over, eps, x, scales, dy, weight, bias, gate, lengths, stats):
    code = _dtype_code(dy)
    if scales is not None:
        _check_packed("x", x, scales, dy.shape)
        if stats is not None:
            raise ValueError("stats do not go with a Packed8 x: they are those of the unpacked one")
    else:
        _expect("x", x, dy.shape, dy.dtype)
    (B, T, C), seq, silu = _group_args(dy.shape, dy.dtype, groups, weight, bias, gate, activation, over, lengths, stats)
    ws_bytes = 0
    if seq or weight is not None or bias is not None:
        ws_bytes = _workspace("dynconv_groupnorm_bwd_workspace_size", B, T, C, groups, seq, int(stats is not None), code)
    return ((C,), ws_bytes, _st(x, 3), _st(scales, 3), _st(gate, 3), _st(dy, 3), _dense(dy.shape, 3),
            (B, T, C, groups, seq, silu, float(eps), code))


def dynconv_groupnorm_bwd(x, groups: int, dy, weight=None, bias=None, gate=None, activation: str | None = None,
                          over: str = "token", lengths=None, eps: float = 1e-5, stats=None):
    """(dx, dweight, dbias, dgate) of <dy, y> for dynconv_groupnorm_fwd with the same arguments, None where
    there is no such input; dweight and dbias are float32 [C]. x may be a Packed8 of what the forward took:
    the gradients are then those at the values it stands for, and no stats are taken. stats: what the forward
    returned with want_stats; recomputed without."""
    x, scales = x if isinstance(x, Packed8) else (x, None)
    column, ws_bytes, xs, xcs, gs, dys, new, sizes = _plan(_group_bwd_plan, (groups, activation, over, eps), x, scales, dy,
                                                           weight, bias, gate, lengths, stats)
    dev = _require_device(x, scales, dy, weight, bias, gate, lengths, stats)
    dx, dgate = dy.new_empty(dy.shape), dy.new_empty(dy.shape) if gate is not None else None
    dw, db = (None if t is None else dy.new_empty(column, dtype=torch.float32) for t in (weight, bias))
    work = dy.new_empty(ws_bytes, dtype=torch.uint8) if ws_bytes else None
    _launch("dynconv_groupnorm_bwd", dev, x.data_ptr(), xs, _dp(scales), xcs, _dp(weight), _dp(bias), _dp(gate), gs, _dp(lengths),
            _dp(stats), dy.data_ptr(), dys, dx.data_ptr(), new, _dp(dw), _dp(db), _dp(dgate), new, *sizes, _dp(work), ws_bytes)
    return dx, dw, db, dgate
