"""PyTorch-facing wrappers of the decoder-layer operators: the residual
addition with its RMS norm or layer norm (and gradients), the products with 4-bit and
8-bit weights, the linear layer with an adapter per row, and the
mixture-of-experts FFN of a few tokens.  Shape, type and stride checks, output allocation and the
current stream; every step of the computation runs in the HIP kernels.
"""
from __future__ import annotations

import math
from typing import Optional

import torch

from . import binding

_STREAM = {torch.bfloat16: 0, torch.float32: 1}
_BF16, _F32, _U8, _I32, _E4M3 = torch.bfloat16, torch.float32, torch.uint8, torch.int32, torch.float8_e4m3fn


# The checks run on every call, ahead of kernels of a few microseconds: they
# use what is cheap to ask of a tensor (its device's index, not the device).
def _check(t: torch.Tensor, name: str, dtype: torch.dtype, shape: tuple, index: int) -> None:
    if t.dtype is dtype and t.shape == shape and t.get_device() == index and t.is_contiguous():
        return
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {list(shape)} tensor, got {list(t.shape)}")
    raise ValueError(f"{name} must be on cuda:{index}, got {t.device}")


def _operand(t: torch.Tensor, name: str, dtypes: tuple) -> int:
    """The device index of the operand that sets the others' sizes."""
    if t.dtype not in dtypes:
        raise TypeError(f"{name} must be {' or '.join(str(d) for d in dtypes)}, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be on a GPU, got {t.device}")
    if t.dim() != 2:
        raise ValueError(f"{name} must be 2-D, got shape {tuple(t.shape)}")
    return t.get_device()


def _stream(index: int) -> int:
    # (kernels are launched on the current device)
    if index != torch._C._cuda_getDevice():
        raise ValueError(f"the operands are on cuda:{index}, the current device is cuda:{torch.cuda.current_device()}")
    return torch._C._cuda_getCurrentRawStream(index)


def _rows(x: torch.Tensor, name: str) -> int:
    """Row stride of a 2-D tensor whose rows are contiguous and apart."""
    rows, hidden = x.shape
    if x.is_contiguous():
        return hidden
    if rows <= 1 or hidden == 0:
        ld = hidden
    else:
        ld = x.stride(0)
    if (hidden > 1 and x.stride(1) != 1) or ld < hidden:
        raise ValueError(f"{name} must have contiguous rows that do not overlap")
    return ld


def _norm(fn, x, weight, residual, eps, h, out_dtype):
    index = _operand(x, "x", (_BF16, _F32))
    rows, hidden = x.shape
    ld = _rows(x, "x")
    dtype = x.dtype
    _check(weight, "weight", _BF16, (hidden,), index)
    if residual is None:
        if h is not None:
            raise ValueError("h is written only with a residual")
        h_out, rp, hp = x, None, None
    else:
        _check(residual, "residual", dtype, (rows, hidden), index)
        if h is None:
            h = torch.empty_like(residual)
        else:
            _check(h, "h", dtype, (rows, hidden), index)
        h_out, rp, hp = h, residual.data_ptr(), h.data_ptr()
    stream = _stream(index)
    y = torch.empty(rows, hidden, dtype=out_dtype, device=x.device)
    stat = torch.empty(rows, dtype=_F32, device=x.device)
    st = fn(x.data_ptr(), ld, rp, weight.data_ptr(), hp, y.data_ptr(), stat.data_ptr(), rows, hidden, eps,
            _STREAM[dtype], stream)
    if st:
        binding.check(st, fn.__name__)
    if not hidden:  # (no launch: the mean of no values is 0, and so is their largest)
        stat.fill_(2.0 ** -126 if out_dtype is _E4M3 else eps ** -0.5 if eps else math.inf)
    return y, stat, h_out


def rms_norm(x: torch.Tensor, weight: torch.Tensor, residual: Optional[torch.Tensor] = None,
             eps: float = 1e-6, h: Optional[torch.Tensor] = None):
    """Residual addition and RMS norm of the rows of x [rows, hidden]:
    h = x + residual in x's type (bf16 or fp32; h is x without a residual),
    rstd = 1 / sqrt(mean(h^2) + eps), y = h * rstd * weight in bf16.
    Returns (y, h, rstd).  x may have a row stride; `h` may name the tensor
    to write the sum to, residual itself or x among them.  Rows of no values
    have rstd 1 / sqrt(eps)."""
    y, rstd, h = _norm(binding.load().mm_rms_norm, x, weight, residual, eps, h, _BF16)
    return y, h, rstd


def rms_norm_q8(x: torch.Tensor, weight: torch.Tensor, residual: Optional[torch.Tensor] = None,
                eps: float = 1e-6, h: Optional[torch.Tensor] = None):
    """rms_norm with an 8-bit output, the activations linear_q8 takes: returns
    (q, scale, h) with q e4m3 [rows, hidden] and scale fp32 [rows]; q stands
    for q * scale[:, None], scale = max(max|y| / 448, 2^-126) of each row (2^-126
    for rows of no values)."""
    return _norm(binding.load().mm_rms_norm_q8, x, weight, residual, eps, h, _E4M3)


def rms_norm_backward(dy: torch.Tensor, h: torch.Tensor, weight: torch.Tensor, rstd: torch.Tensor,
                      dres: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None):
    """Gradient of rms_norm, from what it returned: dy bf16 [rows, hidden] is
    the gradient of y, dres (h's type) the gradient that reached h past the
    norm.  Returns (dh, dweight): dh in h's type is the gradient of x and of
    residual, dweight [hidden] is fp32.  `out` may name the tensor for dh,
    dres itself among them."""
    index = _operand(h, "h", (_BF16, _F32))
    rows, hidden = shape = h.shape
    dtype = h.dtype
    _check(h, "h", dtype, shape, index)
    _check(dy, "dy", _BF16, shape, index)
    _check(weight, "weight", _BF16, (hidden,), index)
    _check(rstd, "rstd", _F32, (rows,), index)
    if dres is not None:
        _check(dres, "dres", dtype, shape, index)
    if out is None:
        out = torch.empty_like(h)
    else:
        _check(out, "out", dtype, shape, index)
    stream = _stream(index)
    dweight = torch.empty(hidden, dtype=_F32, device=h.device)
    nbytes = binding.rms_norm_backward_workspace_size(rows, hidden)
    ws = torch.empty(nbytes, dtype=_U8, device=h.device) if nbytes else None
    st = binding.load().mm_rms_norm_backward(
        dy.data_ptr(), h.data_ptr(), weight.data_ptr(), rstd.data_ptr(),
        None if dres is None else dres.data_ptr(), out.data_ptr(), dweight.data_ptr(), rows, hidden,
        _STREAM[dtype], None if ws is None else ws.data_ptr(), nbytes, stream)
    if st:
        binding.check(st, "mm_rms_norm_backward")
    return out, dweight


def _product(x, M, N, bias, epilogue, out, index):
    epi = binding.EPILOGUES.get(epilogue)
    if epi is None:
        raise ValueError(f"unknown epilogue {epilogue!r}")
    bp = None
    if epi & 1:  # bias, bias_gelu_tanh
        if bias is None:
            raise ValueError(f"epilogue {epilogue!r} needs a bias")
        _check(bias, "bias", _BF16, (N,), index)
        bp = bias.data_ptr()
    if out is None:
        out = torch.empty(M, N, dtype=_BF16, device=x.device)
    else:
        _check(out, "out", _BF16, (M, N), index)
    return epi, bp, out


def pack_w4(codes: torch.Tensor) -> torch.Tensor:
    """Packs 4-bit codes (uint8 [N, K], values 0..15) into the layout linear_w4
    reads: uint8 [ceil(N/16), ceil(K/128), 1024] (see mm_linear_w4 in mm.h)."""
    index = _operand(codes, "codes", (_U8,))
    N, K = codes.shape
    _check(codes, "codes", _U8, (N, K), index)
    stream = _stream(index)
    packed = torch.empty((-(-N // 16), -(-K // 128), 1024), dtype=_U8, device=codes.device)
    st = binding.load().mm_w4_pack(codes.data_ptr(), packed.data_ptr(), N, K, stream)
    if st:
        binding.check(st, "mm_w4_pack")
    return packed


def linear_w4(x: torch.Tensor, W: torch.Tensor, scales: torch.Tensor, zeros: Optional[torch.Tensor] = None,
              bias: Optional[torch.Tensor] = None, epilogue: str = "none", group: int = 128,
              out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """out = epi(x @ Wd.T + bias) with x bf16 [M, K] and a 4-bit weight
    Wd[n, k] = (code[n, k] - zeros[k // group, n]) * scales[k // group, n]:
    W the codes as pack_w4 lays them out, scales bf16 [ceil(K / group), N],
    zeros uint8 of the same shape (8 everywhere when absent), group 32, 64 or
    128.  Epilogues and bias as for linear; bf16 output."""
    index = _operand(x, "x", (_BF16,))
    M, K = x.shape
    if not x.is_contiguous():
        raise ValueError("x must be contiguous")
    if group not in (32, 64, 128):
        raise ValueError(f"group must be 32, 64 or 128, got {group}")
    if scales.dim() != 2:
        raise ValueError(f"scales must be 2-D, got shape {tuple(scales.shape)}")
    N = scales.shape[1]
    groups = -(-K // group)
    _check(scales, "scales", _BF16, (groups, N), index)
    _check(W, "W", _U8, (-(-N // 16), -(-K // 128), 1024), index)
    zp = None
    if zeros is not None:
        _check(zeros, "zeros", _U8, (groups, N), index)
        zp = zeros.data_ptr()
    stream = _stream(index)
    epi, bp, out = _product(x, M, N, bias, epilogue, out, index)
    st = binding.load().mm_linear_w4(x.data_ptr(), W.data_ptr(), scales.data_ptr(), zp, bp, out.data_ptr(), M, N, K,
                                     group, epi, stream)
    if st:
        binding.check(st, "mm_linear_w4")
    return out


def linear_q8(x: torch.Tensor, x_scale: torch.Tensor, W: torch.Tensor, w_scale: torch.Tensor,
              bias: Optional[torch.Tensor] = None, epilogue: str = "none",
              out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """out = epi(x_scale[:, None] * w_scale * (x @ W.T) + bias) with e4m3 x
    [M, K] and W [N, K] (K a multiple of 16) and fp32 row scales x_scale [M],
    w_scale [N]; bf16 output, sums as mm_linear_q8 in mm.h says.  Epilogues and
    bias as for linear."""
    index = _operand(x, "x", (_E4M3,))
    M, K = x.shape
    if not x.is_contiguous():
        raise ValueError("x must be contiguous")
    if W.dim() != 2:
        raise ValueError(f"W must be 2-D, got shape {tuple(W.shape)}")
    N = W.shape[0]
    _check(W, "W", _E4M3, (N, K), index)
    _check(x_scale, "x_scale", _F32, (M,), index)
    _check(w_scale, "w_scale", _F32, (N,), index)
    stream = _stream(index)
    epi, bp, out = _product(x, M, N, bias, epilogue, out, index)
    ws = wp = None
    nbytes = 0
    if M > 64:  # (decode rows never use one)
        nbytes = binding.linear_q8_workspace_size(M, N, K)
        if nbytes:
            ws = torch.empty(nbytes, dtype=_U8, device=x.device)
            wp = ws.data_ptr()
    st = binding.load().mm_linear_q8(x.data_ptr(), x_scale.data_ptr(), W.data_ptr(), w_scale.data_ptr(), bp,
                                     out.data_ptr(), M, N, K, epi, wp, nbytes, stream)
    if st:
        binding.check(st, "mm_linear_q8")
    return out


def layer_norm(x: torch.Tensor, weight: torch.Tensor, bias: Optional[torch.Tensor] = None,
               residual: Optional[torch.Tensor] = None, eps: float = 1e-5, h: Optional[torch.Tensor] = None):
    """Residual addition and layer norm of the rows of x [rows, hidden]:
    h = x + residual in x's type (bf16 or fp32; h is x without a residual),
    mean = mean(h), rstd = 1 / sqrt(mean((h - mean)^2) + eps), y = (h - mean) *
    rstd * weight + bias in bf16.  Returns (y, h, mean, rstd).  x may have a row
    stride; `h` may name the tensor to write the sum to, residual itself or x
    among them.  Rows of no values have mean 0 and rstd 1 / sqrt(eps)."""
    index = _operand(x, "x", (_BF16, _F32))
    rows, hidden = x.shape
    ld = _rows(x, "x")
    dtype = x.dtype
    _check(weight, "weight", _BF16, (hidden,), index)
    if bias is not None:
        _check(bias, "bias", _BF16, (hidden,), index)
    if residual is None:
        if h is not None:
            raise ValueError("h is written only with a residual")
        h_out, rp, hp = x, None, None
    else:
        _check(residual, "residual", dtype, (rows, hidden), index)
        if h is None:
            h = torch.empty_like(residual)
        else:
            _check(h, "h", dtype, (rows, hidden), index)
        h_out, rp, hp = h, residual.data_ptr(), h.data_ptr()
    stream = _stream(index)
    y = torch.empty(rows, hidden, dtype=_BF16, device=x.device)
    mean, rstd = torch.empty(2, rows, dtype=_F32, device=x.device)
    st = binding.load().mm_layer_norm(
        x.data_ptr(), ld, rp, weight.data_ptr(), None if bias is None else bias.data_ptr(), hp, y.data_ptr(),
        mean.data_ptr(), rstd.data_ptr(), rows, hidden, eps, _STREAM[dtype], stream)
    if st:
        binding.check(st, "mm_layer_norm")
    if not hidden:  # (no launch: the mean of no values is 0)
        mean.zero_()
        rstd.fill_(eps ** -0.5 if eps else math.inf)
    return y, h_out, mean, rstd


def layer_norm_backward(dy: torch.Tensor, h: torch.Tensor, weight: torch.Tensor, mean: torch.Tensor,
                        rstd: torch.Tensor, dres: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None):
    """Gradient of layer_norm, from what it returned: dy bf16 [rows, hidden] is
    the gradient of y, dres (h's type) the gradient that reached h past the
    norm.  Returns (dh, dweight, dbias): dh in h's type is the gradient of x and
    of residual, dweight and dbias [hidden] are fp32.  `out` may name the tensor
    for dh, dres itself among them."""
    index = _operand(h, "h", (_BF16, _F32))
    rows, hidden = shape = h.shape
    dtype = h.dtype
    _check(h, "h", dtype, shape, index)
    _check(dy, "dy", _BF16, shape, index)
    _check(weight, "weight", _BF16, (hidden,), index)
    _check(mean, "mean", _F32, (rows,), index)
    _check(rstd, "rstd", _F32, (rows,), index)
    if dres is not None:
        _check(dres, "dres", dtype, shape, index)
    if out is None:
        out = torch.empty_like(h)
    else:
        _check(out, "out", dtype, shape, index)
    stream = _stream(index)
    dweight = torch.empty(hidden, dtype=_F32, device=h.device)
    dbias = torch.empty(hidden, dtype=_F32, device=h.device)
    nbytes = binding.layer_norm_backward_workspace_size(rows, hidden)
    ws = torch.empty(nbytes, dtype=_U8, device=h.device) if nbytes else None
    st = binding.load().mm_layer_norm_backward(
        dy.data_ptr(), h.data_ptr(), weight.data_ptr(), mean.data_ptr(), rstd.data_ptr(),
        None if dres is None else dres.data_ptr(), out.data_ptr(), dweight.data_ptr(), dbias.data_ptr(), rows, hidden,
        _STREAM[dtype], None if ws is None else ws.data_ptr(), nbytes, stream)
    if st:
        binding.check(st, "mm_layer_norm_backward")
    return out, dweight, dbias


def linear_lora(x: torch.Tensor, W: torch.Tensor, A: torch.Tensor, B: torch.Tensor, index: torch.Tensor,
                scale: torch.Tensor, bias: Optional[torch.Tensor] = None, epilogue: str = "none",
                out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Linear layer of many requests at once, each row with a low-rank adapter:
    out[m] = epi(x[m] @ W.T + bias + scale[a] * (x[m] @ A[a].T) @ B[a].T) with
    a = index[m]; a row whose index names no adapter (-1) goes without one.
    x [M, K], W [N, K], A [adapters, rank, K] and B [adapters, N, rank] bf16,
    index int32 [M], scale fp32 [adapters]; K and rank multiples of 8, rank at
    most 256.  Epilogues and bias as for linear; bf16 output."""
    dev = _operand(x, "x", (_BF16,))
    M, K = x.shape
    if not x.is_contiguous():
        raise ValueError("x must be contiguous")
    if W.dim() != 2:
        raise ValueError(f"W must be 2-D, got shape {tuple(W.shape)}")
    if A.dim() != 3:
        raise ValueError(f"A must be 3-D, got shape {tuple(A.shape)}")
    N = W.shape[0]
    adapters, rank, _ = A.shape
    _check(W, "W", _BF16, (N, K), dev)
    _check(A, "A", _BF16, (adapters, rank, K), dev)
    _check(B, "B", _BF16, (adapters, N, rank), dev)
    _check(index, "index", _I32, (M,), dev)
    _check(scale, "scale", _F32, (adapters,), dev)
    stream = _stream(dev)
    epi, bp, out = _product(x, M, N, bias, epilogue, out, dev)
    nbytes = binding.linear_lora_workspace_size(M, N, K, rank, adapters)
    ws = torch.empty(nbytes, dtype=_U8, device=x.device) if nbytes else None
    st = binding.load().mm_linear_lora(
        x.data_ptr(), W.data_ptr(), A.data_ptr(), B.data_ptr(), index.data_ptr(), scale.data_ptr(), bp, out.data_ptr(),
        M, N, K, rank, adapters, epi, None if ws is None else ws.data_ptr(), nbytes, stream)
    if st:
        binding.check(st, "mm_linear_lora")
    return out


def moe_ffn(x: torch.Tensor, logits: torch.Tensor, W_gate: torch.Tensor, W_up: torch.Tensor, W_down: torch.Tensor,
            top_k: int, renormalize: bool = True, out: Optional[torch.Tensor] = None):
    """Mixture-of-experts form of ffn_swiglu with its second layer, for a few
    tokens (at most 64): out[t] = sum over j of weights[t, j] * W_down[e] @
    (SiLU(W_gate[e] @ x[t]) * (W_up[e] @ x[t])), e = experts[t, j] being the
    top_k largest logits of the token, in descending order (of equal ones the
    lower index first), and weights their softmax (renormalize), or their part
    of the softmax over all.  x bf16 [tokens, H], logits fp32 [tokens, experts],
    W_gate and W_up bf16 [experts, I, H], W_down bf16 [experts, H, I].  Returns
    (out, experts, weights): bf16 [tokens, H], int32 and fp32 [tokens, top_k].
    Logits of -inf take no part: slots left without an expert hold -1 and weight
    0, and a token without any (a padded row) gets zeros."""
    index = _operand(x, "x", (_BF16,))
    T, H = x.shape
    if not x.is_contiguous():
        raise ValueError("x must be contiguous")
    if W_gate.dim() != 3:
        raise ValueError(f"W_gate must be 3-D, got shape {tuple(W_gate.shape)}")
    E, I, _ = W_gate.shape
    _check(logits, "logits", _F32, (T, E), index)
    _check(W_gate, "W_gate", _BF16, (E, I, H), index)
    _check(W_up, "W_up", _BF16, (E, I, H), index)
    _check(W_down, "W_down", _BF16, (E, H, I), index)
    if out is not None:
        _check(out, "out", _BF16, (T, H), index)
    stream = _stream(index)
    nbytes = binding.moe_ffn_workspace_size(T, E, H, I, top_k)
    if out is None:
        out = torch.empty(T, H, dtype=_BF16, device=x.device)
    experts = torch.empty(T, top_k, dtype=_I32, device=x.device)
    weights = torch.empty(T, top_k, dtype=_F32, device=x.device)
    ws = torch.empty(nbytes, dtype=_U8, device=x.device) if nbytes else None
    st = binding.load().mm_moe_ffn(
        x.data_ptr(), logits.data_ptr(), W_gate.data_ptr(), W_up.data_ptr(), W_down.data_ptr(), out.data_ptr(),
        experts.data_ptr(), weights.data_ptr(), T, E, H, I, top_k, int(renormalize),
        None if ws is None else ws.data_ptr(), nbytes, stream)
    if st:
        binding.check(st, "mm_moe_ffn")
    return out, experts, weights
