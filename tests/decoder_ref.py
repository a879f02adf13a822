"""The decoder-layer operators from their definitions, in 64 bits on the CPU,
and the layout of packed 4-bit weights.  Used by the tests only."""
import math

import torch

E4M3_MAX = 448.0
TINY = 2.0 ** -126


def norm(x, weight, residual, eps):
    """(h as stored, rstd, y before rounding); h and y in 64 bits."""
    h = x if residual is None else (x.float() + residual.float()).to(x.dtype)
    h = h.double()
    rstd = 1.0 / torch.sqrt((h * h).mean(1) + eps)
    return h, rstd, h * rstd[:, None] * weight.double()


def norm_loss(x, weight, residual, eps, cy, ch):
    """sum(cy y) + sum(ch h) in 64 bits, without the stream's rounding."""
    h = x + residual
    y = h / torch.sqrt((h * h).mean(1, keepdim=True) + eps) * weight
    return (cy * y).sum() + (ch * h).sum()


def norm_grad(dy, h, weight, rstd, dres):
    dy, h, w, r = dy.double(), h.double(), weight.double(), rstd.double()[:, None]
    g, n = dy * w, h * r
    dh = r * (g - n * (g * n).mean(1, keepdim=True))
    if dres is not None:
        dh = dh + dres.double()
    return dh, (dy * n).sum(0)


def pack(codes):
    """Packed bytes of codes [N, K], word by word from the layout's definition."""
    N, K = codes.shape
    nb, kb = -(-N // 16), -(-K // 128)
    full = torch.zeros((nb * 16, kb * 128), dtype=torch.int64)
    full[:N, :K] = codes.long() & 15
    out = torch.zeros((nb, kb, 256), dtype=torch.int64)
    for g in range(4):
        for j in range(4):
            for e in range(8):
                k = 32 * j + 8 * g + e
                shift = 4 * (e // 2 + 4 * (e % 2))
                vals = full.view(nb, 16, kb, 128)[:, :, :, k].permute(0, 2, 1)  # [nb, kb, 16]
                out[:, :, [(16 * g + n) * 4 + j for n in range(16)]] |= vals << shift
    b = torch.stack([(out >> (8 * i)) & 255 for i in range(4)], dim=-1)
    return b.reshape(nb, kb, 1024).to(torch.uint8)


def w4_weight(codes, scales, zeros, group):
    N, K = codes.shape
    at = torch.arange(K) // group
    z = 8.0 if zeros is None else zeros.t().double()[:, at]
    return (codes.double() - z) * scales.t().double()[:, at]


def gelu(t):
    return 0.5 * t * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (t + 0.044715 * t ** 3)))


def epilogue(t, bias, kind):
    if "bias" in kind:
        t = t + bias.double()
    return (gelu(t) if "gelu" in kind else t), t
