"""Layer norm, the linear layer with adapters and the mixture-of-experts FFN from
their definitions, in 64 bits on the inputs' device.  Used by the tests only."""
import math

import torch

from decoder_ref import epilogue  # noqa: F401 (the linear layers')


def norm(x, weight, bias, residual, eps):
    """(h as stored, mean, rstd, y before rounding), in 64 bits."""
    h = x if residual is None else (x.float() + residual.float()).to(x.dtype)
    h = h.double()
    mean = h.mean(1)
    d = h - mean[:, None]
    rstd = 1.0 / torch.sqrt((d * d).mean(1) + eps)
    y = d * rstd[:, None] * weight.double()
    return h, mean, rstd, y if bias is None else y + bias.double()


def norm_loss(x, weight, bias, residual, eps, cy, ch):
    """sum(cy y) + sum(ch h) in 64 bits, without the stream's rounding."""
    h = x + residual
    d = h - h.mean(1, keepdim=True)
    y = d / torch.sqrt((d * d).mean(1, keepdim=True) + eps) * weight + bias
    return (cy * y).sum() + (ch * h).sum()


def norm_grad(dy, h, weight, mean, rstd, dres):
    dy, w, r = dy.double(), weight.double(), rstd.double()[:, None]
    n = (h.double() - mean.double()[:, None]) * r
    g = dy * w
    dh = r * (g - g.mean(1, keepdim=True) - n * (g * n).mean(1, keepdim=True))
    if dres is not None:
        dh = dh + dres.double()
    return dh, (dy * n).sum(0), dy.sum(0)


def lora(x, W, A, B, index, scale):
    """The sums before bias and epilogue."""
    y = x.double() @ W.double().t()
    for m, a in enumerate(index.tolist()):
        if 0 <= a < A.shape[0]:
            y[m] += scale[a].double() * (B[a].double() @ (A[a].double() @ x[m].double()))
    return y


def route(logits, top_k, renormalize):
    """experts (int32) and weights (64 bits) [T, top_k] of logits on the CPU."""
    T, E = logits.shape
    experts = torch.full((T, top_k), -1, dtype=torch.int32)
    weights = torch.zeros((T, top_k), dtype=torch.float64)
    for t, row in enumerate(logits.double().tolist()):
        # NaN first, then descending, equal ones by index
        order = sorted((e for e in range(E) if row[e] != -math.inf),
                       key=lambda e: (0, 0.0, e) if math.isnan(row[e]) else (1, -row[e], e))
        chosen = order[:top_k]
        if not chosen:
            continue
        v = torch.tensor([row[e] for e in (chosen if renormalize else order)], dtype=torch.float64)
        p = torch.exp(v - v[0])
        p = p / p.sum()
        experts[t, :len(chosen)] = torch.tensor(chosen, dtype=torch.int32)
        weights[t, :len(chosen)] = p[:len(chosen)]
    return experts, weights


def moe(x, experts, weights, W_gate, W_up, W_down):
    """(out, size): the sums, and the same with the magnitudes of every term."""
    T, H = x.shape
    out = torch.zeros((T, H), dtype=torch.float64, device=x.device)
    size = torch.zeros_like(out)
    xd = x.double()
    for e in sorted(set(experts.flatten().tolist()) - {-1}):
        at = (experts == e).nonzero()
        rows, w = at[:, 0].to(x.device), weights[at[:, 0], at[:, 1]].to(x.device)[:, None]
        g = xd[rows] @ W_gate[e].double().t().contiguous()
        u = xd[rows] @ W_up[e].double().t().contiguous()
        h = g / (1.0 + torch.exp(-g)) * u * w
        down = W_down[e].double().t().contiguous()
        out.index_add_(0, rows, h @ down)
        # |SiLU'| < 1.1: what an error of g or u is worth, and h itself
        gs = xd[rows].abs() @ W_gate[e].double().abs().t().contiguous()
        us = xd[rows].abs() @ W_up[e].double().abs().t().contiguous()
        hs = (1.1 * gs * u.abs() + g.abs() * us) * w + h.abs()
        size.index_add_(0, rows, hs @ down.abs())
    return out, size
