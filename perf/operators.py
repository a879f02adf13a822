"""Cases of the quantised decoder operators: the residual addition with its
root-mean-square norm (bf16 or e4m3 output, and the gradient), the product
with 4-bit group-scaled weights, and the product of e4m3 operands with row
scales.

``own`` selects what run() calls: False computes the operators from elementary
torch operations, True calls dense_bf16_gemm_amd.  Inputs come from the seed
alone and are the same for both.

Packed 4-bit weights: W [N, K] holds whole numbers 0..15 and stands for
(W - zero) * scale.  It is stored as uint8 [ceil(N/16), ceil(K/128), 1024]:
a kilobyte covers 16 rows by 128 k, 32-bit word (g, n, j) of it (g = 0..3,
n = 0..15, j = 0..3, in that order) covers row n, k = 32 j + 8 g .. + 7, with
k + 2p in its nibble p and k + 2p + 1 in its nibble p + 4 (p = 0..3).  What
pads N and K is never read as a weight.  scales [ceil(K/group), N] are bf16,
zeros [ceil(K/group), N] uint8 (absent: 8 everywhere).
"""
import math

import torch

own = False

EPS = 1e-6
E4M3_MAX = 448.0
TINY = 2.0 ** -126  # smallest scale of a quantised row
NIBBLE_SHIFTS = (0, 16, 4, 20, 8, 24, 12, 28)  # of k = 0..7 in a packed word


def listed():
    return [
        # the smallest call: one new token's residual stream ahead of an 8-bit product
        dict(name="norm_q8_token", op="norm_q8", rows=1, hidden=8192, stream="bf16", residual=True),
        # a prompt of 4096 tokens ahead of an 8-bit product
        dict(name="norm_q8_prompt", op="norm_q8", rows=4096, hidden=8192, stream="bf16", residual=True),
        # training forward, fp32 residual stream, a ragged batch and width
        dict(name="norm_train_f32", op="norm", rows=2047, hidden=5000, stream="f32", residual=True),
        # its gradient at a training batch's size, bf16 stream, with the residual path's gradient
        dict(name="norm_backward", op="norm_backward", rows=8192, hidden=4096, stream="bf16", residual=True),
        # one token through a square projection in 4 bits: latency counts
        dict(name="w4_token", op="w4", M=1, N=4096, K=4096, group=128, zeros=False, epilogue="none"),
        # the decode step of a batch of 16 (bench.py's decode shape), asymmetric weights
        dict(name="w4_decode_16", op="w4", M=16, N=28672, K=8192, group=128, zeros=True, epilogue="bias_gelu_tanh"),
        # a batch of 64 sequences, finer groups
        dict(name="w4_decode_64", op="w4", M=64, N=14336, K=4096, group=64, zeros=False, epilogue="none"),
        # odd batch, odd width, K that ends inside a group and a packed kilobyte
        dict(name="w4_ragged", op="w4", M=37, N=3001, K=4104, group=32, zeros=True, epilogue="bias"),
        # one token through a square projection in 8 bits
        dict(name="q8_token", op="q8", M=1, N=8192, K=8192, epilogue="none"),
        # the decode step of a batch of 16 in 8 bits
        dict(name="q8_decode_16", op="q8", M=16, N=28672, K=8192, epilogue="bias"),
        # a ragged prompt
        dict(name="q8_prompt_ragged", op="q8", M=2047, N=3001, K=4112, epilogue="gelu_tanh"),
        # the headline linear layer (8192 tokens, bias and GELU) in 8 bits: the largest
        dict(name="q8_prompt_8192", op="q8", M=8192, N=8192, K=8192, epilogue="bias_gelu_tanh"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _size(rng, units, lo, hi):
    """An odd multiple of one of `units`, spread over the logarithm of lo..hi:
    widths in use are multiples of 512, ragged ones of the least the operator takes."""
    unit = rng.choice(units)
    return unit * (2 * _log(rng, lo // (2 * unit), (hi // unit - 1) // 2) + 1)


def draw(rng):
    op = rng.choice(["norm", "norm_q8", "norm_backward", "w4", "w4", "q8", "q8"])
    if op.startswith("norm"):
        hidden = _size(rng, (512, 8), 1024, 16384)
        rows = min(_log(rng, 1, 8192), (1 << 25) // hidden)
        return dict(op=op, rows=rows, hidden=hidden, stream=rng.choice(["bf16", "f32"]),
                    residual=rng.random() < 0.75)
    epilogue = rng.choice(["none", "bias", "gelu_tanh", "bias_gelu_tanh"])
    n = _size(rng, (512, 1), 1024, 28672)
    if op == "w4":
        return dict(op=op, M=_log(rng, 1, 64), N=n, K=_size(rng, (512, 8), 1024, 8192),
                    group=rng.choice([32, 64, 128]), zeros=rng.random() < 0.5, epilogue=epilogue)
    k = _size(rng, (512, 16), 1024, 8192)
    m = min(_log(rng, 1, 8192), (1 << 39) // (n * k))
    return dict(op=op, M=m, N=n, K=k, epilogue=epilogue)


def _rowscaled(t):
    """e4m3 rows and their fp32 scales."""
    scale = (t.abs().amax(dim=1) / E4M3_MAX).clamp_min(TINY)
    return (t / scale[:, None]).to(torch.float8_e4m3fn), scale


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def randn(shape, std=1.0, mean=0.0):
        return torch.randn(shape, generator=gen, device="cuda") * std + mean

    c = dict(case)
    if c["op"].startswith("norm"):
        rows, hidden = c["rows"], c["hidden"]
        t = torch.bfloat16 if c["stream"] == "bf16" else torch.float32
        st = {"weight": randn(hidden, 0.1, 1.0).bfloat16()}
        if c["op"] == "norm_backward":
            h = randn((rows, hidden), 2.0).to(t)
            st["h"] = h
            st["rstd"] = torch.rsqrt(h.float().square().mean(dim=1) + EPS)
            st["dy"] = randn((rows, hidden), 1e-3).bfloat16()
            st["dres"] = randn((rows, hidden), 1e-3).to(t) if c["residual"] else None
        else:
            st["x"] = randn((rows, hidden), 0.5).to(t)
            st["residual"] = randn((rows, hidden), 2.0).to(t) if c["residual"] else None
    else:
        M, N, K = c["M"], c["N"], c["K"]
        st = {"bias": randn(N).bfloat16() if "bias" in c["epilogue"] else None}
        x = randn((M, K)).bfloat16()
        if c["op"] == "w4":
            st["x"] = x
            st["W"] = torch.randint(0, 256, (-(-N // 16), -(-K // 128), 1024), generator=gen, device="cuda",
                                    dtype=torch.uint8)
            groups = -(-K // c["group"])
            # the spread of a code (4.6) times this gives rows of unit norm
            st["scales"] = ((0.5 + torch.rand((groups, N), generator=gen, device="cuda"))
                            * (K ** -0.5 / 4.6)).bfloat16()
            st["zeros"] = (torch.randint(6, 11, (groups, N), generator=gen, device="cuda", dtype=torch.uint8)
                           if c["zeros"] else None)
        else:
            st["x"], st["x_scale"] = _rowscaled(x.float())
            st["W"], st["w_scale"] = _rowscaled(randn((N, K), K ** -0.5))
    return c, st


# ---- plain forms -----------------------------------------------------------

def _codes(W, N, K):
    """The whole numbers [N, K] of a packed 4-bit weight."""
    words = W.view(torch.int32).view(W.shape[0], W.shape[1], 4, 16, 4, 1)
    shifts = torch.tensor(NIBBLE_SHIFTS, dtype=torch.int32, device=W.device)
    codes = (words >> shifts) & 15
    return codes.permute(0, 3, 1, 4, 2, 5).reshape(W.shape[0] * 16, W.shape[1] * 128)[:N, :K]


def _epilogue(y, bias, kind):
    if bias is not None:
        y = y + bias.float()
    if kind.endswith("gelu_tanh"):
        y = 0.5 * y * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (y + 0.044715 * y * y * y)))
    return y.bfloat16()


def _plain(c, st):
    op = c["op"]
    if op in ("norm", "norm_q8"):
        x = st["x"]
        h = x if st["residual"] is None else (x.float() + st["residual"].float()).to(x.dtype)
        hf = h.float()
        rstd = torch.rsqrt(hf.square().mean(dim=1) + EPS)
        y = hf * rstd[:, None] * st["weight"].float()
        if op == "norm":
            return {"y": y.bfloat16(), "h": h, "rstd": rstd}
        q, scale = _rowscaled(y)
        return {"q": q, "scale": scale, "h": h}
    if op == "norm_backward":
        hf, dy, r = st["h"].float(), st["dy"].float(), st["rstd"][:, None]
        g = dy * st["weight"].float()
        n = hf * r
        dh = r * (g - n * (g * n).mean(dim=1, keepdim=True))
        if st["dres"] is not None:
            dh = dh + st["dres"].float()
        return {"dh": dh.to(st["h"].dtype), "dweight": (dy * n).sum(dim=0)}
    M, N, K = c["M"], c["N"], c["K"]
    if op == "w4":
        group = torch.arange(K, device=st["x"].device) // c["group"]
        w = _codes(st["W"], N, K).float()
        w = w - (8.0 if st["zeros"] is None else st["zeros"].t().float()[:, group])
        w = w * st["scales"].t().float()[:, group]
        return _epilogue(st["x"].float() @ w.t(), st["bias"], c["epilogue"])
    y = st["x"].float() @ st["W"].float().t()
    return _epilogue(y * st["x_scale"][:, None] * st["w_scale"], st["bias"], c["epilogue"])


# ---- the framework's operators ---------------------------------------------

def _own(c, st):
    import dense_bf16_gemm_amd as mm

    op = c["op"]
    if op == "norm":
        y, h, rstd = mm.rms_norm(st["x"], st["weight"], st["residual"], eps=EPS)
        return {"y": y, "h": h, "rstd": rstd}
    if op == "norm_q8":
        q, scale, h = mm.rms_norm_q8(st["x"], st["weight"], st["residual"], eps=EPS)
        return {"q": q, "scale": scale, "h": h}
    if op == "norm_backward":
        dh, dweight = mm.rms_norm_backward(st["dy"], st["h"], st["weight"], st["rstd"], st["dres"])
        return {"dh": dh, "dweight": dweight}
    if op == "w4":
        return mm.linear_w4(st["x"], st["W"], st["scales"], st["zeros"], st["bias"], c["epilogue"],
                            group=c["group"])
    return mm.linear_q8(st["x"], st["x_scale"], st["W"], st["w_scale"], st["bias"], c["epilogue"])


def run(state):
    return _own(*state) if own else _plain(*state)


# ---- work and the 64-bit values --------------------------------------------

def work(case):
    c = case
    if c["op"].startswith("norm"):
        n, e = c["rows"] * c["hidden"], 2 if c["stream"] == "bf16" else 4
        if c["op"] == "norm_backward":
            per = 2 + e + (e if c["residual"] else 0) + e  # dy, h, dres; dh
            return {"bytes": n * per + 4 * c["rows"] + 6 * c["hidden"], "flops": 9 * n}
        per = e + (2 * e if c["residual"] else 0) + (1 if c["op"] == "norm_q8" else 2)
        return {"bytes": n * per + 4 * c["rows"] + 2 * c["hidden"], "flops": 5 * n}
    M, N, K = c["M"], c["N"], c["K"]
    out = 2 * M * N + (2 * N if "bias" in c["epilogue"] else 0)
    if c["op"] == "w4":
        groups = -(-K // c["group"])
        return {"bytes": N * K // 2 + groups * N * (3 if c["zeros"] else 2) + 2 * M * K + out,
                "flops": 2 * M * N * K}
    return {"bytes": N * K + M * K + 4 * (M + N) + out, "flops": 2 * M * N * K}


def exact(case, seed):
    c, st = prepare(case, seed)
    d = {k: v for k, v in st.items() if v is not None}
    op = c["op"]
    if op in ("norm", "norm_q8"):
        total = d["x"].double()
        if "residual" in d:
            total = total + d["residual"].double()
        h = total.to(d["x"].dtype).double()  # the stream's own rounding is part of the operator
        norm = ((h ** 2).sum(-1) / c["hidden"] + EPS).sqrt()
        y = h / norm.unsqueeze(-1) * d["weight"].double()
        if op == "norm":
            return {"y": y, "h": total, "rstd": 1.0 / norm}
        top = torch.maximum(y.max(-1).values, -y.min(-1).values)
        scale = (top / E4M3_MAX).clamp(min=TINY)
        return {"q": y / scale.unsqueeze(-1), "scale": scale, "h": total}
    if op == "norm_backward":
        h, dy, r = d["h"].double(), d["dy"].double(), d["rstd"].double().unsqueeze(-1)
        wdy = dy * d["weight"].double()
        along = (wdy * h).sum(-1, keepdim=True) * r ** 3 / c["hidden"]
        dh = r * wdy - along * h
        if "dres" in d:
            dh = dh + d["dres"].double()
        return {"dh": dh, "dweight": torch.mv((dy * h).t(), r.squeeze(-1))}
    M, N, K = c["M"], c["N"], c["K"]
    if op == "w4":
        # byte b of a word: nibbles 2b and 2b + 1; k of nibble p is 2p, of nibble p + 4 is 2p + 1
        b = d["W"].reshape(-1, d["W"].shape[1], 4, 16, 4, 4)
        nib = torch.stack((b % 16, b // 16), dim=-1).flatten(-2)
        w = torch.empty((b.shape[0], 16, b.shape[1], 4, 4, 8), dtype=torch.float64, device="cuda")
        nib = nib.permute(0, 3, 1, 4, 2, 5)
        w[..., 0::2] = nib[..., :4]
        w[..., 1::2] = nib[..., 4:]
        w = w.reshape(b.shape[0] * 16, -1)[:N, :K]
        zero = d["zeros"].double().repeat_interleave(c["group"], 0)[:K].t() if "zeros" in d else 8.0
        w = (w - zero) * d["scales"].double().repeat_interleave(c["group"], 0)[:K].t()
        y = torch.mm(d["x"].double(), w.t().contiguous())
    else:
        y = torch.mm(d["x"].double() * d["x_scale"].double().unsqueeze(-1),
                     (d["W"].double() * d["w_scale"].double().unsqueeze(-1)).t().contiguous())
    if "bias" in d:
        y = y + d["bias"].double()
    if "gelu" in c["epilogue"]:
        y = y / (1.0 + torch.exp(-2.0 * math.sqrt(2.0 / math.pi) * (y + 0.044715 * y ** 3)))
    return y
