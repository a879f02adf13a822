"""Cases of a decoder layer's operators beside its products: layer norm with
the residual's addition (and its gradient), the linear layer of many requests
with a low-rank adapter each, and the mixture-of-experts FFN of a few tokens.

``own`` selects what run() calls: False computes the operators from elementary
torch operations, True calls dense_bf16_gemm_amd.  Inputs come from the seed
alone and are the same for both.
"""
import math

import torch

own = False

EPS = 1e-5


def listed():
    return [
        # the smallest call: one new token's residual stream
        dict(name="norm_token", op="norm", rows=1, hidden=8192, stream="bf16", residual=True),
        # training forward, fp32 residual stream, a ragged batch and width
        dict(name="norm_train_f32", op="norm", rows=2047, hidden=5000, stream="f32", residual=True),
        # the gradient at a training batch's size, bf16 stream, with the residual path's gradient
        dict(name="norm_backward", op="norm_backward", rows=8192, hidden=4096, stream="bf16", residual=True),
        # the gradient of a short ragged batch, fp32 stream
        dict(name="norm_backward_short", op="norm_backward", rows=300, hidden=5000, stream="f32", residual=False),
        # one token with its adapter through a square projection: latency counts
        dict(name="lora_token", op="lora", M=1, N=8192, K=8192, rank=16, adapters=32, requests=1, epilogue="none"),
        # the decode step of 16 requests (bench.py's decode shape), each with an adapter of its own choice
        dict(name="lora_decode_16", op="lora", M=16, N=28672, K=8192, rank=16, adapters=16, requests=16,
             epilogue="bias"),
        # 64 requests on few adapters of a high rank
        dict(name="lora_decode_64", op="lora", M=64, N=14336, K=4096, rank=64, adapters=8, requests=64,
             epilogue="none"),
        # ragged prompts of five requests in one batch
        dict(name="lora_prompts_ragged", op="lora", M=2047, N=3001, K=4104, rank=32, adapters=24, requests=5,
             epilogue="gelu_tanh"),
        # the headline linear layer (8192 tokens, bias and GELU) for eight requests: the most operations
        dict(name="lora_prompts_8192", op="lora", M=8192, N=8192, K=8192, rank=16, adapters=16, requests=8,
             epilogue="bias_gelu_tanh"),
        # one token, two of eight wide experts (the FFN sizes of bench.py)
        dict(name="moe_token", op="moe", T=1, E=8, H=4096, I=14336, top_k=2, renormalize=True, padded=0),
        # 16 sequences, eight of 128 narrow experts: the most bytes
        dict(name="moe_batch_16", op="moe", T=16, E=128, H=4096, I=1536, top_k=8, renormalize=True, padded=0),
        # a padded batch, odd sizes throughout, weights not renormalized
        dict(name="moe_ragged", op="moe", T=61, E=60, H=2056, I=1416, top_k=4, renormalize=False, padded=3),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _size(rng, units, lo, hi):
    """An odd multiple of one of `units`, spread over the logarithm of lo..hi:
    widths in use are multiples of 512, ragged ones of the least the operator takes."""
    unit = rng.choice(units)
    return unit * (2 * _log(rng, max(1, lo // (2 * unit)), (hi // unit - 1) // 2) + 1)


def draw(rng):
    op = rng.choice(["norm", "norm_backward", "lora", "lora", "lora", "moe", "moe", "moe"])
    if op.startswith("norm"):
        hidden = _size(rng, (512, 8), 256, 16384)
        rows = min(_log(rng, 1, 8192), (1 << 25) // hidden)
        return dict(op=op, rows=rows, hidden=hidden, stream=rng.choice(["bf16", "f32"]),
                    residual=rng.random() < 0.75)
    if op == "lora":
        n, k = _size(rng, (512, 1), 1024, 28672), _size(rng, (512, 8), 1024, 8192)
        m = min(_log(rng, 1, 8192), (1 << 39) // (n * k))
        return dict(op=op, M=m, N=n, K=k, rank=rng.choice([8, 16, 24, 32, 64, 128]), adapters=_log(rng, 1, 64),
                    requests=m if m <= 64 else _log(rng, 1, 64),
                    epilogue=rng.choice(["none", "bias", "gelu_tanh", "bias_gelu_tanh"]))
    h, e = _size(rng, (512, 8), 1024, 8192), _log(rng, 4, 128)
    i = min(_size(rng, (512, 8), 512, 14336), (400 << 20) // (e * h) // 8 * 8)
    t = _log(rng, 1, 64)
    return dict(op=op, T=t, E=e, H=h, I=i, top_k=min(e, rng.choice([1, 2, 4, 6, 8])),
                renormalize=rng.random() < 0.7, padded=rng.choice([0, 0, 0, min(2, t - 1)]))


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def randn(shape, std=1.0, mean=0.0):
        return torch.randn(shape, generator=gen, device="cuda") * std + mean

    def stack(count, shape, std):
        """bf16 [count, *shape], made one after the other (less fp32 memory at a time)"""
        out = torch.empty((count, *shape), dtype=torch.bfloat16, device="cuda")
        for i in range(count):
            out[i] = randn(shape, std)
        return out

    c = dict(case)
    if c["op"].startswith("norm"):
        rows, hidden = c["rows"], c["hidden"]
        t = torch.bfloat16 if c["stream"] == "bf16" else torch.float32
        st = {"weight": randn(hidden, 0.1, 1.0).bfloat16(), "bias": randn(hidden, 0.1).bfloat16()}
        h = randn((rows, hidden), 2.0, 0.3).to(t)
        if c["op"] == "norm_backward":
            hf = h.double()
            st["h"] = h
            st["mean"] = hf.mean(dim=1).float()
            st["rstd"] = torch.rsqrt(hf.var(dim=1, correction=0) + EPS).float()
            st["dy"] = randn((rows, hidden), 1e-3).bfloat16()
            st["dres"] = randn((rows, hidden), 1e-3).to(t) if c["residual"] else None
        else:
            st["x"] = randn((rows, hidden), 0.5).to(t) if c["residual"] else h
            st["residual"] = h if c["residual"] else None
    elif c["op"] == "lora":
        M, N, K, R, L, n = c["M"], c["N"], c["K"], c["rank"], c["adapters"], c["requests"]
        st = {"x": randn((M, K)).bfloat16(), "W": randn((N, K), K ** -0.5).bfloat16(),
              "A": randn((L, R, K), K ** -0.5).bfloat16(), "B": randn((L, N, R), 0.1 * R ** -0.5).bfloat16(),
              "scale": 1.0 + torch.rand(L, generator=gen, device="cuda"),
              "bias": randn(N).bfloat16() if "bias" in c["epilogue"] else None}
        # requests follow one another in the batch; one in nine or so runs without an adapter
        choice = torch.randint(0, L, (n,), generator=gen, device="cuda")
        choice[torch.rand(n, generator=gen, device="cuda") < 1 / 9] = -1
        if n < M:
            ends = torch.sort(torch.randint(1, M, (n - 1,), generator=gen, device="cuda")).values
            of_row = torch.searchsorted(ends, torch.arange(M, device="cuda"), right=True)
        else:
            of_row = torch.arange(M, device="cuda")
        st["index"] = choice[of_row].int()
    else:
        T, E, H, I = c["T"], c["E"], c["H"], c["I"]
        st = {"x": randn((T, H)).bfloat16(), "logits": randn((T, E), 1.5)}
        # the last rows of a padded batch are tokens that take no expert
        st["logits"][T - c["padded"]:] = -math.inf
        st["W_gate"] = stack(E, (I, H), H ** -0.5)
        st["W_up"] = stack(E, (I, H), H ** -0.5)
        st["W_down"] = stack(E, (H, I), I ** -0.5)
    return c, st


# ---- plain forms -----------------------------------------------------------

def _silu(t):
    return t / (1.0 + torch.exp(-t))


def _plain(c, st):
    op = c["op"]
    if op == "norm":
        x = st["x"]
        h = x if st["residual"] is None else (x.float() + st["residual"].float()).to(x.dtype)
        hf = h.float()
        mean = hf.mean(dim=1)
        d = hf - mean[:, None]
        rstd = torch.rsqrt(d.square().mean(dim=1) + EPS)
        y = d * rstd[:, None] * st["weight"].float() + st["bias"].float()
        return {"y": y.bfloat16(), "h": h, "mean": mean, "rstd": rstd}
    if op == "norm_backward":
        dy, r = st["dy"].float(), st["rstd"][:, None]
        n = (st["h"].float() - st["mean"][:, None]) * r
        g = dy * st["weight"].float()
        dh = r * (g - g.mean(dim=1, keepdim=True) - n * (g * n).mean(dim=1, keepdim=True))
        if st["dres"] is not None:
            dh = dh + st["dres"].float()
        return {"dh": dh.to(st["h"].dtype), "dweight": (dy * n).sum(dim=0), "dbias": dy.sum(dim=0)}
    if op == "lora":
        x, index = st["x"].float(), st["index"].long()
        L, R, K = st["A"].shape
        # every adapter's part of every row, of which the row's own stays
        part = (x @ st["A"].float().reshape(L * R, K).t()).reshape(-1, L, R)
        mine = index[:, None] == torch.arange(L, device=x.device)
        part = torch.where(mine[:, :, None], part * st["scale"][:, None], 0.0).reshape(-1, L * R)
        y = x @ st["W"].float().t() + part @ st["B"].float().permute(0, 2, 1).reshape(L * R, -1)
        if st["bias"] is not None:
            y = y + st["bias"].float()
        if c["epilogue"].endswith("gelu_tanh"):
            y = 0.5 * y * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (y + 0.044715 * y * y * y)))
        return y.bfloat16()
    logits, k = st["logits"], c["top_k"]
    T, E = logits.shape
    values, order = torch.sort(logits, dim=1, descending=True, stable=True)
    values, ids = values[:, :k], order[:, :k]
    live = values > -math.inf
    top = values[:, :1]
    share = torch.where(live, torch.exp(values - top), 0.0)
    over = share if c["renormalize"] else torch.where(logits > -math.inf, torch.exp(logits - top), 0.0)
    weights = torch.where(live, share / over.sum(dim=1, keepdim=True), 0.0)
    x = st["x"].float()
    if T * k < E:  # the experts' weights of each token
        at, rows = ids.reshape(-1), x.repeat_interleave(k, dim=0)[:, :, None]
        g = torch.matmul(st["W_gate"][at].float(), rows)
        u = torch.matmul(st["W_up"][at].float(), rows)
        y = torch.matmul(st["W_down"][at].float(), _silu(g) * u).reshape(T, k, -1)
        y = torch.where(live[:, :, None], y * weights[:, :, None], 0.0).sum(dim=1)
    else:  # every token through every expert
        dense = torch.zeros((T, E), device=x.device).scatter_(1, ids, weights)
        y = torch.zeros_like(x)
        for e in range(E):
            h = _silu(x @ st["W_gate"][e].float().t()) * (x @ st["W_up"][e].float().t())
            y = y + dense[:, e, None] * (h @ st["W_down"][e].float().t())
    return {"y": y.bfloat16(), "experts": torch.where(live, ids, -1).int(), "weights": weights}


# ---- the framework's operators ---------------------------------------------

def _own(c, st):
    import dense_bf16_gemm_amd as mm

    op = c["op"]
    if op == "norm":
        y, h, mean, rstd = mm.layer_norm(st["x"], st["weight"], st["bias"], st["residual"], eps=EPS)
        return {"y": y, "h": h, "mean": mean, "rstd": rstd}
    if op == "norm_backward":
        dh, dweight, dbias = mm.layer_norm_backward(st["dy"], st["h"], st["weight"], st["mean"], st["rstd"],
                                                    st["dres"])
        return {"dh": dh, "dweight": dweight, "dbias": dbias}
    if op == "lora":
        return mm.linear_lora(st["x"], st["W"], st["A"], st["B"], st["index"], st["scale"], st["bias"],
                              c["epilogue"])
    y, experts, weights = mm.moe_ffn(st["x"], st["logits"], st["W_gate"], st["W_up"], st["W_down"], c["top_k"],
                                     renormalize=c["renormalize"])
    return {"y": y, "experts": experts, "weights": weights}


def run(state):
    return _own(*state) if own else _plain(*state)


# ---- work and the 64-bit values --------------------------------------------

def _used(count, picks):
    """How many of `count` are picked at least once, on the average of `picks` free choices."""
    return count * (1.0 - (1.0 - 1.0 / count) ** picks)


def work(case):
    c = case
    if c["op"].startswith("norm"):
        n, e = c["rows"] * c["hidden"], 2 if c["stream"] == "bf16" else 4
        if c["op"] == "norm_backward":
            per = 2 + e + (e if c["residual"] else 0) + e  # dy, h, dres; dh
            return {"bytes": n * per + 8 * c["rows"] + 10 * c["hidden"], "flops": 13 * n}
        per = e + (2 * e if c["residual"] else 0) + 2
        return {"bytes": n * per + 8 * c["rows"] + 4 * c["hidden"], "flops": 8 * n}
    if c["op"] == "lora":
        M, N, K, R = c["M"], c["N"], c["K"], c["rank"]
        used = _used(c["adapters"], c["requests"] * 8 / 9)
        out = 2 * M * N + (2 * N if "bias" in c["epilogue"] else 0)
        return {"bytes": 2 * (N * K + M * K) + out + 4 * M + int(used * 2 * R * (N + K)),
                "flops": 2 * M * N * K + 2 * M * R * (N + K) * 8 // 9}
    T, E, H, I, k = c["T"], c["E"], c["H"], c["I"], c["top_k"]
    live = T - c["padded"]
    used = E * (1.0 - (1.0 - k / E) ** live)  # experts that a token takes, on the average
    return {"bytes": int(used * 6 * H * I) + 4 * T * H + 4 * T * E + 8 * T * k, "flops": 6 * live * k * H * I}


def exact(case, seed):
    c, st = prepare(case, seed)
    d = {k: v for k, v in st.items() if v is not None}
    op = c["op"]
    if op == "norm":
        total = d["x"].double()
        if "residual" in d:
            total = total + d["residual"].double()
        h = total.to(d["x"].dtype).double()  # the stream's own rounding is part of the operator
        mean = h.sum(-1) / c["hidden"]
        spread = ((h - mean.unsqueeze(-1)) ** 2).sum(-1) / c["hidden"]
        r = 1.0 / (spread + EPS).sqrt()
        y = torch.addcmul(d["bias"].double(), (h - mean.unsqueeze(-1)) * r.unsqueeze(-1), d["weight"].double())
        return {"y": y, "h": total, "mean": mean, "rstd": r}
    if op == "norm_backward":
        r, dy = d["rstd"].double().unsqueeze(-1), d["dy"].double()
        z = d["h"].double() - d["mean"].double().unsqueeze(-1)
        wdy = dy * d["weight"].double()
        along = (wdy * z).sum(-1, keepdim=True) * r ** 2 / c["hidden"]
        dh = r * (wdy - z * along) - r * wdy.sum(-1, keepdim=True) / c["hidden"]
        if "dres" in d:
            dh = dh + d["dres"].double()
        return {"dh": dh, "dweight": torch.mv((dy * z).t(), r.squeeze(-1)),
                "dbias": torch.mv(dy.t(), torch.ones_like(r.squeeze(-1)))}
    if op == "lora":
        x = d["x"].double()
        y = torch.mm(x, d["W"].double().t().contiguous())
        for a in d["index"].unique().tolist():
            if a >= 0:
                rows = (d["index"] == a).nonzero().flatten()
                low = torch.mm(x[rows], d["A"][a].double().t().contiguous()) * d["scale"][a].double()
                y[rows] += torch.mm(low, d["B"][a].double().t().contiguous())
        if "bias" in d:
            y += d["bias"].double()
        if "gelu" in c["epilogue"]:
            y = y / (1.0 + torch.exp(-2.0 * math.sqrt(2.0 / math.pi) * (y + 0.044715 * y ** 3)))
        return y
    logits, x = d["logits"].double().cpu(), d["x"].double()
    y = torch.zeros_like(x)
    weights = torch.zeros((c["T"], c["top_k"]), dtype=torch.float64)
    takers = {}
    for t, row in enumerate(logits.tolist()):
        chosen = sorted((e for e in range(c["E"]) if row[e] > -math.inf), key=lambda e: (-row[e], e))
        pool = chosen[:c["top_k"]] if c["renormalize"] else chosen
        norm = math.fsum(math.exp(row[e] - row[chosen[0]]) for e in pool)
        for j, e in enumerate(chosen[:c["top_k"]]):
            weights[t, j] = math.exp(row[e] - row[chosen[0]]) / norm
            takers.setdefault(e, []).append((t, weights[t, j].item()))
    for e, those in takers.items():
        rows = torch.tensor([t for t, _ in those], device=x.device)
        share = torch.tensor([w for _, w in those], dtype=torch.float64, device=x.device)
        g = torch.mm(x[rows], d["W_gate"][e].double().t().contiguous())
        u = torch.mm(x[rows], d["W_up"][e].double().t().contiguous())
        part = torch.mm(g * torch.sigmoid(g) * u, d["W_down"][e].double().t().contiguous())
        y.index_add_(0, rows, part * share.unsqueeze(-1))
    return {"y": y, "experts": None, "weights": weights}
