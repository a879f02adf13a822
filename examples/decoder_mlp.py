"""The decoder-layer operators together, as a served model and a training step
use them, on random weights.

    python examples/decoder_mlp.py [--hidden 4096] [--ffn 14336] [--prompt 512] [--batch 16] [--steps 4]

Serving: each layer adds the block's output to the residual stream, norms it
and writes 8-bit activations with row scales in one kernel (rms_norm_q8),
multiplies them with an 8-bit up projection, bias and GELU in the product's
epilogue (linear_q8), and takes the result back to the stream's width: with
an 8-bit weight for a prompt, with a 4-bit weight (linear_w4) for the decode
steps, which are captured into a graph once and replayed.

Training: the norm ahead of a linear layer, forward and backward, the
residual path's gradient added in the norm's own kernel.

Both print a time and how far the result is from the same layer in fp32 with
the weights that the quantised ones stand for.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import dense_bf16_gemm_amd as mm  # noqa: E402

GROUP = 64


def rowscaled(w):
    """e4m3 rows of a weight and their scales."""
    scale = (w.abs().amax(dim=1) / 448.0).clamp_min(2.0 ** -126)
    return (w / scale[:, None]).to(torch.float8_e4m3fn), scale


def quantise_w4(w):
    """Codes, scales and zeros of a weight by groups of GROUP inputs."""
    n, k = w.shape
    parts = w.view(n, k // GROUP, GROUP)
    lo, hi = parts.amin(dim=2), parts.amax(dim=2)
    scale = ((hi - lo) / 15.0).clamp_min(1e-8).bfloat16()
    zero = (-lo / scale.float()).round().clamp(0, 15)
    codes = (parts / scale.float()[:, :, None] + zero[:, :, None]).round().clamp(0, 15)
    return (codes.view(n, k).to(torch.uint8), scale.t().contiguous(), zero.t().contiguous().to(torch.uint8))


class Mlp:
    """One layer's norm and MLP with random quantised weights."""

    def __init__(self, hidden, ffn, gen, dev):
        def randn(*shape, std=1.0):
            return torch.randn(shape, generator=gen, device=dev) * std

        self.norm = (1.0 + randn(hidden, std=0.1)).bfloat16()
        self.bias = randn(ffn, std=0.1).bfloat16()
        self.up = rowscaled(randn(ffn, hidden, std=hidden ** -0.5))
        down = randn(hidden, ffn, std=ffn ** -0.5)
        self.down_q8 = rowscaled(down)
        codes, self.scales, self.zeros = quantise_w4(down)
        self.down_w4 = mm.pack_w4(codes)
        by_k = torch.arange(ffn, device=dev) // GROUP
        self.down_f32 = (codes.float() - self.zeros.float().t()[:, by_k]) * self.scales.float().t()[:, by_k]

    def decode(self, x, stream):
        """x: the block before's output, added to the residual stream."""
        q, scale, stream = mm.rms_norm_q8(x, self.norm, stream)
        mid = mm.linear_q8(q, scale, *self.up, self.bias, "bias_gelu_tanh")
        return mm.linear_w4(mid, self.down_w4, self.scales, self.zeros, group=GROUP), stream

    def prompt(self, x, stream):
        q, scale, stream = mm.rms_norm_q8(x, self.norm, stream)
        mid = mm.linear_q8(q, scale, *self.up, self.bias, "bias_gelu_tanh")
        q, scale = rowscaled(mid.float())
        return mm.linear_q8(q, scale, *self.down_q8), stream

    def plain(self, x, stream, down):
        h = (x + stream).float()
        y = h * torch.rsqrt(h.square().mean(dim=1, keepdim=True) + 1e-6) * self.norm.float()
        up = self.up[0].float() * self.up[1][:, None]
        mid = torch.nn.functional.gelu(y @ up.t() + self.bias.float(), approximate="tanh")
        return mid @ down.t()


def distance(got, want):
    return float((got.float() - want).norm() / want.norm())


def timed(fn, calls=20):
    fn()
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    start.record()
    for _ in range(calls):
        fn()
    end.record()
    end.synchronize()
    return start.elapsed_time(end) * 1e3 / calls


def serve(args, gen, dev):
    mlp = Mlp(args.hidden, args.ffn, gen, dev)

    def randn(rows):
        return torch.randn((rows, args.hidden), generator=gen, device=dev).bfloat16()

    x, stream = randn(args.prompt), randn(args.prompt)
    y, _ = mlp.prompt(x, stream)
    off = distance(y, mlp.plain(x, stream, mlp.down_q8[0].float() * mlp.down_q8[1][:, None]))
    print(f"prompt of {args.prompt}: {timed(lambda: mlp.prompt(x, stream)):.1f} us, off by {off:.4f}")

    for rows in (1, args.batch):
        x, stream = randn(rows), randn(rows)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            mlp.decode(x, stream)
        torch.cuda.current_stream().wait_stream(side)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            y, h = mlp.decode(x, stream)
        worst = 0.0
        for _ in range(args.steps):  # each step's output and stream are the next one's inputs
            want = mlp.plain(x, stream, mlp.down_f32)
            graph.replay()
            worst = max(worst, distance(y, want))
            x.copy_(y)
            stream.copy_(h)
        print(f"decode, {rows} rows: {timed(graph.replay):.1f} us, off by {worst:.4f} at most in {args.steps} steps")
        if not worst < 0.1:
            raise SystemExit("decode step off")
    if not off < 0.1:
        raise SystemExit("prompt off")


def train(args, gen, dev):
    """y = linear(norm(x + residual)), loss = sum(y * c): gradients of the
    stream and of the norm's weight against autograd's in fp32."""
    rows = args.prompt
    x, res, c = (torch.randn((rows, args.hidden), generator=gen, device=dev) for _ in range(3))
    weight = (1.0 + 0.1 * torch.randn(args.hidden, generator=gen, device=dev)).bfloat16()
    W = (torch.randn((args.hidden, args.hidden), generator=gen, device=dev) * args.hidden ** -0.5).bfloat16()
    c = c.bfloat16()

    def step():
        y, h, rstd = mm.rms_norm(x, weight, res)
        out = mm.linear(y, W)
        dy = mm.matmul(c, W)
        # the stream goes on past the norm with gradient c as well
        dh, dw = mm.rms_norm_backward(dy, h, weight, rstd, c.float())
        return out, dh, dw

    out, dh, dw = step()
    xs = x.clone().requires_grad_()
    ws = weight.float().requires_grad_()
    h = xs + res
    n = h * torch.rsqrt(h.square().mean(dim=1, keepdim=True) + 1e-6) * ws
    want = n @ W.float().t()
    ((want + h) * c.float()).sum().backward()
    off = [distance(out, want.detach()), distance(dh, xs.grad), distance(dw, ws.grad)]
    print(f"training step of {rows} rows: {timed(step):.1f} us, output, dh and dweight off by "
          + ", ".join(f"{v:.4f}" for v in off))
    if not max(off) < 0.02:
        raise SystemExit("training step off")


def main(argv=None):
    parser = argparse.ArgumentParser(description=__doc__.split("\n\n")[0])
    for name, value in (("hidden", 4096), ("ffn", 14336), ("prompt", 512), ("batch", 16), ("steps", 4)):
        parser.add_argument(f"--{name}", type=int, default=value)
    args = parser.parse_args(argv)
    if args.hidden % 16 or args.ffn % GROUP:
        parser.error(f"hidden must be a multiple of 16 and ffn of {GROUP}")
    if min(args.hidden, args.ffn, args.prompt, args.batch, args.steps) < 1:
        parser.error("sizes and steps must be positive")
    if not torch.cuda.is_available():
        raise SystemExit("this example needs a GPU")
    dev = torch.device("cuda:0")
    gen = torch.Generator(device=dev).manual_seed(1)
    serve(args, gen, dev)
    train(args, gen, dev)


if __name__ == "__main__":
    main()
