"""The linear layer with an adapter per row, on the GPU against its 64-bit form.

Inputs of small whole numbers make every sum exact, and such outputs have to match
bit for bit; the tolerances of random ones count roundings (u = 2^-24).
"""
import pytest
import torch

import dense_bf16_gemm_amd as mm
import layer_ref as ref
from dense_bf16_gemm_amd import binding
from test_gpu_decoder import BF16, U, close, dev, gen, guarded, randn, same_class  # noqa: F401 (dev is a fixture)

pytestmark = pytest.mark.gpu


def on(dev, *ts):  # noqa: F811
    return [None if t is None else t.to(dev) for t in ts]


def choices(M, L, how, g):
    """Adapters of the rows: each its own, in runs (requests), or all one; -1 among them."""
    if how == "mixed":
        return torch.randint(-1, L, (M,), generator=g, dtype=torch.int32)
    if how == "one":
        return torch.full((M,), L - 1, dtype=torch.int32)
    cuts = torch.sort(torch.randint(0, M + 1, (6,), generator=g)).values
    return torch.randint(-1, L, (7,), generator=g, dtype=torch.int32)[torch.searchsorted(cuts, torch.arange(M), right=True)]


def inputs(M, N, K, R, L, how, seed, exact=False):
    g = gen(seed)
    if exact:
        # |A x| <= 2 * 2 K / 16 or so stays a whole number of 16 bits; every sum is below 2^24
        def whole(shape, top, rare=1):
            v = torch.randint(-top, top + 1, shape, generator=g)
            return (v * (torch.randint(0, rare, shape, generator=g) == 0)).bfloat16()

        x, W = whole((M, K), 2), whole((N, K), 2)
        A, B = whole((L, R, K), 1, 4), whole((L, N, R), 2)
        scale = 2.0 ** torch.randint(-1, 3, (L,), generator=g).float()
    else:
        x, W = randn(g, (M, K)).bfloat16(), randn(g, (N, K), K ** -0.5).bfloat16()
        A, B = randn(g, (L, R, K), K ** -0.5).bfloat16(), randn(g, (L, N, R), R ** -0.5).bfloat16()
        scale = randn(g, L, 0.3, 1.0)
    return [x, W, A, B, choices(M, L, how, g), scale], randn(g, N).bfloat16()


SHAPES = [(1, 16, 64, 8, 1), (1, 1, 8, 8, 3), (1, 520, 2056, 16, 4), (2, 70, 136, 24, 2), (5, 333, 1000, 64, 40),
          (16, 130, 4104, 16, 16), (15, 17, 8, 256, 5), (16, 264, 8200, 128, 3), (17, 100, 520, 8, 70), (31, 48, 72, 40, 6),
          (32, 513, 1032, 72, 9), (33, 65, 264, 16, 5), (64, 257, 1024, 32, 80), (65, 70, 200, 16, 3),
          (100, 300, 136, 136, 4), (200, 517, 1032, 8, 12), (300, 128, 4096, 256, 2), (513, 1030, 392, 64, 7)]


@pytest.mark.parametrize("M,N,K,R,L", SHAPES)
@pytest.mark.parametrize("how", ["mixed", "runs", "one"])
def test_linear_lora_exact(dev, M, N, K, R, L, how):  # noqa: F811
    args, _ = inputs(M, N, K, R, L, how, M + N + K, exact=True)
    low = args[0].double() @ args[2].double().transpose(1, 2)
    assert float(low.abs().max() * 4) < 2 ** 15  # (16 bits of significand hold them)
    out, intact = guarded((M, N), torch.bfloat16, dev)
    got = mm.linear_lora(*on(dev, *args), out=out)
    intact()
    want = ref.lora(*args)
    assert float(want.abs().max()) < 2 ** 23 and got is out
    assert torch.equal(got.cpu(), want.float().bfloat16())


# one column, and fewer than a store's eight, of more rows than the decode kernels take
@pytest.mark.parametrize("M,N,K,R,L", [(70, 1, 8, 8, 1), (200, 3, 72, 8, 2), (130, 9, 2056, 256, 130), (1030, 7, 4096, 16, 3)])
def test_linear_lora_exact_narrow(dev, M, N, K, R, L):  # noqa: F811
    test_linear_lora_exact(dev, M, N, K, R, L, "mixed")


# K in slices and many columns: the parts of one, two and four blocks of 16 rows joined
@pytest.mark.parametrize("M,N,K,R,L", [(5, 8193, 8264, 24, 2), (20, 8200, 4200, 16, 3), (40, 8208, 136, 8, 4), (32, 70, 4104, 40, 9),
                                       (64, 8192, 2056, 256, 2)])
def test_linear_lora_exact_joined(dev, M, N, K, R, L):  # noqa: F811
    test_linear_lora_exact(dev, M, N, K, R, L, "mixed")


@pytest.mark.parametrize("M,N,K,R,L,how,epi", [
    (1, 1001, 4096, 16, 8, "mixed", "none"), (4, 1024, 2056, 64, 3, "mixed", "bias"),
    (16, 512, 8192, 16, 16, "mixed", "gelu_tanh"), (30, 300, 2000, 128, 5, "mixed", "bias_gelu_tanh"),
    (50, 257, 4096, 32, 4, "runs", "bias"), (64, 1030, 1032, 8, 64, "mixed", "none"),
    (130, 515, 4104, 16, 3, "runs", "bias_gelu_tanh"), (600, 1030, 1032, 64, 9, "runs", "gelu_tanh"),
    (1000, 258, 520, 24, 40, "mixed", "bias")])
def test_linear_lora(dev, M, N, K, R, L, how, epi):  # noqa: F811
    args, bias = inputs(M, N, K, R, L, how, M * 3 + N)
    d = on(dev, *args)
    b = bias.to(dev) if "bias" in epi else None
    got = mm.linear_lora(*d, b, epi)
    sums = ref.lora(*args)
    want, t = ref.epilogue(sums, bias, epi)
    x, W, A, B, index, scale = args
    # additions of one output, in any order: one for each product and each joined part
    # (8 waves, 16 slices); s v is cut to 16 bits of significand
    acc = (K + 64) * U * (x.double().abs() @ W.double().abs().t())
    for m, a in enumerate(index.tolist()):
        if a < 0:
            continue
        v = A[a].double() @ x[m].double()
        err = (K + 64) * U * (A[a].double().abs() @ x[m].double().abs()) + 2.0 ** -16 * v.abs() + R * U * v.abs()
        acc[m] += scale[a].double().abs() * (B[a].double().abs() @ err)
    # GELU: slope at most 1.13; its exponential and reciprocal 1e-5 of |t|
    close(got, want, BF16 * want.abs() + 1.14 * acc * (1 + BF16) + 1e-5 * t.abs(), epi)
    assert torch.equal(got, mm.linear_lora(*d, b, epi)), "not reproducible"


@pytest.mark.parametrize("M", [5, 20, 40, 200])
def test_linear_lora_rows_do_not_touch_each_other(dev, M):  # noqa: F811
    """A row's bits do not depend on the adapters of the rows beside it; an index that
    names none is no adapter; adapters that no row takes may hold anything."""
    N, K, R, L = 130, 520, 16, 6
    (x, W, A, B, index, scale), _ = inputs(M, N, K, R, L, "mixed", M)
    index[0], index[1], index[2] = 3, -1, -7
    d = on(dev, x, W, A, B, index, scale)
    got = mm.linear_lora(*d)
    none = mm.linear_lora(*d[:4], torch.full_like(d[4], -1), d[5])
    off = (index < 0).to(dev)
    assert torch.equal(got[off], none[off])
    other = d[4].clone()
    other[2:] = L + 5  # (names none)
    alone = mm.linear_lora(*d[:4], other, d[5])
    assert torch.equal(alone[0], got[0]) and torch.equal(alone[2:], none[2:])
    A2, B2, s2 = d[2].clone(), d[3].clone(), d[5].clone()
    index3 = d[4].clone()
    index3[index3 == 4] = -1
    A2[4], B2[4], s2[4] = float("nan"), float("inf"), float("nan")
    assert torch.equal(mm.linear_lora(d[0], d[1], A2, B2, index3, s2), mm.linear_lora(*d[:4], index3, d[5]))


@pytest.mark.parametrize("M,N,K,R", [(5, 130, 520, 16), (30, 130, 2056, 8), (50, 200, 520, 40), (150, 130, 520, 16),
                                     (300, 2100, 264, 72), (700, 3000, 1032, 16), (2100, 2100, 328, 8)])
@pytest.mark.parametrize("value", [float("inf"), -float("inf"), float("nan")])
def test_linear_lora_broken_adapter(dev, M, N, K, R, value):  # noqa: F811
    """An infinity or a NaN in an adapter's B: its rows lose that column (NaN, or an
    infinity), all other outputs keep their bits."""
    (x, W, A, B, index, scale), _ = inputs(M, N, K, R, 5, "mixed", M)
    index[:3] = torch.tensor([2, 0, -1])
    d = on(dev, x, W, A, B, index, scale)
    want = mm.linear_lora(*d, epilogue="gelu_tanh").cpu()
    assert want.isfinite().all()
    broken = torch.zeros((5, N), dtype=torch.bool)
    for a, n, r in ((2, 0, 0), (2, 77, R - 1), (0, N - 1, R // 2), (0, 64, 1)):
        d[3][a, n, r] = value
        broken[a, n] = True
    got = mm.linear_lora(*d, epilogue="gelu_tanh").cpu()
    bad = torch.where(index[:, None] >= 0, broken[index.clamp(min=0).long()], False)
    assert torch.equal(got[~bad], want[~bad])
    assert not got[bad].isfinite().any()  # (gelu(-inf) is NaN)


@pytest.mark.parametrize("M", [4, 30, 50, 150])
def test_linear_lora_not_finite(dev, M):  # noqa: F811
    """Infinite and NaN operands give each output the class of the definition's sums."""
    (x, W, A, B, index, scale), _ = inputs(M, 70, 392, 8, 3, "mixed", 9, exact=True)
    index[:4] = torch.tensor([0, 1, 2, -1])
    x[0, 3], x[1, 391], W[5, 100] = float("inf"), float("nan"), -float("inf")
    A[2, 1, 7] = float("inf")
    B[1, 9, 3] = float("nan")
    got = mm.linear_lora(*on(dev, x, W, A, B, index, scale)).float().cpu()
    same_class(got, ref.lora(x, W, A, B, index, scale).float())


def test_linear_lora_without_terms(dev):  # noqa: F811
    """Nothing in the adapters, no adapters, no K, no rows, no columns."""
    (x, W, A, B, index, scale), bias = inputs(9, 48, 64, 8, 3, "mixed", 1)
    d, b = on(dev, x, W, A, B, index, scale), bias.to(dev)
    plain = mm.linear(d[0], d[1], b, "bias")
    assert torch.equal(mm.linear_lora(d[0], d[1], d[2][:, :0].contiguous(), d[3][:, :, :0].contiguous(), d[4], d[5], b,
                                      "bias"), plain)
    assert torch.equal(mm.linear_lora(d[0], d[1], d[2][:0], d[3][:0], d[4], d[5][:0], b, "bias"), plain)
    got = mm.linear_lora(d[0][:, :0].contiguous(), d[1][:, :0].contiguous(), d[2][:, :, :0].contiguous(), d[3], d[4],
                         d[5], b, "bias")
    assert torch.equal(got, b.expand(9, 48))
    assert mm.linear_lora(d[0][:0], *d[1:4], d[4][:0], d[5]).shape == (0, 48)
    assert mm.linear_lora(d[0], d[1][:0], d[2], d[3][:, :0].contiguous(), d[4], d[5]).shape == (9, 0)


@pytest.mark.parametrize("M,workspace", [(7, 1), (90, 1)])
def test_linear_lora_keeps_inside_its_workspace(dev, M, workspace):  # noqa: F811
    """The bytes behind the reported workspace stay as they were, and a workspace
    full of NaN serves as well as any."""
    args, _ = inputs(M, 300, 1032, 24, 4, "mixed", 5)
    d = on(dev, *args)
    want = mm.linear_lora(*d)
    nbytes = binding.linear_lora_workspace_size(M, 300, 1032, 24, 4)
    ws = torch.full((nbytes + 256,), 0xFF, dtype=torch.uint8, device=dev)
    out = torch.empty_like(want)
    binding.check(binding.load().mm_linear_lora(*(t.data_ptr() for t in d), None, out.data_ptr(), M, 300, 1032, 24, 4, 0,
                                                ws.data_ptr(), nbytes, torch.cuda.current_stream().cuda_stream),
                  "mm_linear_lora")
    assert torch.equal(out, want) and bool((ws[nbytes:] == 0xFF).all())


def test_linear_lora_past_32_bits(dev):  # noqa: F811
    """A weight and stacks of adapters of more than 2^32 bytes each: the last columns
    and the last adapter against the same alone."""
    N, K, R, L = 300016, 8192, 16, 600
    (x, _, _, _, _, _), _ = inputs(4, 8, K, 8, 1, "one", 6)
    W = torch.zeros((N, K), dtype=torch.bfloat16, device=dev)
    A = torch.zeros((L * 28, R, K), dtype=torch.bfloat16, device=dev)
    B = torch.zeros((L, N, R), dtype=torch.bfloat16, device=dev)
    g = gen(7)
    W[-40:] = randn(g, (40, K), K ** -0.5).bfloat16().to(dev)
    A[L - 1] = randn(g, (R, K), K ** -0.5).bfloat16().to(dev)
    B[-1, -40:] = randn(g, (40, R), R ** -0.5).bfloat16().to(dev)
    x = x.to(dev)
    index = torch.tensor([L - 1, -1, L - 1, 0], dtype=torch.int32, device=dev)
    scale = torch.ones(L, device=dev)
    got = mm.linear_lora(x, W, A[:L], B, index, scale)
    want = mm.linear_lora(x, W[-40:], A[L - 1:L], B[-1:, -40:].contiguous(), torch.where(index == 0, -1, index).clamp(max=0),
                          scale[:1])
    assert torch.equal(got[:, -40:], want)
    del B
    B = torch.zeros((L * 28, 40, R), dtype=torch.bfloat16, device=dev)
    A[-1], B[-1] = A[L - 1], randn(g, (40, R)).bfloat16().to(dev)
    last = torch.where(index > 0, L * 28 - 1, -1).int()
    got = mm.linear_lora(x, W[-40:], A, B, last, torch.ones(L * 28, device=dev))
    want = mm.linear_lora(x, W[-40:], A[-1:], B[-1:], last.clamp(max=0), scale[:1])
    assert torch.equal(got, want)
