"""The mixture-of-experts FFN of a few tokens on the GPU against its 64-bit form, and a
decoder layer's step of layer norm, linear layers with adapters and experts.
"""
import math

import pytest
import torch

import dense_bf16_gemm_amd as mm
import layer_ref as ref
from dense_bf16_gemm_amd import binding
from test_gpu_decoder import BF16, U, close, dev, gen, guarded, randn  # noqa: F401 (dev is a fixture)

pytestmark = pytest.mark.gpu


def on(dev, *ts):  # noqa: F811
    return [None if t is None else t.to(dev) for t in ts]


def inputs(T, E, H, I, seed):
    g = gen(seed)
    x = randn(g, (T, H)).bfloat16()
    logits = randn(g, (T, E), 1.5)
    gate, up = (randn(g, (E, I, H), H ** -0.5).bfloat16() for _ in range(2))
    return x, logits, gate, up, randn(g, (E, H, I), I ** -0.5).bfloat16()


def check(got, x, logits, gate, up, down, k, renormalize):
    out, experts, weights = got
    we, ww = ref.route(logits, k, renormalize)
    assert experts.dtype == torch.int32 and weights.dtype == torch.float32
    assert torch.equal(experts.cpu(), we)
    # exponentials of differences (exact to u |difference|, at most 20 here) to 4 u, at most
    # 8 + 6 additions, a division
    close(weights, ww, 64 * U * ww, "weights")
    want, size = ref.moe(x, we, ww, gate, up, down)
    H, I = x.shape[1], gate.shape[1]
    # every addition of either layer, in any order; SiLU's exponential and reciprocal, the
    # weights and 16 bits of significand between the layers
    acc = ((H + I + 64 * k + 64) * U + 2.0 ** -16 + 2.0 ** -17) * size
    close(out, want, BF16 * want.abs() + acc * (1 + BF16), "out")


SHAPES = [(1, 8, 256, 512, 2), (1, 1, 8, 8, 1), (1, 64, 136, 72, 8), (2, 5, 520, 264, 3), (3, 130, 64, 40, 16),
          (16, 16, 264, 136, 4), (7, 300, 72, 200, 6), (13, 512, 16, 24, 10), (17, 4, 1032, 520, 2), (32, 32, 200, 328, 8),
          (33, 3, 392, 72, 3), (64, 8, 512, 256, 2), (61, 60, 264, 136, 4), (64, 64, 72, 1032, 16), (50, 2, 2056, 264, 1)]


@pytest.mark.parametrize("T,E,H,I,k", SHAPES)
@pytest.mark.parametrize("renormalize", [True, False])
def test_moe_ffn(dev, T, E, H, I, k, renormalize):  # noqa: F811
    args = inputs(T, E, H, I, T + E + H)
    out, intact = guarded((T, H), torch.bfloat16, dev)
    d = on(dev, *args)
    got = mm.moe_ffn(*d, k, renormalize, out=out)
    intact()
    check(got, *args, k, renormalize)
    for a, b in zip(got, mm.moe_ffn(*d, k, renormalize)):
        assert torch.equal(a, b), "not reproducible"


@pytest.mark.parametrize("T", [5, 30, 64])
def test_moe_ffn_all_tokens_on_one_expert(dev, T):  # noqa: F811
    args = list(inputs(T, 9, 264, 520, T))
    args[1] = torch.full((T, 9), -math.inf)
    args[1][:, 7] = 2.5
    check(mm.moe_ffn(*on(dev, *args), 1), *args, 1, True)
    got = mm.moe_ffn(*on(dev, *args), 3)  # (two slots of each token stay empty)
    check(got, *args, 3, True)
    assert (got[1][:, 0] == 7).all() and (got[1][:, 1:] == -1).all() and (got[2][:, 0] == 1).all()


def test_moe_ffn_masked_logits_ties_and_padded_rows(dev):  # noqa: F811
    T, E, H, I, k = 9, 70, 136, 72, 4
    args = list(inputs(T, E, H, I, 3))
    logits = args[1]
    logits[0] = -math.inf                        # a padded row
    logits[1] = -math.inf
    logits[1, 69] = -torch.finfo(torch.float32).max  # one expert, with the lowest finite value
    logits[2] = torch.finfo(torch.float32).min   # a row of the lowest value: ties, the lowest indices
    logits[3] = 1.0
    logits[4, ::2] = 0.0
    logits[4, 1::2] = -0.0                       # both zeros are the same
    logits[5, 10:] = -math.inf
    logits[6] = torch.round(logits[6])           # many ties
    logits[8] = -math.inf
    for renormalize in (True, False):
        got = mm.moe_ffn(*on(dev, *args), k, renormalize)
        check(got, *args, k, renormalize)
    experts = got[1].cpu()
    assert experts[2].tolist() == experts[3].tolist() == experts[4].tolist() == [0, 1, 2, 3]
    assert (got[0][[0, 8]] == 0).all() and (got[2][[0, 8]] == 0).all()
    # no token at all
    args[1] = torch.full_like(logits, -math.inf)
    got = mm.moe_ffn(*on(dev, *args), k)
    assert (got[0] == 0).all() and (got[1] == -1).all() and (got[2] == 0).all()


def test_moe_ffn_not_finite(dev):  # noqa: F811
    """Logits of NaN or plus infinity make their token's weights NaN, as does a NaN among
    the activations of the output; other tokens, and what only idle experts hold, stay out of it."""
    T, E, H, I, k = 6, 12, 136, 72, 2
    x, logits, gate, up, down = inputs(T, E, H, I, 4)
    logits[:, 11] = -math.inf  # idle
    clean = mm.moe_ffn(*on(dev, x, logits, gate, up, down), k)
    logits[1, 5] = math.nan
    logits[2, 6] = math.inf
    x[4, 100] = math.nan
    gate[11], up[11], down[11] = math.nan, math.inf, math.nan
    out, experts, weights = (t.cpu() for t in mm.moe_ffn(*on(dev, x, logits, gate, up, down), k))
    assert int(experts[1, 0]) == 5 and int(experts[2, 0]) == 6
    assert weights[1].isnan().all() and weights[2].isnan().all()
    assert out[[1, 2, 4]].isnan().all()
    for t in (0, 3, 5):
        assert torch.equal(out[t], clean[0][t].cpu()) and torch.equal(weights[t], clean[2][t].cpu())
    # an infinite weight of an expert in use
    e = int(experts[0, 0])
    takers = (experts == e).any(1)
    down[e, 7, 3] = math.inf
    out2 = mm.moe_ffn(*on(dev, x, logits, gate, up, down), k)[0].cpu()
    assert not out2[takers][:, 7].isfinite().any()
    fine = ~takers & torch.tensor([True, False, False, True, False, True])
    assert torch.equal(out2[fine], out[fine])


def test_moe_ffn_sums_that_are_exact(dev):  # noqa: F811
    """Weights of 1 (one expert per token), gates far above zero (SiLU(g) = g to fp32) and
    whole numbers: outputs are the rounded exact sums."""
    T, E, H, I = 20, 6, 72, 136
    g = gen(8)
    x = torch.randint(0, 3, (T, H), generator=g).bfloat16()
    x[:, 0] = 1
    gate = torch.zeros((E, I, H)).bfloat16()
    gate[:, :, 0] = torch.randint(1, 5, (E, I), generator=g).bfloat16() * 64  # g = 64 .. 256: exp(-g) is below u
    up = torch.randint(-1, 2, (E, I, H), generator=g).bfloat16()
    down = torch.randint(-2, 3, (E, H, I), generator=g).bfloat16()
    logits = torch.randn((T, E), generator=g)
    out, experts, _ = mm.moe_ffn(*on(dev, x, logits, gate, up, down), 1)
    want = torch.zeros((T, H), dtype=torch.float64)
    for t in range(T):
        e = int(experts[t, 0])
        mid = (gate[e].double() @ x[t].double()) * (up[e].double() @ x[t].double())
        assert float(mid.abs().max()) < 2 ** 15
        want[t] = down[e].double() @ mid
    # the reciprocal instruction of 1 + 0 is 1
    assert torch.equal(out.cpu(), want.float().bfloat16())


def test_moe_ffn_without_terms(dev):  # noqa: F811
    x, logits, gate, up, down = on(dev, *inputs(5, 6, 64, 24, 2))
    out, experts, weights = mm.moe_ffn(x, logits, gate[:, :0].contiguous(), up[:, :0].contiguous(),
                                       down[:, :, :0].contiguous(), 2)
    assert (out == 0).all() and torch.equal(experts, mm.moe_ffn(x, logits, gate, up, down, 2)[1])
    assert torch.allclose(weights.sum(1), torch.ones(5, device=x.device))
    out, experts, weights = mm.moe_ffn(x, logits, gate, up, down, 0)
    assert (out == 0).all() and experts.shape == weights.shape == (5, 0)
    assert mm.moe_ffn(x[:0], logits[:0], gate, up, down, 2)[0].shape == (0, 64)
    with pytest.raises(binding.MMError, match="64 tokens"):
        mm.moe_ffn(x.repeat(13, 1), logits.repeat(13, 1), gate, up, down, 2)
    with pytest.raises(binding.MMError, match="top_k"):
        mm.moe_ffn(x, logits, gate, up, down, 7)


@pytest.mark.parametrize("T", [5, 40])
def test_moe_ffn_of_empty_sizes(dev, T):  # noqa: F811
    """No values per token, no experts at all, and experts so wide that only their count says no."""
    x, logits, gate, up, down = on(dev, *inputs(T, 6, 64, 24, 2))
    want = mm.moe_ffn(x, logits, gate, up, down, 2)
    out, experts, weights = mm.moe_ffn(x[:, :0].contiguous(), logits, gate[:, :, :0].contiguous(),
                                       up[:, :, :0].contiguous(), down[:, :0].contiguous(), 2)
    assert out.shape == (T, 0) and torch.equal(experts, want[1]) and torch.equal(weights, want[2])
    for H, I in ((64, 24), (4096, 2048)):
        wide = torch.ones((T, H), dtype=torch.bfloat16, device=dev)
        none = torch.empty((0, I, H), dtype=torch.bfloat16, device=dev)
        out, experts, _ = mm.moe_ffn(wide, logits[:, :0].contiguous(), none, none, none.reshape(0, H, I), 0)
        assert (out == 0).all() and out.shape == (T, H) and experts.shape == (T, 0)


@pytest.mark.parametrize("T", [3, 40])
def test_moe_ffn_keeps_inside_its_workspace(dev, T):  # noqa: F811
    E, H, I, k = 10, 136, 264, 3
    x, logits, gate, up, down = on(dev, *inputs(T, E, H, I, 12))
    want = mm.moe_ffn(x, logits, gate, up, down, k)
    nbytes = binding.moe_ffn_workspace_size(T, E, H, I, k)
    ws = torch.full((nbytes + 256,), 0xFF, dtype=torch.uint8, device=dev)
    out, experts, weights = (torch.empty_like(t) for t in want)
    binding.check(binding.load().mm_moe_ffn(
        x.data_ptr(), logits.data_ptr(), gate.data_ptr(), up.data_ptr(), down.data_ptr(), out.data_ptr(),
        experts.data_ptr(), weights.data_ptr(), T, E, H, I, k, 1, ws.data_ptr(), nbytes,
        torch.cuda.current_stream().cuda_stream), "mm_moe_ffn")
    assert all(torch.equal(a, b) for a, b in zip((out, experts, weights), want)) and bool((ws[nbytes:] == 0xFF).all())


def test_moe_ffn_past_32_bits(dev):  # noqa: F811
    """Weights of more than 2^32 bytes each: the last expert against the same alone."""
    T, E, H, I = 4, 150, 4096, 4096
    x, _, g1, u1, d1 = on(dev, *inputs(T, 1, H, I, 5))
    gate, up, down = (torch.zeros((E, I, H), dtype=torch.bfloat16, device=dev) for _ in range(3))
    gate[-1], up[-1], down[-1] = g1[0], u1[0], d1[0]
    logits = torch.zeros((T, E), device=dev)
    logits[:, -1] = 20.0
    out, experts, weights = mm.moe_ffn(x, logits, gate, up, down, 1)
    assert (experts == E - 1).all() and (weights == 1).all()
    assert torch.equal(out, mm.moe_ffn(x, logits[:, -1:].contiguous(), g1, u1, d1, 1)[0])


# ---- experts of several tokens and many weights ---------------------------------

# One and two blocks of 16 tokens to a group, steps per wave 2, 4 and 8, slices of I 1, 2 and 3, ragged
# H and I, an expert of more tokens than a group
LARGE = [(9, 2, 2056, 1032, 1), (33, 3, 1416, 2056, 2), (64, 8, 4088, 520, 1), (40, 5, 8192, 264, 1), (64, 4, 520, 4104, 3),
         (17, 4, 512, 8200, 1), (64, 1, 2600, 840, 1), (12, 3, 8184, 264, 2), (61, 16, 1032, 2040, 4), (64, 2, 4096, 512, 2),
         (40, 3, 8192, 264, 1), (12, 1, 8184, 264, 1), (16, 2, 4096, 2056, 1)]


@pytest.mark.parametrize("T,E,H,I,k", LARGE)
def test_moe_ffn_large(dev, T, E, H, I, k):  # noqa: F811
    args = inputs(T, E, H, I, T + E + H)
    out, intact = guarded((T, H), torch.bfloat16, dev)
    d = on(dev, *args)
    got = mm.moe_ffn(*d, k, out=out)
    intact()
    check(got, *args, k, True)
    for a, b in zip(got, mm.moe_ffn(*d, k)):
        assert torch.equal(a, b), "not reproducible"
    # padded rows, tokens of one expert, and one that all others have
    logits = args[1]
    logits[0] = logits[T // 2] = -math.inf
    logits[1, 1:] = -math.inf
    logits[2:T // 2, 0] = 16.0
    got = mm.moe_ffn(*on(dev, *args), k, False)
    check(got, *args, k, False)
    assert (got[0][[0, T // 2]] == 0).all() and (got[1][[0, T // 2]] == -1).all()
    assert int(got[1][1, 0]) == 0 and (got[1][1, 1:] == -1).all()
    logits[:] = -math.inf
    got = mm.moe_ffn(*on(dev, *args), k)
    assert (got[0] == 0).all() and (got[1] == -1).all() and (got[2] == 0).all()


@pytest.mark.parametrize("T,E,H,I", [(20, 5, 1032, 2056), (64, 4, 2056, 1032), (33, 6, 520, 4104)])
def test_moe_ffn_large_sums_that_are_exact(dev, T, E, H, I):  # noqa: F811
    """As above, with two thirds of the terms of the second layer zero so that the sums stay exact."""
    g = gen(T)
    x = torch.randint(0, 2, (T, H), generator=g).bfloat16()
    x[:, 0] = 1
    gate = torch.zeros((E, I, H)).bfloat16()
    gate[:, :, 0] = torch.randint(1, 3, (E, I), generator=g).bfloat16() * 64
    up = torch.zeros((E, I, H)).bfloat16()
    up[:, torch.arange(I), torch.arange(I) % H] = torch.randint(-1, 2, (E, I), generator=g).bfloat16()
    up[:, :, H - 1] += 1
    down = torch.randint(-1, 2, (E, H, I), generator=g).bfloat16()
    down[:, :, ::3] = 0
    logits = torch.randn((T, E), generator=g)
    out, experts, _ = mm.moe_ffn(*on(dev, x, logits, gate, up, down), 1)
    assert len(set(experts.flatten().tolist())) == E
    for t in range(T):
        e = int(experts[t, 0])
        mid = (gate[e].double() @ x[t].double()) * (up[e].double() @ x[t].double())
        assert float(down[e].double().abs().max()) * float(mid.abs().sum()) < 2 ** 24 * 64
        want = down[e].double() @ mid
        assert torch.equal(out[t].cpu(), want.float().bfloat16()), t


def test_moe_ffn_large_not_finite(dev):  # noqa: F811
    """A token's NaN, and weights that are not finite, reach the tokens that have them and no other;
    idle experts' weights are not in the sums."""
    T, E, H, I, k = 40, 7, 1032, 2056, 1
    x, logits, gate, up, down = inputs(T, E, H, I, 4)
    logits[:, 6] = -math.inf
    clean, experts, _ = (t.cpu() for t in mm.moe_ffn(*on(dev, x, logits, gate, up, down), k))
    x[4, 100] = math.nan
    gate[6], up[6], down[6] = math.nan, math.inf, math.nan
    e = int(experts[5, 0])
    down[e, 7, 3] = math.inf
    down[e, 9, I - 1] = math.nan
    gate[e, I - 1, H - 1] = math.nan
    out = mm.moe_ffn(*on(dev, x, logits, gate, up, down), k)[0].cpu()
    hit = experts[:, 0] == e
    assert out[hit].isnan().all() and out[4].isnan().all()
    hit[4] = True
    assert torch.equal(out[~hit], clean[~hit])


@pytest.mark.parametrize("T,E,H,I,k", [(20, 3, 1032, 2056, 2), (20, 5, 520, 8200, 1)])
def test_moe_ffn_large_keeps_inside_its_workspace(dev, T, E, H, I, k):  # noqa: F811
    x, logits, gate, up, down = on(dev, *inputs(T, E, H, I, 12))
    want = mm.moe_ffn(x, logits, gate, up, down, k)
    nbytes = binding.moe_ffn_workspace_size(T, E, H, I, k)
    ws = torch.full((nbytes + 256,), 0xFF, dtype=torch.uint8, device=dev)
    out, experts, weights = (torch.empty_like(t) for t in want)
    binding.check(binding.load().mm_moe_ffn(
        x.data_ptr(), logits.data_ptr(), gate.data_ptr(), up.data_ptr(), down.data_ptr(), out.data_ptr(),
        experts.data_ptr(), weights.data_ptr(), T, E, H, I, k, 1, ws.data_ptr(), nbytes,
        torch.cuda.current_stream().cuda_stream), "mm_moe_ffn")
    assert all(torch.equal(a, b) for a, b in zip((out, experts, weights), want)) and bool((ws[nbytes:] == 0xFF).all())


def test_moe_ffn_large_replays_from_a_graph(dev):  # noqa: F811
    """The experts of a replay are those of its own logits."""
    T, E, H, I, k = 24, 4, 1032, 2056, 2
    x, logits, gate, up, down = on(dev, *inputs(T, E, H, I, 31))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        mm.moe_ffn(x, logits, gate, up, down, k)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = mm.moe_ffn(x, logits, gate, up, down, k)
    for i in range(4):
        logits.copy_(randn(gen(100 + i), (T, E)))
        if i == 2:
            logits[3:] = -math.inf
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, mm.moe_ffn(x, logits, gate, up, down, k)):
            assert torch.equal(a, b), i
        torch.cuda.synchronize()


# ---- a decoder layer's step ----------------------------------------------------

def layer_inputs(dev, M, H, I, E):  # noqa: F811
    g = gen(M + H)
    p = {"x": randn(g, (M, H)), "res": randn(g, (M, H)), "w1": randn(g, H, 0.1, 1.0), "b1": randn(g, H, 0.1),
         "w2": randn(g, H, 0.1, 1.0), "b2": randn(g, H, 0.1), "W": randn(g, (H, H), H ** -0.5), "bias": randn(g, H),
         "A": randn(g, (5, 16, H), H ** -0.5), "B": randn(g, (5, H, 16), 0.1), "router": randn(g, (E, H), 2 * H ** -0.5),
         "gate": randn(g, (E, I, H), H ** -0.5), "up": randn(g, (E, I, H), H ** -0.5), "down": randn(g, (E, H, I), I ** -0.5)}
    p = {k: v.bfloat16().to(dev) for k, v in p.items()}
    p["scale"] = torch.rand(5, generator=g).to(dev) + 0.5
    p["index"] = torch.randint(-1, 5, (M,), generator=g, dtype=torch.int32).to(dev)
    return p


def layer(p):
    """One step: norm, a projection with the requests' adapters, norm, router and experts."""
    y, h, _, _ = mm.layer_norm(p["x"], p["w1"], p["b1"], p["res"])
    z = mm.linear_lora(y, p["W"], p["A"], p["B"], p["index"], p["scale"], p["bias"], "bias")
    y2, h2, mean, rstd = mm.layer_norm(z, p["w2"], p["b2"], h)
    logits = mm.matmul(y2, p["router"].t(), out_dtype=torch.float32)
    out, experts, weights = mm.moe_ffn(y2, logits, p["gate"], p["up"], p["down"], 2)
    dh, dw, db = mm.layer_norm_backward(out, h2, p["w2"], mean, rstd, z)
    return y, z, y2, h2, logits, out, experts, weights, dh, dw, db


@pytest.mark.parametrize("M", [1, 24, 64])
def test_layer_on_another_stream(dev, M):  # noqa: F811
    p = layer_inputs(dev, M, 520, 264, 8)
    want = layer(p)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = layer(p)
    side.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    # each operator against 64 bits, from what the one before it wrote
    y, z, y2, h2, logits, out, experts, weights, dh, dw, db = (t.cpu() for t in want)
    c = {k: v.cpu() for k, v in p.items()}
    sums = ref.lora(y, c["W"], c["A"], c["B"], c["index"], c["scale"]) + c["bias"].double()
    size = y.double().abs() @ c["W"].double().abs().t() + 20
    close(z, sums, BF16 * sums.abs() + 700 * U * size + 2.0 ** -15 * size, "projection")
    check((out, experts, weights), y2, logits, c["gate"], c["up"], c["down"], 2, True)


def test_layer_replays_from_a_graph(dev):  # noqa: F811
    p = layer_inputs(dev, 8, 520, 264, 8)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        layer(p)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = layer(p)
    for i in range(4):
        p["x"].copy_(randn(gen(100 + i), (8, 520)).bfloat16())
        p["index"].copy_(torch.randint(-1, 5, (8,), generator=gen(i), dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        want = layer(p)
        torch.cuda.synchronize()
        for a, b in zip(outs, want):
            assert torch.equal(a, b), i


def test_two_graphs_at_once_have_their_own_workspaces(dev):  # noqa: F811
    """Two captured steps replayed on two streams at the same time."""
    steps = []
    for M in (4, 50):
        p = layer_inputs(dev, M, 520, 264, 8)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            layer(p)
        side.synchronize()
        want = layer(p)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs = layer(p)
        steps.append((side, graph, outs, want, p))  # (a graph reads its inputs' memory: they stay)
    torch.cuda.synchronize()
    for _ in range(3):
        for side, graph, _, _, _ in steps:
            with torch.cuda.stream(side):
                for _ in range(5):
                    graph.replay()
    torch.cuda.synchronize()
    for _, _, outs, want, _ in steps:
        for a, b in zip(outs, want):
            assert torch.equal(a, b)
