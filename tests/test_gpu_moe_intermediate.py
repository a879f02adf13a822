"""What stands between the two layers of the mixture-of-experts FFN, on the GPU.

Whole numbers make every sum exact, so outputs have to match bit for bit.
"""
import pytest
import torch

import dense_bf16_gemm_amd as mm
from test_gpu_decoder import dev, gen, same_class  # noqa: F401 (dev is a fixture)

pytestmark = pytest.mark.gpu

# One, several and 64 tokens; the output's columns on one workgroup and on several; experts of several
# tokens with one and two blocks of 16 tokens to a group, slices of I, ragged sizes
SHAPES = [(1, 8, 256, 512), (5, 3, 72, 200), (8, 4, 4104, 72), (17, 12, 264, 136), (64, 64, 72, 1032), (64, 9, 1032, 264),
          (20, 5, 1032, 2056), (64, 4, 2056, 1032), (33, 2, 520, 4104), (64, 2, 4096, 512), (12, 1, 8184, 264),
          (40, 3, 2600, 3208), (40, 8, 4104, 2056)]


@pytest.mark.parametrize("T,E,H,I", SHAPES)
def test_moe_ffn_keeps_all_bits_between_the_layers(dev, T, E, H, I):  # noqa: F811
    """Products g u of up to 19 bits, which the second layer takes in differences of
    neighbours: a value held with fewer bits is off by whole numbers.

    One expert per token has weight 1, gates of 64 and more have SiLU(g) = g in fp32
    (exp(-64) is below half a step of 1, and the reciprocal of 1 is 1).  Row n of the second layer has 8
    pairs of +1 and -1, so every partial sum stays below 16 * 2^19 = 2^23."""
    g = gen(T + H + I)
    x = torch.zeros((T, H))
    x[:, 0] = 3.0
    x[:, H - 1] = torch.randint(1, 3, (T,), generator=g).float()
    gate, up = torch.zeros((E, I, H)), torch.zeros((E, I, H))
    gate[:, :, 0] = torch.randint(64, 256, (E, I), generator=g).float()   # g = 192 .. 765
    up[:, :, H - 1] = torch.randint(-255, 256, (E, I), generator=g).float()  # u = -510 .. 510
    down = torch.zeros((E, H, I))
    for e in range(E):
        at = torch.randint(0, I // 2, (H, 8), generator=g)
        down[e].scatter_(1, 2 * at, 1.0)
        down[e].scatter_(1, 2 * at + 1, -1.0)
    logits = torch.randn((T, E), generator=g)
    args = [t.bfloat16() for t in (x, gate, up, down)]
    assert all(torch.equal(a.float(), t) for a, t in zip(args, (x, gate, up, down)))
    d = [t.to(dev) for t in (args[0], logits, *args[1:])]
    out, experts, weights = (t.cpu() for t in mm.moe_ffn(*d, 1))
    assert (weights == 1).all()
    wide = 0
    for e in set(experts[:, 0].tolist()):
        rows = (experts[:, 0] == e).nonzero().flatten()
        mid = (x[rows, :1] * gate[e, :, 0]).double() * (x[rows, H - 1:] * up[e, :, H - 1]).double()
        assert float(mid.abs().max()) < 2 ** 19
        wide += int((mid.abs() >= 2 ** 17).logical_and(mid.long() % 2 == 1).sum())
        want = mid @ down[e].double().t()
        assert torch.equal(out[rows], want.float().bfloat16()), e
    assert wide  # (products that 16 bits do not hold)


@pytest.mark.parametrize("T,E,H,I", [(1, 3, 256, 512), (5, 3, 72, 200), (8, 4, 4104, 72), (17, 12, 264, 136), (64, 6, 1032, 264),
                                     (20, 2, 1032, 2056), (64, 4, 2056, 1032), (33, 2, 520, 4104), (40, 8, 4104, 2056)])
@pytest.mark.parametrize("k", [1, 2])
def test_moe_ffn_infinities_of_W_down(dev, T, E, H, I, k):  # noqa: F811
    """An infinity in W_down gives the tokens of its expert the infinity or NaN of the definition's
    sum, also where what it meets is a whole number (whose further parts are 0) or exactly 0."""
    g = gen(T + H + I + k)
    x = torch.zeros((T, H))
    x[:, 0] = torch.randint(1, 4, (T,), generator=g).float()
    x[:, 1] = torch.randint(0, 2, (T,), generator=g) * 2.0 - 1.0
    gate, up = torch.zeros((E, I, H)), torch.zeros((E, I, H))
    gate[:, :, 0] = torch.randint(64, 100, (E, I), generator=g).float()
    up[:, :, 1] = torch.randint(-3, 4, (E, I), generator=g).float()  # zeros among them
    up[:, 3, 1], up[:, 5, 1], up[:, I - 1, 1] = 0.0, 2.0, -3.0
    down = torch.randint(-1, 2, (E, H, I), generator=g).float()
    inf = float("inf")
    for n, i, v in ((0, 5, inf), (1, 5, -inf), (2, I - 1, inf), (3, 3, inf), (H - 1, I - 1, -inf), (17, 8, inf), (40, 8, -inf)):
        down[0, n, i] = v
    down[1, 4, 5], down[1, 4, I - 1] = inf, inf   # of two signs: NaN
    down[1, 6, 7] = float("nan")
    down[E - 1, 5, 5] = inf
    logits = torch.randn((T, E), generator=g)
    logits[0] = torch.arange(E).float().flip(0)
    logits[T // 2] = -inf if T > 1 else logits[0]
    args = [t.bfloat16() for t in (x, gate, up, down)]
    d = [t.to(dev) for t in (args[0], logits, *args[1:])]
    out, experts, weights = (t.cpu() for t in mm.moe_ffn(*d, k))
    want = torch.zeros((T, H), dtype=torch.float64)
    for t in range(T):
        for j, e in enumerate(experts[t].tolist()):
            if e >= 0:
                mid = weights[t, j].double() * (gate[e, :, 0] * x[t, 0]).double() * (up[e, :, 1] * x[t, 1]).double()
                want[t] += (down[e].double() * mid).sum(1)
    assert not want.isfinite().all()
    same_class(out.float(), want.float())
    if k == 1:  # (weights of 1: whole numbers)
        fine = want.isfinite()
        assert torch.equal(out[fine], want.float().bfloat16()[fine])
