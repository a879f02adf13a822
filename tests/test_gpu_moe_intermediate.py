"""What stands between the two layers of the mixture-of-experts FFN, on the GPU.

Whole numbers make every sum exact, so outputs have to match bit for bit.
"""
import pytest
import torch

import dense_bf16_gemm_amd as mm
from test_gpu_decoder import dev, gen  # noqa: F401 (dev is a fixture)

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
