"""The adapters' term of the linear layer with an adapter per row, on the GPU: what it
keeps between its two products, and what a row's bits depend on.
"""
import pytest
import torch

import dense_bf16_gemm_amd as mm
import layer_ref as ref
from dense_bf16_gemm_amd import binding
from test_gpu_decoder import dev, gen, guarded, same_class  # noqa: F401 (dev is a fixture)
from test_gpu_linear_lora import choices, inputs, on

pytestmark = pytest.mark.gpu

# rows in one launch with K whole (one and two blocks of 16) and with K in slices, up to 64, tiles with K
# whole and in slices; ranks whose parts end inside a step of 32 or 64
SHAPES = [(1, 70, 136, 8, 2), (9, 130, 1032, 24, 3), (16, 513, 4104, 16, 16), (30, 257, 2056, 72, 5), (32, 64, 4096, 256, 4),
          (5, 333, 8264, 40, 3), (32, 70, 4104, 16, 9), (64, 257, 1024, 32, 30), (50, 130, 2056, 136, 4), (65, 70, 200, 16, 3),
          (130, 515, 4104, 24, 3), (200, 517, 1032, 8, 12), (300, 300, 72, 72, 6), (513, 1030, 392, 64, 7), (2100, 2100, 328, 40, 8),
          (700, 3000, 1032, 16, 5), (260, 140, 136, 256, 3), (64, 10248, 136, 72, 5), (40, 10241, 2056, 64, 30)]


@pytest.mark.parametrize("M,N,K,R,L", SHAPES)
@pytest.mark.parametrize("how", ["mixed", "runs"])
def test_linear_lora_keeps_all_bits_between_the_products(dev, M, N, K, R, L, how):  # noqa: F811
    """Values s A x of 18 to 21 bits, neighbours of which differ by less than 2^10: B takes such
    differences, so that one held with fewer bits is off by whole numbers.  Everything is a
    whole number below 2^24, so outputs have to match bit for bit."""
    g = gen(M + N + K + R)

    def sparse(shape, top):
        """Whole numbers up to top, four or so of them along the last axis, the first and last two of it among them."""
        v = torch.randint(-top, top + 1, shape, generator=g)
        keep = torch.randint(0, max(1, shape[-1] // 2), shape, generator=g) == 0
        keep[..., 0] = keep[..., -1] = keep[..., -2] = True
        return (v * keep).float()

    x = torch.randint(-127, 128, (M, K), generator=g).float()
    x[:, :24] = torch.randint(64, 128, (M, 24), generator=g).float()
    W = sparse((N, K), 1)
    A = sparse((L, R, K), 255)
    A[:, :, :24] = 255.0  # (24 * 64 * 255 is 2^18.6)
    A[:, 1::2] = A[:, ::2]
    A[:, 1::2, -1] = torch.randint(-3, 4, (L, R // 2), generator=g) + A[:, 1::2, -1].clamp(-252, 252)
    A[:, ::2, -1] = A[:, ::2, -1].clamp(-252, 252)
    B = torch.zeros((L, N, R))
    pair = torch.randint(0, R // 2, (L, N, 1), generator=g)
    B.scatter_(2, 2 * pair, 1.0)
    B.scatter_(2, 2 * pair + 1, -1.0)
    scale = 2.0 ** torch.randint(0, 2, (L,), generator=g).float()
    bf = [t.bfloat16() for t in (x, W, A, B)]
    assert all(torch.equal(b.float(), t) for b, t in zip(bf, (x, W, A, B)))
    index = choices(M, L, how, g)
    index[0].clamp_(min=0)
    low = x.double() @ A.double().reshape(L * R, K).t()
    size = x.double().abs() @ A.double().abs().reshape(L * R, K).t()
    assert float(size.max()) * 2 < 2 ** 22 and float(low.abs().min()) > 2 ** 17 and bool((low.long() % 2 == 1).any())
    got = mm.linear_lora(*on(dev, *bf, index, scale)).cpu()
    want = ref.lora(*bf, index, scale)
    assert torch.equal(got, want.float().bfloat16())


# rows in one launch, in slices of K, up to 64, tiles with K whole (256 columns to a tile: many) and in slices
@pytest.mark.parametrize("M,N,K,R", [(5, 4096, 4096, 16), (16, 4096, 4096, 16), (16, 2048, 8192, 64), (30, 4096, 2056, 24),
                                     (32, 4096, 4096, 16), (12, 4096, 8264, 16), (32, 2048, 4104, 40), (40, 4096, 2056, 16),
                                     (64, 4096, 4096, 16), (90, 4096, 1032, 24), (300, 2100, 1032, 16), (600, 4096, 520, 40), (50, 10248, 520, 64)])
def test_linear_lora_row_does_not_depend_on_other_rows_adapters(dev, M, N, K, R):  # noqa: F811
    """The bits of a row stay when other rows take other adapters, more, fewer or none.

    All rows are one, and the bias takes off what a sum is to 8 bits: of what is left, a sum in
    another order changes bits that the output has."""
    L = min(M, 40)
    g = gen(M + K)
    x = torch.randn((1, K), generator=g).bfloat16().expand(M, K).contiguous()
    W = (torch.randn((N, K), generator=g) * K ** -0.5).bfloat16()
    A = (torch.randn((L, R, K), generator=g) * K ** -0.5).bfloat16()
    B = (torch.randn((L, N, R), generator=g) * R ** -0.5).bfloat16()
    A[1:], B[1:] = A[:1].clone(), B[:1].clone()  # (the same in all, so that one bias does for all)
    index = torch.arange(M, dtype=torch.int32) % L
    scale = torch.full((L,), 1.25)
    d = on(dev, x, W, A, B, index, scale)
    bias = -mm.linear_lora(*d)[0]
    want = mm.linear_lora(*d, bias, "bias")
    assert float((want != 0).float().mean()) > 0.9
    rows = torch.arange(M)
    for kept in (rows % 2 == 1, rows % 3 == 2, rows >= M - 2, rows >= M // 2):
        for others in (torch.full_like(index, -1), index.flip(0), (index * 7 + 3) % L, torch.zeros_like(index)):
            other = torch.where(kept, index, others).int().to(dev)
            got = mm.linear_lora(*d[:4], other, scale.to(dev), bias, "bias")
            assert torch.equal(got[kept.to(dev)], want[kept.to(dev)])


@pytest.mark.parametrize("M,N,K,R", [(1, 70, 64, 8), (9, 130, 1032, 24), (30, 70, 392, 40), (12, 130, 8264, 16), (32, 70, 4104, 8),
                                     (50, 200, 520, 40), (90, 130, 1032, 16), (150, 130, 520, 16), (300, 2100, 264, 72),
                                     (700, 3000, 1032, 16), (2100, 2100, 328, 8), (40, 10248, 264, 64)])
@pytest.mark.parametrize("epi", ["none", "gelu_tanh"])
def test_linear_lora_infinities_of_B(dev, M, N, K, R, epi):  # noqa: F811
    """An infinity in B gives its rows the infinity or NaN of the definition's sum, also where
    values of A x are whole numbers (whose further parts are 0) or exactly 0."""
    L = 4
    (x, W, A, B, index, scale), _ = inputs(M, N, K, R, L, "mixed", M + N, exact=True)
    index[0] = 1
    A[1, 0], A[1, 1] = 0, 0                             # exactly 0: 0 times an infinity is NaN
    A[2, 2] = 0
    A[2, 2, :4] = torch.tensor([1.0, 0.5, 0.25, 2.0])
    inf = float("inf")
    for a, n, r, v in ((1, 3, 0, inf), (1, 4, 3, inf), (1, 5, 3, -inf), (2, 6, 2, inf), (2, 7, 2, -inf), (0, N - 1, R - 1, inf),
                       (0, 8, 4, inf), (0, 8, 5, -inf), (3, 9, 1, inf), (3, 9, 6, inf), (3, 64, 7, -inf), (1, 64, 2, float("nan"))):
        B[a, n, r] = v
    if M > 8:
        # s A x itself infinite or NaN, by finite and infinite values of B
        index[3:6] = torch.tensor([3, 3, 0])
        x[3, 5], x[4, 6] = inf, -inf
        A[3, 1, 5], A[3, 6, 5], A[3, 1, 6] = 1.0, 1.0, 2.0
        A[0, 5, 7], W[11, 5] = inf, 0.0
    got = mm.linear_lora(*on(dev, x, W, A, B, index, scale), epilogue=epi).float().cpu()
    want = ref.lora(x, W, A, B, index, scale).float()
    assert want.isinf().any() and want.isnan().any()
    if epi == "gelu_tanh":  # t times 0 is NaN for minus infinity, here as in linear
        want = torch.where(want == -inf, float("nan"), want)
    same_class(got, want)
    if epi == "none":
        fine = want.isfinite()
        assert torch.equal(got[fine], want.bfloat16().float()[fine])


TILE_ROWS = 9224  # bytes of a tile's table: a count, 256 adapters, 256 masks of 256 rows


def up256(n):
    return -(-n // 256) * 256


# the last region of the workspace: sums of W x of slices of K (12 rows: two; 50, in one and in two; 90: tiles in five), or
# the tables of tiles with K whole (of 128 rows by 128 columns, and by 64)
@pytest.mark.parametrize("M,N,K,R,L,region", [(12, 300, 8264, 24, 4, 2 * 12 * 300 * 4), (50, 300, 2056, 24, 30, 2 * 50 * 300 * 4),
                                              (33, 130, 520, 8, 3, 33 * 130 * 4), (90, 300, 1032, 24, 4, 5 * 90 * 300 * 4),
                                              (200, 14336, 4096, 40, 150, "128"), (300, 2100, 264, 8, 300, "128")])
def test_linear_lora_stays_inside_its_workspace(dev, M, N, K, R, L, region):  # noqa: F811
    """The bytes behind the reported workspace stay as they were, its last region is written, and a
    workspace full of NaN serves as well as any."""
    args, _ = inputs(M, N, K, R, L, "mixed", 5)
    d = on(dev, *args)
    want = mm.linear_lora(*d)
    nbytes = binding.linear_lora_workspace_size(M, N, K, R, L)
    ws = torch.full((nbytes + 4096,), 0xFF, dtype=torch.uint8, device=dev)
    out, intact = guarded((M, N), torch.bfloat16, dev)
    binding.check(binding.load().mm_linear_lora(*(t.data_ptr() for t in d), None, out.data_ptr(), M, N, K, R, L, 0,
                                                ws.data_ptr(), nbytes, torch.cuda.current_stream().cuda_stream),
                  "mm_linear_lora")
    assert torch.equal(out, want) and bool((ws[nbytes:] == 0xFF).all())
    intact()
    if region == "128":
        tiles = -(-M // 128)
        table = ws[nbytes - up256(tiles * TILE_ROWS):][:tiles * TILE_ROWS].reshape(tiles, TILE_ROWS)
        for t in range(tiles):
            mine = args[4][128 * t:128 * (t + 1)]
            first = list(dict.fromkeys(a for a in mine.tolist() if a >= 0))  # in the order of their first rows
            got = table[t].cpu()
            assert int(got[:4].view(torch.int32)) == len(first)
            assert got[4:4 + 4 * len(first)].view(torch.int32).tolist() == first
    else:
        sums = ws[nbytes - up256(region):nbytes][:region].view(torch.float32)
        assert bool(sums.isfinite().all())
