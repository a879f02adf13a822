"""The decoder-layer operators on the GPU against their 64-bit forms.

Tolerances count roundings (u = 2^-24 in fp32, half a step of the output's
type at the end), not observed errors; each is derived where it is used.
Inputs of whole numbers and powers of two make every intermediate exact, and
such outputs have to match bit for bit.
"""
import pytest
import torch

import dense_bf16_gemm_amd as mm
import decoder_ref as ref
from dense_bf16_gemm_amd import binding

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
BF16 = torch.finfo(torch.bfloat16).eps / 2
E4M3 = torch.finfo(torch.float8_e4m3fn).eps / 2


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch.device("cuda:0")


def gen(seed):
    return torch.Generator().manual_seed(seed)


def randn(g, shape, std=1.0, mean=0.0):
    return torch.randn(shape, generator=g) * std + mean


def guarded(shape, dtype, dev):
    """A contiguous tensor inside a buffer whose other bytes are 0x5a, and a
    check that they still are."""
    n = 1
    for s in shape:
        n *= s
    size = n * torch.empty(0, dtype=dtype).element_size()
    buf = torch.full((size + 512,), 0x5A, dtype=torch.uint8, device=dev)
    t = buf[256:256 + size].view(dtype).view(shape)

    def intact():
        assert bool((buf[:256] == 0x5A).all()) and bool((buf[256 + size:] == 0x5A).all()), "write out of bounds"

    return t, intact


def close(got, want, tol, what):
    got = got.double().cpu()
    err = (got - want).abs() - tol
    assert not torch.isnan(got).any(), what
    assert float(err.max()) <= 0, (what, float(err.max()), float((got - want).abs().max()))


# ---- RMS norm ---------------------------------------------------------------

NORM = [(1, 8), (1, 8192), (3, 64), (5, 520), (300, 1032), (257, 2048), (130, 4096), (261, 5000), (2, 16384),
        (259, 16392), (3, 32768)]


def norm_inputs(rows, hidden, dtype, residual, seed):
    g = gen(seed)
    x = randn(g, (rows, hidden), 0.5).to(dtype)
    res = randn(g, (rows, hidden), 2.0).to(dtype) if residual else None
    return x, randn(g, hidden, 0.3, 1.0).bfloat16(), res


# a sum of squares of `hidden` values: at most 32 sequential and 6 + 16 joining
# additions and one squaring each, then the mean, eps, root and reciprocal
NORM_U = 64 * U


@pytest.mark.parametrize("rows,hidden", NORM)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("residual", [False, True])
def test_rms_norm(dev, rows, hidden, dtype, residual):
    x, w, res = norm_inputs(rows, hidden, dtype, residual, rows + hidden)
    rd = res.to(dev) if residual else None
    y, h, rstd = mm.rms_norm(x.to(dev), w.to(dev), rd, eps=1e-5)
    q, scale, h2 = mm.rms_norm_q8(x.to(dev), w.to(dev), rd, eps=1e-5)
    wh, wr, wy = ref.norm(x, w, res, 1e-5)
    assert y.dtype == torch.bfloat16 and q.dtype == torch.float8_e4m3fn and scale.dtype == torch.float32
    assert torch.equal(h.cpu().double(), wh) and torch.equal(h2.cpu().double(), wh)
    close(rstd, wr, NORM_U * wr, "rstd")
    close(y, wy, (BF16 + 2 * NORM_U) * wy.abs(), "y")
    ws = (wy.abs().amax(1) / ref.E4M3_MAX).clamp_min(ref.TINY)
    close(scale, ws, 2 * NORM_U * ws, "scale")
    # e4m3: half a step, relative above 2^-6 and 2^-10 below
    val = q.float().cpu().double() * scale.cpu().double()[:, None]
    tol = (E4M3 + 4 * NORM_U) * wy.abs() + 2.0 ** -10 * ws[:, None]
    close(val, wy, tol, "q")


@pytest.mark.parametrize("hidden", [4096, 8192])
def test_rms_norm_rstd_is_mostly_the_nearest(dev, hidden):
    """A sum in fp32 and one rounding after it leave most rows' rstd the nearest
    fp32 value; a square root and a division, each rounded, left 61 %."""
    x = randn(gen(hidden), (4096, hidden), 2.0).bfloat16().to(dev)
    _, _, rstd = mm.rms_norm(x, torch.ones(hidden, device=dev).bfloat16())
    want = (1.0 / (x.double().square().mean(1) + 1e-6).sqrt()).float()
    assert float((rstd == want).float().mean()) >= 0.7


@pytest.mark.parametrize("rows,hidden", [(1, 8192), (64, 4096), (300, 1032), (5, 16384)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_rms_norm_q8_codes_are_the_rounded_quotients(dev, rows, hidden, dtype):
    """scale and q bit for bit from the fp32 y: max|y| / 448 and y / scale, each
    rounded once.  (Quotients at the border of two codes are common, since the
    values have few bits: a product with a rounded 1 / scale misses some.)"""
    x, w, res = norm_inputs(rows, hidden, dtype, True, rows + hidden)
    for weight in (w, w.clone().index_fill_(0, torch.tensor([3]), float("inf"))):
        args = on(dev, x, weight, res)
        _, h, rstd = mm.rms_norm(*args)
        q, scale, _ = mm.rms_norm_q8(*args)
        y = h.float().cpu() * rstd.cpu()[:, None] * weight.float()
        want = (y.abs().amax(1) / ref.E4M3_MAX).clamp_min(ref.TINY)
        assert torch.equal(scale.cpu(), want)
        codes = (y / want[:, None]).to(torch.float8_e4m3fn).float().nan_to_num(1000.0)
        assert int((q.float().cpu().nan_to_num(1000.0) != codes).sum()) == 0


def test_rms_norm_in_place_strided_and_written_where_told(dev):
    g = gen(3)
    wide = randn(g, (37, 1200)).bfloat16().to(dev)
    x = wide[:, 8:8 + 1032]  # row stride 1200
    w = randn(g, 1032).bfloat16().to(dev)
    res = randn(g, (37, 1032)).bfloat16().to(dev)
    y0, h0, r0 = mm.rms_norm(x.contiguous(), w, res)
    y1, h1, r1 = mm.rms_norm(x, w, res)
    assert torch.equal(y0, y1) and torch.equal(h0, h1) and torch.equal(r0, r1)
    into, intact = guarded((37, 1032), torch.bfloat16, dev)
    _, h2, _ = mm.rms_norm(x, w, res, h=into)
    intact()
    assert h2 is into and torch.equal(h2, h0)
    keep = res.clone()
    y3, h3, _ = mm.rms_norm(x, w, keep, h=keep)  # the residual stream updated in place
    assert h3 is keep and torch.equal(keep, h0) and torch.equal(y3, y0)
    xc = x.contiguous()
    q, s, h4 = mm.rms_norm_q8(xc, w, res, h=xc)
    assert torch.equal(xc, h0)
    q0, s0, _ = mm.rms_norm_q8(x, w, res)
    assert torch.equal(q.view(torch.uint8), q0.view(torch.uint8)) and torch.equal(s, s0)


def test_rms_norm_rows_of_zeros_and_not_finite(dev):
    x = torch.ones((6, 264))
    x[0] = 0.0
    x[1, 5] = float("nan")
    x[2, 7] = float("inf")
    x[3, 9] = -float("inf")
    x[4] = 1e-30
    w = torch.ones(264).bfloat16().to(dev)
    for dtype in (torch.bfloat16, torch.float32):
        xd = x.to(dtype).to(dev)
        y, _, rstd = mm.rms_norm(xd, w)
        q, s, _ = mm.rms_norm_q8(xd, w)
        y, q, rstd, s = y.float().cpu(), q.float().cpu(), rstd.cpu(), s.cpu()
        assert torch.equal(y[0], torch.zeros(264)) and torch.equal(q[0], torch.zeros(264))
        assert float(s[0]) == 2.0 ** -126 and abs(float(rstd[0]) - 1e3) < 1e3 * NORM_U
        assert y[1].isnan().all() and q[1].isnan().all() and s[1].isnan() and rstd[1].isnan()
        for row, at in ((2, 7), (3, 9)):  # 1 / inf = 0: zeros, and inf * 0 = NaN
            assert float(rstd[row]) == 0.0 and y[row, at].isnan()
            assert int(y[row].isnan().sum()) == 1 and float(y[row].nan_to_num().abs().max()) == 0.0
            assert s[row].isnan() and q[row].isnan().all()
        assert (y[5] == 1.0).all() and (q[5] == 448.0).all()
    # eps = 0 and a row of zeros: 0 * inf
    y, _, rstd = mm.rms_norm(torch.zeros((2, 8), device=dev), w[:8].contiguous(), eps=0.0)
    assert y.isnan().all() and rstd.isinf().all()


def test_rms_norm_empty(dev):
    w = torch.ones(64, device=dev).bfloat16()
    y, h, rstd = mm.rms_norm(torch.empty((0, 64), device=dev).bfloat16(), w)
    assert y.shape == (0, 64) and rstd.shape == (0,)
    e = torch.empty((0, 64), device=dev)
    dh, dw = mm.rms_norm_backward(e.bfloat16(), e, w, torch.empty(0, device=dev))
    assert dh.shape == (0, 64) and torch.equal(dw, torch.zeros(64, device=dev))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("residual", [False, True])
def test_rms_norm_of_no_values(dev, dtype, residual):
    """Rows without values: the mean of none is 0, the largest of none is 0."""
    x = torch.empty((300, 0), dtype=dtype, device=dev)
    res = x.clone() if residual else None
    w = torch.empty(0, dtype=torch.bfloat16, device=dev)
    for _ in range(3):
        junk = torch.full((300,), float("nan"), device=dev)  # what the statistics' memory may hold
        del junk
        y, h, rstd = mm.rms_norm(x, w, res, eps=0.25)
        assert y.shape == h.shape == (300, 0) and rstd.dtype == torch.float32
        assert torch.equal(rstd, torch.full((300,), 2.0, device=dev))
        del rstd
        junk = torch.full((300,), float("nan"), device=dev)
        del junk
        q, scale, h = mm.rms_norm_q8(x, w, res)
        assert q.shape == (300, 0) and torch.equal(scale, torch.full((300,), ref.TINY, device=dev))
        bias = torch.ones(24, device=dev).bfloat16()
        W = torch.empty((24, 0), device=dev).to(torch.float8_e4m3fn)
        out = mm.linear_q8(q, scale, W, torch.ones(24, device=dev), bias, "bias")
        assert torch.equal(out, bias.expand(300, 24))
        del scale
    _, _, rstd = mm.rms_norm(x, w, eps=0.0)
    assert rstd.isposinf().all()
    dh, dw = mm.rms_norm_backward(torch.empty((300, 0), device=dev).bfloat16(), x, w, rstd, res)
    assert dh.shape == (300, 0) and dw.shape == (0,)


@pytest.mark.parametrize("rows,hidden", [(1, 8), (2, 2056), (700, 520), (1500, 1024), (2200, 64), (300, 4096),
                                         (37, 5000), (9, 16384), (5, 16392), (3, 32768)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("dres", [False, True])
def test_rms_norm_backward(dev, rows, hidden, dtype, dres):
    g = gen(rows * 7 + hidden)
    h = randn(g, (rows, hidden), 2.0).to(dtype)
    dy = randn(g, (rows, hidden)).bfloat16()
    w = randn(g, hidden, 0.3, 1.0).bfloat16()
    d = randn(g, (rows, hidden)).to(dtype) if dres else None
    rstd = torch.rsqrt(h.float().square().mean(1) + 1e-6)
    got, gw = mm.rms_norm_backward(dy.to(dev), h.to(dev), w.to(dev), rstd.to(dev), d.to(dev) if dres else None)
    dh, dw = ref.norm_grad(dy, h, w, rstd, d)
    assert got.dtype == dtype and gw.dtype == torch.float32
    # mean(g n): 32 sequential + 22 joining additions, two products each;
    # then six roundings of the terms it meets, and the output's
    r = rstd.double()[:, None]
    gg, n = (dy.double() * w.double()).abs(), h.double().abs() * r
    terms = r * (gg + n * (gg * n).mean(1, keepdim=True)) + (d.double().abs() if dres else 0.0)
    half = torch.finfo(dtype).eps / 2
    close(got, dh, half * dh.abs() + NORM_U * terms, "dh")
    # dweight: every row is added once, in some order of at most rows + 32 steps
    close(gw, dw, (rows + 40) * U * (dy.double().abs() * n).sum(0), "dweight")
    again, gw2 = mm.rms_norm_backward(dy.to(dev), h.to(dev), w.to(dev), rstd.to(dev), d.to(dev) if dres else None)
    assert torch.equal(again, got) and torch.equal(gw, gw2), "not reproducible"
    if dres:
        buf = d.to(dev)
        inplace, _ = mm.rms_norm_backward(dy.to(dev), h.to(dev), w.to(dev), rstd.to(dev), buf, out=buf)
        assert inplace is buf and torch.equal(buf, got)


@pytest.mark.parametrize("rows,hidden", [(2048, 1032), (2049, 64), (2049, 520), (2050, 4096), (3100, 5000), (2049, 8192),
                                         (2051, 16384), (2049, 16392), (2055, 32768)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("dres", [False, True])
def test_rms_norm_backward_many_rows(dev, rows, hidden, dtype, dres):
    """Both sides of the row count from which the gradient is two launches;
    the 64-bit form runs on the GPU."""
    g = torch.Generator(device=dev).manual_seed(rows + hidden)
    h = (torch.randn((rows, hidden), generator=g, device=dev) * 2.0).to(dtype)
    dy = torch.randn((rows, hidden), generator=g, device=dev).bfloat16()
    w = (torch.randn(hidden, generator=g, device=dev) * 0.3 + 1.0).bfloat16()
    d = torch.randn((rows, hidden), generator=g, device=dev).to(dtype) if dres else None
    rstd = torch.rsqrt(h.float().square().mean(1) + 1e-6)
    got, gw = mm.rms_norm_backward(dy, h, w, rstd, d)
    dh, dw = ref.norm_grad(dy, h, w, rstd, d)
    # (tolerances as in test_rms_norm_backward)
    r = rstd.double()[:, None]
    gg, n = (dy.double() * w.double()).abs(), h.double().abs() * r
    terms = r * (gg + n * (gg * n).mean(1, keepdim=True)) + (d.double().abs() if dres else 0.0)
    off = (got.double() - dh).abs() - (torch.finfo(dtype).eps / 2 * dh.abs() + NORM_U * terms)
    assert float(off.max()) <= 0, float(off.max())
    off = (gw.double() - dw).abs() - (rows + 40) * U * (dy.double().abs() * n).sum(0)
    assert float(off.max()) <= 0, float(off.max())
    again, gw2 = mm.rms_norm_backward(dy, h, w, rstd, d)
    assert torch.equal(again, got) and torch.equal(gw, gw2), "not reproducible"


@pytest.mark.parametrize("rows,hidden", [(2049, 64), (2051, 520), (3100, 4096), (2500, 8192), (2049, 16392)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_rms_norm_backward_many_rows_in_place(dev, rows, hidden, dtype):
    """dh over dres, with counts of rows that leave workgroups with one row fewer than others."""
    g = torch.Generator(device=dev).manual_seed(rows)
    h, d = (torch.randn((rows, hidden), generator=g, device=dev).to(dtype) for _ in range(2))
    dy = torch.randn((rows, hidden), generator=g, device=dev).bfloat16()
    w = torch.randn(hidden, generator=g, device=dev).bfloat16()
    rstd = torch.rsqrt(h.float().square().mean(1) + 1e-6)
    dh, dw = mm.rms_norm_backward(dy, h, w, rstd, d)
    into, dw2 = mm.rms_norm_backward(dy, h, w, rstd, d, out=d)
    assert into is d and torch.equal(d, dh) and torch.equal(dw2, dw)


def test_rms_norm_past_32_bits(dev):
    """rows * hidden past 2^31 elements: the last rows against the same rows alone."""
    rows, hidden = 66000, 32768
    x = torch.zeros((rows, hidden), dtype=torch.bfloat16, device=dev)
    x[-3:] = randn(gen(1), (3, hidden)).bfloat16().to(dev)
    w = randn(gen(2), hidden).bfloat16().to(dev)
    y, _, rstd = mm.rms_norm(x, w)
    want, _, wr = mm.rms_norm(x[-3:].contiguous(), w)
    assert torch.equal(rstd[-3:], wr)
    close(y[-3:], want.double().cpu(), 2 * BF16 * want.double().abs().cpu(), "last rows")


@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("q8", [False, True])
def test_rms_norm_of_more_rows_than_a_launch_takes(dev, residual, q8):
    """64 threads a row: 2^26 rows are 2^32 threads."""
    rows, hidden, tail = (1 << 26) + 3, 8, 1000
    x = torch.zeros((rows, hidden), dtype=torch.bfloat16, device=dev)
    x[-tail:] = randn(gen(1), (tail, hidden)).bfloat16().to(dev)
    x[0] = x[-1]
    res = torch.ones_like(x) if residual else None
    w = randn(gen(2), hidden).bfloat16().to(dev)
    fn = mm.rms_norm_q8 if q8 else mm.rms_norm
    got = fn(x, w, res)
    want = fn(x[-tail:].contiguous(), w, res[-tail:].contiguous() if residual else None)
    for g, e in zip(got, want):
        g, e = (t.float() if t.dtype == torch.float8_e4m3fn else t for t in (g[-tail:], e))
        assert torch.equal(g, e)
    same = [t.float() if t.dtype == torch.float8_e4m3fn else t for t in (got[0][0], got[0][-1])]
    assert torch.equal(*same)
    # rows of zeros (of ones with the residual), the same all along
    middle = got[1][1:rows - tail]
    assert bool((middle == middle[0]).all())


# ---- products with 4-bit weights -------------------------------------------

def w4_inputs(M, N, K, group, zeros, seed, exact=False):
    g = gen(seed)
    codes = torch.randint(0, 16, (N, K), generator=g, dtype=torch.uint8)
    groups = -(-K // group)
    z = torch.randint(0, 16, (groups, N), generator=g, dtype=torch.uint8) if zeros else None
    if exact:  # whole numbers and powers of two: every sum is exact in fp32
        x = torch.randint(-2, 3, (M, K), generator=g).bfloat16()
        s = (2.0 ** torch.randint(-2, 3, (groups, N), generator=g)).bfloat16()
    else:
        x = randn(g, (M, K)).bfloat16()
        s = (randn(g, (groups, N), 0.3, 1.0) * K ** -0.5).bfloat16()
    return x, codes, s, z, randn(g, N).bfloat16()


def on(dev, *ts):
    return [None if t is None else t.to(dev) for t in ts]


@pytest.mark.parametrize("N,K", [(1, 8), (16, 128), (33, 136), (257, 1000), (16, 4096)])
def test_pack_w4(dev, N, K):
    codes = torch.randint(0, 16, (N, K), generator=gen(N + K), dtype=torch.uint8)
    assert torch.equal(mm.pack_w4(codes.to(dev)).cpu(), ref.pack(codes))


W4 = [(1, 16, 128), (1, 1, 8), (1, 4096, 2048), (2, 65, 136), (5, 130, 1000), (15, 100, 520), (16, 333, 1024),
      (17, 47, 2056), (32, 129, 640), (33, 64, 384), (37, 3001, 264), (64, 515, 1280), (65, 70, 256),
      (200, 97, 392), (1, 16421, 264), (4, 9001, 1160), (16, 16450, 264), (13, 9001, 392), (30, 16421, 136),
      (32, 9001, 1160), (64, 16450, 136), (50, 9001, 264)]


@pytest.mark.parametrize("M,N,K", W4)
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("zeros", [False, True])
def test_linear_w4_exact(dev, M, N, K, group, zeros):
    """Whole-number operands: every partial sum is a multiple of 1/4 below
    2^22, so fp32 holds it and the result is the rounded exact sum."""
    x, codes, s, z, _ = w4_inputs(M, N, K, group, zeros, M + N + K, exact=True)
    out, intact = guarded((M, N), torch.bfloat16, dev)
    xd, sd, zd = on(dev, x, s, z)
    got = mm.linear_w4(xd, mm.pack_w4(codes.to(dev)), sd, zd, group=group, out=out)
    intact()
    want = (x.double() @ ref.w4_weight(codes, s, z, group).t()).float().bfloat16()
    assert torch.equal(got.cpu(), want)


@pytest.mark.parametrize("M,N,K", [(65, 70, 8), (65, 100, 64), (71, 50, 8), (66, 64, 16), (129, 67, 392),
                                   (193, 97, 4104), (257, 130, 1032)])
@pytest.mark.parametrize("group", [32, 64, 128])
def test_linear_w4_few_rows_in_the_last_block(dev, M, N, K, group):
    """Blocks of 64 rows, few in the last, and a K that ends in the first half
    of a step: the second half's copies lie past all of the block's rows."""
    x, codes, s, z, _ = w4_inputs(M, N, K, group, True, M + N + K, exact=True)
    out, intact = guarded((M, N), torch.bfloat16, dev)
    xd, sd, zd = on(dev, x, s, z)
    got = mm.linear_w4(xd, mm.pack_w4(codes.to(dev)), sd, zd, group=group, out=out)
    intact()
    want = (x.double() @ ref.w4_weight(codes, s, z, group).t()).float().bfloat16()
    assert torch.equal(got.cpu(), want)


@pytest.mark.parametrize("M,N,K,group,zeros,epi", [
    (1, 4096, 4096, 128, False, "none"), (3, 1001, 4104, 32, True, "bias"), (16, 512, 8192, 64, True, "gelu_tanh"),
    (31, 300, 2000, 128, True, "bias_gelu_tanh"), (64, 257, 4096, 64, False, "bias_gelu_tanh"),
    (100, 130, 1032, 32, True, "none")])
def test_linear_w4(dev, M, N, K, group, zeros, epi):
    x, codes, s, z, bias = w4_inputs(M, N, K, group, zeros, M * 3 + N)
    xd, sd, zd, bd = on(dev, x, s, z, bias)
    W = mm.pack_w4(codes.to(dev))
    # what pads N and K may hold anything
    if N % 16:
        W.view(W.shape[0], W.shape[1], 4, 16, 16)[-1, :, :, N % 16:] = 0xFF
    got = mm.linear_w4(xd, W, sd, zd, bd if "bias" in epi else None, epi, group=group)
    w = ref.w4_weight(codes, s, z, group)
    want, t = ref.epilogue(x.double() @ w.t(), bias, epi)
    # the sums run over x (16 + code) and (16 + zero) sum x: at most 128 + 8
    # additions in a group, one per group and wave, 8 waves
    at = torch.arange(K) // group
    zz = 8.0 if z is None else z.t().double()[:, at]
    size = (codes.double() + 32.0 + zz) * s.double().abs().t()[:, at]
    acc = (160 + K // group) * U * (x.double().abs() @ size.t())
    # GELU: slope at most 1.13; its exponential and reciprocal 1e-5 of |t|
    close(got, want, BF16 * want.abs() + 1.14 * acc + 1e-5 * t.abs(), epi)
    again = mm.linear_w4(xd, W, sd, zd, bd if "bias" in epi else None, epi, group=group)
    assert torch.equal(got, again), "not reproducible"


def same_class(got, want):
    assert torch.equal(got.isnan(), want.isnan())
    inf = want.isinf()
    assert torch.equal(got.isinf(), inf) and torch.equal(got[inf], want[inf])


@pytest.mark.parametrize("M", [3, 20, 40])
def test_linear_w4_not_finite(dev, M):
    """Infinite and NaN activations give each output the class of the sum."""
    x, codes, s, z, _ = w4_inputs(M, 70, 392, 64, True, 9)
    codes[codes == 8] = 9  # some weights are zero only where z says so
    x[0, 3] = float("inf")
    x[1, 200] = -float("inf")
    x[2, 5], x[2, 390] = float("nan"), 1.0
    got = mm.linear_w4(*on(dev, x), mm.pack_w4(codes.to(dev)), *on(dev, s, z), group=64).float().cpu()
    want = x.double() @ ref.w4_weight(codes, s, z, 64).t()
    same_class(got[:3], want[:3].float())
    assert got[3:].isfinite().all()


@pytest.mark.parametrize("M", [2, 30, 64])
def test_linear_w4_sums_that_only_the_offset_form_overflows(dev, M):
    """x (16 + code) passes fp32's range where x (code - zero) does not, and an
    infinite scale takes its own column alone."""
    N, K, group = 70, 392, 64
    x, codes, s, z, _ = w4_inputs(M, N, K, group, True, 12, exact=True)
    x[1] = 0.0
    x[1, 3], x[1, 390] = 2.0 ** 125, -2.0 ** 124
    codes[:, 3], codes[:, 390] = 9, 12
    z[0], z[6] = 8, 7
    s[0], s[6] = 2.0, 0.5
    s[2, 5] = float("inf")
    got = mm.linear_w4(*on(dev, x), mm.pack_w4(codes.to(dev)), *on(dev, s, z), group=group).cpu()
    want = (x.double() @ ref.w4_weight(codes, s, z, group).t()).float().bfloat16()
    same_class(got.float(), want.float())
    fine = want.isfinite()
    assert fine[1].sum() == N - 1 and torch.equal(got[fine], want[fine])


@pytest.mark.parametrize("rows", ["one", "all"])
@pytest.mark.parametrize("what", ["a NaN", "NaN", "an infinity", "infinities"])
def test_linear_w4_not_finite_takes_no_hundredfold(dev, rows, what):
    """Padded rows may hold anything: a call whose outputs are not finite takes
    longer, but by no orders of magnitude (here at most 25 times and 1 ms)."""
    M, N, K = 16, 8192, 8192
    W = torch.randint(0, 256, (N // 16, K // 128, 1024), generator=gen(32), dtype=torch.uint8).to(dev)
    x = randn(gen(33), (M, K)).bfloat16()
    s = (randn(gen(34), (K // 128, N), 0.3, 1.0) * K ** -0.5).bfloat16().to(dev)
    bad = x.clone()
    value = float("nan") if "NaN" in what else float("inf")
    for row in ([M - 1] if rows == "one" else range(M)):
        bad[row, slice(None) if what in ("NaN", "infinities") else 17 * row + 5] = value

    def median(t):
        times = []
        for _ in range(6):
            start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            start.record()
            mm.linear_w4(t, W, s)
            end.record()
            end.synchronize()
            times.append(start.elapsed_time(end))
        return sorted(times[1:])[2]

    fine, slow = median(x.to(dev)), median(bad.to(dev))
    print(f"{fine * 1e3:.0f} us, not finite {slow * 1e3:.0f} us")
    assert slow <= 25 * fine and slow <= 1.0


def test_linear_w4_empty(dev):
    bias = randn(gen(1), 40).bfloat16().to(dev)
    s = torch.ones((0, 40), device=dev).bfloat16()
    W = torch.empty((3, 0, 1024), dtype=torch.uint8, device=dev)
    got = mm.linear_w4(torch.empty((5, 0), device=dev).bfloat16(), W, s, None, bias, "bias")
    assert torch.equal(got, bias.expand(5, 40))
    x, codes, s, z, _ = w4_inputs(1, 40, 128, 128, False, 1)
    assert mm.linear_w4(torch.empty((0, 128), device=dev).bfloat16(), mm.pack_w4(codes.to(dev)),
                        s.to(dev)).shape == (0, 40)


def test_linear_w4_past_32_bits(dev):
    """A weight of 5 GB: the last columns against the same rows alone."""
    N, K = 300016, 32768
    W = torch.zeros((N // 16, K // 128, 1024), dtype=torch.uint8, device=dev)
    tail = torch.randint(0, 256, (3, K // 128, 1024), generator=gen(4), dtype=torch.uint8).to(dev)
    W[-3:] = tail
    s = torch.full((K // 128, N), 2.0 ** -8, device=dev).bfloat16()
    x = randn(gen(5), (2, K)).bfloat16().to(dev)
    got = mm.linear_w4(x, W, s)
    want = mm.linear_w4(x, tail.contiguous(), s[:, -48:].contiguous())
    assert torch.equal(got[:, -48:], want)


def test_pack_w4_of_more_words_than_a_launch_takes(dev):
    """A packed weight past 16 GiB (2^32 words, a thread each)."""
    N, K = (1 << 21) + 16, 1 << 14
    codes = torch.zeros((N, K), dtype=torch.uint8, device=dev)
    tail = torch.randint(0, 16, (16, K), generator=gen(6), dtype=torch.uint8).to(dev)
    codes[-16:] = tail
    codes[:16] = tail
    packed = mm.pack_w4(codes)
    want = mm.pack_w4(tail)[0]
    assert torch.equal(packed[0], want) and torch.equal(packed[-1], want)
    assert not bool(packed[1:-1].view(torch.int64).any())


@pytest.mark.parametrize("M,N,K", [(1431655777, 3, 8), (65535 * 64 + 70, 20, 128)])
def test_linear_w4_of_more_rows_than_a_launch_takes(dev, M, N, K):
    """Few columns: a thread per output.  Otherwise 65535 blocks of 64 rows."""
    _, codes, s, z, bias = w4_inputs(1, N, K, 32, True, 9)
    x = torch.zeros((M, K), dtype=torch.bfloat16, device=dev)
    tail = randn(gen(7), (200, K)).bfloat16().to(dev)
    x[-200:] = tail
    x[:200] = tail
    W = mm.pack_w4(codes.to(dev))
    args = (*on(dev, s, z, bias), "bias", 32)
    got = mm.linear_w4(x, W, *args)
    want = mm.linear_w4(tail, W, *args)
    assert torch.equal(got[-200:], want) and torch.equal(got[:200], want)
    assert torch.equal(got[200:-200].amax(0), bias.to(dev)) and torch.equal(got[200:-200].amin(0), bias.to(dev))


# ---- products of e4m3 operands ---------------------------------------------

def q8_inputs(M, N, K, seed, exact=False):
    g = gen(seed)
    if exact:
        x = torch.randint(-4, 5, (M, K), generator=g).float()
        W = torch.randint(-4, 5, (N, K), generator=g).float()
        xs, ws = 2.0 ** torch.randint(-2, 3, (M,), generator=g), 2.0 ** torch.randint(-2, 3, (N,), generator=g)
    else:
        x, W = randn(g, (M, K), 60.0), randn(g, (N, K), 60.0)
        xs, ws = randn(g, M, 0.1, 1.0), randn(g, N, 0.1, 1.0) * (K ** -0.5 / 3600)
    return (x.clamp(-448, 448).to(torch.float8_e4m3fn), xs.float(), W.clamp(-448, 448).to(torch.float8_e4m3fn),
            ws.float(), randn(g, N).bfloat16())


Q8 = [(1, 1, 16), (1, 64, 128), (1, 3001, 2048), (2, 65, 144), (7, 130, 1008), (16, 333, 1024), (17, 47, 2064),
      (32, 129, 640), (33, 64, 384), (64, 515, 1280), (65, 128, 256), (100, 200, 16), (128, 128, 128),
      (129, 131, 400), (255, 257, 1040), (256, 256, 1024), (300, 700, 272), (513, 300, 528), (700, 1030, 640),
      # K cut into chunks (the last one shorter, and ragged)
      (70, 1001, 4096), (130, 300, 4112), (256, 512, 1296), (1000, 520, 2064),
      # each kind of tile, several tiles per workgroup, ragged edges
      (2050, 2056, 144), (3000, 4100, 272), (1030, 9001, 400)]


@pytest.mark.parametrize("M,N,K", Q8)
def test_linear_q8_exact(dev, M, N, K):
    """Whole-number operands, power-of-two scales: the result is the rounded exact sum."""
    x, xs, W, ws, _ = q8_inputs(M, N, K, M + N + K, exact=True)
    out, intact = guarded((M, N), torch.bfloat16, dev)
    got = mm.linear_q8(*on(dev, x, xs, W, ws), out=out)
    intact()
    want = ((x.double() @ W.double().t()) * xs.double()[:, None] * ws.double()).float().bfloat16()
    assert torch.equal(got.cpu(), want)


@pytest.mark.parametrize("M,N,K", [
    # 256 x 256 tiles whole and in chunks, 256 x 128, 128 x 128 with short and with
    # long rings, 128 x 64
    (129, 36981, 144), (144, 10898, 9344), (142, 21458, 144), (11208, 70, 8368), (79, 33206, 144), (67, 16681, 5248),
    (16393, 66, 144), (6389, 69, 3360), (67, 71, 144), (71, 66, 1616),
    # few rows by a wide weight
    (33, 11000, 272), (64, 14001, 1040), (47, 33000, 144)])
def test_linear_q8_every_tile_exact(dev, M, N, K):
    x, xs, W, ws, _ = q8_inputs(M, N, K, M + N + K, exact=True)
    out, intact = guarded((M, N), torch.bfloat16, dev)
    got = mm.linear_q8(*on(dev, x, xs, W, ws), out=out)
    intact()
    # (sums of at most 16 K: exact in fp32)
    want = ((x.float() @ W.float().t()) * xs[:, None] * ws).bfloat16()
    assert torch.equal(got.cpu(), want)


def test_linear_q8_without_a_workspace(dev):
    """The same product uncut: equal to fp32 rounding, here exactly (whole numbers)."""
    M, N, K = 130, 300, 4112
    x, xs, W, ws, _ = q8_inputs(M, N, K, 6, exact=True)
    assert binding.linear_q8_workspace_size(M, N, K) > 0
    args = on(dev, x, xs, W, ws)
    out = torch.empty((M, N), dtype=torch.bfloat16, device=dev)
    binding.check(binding.load().mm_linear_q8(*(t.data_ptr() for t in args), None, out.data_ptr(), M, N, K, 0, None, 0,
                                              torch.cuda.current_stream().cuda_stream), "mm_linear_q8")
    assert torch.equal(out, mm.linear_q8(*args))


@pytest.mark.parametrize("M,N,K,epi", [
    (1, 2048, 4096, "none"), (5, 1001, 4112, "bias"), (16, 512, 8192, "gelu_tanh"), (40, 300, 2000, "bias_gelu_tanh"),
    (130, 257, 4096, "bias_gelu_tanh"), (256, 512, 1024, "bias"), (300, 515, 1040, "none"),
    (1000, 2100, 4112, "gelu_tanh")])
def test_linear_q8(dev, M, N, K, epi):
    x, xs, W, ws, bias = q8_inputs(M, N, K, M * 3 + N)
    args = on(dev, x, xs, W, ws)
    b = bias.to(dev) if "bias" in epi else None
    got = mm.linear_q8(*args, b, epi)
    xd, wd = x.double(), W.double()
    scale = xs.double()[:, None] * ws.double()
    want, t = ref.epilogue((xd @ wd.t()) * scale, bias, epi)
    # 128 products and sums per instruction, one instruction per 128 k, 8
    # waves' parts; a sum may be truncated (a whole step, 2 U), then two scales
    acc = (128 + K // 128 + 12) * 2 * U * (xd.abs() @ wd.abs().t()) * scale.abs() + 4 * U * t.abs()
    close(got, want, BF16 * want.abs() + 1.14 * acc + 1e-5 * t.abs(), epi)
    assert torch.equal(got, mm.linear_q8(*args, b, epi)), "not reproducible"


@pytest.mark.parametrize("M", [4, 20, 70, 300])
def test_linear_q8_not_finite(dev, M):
    x, xs, W, ws, _ = q8_inputs(M, 70, 400, 11)
    nan = torch.tensor(float("nan"))
    x[0, 7] = nan.to(torch.float8_e4m3fn)
    xs[1], xs[2] = float("inf"), float("nan")
    W[5, 399] = nan.to(torch.float8_e4m3fn)
    got = mm.linear_q8(*on(dev, x, xs, W, ws)).float().cpu()
    want = (x.double() @ W.double().t()) * xs.double()[:, None] * ws.double()
    same_class(got, want.float())


def test_linear_q8_empty(dev):
    bias = randn(gen(1), 48).bfloat16().to(dev)
    for M in (5, 200):
        got = mm.linear_q8(torch.empty((M, 0), device=dev).to(torch.float8_e4m3fn), torch.ones(M, device=dev),
                           torch.empty((48, 0), device=dev).to(torch.float8_e4m3fn), torch.ones(48, device=dev),
                           bias, "bias")
        assert torch.equal(got, bias.expand(M, 48))


def test_linear_q8_of_no_k_and_more_rows_than_a_launch_takes(dev):
    M, N = 65535 * 64 + 70, 20
    bias = randn(gen(1), N).bfloat16().to(dev)
    got = mm.linear_q8(torch.empty((M, 0), device=dev).to(torch.float8_e4m3fn), torch.ones(M, device=dev),
                       torch.empty((N, 0), device=dev).to(torch.float8_e4m3fn), torch.ones(N, device=dev), bias, "bias")
    assert torch.equal(got.amax(0), bias) and torch.equal(got.amin(0), bias)


@pytest.mark.parametrize("M", [2, 130])
def test_linear_q8_past_32_bits(dev, M):
    """A weight of 4.6 GB: the last columns against the same rows alone."""
    N, K = 140010, 32768
    W = torch.zeros((N, K), dtype=torch.uint8, device=dev)
    tail = q8_inputs(1, 40, K, 3)[2].to(dev)
    W[-40:] = tail.view(torch.uint8)
    W = W.view(torch.float8_e4m3fn)
    x, xs, _, _, _ = on(dev, *q8_inputs(M, 1, K, 4))
    ws = torch.full((N,), 2.0 ** -12, device=dev)
    got = mm.linear_q8(x, xs, W, ws)
    want = mm.linear_q8(x, xs, tail, ws[-40:].contiguous())
    assert torch.equal(got[:, -40:], want)


# ---- streams, graphs, the operators together --------------------------------

def block(x, res, w_norm, up, down, bias):
    """A decoder layer's MLP as it is served: norm to 8 bits, an 8-bit product
    with bias and GELU, a 4-bit product back to the stream."""
    q, scale, h = mm.rms_norm_q8(x, w_norm, res)
    mid = mm.linear_q8(q, scale, up[0], up[1], bias, "bias_gelu_tanh")
    return mm.linear_w4(mid, down[0], down[1], down[2], group=64), h


def block_inputs(dev, M, H, F):
    g = gen(M + H + F)
    x, res = (randn(g, (M, H)).bfloat16().to(dev) for _ in range(2))
    w = randn(g, H, 0.1, 1.0).bfloat16().to(dev)
    _, _, W, ws, bias = q8_inputs(1, F, H, 21)
    _, codes, s, z, _ = w4_inputs(1, H, F, 64, True, 22)
    return x, res, w, on(dev, W, ws), [mm.pack_w4(codes.to(dev)), *on(dev, s, z)], bias.to(dev), codes


@pytest.mark.parametrize("M", [1, 20, 150])
def test_operators_together_on_another_stream(dev, M):
    x, res, w, up, down, bias, codes = block_inputs(dev, M, 512, 1280)
    y0, h0 = block(x, res, w, up, down, bias)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        y1, h1 = block(x, res, w, up, down, bias)
    side.synchronize()
    assert torch.equal(y0, y1) and torch.equal(h0, h1)
    # against 64 bits, from the 8-bit values the norm wrote
    q, scale, _ = mm.rms_norm_q8(x, w, res)
    mid = mm.linear_q8(q, scale, up[0], up[1], bias, "bias_gelu_tanh").cpu()
    want = mid.double() @ ref.w4_weight(codes, down[1].cpu(), down[2].cpu(), 64).t()
    size = (codes.double() + 47.0) * down[1].cpu().double().abs().t()[:, torch.arange(1280) // 64]
    close(y0, want, BF16 * want.abs() + 200 * U * (mid.double().abs() @ size.t()), "block")


def test_operators_replay_from_a_graph(dev):
    x, res, w, up, down, bias, _ = block_inputs(dev, 8, 512, 1280)
    dy = randn(gen(8), (8, 512)).bfloat16().to(dev)

    def step():
        y, h = block(x, res, w, up, down, bias)
        z, _, rstd = mm.rms_norm(y, w, h)
        dh, dw = mm.rms_norm_backward(dy, h, w, rstd, z)
        return y, h, z, dh, dw

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
    for i in range(4):
        x.copy_(randn(gen(100 + i), (8, 512)).bfloat16())
        graph.replay()
        torch.cuda.synchronize()
        want = step()
        torch.cuda.synchronize()
        for a, b in zip(outs, want):
            assert torch.equal(a, b), i
