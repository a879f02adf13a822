"""Layer norm and its gradient on the GPU against the 64-bit forms.

Tolerances count roundings (u = 2^-24 in fp32, half a step of the output's type at
the end), not observed errors; each is derived where it is used.
"""
import pytest
import torch

import dense_bf16_gemm_amd as mm
import layer_ref as ref
from test_gpu_decoder import BF16, U, close, dev, gen, guarded, randn  # noqa: F401 (dev is a fixture)

pytestmark = pytest.mark.gpu

# a sum of `hidden` values: at most 32 sequential and 6 + 16 joining additions, one
# operation for each term, then the division, eps and the root
NORM_U = 64 * U
SHAPES = [(1, 8), (1, 8192), (3, 64), (5, 520), (300, 1032), (257, 2048), (130, 4096), (261, 5000), (2, 16384),
          (259, 16392), (3, 32768)]


def inputs(rows, hidden, dtype, residual, seed, shift=0.0):
    g = gen(seed)
    x = randn(g, (rows, hidden), 0.5, shift).to(dtype)
    res = randn(g, (rows, hidden), 2.0).to(dtype) if residual else None
    return x, randn(g, hidden, 0.3, 1.0).bfloat16(), randn(g, hidden, 0.5).bfloat16(), res


def on(dev, *ts):  # noqa: F811
    return [None if t is None else t.to(dev) for t in ts]


def check_norm(got, want, w, b):
    y, h, mean, rstd = got
    wh, wm, wr, wy = want
    assert torch.equal(h.cpu().double(), wh)
    size = wh.abs().mean(1)
    close(mean, wm, NORM_U * size, "mean")
    # the mean's error moves every difference by as much: relative to their spread, by rstd
    off = NORM_U * size * wr
    close(rstd, wr, (NORM_U + off + off * off) * wr, "rstd")
    n = (wh - wm[:, None]).abs() * wr[:, None]
    tol = (n * (NORM_U + off[:, None] + 4 * U) + off[:, None]) * w.double().abs() * (1 + BF16)
    close(y, wy, BF16 * wy.abs() + tol + 2 * U * (b.double().abs() if b is not None else 0.0), "y")


@pytest.mark.parametrize("rows,hidden", SHAPES)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("bias", [False, True])
def test_layer_norm(dev, rows, hidden, dtype, residual, bias):  # noqa: F811
    x, w, b, res = inputs(rows, hidden, dtype, residual, rows + hidden)
    b = b if bias else None
    got = mm.layer_norm(*on(dev, x, w, b, res), eps=1e-5)
    assert got[0].dtype == torch.bfloat16 and got[2].dtype == got[3].dtype == torch.float32
    check_norm(got, ref.norm(x, w, b, res, 1e-5), w, b)


@pytest.mark.parametrize("hidden", [512, 8192])
def test_layer_norm_of_rows_far_from_zero(dev, hidden):  # noqa: F811
    """A mean 4000 times the spread: mean(h^2) - mean^2 in fp32 would leave nothing
    of the variance, the squares of differences leave all of it."""
    x, w, b, _ = inputs(33, hidden, torch.float32, False, hidden, shift=2000.0)
    got = mm.layer_norm(*on(dev, x, w, b), eps=1e-5)
    check_norm(got, ref.norm(x, w, b, None, 1e-5), w, b)


def test_layer_norm_in_place_strided_and_written_where_told(dev):  # noqa: F811
    g = gen(3)
    wide = randn(g, (37, 1200)).bfloat16().to(dev)
    x = wide[:, 8:8 + 1032]  # row stride 1200
    w, b = randn(g, (2, 1032)).bfloat16().to(dev)
    res = randn(g, (37, 1032)).bfloat16().to(dev)
    want = mm.layer_norm(x.contiguous(), w, b, res)
    for a, c in zip(mm.layer_norm(x, w, b, res), want):
        assert torch.equal(a, c)
    into, intact = guarded((37, 1032), torch.bfloat16, dev)
    y, h, _, _ = mm.layer_norm(x, w, b, res, h=into)
    intact()
    assert h is into and torch.equal(h, want[1]) and torch.equal(y, want[0])
    keep = res.clone()
    y, h, _, _ = mm.layer_norm(x, w, b, keep, h=keep)  # the residual stream updated in place
    assert h is keep and torch.equal(keep, want[1]) and torch.equal(y, want[0])
    xc = x.contiguous()
    y, h, _, _ = mm.layer_norm(xc, w, b, res, h=xc)
    assert torch.equal(xc, want[1]) and torch.equal(y, want[0])
    with pytest.raises(ValueError, match="only with a residual"):
        mm.layer_norm(xc, w, b, h=xc)


def test_layer_norm_rows_of_one_value_and_not_finite(dev):  # noqa: F811
    x = torch.randn((6, 264), generator=gen(1))
    x[0] = 0.0
    x[1] = 3.0
    x[2, 5] = float("nan")
    x[3, 7] = float("inf")
    x[4, 9] = -float("inf")
    w, b = torch.ones((2, 264)).bfloat16().to(dev)
    for dtype in (torch.bfloat16, torch.float32):
        y, _, mean, rstd = (t.float().cpu() for t in mm.layer_norm(x.to(dtype).to(dev), w, b, eps=1e-6))
        for row in (0, 1):  # no spread: the bias
            assert torch.equal(y[row], torch.ones(264)) and abs(float(rstd[row]) - 1e3) < 1e3 * NORM_U
        assert y[2:5].isnan().all() and rstd[2:5].isnan().all()
        assert mean[2].isnan() and float(mean[3]) == float("inf") and float(mean[4]) == -float("inf")
        assert y[5].isfinite().all()


def test_layer_norm_empty(dev):  # noqa: F811
    w = torch.ones(64, device=dev).bfloat16()
    e = torch.empty((0, 64), device=dev)
    y, h, mean, rstd = mm.layer_norm(e, w)
    assert y.shape == (0, 64) and mean.shape == rstd.shape == (0,)
    dh, dw, db = mm.layer_norm_backward(e.bfloat16(), e, w, mean, rstd)
    assert dh.shape == (0, 64) and torch.equal(dw, torch.zeros(64, device=dev)) and torch.equal(db, dw)
    n = torch.empty((3, 0), device=dev)
    y, h, mean, rstd = mm.layer_norm(n, w[:0], eps=0.25)
    assert y.shape == (3, 0) and mean.tolist() == [0.0] * 3 and rstd.tolist() == [2.0] * 3
    dh, dw, db = mm.layer_norm_backward(n.bfloat16(), n, w[:0], mean, rstd)
    assert dh.shape == (3, 0) and dw.shape == db.shape == (0,)


def grad_inputs(rows, hidden, dtype, dres, device, seed):
    g = torch.Generator(device=device).manual_seed(seed)

    def rn(shape, std=1.0, mean=0.0):
        return torch.randn(shape, generator=g, device=device) * std + mean

    h = rn((rows, hidden), 2.0, 0.5).to(dtype)
    dy = rn((rows, hidden)).bfloat16()
    w = rn(hidden, 0.3, 1.0).bfloat16()
    d = rn((rows, hidden)).to(dtype) if dres else None
    hd = h.double()
    return dy, h, w, hd.mean(1).float(), (hd.var(1, correction=0) + 1e-6).rsqrt().float(), d


def check_grad(dev, args, got):  # noqa: F811
    dy, h, w, mean, rstd, d = args
    rows, dtype = h.shape[0], h.dtype
    dh, dw, db = ref.norm_grad(*args)
    assert got[0].dtype == dtype and got[1].dtype == got[2].dtype == torch.float32
    # mean(g), mean(g n): sums as above with two products each; then six roundings of
    # the terms they meet, and the output's
    r = rstd.double()[:, None]
    gg, n = (dy.double() * w.double()).abs(), (h.double() - mean.double()[:, None]).abs() * r
    terms = r * (gg + gg.mean(1, keepdim=True) + n * (gg * n).mean(1, keepdim=True)) + (d.double().abs() if d is not None else 0)
    half = torch.finfo(dtype).eps / 2
    close(got[0], dh.cpu(), (half * dh.abs() + NORM_U * terms).cpu(), "dh")
    # every row is added once, in some order of at most rows + 40 steps
    close(got[1], dw.cpu(), ((rows + 40) * U * (dy.double().abs() * n).sum(0)).cpu(), "dweight")
    close(got[2], db.cpu(), ((rows + 40) * U * dy.double().abs().sum(0)).cpu(), "dbias")


@pytest.mark.parametrize("rows,hidden", [(1, 8), (2, 2056), (700, 520), (1500, 1024), (2048, 64), (300, 4096), (37, 5000),
                                         (9, 16384), (5, 16392), (3, 32768), (2049, 64), (2049, 520), (2050, 4096),
                                         (2300, 5000), (2049, 8192), (2051, 16384), (2049, 16392)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("dres", [False, True])
def test_layer_norm_backward(dev, rows, hidden, dtype, dres):  # noqa: F811
    """Both sides of the row count from which the gradient is two launches."""
    args = grad_inputs(rows, hidden, dtype, dres, dev, rows * 7 + hidden)
    got = mm.layer_norm_backward(*args)
    check_grad(dev, args, got)
    for a, b in zip(got, mm.layer_norm_backward(*args)):
        assert torch.equal(a, b), "not reproducible"
    if dres:
        buf = args[5].clone()
        inplace = mm.layer_norm_backward(*args[:5], buf, out=buf)
        assert inplace[0] is buf and all(torch.equal(a, b) for a, b in zip(got, inplace))
    into, intact = guarded((rows, hidden), dtype, dev)
    mm.layer_norm_backward(*args, out=into)
    intact()
    assert torch.equal(into, got[0])


def test_layer_norm_gradient_by_differences(dev):  # noqa: F811
    """The gradient of sum(cy y) + sum(ch h) along a random direction of every input
    against the 64-bit forward form's central difference."""
    rows, hidden, eps, step = 6, 264, 1e-3, 1e-4
    g = gen(2)
    x, res, cy, ch = (randn(g, (rows, hidden)) for _ in range(4))
    w, b = randn(g, (2, hidden), 0.3, 1.0).bfloat16()
    cy = cy.bfloat16()
    _, h, mean, rstd = mm.layer_norm(*on(dev, x, w, b, res), eps=eps)
    dh, dw, db = (t.double().cpu() for t in mm.layer_norm_backward(*on(dev, cy), h, w.to(dev), mean, rstd, ch.to(dev)))
    # h is x + res rounded once: the forms differentiate there
    base = [h.double().cpu(), w.double(), b.double(), torch.zeros((rows, hidden), dtype=torch.float64)]
    for at, grad in ((0, dh), (1, dw), (2, db)):
        v = torch.randn(grad.shape, generator=g, dtype=torch.float64)
        values = [ref.norm_loss(*(t + sign * step * v if i == at else t for i, t in enumerate(base)), eps, cy.double(),
                                ch.double()) for sign in (1, -1)]
        want = (values[0] - values[1]) / (2 * step)
        # fp32 gradients: 2^-17 of the terms they add; the difference's own error, a
        # third derivative (some 10 per element) times step^2 / 6
        size = float((grad.abs() * v.abs()).sum()) * 2.0 ** -17 + 10 * rows * hidden * step ** 2
        assert abs(float((grad * v).sum()) - float(want)) <= size, at


def test_layer_norm_past_32_bits(dev):  # noqa: F811
    """More than 2^32 bytes of stream: the last rows equal the same rows alone."""
    rows, hidden = 68000, 32768
    x = torch.zeros((rows, hidden), dtype=torch.bfloat16, device=dev)
    tail = randn(gen(4), (5, hidden)).bfloat16().to(dev)
    x[-5:] = tail
    w, b = (randn(gen(5), (2, hidden)).bfloat16().to(dev))
    got = mm.layer_norm(x, w, b)
    want = mm.layer_norm(tail, w, b)
    assert torch.equal(got[0][-5:], want[0]) and torch.equal(got[2][-5:], want[2]) and torch.equal(got[3][-5:], want[3])
    del got
    dy = torch.zeros_like(x)
    dy[-5:] = tail.flip(0)
    mean, rstd = torch.zeros(rows, device=dev), torch.ones(rows, device=dev)
    mean[-5:], rstd[-5:] = want[2], want[3]
    dh, dw, db = mm.layer_norm_backward(dy, x, w, mean, rstd)
    few = mm.layer_norm_backward(tail.flip(0).contiguous(), tail, w, want[2], want[3])
    assert torch.equal(dh[-5:], few[0]) and bool((dh[0] == 0).all())
    # (the same five terms in another order)
    size = ((tail.flip(0).double().abs() * ((tail.double() - want[2].double()[:, None]) * want[3].double()[:, None]).abs()).sum(0))
    close(dw, few[1].double().cpu(), (16 * U * size).cpu(), "dweight")
    close(db, few[2].double().cpu(), (16 * U * tail.double().abs().sum(0)).cpu(), "dbias")
