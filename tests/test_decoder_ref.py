"""Pins of the 64-bit forms the decoder operators are tested against, and the
host-side refusals of those operators (CPU only: no test here launches a
kernel or passes validation with a pointer that is not real device memory)."""
import ctypes

import pytest
import torch

import dense_bf16_gemm_amd as mm
import decoder_ref as ref
from dense_bf16_gemm_amd import binding

P = [0x10000000 * (i + 1) for i in range(12)]  # fake, never dereferenced
NULL = None
INVALID, UNSUPPORTED, MISALIGNED = (binding.MM_ERR_INVALID_VALUE, binding.MM_ERR_UNSUPPORTED,
                                    binding.MM_ERR_MISALIGNED)


@pytest.fixture(scope="module")
def lib():
    return binding.load()


def test_gradient_is_the_forward_forms_by_differences():
    gen = torch.Generator().manual_seed(5)
    r, n = 3, 16
    x, res, cy, ch = (torch.randn((r, n), generator=gen, dtype=torch.float64) for _ in range(4))
    w = torch.randn(n, generator=gen, dtype=torch.float64)
    eps = 1e-3
    h = x + res
    rstd = 1.0 / torch.sqrt((h * h).mean(1) + eps)
    dh, dw = ref.norm_grad(cy, h, w, rstd, ch)
    step = 1e-5

    def diff(t, i):
        a, b = t.clone(), t.clone()
        a.view(-1)[i] += step
        b.view(-1)[i] -= step
        return a, b

    for i in range(r * n):
        a, b = diff(x, i)
        d = (ref.norm_loss(a, w, res, eps, cy, ch) - ref.norm_loss(b, w, res, eps, cy, ch)) / (2 * step)
        assert abs(d - dh.view(-1)[i]) < 1e-8
        a, b = diff(res, i)
        d = (ref.norm_loss(x, w, a, eps, cy, ch) - ref.norm_loss(x, w, b, eps, cy, ch)) / (2 * step)
        assert abs(d - dh.view(-1)[i]) < 1e-8
    for i in range(n):
        a, b = diff(w, i)
        d = (ref.norm_loss(x, a, res, eps, cy, ch) - ref.norm_loss(x, b, res, eps, cy, ch)) / (2 * step)
        assert abs(d - dw[i]) < 1e-8


def test_pack_by_hand():
    codes = torch.zeros((17, 136), dtype=torch.uint8)
    codes[3, 41] = 5     # k = 32 + 8 + 1: word (g=1, n=3, j=1), nibble 4
    codes[16, 130] = 9   # second block of rows and of k: k = 2, word (0, 0, 0), nibble 1
    packed = ref.pack(codes)
    assert packed.shape == (2, 2, 1024)
    assert packed[0, 0, ((16 * 1 + 3) * 4 + 1) * 4 + 2] == 5
    assert packed[1, 1, 0] == 9 << 4
    assert int((packed != 0).sum()) == 2


def test_weight_of_codes():
    codes = torch.tensor([[0, 15, 8, 3] * 16])
    scales = torch.tensor([[2.0], [0.5]]).bfloat16()
    w = ref.w4_weight(codes, scales, None, 32)
    assert w[0, :4].tolist() == [-16.0, 14.0, 0.0, -10.0] and w[0, 32:36].tolist() == [-4.0, 3.5, 0.0, -2.5]
    w = ref.w4_weight(codes, scales, torch.tensor([[3], [0]], dtype=torch.uint8), 32)
    assert w[0, :4].tolist() == [-6.0, 24.0, 10.0, 0.0] and w[0, 32:36].tolist() == [0.0, 7.5, 4.0, 1.5]


def norm(lib, fn="mm_rms_norm", x=P[0], ld=64, res=P[1], w=P[2], h=P[3], y=P[4], stat=P[5], rows=4, hidden=64,
         eps=1e-6, dtype=0):
    return getattr(lib, fn)(x, ld, res, w, h, y, stat, rows, hidden, eps, dtype, None)


@pytest.mark.parametrize("fn", ["mm_rms_norm", "mm_rms_norm_q8"])
def test_norm_refusals(lib, fn):
    for bad in (dict(x=NULL), dict(w=NULL), dict(y=NULL), dict(stat=NULL), dict(h=NULL), dict(rows=-1),
                dict(hidden=-8), dict(eps=-1.0), dict(eps=float("nan")), dict(dtype=2), dict(ld=56),
                dict(y=P[0]), dict(y=P[1] + 16), dict(h=P[0] + 16), dict(h=P[1] + 128), dict(h=P[2]),
                dict(stat=P[0]), dict(y=P[3]), dict(stat=P[4] + 4),
                dict(h=P[0], ld=72)):
        assert norm(lib, fn, **bad) == INVALID, bad
    for bad in (dict(hidden=60), dict(ld=68), dict(x=P[0] + 8), dict(w=P[2] + 2), dict(y=P[4] + 8),
                dict(stat=P[5] + 2), dict(res=P[1] + 8), dict(h=P[3] + 4)):
        assert norm(lib, fn, **bad) == MISALIGNED, bad
    assert norm(lib, fn, hidden=32776, ld=32776) == UNSUPPORTED
    assert norm(lib, fn, rows=1 << 31) == UNSUPPORTED
    assert norm(lib, fn, rows=0, x=NULL, y=NULL) == binding.MM_OK
    assert norm(lib, fn, hidden=0, ld=0) == binding.MM_OK
    assert "ld_x" in (norm(lib, fn, ld=56), lib.mm_last_error().decode())[1]


def test_norm_gradient_refusals(lib):
    def grad(dy=P[0], h=P[1], w=P[2], rstd=P[3], dres=P[4], dh=P[5], dw=P[6], rows=4, hidden=64, dtype=0, ws=P[7],
             nbytes=1 << 20):
        return lib.mm_rms_norm_backward(dy, h, w, rstd, dres, dh, dw, rows, hidden, dtype, ws, nbytes, None)

    for bad in (dict(dy=NULL), dict(h=NULL), dict(w=NULL), dict(rstd=NULL), dict(dh=NULL), dict(dw=NULL),
                dict(ws=NULL, rows=4096), dict(rows=-1), dict(dtype=3), dict(nbytes=-1), dict(dh=P[0]), dict(dh=P[1]),
                dict(dh=P[4] + 16), dict(dw=P[2]), dict(ws=P[5]), dict(dw=P[5] + 16)):
        assert grad(**bad) == INVALID, bad
    for bad in (dict(hidden=4), dict(dy=P[0] + 2), dict(dw=P[6] + 4), dict(ws=P[7] + 4), dict(dres=P[4] + 8)):
        assert grad(**bad) == MISALIGNED, bad
    assert grad(hidden=40000) == UNSUPPORTED
    n = ctypes.c_int64(7)
    assert lib.mm_rms_norm_backward_workspace_size(-1, 64, ctypes.byref(n)) == INVALID
    assert lib.mm_rms_norm_backward_workspace_size(4, 64, None) == INVALID
    assert lib.mm_rms_norm_backward_workspace_size(0, 64, ctypes.byref(n)) == binding.MM_OK and n.value == 0


def test_w4_refusals(lib):
    def w4(x=P[0], W=P[1], s=P[2], z=NULL, b=P[3], out=P[4], M=4, N=64, K=128, group=128, epi=1):
        return lib.mm_linear_w4(x, W, s, z, b, out, M, N, K, group, epi, None)

    for bad in (dict(x=NULL), dict(W=NULL), dict(s=NULL), dict(b=NULL), dict(out=NULL), dict(M=-1), dict(epi=7),
                dict(out=P[0]), dict(out=P[1] + 256), dict(out=P[2]), dict(out=P[3]), dict(z=P[4])):
        assert w4(**bad) == INVALID, bad
    for bad in (dict(group=16), dict(group=0), dict(group=256), dict(K=1 << 31), dict(M=1 << 31)):
        assert w4(**bad) == UNSUPPORTED, bad
    for bad in (dict(K=124), dict(x=P[0] + 2), dict(W=P[1] + 8), dict(s=P[2] + 1), dict(out=P[4] + 1),
                dict(b=P[3] + 1)):
        assert w4(**bad) == MISALIGNED, bad
    assert w4(M=0, x=NULL) == binding.MM_OK and w4(N=0, out=NULL) == binding.MM_OK
    assert lib.mm_w4_pack(NULL, P[1], 4, 8, None) == INVALID
    assert lib.mm_w4_pack(P[0], P[0], 4, 8, None) == INVALID
    assert lib.mm_w4_pack(P[0], P[1] + 4, 4, 8, None) == MISALIGNED
    assert lib.mm_w4_pack(P[0], P[1], -4, 8, None) == INVALID
    assert lib.mm_w4_pack(NULL, NULL, 0, 8, None) == binding.MM_OK


def test_q8_refusals(lib):
    def q8(x=P[0], xs=P[1], W=P[2], ws=P[3], b=P[4], out=P[5], M=4, N=64, K=128, epi=3, work=NULL, nbytes=0):
        return lib.mm_linear_q8(x, xs, W, ws, b, out, M, N, K, epi, work, nbytes, None)

    for bad in (dict(x=NULL), dict(xs=NULL), dict(W=NULL), dict(ws=NULL), dict(b=NULL), dict(out=NULL), dict(N=-1),
                dict(epi=4), dict(out=P[0]), dict(out=P[1]), dict(out=P[2] + 64), dict(out=P[3]), dict(out=P[4]), dict(nbytes=-1),
                dict(work=P[5], nbytes=4096), dict(work=P[0], nbytes=4096), dict(work=P[3], nbytes=4096),
                dict(work=P[6], nbytes=16, M=128, N=512, K=8192)):
        assert q8(**bad) == INVALID, bad
    for bad in (dict(K=(1 << 22) + 16), dict(N=1 << 31)):
        assert q8(**bad) == UNSUPPORTED, bad
    for bad in (dict(K=120), dict(x=P[0] + 8), dict(W=P[2] + 4), dict(xs=P[1] + 2), dict(out=P[5] + 1)):
        assert q8(**bad) == MISALIGNED, bad
    assert q8(work=P[6] + 4, nbytes=1 << 40, M=128, N=512, K=8192) == MISALIGNED
    assert q8(M=0, x=NULL) == binding.MM_OK and q8(N=0) == binding.MM_OK
    n = ctypes.c_int64(5)
    assert lib.mm_linear_q8_workspace_size(4, 64, 128, ctypes.byref(n)) == binding.MM_OK and n.value == 0
    assert lib.mm_linear_q8_workspace_size(8192, 8192, 8192, ctypes.byref(n)) == binding.MM_OK and n.value == 0
    # 4 tiles of 128 x 128 in 8 chunks
    assert lib.mm_linear_q8_workspace_size(128, 512, 8192, ctypes.byref(n)) == binding.MM_OK
    assert n.value == 4 * 8 * 128 * 128 * 4
    assert lib.mm_linear_q8_workspace_size(-1, 64, 128, ctypes.byref(n)) == INVALID
    assert lib.mm_linear_q8_workspace_size(4, 64, 128, None) == INVALID


def test_widths_past_one_launch_are_refused(lib):
    """Before any device call, wherever the products of few rows would need more
    than the 2^32 - 1 threads of a launch."""
    A = [(i + 1) << 50 for i in range(6)]
    wide = 1 << 29
    for M in (1, 16, 64, 1000):
        assert lib.mm_linear_w4(A[0], A[1], A[2], NULL, NULL, A[3], M, wide, 128, 128, 0, None) == UNSUPPORTED
        assert "2^29" in lib.mm_last_error().decode()
    for M, K in ((1, 128), (16, 128), (32, 128), (1, 0), (100, 0)):
        assert lib.mm_linear_q8(A[0], A[1], A[2], A[3], NULL, A[4], M, wide, K, 0, NULL, 0, None) == UNSUPPORTED
        assert "2^29" in lib.mm_last_error().decode()


def test_python_checks_types_and_devices():
    x = torch.zeros((4, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="GPU"):
        mm.rms_norm(x, torch.zeros(64, dtype=torch.bfloat16))
    with pytest.raises(TypeError, match="x must be"):
        mm.rms_norm(x.half(), x)
    with pytest.raises(TypeError, match="x must be"):
        mm.linear_q8(x, x, x, x)
    with pytest.raises(TypeError, match="codes must be"):
        mm.pack_w4(x)
    with pytest.raises(ValueError, match="GPU"):
        mm.linear_w4(x, x, x)
