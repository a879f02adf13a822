"""Pins of the 64-bit forms that layer norm, the linear layer with adapters and the
mixture-of-experts FFN are tested against, and the host-side refusals of those
operators (CPU only: no test here launches a kernel or passes validation with a
pointer that is not real device memory)."""
import ctypes
import math

import pytest
import torch

import dense_bf16_gemm_amd as mm
import layer_ref as ref
from dense_bf16_gemm_amd import binding

P = [0x10000000 * (i + 1) for i in range(12)]  # fake, never dereferenced
NULL = None
INVALID, UNSUPPORTED, MISALIGNED = (binding.MM_ERR_INVALID_VALUE, binding.MM_ERR_UNSUPPORTED,
                                    binding.MM_ERR_MISALIGNED)


@pytest.fixture(scope="module")
def lib():
    return binding.load()


# ---- the 64-bit forms --------------------------------------------------------

def test_norm_against_torch():
    gen = torch.Generator().manual_seed(3)
    x = torch.randn((5, 24), generator=gen, dtype=torch.float32) * 3 + 100
    w, b = torch.randn((2, 24), generator=gen).bfloat16()
    _, mean, rstd, y = ref.norm(x, w, b, None, 1e-3)
    want = torch.nn.functional.layer_norm(x.double(), (24,), w.double(), b.double(), 1e-3)
    assert torch.allclose(y, want, rtol=1e-12, atol=1e-12)
    assert torch.allclose(mean, x.double().mean(1)) and torch.allclose(rstd, (x.double().var(1, correction=0) + 1e-3) ** -0.5)


def test_gradient_is_the_forward_forms_by_differences():
    gen = torch.Generator().manual_seed(5)
    r, n, eps, step = 3, 16, 1e-3, 1e-5
    x, res, cy, ch = (torch.randn((r, n), generator=gen, dtype=torch.float64) for _ in range(4))
    w, b = torch.randn((2, n), generator=gen, dtype=torch.float64)
    h = x + res
    mean = h.mean(1)
    rstd = 1.0 / torch.sqrt(h.var(1, correction=0) + eps)
    dh, dw, db = ref.norm_grad(cy, h, w, mean, rstd, ch)

    def difference(at, i):
        args = [x, w, b, res]
        values = []
        for sign in (1, -1):
            t = args[at].clone()
            t.view(-1)[i] += sign * step
            values.append(ref.norm_loss(*(t if q == at else a for q, a in enumerate(args)), eps, cy, ch))
        return (values[0] - values[1]) / (2 * step)

    for i in range(r * n):
        assert abs(difference(0, i) - dh.view(-1)[i]) < 1e-8 and abs(difference(3, i) - dh.view(-1)[i]) < 1e-8
    for i in range(n):
        assert abs(difference(1, i) - dw[i]) < 1e-8 and abs(difference(2, i) - db[i]) < 1e-8


def test_lora_by_hand():
    x = torch.tensor([[1.0, 2.0], [3.0, 4.0], [5.0, 6.0], [1.0, 0.0]])
    W = torch.tensor([[1.0, 0.0], [0.0, 1.0], [1.0, 1.0]])
    A = torch.tensor([[[1.0, 1.0]], [[2.0, -1.0]]])
    B = torch.tensor([[[1.0], [0.0], [-1.0]], [[0.0], [1.0], [2.0]]])
    y = ref.lora(x, W, A, B, torch.tensor([1, -1, 0, 2]), torch.tensor([10.0, 100.0]))
    assert y.tolist() == [[1, 2, 3], [3, 4, 7], [5 + 110, 6, 11 - 110], [1, 0, 1]]


def test_route_by_hand():
    inf, nan = math.inf, math.nan
    logits = torch.tensor([[0.0, 1.0, 1.0, -1.0], [-inf, 2.0, -inf, -inf], [-inf] * 4, [0.0, -0.0, nan, inf]])
    experts, weights = ref.route(logits, 2, True)
    assert experts.tolist() == [[1, 2], [1, -1], [-1, -1], [2, 3]]
    assert weights[:3].tolist() == [[0.5, 0.5], [1.0, 0.0], [0.0, 0.0]] and weights[3].isnan().all()
    _, weights = ref.route(logits[:1], 2, False)
    assert torch.allclose(weights, torch.softmax(logits[:1].double(), 1)[:, 1:3])


def test_moe_against_one_token_at_a_time():
    gen = torch.Generator().manual_seed(1)
    T, E, H, I, k = 5, 4, 6, 7, 2
    x = torch.randn((T, H), generator=gen, dtype=torch.float64)
    g, u = torch.randn((2, E, I, H), generator=gen, dtype=torch.float64)
    d = torch.randn((E, H, I), generator=gen, dtype=torch.float64)
    experts, weights = ref.route(torch.randn((T, E), generator=gen), k, True)
    out, size = ref.moe(x, experts, weights, g, u, d)
    for t in range(T):
        want = sum(weights[t, j] * d[e] @ (torch.nn.functional.silu(g[e] @ x[t]) * (u[e] @ x[t]))
                   for j, e in enumerate(experts[t].tolist()))
        assert torch.allclose(out[t], want, rtol=1e-12, atol=1e-12)
    assert (size >= out.abs()).all()


# ---- refusals ----------------------------------------------------------------

def layer_norm(lib, x=P[0], ld=64, res=P[1], w=P[2], b=P[3], h=P[4], y=P[5], mean=P[6], rstd=P[7], rows=4, hidden=64,
               eps=1e-5, dtype=0):
    return lib.mm_layer_norm(x, ld, res, w, b, h, y, mean, rstd, rows, hidden, eps, dtype, None)


def test_layer_norm_refusals(lib):
    for bad in (dict(x=NULL), dict(w=NULL), dict(y=NULL), dict(mean=NULL), dict(rstd=NULL), dict(h=NULL), dict(rows=-1),
                dict(hidden=-8), dict(eps=-1.0), dict(eps=float("nan")), dict(dtype=2), dict(ld=56),
                dict(y=P[0]), dict(y=P[1] + 16), dict(y=P[3]), dict(h=P[0] + 16), dict(h=P[1] + 128), dict(h=P[2]),
                dict(h=P[3]), dict(h=P[5] + 16), dict(mean=P[0]), dict(rstd=P[6] + 4), dict(rstd=P[4] + 4),
                dict(mean=P[5] + 4), dict(h=P[0], ld=72)):
        assert layer_norm(lib, **bad) == INVALID, bad
    for bad in (dict(hidden=60), dict(ld=68), dict(x=P[0] + 8), dict(w=P[2] + 2), dict(b=P[3] + 2), dict(y=P[5] + 8),
                dict(mean=P[6] + 2), dict(rstd=P[7] + 1), dict(res=P[1] + 8), dict(h=P[4] + 4)):
        assert layer_norm(lib, **bad) == MISALIGNED, bad
    assert layer_norm(lib, hidden=32776, ld=32776) == UNSUPPORTED
    assert layer_norm(lib, rows=1 << 31) == UNSUPPORTED
    assert layer_norm(lib, rows=0, x=NULL, y=NULL) == binding.MM_OK
    assert layer_norm(lib, hidden=0, ld=0) == binding.MM_OK


def test_layer_norm_gradient_refusals(lib):
    def grad(dy=P[0], h=P[1], w=P[2], mean=P[3], rstd=P[4], dres=P[5], dh=P[6], dw=P[7], db=P[8], rows=4, hidden=64,
             dtype=0, ws=P[9], nbytes=1 << 20):
        return lib.mm_layer_norm_backward(dy, h, w, mean, rstd, dres, dh, dw, db, rows, hidden, dtype, ws, nbytes, None)

    for bad in (dict(dy=NULL), dict(h=NULL), dict(w=NULL), dict(mean=NULL), dict(rstd=NULL), dict(dh=NULL),
                dict(dw=NULL), dict(db=NULL), dict(ws=NULL, rows=4096), dict(rows=-1), dict(dtype=3), dict(nbytes=-1),
                dict(dh=P[0]), dict(dh=P[1]), dict(dh=P[5] + 16), dict(dw=P[2]), dict(ws=P[6]), dict(ws=P[5]),
                dict(dw=P[6] + 16), dict(db=P[7] + 16), dict(db=P[3]), dict(dw=P[5] + 64)):
        assert grad(**bad) == INVALID, bad
    for bad in (dict(hidden=4), dict(dy=P[0] + 2), dict(dw=P[7] + 4), dict(db=P[8] + 8), dict(ws=P[9] + 4),
                dict(dres=P[5] + 8)):
        assert grad(**bad) == MISALIGNED, bad
    assert grad(hidden=40000) == UNSUPPORTED
    n = ctypes.c_int64(7)
    assert lib.mm_layer_norm_backward_workspace_size(-1, 64, ctypes.byref(n)) == INVALID
    assert lib.mm_layer_norm_backward_workspace_size(4, 64, None) == INVALID
    assert lib.mm_layer_norm_backward_workspace_size(0, 64, ctypes.byref(n)) == binding.MM_OK and n.value == 0


def test_linear_lora_refusals(lib):
    def lora(x=P[0], W=P[1], A=P[2], B=P[3], index=P[4], scale=P[5], bias=P[6], out=P[7], M=4, N=64, K=128, rank=16,
             adapters=3, epi=1, ws=P[8], nbytes=1 << 24):
        return lib.mm_linear_lora(x, W, A, B, index, scale, bias, out, M, N, K, rank, adapters, epi, ws, nbytes, None)

    for bad in (dict(x=NULL), dict(W=NULL), dict(A=NULL), dict(B=NULL), dict(index=NULL), dict(scale=NULL),
                dict(bias=NULL), dict(out=NULL), dict(ws=NULL), dict(M=-1), dict(rank=-8), dict(adapters=-1),
                dict(epi=7), dict(out=P[0]), dict(out=P[1] + 256), dict(out=P[2]), dict(out=P[3]), dict(out=P[4]),
                dict(out=P[5]), dict(out=P[6]), dict(ws=P[7]), dict(ws=P[0]), dict(ws=P[3]), dict(nbytes=-1),
                dict(nbytes=64)):
        assert lora(**bad) == INVALID, bad
    for bad in (dict(K=1 << 31), dict(M=1 << 31), dict(K=(1 << 22) + 8), dict(rank=264), dict(adapters=1 << 31),
                dict(N=1 << 27)):
        assert lora(**bad) == UNSUPPORTED, bad
    for bad in (dict(K=124), dict(rank=12), dict(x=P[0] + 2), dict(W=P[1] + 8), dict(A=P[2] + 8), dict(B=P[3] + 4),
                dict(index=P[4] + 2), dict(scale=P[5] + 1), dict(out=P[7] + 1), dict(bias=P[6] + 1), dict(ws=P[8] + 16)):
        assert lora(**bad) == MISALIGNED, bad
    assert lora(M=0, x=NULL) == binding.MM_OK and lora(N=0, out=NULL) == binding.MM_OK
    n = ctypes.c_int64(5)
    size = lib.mm_linear_lora_workspace_size
    assert size(4, 64, 128, 0, 3, ctypes.byref(n)) == binding.MM_OK and n.value == 0
    assert size(4, 64, 128, 16, 3, ctypes.byref(n)) == binding.MM_OK and n.value > 0
    assert size(-4, 64, 128, 16, 3, ctypes.byref(n)) == INVALID
    assert size(4, 64, 128, 16, 3, None) == INVALID


def test_moe_refusals(lib):
    def moe(x=P[0], logits=P[1], g=P[2], u=P[3], d=P[4], out=P[5], experts=P[6], weights=P[7], T=4, E=8, H=64, I=32, k=2,
            ws=P[8], nbytes=1 << 20):
        return lib.mm_moe_ffn(x, logits, g, u, d, out, experts, weights, T, E, H, I, k, 1, ws, nbytes, None)

    for bad in (dict(x=NULL), dict(logits=NULL), dict(g=NULL), dict(u=NULL), dict(d=NULL), dict(out=NULL),
                dict(experts=NULL), dict(weights=NULL), dict(ws=NULL), dict(T=-1), dict(E=-1), dict(k=-1), dict(k=9),
                dict(out=P[0]), dict(out=P[2] + 64), dict(experts=P[1]), dict(weights=P[6]), dict(ws=P[4]), dict(ws=P[5]),
                dict(nbytes=-1), dict(nbytes=4096)):
        assert moe(**bad) == INVALID, bad
    for bad in (dict(T=65), dict(E=513), dict(E=40, k=17), dict(H=(1 << 18) + 8), dict(I=(1 << 18) + 8)):
        assert moe(**bad) == UNSUPPORTED, bad
    for bad in (dict(H=60), dict(I=36), dict(x=P[0] + 8), dict(g=P[2] + 2), dict(d=P[4] + 8), dict(logits=P[1] + 2),
                dict(experts=P[6] + 2), dict(out=P[5] + 1), dict(ws=P[8] + 64)):
        assert moe(**bad) == MISALIGNED, bad
    assert moe(T=0, x=NULL) == binding.MM_OK
    n = ctypes.c_int64(5)
    assert lib.mm_moe_ffn_workspace_size(0, 8, 64, 32, 2, ctypes.byref(n)) == binding.MM_OK and n.value == 0
    assert lib.mm_moe_ffn_workspace_size(4, 8, 64, 32, 2, None) == INVALID
    assert lib.mm_moe_ffn_workspace_size(4, 8, 64, 32, 9, ctypes.byref(n)) == INVALID


def test_python_checks_types_and_devices():
    x = torch.zeros((4, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="GPU"):
        mm.layer_norm(x, torch.zeros(64, dtype=torch.bfloat16))
    with pytest.raises(TypeError, match="x must be"):
        mm.layer_norm(x.half(), x)
    with pytest.raises(TypeError, match="h must be"):
        mm.layer_norm_backward(x, x.half(), x, x, x)
    with pytest.raises(TypeError, match="x must be"):
        mm.linear_lora(x.float(), x, x, x, x, x)
    with pytest.raises(ValueError, match="GPU"):
        mm.moe_ffn(x, x, x, x, x, 2)
