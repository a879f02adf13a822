"""Race check of the 4-bit and 8-bit products: the library built with
MM_DEBUG_FULL_SYNC (every copy into LDS drained before its step; the tile
kernel also waits at a barrier before each) against the normal build, bit for
bit.

The extra waits change only timing, so any difference means that the normal
build reads a tile before its copy landed, or copies over one still being
read.  The cases take every kernel: each count of activation rows, whole and
half staging steps, ragged last steps, one step and many, and the tile kernel
with its K whole and in chunks and several tiles per workgroup.
"""
import pytest
import torch

import decoder_ref as ref
from dense_bf16_gemm_amd import binding
from test_gpu_decoder import q8_inputs, w4_inputs
from test_gpu_sync import assert_same, libs, run_both, say, stream  # noqa: F401 (libs is a fixture)

pytestmark = pytest.mark.gpu


def ptr(t):
    return t.data_ptr() if t is not None else None


@pytest.mark.parametrize("M,N,K,group,zeros", [
    (1, 520, 8200, 32, True), (4, 4800, 2048, 128, False), (13, 1000, 4104, 64, True), (31, 9600, 1032, 32, False),
    (37, 3001, 4104, 128, True), (48, 5000, 128, 64, False), (64, 9600, 2056, 32, True), (61, 300, 8192, 128, False),
    (150, 1000, 1160, 64, False),
])
def test_linear_w4(libs, M, N, K, group, zeros):  # noqa: F811
    dev = torch.device("cuda:0")
    x, codes, s, z, _ = w4_inputs(M, N, K, group, zeros, 40 + M)
    packed = ref.pack(codes).to(dev)
    x, s, z = x.to(dev), s.to(dev), z.to(dev) if z is not None else None
    out = torch.empty((M, N), dtype=torch.bfloat16, device=dev)
    say("linear_w4", M, N, K, group, zeros)
    assert_same(run_both(libs, None, lambda lib: binding.check(lib.mm_linear_w4(
        x.data_ptr(), packed.data_ptr(), s.data_ptr(), ptr(z), None, out.data_ptr(), M, N, K, group, 0, stream()),
        "mm_linear_w4"), [out]))


@pytest.mark.parametrize("M,N,K,ws", [
    (1, 520, 8208, False), (4, 14000, 2048, False), (13, 1000, 4112, False), (32, 9600, 1040, False),
    (64, 9600, 2064, False), (50, 300, 8192, False),
    (70, 520, 16400, False), (70, 520, 16400, True), (300, 3001, 4112, True), (1100, 4200, 1040, True),
    (2500, 8200, 272, False), (4096, 4096, 1024, True), (142, 21458, 1040, True), (11208, 70, 8368, True),
    (67, 16681, 5248, True), (6389, 69, 3360, True), (16393, 66, 1040, False), (71, 66, 8016, True),
])
def test_linear_q8(libs, M, N, K, ws):  # noqa: F811
    dev = torch.device("cuda:0")
    x, xs, W, s, _ = (t.to(dev) for t in q8_inputs(M, N, K, 60 + M))
    nbytes = binding.linear_q8_workspace_size(M, N, K) if ws else 0
    wsp = torch.empty(max(nbytes, 16), dtype=torch.uint8, device=dev)
    out = torch.empty((M, N), dtype=torch.bfloat16, device=dev)
    say("linear_q8", M, N, K, nbytes)
    assert_same(run_both(libs, None, lambda lib: binding.check(lib.mm_linear_q8(
        x.data_ptr(), xs.data_ptr(), W.data_ptr(), s.data_ptr(), None, out.data_ptr(), M, N, K, 0,
        wsp.data_ptr() if nbytes else None, nbytes, stream()), "mm_linear_q8"), [out]))
