"""Race check of the tiles of the linear layer with adapters: the library built with
MM_DEBUG_FULL_SYNC (every copy into LDS drained, and every wave at a barrier, before
each super-step) against the normal build, bit for bit.

The cases take every kind of tile, K whole and in slices, several tiles per
workgroup, ragged last super-steps, and none, one and many adapters to a tile.
"""
import pytest
import torch

from dense_bf16_gemm_amd import binding
from test_gpu_linear_lora import inputs
from test_gpu_sync import assert_same, libs, run_both, say, stream  # noqa: F401 (libs is a fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M,N,K,R,L,how", [
    (70, 520, 8200, 16, 3, "mixed"), (300, 3001, 2056, 64, 4, "runs"), (1100, 4200, 520, 8, 40, "mixed"),
    (2500, 8200, 136, 32, 5, "runs"), (4096, 4096, 512, 16, 6, "runs"), (142, 21458, 520, 24, 2, "one"),
    (11208, 70, 4184, 16, 3, "runs"), (67, 16681, 2624, 128, 9, "mixed"), (6389, 69, 1680, 16, 4, "runs"),
    (8200, 2300, 64, 256, 2, "runs"), (2047, 3001, 4104, 32, 24, "runs"), (3000, 2500, 1032, 16, 300, "mixed"),
    (1024, 1024, 4096, 16, 2, "one"), (5000, 5000, 8, 8, 2, "mixed"),
])
def test_linear_lora(libs, M, N, K, R, L, how):  # noqa: F811
    dev = torch.device("cuda:0")
    args, bias = inputs(M, N, K, R, L, how, 40 + M)
    x, W, A, B, index, scale = (t.to(dev) for t in args)
    bias = bias.to(dev)
    nbytes = binding.linear_lora_workspace_size(M, N, K, R, L)
    ws = torch.empty(nbytes, dtype=torch.uint8, device=dev)
    out = torch.empty((M, N), dtype=torch.bfloat16, device=dev)
    say("linear_lora", M, N, K, R, L, how)
    assert_same(run_both(libs, None, lambda lib: binding.check(lib.mm_linear_lora(
        x.data_ptr(), W.data_ptr(), A.data_ptr(), B.data_ptr(), index.data_ptr(), scale.data_ptr(), bias.data_ptr(),
        out.data_ptr(), M, N, K, R, L, 3, ws.data_ptr(), nbytes, stream()), "mm_linear_lora"), [out]))
