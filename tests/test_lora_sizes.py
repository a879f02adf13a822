"""Sizes of the linear layer with an adapter per row that the library refuses, by both of
its entry points alike (CPU only: nothing here launches a kernel)."""
import ctypes

import pytest

from dense_bf16_gemm_amd import binding

P = [0x10000000000 * (i + 1) for i in range(9)]  # fake, never dereferenced
MOST = (1 << 21) - 32  # rows: 65535 blocks of 32


def both(M, N=64, K=128, rank=16, adapters=3):
    lib, n = binding.load(), ctypes.c_int64(7)
    size = lib.mm_linear_lora_workspace_size(M, N, K, rank, adapters, ctypes.byref(n))
    # (no workspace: what the sizes are refused for comes before what the call lacks)
    call = lib.mm_linear_lora(*P[:6], None, P[7], M, N, K, rank, adapters, 0, None, 0, None)
    return size, n.value, call


@pytest.mark.parametrize("sizes", [dict(M=MOST + 1), dict(M=1 << 22), dict(M=(1 << 31) - 1), dict(M=1 << 31), dict(M=4, K=1 << 22),
                                   dict(M=4, N=(1 << 27) - 15), dict(M=4, rank=264)])
def test_both_entry_points_refuse(sizes):
    size, n, call = both(**sizes)
    assert size == call == binding.MM_ERR_UNSUPPORTED and n == 0


def test_the_largest_row_count_has_a_workspace():
    size, n, call = both(MOST)
    assert size == binding.MM_OK and n > 0 and call == binding.MM_ERR_INVALID_VALUE  # (the workspace is missing)


def test_rows_without_adapters_are_the_linear_layers():
    """With nothing in the adapters the call is mm_linear, whose rows go further and which needs no
    workspace (asked for only: the call would launch)."""
    for sizes in ((64, 128, 0, 3), (64, 128, 16, 0), (64, 0, 16, 3)):
        n = ctypes.c_int64(7)
        assert binding.load().mm_linear_lora_workspace_size(MOST + 1, *sizes, ctypes.byref(n)) == binding.MM_OK
        assert n.value == 0
