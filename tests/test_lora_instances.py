"""The instances of the rows' kernel of the linear layer with an adapter per row that the
library holds are those that a call reaches (CPU only)."""
import re

from dense_bf16_gemm_amd import build

WAVES = 16


def plan(M, K):
    """Blocks of 16 rows, steps of 64 k per wave, whether the kernel writes the output: the
    host's rule for up to 64 rows."""
    blocks = 1 if M <= 16 else 2 if M <= 32 else 4
    steps = -(-K // 64)
    slices = -(-steps // (WAVES * (8 // blocks)))
    per_wave = 2
    while WAVES * per_wave * slices < steps:
        per_wave *= 2
    return blocks, per_wave, slices == 1 and blocks < 4


def test_rows_kernel_instances():
    # (every count of steps up to some 400, and the longest K)
    reached = {plan(M, K) for M in (1, 16, 17, 32, 33, 64) for K in [*range(8, 26000, 56), (1 << 22) - 8]}
    built = set()
    for name in build.resource_usage(build.REMARKS_DECODER):
        m = re.match(r"_ZN3mmk9lora_rowsILi(\d)ELi(\d)ELb([01])E", name)
        if m:
            built.add((int(m.group(1)), int(m.group(2)), m.group(3) == "1"))
    assert built == reached
