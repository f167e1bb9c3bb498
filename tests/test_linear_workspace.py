"""Sizes of the linear workspace (host arithmetic, no GPU)."""

import pytest

from bit_nf4_quantized_blk_b200 import binding, build

# (M, N, K, r): bytes.  What the calls on bf16 activations need; the backward from a checkpoint uses the same buffer.
FUSED = {
    (1, 4096, 4096, 16): 2656000,
    (16, 14336, 4096, 16): 9466112,
    (17, 64, 64, 8): 52992,
    (33, 1024, 4096, 8): 2126592,
    (2048, 1024, 4096, 16): 24674560,
    (1999, 2048, 8192, 64): 27393536,
    (8192, 14336, 4096, 16): 56295680,
    (8192, 4096, 14336, 16): 45220096,
    (1500, 1032, 2112, 40): 22551040,
    (65536, 14336, 4096, 64): 166265088,
    (2**25, 8, 64, 8): 38664558336,
}
DENSE = {(1, 4096, 4096, 16): 35161856, (16, 14336, 4096, 16): 123236608, (17, 64, 64, 8): 60160}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    binding.lib()


def test_a_checkpoint_costs_other_callers_no_workspace():
    """A buffer that served the forward and the backward on bf16 activations still does."""
    for shape, size in FUSED.items():
        assert binding.qlora_linear_ws_bytes(*shape) <= size, shape
    with binding.weight_path(binding.WEIGHT_PATH_DENSE):
        for shape, size in DENSE.items():
            assert binding.qlora_linear_ws_bytes(*shape) <= size, shape
