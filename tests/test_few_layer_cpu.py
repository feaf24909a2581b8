"""Which forwards of a layer with few=True are the one call (no GPU)."""
import pytest

from quantized_grouped_gemm_token_amd import ops
from quantized_grouped_gemm_token_amd.layer import W4A8MoE, W4A8MoEChannel, W4A8MoEMxfp4

LAYERS = [W4A8MoE, W4A8MoEChannel, W4A8MoEMxfp4]


def layer(cls, few=True):
    moe = cls.__new__(cls)                                   # (a constructor prepacks, on a GPU)
    moe.few, moe.H, moe.k, moe.I, moe.steps = few, 128, 1, 128, ("front",) + cls.STEPS[3:]
    return moe


@pytest.mark.parametrize("cls", LAYERS)
def test_a_kernel_asked_for_takes_the_steps(cls):
    moe = layer(cls)
    assert moe.uses_few(4) and moe.uses_few(4, ops.W4A8_GG_AUTO)
    for algo in (ops.W4A8_GG_STREAM, ops.W4A8_GG_TILED):
        assert not moe.uses_few(4, algo)
