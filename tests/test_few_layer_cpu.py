"""Which forwards of a layer with few=True are the one call, and what it says about events (no GPU)."""
import pytest
import torch

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
        assert moe.steps_for(4, algo) == moe.steps
    assert moe.steps_for(4) == ("few",)
    assert moe.steps_for(17) == moe.steps
    assert layer(cls, few=False).steps_for(4) == moe.steps


@pytest.mark.parametrize("cls", LAYERS)
def test_events_of_other_steps_are_refused(cls):
    moe = layer(cls)
    x, lg = torch.zeros((2, 128), dtype=torch.bfloat16), torch.zeros((2, 1))
    with pytest.raises(ValueError, match="steps_for"):
        moe.forward(x, lg, events={s: (None, None) for s in moe.steps})
