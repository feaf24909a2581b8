"""A layer with few=True whose caller asks for a GEMM kernel or for the times of steps."""
import pytest
import torch

from gpu_util import bf16_to_dev, say, to_dev
from quantized_grouped_gemm_token_amd import ops
from quantized_grouped_gemm_token_amd.layer import W4A8MoE, W4A8MoEChannel, W4A8MoEMxfp4
from test_gpu_few import FORMS, make

pytestmark = pytest.mark.gpu

LAYER = {"g128": W4A8MoE, "channel": W4A8MoEChannel, "mxfp4": W4A8MoEMxfp4}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    assert ops.w4a8_moe_device_supported(), "the current device is not a gfx950"
    yield
    torch.cuda.synchronize()


@pytest.mark.parametrize("form", FORMS)
def test_layer_few_with_a_kernel_asked_for(form):
    """algo other than AUTO: that kernel's bits, eager and captured."""
    T, H, I, E, k = 6, 512, 256, 16, 4
    x_bits, logits, weights = make(form, T, H, I, E, k, seed=91)
    x, lg = bf16_to_dev(x_bits), to_dev(logits)
    few, steps = (LAYER[form](*(to_dev(a) for a in weights), k=k, few=f) for f in (True, False))
    for algo in (ops.W4A8_GG_STREAM, ops.W4A8_GG_TILED):
        say(f"layer {form} few=True, algo={algo}")
        assert torch.equal(few(x, lg, algo=algo), steps(x, lg, algo=algo))
    y = torch.empty((T, H), device="cuda:0")
    g = few.capture(x, lg, y, algo=ops.W4A8_GG_STREAM)
    ref = steps(x, lg, algo=ops.W4A8_GG_STREAM)
    for _ in range(3):
        y.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, ref)


@pytest.mark.parametrize("form", FORMS)
def test_layer_few_events(form):
    """Events keyed by steps_for are recorded whichever path a forward takes; others are refused."""
    T, H, I, E, k = 6, 512, 256, 16, 4
    x_bits, logits, weights = make(form, T, H, I, E, k, seed=92)
    x, lg = bf16_to_dev(x_bits), to_dev(logits)
    few = LAYER[form](*(to_dev(a) for a in weights), k=k, few=True)
    for algo in (ops.W4A8_GG_AUTO, ops.W4A8_GG_STREAM, ops.W4A8_GG_TILED):
        say(f"layer {form} few=True, algo={algo}, events")
        ev = {n: (torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True))
              for n in few.steps_for(T, algo)}
        want = few(x, lg, algo=algo)
        assert torch.equal(few(x, lg, algo=algo, events=ev), want)
        torch.cuda.synchronize()
        assert all(a.elapsed_time(b) >= 0 for a, b in ev.values())
    with pytest.raises(ValueError):
        few(x, lg, events={n: None for n in few.steps})
