"""act and y of the few-token layer, each against 64 bits from the values its own kernel starts with.

The bounds (few_accuracy.py) are mean squares of the roundings of fp32 sums: the errors of the FP8 matrix cores
would be several times over them (test_few_accuracy_cpu.py).
"""
import numpy as np
import pytest
import torch

import oracle
from few_accuracy import act_reference, errors, scaled, y_reference
from gpu_util import bf16_to_dev, host, say, to_dev
from quantized_grouped_gemm_token_amd import ops
from test_gpu_few import CALL, FORMS, make, prepack
from test_gpu_matvec import STORED, exact, make as make_mv

pytestmark = pytest.mark.gpu

# T, H, I, E, k
SHAPES = [
    (1, 256, 128, 8, 2), (16, 256, 128, 8, 2), (5, 1152, 384, 60, 6), (16, 1024, 640, 12, 8), (2, 2048, 768, 128, 8),
    (9, 4352, 512, 24, 3), (2, 8192, 640, 16, 8), (16, 384, 2176, 5, 2), (4, 6144, 2048, 4, 1), (12, 512, 256, 40, 7),
]


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    assert ops.w4a8_moe_device_supported(), "the current device is not a gfx950"
    yield
    torch.cuda.synchronize()


def act_in(ws, T, k, I):
    """act [T k][I] in a workspace: in front of the maxima [T k][I/16], 256 x 2 x T x 32 sums and 256 counts."""
    behind = T * k * (I + I // 16) + 256 * 2 * T * 32 + 256
    at = ws.numel() - 4 * behind
    return host(ws[at:at + 4 * T * k * I].view(torch.float32)).reshape(T * k, I)


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("T,H,I,E,k", SHAPES)
def test_few_act_and_y_to_fp32_rounding(form, T, H, I, E, k):
    x_bits, logits, weights = make(form, T, H, I, E, k, seed=T + H + I)
    w13, s13, w2, s2 = weights
    say(f"few {form} T={T} H={H} I={I} E={E} k={k}: act and y to fp32 rounding")
    ws = torch.zeros(ops.w4a8_moe_few_workspace_bytes(T, k, I), dtype=torch.uint8, device="cuda:0")
    ids = torch.empty((T, k), dtype=torch.int32, device="cuda:0")
    w = torch.empty((T, k), device="cuda:0")
    y = host(CALL[form](bf16_to_dev(x_bits), to_dev(logits), k, *prepack(form, weights), ids=ids, w=w, workspace=ws))
    act, ids, w = act_in(ws, T, k, I), host(ids), host(w)
    rms, top = errors(act, *act_reference(form, x_bits, ids, w13, s13))
    rms_y, top_y = errors(y, *y_reference(form, act, ids, w, w2, s2))
    say(f"  act {rms:.3f} (largest {top:.2f}), y {rms_y:.3f} (largest {top_y:.2f}) of the bound")
    assert rms <= 1 and top <= 8, "act"                      # (8: of 10^6 evenly spread sums none is near)
    assert rms_y <= 1 and top_y <= 8, "y"


@pytest.mark.parametrize("binades", [0, 24])
@pytest.mark.parametrize("form", ["g128", "mxfp4"])
def test_one_group_on_the_bf16_matrix_cores(form, binades):
    """K = 128, scale 1: the products and sums of one group, eight (MXFP4: four) instructions in a row.

    An instruction's order of adding is its own, so what holds for any is all that bounds an element: an fp32 sum of
    n terms takes n - 1 additions, each off by at most U of a partial sum <= sum |products|.  In the mean square the
    instructions are as good as if each rounded its result once."""
    T, N, K = 16, 4096, 128
    rng = np.random.Generator(np.random.PCG64(binades))
    _, w, s = make_mv(form, T, N, K, rng)
    s = np.full_like(s, 127 if form == "mxfp4" else 1)
    # (normally distributed, and spread over 24 binades: the former hardly round at all in one group)
    x = rng.standard_normal((T, K)) * np.exp2(rng.uniform(-binades / 2, binades / 2, (T, K)))
    x_bits = oracle.f32_to_bf16_bits(x.astype(np.float32))
    want, _ = exact(form, x_bits, w, s)
    x = oracle.bf16_bits_to_f32(x_bits).astype(np.float64)
    B = np.abs(x) @ scaled(form, w, s)[1].T
    say(f"one group {form}, {binades} binades")
    err = (host(STORED[form](bf16_to_dev(x_bits), to_dev(w), to_dev(s))).astype(np.float64) - want) / B
    top, rms = float(np.abs(err).max()), float(np.sqrt(np.mean(err ** 2)))
    say(f"  largest {top:.2e}, rms {rms:.2e} of sum |products|")
    n = 8 if form == "g128" else 4
    assert top <= (32 * n - 1) * 2.0 ** -24 and rms <= (n / 3) ** 0.5 * 2.0 ** -24
