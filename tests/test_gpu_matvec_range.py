"""Matrix-vector products at the ends of their numbers: E8M0 scales, large activations."""
import numpy as np
import pytest
import torch

import oracle
from gpu_util import bf16_to_dev, say, to_dev
from oracle import mxfp4_oracle as mx
from quantized_grouped_gemm_token_amd import ops
from test_gpu_few import CALL, make as make_layer, prepack as prepack_layer
from test_gpu_matvec import BLK, STORED, check, exact, make, prepack

pytestmark = pytest.mark.gpu


@pytest.fixture
def rng():
    return np.random.Generator(np.random.PCG64(7))


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    assert ops.w4a8_moe_device_supported(), "the current device is not a gfx950"
    yield
    torch.cuda.synchronize()


@pytest.mark.parametrize("prepacked", [False, True])
@pytest.mark.parametrize("byte", [0, 1, 2, 3, 127, 251, 252, 253, 254, 255])
def test_matvec_mxfp4_every_code_at_the_ends_of_the_scales(byte, prepacked):
    """One weight per output, one activation: the value itself, a subnormal one included; an infinity from 2^128 on
    (no fp32 value), NaN for byte 255."""
    K, N = 128, 16
    w = np.zeros((N, K // 2), np.uint8)
    w[:, 35] = np.arange(16)                                 # code n at k = 70, in the third block
    s = np.full((N, K // 32), 127, np.uint8)
    s[:, 2] = byte
    say(f"matvec mxfp4 scale byte {byte}, prepacked={prepacked}")
    wd, sd = prepack("mxfp4", w, s) if prepacked else (to_dev(w), to_dev(s))
    call = (BLK if prepacked else STORED)["mxfp4"]
    code = mx.e2m1_decode(np.arange(16, dtype=np.uint8)).astype(np.float64)
    # activations whose products are the smallest fp32 values that hold a code, ordinary and near the largest: exact
    for e in (-14, 0, 100) if byte < 4 else (-100, -14, 0):
        x = np.zeros((1, K), np.float32)
        x[0, 70] = 2.0 ** e
        y = call(bf16_to_dev(oracle.f32_to_bf16_bits(x)), wd, sd).double().cpu().numpy()[0]
        if byte == 255:
            assert np.isnan(y).all()
            continue
        weight = code * 2.0 ** (byte - 127)
        want = np.where(np.abs(weight) < 2.0 ** 128, weight * 2.0 ** e, np.copysign(np.inf, weight))
        assert np.array_equal(y, want), (e, y, want)


@pytest.mark.parametrize("form", ["g128", "channel"])
def test_matvec_int4_largest_activations(form, rng):
    """Activations of up to 2^116: a group's sums of x (q + 8) and of -8 x stay finite."""
    T, N, K = 4, 48, 1152
    x_bits, w, s = make(form, T, N, K, rng)
    x = oracle.bf16_bits_to_f32(x_bits)
    x = np.sign(x) * np.exp2(rng.integers(100, 117, size=x.shape)).astype(np.float32)
    x[1] = 2.0 ** 116                                        # every element of one sign
    x_bits, s = oracle.f32_to_bf16_bits(x), (s * np.float32(2.0 ** -20)).astype(np.float32)
    want, tol = exact(form, x_bits, w, s)
    say(f"matvec {form} largest activations")
    xd = bf16_to_dev(x_bits)
    y = STORED[form](xd, to_dev(w), to_dev(s))
    assert torch.isfinite(y).all()
    check(y, want, tol, "stored")
    blk = BLK[form](xd, *prepack(form, w, s))
    assert torch.equal(blk, y)


@pytest.mark.parametrize("form", ["g128", "channel"])
def test_matvec_int4_infinite_activations_give_nan(form, rng):
    x_bits, w, s = make(form, 3, 32, 256, rng)
    x = bf16_to_dev(x_bits)
    x[1, 77], x[2, 3] = float("inf"), float("-inf")
    say(f"matvec {form} infinities in x")
    y = STORED[form](x, to_dev(w), to_dev(s))
    assert torch.isfinite(y[0]).all() and torch.isnan(y[1:]).all()


def test_few_mxfp4_scale_of_nan():
    """Scale byte 255 in one row of w2: that column of y is NaN for the tokens that take the expert, nothing else."""
    T, H, I, E, k = 4, 256, 128, 4, 1
    x_bits, logits, weights = make_layer("mxfp4", T, H, I, E, k, seed=13)
    logits[:] = -5.0
    logits[np.arange(T), [0, 2, 2, 3]] = 1.0
    x, lg = bf16_to_dev(x_bits), to_dev(logits)
    say("few mxfp4 scale byte 255")
    want = CALL["mxfp4"](x, lg, k, *prepack_layer("mxfp4", weights))
    weights[3][2, 37, 1] = 255
    y = CALL["mxfp4"](x, lg, k, *prepack_layer("mxfp4", weights))
    bad = torch.zeros_like(y, dtype=torch.bool)
    bad[1:3, 37] = True
    assert torch.isnan(y[bad]).all() and torch.equal(y[~bad], want[~bad])


@pytest.mark.parametrize("T,N", [(3, 37), (16, 8200), (1, 1)])
@pytest.mark.parametrize("K", [6176, 6240, 12352, 18464])
def test_matvec_mxfp4_long_rows_that_end_inside_a_group(K, T, N, rng):
    """Stored rows of several parts whose last group is not whole; what follows a row of x is NaN."""
    x_bits, w, s = make("mxfp4", T, N, K, rng)
    want, tol = exact("mxfp4", x_bits, w, s)
    say(f"matvec mxfp4 T={T} N={N} K={K}")
    wide = torch.full((T, K + 8), float("nan"), dtype=torch.bfloat16, device="cuda:0")
    wide[:, :K] = bf16_to_dev(x_bits)
    wd, sd = to_dev(w), to_dev(s)
    y = STORED["mxfp4"](wide[:, :K], wd, sd)
    check(y, want, tol, "strided")
    assert torch.equal(STORED["mxfp4"](bf16_to_dev(x_bits), wd, sd), y)
