"""y in memory that the call also reads: refused by the matrix-vector products, allowed by the few-token layer."""
import numpy as np
import pytest
import torch

from gpu_util import bf16_to_dev, say, to_dev
from quantized_grouped_gemm_token_amd import ops
from test_gpu_few import CALL, FORMS, make as make_layer, prepack as prepack_layer
from test_gpu_matvec import BLK, STORED, make, prepack

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


@pytest.mark.parametrize("form", FORMS)
def test_matvec_refuses_a_y_that_overlaps_x(form, rng):
    T, N, K = 3, 256, 256
    x_bits, w, s = make(form, T, N, K, rng)
    wd, sd = to_dev(w), to_dev(s)
    buf = torch.zeros(T * 3 * K, dtype=torch.bfloat16, device="cuda:0")
    x = buf[:T * K].view(T, K)
    x.copy_(bf16_to_dev(x_bits))
    say(f"matvec {form}: y over x")
    want = STORED[form](x, wd, sd, y_dtype=torch.bfloat16)
    for y in (x, buf[K:K + T * N].view(T, N), buf[T * K - 1:T * K - 1 + T * N].view(T, N)):
        with pytest.raises(ValueError, match="overlap"):
            STORED[form](x, wd, sd, y=y)
        with pytest.raises(ValueError, match="overlap"):
            BLK[form](x, *prepack(form, w, s), y=y)
    with pytest.raises(ValueError, match="overlap"):         # one row, and an output of another type in its memory
        STORED[form](x[1:2], wd, sd, y=buf[K:K + 2 * N].view(torch.float32).view(1, N))
    with pytest.raises(ops.W4A8Error):
        STORED[form](x[:1].expand(T, K), wd, sd, y=torch.empty(T, N, dtype=torch.bfloat16, device="cuda:0"))
    # next to x, in the same buffer
    y = STORED[form](x, wd, sd, y=buf[T * K:T * K + T * N].view(T, N))
    assert torch.equal(y, want)
    # the rows of x apart, y in the gap between two of them
    wide = torch.zeros(2, 4 * K, dtype=torch.bfloat16, device="cuda:0")
    wide[:, :K] = x[:2]
    y = STORED[form](wide[:, :K], wd, sd, y=wide[0, K:K + 2 * N].view(2, N))
    assert torch.equal(y, want[:2])


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("T", [1, 7, 16])
def test_few_in_place(form, T):
    H, I, E, k = 512, 640, 12, 3
    x_bits, logits, weights = make_layer(form, T, H, I, E, k, seed=17)
    x, lg, packed = bf16_to_dev(x_bits), to_dev(logits), prepack_layer(form, weights)
    say(f"few {form} T={T}: y over x, then over the logits")
    want = CALL[form](x, lg, k, *packed, y_dtype=torch.bfloat16)
    for _ in range(3):
        h = x.clone()
        assert torch.equal(CALL[form](h, lg, k, *packed, y=h), want)
    buf = torch.zeros(T * H, dtype=torch.float32, device="cuda:0")
    l2 = buf[:T * E].view(T, E)
    l2.copy_(lg)
    assert torch.equal(CALL[form](x, l2, k, *packed, y=buf.view(T, H)), CALL[form](x, lg, k, *packed))
