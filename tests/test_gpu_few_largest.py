"""The largest sizes that the few-token layer and the matrix-vector products admit."""
import numpy as np
import pytest
import torch

import oracle
from few_accuracy import U, errors, product
from gpu_util import bf16_to_dev, host, say, to_dev
from quantized_grouped_gemm_token_amd import ops
from test_gpu_few import CALL, FORMS, check, make as make_layer, prepack as prepack_layer
from test_gpu_matvec import BLK, STORED, make, prepack

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    assert ops.w4a8_moe_device_supported(), "the current device is not a gfx950"
    yield
    torch.cuda.synchronize()
    torch.cuda.empty_cache()


@pytest.mark.parametrize("form", FORMS)
def test_matvec_longest_rows(form):
    """K = 2^22.  The bound is the mean square of the sums' roundings: each of a wave's K / 1024 groups (MXFP4: four
    products of a group) and the 8 waves round a sum of at most P, the group-128 form's products one of at most B_g.
    (few_accuracy.py; per channel the scale is last, and the groups' products round the same B_g.)"""
    T, N, K = 2, 16, 1 << 22
    rng = np.random.Generator(np.random.PCG64(22))
    x_bits, w, s = make(form, T, N, K, rng)
    say(f"matvec {form} K=2^22")
    xd = bf16_to_dev(x_bits)
    y = STORED[form](xd, to_dev(w), to_dev(s))
    assert torch.equal(BLK[form](xd, *prepack(form, w, s)), y)
    x = oracle.bf16_bits_to_f32(x_bits).astype(np.float64)
    if form == "channel":                                    # as a group-128 matrix of equal scales
        want, G2, P = product("g128", x, w, np.repeat(s[:, None], K // 128, 1))
    else:
        want, G2, P = product(form, x, w, s)
    n = (4 if form == "mxfp4" else 1) * (K // 1024) + 8
    rms, top = errors(host(y), want, np.sqrt((U * U / 3) * (9 * G2 + n * P * P)), 2 * U * np.abs(want))
    say(f"  {rms:.3f} (largest {top:.2f}) of the bound")
    assert rms <= 1 and top <= 8


@pytest.mark.parametrize("T", [1, 16])
@pytest.mark.parametrize("form", FORMS)
def test_matvec_most_outputs(form, T):
    """N = 2^24: every output as from the small matrices that the large one is made of."""
    N, K, part = 1 << 24, 128, 1 << 12
    rng = np.random.Generator(np.random.PCG64(24))
    x_bits, w, s = make(form, T, part, K, rng)
    x, wd, sd = bf16_to_dev(x_bits), to_dev(w), to_dev(s)
    say(f"matvec {form} T={T} N=2^24")
    want = STORED[form](x, wd, sd, y_dtype=torch.bfloat16)
    many = [t.repeat(N // part, *[1] * (t.dim() - 1)) for t in (wd, sd)]
    many[0][-1].zero_()                                      # .. but for the last row
    y = STORED[form](x, *many, y_dtype=torch.bfloat16)
    assert torch.equal(y.view(T, N // part, part)[:, :-1], want[:, None].expand(T, N // part - 1, part))
    assert torch.equal(y[:, N - part:N - 1], want[:, :-1])
    last = many[0][-1:].contiguous(), many[1][-1:].contiguous()
    assert torch.equal(y[:, N - 1:], STORED[form](x, *last, y_dtype=torch.bfloat16))


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("T,H,I,E,k", [(1, 256, 128, 1024, 256), (16, 7168, 128, 16, 16), (16, 128, 128, 1024, 16),
                                       (1, 8192, 128, 2, 2)])
def test_few_most_picks_and_codes(form, T, H, I, E, k):
    x_bits, logits, weights = make_layer(form, T, H, I, E, k, seed=T + k)
    say(f"few {form} T={T} H={H} I={I} E={E} k={k}")
    lg = to_dev(logits)
    ids, w = torch.empty((T, k), dtype=torch.int32, device="cuda:0"), torch.empty((T, k), device="cuda:0")
    y = CALL[form](bf16_to_dev(x_bits), lg, k, *prepack_layer(form, weights), ids=ids, w=w)
    check(form, x_bits, logits, weights, k, y, torch.float32)
    ids_r, w_r = ops.w4a8_moe_route(lg, k)
    assert torch.equal(ids, ids_r) and torch.equal(w.view(torch.int32), w_r.view(torch.int32))


@pytest.mark.parametrize("form", FORMS)
def test_few_longest_act_rows_of_every_pick(form):
    """16 tokens x 16 picks of I = 65536: the largest workspace.  One expert's weights for all, so that every token's
    y is what it is with that expert alone, up to rounding."""
    T, H, I, E, k = 16, 128, 65536, 16, 16
    x_bits, _, weights = make_layer(form, T, H, I, 1, 1, seed=5)
    packed = prepack_layer(form, weights)
    many = [t.expand(E, *t.shape[1:]).contiguous() for t in packed]
    gen = torch.Generator(device="cuda:0").manual_seed(5)
    lg = torch.randn(T, E, generator=gen, device="cuda:0")
    x = bf16_to_dev(x_bits)
    say(f"few {form} T={T} I={I} k={k}")
    one = CALL[form](x, lg[:, :1].contiguous(), 1, *packed)
    y = CALL[form](x, lg, k, *many)
    # (weights that sum to 1 and equal terms; sums of 16 x 512 groups instead of 512)
    assert float((y - one).norm() / one.norm()) <= 1e-5
