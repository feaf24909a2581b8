"""The accuracy bounds of the few-token layer's tests notice the errors they are there for (no GPU)."""
import numpy as np
import pytest

import oracle
from few_accuracy import act_reference, errors, y_reference
from oracle import mxfp4_oracle as mx

FORMS = ("g128", "mxfp4")                                    # (the INT8 form's sums are exact)


def expert(form, rng, E, N, K):
    if form == "mxfp4":
        return (rng.integers(0, 256, size=(E, N, K // 2), dtype=np.uint8),
                (121 + rng.integers(-1, 2, size=(E, N, K // 32))).astype(np.uint8))
    return (rng.integers(0, 2**32, size=(E, N, K // 8), dtype=np.uint32).view(np.int32),
            rng.lognormal(-4, 0.5, size=(E, N, K // 128)).astype(np.float32))


@pytest.mark.parametrize("H,I", [(256, 128), (2048, 640)])
@pytest.mark.parametrize("form", FORMS)
def test_bounds_notice_less_exact_products(form, H, I):
    """The FP8 matrix cores' error (up to 7.5e-6 of a group's sum of magnitudes, taken here as evenly spread) is over
    the bound; the roundings of fp32 results alone are far below it."""
    rng = np.random.Generator(np.random.PCG64(7))
    T, E, k = 3, 4, 2
    x_bits = oracle.f32_to_bf16_bits(rng.standard_normal((T, H)).astype(np.float32))
    ids = np.array([[0, 1], [1, 2], [3, 0]])
    weights = np.full((T, k), 0.5, np.float32)
    w13, s13 = expert(form, rng, E, 2 * I, H)
    w2, s2 = expert(form, rng, E, H, I)
    noise = lambda shape: rng.uniform(-7.5e-6, 7.5e-6, shape)  # noqa: E731
    act, root, rest = act_reference(form, x_bits, ids, w13, s13)
    assert errors(act.astype(np.float32), act, root, rest)[0] < 0.1
    off, _, _ = act_reference(form, x_bits, ids, w13, s13, noise)
    assert errors(off, act, root, rest)[0] > 2
    act32 = act.astype(np.float32)
    y, root, rest = y_reference(form, act32, ids, weights, w2, s2)
    assert errors(y.astype(np.float32), y, root, rest)[0] < 0.1
    off, _, _ = y_reference(form, act32, ids, weights, w2, s2, noise)
    assert errors(off, y, root, rest)[0] > 2
