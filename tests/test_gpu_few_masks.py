"""Masked logits (-infinity, NaN) in the few-token layer: a masked expert is not routed.

Whatever a masked expert holds does not reach y, a token with nothing but masks has
weights and a row of y that are zero, and y agrees with the layer's steps, which skip
the same routed rows.
"""
import numpy as np
import pytest
import torch

from gpu_util import bf16_to_dev, host, say, to_dev
from quantized_grouped_gemm_token_amd import ops
from quantized_grouped_gemm_token_amd.layer import W4A8MoE, W4A8MoEChannel, W4A8MoEMxfp4
from test_gpu_few import CALL, FORMS, check, make, prepack

pytestmark = pytest.mark.gpu

LAYER = {"g128": W4A8MoE, "channel": W4A8MoEChannel, "mxfp4": W4A8MoEMxfp4}
INF, NAN = np.inf, np.nan


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    assert ops.w4a8_moe_device_supported(), "the current device is not a gfx950"
    yield
    torch.cuda.synchronize()


def run(form, x_bits, logits, packed, k, y_dtype=torch.float32, **kw):
    """y, ids, w of a call whose outputs and workspace start as NaN."""
    T, H = x_bits.shape
    I = packed[0].shape[1] * 8
    ids = torch.full((T, k), -7, dtype=torch.int32, device="cuda:0")
    w = torch.full((T, k), NAN, device="cuda:0")
    y = torch.full((T, H), NAN, dtype=y_dtype, device="cuda:0")
    ws = torch.full((ops.w4a8_moe_few_workspace_bytes(T, k, I),), 255, dtype=torch.uint8, device="cuda:0")
    CALL[form](bf16_to_dev(x_bits), to_dev(logits), k, *packed, y=y, ids=ids, w=w, workspace=ws, **kw)
    return y, host(ids), host(w)


@pytest.mark.parametrize("renormalize", [True, False])
@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("T,H,I,E,k", [(5, 384, 256, 60, 4), (16, 512, 256, 300, 16), (12, 4352, 512, 24, 3)])
def test_few_a_masked_token_gives_a_zero_row(form, T, H, I, E, k, renormalize):
    """Padding tokens: nothing but -infinity in their rows of logits."""
    x_bits, logits, weights = make(form, T, H, I, E, k, seed=81)
    masked = [0, T // 2, T - 1]
    rest = [t for t in range(T) if t not in masked]
    whole = logits.copy()
    logits[masked] = -INF
    say(f"few {form} T={T} H={H} masked tokens, renormalize={renormalize}")
    y, ids, w = run(form, x_bits, logits, prepack(form, weights), k, renormalize=renormalize)
    assert (host(y)[masked] == 0).all() and (w[masked] == 0).all()
    assert (ids[masked] == np.arange(k)).all()
    check(form, x_bits[rest], whole[rest], weights, k, y[rest], torch.float32, renormalize)
    ids_r, w_r = (host(a) for a in ops.w4a8_moe_route(to_dev(logits), k, renormalize=renormalize))
    assert np.array_equal(ids[rest], ids_r[rest]) and np.array_equal(w[rest].view(np.int32), w_r[rest].view(np.int32))


@pytest.mark.parametrize("y_dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("T,H,I", [(1, 256, 128), (16, 256, 128), (3, 6144, 128), (16, 4096, 1024)])
def test_few_nothing_is_routed(form, T, H, I, y_dtype):
    """Every token masked: no expert is read, y is zero."""
    E, k = 6, 2
    x_bits, logits, weights = make(form, T, H, I, E, k, seed=82)
    say(f"few {form} T={T} H={H} I={I}: every logit masked, {y_dtype}")
    for mask in (-INF, NAN):
        logits[:] = mask
        y, ids, w = run(form, x_bits, logits, prepack(form, weights), k, y_dtype)
        assert not y.view(torch.int32 if y_dtype == torch.float32 else torch.int16).any()       # (+0)
        assert (w == 0).all() and (ids == np.arange(k)).all()


@pytest.mark.parametrize("bad", [NAN, INF])
@pytest.mark.parametrize("form", ["g128", "channel"])
def test_few_masked_experts_that_are_not_finite_are_not_read(form, bad):
    """Rows with fewer unmasked experts than picks: experts 0 .. 3 rank next, and their scales are not finite."""
    T, H, I, E, k = 6, 512, 256, 20, 4
    x_bits, logits, weights = make(form, T, H, I, E, k, seed=83)
    whole = [a.copy() for a in weights]
    weights[1][:4], weights[3][:4] = bad, bad
    mask = np.zeros((T, E), bool)
    mask[:, :4] = True                                       # masked for everyone
    for t in range(T):
        mask[t, 5 + t % 3:] = True                           # one to three experts left
    lg = np.where(mask, np.where(np.arange(E) % 2, NAN, -INF), logits).astype(np.float32)
    say(f"few {form}: masked experts hold {bad}")
    y, ids, w = run(form, x_bits, lg, prepack(form, weights), k)
    assert ((ids >= 0) & (ids < E)).all() and all(len(set(r)) == k for r in ids.tolist())
    assert (w[np.take_along_axis(mask, ids, 1)] == 0).all() and np.allclose(w.sum(1), 1, rtol=1e-6)
    low = np.where(mask, -1e30, logits).astype(np.float32)   # the same picks and weights, every expert finite
    check(form, x_bits, low, whole, k, y, torch.float32)
    ref = host(LAYER[form](*(to_dev(a) for a in weights), k=k)(bf16_to_dev(x_bits), to_dev(lg)))
    assert np.isfinite(ref).all()
    assert np.linalg.norm(host(y) - ref) <= 2e-3 * np.linalg.norm(ref)


@pytest.mark.parametrize("form", FORMS)
def test_layer_few_and_steps_agree_on_masks(form):
    """few=True and the steps: the same y for masked tokens and masked experts."""
    T, H, I, E, k = 7, 512, 256, 16, 4
    x_bits, logits, weights = make(form, T, H, I, E, k, seed=84)
    logits[0] = -INF
    logits[1, 3:] = -INF                                     # three left
    logits[2, :] = NAN
    logits[3, ::2] = NAN
    logits[4, [1, 5, 9]] = -INF
    dev = [to_dev(a) for a in weights]
    x, lg = bf16_to_dev(x_bits), to_dev(logits)
    say(f"layer {form}: masks, few=True against the steps")
    y = LAYER[form](*dev, k=k, few=True)(x, lg)
    ref = LAYER[form](*dev, k=k)(x, lg)
    assert torch.isfinite(ref).all() and torch.isfinite(y).all()
    assert not y[[0, 2]].any() and not ref[[0, 2]].any()
    for t in (1, 3, 4, 5, 6):
        assert float((y[t] - ref[t]).norm() / ref[t].norm()) <= 2e-3
