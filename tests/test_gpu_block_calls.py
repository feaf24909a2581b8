"""Calls that the operators around the experts admit beside their bindings' usual ones: layer forwards from codes by
every GEMM kernel, and norms with some of their outputs left out."""
import numpy as np
import pytest
import torch

from gpu_util import DEV, say
from quantized_grouped_gemm_token_amd import ops
from test_gpu_block import H, block, router, stream_of
from test_gpu_few import FORMS

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    assert ops.w4a8_moe_device_supported(), "the current device is not a gfx950"
    yield
    torch.cuda.synchronize()


@pytest.mark.parametrize("algo", [ops.W4A8_GG_AUTO, ops.W4A8_GG_TILED], ids=["auto", "tiled"])
@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("T", [1, 5, 16, 17, 40, 130, 1000])
def test_codes_by_every_kernel(form, T, algo):
    """x's own codes give the bits of the steps' forward, also in a layer that would take few tokens in one call (under
    AUTO 40 tokens are left to both kernels' choice on the device, 130 and 1000 take the tiled one)."""
    moe = block(form, 5).moe
    x = stream_of(6, T, torch.bfloat16)
    lg = router(5)(x)
    codes = ops.w4a8_moe_quant_act_i8(x) if form == "channel" else ops.w4a8_moe_quant_act(x)
    say(f"layer {form} T={T} algo={algo} from codes")
    want = moe(x, lg, algo=algo)
    assert not moe.uses_few(T, algo)
    other = torch.zeros_like(x)                              # (x itself is not read)
    for few in (False, True):
        moe.few = few
        assert torch.equal(moe(other, lg, algo=algo, codes=codes), want)
    changed = (codes[0].flip(0), codes[1].flip(0), *(c.flip(0) for c in codes[2:]))
    if T > 1:
        assert not torch.equal(moe(x, lg, algo=algo, codes=changed), want)


@pytest.mark.parametrize("i8", [False, True], ids=["fp8", "i8"])
@pytest.mark.parametrize("T,H", [(3, 512), (5, 2048), (2, 6144), (300, 6144), (300, 12288), (3, 20000)])
def test_outputs_left_out(T, H, i8):
    """The C calls with codes alone, rows alone, and codes without their sums: what is written is what all together
    gives."""
    g = np.random.Generator(np.random.PCG64(T + H))
    x = torch.from_numpy(g.normal(size=(T, H)).astype(np.float32)).to(DEV)
    r = torch.from_numpy(g.normal(size=(T, H)).astype(np.float32)).to(DEV)
    w = torch.from_numpy((1 + 0.2 * g.normal(size=H)).astype(np.float32)).to(DEV)
    end = "_i8" if i8 else ""
    say(f"norms with outputs left out T={T} H={H} i8={i8}")
    new = lambda *shape, dtype: torch.full(shape, 3, dtype=dtype, device=DEV)  # noqa: E731

    def outputs():
        return [new(T, H, dtype=torch.bfloat16), new(T, H, dtype=torch.int8 if i8 else torch.uint8),
                new(T, dtype=torch.float32)] + ([new(T, dtype=torch.int32)] if i8 else [])

    def norm(outs):
        ops._call_on(x.device, "w4a8_moe_norm_quant" + end, x.data_ptr(), 0, T, H, H, w.data_ptr(), 1e-6,
                     *(ops._p(o) for o in outs))

    def residual(outs):
        out = torch.empty_like(x)
        ops._call_on(x.device, "w4a8_moe_residual_norm_quant" + end, x.data_ptr(), 0, H, r.data_ptr(), 0, H, T, H,
                     w.data_ptr(), None, None, 0.5, 1e-6, out.data_ptr(), H, w.data_ptr(), *(ops._p(o) for o in outs))
        return out
    for call in (norm, residual):
        whole = outputs()
        out = call(whole)
        for keep in ((0,), (1, 2), (0, 1, 2)) + (((1, 2, 3),) if i8 else ()):
            part = [o if i in keep else None for i, o in enumerate(outputs())]
            again = call(part)
            for i in keep:
                assert torch.equal(part[i], whole[i]), (call.__name__, keep, i)
            assert out is None or torch.equal(again, out)
