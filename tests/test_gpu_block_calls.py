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


def shifted(t, by=1):
    """t's values in memory that starts `by` elements behind an allocation's start."""
    buf = torch.empty(t.numel() + by, dtype=t.dtype, device=t.device)
    buf[by:] = t.reshape(-1)
    return buf[by:].view(t.shape)


@pytest.mark.parametrize("M", [1, 16, 17, 64, 130, 300, 1500])
def test_vectors_aligned_to_their_elements(M):
    """Scales, bias, addend and result of the products at addresses of their elements' alignment only."""
    g = np.random.Generator(np.random.PCG64(M))
    K, I = 400, 384
    c = lambda *s: torch.from_numpy(g.integers(-128, 128, size=s, dtype=np.int8)).to(DEV)  # noqa: E731
    f = lambda *s: torch.from_numpy(g.normal(size=s).astype(np.float32)).to(DEV)  # noqa: E731
    a, sa, w13, s13, w2, s2 = c(M, K), f(M), c(2 * I, K), 0.01 * f(2 * I), c(K, I), f(K)
    bias, add = f(2 * I), f(M, K)
    say(f"products with vectors at any element M={M}")
    for dt in (torch.float32, torch.bfloat16):
        want = ops.w4a8_moe_dense_i8(a, sa, w13, s13, bias=bias, y_dtype=dt)
        y = shifted(torch.zeros(M, 2 * I, dtype=dt, device=DEV))
        ops.w4a8_moe_dense_i8(a, shifted(sa), w13, shifted(s13, 3), bias=shifted(bias), y=y)
        assert torch.equal(y, want)
        want = ops.w4a8_moe_mlp_i8(a, sa, w13, s13, w2, s2, add=add.to(dt), y_dtype=dt)
        y = shifted(add.to(dt))
        ops.w4a8_moe_mlp_i8(a, shifted(sa, 2), w13, shifted(s13), w2, shifted(s2, 3), add=y, y=y)
        assert torch.equal(y, want)


@pytest.mark.parametrize("T,H", [(3, 512), (5, 2048), (2, 6144), (300, 6144), (300, 12288), (3, 20000)])
def test_norm_vectors_aligned_to_their_elements(T, H):
    g = np.random.Generator(np.random.PCG64(T + H))
    f = lambda *s: torch.from_numpy(g.normal(size=s).astype(np.float32)).to(DEV)  # noqa: E731
    y, r, w, gate, tg = f(T, H), f(T, H), f(H), f(H), f(T)
    say(f"norms with vectors at any element T={T} H={H}")
    for r_scale in (0.0, -1.5):
        kw = dict(post_weight=w, gate=gate, r_scale=r_scale)
        sums = torch.zeros(T, dtype=torch.int32, device=DEV)
        want = ops.w4a8_moe_residual_norm_quant_i8(y, r, w, token_gate=tg, rowsum=sums, **kw)
        q, s, more = shifted(torch.zeros_like(want[2]), 8), shifted(torch.zeros_like(want[3])), shifted(torch.zeros_like(sums))
        got = ops.w4a8_moe_residual_norm_quant_i8(y, r, w, token_gate=shifted(tg), qx=q, sx=s, rowsum=more, **kw)
        for a, b in zip((*got, more), (*want, sums)):
            assert torch.equal(a, b)
        n = y.double() * w.double() / torch.sqrt((y.double() ** 2).mean(1, keepdim=True) + 1e-6)
        p = n * gate.double() * tg.double()[:, None]
        out = r_scale * r.double() + p
        # the norm's fp32 error and two products, then the sum's rounding (a term and the sum may be one FMA)
        tol = (40 + 2) * 2.0 ** -24 * p.abs() + 2.0 ** -24 * out.abs()
        assert bool(((got[0].double() - out).abs() <= tol).all())
