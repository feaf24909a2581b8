"""The few-token layer's and the matrix-vector product's host checks, without a GPU.

Pointers passed here are never dereferenced: every call fails a host check (or, on a
machine without a gfx950, the device check).
"""
import pytest
import torch

from quantized_grouped_gemm_token_amd import ops

OK, ERR_NULL, ERR_SHAPE, ERR_ALIGN, ERR_DEVICE, ERR_HIP, ERR_WORKSPACE = range(7)
P = 0x10000          # a fake, 64 KiB-aligned address (never dereferenced)

FEW = ["w4a8_moe_few_prepacked", "w4a8_moe_few_i8_prepacked", "w4a8_moe_few_mxfp4_prepacked"]
MATVEC = ["w4a8_moe_matvec", "w4a8_moe_matvec_prepacked", "w4a8_moe_matvec_channel",
          "w4a8_moe_matvec_channel_prepacked", "w4a8_moe_matvec_mxfp4", "w4a8_moe_matvec_mxfp4_prepacked"]


@pytest.fixture(scope="module")
def L():
    return ops.lib()


@pytest.mark.parametrize("name", FEW)
def test_few_checks(L, name):
    f = getattr(L, name)
    good = dict(x=P, T=4, H=256, ld=256, lg=P, E=8, k=2, renorm=1, w13=P, s13=P, w2=P, s2=P, I=128, ids=None, w=None,
                y=P, dt=0, ws=P, nbytes=1 << 20)

    def call(**kw):
        return f(*dict(good, **kw).values(), None)
    assert call(T=17) == ERR_SHAPE
    assert call(T=-1) == ERR_SHAPE
    assert call(H=192) == ERR_SHAPE                          # H % 128
    assert call(H=8320, ld=8320) == ERR_SHAPE                # H > 8192
    assert call(T=15, H=8192, ld=8192) == ERR_SHAPE          # T H > 114688
    assert call(H=0) == ERR_SHAPE
    assert call(ld=248) == ERR_SHAPE
    assert call(ld=260) == ERR_SHAPE
    assert call(E=0) == ERR_SHAPE
    assert call(E=2000) == ERR_SHAPE
    assert call(k=9) == ERR_SHAPE                            # k > E
    assert call(k=0) == ERR_SHAPE
    assert call(T=16, E=64, k=17) == ERR_SHAPE               # T k > 256
    assert call(I=64) == ERR_SHAPE
    assert call(I=-128) == ERR_SHAPE
    assert call(dt=2) == ERR_SHAPE
    for arg in ("x", "lg", "w13", "s13", "w2", "s2", "y", "ws"):
        assert call(**{arg: None}) == ERR_NULL, arg
    for arg in ("x", "w13", "w2", "ws"):
        assert call(**{arg: P + 8}) == ERR_ALIGN, arg
    for arg in ("lg", "s13", "s2", "ids", "w", "y"):
        assert call(**{arg: P + 2}) == ERR_ALIGN, arg
    assert call(y=P + 1, dt=1) == ERR_ALIGN
    need = L.w4a8_moe_few_workspace_bytes(4, 2, 128)
    assert call(nbytes=need - 1) == ERR_WORKSPACE
    assert name[len("w4a8_moe_"):] in ops.last_error()
    assert call(T=0, x=None, lg=None, y=None, ws=None, nbytes=0) == OK
    if not L.w4a8_moe_device_supported():
        assert call(nbytes=need) == ERR_DEVICE
        assert call(y=P + 2, dt=1, ids=P, w=P) == ERR_DEVICE


def test_few_workspace_bytes(L):
    ws = L.w4a8_moe_few_workspace_bytes
    assert 0 < ws(0, 1, 128) < ws(1, 8, 2048) < ws(2, 8, 2048) < ws(16, 8, 2048) < 1 << 22
    for bad in ((17, 1, 128), (-1, 1, 128), (16, 17, 128), (1, 0, 128), (1, 1, 100), (1, 1, 0), (1, 257, 128),
                (1, 1, 65664)):
        assert ws(*bad) == -1
        with pytest.raises(ValueError):
            ops.w4a8_moe_few_workspace_bytes(*bad)


def test_few_layers_of_larger_experts_take_the_steps():
    from quantized_grouped_gemm_token_amd.layer import W4A8MoE
    moe = W4A8MoE.__new__(W4A8MoE)
    moe.few, moe.H, moe.k, moe.I = True, 128, 1, ops.FEW_MAX_I
    assert moe.uses_few(1) and not moe.uses_few(17)
    moe.I += 128
    assert not moe.uses_few(1)
    with pytest.raises(ValueError):
        ops.w4a8_moe_few_workspace_bytes(1, 1, moe.I)


def test_few_fits_is_the_rule(L):
    for T, H, k in [(1, 8192, 8), (14, 8192, 8), (15, 8192, 8), (16, 7168, 8), (16, 7296, 8), (17, 128, 1),
                    (16, 128, 16), (16, 128, 17), (1, 8320, 1), (1, 128, 256), (1, 128, 257)]:
        st = L.w4a8_moe_few_prepacked(P, T, H, H, P, 1024, k, 1, P, P, P, P, 128, None, None, P, 0, None, 0, None)
        assert (st != ERR_SHAPE) == ops.w4a8_moe_few_fits(T, H, k), (T, H, k)


@pytest.mark.parametrize("name", MATVEC)
def test_matvec_checks(L, name):
    f = getattr(L, name)
    stored = "prepacked" not in name
    good = dict(x=P, T=4, K=256, ld=256, w=P, s=P, N=64, y=P, dt=0)

    def call(**kw):
        return f(*dict(good, **kw).values(), None)
    assert call(T=17) == ERR_SHAPE
    assert call(T=-1) == ERR_SHAPE
    assert call(K=0) == ERR_SHAPE
    assert call(K=240, ld=256) == ERR_SHAPE
    if name != "w4a8_moe_matvec_mxfp4":
        assert call(K=160) == ERR_SHAPE                      # K % 128 (stored MXFP4: K % 32)
    assert call(ld=248) == ERR_SHAPE
    assert call(ld=260) == ERR_SHAPE
    assert call(N=0) == ERR_SHAPE
    assert call(N=-16) == ERR_SHAPE
    assert stored or call(N=40) == ERR_SHAPE                 # N % 16 in the GEMM storage
    assert call(dt=3) == ERR_SHAPE
    for arg in ("x", "w", "s", "y"):
        assert call(**{arg: None}) == ERR_NULL, arg
    assert call(x=P + 8) == ERR_ALIGN
    assert call(w=P + 8) == ERR_ALIGN
    assert call(y=P + 2) == ERR_ALIGN
    assert call(y=P + 1, dt=1) == ERR_ALIGN
    assert name == "w4a8_moe_matvec_mxfp4" or call(s=P + 2) == ERR_ALIGN
    assert name[len("w4a8_moe_"):] in ops.last_error() or name == "w4a8_moe_matvec_mxfp4"
    assert call(T=0, x=None, y=None) == OK
    if not L.w4a8_moe_device_supported():
        assert call() == ERR_DEVICE
        assert call(N=16, y=P + 2, dt=1) == ERR_DEVICE
        if stored:
            assert call(N=1) == ERR_DEVICE


def test_binding_refuses_before_the_library():
    x = torch.zeros((2, 256), dtype=torch.bfloat16)
    with pytest.raises(TypeError):
        ops.w4a8_moe_matvec(x.float(), x, x)
    with pytest.raises(ValueError):
        ops.w4a8_moe_matvec(x, x, x)                         # not on a GPU
    with pytest.raises(TypeError):
        ops.w4a8_moe_few_prepacked(x.float(), x, 1, x, x, x, x)
    with pytest.raises(ValueError):
        ops.w4a8_moe_few_prepacked(x, x, 1, x, x, x, x)
    with pytest.raises(TypeError):
        ops.w4a8_moe_few_prepacked([1.0], x, 1, x, x, x, x)
