"""The host checks of the operators around the experts, without a GPU.

Pointers passed here are never dereferenced: every call fails a host check (or, on a
machine without a gfx950, the device check).
"""
import os
import re

import pytest
import torch

from quantized_grouped_gemm_token_amd import ops

OK, ERR_NULL, ERR_SHAPE, ERR_ALIGN, ERR_DEVICE, ERR_HIP, ERR_WORKSPACE = range(7)
P = 0x10000          # a fake, 64 KiB-aligned address (never dereferenced)
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
NAN, INF = float("nan"), float("inf")


def bound(name):
    return ops._function(name)


def absent():
    return not ops.lib().w4a8_moe_device_supported()


def test_every_declared_symbol_is_bound():
    text = open(os.path.join(ROOT, "include", "w4a8_block.h")).read()
    names = set(re.findall(r"\b(?:int|int64_t) (w4a8_moe_\w+)\s*\(", text))
    assert names == set(ops._BLOCK_SIGNATURES)
    for n in names:
        assert len(bound(n).argtypes) == re.search(n + r"\(([^;]*)\);", text).group(1).count(",") + 1, n


def test_dense_checks():
    f = bound("w4a8_moe_dense_i8")
    good = dict(a=P, sa=P, M=300, K=256, ld=256, w=P, sw=P, bias=None, N=100, add=None, y=P, dt=0)

    def call(**kw):
        return f(*dict(good, **kw).values(), None)
    assert call(M=-1) == ERR_SHAPE
    assert call(M=1 << 31) == ERR_SHAPE
    for K in (0, 8, 250, -16, 1 << 17):
        assert call(K=K, ld=1 << 18) == ERR_SHAPE, K
    for ld in (240, 250, 264, (1 << 22) + 16):
        assert call(ld=ld) == ERR_SHAPE, ld
    for N in (0, -1, (1 << 24) + 1):
        assert call(N=N) == ERR_SHAPE, N
    assert call(M=1 << 20, N=(1 << 20) + 1) == ERR_SHAPE
    assert call(dt=2) == ERR_SHAPE
    assert "dense_i8" in ops.last_error()
    for arg in ("a", "sa", "w", "sw", "y"):
        assert call(**{arg: None}) == ERR_NULL, arg
    for arg in ("a", "w"):
        assert call(**{arg: P + 8}) == ERR_ALIGN, arg
    for arg in ("sa", "sw", "bias", "add", "y"):
        assert call(**{arg: P + 2}) == ERR_ALIGN, arg
    assert call(y=P + 1, dt=1) == ERR_ALIGN
    assert call(M=0, a=None, sa=None, y=None) == OK
    if absent():
        assert call() == ERR_DEVICE
        assert call(bias=P, add=P, y=P + 2, dt=1) == ERR_DEVICE


def test_mlp_checks():
    f = bound("w4a8_moe_mlp_i8")
    good = dict(a=P, sa=P, M=30, H=144, ld=144, w13=P, s13=P, w2=P, s2=P, I=256, add=None, y=P, dt=0, ws=P,
                nbytes=1 << 40)

    def call(**kw):
        return f(*dict(good, **kw).values(), None)
    assert call(M=-1) == ERR_SHAPE
    for H in (0, 8, 1 << 17):
        assert call(H=H, ld=1 << 18) == ERR_SHAPE, H
    assert call(ld=128) == ERR_SHAPE
    assert call(ld=152) == ERR_SHAPE
    for I in (0, 64, -128, 65664):
        assert call(I=I) == ERR_SHAPE, I
    assert call(dt=-1) == ERR_SHAPE
    for arg in ("a", "sa", "w13", "s13", "w2", "s2", "y", "ws"):
        assert call(**{arg: None}) == ERR_NULL, arg
    for arg in ("a", "w13", "w2", "ws"):
        assert call(**{arg: P + 8}) == ERR_ALIGN, arg
    for arg in ("sa", "s13", "s2", "add", "y"):
        assert call(**{arg: P + 2}) == ERR_ALIGN, arg
    need = bound("w4a8_moe_mlp_i8_workspace_bytes")(30, 144, 256)
    assert need > 0 and call(nbytes=need - 1) == ERR_WORKSPACE
    assert call(M=0, a=None, y=None, ws=None, nbytes=0) == OK
    if absent():
        assert call(nbytes=need) == ERR_DEVICE
        assert call(add=P + 2, y=P + 2, dt=1) == ERR_DEVICE


def test_workspace_sizes():
    m = bound("w4a8_moe_mlp_i8_workspace_bytes")
    assert m(0, 128, 128) >= 0
    assert 0 < m(1, 6144, 2048) <= m(16, 6144, 2048) < m(4096, 6144, 2048)
    for bad in ((-1, 128, 128), (1, 8, 128), (1, 128, 64)):
        assert m(*bad) == -1
        with pytest.raises(ValueError):
            ops.w4a8_moe_mlp_i8_workspace_bytes(*bad)


@pytest.mark.parametrize("i8", [False, True])
def test_norm_checks(i8):
    f = bound("w4a8_moe_norm_quant" + ("_i8" if i8 else ""))
    good = dict(x=P, dt=1, T=4, H=64, ld=64, w=P, eps=1e-6, xn=P, q=P, s=P)
    if i8:
        good["rowsum"] = None

    def call(**kw):
        return f(*dict(good, **kw).values(), None)
    assert call(T=-1) == ERR_SHAPE
    assert call(T=1 << 31) == ERR_SHAPE
    for H in (0, -8, 60, 32776):
        assert call(H=H, ld=1 << 20) == ERR_SHAPE, H
    assert call(ld=56) == ERR_SHAPE
    assert call(ld=68) == ERR_SHAPE                          # 136 bytes in bf16
    assert call(dt=0, ld=66) == ERR_SHAPE
    assert call(dt=2) == ERR_SHAPE
    for eps in (0.0, -1e-6, 1e-31, NAN, INF):
        assert call(eps=eps) == ERR_SHAPE, eps
    for arg in ("x", "w", "q", "s"):
        assert call(**{arg: None}) == ERR_NULL, arg
    assert call(xn=None, q=None, s=None) == ERR_NULL
    for arg, by in (("x", 8), ("w", 8), ("xn", 8), ("q", 4), ("s", 2)):
        assert call(**{arg: P + by}) == ERR_ALIGN, arg
    if i8:
        assert call(q=None, s=None, rowsum=P) == ERR_NULL
        assert call(rowsum=P + 2) == ERR_ALIGN
    assert call(T=0, x=None, w=None, xn=None, q=None, s=None) == OK
    if absent():
        for kw in ({}, dict(xn=None), dict(q=None, s=None), dict(dt=0, ld=68)):
            assert call(**kw) == ERR_DEVICE


@pytest.mark.parametrize("form", ["", "_quant", "_quant_i8"])
def test_residual_checks(form):
    f = bound("w4a8_moe_residual_norm" + form)
    good = dict(y=P, ydt=1, ld_y=64, r=P, rdt=0, ld_r=64, T=4, H=64, post=None, gate=None, tg=None, rs=1.0, eps=1e-6,
                out=P, ld_out=64)
    if form:
        good.update(w=P, xn=P, q=P, s=P)
    if form == "_quant_i8":
        good["rowsum"] = None

    def call(**kw):
        return f(*dict(good, **kw).values(), None)
    assert call(T=-1) == ERR_SHAPE
    assert call(H=60) == ERR_SHAPE
    for ld in ("ld_y", "ld_r", "ld_out"):
        assert call(**{ld: 56}) == ERR_SHAPE, ld
        assert call(**{ld: 66}) == ERR_SHAPE, ld
    for dt in ("ydt", "rdt"):
        assert call(**{dt: 3}) == ERR_SHAPE, dt
    assert call(eps=0.0) == ERR_SHAPE
    for rs in (NAN, INF, -INF):
        assert call(rs=rs) == ERR_SHAPE
    for arg in ("y", "r", "out") + (("w", "q", "s") if form else ()):
        assert call(**{arg: None}) == ERR_NULL, arg
    for arg in ("y", "r", "out", "post", "gate") + (("w", "xn") if form else ()):
        assert call(**{arg: P + 8}) == ERR_ALIGN, arg
    assert call(tg=P + 2) == ERR_ALIGN
    assert call(T=0, y=None, r=None, out=None) == OK
    if absent():
        assert call() == ERR_DEVICE
        assert call(post=P, gate=P, tg=P + 4, rs=0.0, ydt=0, rdt=1) == ERR_DEVICE


def test_bindings_refuse_before_the_library():
    i8 = lambda *s: torch.zeros(*s, dtype=torch.int8)  # noqa: E731
    f = lambda *s: torch.zeros(*s)  # noqa: E731
    with pytest.raises(ValueError, match="GPU"):
        ops.w4a8_moe_dense_i8(i8(2, 16), f(2), i8(4, 16), f(4))
    with pytest.raises(TypeError, match="a must be"):
        ops.w4a8_moe_dense_i8(f(2, 16), f(2), i8(4, 16), f(4))
    with pytest.raises(TypeError, match="x must be"):
        ops.w4a8_moe_norm_quant(torch.zeros(2, 16, dtype=torch.float16), f(16))
    with pytest.raises(ValueError, match="GPU"):
        ops.w4a8_moe_residual_norm(f(2, 16), f(2, 16))
    with pytest.raises(TypeError, match="y must be a torch.Tensor"):
        ops.w4a8_moe_residual_norm(None, f(2, 16))


def test_overlaps_are_told_from_rows_between_rows():
    b = torch.zeros(6, 64)
    with pytest.raises(ValueError, match="out must not overlap r"):
        ops._no_overlap(b[:, :32], "out", ("r", b[:, 16:48]))
    with pytest.raises(ValueError):
        ops._no_overlap(b[1:], "out", ("r", b[:-1]))
    ops._no_overlap(b[:, :32], "out", ("r", b[:, 32:]), ("gate", None), ("y", torch.zeros(6, 32)))
    ops._no_overlap(b[:, 32:], "out", ("r", b[:, :32]))
    ops._no_overlap(b[:3], "out", ("r", b[3:]))
    with pytest.raises(ValueError):                          # the same rows, another distance between them
        ops._no_overlap(b.view(3, 128)[:, :32], "out", ("r", b[:, 32:]))
