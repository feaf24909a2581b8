"""Norms before and after a block, their codes, gates and residual, against 64-bit forms."""
import numpy as np
import pytest
import torch

from block_ref import HALF_BF16, HALF_F32, NORM_REL, check_codes, rms
from gpu_util import DEV, say
from quantized_grouped_gemm_token_amd import ops

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
EPS = 1e-6


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    assert ops.w4a8_moe_device_supported(), "the current device is not a gfx950"
    yield
    torch.cuda.synchronize()


def f64(t):
    torch.cuda.synchronize()
    return t.double().cpu().numpy()


def rows(g, T, H, dtype, pad=0, gain=1.0):
    x = g.normal(size=(T, H)) * gain
    x[:, g.random(H) < 0.01] *= 20
    buf = torch.full((T, H + pad), 99.0, dtype=TYPES[dtype], device=DEV)
    buf[:, :H] = torch.from_numpy(x).to(DEV)
    return buf[:, :H]


def vec(g, H):
    return torch.from_numpy((1 + 0.2 * g.normal(size=H)).astype(np.float32)).to(DEV)


def check_norm(n, xn, q, s, fp8, what, rel=NORM_REL, absolute=0.0):
    """n in 64 bits; the kernel's fp32 norm is within rel of it (and `absolute` of each row's largest value)."""
    top = np.abs(n).max(1, keepdims=True)
    tol = rel * np.abs(n) + absolute * top
    tol = tol + HALF_BF16 * (np.abs(n) + tol) + 2.0 ** -134   # (half a step of bf16's smallest)
    bad = ~(np.abs(f64(xn) - n) <= tol)
    assert not bad.any(), f"{what}: {int(bad.sum())} of xn off"
    check_codes(n, rel, absolute, q.cpu().numpy(), f64(s), fp8, what)


SIZES = [(1, 8, 0), (1, 6144, 0), (3, 16, 8), (5, 64, 0), (4, 504, 8), (7, 512, 0), (6, 520, 0), (9, 1024, 16),
         (2, 1032, 0), (33, 2048, 0), (5, 2056, 8), (3, 2920, 24), (4, 4096, 0), (2, 4104, 0), (128, 6144, 0),
         (2, 6152, 0), (3, 8192, 0), (2, 8200, 8), (2, 16384, 0), (2, 16392, 0), (3, 32768, 0), (1001, 296, 8)]


@pytest.mark.parametrize("form", ["fp8", "i8"])
@pytest.mark.parametrize("x", ["bf16", "f32"])
@pytest.mark.parametrize("T,H,pad", SIZES)
def test_norm_before(T, H, pad, x, form):
    g = np.random.Generator(np.random.PCG64(T * 100 + H))
    xt, w = rows(g, T, H, x, pad), vec(g, H)
    fn = ops.w4a8_moe_norm_quant if form == "fp8" else ops.w4a8_moe_norm_quant_i8
    say(f"norm_quant T={T} H={H} {x} {form} pad={pad}")
    if form == "i8":
        rowsum = torch.full((T,), 7, dtype=torch.int32, device=DEV)
        xn, q, s = fn(xt, w, EPS, rowsum=rowsum)
        assert torch.equal(rowsum, q.sum(1, dtype=torch.int32))
        for a, b in zip(fn(xt, w, EPS), (xn, q, s)):          # without the sums
            assert torch.equal(a, b)
    else:
        xn, q, s = fn(xt, w, EPS)
    assert xn.dtype is torch.bfloat16 and q.dtype is (torch.uint8 if form == "fp8" else torch.int8)
    check_norm(rms(f64(xt), f64(w), EPS), xn, q, s, form == "fp8", f"T={T} H={H}")


CASES = [dict(post=True, gate=True, token_gate=True), dict(post=True), dict(gate=True), dict(token_gate=True), dict()]


def residual_ref(y, r, post, gate, token_gate, r_scale):
    """(out, its fp32 error) in 64 bits."""
    p = f64(y)
    rel = 0.0
    if post is not None:
        p, rel = rms(p, f64(post), EPS), NORM_REL
    for v in (gate, None if token_gate is None else token_gate[:, None]):
        if v is not None:
            p, rel = p * f64(v), rel + HALF_F32
    out = r_scale * f64(r) + p
    return out, rel * np.abs(p) + HALF_F32 * np.abs(out)


@pytest.mark.parametrize("case", range(len(CASES)))
@pytest.mark.parametrize("form", ["none", "fp8", "i8"])
@pytest.mark.parametrize("y,r", [("f32", "f32"), ("bf16", "bf16"), ("bf16", "f32"), ("f32", "bf16")])
@pytest.mark.parametrize("T,H,pad", [(1, 6144, 0), (5, 8, 8), (9, 1000, 0), (130, 2920, 24), (3, 16384, 0), (2, 32768, 0)])
def test_residual(T, H, pad, y, r, form, case):
    g = np.random.Generator(np.random.PCG64(T * 100 + H + case))
    has = CASES[case]
    yt, rt = rows(g, T, H, y, pad), rows(g, T, H, r, 2 * pad)
    kw = dict(post_weight=vec(g, H) if has.get("post") else None, gate=vec(g, H) if has.get("gate") else None,
              token_gate=torch.rand(T, device=DEV) if has.get("token_gate") else None, r_scale=0.75, eps=EPS)
    say(f"residual T={T} H={H} {y} {r} {form} {has}")
    want, tol = residual_ref(yt, rt, kw["post_weight"], kw["gate"], kw["token_gate"], 0.75)
    if form == "none":
        out = ops.w4a8_moe_residual_norm(yt, rt, **kw)
    else:
        fn = ops.w4a8_moe_residual_norm_quant if form == "fp8" else ops.w4a8_moe_residual_norm_quant_i8
        nw = vec(g, H)
        out, xn, q, s = fn(yt, rt, nw, **kw)
    assert out.dtype is TYPES[r] and out.is_contiguous()
    bound = tol + (HALF_BF16 * (np.abs(want) + tol) if r == "bf16" else 0)
    bad = ~(np.abs(f64(out) - want) <= bound)
    assert not bad.any(), f"{int(bad.sum())} of out off"
    if form != "none":
        # the error of the sum next to its row's root mean square (where terms cancel, theirs stays), in each value
        # and in the mean square
        n = rms(want, f64(nw), EPS)
        off = tol.max(1) / np.sqrt((want * want).mean(1) + EPS)
        absolute = float((off * np.abs(f64(nw)).max() / np.abs(n).max(1)).max())
        check_norm(n, xn, q, s, form == "fp8", "next norm", NORM_REL + 1.01 * float(off.max()), 1.01 * absolute)
        assert torch.equal(ops.w4a8_moe_residual_norm(yt, rt, **kw), out)
    # over the residual itself (same row distance), and over y where the types are alike
    if not pad:
        for target in [rt.clone()] + ([yt.clone()] if y == r else []):
            args = (yt, target) if target.dtype is rt.dtype and torch.equal(target, rt) else (target, rt)
            assert ops.w4a8_moe_residual_norm(*args, out=target, **kw) is target
            assert torch.equal(target, out)


@pytest.mark.parametrize("H", [64, 6144, 20000])
@pytest.mark.parametrize("x", ["bf16", "f32"])
def test_rows_at_the_ends_of_the_range(x, H):
    """Zero rows, rows whose squares overflow or vanish, rows next to eps, and NaN and infinity in rows of their own."""
    g = np.random.Generator(np.random.PCG64(H))
    gains = [0.0, 1.0, 1e-3, 1e-12, 1e-30, 1e-37, 1e15, 1e19, 1e25, 1e36]
    xt = torch.cat([rows(g, 1, H, x, gain=k) for k in gains] + [rows(g, 3, H, x)])
    xt[-2, 5], xt[-1, 3], w = float("nan"), float("inf"), vec(g, H)
    for fp8, fn in ((True, ops.w4a8_moe_norm_quant), (False, ops.w4a8_moe_norm_quant_i8)):
        say(f"norm_quant H={H} {x} ends of the range")
        xn, q, s = fn(xt, w, EPS)
        k = len(gains) + 1
        v = f64(xt[:k])
        check_norm(rms(v, f64(w), EPS), xn[:k], q[:k], s[:k], fp8, "ends", absolute=2.0 ** -24)
        assert bool((xn[0] == 0).all()) and float(s[0]) == 1.0 and bool((q[0] == 0).all() if not fp8 else ((q[0] & 127) == 0).all())
        assert bool(torch.isnan(s[k:]).all())                # a row with a NaN or an infinity says so
        alone = fn(xt[:k].contiguous(), w, EPS)
        for a, b in zip(alone, (xn, q, s)):                  # and leaves the others as they are
            assert torch.equal(a, b[:k])


@pytest.mark.parametrize("eps", [2.0 ** -100, 1e-12, 1e-2, 10.0])
def test_eps(eps):
    g = np.random.Generator(np.random.PCG64(3))
    x = torch.cat([rows(g, 1, 512, "f32", gain=k) for k in (1.0, 1e-3, 1e-6, 1e-13, 1e-15, 1e-18)])
    w = vec(g, 512)
    xn, q, s = ops.w4a8_moe_norm_quant(x, w, eps)
    check_norm(rms(f64(x), f64(w), eps), xn, q, s, True, f"eps={eps}")


@pytest.mark.parametrize("T,H", [(1, 128), (7, 2048), (5, 6144)])
def test_memory_around_the_results_is_left(T, H):
    g = np.random.Generator(np.random.PCG64(T))
    y, r, w = rows(g, T, H, "bf16"), rows(g, T, H, "f32"), vec(g, H)
    guard = lambda n, dt: torch.full((n + 512,), 3, dtype=dt, device=DEV)  # noqa: E731
    bo, bx, bq, bs, br = guard(T * H, torch.float32), guard(T * H, torch.bfloat16), guard(T * H, torch.int8), \
        guard(T, torch.float32), guard(T, torch.int32)
    cut = lambda b, *sh: b[256:256 + int(np.prod(sh))].view(*sh)  # noqa: E731
    say(f"residual_norm_quant_i8 guard T={T} H={H}")
    got = ops.w4a8_moe_residual_norm_quant_i8(y, r, w, out=cut(bo, T, H), xn=cut(bx, T, H), qx=cut(bq, T, H),
                                              sx=cut(bs, T), rowsum=cut(br, T))
    want = ops.w4a8_moe_residual_norm_quant_i8(y, r, w)
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    for b, n in ((bo, T * H), (bx, T * H), (bq, T * H), (bs, T), (br, T)):
        assert bool((b[:256] == 3).all()) and bool((b[256 + n:] == 3).all())


def test_rows_between_rows():
    """y and r as the two halves of one buffer's rows, out the residual's half."""
    g = np.random.Generator(np.random.PCG64(1))
    both = torch.from_numpy(g.normal(size=(6, 512)).astype(np.float32)).to(DEV)
    y, r = both[:, :256], both[:, 256:]
    want = ops.w4a8_moe_residual_norm(y.contiguous(), r.contiguous())
    ops.w4a8_moe_residual_norm(y, r, out=r)
    assert torch.equal(r, want)


@pytest.mark.parametrize("T", [1, 300])
def test_graph_and_stream(T):
    g = np.random.Generator(np.random.PCG64(T))
    H = 6144
    y, r, w, pw = rows(g, T, H, "bf16"), rows(g, T, H, "f32"), vec(g, H), vec(g, H)
    want = ops.w4a8_moe_residual_norm_quant(y, r, w, pw)
    outs = [torch.zeros_like(t) for t in want]
    torch.cuda.synchronize()
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        ops.w4a8_moe_residual_norm_quant(y, r, w, pw, out=outs[0], xn=outs[1], qx=outs[2], sx=outs[3])
    for rep in range(3):
        for t in outs:
            t.zero_()
        gr.replay()
        eager = ops.w4a8_moe_norm_quant(y, w)
        torch.cuda.synchronize()
        for a, b in zip(outs, want):
            assert torch.equal(a, b)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = ops.w4a8_moe_norm_quant(y, w)
    torch.cuda.synchronize()
    for a, b in zip(other, eager):
        assert torch.equal(a, b)


@pytest.mark.parametrize("y,r", [("bf16", "bf16"), ("f32", "f32")])
@pytest.mark.parametrize("T,H", [(300, 4096), (257, 4104), (300, 6144), (300, 8192), (300, 16384), (260, 20000),
                                 (17000, 2056)])
def test_many_rows(T, H, y, r):
    """More rows than CUs, each number of threads to a row, and rows marked as read once (the largest)."""
    g = np.random.Generator(np.random.PCG64(T + H))
    base = rows(g, min(T, 300), H, y), rows(g, min(T, 300), H, r)
    yt, rt = (b.repeat(-(-T // b.shape[0]), 1)[:T].contiguous() for b in base)
    nw, pw = vec(g, H), vec(g, H)
    say(f"residual_norm_quant T={T} H={H} {y} {r}")
    got = ops.w4a8_moe_residual_norm_quant(yt, rt, nw, pw, r_scale=0.5)
    n = base[0].shape[0]
    want, tol = residual_ref(base[0], base[1], pw, None, None, 0.5)
    bound = tol + (HALF_BF16 * (np.abs(want) + tol) if r == "bf16" else 0)
    assert np.all(np.abs(f64(got[0][:n]) - want) <= bound)
    ref = rms(want, f64(nw), EPS)
    off = tol.max(1) / np.sqrt((want * want).mean(1) + EPS)
    absolute = float((off * np.abs(f64(nw)).max() / np.abs(ref).max(1)).max())
    check_norm(ref, got[1][:n], got[2][:n], got[3][:n], True, "next norm", NORM_REL + 1.01 * float(off.max()),
               1.01 * absolute)
    for t in got:                                            # the same rows again
        for k in range(n, T - n + 1, n):
            assert torch.equal(t[k:k + n], t[:n])
    x8 = ops.w4a8_moe_norm_quant_i8(yt, nw, EPS)
    check_norm(rms(f64(base[0]), f64(nw), EPS), x8[0][:n], x8[1][:n], x8[2][:n], False, "norm")


@pytest.mark.parametrize("i8", [False, True], ids=["fp8", "i8"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("T,H", [(2000, 6144), (300, 264), (40, 32768)])
def test_codes_are_the_nearest(i8, dtype, T, H):
    """The code of every value is the nearest to its quotient by the row's largest value (the norm's factor is in
    neither): products of two fp32 values are exact in 64 bits, the quotient is off by 2^-52 of itself, and quotients
    within 2^-42 of a border (the kernel takes 2^-43 for a tie) may have either code."""
    gen = torch.Generator(device=DEV).manual_seed(T + H)
    x = torch.randn(T, H, device=DEV, generator=gen).to(dtype)
    w = 1 + 0.2 * torch.randn(H, device=DEV, generator=gen)
    say(f"nearest codes T={T} H={H} {dtype} i8={i8}")
    _, q, _ = (ops.w4a8_moe_norm_quant_i8 if i8 else ops.w4a8_moe_norm_quant)(x, w, 1e-5)
    n = x.double() * w.double()
    v = n / n.abs().amax(1, keepdim=True) * (127.0 if i8 else 448.0)
    if i8:
        got, step = q.double(), torch.ones_like(v)
    else:
        got = q.view(torch.float8_e4m3fn).double()
        e = (torch.frexp(v)[1] - 1).clamp_min(-6)              # 3 bits behind the leading one, 2^-9 the smallest step
        step = torch.ldexp(torch.ones_like(v), e - 3)
    assert bool(((got - v).abs() <= step / 2 + 2.0 ** -42 * v.abs()).all())


def test_no_rows_and_largest():
    w = torch.ones(64, device=DEV)
    xn, q, s = ops.w4a8_moe_norm_quant(torch.empty(0, 64, device=DEV), w)
    assert tuple(xn.shape) == (0, 64) and tuple(s.shape) == (0,)
    assert tuple(ops.w4a8_moe_residual_norm(torch.empty(0, 64, device=DEV), torch.empty(0, 64, device=DEV)).shape) == (0, 64)
    T, H = 400000, 6144                                      # 4.9 GB of bf16: offsets past 32 bits
    x = torch.randn(1000, H, device=DEV).to(torch.bfloat16).repeat(T // 1000, 1)
    say(f"norm_quant T={T} H={H}")
    w = torch.ones(H, device=DEV)
    xn, q, s = ops.w4a8_moe_norm_quant(x, w)
    part = ops.w4a8_moe_norm_quant(x[:1000].contiguous(), w)
    for a, b in zip((xn, q, s), part):
        assert torch.equal(a[-1000:], b) and torch.equal(a[200000:201000], b)


@pytest.mark.parametrize("T,H", [((1 << 26) + 5, 8), ((1 << 22) + 3, 2056)])
def test_more_rows_than_a_launch_has_in_x(T, H):
    gen = torch.Generator(device=DEV).manual_seed(H)
    x = torch.empty(T, H, dtype=torch.bfloat16, device=DEV).normal_(generator=gen)
    w = torch.rand(H, device=DEV, generator=gen)
    say(f"norm T={T} H={H}")
    whole = ops.w4a8_moe_norm_quant_i8(x, w)
    res = ops.w4a8_moe_residual_norm(x, x, post_weight=w)
    for rows in (slice(0, 300), slice((1 << 21) - 150, (1 << 21) + 150), slice(T - 300, T)):
        for got, want in zip(whole, ops.w4a8_moe_norm_quant_i8(x[rows], w)):
            assert torch.equal(got[rows], want)
        assert torch.equal(res[rows], ops.w4a8_moe_residual_norm(x[rows], x[rows], post_weight=w))
