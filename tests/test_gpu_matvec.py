"""Matrix-vector products with 4-bit weights against the exact product in 64 bits.

The bound per element is derived: fp32 sums of G = K/128 groups in 8 parts, whose
terms are x (q + 8) and -8 x for the INT4 forms and x w for MXFP4, plus half a step of
bf16 where y is bf16.
"""
import numpy as np
import pytest
import torch

import oracle
from gpu_util import bf16_to_dev, say, to_dev
from oracle import mxfp4_oracle as mx
from quantized_grouped_gemm_token_amd import ops

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
FORMS = ("g128", "channel", "mxfp4")
STORED = {"g128": ops.w4a8_moe_matvec, "channel": ops.w4a8_moe_matvec_channel, "mxfp4": ops.w4a8_moe_matvec_mxfp4}
BLK = {"g128": ops.w4a8_moe_matvec_prepacked, "channel": ops.w4a8_moe_matvec_channel_prepacked,
       "mxfp4": ops.w4a8_moe_matvec_mxfp4_prepacked}

# T, N, K
SHAPES = [
    (1, 16, 128), (16, 16, 128),     # one group: seven waves without work
    (1, 1, 256), (3, 17, 384),       # fewer outputs than a tile, one more than a tile
    (5, 4096, 256), (16, 80, 6144),
    (2, 1000, 1152),                 # nine groups: two waves' shares are not whole
    (9, 33, 16512),                  # 129 groups
    (8, 6144, 2048), (4, 2049, 1024),
    (1, 8208, 640), (16, 8192, 384),
    (16, 16400, 256),                # steps of 32 columns, the last of 16
    (3, 8208, 6272),                 # .. and K in parts
]


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    assert ops.w4a8_moe_device_supported(), "the current device is not a gfx950"
    yield
    torch.cuda.synchronize()


def make(form, T, N, K, rng):
    x = rng.standard_normal((T, K)).astype(np.float32)
    x[:, rng.random(K) < 0.01] *= 20
    x_bits = oracle.f32_to_bf16_bits(x)
    if form == "mxfp4":
        w = rng.integers(0, 256, size=(N, K // 2), dtype=np.uint8)
        s = (127 + np.rint(rng.normal(-6, 1, size=(N, K // 32)))).astype(np.uint8)
    else:
        w = rng.integers(0, 2**32, size=(N, K // 8), dtype=np.uint32).view(np.int32)
        s = rng.lognormal(-4, 0.5, size=(N, K // 128) if form == "g128" else (N,)).astype(np.float32)
    return x_bits, w, s


def exact(form, x_bits, w, s):
    """(y, tol): the product in 64 bits, and the bound of an fp32 sum of its terms."""
    x = oracle.bf16_bits_to_f32(x_bits).astype(np.float64)
    K = x.shape[1]
    if form == "mxfp4":
        W = mx.dequant_mxfp4(w, s).astype(np.float64)
        B = np.abs(W)
    else:
        q = oracle.int4_unpack(w).astype(np.float64)
        f = np.repeat(s.astype(np.float64), 128, -1) if form == "g128" else s.astype(np.float64)[:, None]
        W, B = q * f, (q + 16) * np.abs(f)
    # at most G + 8 (waves) + 8 rounded additions and products in a row
    return x @ W.T, (-(-K // 128) + 16) * U * (np.abs(x) @ B.T) + 2.0 ** -126


def prepack(form, w, s):
    if form == "mxfp4":
        wb, sb = ops.w4a8_moe_prepack_mxfp4(to_dev(w[None]), to_dev(s[None]))
        return wb[0], sb[0]
    if form == "channel":
        return ops.w4a8_moe_prepack_int4(to_dev(w[None]))[0][0], to_dev(s)
    wb, sb = ops.w4a8_moe_prepack_int4(to_dev(w[None]), to_dev(s[None]))
    return wb[0], sb[0]


def check(y, want, tol, what):
    got = y.double().cpu().numpy()
    if y.dtype == torch.bfloat16:
        tol = tol + 2.0 ** -8 * (np.abs(want) + tol)
    off = np.abs(got - want)
    assert (off <= tol).all(), f"{what}: off by up to {float((off / tol).max()):.2f} of the bound"


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("T,N,K", SHAPES)
def test_matvec_against_64_bits(form, T, N, K, rng):
    x_bits, w, s = make(form, T, N, K, rng)
    want, tol = exact(form, x_bits, w, s)
    say(f"matvec {form} T={T} N={N} K={K}")
    x, wd, sd = bf16_to_dev(x_bits), to_dev(w), to_dev(s)
    y = STORED[form](x, wd, sd)
    check(y, want, tol, "stored")
    assert torch.equal(STORED[form](x, wd, sd, y_dtype=torch.bfloat16), y.to(torch.bfloat16))
    if N % 16 == 0:
        blk = BLK[form](x, *prepack(form, w, s))
        check(blk, want, tol, "GEMM storage")
        assert torch.equal(blk, y)                          # the same values in the same order
    for t in {0, T - 1}:                                    # a row's result does not depend on the others
        assert torch.equal(STORED[form](x[t:t + 1], wd, sd), y[t:t + 1])


@pytest.mark.parametrize("form", FORMS)
def test_matvec_a_row_that_is_not_finite_keeps_to_itself(form, rng):
    T, N, K = 6, 48, 1152
    x_bits, w, s = make(form, T, N, K, rng)
    say(f"matvec {form} with NaN and infinities in x")
    x, wd, sd = bf16_to_dev(x_bits), to_dev(w), to_dev(s)
    want = STORED[form](x, wd, sd)
    bad = x.clone()
    bad[2, 5], bad[5, :] = float("nan"), float("inf")
    got = STORED[form](bad, wd, sd)
    assert torch.equal(got[[0, 1, 3, 4]], want[[0, 1, 3, 4]])
    assert not torch.isfinite(got[[2, 5]]).any()


@pytest.mark.parametrize("K", [32, 96, 160, 2912, 4064])
def test_matvec_mxfp4_rows_that_end_inside_a_group(K, rng):
    T, N = 3, 37
    x_bits, w, s = make("mxfp4", T, N, K, rng)
    want, tol = exact("mxfp4", x_bits, w, s)
    say(f"matvec mxfp4 K={K}")
    # x's rows end at the end of their allocation, and what follows a row in a wider one is NaN
    check(ops.w4a8_moe_matvec_mxfp4(bf16_to_dev(x_bits), to_dev(w), to_dev(s)), want, tol, "whole")
    wide = torch.full((T, K + 40), float("nan"), dtype=torch.bfloat16, device="cuda:0")
    wide[:, :K] = bf16_to_dev(x_bits)
    y = ops.w4a8_moe_matvec_mxfp4(wide[:, :K], to_dev(w), to_dev(s))
    check(y, want, tol, "strided")


def test_matvec_mxfp4_scale_range():
    """Block scales at both ends of E8M0: 2^-127 to 2^120."""
    K, N = 128, 16
    x = np.ones((1, K), np.float32)
    w = np.full((N, K // 2), 0x22, np.uint8)                # every code 1.0
    s = np.zeros((N, K // 32), np.uint8)
    s[:8] = np.arange(8)[:, None] * 35                      # 2^-127, 2^-92, ..., 2^118
    s[8:] = 127
    say("matvec mxfp4 scale range")
    y = ops.w4a8_moe_matvec_mxfp4(bf16_to_dev(oracle.f32_to_bf16_bits(x)), to_dev(w), to_dev(s)).double().cpu().numpy()
    want = 128.0 * np.exp2(s[:, 0].astype(np.float64) - 127)
    assert np.allclose(y[0, 1:], want[1:], rtol=1e-6)
    assert abs(y[0, 0] - want[0]) <= 2.0 ** -120            # subnormal terms may be flushed


def test_matvec_strides_and_neighbours(rng):
    T, N, K = 5, 50, 512
    x_bits, w, s = make("g128", T, N, K, rng)
    x, wd, sd = bf16_to_dev(x_bits), to_dev(w), to_dev(s)
    say("matvec strided x, y inside a larger buffer")
    want = ops.w4a8_moe_matvec(x, wd, sd)
    wide = torch.full((T, K + 8), float("nan"), dtype=torch.bfloat16, device="cuda:0")
    wide[:, :K] = x
    assert torch.equal(ops.w4a8_moe_matvec(wide[:, :K], wd, sd), want)
    buf = torch.full((T + 2, N), 9.0, device="cuda:0")
    ops.w4a8_moe_matvec(x, wd, sd, y=buf[1:1 + T])
    assert torch.equal(buf[1:1 + T], want) and (buf[0] == 9).all() and (buf[-1] == 9).all()
    flat = torch.full((T * N + 3,), 9.0, dtype=torch.bfloat16, device="cuda:0")
    ops.w4a8_moe_matvec(x, wd, sd, y=flat[1:1 + T * N].view(T, N))      # two-byte aligned
    assert torch.equal(flat[1:1 + T * N].view(T, N), want.to(torch.bfloat16))
    assert (flat[:1] == 9).all() and (flat[-2:] == 9).all()
    assert ops.w4a8_moe_matvec(x[:0], wd, sd).shape == (0, N)


def test_matvec_far_rows():
    """Outputs whose weights start past 2^32 bytes give what they give in a small matrix."""
    N, K = 16 * 90000, 6144
    gen = torch.Generator(device="cuda:0").manual_seed(3)
    w = torch.randint(-2**31, 2**31, (N // 16, K // 128, 16, 16), generator=gen, device="cuda:0", dtype=torch.int32)
    s = torch.rand(K // 128, N, generator=gen, device="cuda:0") * 0.01
    assert w[-1:].data_ptr() - w.data_ptr() > 2**32
    x = torch.randn(2, K, generator=gen, device="cuda:0").to(torch.bfloat16)
    say("matvec with rows past 4 GiB")
    y = ops.w4a8_moe_matvec_prepacked(x, w, s)
    tail = ops.w4a8_moe_matvec_prepacked(x, w[-3:].contiguous(), s[:, -48:].contiguous())
    assert torch.equal(y[:, -48:], tail) and float(tail.abs().max()) > 0
    rows = w.view(N, K // 8)                               # the same bytes taken as stored rows
    sr = torch.rand(N, generator=gen, device="cuda:0")
    y = ops.w4a8_moe_matvec_channel(x, rows, sr)
    tail = ops.w4a8_moe_matvec_channel(x, rows[-33:].contiguous(), sr[-33:].contiguous())
    assert torch.equal(y[:, -33:], tail)


@pytest.mark.parametrize("form", FORMS)
def test_matvec_graph_and_streams(form, rng):
    T, N, K = 4, 512, 1024
    x_bits, w, s = make(form, T, N, K, rng)
    x, wb = bf16_to_dev(x_bits), prepack(form, w, s)
    xs = [x, x * 2, -x]
    want = [BLK[form](a, *wb) for a in xs]
    buf, y = x.clone(), torch.empty_like(want[0])
    say(f"matvec {form} captured")
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        BLK[form](buf, *wb, y=y)
    for i in range(4):
        buf.copy_(xs[i % 3])
        y.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want[i % 3])
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    for _ in range(20):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                got[i].append(BLK[form](xs[i], *wb))
    torch.cuda.synchronize()
    assert all(torch.equal(v, want[i]) for i in range(2) for v in got[i])


def test_layer_and_projections_together(rng):
    """A decode step as they are used: a 4-bit projection, the router's logits, the layer, a 4-bit output head."""
    T, H, I, E, k, V = 3, 512, 256, 8, 2, 1000
    from test_gpu_few import make as make_layer, prepack as prepack_layer, reference
    x_bits, w, s = make("g128", T, H, H, rng)
    _, wh, sh = make("mxfp4", T, V, H, rng)
    _, logits, experts = make_layer("g128", T, H, I, E, k, seed=9)
    packed, lg = prepack_layer("g128", experts), to_dev(logits)
    say("projection, layer, head in a row")
    h = ops.w4a8_moe_matvec(bf16_to_dev(x_bits), to_dev(w), to_dev(s), y_dtype=torch.bfloat16)
    y = ops.w4a8_moe_few_prepacked(h, lg, k, *packed, y_dtype=torch.bfloat16)
    out = ops.w4a8_moe_matvec_mxfp4(y, to_dev(wh), to_dev(sh))
    # each step against 64 bits on the bits the step before it gave
    bits = lambda t: t.view(torch.int16).cpu().numpy().view(np.uint16)  # noqa: E731
    check(h, *exact("g128", x_bits, w, s), "projection")
    _, _, ref, tol = reference("g128", bits(h), logits, experts, k)
    check(y, ref, tol, "layer")
    check(out, *exact("mxfp4", bits(y), wh, sh), "head")


def test_matvec_refusals(rng):
    x_bits, w, s = make("g128", 2, 32, 256, rng)
    x, wd, sd = bf16_to_dev(x_bits), to_dev(w), to_dev(s)
    call = ops.w4a8_moe_matvec
    say("matvec refusals")
    with pytest.raises(TypeError):
        call(x.half(), wd, sd)
    with pytest.raises(ValueError):
        call(x[:, :128], wd, sd)                            # another K than the weights
    with pytest.raises(ValueError):
        call(x, wd, sd[:, :1].contiguous())
    with pytest.raises(TypeError):
        call(x, wd.view(torch.uint8), sd)
    with pytest.raises(ValueError):
        call(x, wd[:, :16], sd)                             # weights that are not contiguous
    with pytest.raises(ops.W4A8Error):
        call(x.repeat(9, 1), wd, sd)                        # 18 rows
    with pytest.raises(ops.W4A8Error):
        call(torch.zeros(2 * 256 + 1, dtype=torch.bfloat16, device="cuda:0")[1:].view(2, 256), wd, sd)
    with pytest.raises(ValueError):
        call(x, wd, sd, y=torch.empty(2, 33, device="cuda:0"))
    with pytest.raises(TypeError):
        call(x, wd, sd, y=torch.empty(2, 32, dtype=torch.float64, device="cuda:0"))
    with pytest.raises(ValueError):
        ops.w4a8_moe_matvec_prepacked(x, wd.view(2, 2, 32, 8), sd)
