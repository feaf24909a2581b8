"""Dense products in 8-bit integers and the gated block on them, against 64-bit forms."""
import numpy as np
import pytest
import torch

from block_ref import check_dense, check_mlp, dense_f32
from gpu_util import DEV, say
from quantized_grouped_gemm_token_amd import ops

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    assert ops.w4a8_moe_device_supported(), "the current device is not a gfx950"
    yield
    torch.cuda.synchronize()


def codes(g, rows, K):
    return g.integers(-128, 128, size=(rows, K), dtype=np.int8)


def scales(g, n, K):
    return np.exp(g.normal(-np.log(5000.0 * np.sqrt(K)) / 2, 0.3, n)).astype(np.float32)


def strided(x: np.ndarray, ld: int) -> torch.Tensor:
    buf = torch.zeros(x.shape[0], ld, dtype=torch.from_numpy(x).dtype, device=DEV)
    buf[:, x.shape[1]:] = 77
    buf[:, :x.shape[1]] = torch.from_numpy(x).to(DEV)
    return buf[:, :x.shape[1]]


def dev(x):
    return None if x is None else torch.from_numpy(np.ascontiguousarray(x)).to(DEV)


def f64(t):
    torch.cuda.synchronize()
    return t.double().cpu().numpy()


# one row, the ends of tiles and of their parts, one output, K of one chunk, tails of every kind, strides
SHAPES = [(1, 1, 16, 0), (1, 64, 128, 0), (1, 6144, 6144, 0), (2, 17, 48, 16), (3, 100, 144, 0), (5, 257, 6128, 0),
          (8, 1000, 2048, 0), (15, 33, 112, 64), (16, 512, 640, 0), (17, 65, 128, 0), (31, 129, 272, 16),
          (33, 640, 1040, 0), (63, 127, 256, 0), (64, 64, 64, 0), (65, 300, 2896, 32), (77, 501, 2896, 32),
          (128, 128, 128, 0), (128, 768, 6144, 0), (129, 257, 384, 0), (200, 1000, 1008, 0), (255, 255, 80, 16),
          (256, 256, 256, 0), (257, 513, 400, 0), (300, 2048, 1024, 0), (513, 771, 528, 16), (1000, 1001, 2064, 0)]


@pytest.mark.parametrize("M,N,K,pad", SHAPES)
def test_products_are_exact(M, N, K, pad):
    g = np.random.Generator(np.random.PCG64(M * 1000003 + N * 1009 + K))
    a, w = codes(g, M, K), codes(g, N, K)
    sa, sw = scales(g, M, K), scales(g, N, K)
    say(f"dense_i8 M={M} N={N} K={K} pad={pad}")
    y = ops.w4a8_moe_dense_i8(strided(a, K + pad), dev(sa), dev(w), dev(sw))
    assert y.dtype is torch.float32 and tuple(y.shape) == (M, N)
    want = dense_f32(a, sa, w, sw)
    got = y.cpu().numpy()
    assert np.array_equal(got, want), f"{int((got != want).sum())} of {want.size} differ"
    y16 = ops.w4a8_moe_dense_i8(strided(a, K + pad), dev(sa), dev(w), dev(sw), y_dtype=torch.bfloat16)
    assert torch.equal(y16.cpu(), torch.from_numpy(want).to(torch.bfloat16))


@pytest.mark.parametrize("y", ["f32", "bf16"])
@pytest.mark.parametrize("M,N,K,pad", [(1, 96, 64, 0), (7, 333, 1040, 16), (40, 130, 208, 0), (130, 200, 128, 0),
                                       (300, 515, 272, 48)])
def test_bias_and_addend(M, N, K, pad, y):
    g = np.random.Generator(np.random.PCG64(M + N + K))
    a, w, sa, sw = codes(g, M, K), codes(g, N, K), scales(g, M, K), scales(g, N, K)
    bias = g.normal(size=N).astype(np.float32)
    add = torch.from_numpy(g.normal(size=(M, N)).astype(np.float32)).to(TYPES[y]).to(DEV)
    at = strided(a, K + pad)
    for b, c in ((bias, None), (None, add), (bias, add)):
        say(f"dense_i8 M={M} N={N} K={K} {y} bias={b is not None} add={c is not None}")
        got = ops.w4a8_moe_dense_i8(at, dev(sa), dev(w), dev(sw), bias=dev(b), add=c, y_dtype=TYPES[y])
        check_dense(f64(got), a, sa, w, sw, b, None if c is None else f64(c), y == "bf16")
    inplace = add.clone()                                     # the addend is the result's own memory
    assert ops.w4a8_moe_dense_i8(at, dev(sa), dev(w), dev(sw), bias=dev(bias), add=inplace, y=inplace) is inplace
    assert torch.equal(inplace, got)


# rows and outputs past every tile's edge (64 x 64, 128 x 64, 128 x 128, 256 x 128 and 256 x 256), K of an odd number
# of steps, few K steps, and for 16 rows and fewer each number of K units of a wave
@pytest.mark.parametrize("M,N,K", [(100, 333, 1008), (500, 2999, 400), (500, 6011, 144), (1000, 6011, 208),
                                   (3001, 3999, 16), (2999, 6001, 400), (4097, 8193, 272), (1025, 12290, 1040),
                                   (3, 260, 2064), (16, 333, 4112), (2, 100, 8208), (7, 77, 12288), (16, 129, 12304),
                                   (9, 4100, 16384), (1, 300, 16400), (16, 35, 40000)])
@pytest.mark.parametrize("y", ["f32", "bf16"])
def test_every_tile(M, N, K, y):
    a, sa, w, sw = _large(M, N, K, M + N + K)
    gen = torch.Generator(device=DEV).manual_seed(N)
    bias = torch.randn(N, device=DEV, generator=gen)
    buf = torch.randn((M + 2) * N, device=DEV, generator=gen).to(TYPES[y])
    edges = buf[:N].clone(), buf[-N:].clone()
    add = buf[N:-N].view(M, N)
    say(f"dense_i8 M={M} N={N} K={K} {y}")
    sums = a.double() @ w.double().t()
    assert torch.equal(ops.w4a8_moe_dense_i8(a, sa, w, sw, y_dtype=TYPES[y]),
                       (sums.float() * sa[:, None] * sw).to(TYPES[y]))
    # with bias and addend check_dense's bound: three half steps of the product, one of each sum, one of bf16
    p = sums * sa.double()[:, None] * sw.double()
    first = p + bias
    want = first + add
    tol = 1.001 * 2.0 ** -24 * (3 * p.abs() + first.abs() + want.abs()) + 2.0 ** -149
    if y == "bf16":
        tol += 2.0 ** -8 * (want.abs() + tol)
    assert ops.w4a8_moe_dense_i8(a, sa, w, sw, bias=bias, add=add, y=add) is add
    assert bool(((add - want).abs() <= tol).all())
    assert torch.equal(buf[:N], edges[0]) and torch.equal(buf[-N:], edges[1])


@pytest.mark.parametrize("M,H,I", [(2, 64, 20480), (16, 32, 12288), (5, 20480, 128), (11, 12304, 256), (1, 8208, 640),
                                   (16, 80, 65536), (40, 80, 20480)])
def test_gated_block_of_long_rows(M, H, I):
    """The few-row kernels' parts of K, on either side of the activation."""
    g = np.random.Generator(np.random.PCG64(M + H + I))
    a, w13, w2 = codes(g, M, H), codes(g, 2 * I, H), codes(g, H, I)
    sa, s13, s2 = scales(g, M, H), scales(g, 2 * I, H), scales(g, H, I)
    say(f"mlp_i8 M={M} H={H} I={I}")
    got = ops.w4a8_moe_mlp_i8(dev(a), dev(sa), dev(w13), dev(s13), dev(w2), dev(s2))
    check_mlp(f64(got), a, sa, w13, s13, w2, s2, None, False, f"M={M} H={H} I={I}")


def test_extreme_codes_and_longest_rows():
    """-128 everywhere over the longest rows: the largest sum, 2^14 (2^17 - 16), is exact."""
    K = (1 << 17) - 16
    a = np.full((3, K), -128, np.int8)
    w = np.full((20, K), -128, np.int8)
    a[1], w[5] = 127, 127
    one = np.ones(3, np.float32), np.ones(20, np.float32)
    say(f"dense_i8 K={K}")
    y = ops.w4a8_moe_dense_i8(dev(a), dev(one[0]), dev(w), dev(one[1]))
    assert np.array_equal(y.cpu().numpy(), dense_f32(a, one[0], w, one[1]))
    many = np.repeat(a, 40, 0)                               # and where rows are many
    y = ops.w4a8_moe_dense_i8(dev(many), dev(np.ones(120, np.float32)), dev(w), dev(one[1]))
    assert np.array_equal(y.cpu().numpy(), dense_f32(many, np.ones(120, np.float32), w, one[1]))


@pytest.mark.parametrize("M", [2, 40, 300])
def test_a_scale_that_is_not_finite_reaches_its_row_only(M):
    g = np.random.Generator(np.random.PCG64(M))
    K, N = 256, 200
    a, w, sa, sw = codes(g, M, K), codes(g, N, K), scales(g, M, K), scales(g, N, K)
    clean = ops.w4a8_moe_dense_i8(dev(a), dev(sa), dev(w), dev(sw)).cpu()
    sa[1] = np.nan
    got = ops.w4a8_moe_dense_i8(dev(a), dev(sa), dev(w), dev(sw)).cpu()
    rows = [m for m in range(M) if m != 1]
    assert torch.equal(got[rows], clean[rows]) and bool(torch.isnan(got[1]).all())


@pytest.mark.parametrize("M", [1, 17, 129, 300])
def test_memory_around_the_result_is_left(M):
    g = np.random.Generator(np.random.PCG64(M))
    K, N = 144, 131
    a, w, sa, sw = codes(g, M, K), codes(g, N, K), scales(g, M, K), scales(g, N, K)
    buf = torch.full(((M + 2) * N,), 5.0, device=DEV)
    y = buf[N:-N].view(M, N)
    say(f"dense_i8 guard M={M}")
    ops.w4a8_moe_dense_i8(dev(a), dev(sa), dev(w), dev(sw), y=y)
    assert np.array_equal(y.cpu().numpy(), dense_f32(a, sa, w, sw))
    assert bool((buf[:N] == 5).all()) and bool((buf[-N:] == 5).all())


@pytest.mark.parametrize("y", ["f32", "bf16"])
@pytest.mark.parametrize("M,H,I,pad", [(1, 16, 128, 0), (1, 6144, 2048, 0), (2, 272, 256, 16), (4, 1040, 1408, 0),
                                       (13, 2944, 1408, 0), (16, 512, 128, 0), (17, 512, 384, 0), (31, 80, 640, 16),
                                       (64, 1024, 512, 0), (77, 208, 128, 0), (130, 144, 384, 0), (300, 528, 1152, 32),
                                       (515, 1024, 256, 0)])
def test_gated_block(M, H, I, pad, y):
    g = np.random.Generator(np.random.PCG64(M * 7 + H + I))
    a, w13, w2 = codes(g, M, H), codes(g, 2 * I, H), codes(g, H, I)
    sa, s13, s2 = scales(g, M, H), scales(g, 2 * I, H), scales(g, H, I)
    add = torch.from_numpy(g.normal(size=(M, H)).astype(np.float32)).to(TYPES[y]).to(DEV)
    at = strided(a, H + pad)
    say(f"mlp_i8 M={M} H={H} I={I} {y}")
    args = at, dev(sa), dev(w13), dev(s13), dev(w2), dev(s2)
    got = ops.w4a8_moe_mlp_i8(*args, y_dtype=TYPES[y])
    check_mlp(f64(got), a, sa, w13, s13, w2, s2, None, y == "bf16", f"M={M} H={H} I={I}")
    more = ops.w4a8_moe_mlp_i8(*args, add=add, y_dtype=TYPES[y])
    check_mlp(f64(more), a, sa, w13, s13, w2, s2, f64(add), y == "bf16", "with an addend")
    again = ops.w4a8_moe_mlp_i8(*args, add=add, y=add, workspace=torch.empty(
        ops.w4a8_moe_mlp_i8_workspace_bytes(M, H, I), dtype=torch.uint8, device=DEV))
    assert again is add and torch.equal(again, more)


@pytest.mark.parametrize("M", [1, 20, 200])
def test_gated_block_of_rows_without_activation(M):
    """Rows of zero codes: act is zero, its scale 1, and y the addend or zero; a NaN scale stays in its row."""
    g = np.random.Generator(np.random.PCG64(M))
    H, I = 256, 128
    a, w13, w2 = codes(g, M, H), codes(g, 2 * I, H), codes(g, H, I)
    sa, s13, s2 = scales(g, M, H), scales(g, 2 * I, H), scales(g, H, I)
    a[0] = 0
    rest = dev(w13), dev(s13), dev(w2), dev(s2)
    y = ops.w4a8_moe_mlp_i8(dev(a), dev(sa), *rest)
    assert bool((y[0] == 0).all())
    check_mlp(f64(y), a, sa, w13, s13, w2, s2)
    sa[0] = np.nan
    a[0] = 1
    z = ops.w4a8_moe_mlp_i8(dev(a), dev(sa), *rest)
    assert torch.equal(z[1:], y[1:]) and not bool(torch.isfinite(z[0]).any())


def test_gated_block_of_large_and_tiny_values():
    """Gates far down silu's tail and far up, and rows whose act is below the fp32 normals of a reciprocal."""
    g = np.random.Generator(np.random.PCG64(9))
    M, H, I = 24, 64, 128
    a, w13, w2 = codes(g, M, H), codes(g, 2 * I, H), codes(g, H, I)
    s13, s2 = np.full(2 * I, 2.0 ** -10, np.float32), scales(g, H, I)
    sa = np.exp2(np.linspace(-60, 6, M)).astype(np.float32)
    say("mlp_i8 rows from 2^-60 to 2^6")
    y = ops.w4a8_moe_mlp_i8(dev(a), dev(sa), dev(w13), dev(s13), dev(w2), dev(s2))
    check_mlp(f64(y), a, sa, w13, s13, w2, s2)


def test_no_rows():
    e = torch.empty
    w, s = torch.ones(32, 64, dtype=torch.int8, device=DEV), torch.ones(32, device=DEV)
    none = e(0, 64, dtype=torch.int8, device=DEV), e(0, device=DEV)
    assert tuple(ops.w4a8_moe_dense_i8(*none, w, s).shape) == (0, 32)
    w13, w2 = torch.ones(256, 64, dtype=torch.int8, device=DEV), torch.ones(64, 128, dtype=torch.int8, device=DEV)
    y = ops.w4a8_moe_mlp_i8(*none, w13, torch.ones(256, device=DEV), w2, torch.ones(64, device=DEV))
    assert tuple(y.shape) == (0, 64)


@pytest.mark.parametrize("M", [1, 9, 130, 600])
def test_streams_and_graphs(M):
    """Two captured graphs of the same weights, replayed in turn with eager calls between, and a call on another stream."""
    g = np.random.Generator(np.random.PCG64(M))
    H, I = 512, 256
    w13, w2 = codes(g, 2 * I, H), codes(g, H, I)
    rest = dev(w13), dev(scales(g, 2 * I, H)), dev(w2), dev(scales(g, H, I))
    ins = [(dev(codes(g, M, H)), dev(scales(g, M, H))) for _ in range(2)]
    want = [ops.w4a8_moe_mlp_i8(*i, *rest) for i in ins]
    want_d = [ops.w4a8_moe_dense_i8(*i, *rest[:2], y_dtype=torch.bfloat16) for i in ins]
    outs = [torch.zeros_like(want[0]) for _ in range(2)]
    outs_d = [torch.zeros_like(want_d[0]) for _ in range(2)]
    torch.cuda.synchronize()
    graphs = []
    for (a, s), y, d in zip(ins, outs, outs_d):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            ops.w4a8_moe_mlp_i8(a, s, *rest, y=y)
            ops.w4a8_moe_dense_i8(a, s, *rest[:2], y=d)
        graphs.append(gr)
    for rep in range(4):
        say(f"replay {rep} M={M}")
        for gr, y, d in zip(graphs, outs, outs_d):
            y.zero_()
            d.zero_()
            gr.replay()
            assert torch.equal(ops.w4a8_moe_mlp_i8(*ins[0], *rest), want[0])
        torch.cuda.synchronize()
        for k in range(2):
            assert torch.equal(outs[k], want[k]) and torch.equal(outs_d[k], want_d[k])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = ops.w4a8_moe_mlp_i8(*ins[1], *rest)
    mine = ops.w4a8_moe_mlp_i8(*ins[0], *rest)               # at the same time, on this stream
    torch.cuda.synchronize()
    assert torch.equal(other, want[1]) and torch.equal(mine, want[0])


def _large(M, N, K, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    c = lambda *s: torch.randint(-128, 128, s, dtype=torch.int8, device=DEV, generator=gen)  # noqa: E731
    f = lambda n: torch.exp(torch.randn(n, device=DEV, generator=gen) * 0.3 - 5)  # noqa: E731
    return c(M, K), f(M), c(N, K), f(N)


@pytest.mark.parametrize("M,N,K", [(1, 131072, 6144), (128, 6144, 6144), (4096, 12288, 6144), (8192, 4096, 6144)])
def test_largest(M, N, K):
    """Every output of the largest calls, against fp64 products on the GPU (exact: integers below 2^53)."""
    a, sa, w, sw = _large(M, N, K, 5)
    say(f"dense_i8 M={M} N={N} K={K}")
    y = ops.w4a8_moe_dense_i8(a, sa, w, sw)
    y16 = ops.w4a8_moe_dense_i8(a, sa, w, sw, y_dtype=torch.bfloat16)
    step = 8192
    for n in range(0, N, step):
        want = (a.double() @ w[n:n + step].double().t()).float() * sa[:, None] * sw[n:n + step]
        assert torch.equal(y[:, n:n + step], want)
        assert torch.equal(y16[:, n:n + step], want.to(torch.bfloat16))


def test_operands_past_32_bits_of_offset():
    """Weights of more than 2^32 bytes, and rows of a further than 2^31 bytes from its first."""
    a, sa, w, sw = _large(2, 70000, 65536, 6)
    say("dense_i8 N=70000 K=65536 (4.6 GB of weights)")
    y = ops.w4a8_moe_dense_i8(a, sa, w, sw)
    at = torch.tensor([0, 1, 32767, 32768, 65535, 65536, 69999], device=DEV)
    assert torch.equal(y[:, at], (a.double() @ w[at].double().t()).float() * sa[:, None] * sw[at])
    del w
    ld = 1 << 22
    M, N, K = 700, 64, 128
    buf = torch.zeros(M, ld, dtype=torch.int8, device=DEV)
    b, sb, w, sw = _large(M, N, K, 7)
    buf[:, :K] = b
    say(f"dense_i8 rows {ld} bytes apart")
    y = ops.w4a8_moe_dense_i8(buf[:, :K], sb, w, sw)
    assert torch.equal(y, (b.double() @ w.double().t()).float() * sb[:, None] * sw)


def test_gated_block_of_more_rows_than_a_launch_has_in_x():
    M, H, I = (1 << 24) + 3, 16, 128
    a, sa, w13, s13 = _large(M, 2 * I, H, 11)
    w2, s2 = _large(H, H, I, 12)[:2]
    say(f"mlp_i8 M={M} H={H} I={I}")
    y = ops.w4a8_moe_mlp_i8(a, sa, w13, s13, w2, s2, y_dtype=torch.bfloat16)
    for rows in (slice(0, 40), slice((1 << 23) - 20, (1 << 23) + 20), slice((1 << 24) - 20, M)):
        assert torch.equal(y[rows], ops.w4a8_moe_mlp_i8(a[rows], sa[rows], w13, s13, w2, s2, y_dtype=torch.bfloat16))
