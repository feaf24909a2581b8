"""The whole layer for a few tokens (two kernels) against the definition in 64 bits.

Routing is bit-exact.  y is held to a bound per element that is derived from the
arithmetic (``reference``): fp32 sums of known length, and, for re-quantized
activations whose quotient lies within the error of act of a border between two
codes, one step of the code.
"""
import numpy as np
import pytest
import torch

import oracle
from gpu_util import bf16_to_dev, host, say, to_dev
from oracle import mxfp4_oracle as mx
from quantized_grouped_gemm_token_amd import ops, workloads
from quantized_grouped_gemm_token_amd.layer import W4A8MoE, W4A8MoEChannel, W4A8MoEMxfp4

pytestmark = pytest.mark.gpu

U = 2.0 ** -24                                   # half a step of fp32, relative
FORMS = ("g128", "channel", "mxfp4")
CALL = {"g128": ops.w4a8_moe_few_prepacked, "channel": ops.w4a8_moe_few_i8_prepacked,
        "mxfp4": ops.w4a8_moe_few_mxfp4_prepacked}

# T, H, I, E, k
SHAPES = [
    (1, 256, 128, 8, 2),             # one token
    (16, 256, 128, 8, 2),            # the benchmark's tiny layer
    (3, 384, 256, 4, 4),             # every token at every expert
    (5, 1152, 384, 60, 6),           # 9 and 3 groups: waves without work, a chunk that is not whole
    (16, 1024, 640, 12, 8),          # experts with many of the tokens
    (2, 2048, 768, 128, 8),          # many small experts
    (7, 896, 128, 1, 1),             # one expert
    (16, 512, 256, 300, 16),         # the most routed rows (256), more than 256 experts
    (1, 128, 128, 1024, 64),         # one group each, the most experts
    (10, 4352, 512, 24, 3),          # gate/up tasks of 32 columns, rows of up to 6144
    (9, 6400, 512, 24, 3),           # .. and of more
    (1, 128, 65536, 2, 1),           # the longest act rows
    (5, 256, 4224, 3, 2),            # .. and ones whose maxima take more than one pass
    (2, 256, 128, 300, 128),         # more picks than a wave has lanes
    (14, 8192, 128, 8, 2),           # the longest rows, the most codes in LDS
    (3, 8192, 128, 64, 8),           # the most column blocks, 17 to 24 pieces in each
    (2, 8192, 640, 16, 8),           # .. and a range of pieces that is nearly a block
    (16, 384, 2176, 5, 2),           # 12 column blocks shared by many workgroups
    (9, 2304, 1280, 20, 3),          # two rows of work per wave in the quantizer's second pass
]


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    assert ops.w4a8_moe_device_supported(), "the current device is not a gfx950"
    yield
    torch.cuda.synchronize()


def make(form, T, H, I, E, k, seed):
    """Host arrays of a workload: x bits, logits, stored weights and scales."""
    wl = workloads.make_custom(T, H, I, E, k, seed=seed)
    if form == "g128":
        w = (wl.w13, wl.s13, wl.w2, wl.s2)
    elif form == "channel":
        s13, s2 = workloads.channel_scales(wl)
        w = (wl.w13, s13, wl.w2, s2)
    else:
        w = workloads.mxfp4_weights(wl)
    return wl.x_bf16, wl.logits, w


def prepack(form, w):
    w13, s13, w2, s2 = (to_dev(a) for a in w)
    if form == "mxfp4":
        return (*ops.w4a8_moe_prepack_mxfp4(w13, s13), *ops.w4a8_moe_prepack_mxfp4(w2, s2))
    if form == "channel":
        return ops.w4a8_moe_prepack_int4(w13)[0], s13, ops.w4a8_moe_prepack_int4(w2)[0], s2
    return (*ops.w4a8_moe_prepack_int4(w13, s13), *ops.w4a8_moe_prepack_int4(w2, s2))


def dequant(form, w, s):
    """(W, B): the weights [N, K] in fp64, and what their products' sizes are summed over: the INT4 form adds
    u x and -8 x, u = q + 8 <= 15, so B = (u + 8) |s|."""
    if form == "mxfp4":
        W = mx.dequant_mxfp4(w[None], s[None])[0].astype(np.float64)
        return W, np.abs(W)
    q = oracle.int4_unpack(w).astype(np.float64)
    f = np.abs(np.repeat(s.astype(np.float64), 128, -1)) if form == "g128" else np.abs(s.astype(np.float64))[:, None]
    return q * f, (q + 16) * f


def code_step(v, int8):
    """The largest distance between neighbouring codes at |v|."""
    if int8:
        return np.ones_like(v)
    e = np.clip(np.floor(np.log2(np.maximum(np.abs(v), 1e-30))), -6, 8)
    return 2.0 ** (e - 3)


def border_distance(v, int8):
    a = np.abs(v)
    if int8:
        return np.abs(a - np.floor(a) - 0.5)
    pos = oracle.E4M3_VALUES[:0x7F].astype(np.float64)
    mids = (pos[:-1] + pos[1:]) / 2
    i = np.clip(np.searchsorted(mids, a), 1, len(mids) - 1)
    return np.minimum(np.abs(a - mids[i - 1]), np.abs(a - mids[i]))


def reference(form, x_bits, logits, weights, k, renormalize=True):
    """(ids, w, y, tol): the layer in 64 bits and how far an element of y may be off."""
    int8 = form == "channel"
    w13, s13, w2, s2 = weights
    T, H = x_bits.shape
    I, E = w2.shape[2] * (2 if form == "mxfp4" else 8), logits.shape[1]
    ids, w = oracle.route(logits, k, renormalize)
    if int8:
        q, sx = oracle.quant_act_i8(x_bits)
        a = q.astype(np.float64)
    else:
        q, sx = oracle.quant_act(x_bits)
        a = oracle.e4m3_decode(q).astype(np.float64)
    y, tol = np.zeros((T, H)), np.zeros((T, H))
    # a sum of G groups: at most G + 8 (waves) + 8 rounded additions and products in a row
    g13, g2 = (H // 128 + 16) * U, (I // 128 + longest_chain(T, k, E, I) + 16) * U
    for e in sorted(set(ids.reshape(-1).tolist())):
        t, j = np.nonzero(ids == e)
        W, B = dequant(form, w13[e], s13[e])
        h = a[t] @ W.T * sx[t].astype(np.float64)[:, None]
        dh = np.abs(h) * 4 * U if int8 else g13 * (np.abs(a[t]) @ B.T) * sx[t].astype(np.float64)[:, None]
        g, u, dg, du = h[:, :I], h[:, I:], dh[:, :I], dh[:, I:]
        silu = g / (1 + np.exp(-g))
        act = silu * u
        # |silu'| <= 1.1; the fast exponential and reciprocal cost 16 steps, and 2^-24 of the row in silu's far tail
        big = np.abs(act).max(1, keepdims=True)
        # (two steps of the subnormals: silu and the product; half a step of sa)
        dact = 1.1 * dg * np.abs(u) + np.abs(silu) * du + 1.1 * dg * du + 32 * U * np.abs(act) + U * big + 2.0 ** -148
        sa = np.where(big > 0, big / (127.0 if int8 else 448.0), 1.0)
        ds = dact.max(1, keepdims=True) / np.maximum(big, 1e-300) + 4 * U + 2.0 ** -150 / sa    # relative error of sa
        v = act / sa
        dv = dact / sa + np.abs(v) * (ds + 4 * U)
        qa = np.clip(np.rint(v), -127, 127) if int8 else \
            oracle.e4m3_decode(oracle.e4m3_encode(v.astype(np.float32))).astype(np.float64)
        flip = np.where(border_distance(v, int8) <= dv, code_step(v, int8), 0.0)
        W, B = dequant(form, w2[e], s2[e])
        o = qa @ W.T * sa
        do = flip @ np.abs(W).T * sa + np.abs(o) * ds + (g2 * (np.abs(qa) @ (np.abs(W) if int8 else B).T)) * sa
        wt = w[t, j].astype(np.float64)[:, None]
        np.add.at(y, t, wt * o)
        np.add.at(tol, t, wt * (do * (1 + ds) + np.abs(o) * 8 * U) + 2.0 ** -150 * np.abs(o / sa))   # (w sa may be subnormal)
    return ids, w, y, tol + 2.0 ** -126


def longest_chain(T, k, E, I):
    """Additions in a row to a wave's tile of y: one per (expert, 4-group chunk) piece."""
    return min(T * k, E) * -(-I // 512) // 8 + 1


def check(form, x_bits, logits, weights, k, y, y_dtype, renormalize=True, what=""):
    ids, w, ref, tol = reference(form, x_bits, logits, weights, k, renormalize)
    got = y.double().cpu().numpy()
    if y_dtype == torch.bfloat16:
        tol = tol + 2.0 ** -8 * (np.abs(ref) + tol)
    off = np.abs(got - ref)
    assert np.isfinite(got).all(), what
    assert (off <= tol).all(), (f"{what}: {int((off > tol).sum())} elements off by up to "
                                f"{float((off / tol).max()):.2f} of their bound")
    return ids, w


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("T,H,I,E,k", SHAPES)
def test_few_against_64_bits(form, T, H, I, E, k):
    x_bits, logits, weights = make(form, T, H, I, E, k, seed=11 * T + E)
    say(f"few {form} T={T} H={H} I={I} E={E} k={k}")
    x, lg, packed = bf16_to_dev(x_bits), to_dev(logits), prepack(form, weights)
    ids = torch.full((T, k), -7, dtype=torch.int32, device="cuda:0")
    w = torch.full((T, k), -7.0, device="cuda:0")
    y = CALL[form](x, lg, k, *packed, ids=ids, w=w)
    check(form, x_bits, logits, weights, k, y, torch.float32, what="fp32")
    ids_r, w_r = ops.w4a8_moe_route(lg, k)
    assert torch.equal(ids, ids_r) and torch.equal(w.view(torch.int32), w_r.view(torch.int32))
    yb = CALL[form](x, lg, k, *packed, y_dtype=torch.bfloat16)
    assert torch.equal(yb, y.to(torch.bfloat16))                     # one rounding of the same sums
    # again, with a workspace full of ones (NaN as fp32): the same bits
    ws = torch.full((ops.w4a8_moe_few_workspace_bytes(T, k, I),), 255, dtype=torch.uint8, device="cuda:0")
    again = CALL[form](x, lg, k, *packed, workspace=ws)
    assert torch.equal(again, y)


@pytest.mark.parametrize("form", FORMS)
def test_few_without_renormalization(form):
    T, H, I, E, k = 4, 512, 256, 70, 5
    x_bits, logits, weights = make(form, T, H, I, E, k, seed=5)
    say(f"few {form} softmax over all experts")
    lg = to_dev(logits)
    ids, w = torch.empty((T, k), dtype=torch.int32, device="cuda:0"), torch.empty((T, k), device="cuda:0")
    y = CALL[form](bf16_to_dev(x_bits), lg, k, *prepack(form, weights), renormalize=False, ids=ids, w=w)
    check(form, x_bits, logits, weights, k, y, torch.float32, renormalize=False)
    ids_r, w_r = ops.w4a8_moe_route(lg, k, renormalize=False)
    assert torch.equal(ids, ids_r) and torch.equal(w.view(torch.int32), w_r.view(torch.int32))


def test_few_ties_masks_and_one_expert_for_all():
    """Equal logits go to the lower expert, masked ones (-inf, the lowest value) come last, and sixteen tokens
    that all pick the same experts are multiplied together."""
    form, T, H, I, E, k = "g128", 16, 256, 128, 130, 3
    x_bits, logits, weights = make(form, T, H, I, E, k, seed=8)
    logits[:] = -np.inf
    logits[:8, [129, 70, 5, 64]] = 1.5                        # four equal: 5, 64, 70
    logits[8:12, 40:] = np.finfo(np.float32).min             # finite lowest values, equal: 40, 41, 42
    logits[12:, 9] = 0.0                                     # one expert left: then the lowest masked ones, weight 0
    logits[15, 3] = -0.0                                     # -0 equals 0: 3 before 9
    say("few ties, masks, shared experts")
    lg = to_dev(logits)
    ids, w = torch.empty((T, k), dtype=torch.int32, device="cuda:0"), torch.empty((T, k), device="cuda:0")
    y = CALL[form](bf16_to_dev(x_bits), lg, k, *prepack(form, weights), ids=ids, w=w)
    ids, w = host(ids), host(w)
    assert (ids[:8] == [5, 64, 70]).all() and np.allclose(w[:8], 1 / 3, rtol=1e-6)
    assert (ids[8:12] == [40, 41, 42]).all() and np.allclose(w[8:12], 1 / 3, rtol=1e-6)
    assert (ids[12:15] == [9, 0, 1]).all() and (w[12:15] == [1, 0, 0]).all()
    assert (ids[15] == [3, 9, 0]).all() and (w[15] == [0.5, 0.5, 0]).all()
    # the same tokens with finite logits that rank alike
    finite = np.where(np.isfinite(logits), logits, -1e30).astype(np.float32)
    finite[8:12] = np.where(np.arange(E) >= 40, 0.0, -1e30)
    check(form, x_bits, finite, weights, k, y, torch.float32)


def test_few_ids_stay_in_range_for_nan_logits():
    T, H, I, E, k = 3, 256, 128, 9, 4
    x_bits, logits, weights = make("g128", T, H, I, E, k, seed=3)
    logits[0, 2], logits[1, :], logits[2, 4] = np.nan, np.nan, np.inf
    say("few with NaN logits")
    ids = torch.full((T, k), -7, dtype=torch.int32, device="cuda:0")
    ops.w4a8_moe_few_prepacked(bf16_to_dev(x_bits), to_dev(logits), k, *prepack("g128", weights), ids=ids)
    ids = host(ids)
    assert ((ids >= 0) & (ids < E)).all() and all(len(set(r)) == k for r in ids.tolist())


@pytest.mark.parametrize("form", FORMS)
def test_few_zero_rows_and_outliers(form):
    """An all-zero token (scale 1, codes 0), one with a single value, one of outliers."""
    T, H, I, E, k = 4, 384, 256, 6, 2
    x_bits, logits, weights = make(form, T, H, I, E, k, seed=21)
    x = oracle.bf16_bits_to_f32(x_bits).copy()
    x[0] = 0
    x[1] = 0
    x[1, 130] = 3.0
    x[2, ::7] *= 1000
    x_bits = oracle.f32_to_bf16_bits(x)
    say(f"few {form} zero rows, outliers")
    y = CALL[form](bf16_to_dev(x_bits), to_dev(logits), k, *prepack(form, weights))
    assert (host(y)[0] == 0).all()
    check(form, x_bits[1:], logits[1:], weights, k, y[1:], torch.float32)


def scale_weights(form, s, exponent):
    """The scales times 2^exponent (MXFP4: E8M0 exponents)."""
    if form == "mxfp4":
        shifted = s.astype(np.int32) + exponent
        assert shifted.min() >= 1 and shifted.max() <= 254
        return shifted.astype(np.uint8)
    return (s * np.float32(2.0 ** exponent)).astype(np.float32)


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("T,H", [(3, 384), (11, 384), (9, 2304)])
def test_few_rows_of_tiny_values(form, T, H):
    """Rows whose largest value over the largest code is subnormal: its reciprocal is infinite.  Tokens first (with
    w13 scaled up), then act (with w13 scaled down and w2 up)."""
    I, E, k = 256, 6, 2
    x_bits, logits, weights = make(form, T, H, I, E, k, seed=22)
    w13, s13, w2, s2 = weights
    say(f"few {form} T={T} H={H} tiny rows of x")
    tiny = oracle.f32_to_bf16_bits(oracle.bf16_bits_to_f32(x_bits) * np.float32(2.0 ** -125))
    up = (w13, scale_weights(form, s13, 100), w2, s2)
    y = CALL[form](bf16_to_dev(tiny), to_dev(logits), k, *prepack(form, up))
    check(form, tiny, logits, up, k, y, torch.float32, what="tiny x")
    for shift, bounded in ((-64, True), (-66, True), (-70, False), (-73, False), (-76, False)):
        say(f"few {form} T={T} H={H} w13 times 2^{shift}")
        low = (w13, scale_weights(form, s13, shift), w2, scale_weights(form, s2, 100))
        y = CALL[form](bf16_to_dev(x_bits), to_dev(logits), k, *prepack(form, low))
        assert torch.isfinite(y).all()
        if bounded:                                          # (further down sa itself has few bits left)
            check(form, x_bits, logits, low, k, y, torch.float32, what=f"tiny act {shift}")


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("T,H", [(4, 512), (16, 512), (12, 2304)])
def test_few_a_token_that_is_not_finite_keeps_to_itself(form, T, H):
    """NaN or infinities in one token's row: the other tokens' results are the same bits."""
    I, E, k = 640, 6, 3
    x_bits, logits, weights = make(form, T, H, I, E, k, seed=23)
    say(f"few {form} T={T} H={H} with a NaN and an infinity in x")
    x, lg, packed = bf16_to_dev(x_bits), to_dev(logits), prepack(form, weights)
    want = CALL[form](x, lg, k, *packed)
    assert torch.isfinite(want).all()
    bad = x.clone()
    bad[1, 7], bad[T - 1, :] = float("nan"), float("-inf")
    got = CALL[form](bad, lg, k, *packed)
    rest = [t for t in range(T) if t not in (1, T - 1)]
    assert torch.equal(got[rest], want[rest])
    if form != "channel":                                    # (an INT8 code has no value for them)
        assert not torch.isfinite(got[[1, T - 1]]).any()


def test_few_strided_rows_and_neighbours_untouched():
    form, T, H, I, E, k = "g128", 6, 512, 256, 10, 3
    x_bits, logits, weights = make(form, T, H, I, E, k, seed=31)
    packed, lg = prepack(form, weights), to_dev(logits)
    x = bf16_to_dev(x_bits)
    wide = torch.full((T, H + 24), float("nan"), dtype=torch.bfloat16, device="cuda:0")
    wide[:, :H] = x
    say("few with strided rows, y inside a larger buffer")
    want = CALL[form](x, lg, k, *packed)
    assert torch.equal(CALL[form](wide[:, :H], lg, k, *packed), want)
    buf = torch.full((T + 4, H), 77.0, device="cuda:0")
    CALL[form](x, lg, k, *packed, y=buf[2:2 + T])
    assert torch.equal(buf[2:2 + T], want) and (buf[:2] == 77).all() and (buf[2 + T:] == 77).all()
    # one token's result does not depend on the others
    for t in (0, T - 1):
        one = CALL[form](x[t:t + 1], lg[t:t + 1], k, *packed)
        ref = want[t:t + 1]
        assert float((one - ref).norm() / ref.norm()) <= 2e-3
    assert CALL[form](x[:0], lg[:0], k, *packed).shape == (0, H)


def test_few_far_experts():
    """Experts whose weights start past 2^32 bytes give what they give in a small array."""
    H, I, E, k = 4096, 2048, 600, 2
    gen = torch.Generator(device="cuda:0").manual_seed(1)
    w13 = torch.randint(-2**31, 2**31, (E, 2 * I // 16, H // 128, 16, 16), generator=gen, device="cuda:0",
                        dtype=torch.int32)
    w2 = torch.randint(-2**31, 2**31, (E, H // 16, I // 128, 16, 16), generator=gen, device="cuda:0",
                       dtype=torch.int32)
    assert w13[-2:].data_ptr() - w13.data_ptr() > 2**32
    s13 = torch.exp(torch.randn(E, H // 128, 2 * I, generator=gen, device="cuda:0") * 0.5 - 4)
    s2 = torch.exp(torch.randn(E, I // 128, H, generator=gen, device="cuda:0") * 0.5 - 4)
    x = torch.randn(2, H, generator=gen, device="cuda:0").to(torch.bfloat16)
    lg = torch.full((2, E), -1e30, device="cuda:0")
    near = torch.tensor([[0.3, 1.0], [2.0, -1.0]], device="cuda:0")
    lg[:, -2:] = near
    say("few with experts past 4 GiB")
    got = ops.w4a8_moe_few_prepacked(x, lg, k, w13, s13, w2, s2)
    want = ops.w4a8_moe_few_prepacked(x, near, k, *(a[-2:].contiguous() for a in (w13, s13, w2, s2)))
    assert torch.equal(got, want) and float(want.abs().max()) > 0


@pytest.mark.parametrize("form", FORMS)
def test_few_graph_replays_follow_the_inputs(form):
    T, H, I, E, k = 5, 512, 256, 24, 4
    x_bits, logits, weights = make(form, T, H, I, E, k, seed=41)
    packed = prepack(form, weights)
    x, lg = bf16_to_dev(x_bits), to_dev(logits)
    sets = [(x, lg), (x * 3, lg.roll(1, 0)), (x.flip(0), -lg)]
    want = [CALL[form](a, b, k, *packed) for a, b in sets]
    xs, ls, y = x.clone(), lg.clone(), torch.empty_like(want[0])
    say(f"few {form} captured twice")
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):                                       # two graphs, their workspaces apart
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            CALL[form](xs, ls, k, *packed, y=y)
        graphs.append(g)
    for i in range(6):
        a, b = sets[i % 3]
        xs.copy_(a)
        ls.copy_(b)
        y.zero_()
        graphs[i % 2].replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want[i % 3]), f"replay {i}"
        other = CALL[form](*sets[(i + 1) % 3], k, *packed)   # eager work between replays
        torch.cuda.synchronize()
        assert torch.equal(other, want[(i + 1) % 3])


def test_few_two_graphs_replayed_in_turn_and_at_once():
    """Two captured layers with matrix-vector products behind them, each with workspaces of its own."""
    T, H, I, E, k = 6, 512, 384, 24, 3
    x_bits, logits, weights = make("mxfp4", T, H, I, E, k, seed=71)
    packed = prepack("mxfp4", weights)
    x, lg = [bf16_to_dev(x_bits) * f for f in (1, 3)], [to_dev(logits), -to_dev(logits)]
    w = torch.randint(0, 256, (300, H // 2), dtype=torch.uint8, device="cuda:0")
    s = torch.randint(118, 124, (300, H // 32), dtype=torch.uint8, device="cuda:0")

    def step(i):
        h = ops.w4a8_moe_few_mxfp4_prepacked(x[i], lg[i], k, *packed, y_dtype=torch.bfloat16)
        return h, ops.w4a8_moe_matvec_mxfp4(h, w, s)

    say("few: two graphs")
    want = [step(i) for i in range(2)]
    torch.cuda.synchronize()
    graphs, got = [], []
    for i in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got.append(step(i))
        graphs.append(g)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for at_once in (False, True, False, True):
        for h, y in got:
            h.zero_()
            y.zero_()
        torch.cuda.synchronize()
        for _ in range(5):
            for i in range(2):
                with torch.cuda.stream(streams[i if at_once else 0]):
                    graphs[i].replay()
        torch.cuda.synchronize()
        for i in range(2):
            assert all(torch.equal(a, b) for a, b in zip(got[i], want[i]))
        assert all(torch.equal(a, b) for i in range(2) for a, b in zip(step(i), want[i]))   # eager work between


def test_few_on_two_streams_at_once():
    T, H, I, E, k = 3, 1024, 512, 32, 4
    x_bits, logits, weights = make("g128", T, H, I, E, k, seed=51)
    packed, x, lg = prepack("g128", weights), bf16_to_dev(x_bits), to_dev(logits)
    want = [ops.w4a8_moe_few_prepacked(x, lg, k, *packed), ops.w4a8_moe_few_prepacked(x * 2, -lg, k, *packed)]
    x2, lg2 = x * 2, -lg
    torch.cuda.synchronize()
    say("few on two streams")
    s = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    for _ in range(20):
        for i, (a, b) in enumerate(((x, lg), (x2, lg2))):
            with torch.cuda.stream(s[i]):
                got[i].append(ops.w4a8_moe_few_prepacked(a, b, k, *packed))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(y, want[i]) for y in got[i])


@pytest.mark.parametrize("form", FORMS)
def test_layer_takes_the_few_path(form):
    """few=True: up to 16 tokens give the call's result, more the steps' (as without the option)."""
    H, I, E, k = 512, 256, 16, 4
    x_bits, logits, weights = make(form, 40, H, I, E, k, seed=61)
    cls = {"g128": W4A8MoE, "channel": W4A8MoEChannel, "mxfp4": W4A8MoEMxfp4}[form]
    dev = [to_dev(a) for a in weights]
    few, steps = cls(*dev, k=k, few=True), cls(*dev, k=k)
    x, lg = bf16_to_dev(x_bits), to_dev(logits)
    say(f"layer {form} few=True")
    packed = prepack(form, weights)
    for T in (1, 7, 16):
        y = few(x[:T], lg[:T])
        assert few.uses_few(T) and not steps.uses_few(T)
        assert torch.equal(y, CALL[form](x[:T], lg[:T], k, *packed))
        ref = steps(x[:T], lg[:T])
        assert float((y - ref).norm() / ref.norm()) <= 2e-3
        yb = few(x[:T], lg[:T], y_dtype=torch.bfloat16)
        assert torch.equal(yb, y.to(torch.bfloat16))
    assert not few.uses_few(17) and not few.uses_few(0)
    assert torch.equal(few(x, lg), steps(x, lg))
    y = torch.empty((3, H), device="cuda:0")
    g = few.capture(x[:3], lg[:3], y)
    for _ in range(3):
        y.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, few(x[:3], lg[:3]))


def test_few_refusals():
    T, H, I, E, k = 2, 256, 128, 4, 2
    x_bits, logits, weights = make("g128", T, H, I, E, k, seed=71)
    packed, x, lg = prepack("g128", weights), bf16_to_dev(x_bits), to_dev(logits)
    call = ops.w4a8_moe_few_prepacked
    say("few refusals")
    with pytest.raises(TypeError):
        call(x.float(), lg, k, *packed)
    with pytest.raises(ValueError):
        call(x, lg[:1], k, *packed)
    with pytest.raises(ValueError):
        call(x, lg[:, :3].contiguous(), k, *packed)          # another number of experts than the weights
    with pytest.raises(ValueError):
        call(x.t(), lg, k, *packed)
    with pytest.raises(ops.W4A8Error):
        call(x, lg, 5, *packed)                              # k > E
    with pytest.raises(ops.W4A8Error):
        call(x.repeat(9, 1), lg.repeat(9, 1), k, *packed)    # 18 tokens
    with pytest.raises(ops.W4A8Error):
        call(x, lg, k, *packed, workspace=torch.empty(64, dtype=torch.uint8, device="cuda:0"))
    odd = torch.zeros(T, H + 1, dtype=torch.bfloat16, device="cuda:0")
    with pytest.raises(ops.W4A8Error):
        call(odd[:, :H], lg, k, *packed)                     # rows not a multiple of 8 elements apart
    with pytest.raises(ops.W4A8Error):
        call(torch.zeros(T * H + 1, dtype=torch.bfloat16, device="cuda:0")[1:].view(T, H), lg, k, *packed)
    with pytest.raises(ValueError):
        call(x, lg, k, packed[0], packed[1][:, :, :-16].contiguous(), *packed[2:])
    with pytest.raises(ValueError):
        call(x, lg, k, *packed, y=torch.empty(T, H + 128, device="cuda:0"))
    with pytest.raises(TypeError):
        call(x, lg, k, *packed, y_dtype=torch.float16)
