"""The norms, the routed experts, the shared expert and the residual as they run together in a decoder block."""
import numpy as np
import pytest
import torch

from block_ref import check_mlp, rms
from gpu_util import DEV, host, say, to_dev
from quantized_grouped_gemm_token_amd import ops
from quantized_grouped_gemm_token_amd.layer import MoEBlock, W4A8MoE, W4A8MoEChannel, W4A8MoEMxfp4, W8A8Mlp
from test_gpu_few import FORMS, make

pytestmark = pytest.mark.gpu

LAYER = {"g128": W4A8MoE, "channel": W4A8MoEChannel, "mxfp4": W4A8MoEMxfp4}
H, I, E, K = 512, 256, 16, 4


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    assert ops.w4a8_moe_device_supported(), "the current device is not a gfx950"
    yield
    torch.cuda.synchronize()


def vec(g, n, mean=0.0, sd=1.0):
    return to_dev((mean + sd * g.normal(size=n)).astype(np.float32))


def shared_expert(g, inner=384):
    w13 = torch.from_numpy(g.normal(size=(2 * inner, H)).astype(np.float32)).to(torch.bfloat16).to(DEV)
    w2 = torch.from_numpy(g.normal(size=(H, inner)).astype(np.float32)).to(torch.bfloat16).to(DEV)
    q13, s13, _ = ops.w4a8_moe_quant_act_i8(w13)
    q2, s2, _ = ops.w4a8_moe_quant_act_i8(w2)
    return W8A8Mlp(q13, s13 * 0.05, q2, s2 * 0.05)


def block(form, seed, shared=True, few=False, post=True, gates=True, r_scale=0.75):
    g = np.random.Generator(np.random.PCG64(seed))
    weights = make(form, 2, H, I, E, K, seed)[2]
    moe = LAYER[form](*(to_dev(a) for a in weights), k=K, few=few)
    return MoEBlock(moe, vec(g, H, 1, 0.2), shared_expert(g) if shared else None, vec(g, H, 1, 0.2) if post else None,
                    vec(g, H) if gates else None, r_scale, 1e-5)


def router(seed):
    g = np.random.Generator(np.random.PCG64(seed + 7))
    w = torch.from_numpy(g.normal(size=(E, H)).astype(np.float32) * 0.1).to(DEV)
    return lambda xn: (xn.float()[:, None, :] * w).sum(-1)       # (no library product: any row alone gives its bits)


def stream_of(seed, T, dtype):
    g = np.random.Generator(np.random.PCG64(seed + 13))
    return torch.from_numpy(g.normal(size=(T, H)).astype(np.float32) * 3).to(dtype).to(DEV)


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("T", [1, 5, 16, 17, 130])
def test_codes_in_place_of_x(form, T):
    """Codes that are x's own give the forward's bits, by every path, and others are the ones that are multiplied."""
    b = block(form, 3)
    say(f"layer {form} T={T} from codes")
    x = stream_of(4, T, torch.bfloat16)
    lg = router(3)(x)
    codes = ops.w4a8_moe_quant_act_i8(x) if form == "channel" else ops.w4a8_moe_quant_act(x)
    for kw in (dict(), dict(front=False), dict(fused=False), dict(scatter=True), dict(few=True)):
        moe = b.moe
        for name, value in kw.items():
            setattr(moe, name, value)
        if "fused" in kw:
            moe._bufs.clear()
        steps_only = moe(x, lg, algo=ops.W4A8_GG_STREAM)
        assert torch.equal(moe(x, lg, algo=ops.W4A8_GG_STREAM, codes=codes), steps_only), kw
        other = torch.zeros_like(x)
        assert torch.equal(moe(other, lg, algo=ops.W4A8_GG_STREAM, codes=codes), steps_only), kw
    assert moe.uses_few(T) == (T <= 16)
    assert torch.equal(moe(other, lg, codes=codes), moe(other, lg, codes=codes, algo=ops.W4A8_GG_AUTO))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("T", [1, 7, 33, 300])
@pytest.mark.parametrize("shared,few,post", [(True, False, True), (False, True, False), (True, True, False),
                                             (False, False, True)])
def test_block_is_its_operators(dtype, form, T, shared, few, post):
    """Two blocks one behind the other, the second's norm made by the first's last pass."""
    say(f"block {form} T={T} {dtype} shared={shared} few={few} post={post}")
    first, second = (block(form, seed, shared, few, post) for seed in (21, 22))
    route, r = router(21), stream_of(23, T, dtype)
    token_gate = vec(np.random.Generator(np.random.PCG64(24)), T)
    before = r.clone()
    out, normed = first(r, route, token_gate, following=second)
    last = second(out, route, normed=normed)
    assert torch.equal(r, before) and last.dtype is dtype

    def by_hand(b, r, token_gate, normed):
        xn, q, s, rs = normed
        took = b.int8 == b.channel and not (few and T <= 16)
        y = b.moe(xn, route(xn), codes=((q, s, rs) if b.channel else (q, s)) if took else None)
        if shared:
            y = ops.w4a8_moe_mlp_i8(q, s, b.shared.w13, b.shared.s13, b.shared.w2, b.shared.s2, add=y)
        return ops.w4a8_moe_residual_norm(y, r, post_weight=b.post_weight, gate=b.gate, token_gate=token_gate,
                                          r_scale=b.r_scale, eps=b.eps)
    mid = by_hand(first, r, token_gate, first.before(r))
    assert torch.equal(out, mid)
    assert torch.equal(last, by_hand(second, mid, None, normed))
    if dtype is torch.float32:                            # (bf16: the norm takes the stream before its rounding)
        alone = second.before(mid)
        assert torch.equal(normed[0], alone[0]) and torch.equal(normed[1], alone[1]) and torch.equal(normed[2], alone[2])
    inplace = r.clone()
    assert first(inplace, route, token_gate, out=inplace) is inplace and torch.equal(inplace, mid)


def test_shared_expert_against_the_definition():
    b = block("channel", 31)
    r = stream_of(32, 40, torch.float32)
    xn, q, s, rs = b.before(r)
    y = b.shared(q, s)
    sh = b.shared
    check_mlp(y.double().cpu().numpy(), host(q), host(s), host(sh.w13), host(sh.s13), host(sh.w2), host(sh.s2))
    n = rms(r.double().cpu().numpy(), host(b.weight), b.eps)
    err = np.abs(host(q) * host(s).astype(np.float64)[:, None] - n)
    assert np.all(err <= 0.502 * host(s).astype(np.float64)[:, None])   # half a code, and the fp32 norm's own error
    assert np.array_equal(host(rs), host(q).astype(np.int64).sum(1))


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("T,few", [(3, True), (3, False), (150, False)])
def test_block_captured(form, T, few):
    """Two blocks in one graph, replayed on new contents with eager calls of the same blocks between."""
    first, second = (block(form, seed, True, few) for seed in (41, 42))
    route = router(41)
    r = stream_of(43, T, torch.float32)
    out = torch.empty_like(r)

    def run(r, out=None):
        mid, normed = first(r, route, following=second)
        return second(mid, route, normed=normed, out=out)
    run(r, out)
    torch.cuda.synchronize()
    say(f"block {form} T={T} few={few} captured")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(r, out)
    torch.cuda.synchronize()
    for i in range(4):
        x = stream_of(50 + i, T, torch.float32)
        want = run(x)
        r.copy_(x)
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want), i
        run(stream_of(60 + i, T, torch.float32))


def test_rows_do_not_meet():
    """A row of NaN, an infinite one and zeros leave the other rows' bits as they are."""
    b = block("channel", 71)
    route, r = router(71), stream_of(72, 24, torch.float32)
    clean = b(r, route)
    bad = r.clone()
    bad[3], bad[9, 5], bad[17] = float("nan"), float("inf"), 0
    xn = b.before(bad)[0]
    lg = route(xn).nan_to_num(0.0)                        # a router's logits are finite
    got = b(bad, lambda _: lg)
    rows = [i for i in range(24) if i not in (3, 9, 17)]
    assert torch.equal(got[rows], clean[rows]) and bool(torch.isfinite(got[17]).all())
    assert bool(torch.isnan(got[3]).all())


@pytest.mark.parametrize("form", FORMS)
def test_no_rows_and_strided_rows(form):
    """No token at all (whatever the strides of such a tensor are), and a stream and a result whose rows are apart."""
    b, route = block(form, 91), router(91)
    for none in (torch.empty(0, H, device=DEV), torch.from_numpy(np.zeros((5, H), np.float32)[:0]).to(DEV),
                 torch.empty(H, 0, device=DEV).t()):
        out, normed = b(none, route, following=b)
        assert tuple(out.shape) == (0, H) and tuple(normed[1].shape) == (0, H)
    r = stream_of(92, 20, torch.float32)
    want = b(r, route)
    wide = torch.full((20, H + 64), 7.0, device=DEV)
    wide[:, :H] = r
    assert torch.equal(b(wide[:, :H], route), want)
    buf = torch.zeros(20, H + 64, device=DEV)
    b(r, route, out=buf[:, :H])
    assert torch.equal(buf[:, :H], want) and bool((buf[:, H:] == 0).all())


def test_refusals():
    b = block("channel", 81)
    r = stream_of(82, 6, torch.float32)
    x = r.bfloat16()
    lg = router(81)(x)
    q, s, rs = ops.w4a8_moe_quant_act_i8(x)
    for codes, error in (((q[:5], s, rs), ValueError), ((q, s[:5], rs), ValueError), ((q, s, rs[:5]), ValueError),
                         ((q, s), TypeError), ((q.view(torch.uint8), s, rs), TypeError), ((q, s, s), TypeError),
                         ((q.cpu(), s, rs), ValueError)):
        with pytest.raises(error):
            b.moe(x, lg, codes=codes)
    with pytest.raises(TypeError):
        block("g128", 81).moe(x, lg, codes=(q, s))
    with pytest.raises(ValueError):
        W8A8Mlp(b.shared.w13, b.shared.s13, b.shared.w2[:, :-128], b.shared.s2)
    other = block("channel", 83)
    other.eps = 1e-3
    with pytest.raises(ValueError):
        b(r, router(81), following=other)
    with pytest.raises(TypeError):
        b(r, router(81), out=x)
