"""Operators of a decoder block around the routed experts, with 8-bit weights and activations, measured on one GPU.

* ``dense``: int8 activation codes (a scale per token) times an int8 weight matrix (a scale per output channel), with
  a bias and an addend: projections, dense layers, an output head.
* ``mlp``: the gated feed-forward block on such weights (a shared expert, a dense layer's block): gate/up products,
  SwiGLU, per-row requantization to int8, down product, an addend (the routed experts' sum).
* ``norm``: RMS norm before a block: the normalized rows in bf16 and their 8-bit codes with a scale per row.
* ``residual``: after a block: RMS norm of its result, gates per channel and per token, the scaled residual; and, for
  the next block, the norm and the codes of that sum.

``run`` computes each in its plain form (elementary torch operations), or with ``own`` set through the package's entry
points.  ``exact`` computes the definition in 64 bits.
"""
from __future__ import annotations

import math

import torch

own = False

DEV = "cuda"
EPS = 1e-6


# ------------------------------------------------------------------ cases
def _dense(name, M, N, K, y="bf16", bias=False, add=False, pad=0):
    return dict(name=name, op="dense", M=M, N=N, K=K, y=y, bias=bias, add=add, pad=pad)


def _mlp(name, M, H, I, add=False, pad=0):
    return dict(name=name, op="mlp", M=M, H=H, I=I, y="bf16", add=add, pad=pad)


def _norm(name, T, H, x="bf16", form="fp8", pad=0):
    return dict(name=name, op="norm", T=T, H=H, x=x, form=form, pad=pad)


def _residual(name, T, H, y, r, post, gate, token_gate, form, pad=0):
    return dict(name=name, op="residual", T=T, H=H, y=y, r=r, post=post, gate=gate, token_gate=token_gate, form=form,
                pad=pad)


def listed():
    return [
        # one decoding sequence through an attention output projection: latency and one read of the weights
        _dense("dense one token", 1, 6144, 6144),
        # an 8-bit output head over a vocabulary, one token, fp32 logits: the most bytes
        _dense("dense head", 1, 131072, 6144, y="f32"),
        # the benchmark's decode batch through a projection with a bias
        _dense("dense decode batch", 128, 6144, 6144, bias=True),
        # odd rows and outputs, a row length that is no multiple of 64, strided rows, bias and addend, fp32
        _dense("dense odd", 77, 5001, 2896, y="f32", bias=True, add=True, pad=32),
        # a long prompt through a wide projection: the most products
        _dense("dense prefill", 8192, 12288, 6144),
        # the shared expert of the benchmark's layer for one token, added to the routed experts' sum
        _mlp("mlp one token", 1, 6144, 2048, add=True),
        # a ragged small batch, odd group counts
        _mlp("mlp thirteen tokens", 13, 2944, 1408),
        # the shared expert over the benchmark's prefill, added to the routed experts' sum
        _mlp("mlp prefill", 8192, 6144, 2048, add=True),
        # the smallest call: one token's norm
        _norm("norm one token", 1, 6144),
        # the norm before the benchmark's longest prefill
        _norm("norm prefill", 16384, 6144),
        # between two blocks of a decode batch: fp32 residual stream, norms on both sides, channel and token gates
        _residual("residual decode batch", 128, 6144, "f32", "f32", True, True, True, "fp8"),
        # after a block of an odd prompt, bf16 all through, strided rows, no norm of the next block
        _residual("residual odd", 1001, 2920, "bf16", "bf16", True, False, True, "none", pad=24),
    ]


def _log(rng, lo, hi):
    return math.exp(rng.uniform(math.log(lo), math.log(hi)))


def draw(rng):
    op = rng.choice(["dense", "dense", "mlp", "norm", "residual"])
    pad = rng.choice([0, 0, 16, 64])
    y = rng.choice(["bf16", "bf16", "f32"])
    if op == "dense":
        M, N, K = int(_log(rng, 1, 8192)), int(_log(rng, 64, 16384)), 16 * int(_log(rng, 8, 512))
        while M * N * K > 8192 * 12288 * 6144:
            M //= 2
        return dict(op=op, M=M, N=N, K=K, y=y, bias=rng.random() < 0.5, add=rng.random() < 0.3, pad=pad)
    if op == "mlp":
        return dict(op=op, M=int(_log(rng, 1, 8192)), H=16 * int(_log(rng, 16, 384)), I=128 * int(_log(rng, 1, 32)),
                    y="bf16", add=rng.random() < 0.5, pad=pad)
    T, H = int(_log(rng, 1, 16384)), 8 * int(_log(rng, 8, 2048))
    while T * H > 16384 * 6144:
        T //= 2
    if op == "norm":
        return dict(op=op, T=T, H=H, x=y, form=rng.choice(["fp8", "i8"]), pad=pad)
    return dict(op=op, T=T, H=H, y=y, r=rng.choice(["bf16", "f32"]), post=rng.random() < 0.7, gate=rng.random() < 0.5,
                token_gate=rng.random() < 0.3, form=rng.choice(["none", "fp8", "i8"]), pad=pad)


# ----------------------------------------------------------------- inputs
def _rows(gen, T, H, dtype, pad, outliers=True):
    """Activations with 1% outlier channels, in rows of H + pad."""
    x = torch.randn(T, H, generator=gen, device=DEV)
    if outliers:
        x = torch.where(torch.rand(H, generator=gen, device=DEV) < 0.01, x * 20, x)
    buf = torch.zeros(T, H + pad, dtype=torch.bfloat16 if dtype == "bf16" else torch.float32, device=DEV)
    buf[:, :H] = x
    return buf[:, :H]


def _codes(gen, T, K, pad):
    """int8 codes and scales of activations, in rows of K + pad."""
    x = _rows(gen, T, K, "f32", 0)
    s = x.abs().amax(1) / 127
    buf = torch.zeros(T, K + pad, dtype=torch.int8, device=DEV)
    buf[:, :K] = torch.round(x / s[:, None]).clamp(-127, 127)
    return buf[:, :K], s


def _weights(gen, N, K):
    """int8 weights with normal codes (a quarter of the range their deviation), scales that keep products near one."""
    w = torch.empty(N, K, dtype=torch.int8, device=DEV)
    for n in range(0, N, 16384):
        w[n:n + 16384] = torch.randn(min(16384, N - n), K, generator=gen, device=DEV).mul_(32).round_().clamp_(-127, 127)
    return w, torch.exp(torch.randn(N, generator=gen, device=DEV) * 0.3 - math.log(32 * math.sqrt(K)))


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    s = dict(case)
    normal = lambda *shape: torch.randn(*shape, generator=gen, device=DEV)  # noqa: E731
    if case["op"] == "dense":
        s["a"], s["a_scale"] = _codes(gen, case["M"], case["K"], case["pad"])
        s["w"], s["w_scale"] = _weights(gen, case["N"], case["K"])
        s["bias"] = normal(case["N"]) if case["bias"] else None
        s["add"] = _rows(gen, case["M"], case["N"], case["y"], 0, False) if case["add"] else None
    elif case["op"] == "mlp":
        s["a"], s["a_scale"] = _codes(gen, case["M"], case["H"], case["pad"])
        s["w13"], s["s13"] = _weights(gen, 2 * case["I"], case["H"])
        s["w2"], s["s2"] = _weights(gen, case["H"], case["I"])
        s["add"] = _rows(gen, case["M"], case["H"], case["y"], 0, False) if case["add"] else None
    elif case["op"] == "norm":
        s["x"] = _rows(gen, case["T"], case["H"], case["x"], case["pad"])
        s["weight"] = 1 + 0.2 * normal(case["H"])
    else:
        s["y"] = _rows(gen, case["T"], case["H"], case["y"], case["pad"], False)
        s["r"] = _rows(gen, case["T"], case["H"], case["r"], case["pad"])
        s["post"] = 1 + 0.2 * normal(case["H"]) if case["post"] else None
        s["gate"] = 0.5 * normal(case["H"]) if case["gate"] else None
        s["token_gate"] = torch.sigmoid(normal(case["T"])) if case["token_gate"] else None
        s["r_scale"] = 0.75
        s["weight"] = 1 + 0.2 * normal(case["H"]) if case["form"] != "none" else None
    return s


# ------------------------------------------------------------- plain form
def _type(name):
    return torch.bfloat16 if name == "bf16" else torch.float32


def _product(a, w):
    """The integer sums of a x w^T: exact in 64 bits, where 32 lose them from K = 1040 on."""
    return torch.matmul(a.double(), w.double().t()).float()


def _plain_dense(a, a_scale, w, w_scale, bias, add, dtype):
    y = _product(a, w) * a_scale[:, None] * w_scale
    if bias is not None:
        y = y + bias
    if add is not None:
        y = y + add.float()
    return y.to(dtype)


def _plain_mlp(s):
    # y is bf16 in every case: act next to a border between two codes falls on either side of it by fp32's rounding
    h = _plain_dense(s["a"], s["a_scale"], s["w13"], s["s13"], None, None, torch.float32)
    gate, up = h[:, :s["I"]], h[:, s["I"]:]
    act = gate / (1 + torch.exp(-gate)) * up
    amax = act.abs().amax(1)
    sa = torch.where(amax > 0, amax / 127, torch.ones_like(amax))
    qa = torch.round(act / sa[:, None]).clamp(-127, 127)
    return _plain_dense(qa, sa, s["w2"], s["s2"], None, s["add"], _type(s["y"]))


def _plain_norm(x, weight):
    return x * torch.rsqrt((x * x).sum(1, keepdim=True) / x.shape[1] + EPS) * weight


def _plain_codes(n, form):
    amax = n.abs().amax(1)
    scale = torch.where(amax > 0, amax / (448 if form == "fp8" else 127), torch.ones_like(amax))
    q = n / scale[:, None]
    codes = q.to(torch.float8_e4m3fn) if form == "fp8" else torch.round(q).clamp(-127, 127).to(torch.bfloat16)
    return {"xn": n.to(torch.bfloat16), "codes": codes, "scale": scale}


def _plain_residual(s):
    p = s["y"].float()
    if s["post"] is not None:
        p = _plain_norm(p, s["post"])
    if s["gate"] is not None:
        p = p * s["gate"]
    if s["token_gate"] is not None:
        p = p * s["token_gate"][:, None]
    out = s["r"].float() * s["r_scale"] + p
    got = {"out": out.to(s["r"].dtype)}
    if s["form"] != "none":
        got.update(_plain_codes(_plain_norm(out, s["weight"]), s["form"]))
    return got


def _plain(s):
    if s["op"] == "dense":
        return _plain_dense(s["a"], s["a_scale"], s["w"], s["w_scale"], s["bias"], s["add"], _type(s["y"]))
    if s["op"] == "mlp":
        return _plain_mlp(s)
    if s["op"] == "norm":
        return _plain_codes(_plain_norm(s["x"].float(), s["weight"]), s["form"])
    return _plain_residual(s)


# ----------------------------------------------------- the package's calls
def _values(form, xn, codes, scale):
    """Codes as the numbers they stand for (of E4M3 the same bytes)."""
    return {"xn": xn, "codes": codes.view(torch.float8_e4m3fn) if form == "fp8" else codes.to(torch.bfloat16),
            "scale": scale}


def _own(s):
    from quantized_grouped_gemm_token_amd import ops
    form = s.get("form")
    if s["op"] == "dense":
        return ops.w4a8_moe_dense_i8(s["a"], s["a_scale"], s["w"], s["w_scale"], bias=s["bias"], add=s["add"],
                                     y_dtype=_type(s["y"]))
    if s["op"] == "mlp":
        return ops.w4a8_moe_mlp_i8(s["a"], s["a_scale"], s["w13"], s["s13"], s["w2"], s["s2"], add=s["add"],
                                   y_dtype=_type(s["y"]))
    if s["op"] == "norm":
        fn = ops.w4a8_moe_norm_quant if form == "fp8" else ops.w4a8_moe_norm_quant_i8
        return _values(form, *fn(s["x"], s["weight"], EPS))
    how = dict(post_weight=s["post"], gate=s["gate"], token_gate=s["token_gate"], r_scale=s["r_scale"], eps=EPS)
    if form == "none":
        return {"out": ops.w4a8_moe_residual_norm(s["y"], s["r"], **how)}
    fn = ops.w4a8_moe_residual_norm_quant if form == "fp8" else ops.w4a8_moe_residual_norm_quant_i8
    out, *coded = fn(s["y"], s["r"], s["weight"], **how)
    return {"out": out, **_values(form, *coded)}


def run(state):
    if own:
        return _own(state)
    return _plain(state)


# ------------------------------------------------------------------- work
def work(case):
    e = {"bf16": 2, "f32": 4}
    if case["op"] == "dense":
        M, N, K, b = case["M"], case["N"], case["K"], e[case["y"]]
        more = 4 * N * case["bias"] + M * N * b * case["add"]
        return {"bytes": M * K + N * K + 4 * (M + N) + more + M * N * b, "flops": 2 * M * N * K}
    if case["op"] == "mlp":
        M, H, I, b = case["M"], case["H"], case["I"], e[case["y"]]
        return {"bytes": 3 * I * H + 4 * (M + 2 * I + H) + M * H + M * H * b * (1 + case["add"]),
                "flops": 6 * M * H * I}
    T, H = case["T"], case["H"]
    codes = T * (3 * H + 4) + 4 * H
    if case["op"] == "norm":
        return {"bytes": T * H * e[case["x"]] + codes, "flops": 6 * T * H}
    return {"bytes": T * H * (e[case["y"]] + 2 * e[case["r"]]) + 4 * H * (case["post"] + case["gate"])
            + 4 * T * case["token_gate"] + codes * (case["form"] != "none"), "flops": 12 * T * H}


# ------------------------------------------------------------------ exact
def _exact_sums(a, w):
    """Integer sums by pieces of the outputs, in fp64 (each below 2^53)."""
    a, step = a.double(), max(1, (1 << 26) // w.shape[1])
    return torch.cat([a @ w[n:n + step].double().t() for n in range(0, w.shape[0], step)], 1)


def _exact_quantized(v, fp8):
    """Codes, as values, and scales of the rows of v."""
    top = v.abs().max(1).values
    scale = torch.where(top > 0, top / (448.0 if fp8 else 127.0), torch.ones_like(top))
    q = v / scale.unsqueeze(1)
    if fp8:                                              # 3 bits behind the leading one, 2^-9 the smallest step
        step = torch.exp2(torch.floor(torch.log2(q.abs().clamp_min(2.0 ** -6))) - 3)
        return torch.round(q / step) * step, scale
    return torch.round(q), scale


def _exact_rms(v, weight):
    return weight.double() * v / torch.sqrt(v.square().mean(1, keepdim=True) + EPS)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "dense":
        y = _exact_sums(s["a"], s["w"]) * torch.outer(s["a_scale"].double(), s["w_scale"].double())
        if case["bias"]:
            y += s["bias"].double()
        return y + s["add"].double() if case["add"] else y
    if case["op"] == "mlp":
        h = _exact_sums(s["a"], s["w13"]) * torch.outer(s["a_scale"].double(), s["s13"].double())
        g, u = h.chunk(2, 1)
        q, sq = _exact_quantized(g * torch.sigmoid(g) * u, False)
        y = _exact_sums(q, s["w2"]) * torch.outer(sq, s["s2"].double())
        return y + s["add"].double() if case["add"] else y
    got = {}
    if case["op"] == "norm":
        n = _exact_rms(s["x"].double(), s["weight"])
    else:
        v = s["y"].double()
        if case["post"]:
            v = _exact_rms(v, s["post"])
        for g in (s["gate"], None if s["token_gate"] is None else s["token_gate"].unsqueeze(1)):
            v = v if g is None else v * g.double()
        got["out"] = v + s["r_scale"] * s["r"].double()
        if case["form"] == "none":
            return got
        n = _exact_rms(got["out"], s["weight"])
    q, sq = _exact_quantized(n, case["form"] == "fp8")
    return {**got, "xn": n, "codes": q, "scale": sq}
