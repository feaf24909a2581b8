"""Two operators for decoding a few tokens with 4-bit weights, measured on one GPU.

* ``few``: the whole routed-expert layer for 1 to 16 tokens: top-k softmax routing, per-token quantization of
  the activations, gate/up, SwiGLU, per-row requantization, down, and the routing-weighted sum.
* ``matvec``: bf16 activations of 1 to 16 tokens times one 4-bit weight matrix, the activations as they are.

Weights come as a serving program holds them: in the GEMM storage (``layout`` "blk") or as a checkpoint stores
them ("rows"), in one of three forms: "g128" (INT4, an fp32 scale per 128 weights), "channel" (INT4, an fp32 scale
per output) and "mx" (E2M1 codes, an E8M0 scale per 32 weights).

``run`` computes each in its plain form (elementary torch operations in fp32), or with ``own`` set through the
package's entry points.  ``exact`` computes the definition in 64 bits.
"""
from __future__ import annotations

import math

import torch

own = False

DEV = "cuda"
GROUP = 128


# ------------------------------------------------------------------ cases
def _few(name, form, T, H, I, E, k, y="bf16"):
    return dict(name=name, op="few", form=form, T=T, H=H, I=I, E=E, k=k, y=y)


def _matvec(name, form, layout, T, N, K, y="bf16", pad=0):
    return dict(name=name, op="matvec", form=form, layout=layout, T=T, N=N, K=K, y=y, pad=pad)


def listed():
    return [
        # the smallest layer the tests and smoke() use: launches and latency only
        _few("few tiny", "g128", 16, 256, 128, 8, 2),
        # one decoding sequence on the benchmark's layer
        _few("few one token", "g128", 1, 6144, 2048, 256, 8),
        # one sequence with three drafted tokens, MXFP4 experts
        _few("few four tokens mx", "mx", 4, 6144, 2048, 256, 8),
        # a small serving batch, nearly every routed row its own expert: the most bytes
        _few("few sixteen tokens", "g128", 16, 6144, 2048, 256, 8),
        # odd group counts, an expert count that is no power of two, INT8 activations
        _few("few ragged int8", "channel", 5, 2944, 1408, 60, 6),
        # one token through a layer of many small experts
        _few("few small experts mx", "mx", 1, 2048, 768, 128, 8),
        # one expert's gate/up as a dense (shared-expert) projection, one token
        _matvec("matvec gate up", "g128", "blk", 1, 4096, 6144),
        # an output head over a vocabulary, one token, fp32 logits
        _matvec("matvec head", "g128", "blk", 1, 131072, 6144, y="f32"),
        # a wide projection for a small batch
        _matvec("matvec sixteen tokens", "g128", "blk", 16, 12288, 6144),
        # weights as a checkpoint stores them, odd output count, a row length of 91 blocks, strided activations
        _matvec("matvec odd mx rows", "mx", "rows", 3, 5001, 2912, pad=32),
        # per-channel scales as stored, eight tokens, the down projection's shape, fp32 result
        _matvec("matvec channel rows", "channel", "rows", 8, 6144, 2048, y="f32"),
    ]


def _log(rng, lo, hi):
    return math.exp(rng.uniform(math.log(lo), math.log(hi)))


def draw(rng):
    form = rng.choice(["g128", "channel", "mx"])
    y = rng.choice(["bf16", "bf16", "f32"])
    T = min(16, int(_log(rng, 1, 17)))
    if rng.random() < 0.5:
        E = max(2, round(_log(rng, 4, 256)))
        return dict(op="few", form=form, T=T, H=128 * max(1, round(_log(rng, 2, 48))),
                    I=128 * max(1, round(_log(rng, 1, 16))), E=E, k=rng.randint(1, min(8, E)), y="bf16")
    layout = rng.choice(["blk", "rows"])
    N = round(_log(rng, 64, 32768))
    K = 128 * max(1, round(_log(rng, 2, 96)))
    if layout == "blk":
        N = 16 * max(1, N // 16)
    elif form == "mx" and rng.random() < 0.5:
        K += 32 * rng.randint(1, 3)              # a last group that is not whole
    return dict(op="matvec", form=form, layout=layout, T=T, N=N, K=K, y=y, pad=rng.choice([0, 0, 8, 64]))


# ----------------------------------------------------------------- inputs
def _weights(gen, form, layout, lead, N, K):
    """Random 4-bit weights [*lead, N, K] in a storage, with scales of the law the package's workloads use."""
    def scale(*shape):
        return torch.exp(torch.randn(*shape, generator=gen, device=DEV) * 0.5 - 4.0)

    def words(*shape):
        return torch.randint(-2**31, 2**31, shape, generator=gen, device=DEV, dtype=torch.int32)

    G = K // GROUP
    blk = layout == "blk"
    if form == "mx":
        b = lambda *s: (127 + torch.round(torch.log2(scale(*s)))).to(torch.uint8)  # noqa: E731
        if blk:
            return words(*lead, N // 16, G, 16, 16).view(torch.uint8), b(*lead, G, N, 4)
        return words(*lead, N, K // 8).view(torch.uint8), b(*lead, N, K // 32)
    w = words(*lead, N // 16, G, 16, 16) if blk else words(*lead, N, K // 8)
    if form == "channel":
        return w, scale(*lead, N)
    return w, scale(*lead, G, N) if blk else scale(*lead, N, G)


def _tokens(gen, T, K, pad):
    """bf16 activations with 1% outlier channels, in rows of K + pad."""
    x = torch.randn(T, K, generator=gen, device=DEV)
    x = torch.where(torch.rand(K, generator=gen, device=DEV) < 0.01, x * 20, x)
    buf = torch.zeros(T, K + pad, dtype=torch.bfloat16, device=DEV)
    buf[:, :K] = x.to(torch.bfloat16)
    return buf[:, :K]


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    s = dict(case)
    if case["op"] == "few":
        T, H, I, E = case["T"], case["H"], case["I"], case["E"]
        s["x"] = _tokens(gen, T, H, 0)
        s["logits"] = torch.randn(T, E, generator=gen, device=DEV)
        s["w13"], s["s13"] = _weights(gen, case["form"], "blk", (E,), 2 * I, H)
        s["w2"], s["s2"] = _weights(gen, case["form"], "blk", (E,), H, I)
    else:
        s["x"] = _tokens(gen, case["T"], case["K"], case["pad"])
        s["w"], s["s"] = _weights(gen, case["form"], case["layout"], (), case["N"], case["K"])
    return s


# ------------------------------------------------------------- plain form
# K elements of an INT4 word: bit position of element j, in the GEMM storage and as stored
_SHIFTS = {"blk": [0, 8, 16, 24, 4, 12, 20, 28], "rows": [0, 4, 8, 12, 16, 20, 24, 28]}
_E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0]


def _plain_weights(form, layout, w, s):
    """fp32 weights [*, N, K] from a storage (any leading dimensions)."""
    blk = layout == "blk"
    if form == "mx":
        codes = torch.stack([w & 15, w >> 4], dim=-1).flatten(-2).to(torch.int32)
        v = torch.tensor(_E2M1, device=w.device)[codes]
    else:
        sh = torch.tensor(_SHIFTS[layout], dtype=torch.int32, device=w.device)
        v = (((w.unsqueeze(-1) >> sh) & 15) - 8).flatten(-2).float()
    if blk:                                              # [*, N/16, G, 16, 128] -> [*, N, K]
        v = v.transpose(-3, -2)
        v = v.reshape(*v.shape[:-4], v.shape[-4] * 16, v.shape[-2] * 128)
    if form == "channel":
        return v * s.unsqueeze(-1)
    if form == "mx":
        f = (s.to(torch.int32) << 23).view(torch.float32)
        if blk:                                          # [*, G, N, 4] -> [*, N, 4 G]
            f = f.transpose(-3, -2).flatten(-2)
        return v * f.repeat_interleave(32, dim=-1)
    f = s.transpose(-2, -1) if blk else s
    return v * f.repeat_interleave(GROUP, dim=-1)


def _plain_quant(x, int8):
    """Values of the quantized rows (codes times their row's scale is left to the caller) and the scales."""
    amax = x.abs().amax(-1, keepdim=True)
    sc = torch.where(amax > 0, amax / (127.0 if int8 else 448.0), torch.ones_like(amax))
    q = x / sc
    q = q.round().clamp(-127, 127) if int8 else q.to(torch.float8_e4m3fn).float()
    return q, sc


def _out(y, kind):
    return y.to(torch.bfloat16) if kind == "bf16" else y


def _plain_few(s):
    k, I, int8 = s["k"], s["I"], s["form"] == "channel"
    order = torch.sort(s["logits"], dim=-1, descending=True, stable=True)
    top, ids = order.values[:, :k], order.indices[:, :k]
    p = torch.exp(top - top[:, :1])
    w = p / p.sum(-1, keepdim=True)
    q, sx = _plain_quant(s["x"].float(), int8)
    flat = ids.reshape(-1)
    w13 = _plain_weights(s["form"], "blk", s["w13"][flat], s["s13"][flat])       # [T k, 2 I, H]
    h = torch.matmul(w13, q.repeat_interleave(k, 0).unsqueeze(-1)).squeeze(-1) * sx.repeat_interleave(k, 0)
    del w13
    gate, up = h[:, :I], h[:, I:]
    act = gate / (1 + torch.exp(-gate)) * up
    qa, sa = _plain_quant(act, int8)
    w2 = _plain_weights(s["form"], "blk", s["w2"][flat], s["s2"][flat])          # [T k, H, I]
    o = torch.matmul(w2, qa.unsqueeze(-1)).squeeze(-1) * sa
    y = (o.view(*w.shape, -1) * w.unsqueeze(-1)).sum(1)
    return _out(y, s["y"])


def _plain_matvec(s):
    w = _plain_weights(s["form"], s["layout"], s["w"], s["s"])
    return _out(torch.matmul(s["x"].float(), w.transpose(0, 1)), s["y"])


# ----------------------------------------------------- the package's calls
def _own(s):
    from quantized_grouped_gemm_token_amd import ops
    dt = torch.bfloat16 if s["y"] == "bf16" else torch.float32
    if s["op"] == "few":
        fn = {"g128": ops.w4a8_moe_few_prepacked, "channel": ops.w4a8_moe_few_i8_prepacked,
              "mx": ops.w4a8_moe_few_mxfp4_prepacked}[s["form"]]
        return fn(s["x"], s["logits"], s["k"], s["w13"], s["s13"], s["w2"], s["s2"], y_dtype=dt)
    blk = s["layout"] == "blk"
    fn = {"g128": ops.w4a8_moe_matvec_prepacked if blk else ops.w4a8_moe_matvec,
          "channel": ops.w4a8_moe_matvec_channel_prepacked if blk else ops.w4a8_moe_matvec_channel,
          "mx": ops.w4a8_moe_matvec_mxfp4_prepacked if blk else ops.w4a8_moe_matvec_mxfp4}[s["form"]]
    return fn(s["x"], s["w"], s["s"], y_dtype=dt)


def run(state):
    if own:
        return _own(state)
    return _plain_few(state) if state["op"] == "few" else _plain_matvec(state)


# ------------------------------------------------------------------- work
def _weight_bytes(form, N, K):
    return N * K / 2 + (4 * N if form == "channel" else N * K / 32)     # g128: 4 bytes per 128, mx: 1 per 32


def work(case):
    out = 2 if case["y"] == "bf16" else 4
    T = case["T"]
    if case["op"] == "few":
        H, I, E, k = case["H"], case["I"], case["E"], case["k"]
        experts = E * (1 - (1 - k / E) ** T)             # touched under uniform routing, each read once
        each = _weight_bytes(case["form"], 2 * I, H) + _weight_bytes(case["form"], H, I)
        return {"bytes": experts * each + T * (2 * H + 4 * E + out * H), "flops": 6 * T * k * H * I}
    N, K = case["N"], case["K"]
    return {"bytes": _weight_bytes(case["form"], N, K) + T * (2 * K + out * N), "flops": 2 * T * N * K}


# ------------------------------------------------------------------ exact
def _exact_matrix(form, layout, w, s):
    """One weight matrix [N, K] in fp64, element by element from the storage's description."""
    blk = layout == "blk"
    raw = w.contiguous().view(torch.uint8)
    if blk:                                              # [N/16, G, 16, 64] bytes -> rows of K/2 bytes
        raw = raw.view(raw.shape[0], raw.shape[1], 16, 64).permute(0, 2, 1, 3)
        raw = raw.reshape(raw.shape[0] * 16, -1)
    lo, hi = (raw & 15).long(), (raw >> 4).long()
    if form == "mx":
        c = torch.stack([lo, hi], -1).view(raw.shape[0], -1)
        mag, e = (c & 1).double(), (c >> 1) & 3
        v = torch.where(e == 0, mag * 0.5, (1 + mag * 0.5) * torch.pow(2.0, (e - 1).double()))
        v = torch.where(c >= 8, -v, v)
        b = s.permute(1, 0, 2).reshape(s.shape[1], -1) if blk else s
        return v * torch.pow(2.0, b.double() - 127).repeat_interleave(32, 1)
    nib = torch.stack([lo, hi], -1).view(raw.shape[0], -1, 8)         # the nibbles of each word, from bit 0
    if blk:
        nib = nib[:, :, [0, 2, 4, 6, 1, 3, 5, 7]]                     # held in the order k0 k4 k1 k5 k2 k6 k3 k7
    v = nib.reshape(raw.shape[0], -1).double() - 8
    if form == "channel":
        return v * s.double()[:, None]
    return v * (s.t() if blk else s).double().repeat_interleave(GROUP, 1)


def _exact_codes(x, int8):
    """Quantized rows by their rule: the fp32 scale, the fp32 quotient (many a bf16 value falls on a border between
    two codes only once the quotient is rounded), then the nearest code, ties to even."""
    amax = x.abs().amax(1, keepdim=True)
    sc = torch.where(amax > 0, amax / (127 if int8 else 448), torch.ones_like(amax)).float().double()
    v = (x / sc).float().double()
    if int8:
        return torch.round(v).clamp(-127, 127), sc
    e = torch.floor(torch.log2(v.abs().clamp_min(1e-300))).clamp(-6, 8)
    step = torch.pow(2.0, e - 3)
    return (torch.round(v / step) * step).clamp(-448, 448), sc


def exact(case, seed):
    s = prepare(case, seed)
    form = case["form"]
    if case["op"] == "matvec":
        x = s["x"].double()
        rows = []
        step = 16 * max(1, (1 << 24) // case["K"])
        for n in range(0, case["N"], step):              # a slice of the outputs at a time
            if case["layout"] == "blk":
                w = s["w"][n // 16:(n + step) // 16]
                sc = s["s"][n:n + step] if form == "channel" else s["s"][:, n:n + step]
            else:
                w, sc = s["w"][n:n + step], s["s"][n:n + step]
            rows.append(x @ _exact_matrix(form, case["layout"], w, sc).t())
        return torch.cat(rows, 1)
    T, k, I, int8 = case["T"], case["k"], case["I"], form == "channel"
    lg = s["logits"].double()
    ids = torch.argsort(lg, dim=1, descending=True, stable=True)[:, :k]
    p = torch.softmax(torch.gather(lg, 1, ids), 1)       # the softmax over all experts, renormalized over the k
    q, sx = _exact_codes(s["x"].double(), int8)
    y = torch.zeros(T, case["H"], dtype=torch.float64, device=DEV)
    for e in sorted(set(ids.flatten().tolist())):        # one expert at a time, its tokens together
        t, j = torch.nonzero(ids == e, as_tuple=True)
        h = (q[t] @ _exact_matrix(form, "blk", s["w13"][e], s["s13"][e]).t()) * sx[t]
        act = h[:, :I] * torch.sigmoid(h[:, :I]) * h[:, I:]
        qa, sa = _exact_codes(act, int8)
        o = (qa @ _exact_matrix(form, "blk", s["w2"][e], s["s2"][e]).t()) * sa
        y[t] += p[t, j][:, None] * o
    return y
