"""How far act and y of the few-token layer may be off, element by element, before a quantizer hides it.

act is compared with 64 bits from the tokens' codes; y with 64 bits from the codes of the very act that the
first kernel left, so that no code can fall on the other side of a border.

The model: a result is a sum of G K groups.  In the group-128 form a group's eight matrix-core products and its
scale round sums of at most B_g = sum |a| (q + 16) |s|; adding up the groups, waves and experts rounds sums of at
most P = sum |a w|, and so do the MXFP4 form's four products of a group, which go on from the group before.  A
rounding is off by at most U = 2^-24 of its sum, evenly spread
over both signs: its mean square is at most U^2 / 3 of the sum's square, and independent ones add in squares.
So an element's mean square error is at most

    V = U^2 / 3 (9 sum_g B_g^2 + n P^2),     n: additions behind the groups' products.
"""
import numpy as np

import oracle
from oracle import mxfp4_oracle as mx

U = 2.0 ** -24


def scaled(form, w, s):
    """(W, B) [N, K] in fp64: the weights, and what a group's rounded sums are made of."""
    if form == "mxfp4":
        W = mx.dequant_mxfp4(w[None], s[None])[0].astype(np.float64)
        return W, np.abs(W)
    q = oracle.int4_unpack(w).astype(np.float64)
    f = np.repeat(s.astype(np.float64), 128, -1) if form == "g128" else s.astype(np.float64)[:, None]
    return q * f, (q + 16) * np.abs(f)


def product(form, a, w, s, noise=None):
    """(h, G2, P) of rows a: a x W, sum_g B_g^2 and P.  noise(shape): an error of every group's sum in units of
    B_g, for showing that the bound notices it."""
    W, B = scaled(form, w, s)
    h, G2, P = a @ W.T, np.zeros((len(a), len(w))), np.abs(a) @ np.abs(W).T
    if form == "channel":                                    # exact int32 sums
        return h, G2, P
    for g in range(0, a.shape[1], 128):
        Bg = np.abs(a[:, g:g + 128]) @ B[:, g:g + 128].T
        if form == "g128":
            G2 += Bg * Bg
        if noise is not None:
            h = h + noise(Bg.shape) * Bg
    return h, G2, P


def token_codes(form, x_bits):
    if form == "channel":
        q, sx = oracle.quant_act_i8(x_bits)
        return q.astype(np.float64), sx.astype(np.float64)[:, None]
    q, sx = oracle.quant_act(x_bits)
    return oracle.e4m3_decode(q).astype(np.float64), sx.astype(np.float64)[:, None]


def act_reference(form, x_bits, ids, w13, s13, noise=None):
    """(act, root of V, rest) [T k, I]: rest bounds what the fast exponential and reciprocal and the last products
    add, at most 32 U of act and U of the row's largest (silu's far tail)."""
    a, sx = token_codes(form, x_bits)
    T, k = ids.shape
    I = w13.shape[1] // 2
    act, V, rest = (np.zeros((T * k, I)) for _ in range(3))
    G = a.shape[1] // 128
    for e in np.unique(ids):
        t, j = np.nonzero(ids == e)
        h, G2, P = product(form, a[t], w13[e], s13[e], noise)
        # behind the groups' products: a wave's G / 8 groups, 8 waves
        n = {"channel": 0, "g128": -(-G // 8) + 8, "mxfp4": 4 * -(-G // 8) + 8}[form]
        v = (U * U / 3) * (9 * G2 + n * P * P) * sx[t] ** 2
        h = h * sx[t]
        v = v + U * U * h * h                                # the token's scale (INT8: and the channel's), worst case
        g, u = h[:, :I], h[:, I:]
        with np.errstate(over="ignore"):
            sig = 1 / (1 + np.exp(-g))
        silu, slope = g * sig, sig * (1 + g * (1 - sig))
        f = t * k + j
        act[f] = silu * u
        V[f] = (slope * u) ** 2 * v[:, :I] + silu ** 2 * v[:, I:]
        rest[f] = 32 * U * np.abs(act[f]) + U * np.abs(act[f]).max(1, keepdims=True)
    return act, np.sqrt(V), rest


def act_codes(form, act):
    """The codes' values and the scales that an fp32 act requantizes to."""
    if form == "channel":
        q, sa = oracle.quant_rows_i8(act)
        return q.astype(np.float64), sa.astype(np.float64)[:, None]
    q, sa = oracle.quant_rows(act)
    return oracle.e4m3_decode(q).astype(np.float64), sa.astype(np.float64)[:, None]


def y_reference(form, act, ids, weights, w2, s2, noise=None):
    """(y, root of V, rest) [T, H] from the bits of act and of the routing weights."""
    qa, sa = act_codes(form, act)
    T, k = ids.shape
    H, G = w2.shape[1], qa.shape[1] // 128
    y, V, P_all, rest = (np.zeros((T, H)) for _ in range(4))
    for e in np.unique(ids):
        t, j = np.nonzero(ids == e)
        f = t * k + j
        o, G2, P = product(form, qa[f], w2[e], s2[e], noise)
        c = weights[t, j].astype(np.float64)[:, None] * sa[f]
        np.add.at(y, t, c * o)
        np.add.at(V, t, (U * U / 3) * 9 * c * c * G2)
        np.add.at(P_all, t, c * P)
        np.add.at(rest, t, 4 * U * np.abs(c * o))            # the factor w sa, its product, INT8: the scale
    # a group at a time into a piece, the pieces into a wave's sums, then 8 waves and the workgroups of a block
    V += (U * U / 3) * ((5 if form == "mxfp4" else 2) * k * G + 8 + 16) * P_all ** 2
    return y, np.sqrt(V), rest


def errors(got, want, root, rest):
    """(rms, largest) error beyond rest, in units of the root of V; INT8 forms have errors of `rest` alone."""
    over = np.maximum(np.abs(got.astype(np.float64) - want) - rest, 0.0)
    unit = np.maximum(root, 2.0 ** -130)
    return float(np.sqrt(np.mean((over / unit) ** 2))), float((over / unit).max())
