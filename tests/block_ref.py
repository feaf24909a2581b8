"""Plain 64-bit forms of the operators around the experts, for their tests (numpy)."""
from __future__ import annotations

import numpy as np

HALF_BF16 = 2.0 ** -8       # half a step of bf16, relative to the value
HALF_F32 = 2.0 ** -24


def int_sums(a, w):
    """sum_k a[m, k] w[n, k], exact: fp64 holds integers below 2^53."""
    return a.astype(np.float64) @ w.astype(np.float64).T


def dense_f32(a, a_scale, w, w_scale):
    """The product without bias and addend as the header rounds it: the sum, then each scale, in fp32."""
    return int_sums(a, w).astype(np.float32) * a_scale[:, None] * w_scale[None, :]


def check_dense(got, a, a_scale, w, w_scale, bias=None, add=None, bf16=False, what=""):
    """got (fp64 values of y) against the definition.  The product carries three roundings (the sum, two scales), the
    bias and the addend one each of what they give; then half a step of bf16."""
    p = int_sums(a, w) * a_scale.astype(np.float64)[:, None] * w_scale.astype(np.float64)
    tol = 3 * HALF_F32 * np.abs(p)
    y = p.copy()
    for more in (bias, add):
        if more is not None:
            y = y + more.astype(np.float64)
            tol = tol + HALF_F32 * np.abs(y)
    tol = 1.001 * tol + 2.0 ** -149
    if bf16:
        tol = tol + HALF_BF16 * (np.abs(y) + tol)
    bad = ~(np.abs(got - y) <= tol)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.size} off, first at {np.argwhere(bad)[0]}"


def check_mlp(got, a, a_scale, w13, s13, w2, s2, add=None, bf16=False, what=""):
    """got against the definition.  act is fp32: h carries three roundings, the hardware exponential, reciprocal and
    three products some ulp (16 in all, and 2^-24 of the row's largest value far down silu's tail), so a code within
    2^-15 of a border between two (127 times 2 x 16 x 2^-24, rounded up) may be either of them."""
    I = w2.shape[1]
    h = int_sums(a, w13) * a_scale.astype(np.float64)[:, None] * s13.astype(np.float64)
    g, u = h[:, :I], h[:, I:]
    with np.errstate(over="ignore"):
        act = g / (1 + np.exp(-g)) * u
    top = np.abs(act).max(1)
    sa = np.where(top > 0, top / 127, 1.0)
    v = act / sa[:, None]
    q = np.rint(v)
    near = np.abs(np.abs(v - np.floor(v)) - 0.5) <= 2.0 ** -15
    y = (q @ w2.astype(np.float64).T) * sa[:, None] * s2.astype(np.float64)
    tol = (near.astype(np.float64) @ np.abs(w2.astype(np.float64)).T) * sa[:, None] * s2
    tol = tol + 24 * HALF_F32 * np.abs(y)                    # sa's error (that of act) and the product's roundings
    if add is not None:
        y = y + add.astype(np.float64)
        tol = tol + HALF_F32 * np.abs(y)
    tol = 1.001 * tol + 2.0 ** -149
    if bf16:
        tol = tol + HALF_BF16 * (np.abs(y) + tol)
    bad = ~(np.abs(got - y) <= tol)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.size} off, first at {np.argwhere(bad)[0]}"


def rms(v, weight, eps):
    return weight.astype(np.float64) * v / np.sqrt((v * v).mean(1, keepdims=True) + eps)


# fp32 error of a norm relative to the value: the sum of squares of 32768 values by 1024 threads is a chain of at most
# 32 FMAs and 26 adds (58 half steps, halved by the root), the quotient and eps 2, the root 2, three products 3.
NORM_REL = 40 * HALF_F32

E4M3 = np.array([(m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)) for e in range(16) for m in range(8)]
                [:127])


def check_codes(n, rel, absolute, q, s, fp8, what=""):
    """Codes q (bytes) and scales s of rows n that the kernel holds to within rel |n| + absolute max |n|.

    A quotient n / s is then off by rel |n / s| and by absolute max |n| / s, which is absolute times the largest code
    whatever n is, and by the scale's own error, rel + absolute and two roundings of it."""
    top = np.abs(n).max(1)
    want = np.where(top > 0, top / (448.0 if fp8 else 127.0), 1.0)
    # (a step of the smallest fp32 where the scale is tiny)
    assert np.all(np.abs(s - want) <= (rel + absolute + 2 * HALF_F32) * want + 2.0 ** -149), f"{what}: scales"
    if fp8:
        mag, val = E4M3[q & 0x7F], np.abs(n) / s[:, None]
        assert np.all(((q & 0x7F) != 0x7F)), f"{what}: a code is NaN"
        i = np.clip(np.searchsorted(E4M3, val), 1, len(E4M3) - 1)
        gap = E4M3[i] - E4M3[i - 1]                          # the distance of the codes around the value
        signs = (q >= 0x80) == (n < 0)
        assert np.all(signs | (mag == 0)), f"{what}: signs"
    else:
        mag, val, gap = np.abs(q.astype(np.float64)), np.abs(n) / s[:, None], 1.0
        assert np.all((np.sign(q) == np.sign(n)) | (q == 0)), f"{what}: signs"
    err = np.abs(mag - val)
    bad = ~(err <= gap / 2 + (2 * rel + absolute + 4 * HALF_F32) * val + 1.01 * absolute * (448 if fp8 else 127))
    bad[top <= 2.0 ** -120] = False                          # scales of a few bits: the codes' steps are theirs
    assert not bad.any(), f"{what}: {int(bad.sum())} codes are not the nearest, first at {np.argwhere(bad)[0]}"
