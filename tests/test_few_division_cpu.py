"""x / s by a reciprocal, as the few-token layer divides a row by its scale: q = fl(x r) with r = fl(1 / s), then
fl(q + r (x - q s)), is the correctly rounded quotient (the kernel's div_by, restated in exact arithmetic)."""
import numpy as np
import pytest


def round_sum(a, b):
    """a + b (fp64, |a| >= |b|) rounded once to fp32."""
    s = a + b
    e = b - (s - a)                                          # what fp64 lost (exact)
    r = s.astype(np.float32)
    # fp64 lands on a border between two fp32 values: its lost part decides, an exact tie goes to even
    lo, hi = np.nextafter(r, np.float32(-np.inf)).astype(np.float64), np.nextafter(r, np.float32(np.inf)).astype(np.float64)
    up, down = (s == (r.astype(np.float64) + hi) / 2) & (e > 0), (s == (r.astype(np.float64) + lo) / 2) & (e < 0)
    return np.where(up, hi, np.where(down, lo, r.astype(np.float64))).astype(np.float32)


def div_by(x, s):
    r = (np.float32(1) / s).astype(np.float32)
    q = (x * r).astype(np.float32)
    x64, s64, q64 = x.astype(np.float64), s.astype(np.float64), q.astype(np.float64)
    res = (x64 - q64 * s64).astype(np.float32)               # 48 bits below x's: exact in fp64, then one rounding
    return round_sum(q64, res.astype(np.float64) * r.astype(np.float64))


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("top", [127, 448])
def test_quotients_are_correctly_rounded(top, bf16):
    rng = np.random.Generator(np.random.PCG64(top))
    for _ in range(10):
        amax = np.exp2(rng.uniform(-70, 100, 500_000)).astype(np.float32)
        x = (amax * rng.uniform(-1, 1, amax.size) * np.exp2(-rng.integers(0, 12, amax.size))).astype(np.float32)
        if bf16:
            amax, x = ((v.view(np.uint32) & np.uint32(0xffff0000)).view(np.float32) for v in (amax, x))
        s = (amax / np.float32(top)).astype(np.float32)
        want = x / s
        got = div_by(x, s)
        assert np.array_equal(got, want)
