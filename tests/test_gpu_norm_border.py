"""Norms of rows whose mean square and eps come next to a power of 4 (rows that were normed before), where the factor
of a row lies on either side of a power of two by its last bit; and of rows whose squares come next to fp32's largest sum."""
import numpy as np
import pytest
import torch

from block_ref import HALF_BF16, HALF_F32, NORM_REL
from gpu_util import DEV, say
from quantized_grouped_gemm_token_amd import ops

pytestmark = pytest.mark.gpu

EPS = 1e-6


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    assert ops.w4a8_moe_device_supported(), "the current device is not a gfx950"
    yield
    torch.cuda.synchronize()


def normed_rows(gen, T, H, dtype, power, near):
    """x / sqrt(mean x^2 + eps) times 2^power, rounded to dtype: its mean square and eps 4^power make 4^power, but for
    the rounding and eps times what mean x^2 lacks to 1.  Mean squares are off by up to `near` more."""
    x = torch.randn(T, H, device=DEV, generator=gen, dtype=torch.float64)
    x = x / torch.sqrt((x * x).mean(1, keepdim=True) + EPS)
    x = x * torch.sqrt(1 + near * (2 * torch.rand(T, 1, device=DEV, generator=gen, dtype=torch.float64) - 1))
    return torch.ldexp(x, torch.tensor(power, device=DEV)).to(dtype)


def check(x, w, eps, xn, q, s, i8):
    """Each code the nearest to the exact quotient by the row's largest product (2^-52 of 64 bits; quotients within
    2^-42 of a border may have either code); xn and scales within the fp32 norm's error, NORM_REL, and their own
    roundings."""
    p = x.double() * w.double()                              # exact
    top = p.abs().amax(1, keepdim=True)
    largest = 127.0 if i8 else 448.0
    v = p / top * largest
    if i8:
        got, step = q.double(), torch.ones_like(v)
    else:
        got = q.view(torch.float8_e4m3fn).double()
        e = (torch.frexp(v)[1] - 1).clamp_min(-6)            # 3 bits behind the leading one, 2^-9 the smallest step
        step = torch.ldexp(torch.ones_like(v), e - 3)
    far = ((got - v).abs() > step / 2 + 2.0 ** -42 * v.abs()).sum(1)
    assert not bool(far.any()), f"{int((far > 0).sum())} of {len(far)} rows have codes that are not the nearest, " \
                                f"up to {int(far.max())} of {x.shape[1]}"
    f = 1 / torch.sqrt((x.double() ** 2).mean(1, keepdim=True) + eps)
    want = top * f / largest
    assert bool(((s.double()[:, None] - want).abs() <= 1.001 * (NORM_REL + 2 * HALF_F32) * want).all())
    n = p * f
    tol = NORM_REL * n.abs()
    assert bool(((xn.double() - n).abs() <= tol + HALF_BF16 * (n.abs() + tol)).all())


# a wave, 128, 256 and 512 threads a row, 1024 for few rows, for residual rows beyond 8192 and for rows beyond 16384
SIZES = [(40000, 512), (20000, 1024), (4000, 2048), (256, 2056), (256, 6144), (300, 6144), (256, 12288), (300, 12288),
         (200, 24576)]


@pytest.mark.parametrize("i8", [False, True], ids=["fp8", "i8"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("T,H", SIZES)
def test_codes_of_normed_rows(T, H, dtype, i8):
    gen = torch.Generator(device=DEV).manual_seed(T + H)
    w = 1 + 0.2 * torch.randn(H, device=DEV, generator=gen)
    say(f"norms of normed rows T={T} H={H} {dtype} i8={i8}")
    for draw in range(max(2, 6000 // T)):
        power = (0, 1, -1)[draw % 3]
        eps = EPS * 4.0 ** power
        x = normed_rows(gen, T, H, dtype, power, 2.0 ** -22 if draw % 2 else 0.0)
        if i8:
            rowsum = torch.full((T,), 7, dtype=torch.int32, device=DEV)
            xn, q, s = ops.w4a8_moe_norm_quant_i8(x, w, eps, rowsum=rowsum)
            assert torch.equal(rowsum, q.sum(1, dtype=torch.int32))
        else:
            xn, q, s = ops.w4a8_moe_norm_quant(x, w, eps)
        check(x, w, np.float32(eps).item(), xn, q, s, i8)
        # the residual form on a block's result of zeros: the same rows again, and the same next norm
        zero = torch.zeros_like(x)
        fn = ops.w4a8_moe_residual_norm_quant_i8 if i8 else ops.w4a8_moe_residual_norm_quant
        out, xn, q, s = fn(zero, x, w, post_weight=w if draw % 2 else None, eps=eps)
        assert torch.equal(out, x)
        check(x, w, np.float32(eps).item(), xn, q, s, i8)


@pytest.mark.parametrize("i8", [False, True], ids=["fp8", "i8"])
@pytest.mark.parametrize("T,H", [(3000, 512), (256, 6144), (300, 12288), (200, 24576)])
def test_rows_whose_squares_come_next_to_the_largest_sum(T, H, i8):
    """Sums of squares within 2^-21 of 2^128: some round to infinity and are taken again of scaled values, some do not;
    each row's codes and scale are right either way."""
    gen = torch.Generator(device=DEV).manual_seed(T + H)
    w = 1 + 0.2 * torch.randn(H, device=DEV, generator=gen)
    x = torch.randn(T, H, device=DEV, generator=gen, dtype=torch.float64)
    near = 1 + 2.0 ** -21 * (2 * torch.rand(T, 1, device=DEV, generator=gen, dtype=torch.float64) - 1)
    x = (x * torch.sqrt(near / (x * x).sum(1, keepdim=True)) * 2.0 ** 64).float()
    say(f"norms of rows next to the largest sum T={T} H={H} i8={i8}")
    fn = ops.w4a8_moe_norm_quant_i8 if i8 else ops.w4a8_moe_norm_quant
    check(x, w, EPS, *fn(x, w, EPS), i8)
    fn = ops.w4a8_moe_residual_norm_quant_i8 if i8 else ops.w4a8_moe_residual_norm_quant
    out, *coded = fn(x, torch.zeros_like(x), w, eps=EPS)
    assert torch.equal(out, x)
    check(x, w, EPS, *coded, i8)
    # and as a block's result that is normed
    out = ops.w4a8_moe_residual_norm(x, torch.zeros_like(x), post_weight=w, eps=EPS)
    n = x.double() * w.double() / torch.sqrt((x.double() ** 2).mean(1, keepdim=True))
    assert bool(((out.double() - n).abs() <= (NORM_REL + HALF_F32) * n.abs()).all())


@pytest.mark.parametrize("i8", [False, True], ids=["fp8", "i8"])
@pytest.mark.parametrize("H,eps", [(8, 3.3e38), (64, 2.0 ** 127), (512, 1e30), (512, 1e36), (6144, 1e33), (20000, 1e35)])
def test_eps_next_to_the_largest_squares(H, eps, i8):
    """An eps that matters next to rows whose sum of squares overflows, or that overflows with a mean square."""
    gen = torch.Generator(device=DEV).manual_seed(H)
    w = 1 + 0.2 * torch.randn(H, device=DEV, generator=gen)
    gains = torch.tensor([1e10, 1e15, 1e17, 1e18, 6e18, 1e19, 2e19, 1e20, 1e25, 1e36], device=DEV, dtype=torch.float64)
    x = torch.randn(len(gains), H, device=DEV, generator=gen, dtype=torch.float64)
    x = (x / x.abs().amax(1, keepdim=True) * gains[:, None]).float()
    say(f"norms with eps={eps} H={H} i8={i8}")
    fn = ops.w4a8_moe_norm_quant_i8 if i8 else ops.w4a8_moe_norm_quant
    check(x, w, np.float32(eps).item(), *fn(x, w, eps), i8)
    y = ops.w4a8_moe_residual_norm(x, torch.zeros_like(x), post_weight=w, eps=eps)
    n = x.double() * w.double() / torch.sqrt((x.double() ** 2).mean(1, keepdim=True) + np.float32(eps).item())
    assert bool(((y.double() - n).abs() <= (NORM_REL + HALF_F32) * n.abs()).all())
