"""The RMS norm and the 8-bit linear layer at the ends of fp32's range, against 64 bits.

Bounds: those at the head of test_linear_gpu.py. Norm: a row whose squares fp32 does not hold is taken times 2^100, which is
exact. Linear: a block's product of scales below 2^-126 is a multiple of 2^-149, so off by at
most 2^-150, of a block's sum of at most 128 x 448^2 < 2^24.62, and the product with that sum by 2^-150 more: 2^-125.25 for
each block. What of it is a normal product's is 2^-150 a block."""
import pytest
import torch

import split_kv_async_gb300 as F
from test_linear_gpu import CODES, HALF, TYPES, check_norm, e4m3, linear_problem, linear_reference, norm_reference, run_linear

pytestmark = pytest.mark.gpu


# ---- RMS norm ----------------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("out", ["same", "e4m3"])
@pytest.mark.parametrize("dim", [648, 4096, 16392])
@pytest.mark.parametrize("power", [-120, -100, -76, -74, -64, -51, -49, -41, 20, 49, 54])
def test_norm_of_rows_of_any_size(power, dim, out, dtype):
    """Rows of about 2^power without an epsilon: their squares lie below what fp32 holds, at its end, and within."""
    check_norm(3, dim, dtype, out, eps=0.0, seed=power & 0xFF, gain=2.0 ** power)


@pytest.mark.parametrize("out", ["same", "e4m3"])
@pytest.mark.parametrize("power,eps", [(-100, 2.0 ** -120), (-60, 2.0 ** -120), (-60, 2.0 ** -140), (-145, 2.0 ** -149), (-70, 1e-6),
                                       (-45, 2.0 ** -99), (-45, 2.0 ** -101), (54, 2.0 ** -120), (0, 3.4e38)])
def test_norm_with_an_epsilon_of_any_size(power, eps, out):
    check_norm(3, 648, "f32", out, eps=eps, seed=5, gain=2.0 ** power)


@pytest.mark.parametrize("dim", [264, 8192])
def test_norm_rows_of_every_size_in_one_call(dim):
    """Small, ordinary, zero and not finite rows one after another on the same threads, 700 of them (more than
    are at work at once)."""
    T = 700
    gen = torch.Generator("cuda").manual_seed(9)
    x = torch.randn(T, dim, generator=gen, device="cuda")
    powers = torch.tensor([-130, 0, 40, -60, -148, 3, -100], device="cuda", dtype=torch.float64)
    x = (x.double().clamp(-1.9, 1.9) * torch.exp2(powers[torch.arange(T, device="cuda") % 7])[:, None]).float()
    x[7] = 0.0
    x[8, 3], x[9, 5] = float("nan"), float("inf")
    p = F.make_norm_params(num_tokens=T, dim=dim, dtype=F.FDPP_F32, eps=0.0)
    out, total = torch.empty_like(x), torch.empty_like(x)
    F.fdpp_rms_norm(x, None, None, p, out, None, total)
    torch.cuda.synchronize()
    _, y = norm_reference(x, None, None, 0.0, 0.0)
    assert torch.equal(out.isnan(), y.isnan())               # the row of zeros (0 / 0), the NaN's, and inf / inf
    err = (out.double() - y).abs().nan_to_num(0.0)
    assert bool((err <= ((HALF["f32"] + 2.0 ** -18) * y.abs() + 1e-37).nan_to_num(0.0)).all())
    keep = ~x.isnan()
    assert torch.equal(total[keep], x[keep]) and bool(total[~keep].isnan().all())


@pytest.mark.parametrize("out", ["same", "e4m3"])
@pytest.mark.parametrize("dim", [256, 4096])
@pytest.mark.parametrize("eps", [0.0, 1e-6])
def test_norm_at_the_largest_sum_of_squares(eps, dim, out):
    """Channels of 2^64 / sqrt(dim) have a sum of squares of 2^128: just below it y is right, from there on 0."""
    limit = 2.0 ** 64 / dim ** 0.5
    x = torch.tensor([[0.99 * limit], [limit], [1.01 * limit], [1e38]], device="cuda").expand(4, dim).contiguous()
    p = F.make_norm_params(num_tokens=4, dim=dim, dtype=F.FDPP_F32, out_dtype=F.FDPP_E4M3 if out == "e4m3" else None, eps=eps)
    o = torch.full((4, dim), 7, device="cuda", dtype=torch.uint8 if out == "e4m3" else torch.float32)
    scales = torch.full((4, dim // 128), 7.0, device="cuda") if out == "e4m3" else None
    F.fdpp_rms_norm(x, None, None, p, o, scales)
    torch.cuda.synchronize()
    y = e4m3(o).double() * scales.double().repeat_interleave(128, 1) if out == "e4m3" else o.double()
    assert bool(((y[0] - 1).abs() <= 2.0 ** -16).all()) and bool((y[1:] == 0).all())


# ---- linear layer ------------------------------------------------------------------------------

def finite_problem(M, N, K, seed):
    x, sx, w, sw = linear_problem(M, N, K, seed)
    return tuple(torch.where((t & 0x7F) == 0x7F, 0, t) if t.dtype == torch.uint8 else t for t in (x, sx, w, sw))


def about(like, power):
    """Scales of 1 to 1.25 times 2^power (in 64 bits, then rounded: the least ones are subnormal)."""
    return ((1 + torch.rand_like(like).double() / 4) * 2.0 ** power).float()


@pytest.mark.parametrize("M", [9, 40, 150, 300])
@pytest.mark.parametrize("px,pw", [(-80, -45), (-126, 1), (-1, -125), (70, 25), (126, -126), (-126, 126)])
def test_linear_scales_whose_product_is_normal(M, px, pw):
    """The stated accuracy holds as long as the scales' product is a normal number (here the least and some large ones),
    whatever each of them is."""
    x, sx, w, sw = finite_problem(M, 392, 528, 3)
    sx, sw = about(sx, px), about(sw, pw)
    got = run_linear(x, sx, w, sw, "f32")
    want, size = linear_reference(x, sx, w, sw)
    bound = 2.0 ** -24 * want.abs() + 2.0 ** -15 * size + sx.shape[1] * 2.0 ** -150
    assert bool(((got.double() - want).abs() <= bound).all())


@pytest.mark.parametrize("M", [9, 40, 150, 300])
@pytest.mark.parametrize("px,pw", [(-80, -60), (-126, -8), (-140, 10), (-149, 0), (-100, -100)])
def test_linear_scales_whose_product_is_subnormal(M, px, pw):
    x, sx, w, sw = finite_problem(M, 392, 528, 4)
    sx, sw = about(sx, px), about(sw, pw)
    got = run_linear(x, sx, w, sw, "f32")
    want, size = linear_reference(x, sx, w, sw)
    bound = 2.0 ** -24 * want.abs() + 2.0 ** -15 * size + sx.shape[1] * 2.0 ** -125.25
    assert bool(((got.double() - want).abs() <= bound).all())


@pytest.mark.parametrize("M", [9, 150])
def test_linear_zero_scales(M):
    """A zero scale takes its block out, beside the largest finite one as well."""
    x, sx, w, sw = finite_problem(M, 200, 528, 5)
    sx[:, 1] = 0.0
    sw[:, 1] = 3.4e38
    sw[:, 2] = 0.0
    got = run_linear(x, sx, w, sw, "f32")
    want, size = linear_reference(x, sx, w, sw)
    assert bool(((got.double() - want).abs() <= 2.0 ** -24 * want.abs() + 2.0 ** -15 * size).all())


@pytest.mark.parametrize("M", [9, 40, 150, 300])
def test_linear_scales_whose_product_is_infinite(M):
    """Infinite, or NaN where the block's sum is 0, in the rows and weight blocks concerned and no others."""
    x, sx, w, sw = finite_problem(M, 392, 528, 6)
    clean = run_linear(x, sx, w, sw, "f32")
    sw[1, 2] = 2.0 ** 30
    sx[3, 2] = 2.0 ** 100
    other = run_linear(x, sx, w, sw, "f32")
    assert not bool(other[3, 128:256].isfinite().any())
    rows = torch.arange(M, device="cuda") != 3
    assert bool(other[rows].isfinite().all()) and bool(other[3, :128].isfinite().all()) and bool(other[3, 256:].isfinite().all())
    cols = (torch.arange(392, device="cuda") // 128) != 1
    assert torch.equal(other[rows][:, cols], clean[rows][:, cols])
