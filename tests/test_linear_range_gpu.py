"""The RMS norm at the ends of fp32's range, against 64 bits.

Bounds: those at the head of test_linear_gpu.py. Norm: a row whose squares fp32 does not hold is taken times 2^100, which is
exact."""
import pytest
import torch

import split_kv_async_gb300 as F
from test_linear_gpu import HALF, check_norm, e4m3, norm_reference

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
