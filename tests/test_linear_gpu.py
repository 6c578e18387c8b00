"""The RMS norm and the 8-bit linear layer on the GPU against 64 bits.

Bounds, from the arithmetic. Norm: a row's sum of squares is made of at most 32 terms in a row per thread and
two trees over the threads, so it is off by less than 2^6 roundings of 2^-24, its square root's reciprocal by
half of that; the sum x + residual, the weight's offset and the products add six roundings: 2^-18 |y| in all,
then the output's rounding (half a step). e4m3: half a step is 2^-4 of a value (2^-10 of the scale below 2^-6).
Linear: a block's 128 products are exact in fp32; their sum, by adders of fp32's width at least, is off by
at most 2^7 x 2^-23 of sum |x w|, the sum over up to 2^7 blocks by 2^7 x 2^-24 of it, the scales' product by
2^-24: 2^-15 of the scaled sum |x w|, then the output's rounding."""
import numpy as np
import pytest
import torch

import split_kv_async_gb300 as F

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
CODES = {"bf16": F.FDPP_BF16, "f32": F.FDPP_F32}
HALF = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}
FP8 = torch.float8_e4m3fn
NAN_BYTE = 0x7F


def filled(rows, stride, dtype, value):
    return torch.full((rows, stride), value, dtype=dtype, device="cuda")


def e4m3(t):
    """uint8 bytes as the fp32 values they stand for."""
    return t.contiguous().view(FP8).float()


# ---- RMS norm ----------------------------------------------------------------------------------

def norm_reference(x, residual, weight, eps, offset):
    r = x.double() + (residual.double() if residual is not None else 0.0)
    y = r / torch.sqrt((r * r).mean(-1, keepdim=True) + eps)
    return r, y * (weight.double() + offset) if weight is not None else y


def check_norm(T, dim, dtype="bf16", out="same", residual=True, weight=True, offset=0.0, pad=0, eps=1e-6, seed=0, gain=1.0,
               in_place=False):
    gen = torch.Generator("cuda").manual_seed(seed)
    tdt = TYPES[dtype]
    stride = dim + pad
    rand = lambda: (gain * torch.randn(T, stride, generator=gen, device="cuda")).to(tdt)  # noqa: E731
    x, res = rand(), rand() if residual else None
    w = torch.randn(dim, generator=gen, device="cuda").to(tdt) if weight else None
    x[:, dim:] = float("nan")
    if residual:
        res[:, dim:] = float("nan")
    r, y = norm_reference(x[:, :dim], None if res is None else res[:, :dim], w, eps, offset)
    blocks = -(-dim // 128)
    total = res if in_place else filled(T, stride, tdt, 7.0)
    kw = dict(num_tokens=T, dim=dim, dtype=CODES[dtype], eps=eps, weight_offset=offset, x_stride=stride, residual_stride=stride,
              sum_stride=stride)
    if out == "same":
        p = F.make_norm_params(out_stride=stride, **kw)
        o, scales = (x if in_place else filled(T, stride, tdt, 7.0)), None
    else:
        p = F.make_norm_params(out_dtype=F.FDPP_E4M3, out_stride=stride + 8, scale_stride=blocks + 3, **kw)
        o, scales = filled(T, p.out_stride, torch.uint8, 0xAB), filled(T, blocks + 3, torch.float32, 7.0)
    F.fdpp_rms_norm(x, res, w, p, o, scales, total)
    torch.cuda.synchronize()
    tiny = 1e-37
    err = (total[:, :dim].double() - r).abs()
    assert bool((err <= (HALF[dtype] + 2.0 ** -23) * r.abs() + tiny).all())
    if not in_place:
        assert bool((total[:, dim:] == 7.0).all())
    if out == "same":
        assert bool(((o[:, :dim].double() - y).abs() <= (HALF[dtype] + 2.0 ** -18) * y.abs() + tiny).all())
        if not in_place:
            assert bool((o[:, dim:] == 7.0).all())
        return
    padded = torch.nn.functional.pad(y, (0, blocks * 128 - dim)).reshape(T, blocks, 128)
    want = (padded.abs().amax(-1) / 448.0).clamp(min=2.0 ** -126)
    s = scales[:, :blocks].double()
    assert bool(((s - want).abs() <= 2.0 ** -17 * want).all())
    each = s.repeat_interleave(128, 1)[:, :dim]
    got = e4m3(o[:, :dim]).double() * each
    assert bool(((got - y).abs() <= (2.0 ** -4 + 2.0 ** -16) * y.abs() + 2.0 ** -10 * each).all())
    assert bool((o[:, dim:] == 0xAB).all()) and bool((scales[:, blocks:] == 7.0).all())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("out", ["same", "e4m3"])
@pytest.mark.parametrize("T,dim", [(1, 8), (1, 128), (3, 136), (7, 256), (9, 504), (33, 1024), (5, 1032), (2, 4096), (3, 4104), (2, 8192),
                                   (1, 16392), (1, 32768)])
def test_norm_sizes(T, dim, dtype, out):
    check_norm(T, dim, dtype, out)


@pytest.mark.parametrize("kw", [dict(residual=False), dict(weight=False), dict(offset=1.0), dict(pad=8), dict(pad=40, T=700),
                                dict(gain=1e-18, dtype="f32"), dict(gain=1e10), dict(in_place=True),
                                dict(in_place=True, dtype="f32"), dict(residual=False, weight=False, T=5, dim=64)])
@pytest.mark.parametrize("out", ["same", "e4m3"])
def test_norm_options(kw, out):
    kw = {**dict(T=6, dim=648), **kw}
    if kw.get("in_place") and out == "e4m3":
        kw["in_place"] = False
    check_norm(out=out, eps=0.0 if kw.get("gain", 1.0) < 1 else 1e-5, seed=3, **kw)


def test_norm_of_zeros_and_of_values_that_are_not_finite():
    T, dim = 5, 384
    x = torch.ones(T, dim, device="cuda")
    x[0] = 0.0
    x[2, 5] = float("nan")
    x[3, 200] = float("inf")
    x[4, :128] = 1e-30
    p = F.make_norm_params(num_tokens=T, dim=dim, dtype=F.FDPP_F32, out_dtype=F.FDPP_E4M3, eps=1e-6)
    out, scales = torch.empty(T, dim, device="cuda", dtype=torch.uint8), torch.empty(T, 3, device="cuda")
    F.fdpp_rms_norm(x, None, None, p, out, scales)
    torch.cuda.synchronize()
    v = e4m3(out)
    assert bool((v[0] == 0).all()) and bool((scales[0] == 2.0 ** -126).all())
    assert bool((v[1] == 448).all())
    assert bool(v[2].isnan().all()) and bool(scales[2].isnan().all())
    # the infinity's row: finite values over an infinite root are 0, the infinity itself inf / inf
    assert bool((v[3, :128] == 0).all()) and bool(v[3, 128:256].isnan().all()) and bool((v[3, 256:] == 0).all())
    assert bool((v[4] == 448).all())               # blocks of very different sizes: each by its own scale


@pytest.mark.parametrize("dim", [8, 24, 136, 1000, 2056])
def test_norm_contiguous_rows_end_where_the_buffer_does(dim):
    """Contiguous e4m3 rows by the binding's defaults, of channels that are no multiple of 16: nothing behind them
    is written."""
    T = 9
    x = torch.randn(T, dim, device="cuda")
    p = F.make_norm_params(num_tokens=T, dim=dim, dtype=F.FDPP_F32, out_dtype=F.FDPP_E4M3)
    buf, scales = torch.full((T * dim + 64,), 0xAB, device="cuda", dtype=torch.uint8), torch.empty(T, p.scale_stride, device="cuda")
    F.fdpp_rms_norm(x, None, None, p, buf, scales)
    torch.cuda.synchronize()
    assert bool((buf[T * dim:] == 0xAB).all())
    _, y = norm_reference(x, None, None, 1e-6, 0.0)
    each = scales.double().repeat_interleave(128, 1)[:, :dim]
    got = e4m3(buf[:T * dim].reshape(T, dim)).double() * each
    assert bool(((got - y).abs() <= (2.0 ** -4 + 2.0 ** -16) * y.abs() + 2.0 ** -10 * each).all())


def test_norm_of_nothing():
    p = F.make_norm_params(num_tokens=0, dim=64, dtype=F.FDPP_F32)
    x = torch.ones(1, 64, device="cuda")
    out = torch.full((1, 64), 3.0, device="cuda")
    F.fdpp_rms_norm(x, None, None, p, out)
    torch.cuda.synchronize()
    assert bool((out == 3.0).all())


# ---- linear layer ------------------------------------------------------------------------------

def linear_problem(M, N, K, seed=0, spread=1.0):
    """e4m3 bytes (values that the type cannot hold become NaN: a few in a million) and scales; `spread`: how
    far (in powers of two) the blocks' scales differ."""
    gen = torch.Generator("cuda").manual_seed(seed)
    kb, nb = -(-K // 128), -(-N // 128)
    byte = lambda r: (torch.randn(r, K, generator=gen, device="cuda") * 100).to(FP8).view(torch.uint8)  # noqa: E731
    scale = lambda *s: torch.exp2(spread * torch.randn(*s, generator=gen, device="cuda"))  # noqa: E731
    return byte(M), scale(M, kb), byte(N), scale(nb, kb)


def linear_reference(x, sx, w, sw):
    """(y, the scaled sum of |x w|) in 64 bits."""
    K = x.shape[1]
    xd = e4m3(x).double() * sx.double().repeat_interleave(128, 1)[:, :K]
    wd = e4m3(w).double() * sw.double().repeat_interleave(128, 0)[:w.shape[0]].repeat_interleave(128, 1)[:, :K]
    return xd @ wd.T, xd.abs() @ wd.abs().T


def run_linear(x, sx, w, sw, out="bf16", split_k=0, xpad=0, wpad=0, ypad=0, spad=0, offset=0):
    """Through the library, every buffer with rows and columns of poison around it."""
    (M, K), N = x.shape, w.shape[0]

    def padded(t, pad, rows):
        o = torch.full((t.shape[0] + rows, K + pad), NAN_BYTE, dtype=torch.uint8, device="cuda")
        o[:t.shape[0], :K] = t
        return o

    xs, wsrc = padded(x, xpad, 3), padded(w, wpad, 3)
    s = torch.full((M + 3, sx.shape[1] + spad), float("nan"), device="cuda")
    s[:M, :sx.shape[1]] = sx
    stride = N + ypad
    y = torch.full((offset + (M + 2) * stride,), 7.0, dtype=TYPES[out], device="cuda")
    p = F.make_scaled_gemm_params(M=M, N=N, K=K, out_dtype=CODES[out], x_stride=K + xpad, w_stride=K + wpad, y_stride=stride,
                                  x_scale_stride=sx.shape[1] + spad, split_k=split_k)
    ws = F.alloc_scaled_gemm_workspace(p)
    F.fdpp_scaled_gemm(xs, s, wsrc, sw, p, ws, y[offset:])
    assert F.fdpp_read_error(ws) == 0
    rows = y[offset:].reshape(M + 2, stride)
    assert bool((y[:offset] == 7.0).all()) and bool((rows[M:] == 7.0).all()) and bool((rows[:, N:] == 7.0).all())
    return rows[:M, :N].clone()


def check_linear(M, N, K, out="bf16", seed=0, spread=1.0, **kw):
    x, sx, w, sw = linear_problem(M, N, K, seed, spread)
    got = run_linear(x, sx, w, sw, out, **kw)
    want, size = linear_reference(x, sx, w, sw)
    assert torch.equal(got.isnan(), want.isnan())      # a NaN operand's row or column, and no other
    err = (got.double() - want).abs().nan_to_num(0.0)
    bound = (HALF[out] * want.abs() + 2.0 ** -15 * size).nan_to_num(0.0)
    assert bool((err <= bound).all()), float((err / bound).max())
    return got


def same(a, b):
    return (a == b) | (a.isnan() & b.isnan())


@pytest.mark.parametrize("M", [1, 7, 16, 17, 33, 64, 100, 128, 129, 200, 300])
@pytest.mark.parametrize("N,K", [(1, 16), (100, 128), (128, 144), (260, 1040), (1000, 2048)])
def test_linear_sizes(M, N, K):
    check_linear(M, N, K, "f32" if (M + N) % 2 else "bf16")


@pytest.mark.parametrize("M", [5, 128])
@pytest.mark.parametrize("split_k", range(1, 9))
def test_linear_splits(M, split_k):
    check_linear(M, 300, 1168, "f32", split_k=split_k)


@pytest.mark.parametrize("M", [3, 140])
@pytest.mark.parametrize("kw", [dict(xpad=16), dict(wpad=32), dict(ypad=1), dict(ypad=7, offset=1), dict(ypad=8, offset=4), dict(spad=3),
                                dict(xpad=112, wpad=16, ypad=3, spad=1, offset=2)])
@pytest.mark.parametrize("out", ["bf16", "f32"])
def test_linear_strides(M, kw, out):
    check_linear(M, 333 if kw.get("offset") else 384, 400, out, **kw)


@pytest.mark.parametrize("M,N,K", [(1024, 5120, 512), (640, 8192 + 72, 1024), (2500, 2056, 272), (8192, 1024, 128)])
def test_linear_many_tiles(M, N, K):
    check_linear(M, N, K)


@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("M,N,K", [
    (1000, 4096, 272), (70, 20000, 144), (129, 10250, 400),      # 128 x 256 tiles, one for an SM at most
    (260, 4000, 8208), (130, 6300, 9216),                        # .. that share out a long K
    (70, 40000, 144),                                            # .. two for an SM: pairs would be half empty
    (1200, 4000, 272),                                           # pairs
])
def test_linear_tiles_of_every_kind(M, N, K, out):
    check_linear(M, N, K, out, ypad=3 if M == 130 else 0)


@pytest.mark.parametrize("split_k", [1, 2, 5, 8])
def test_linear_splits_of_wide_tiles(split_k):
    check_linear(300, 6000, 1168, "f32", split_k=split_k)


@pytest.mark.parametrize("M", [9, 150])
def test_linear_scales_of_every_size(M):
    check_linear(M, 520, 900 // 16 * 16, "f32", spread=12.0)


@pytest.mark.parametrize("M", [20, 300])
def test_linear_values_that_are_not_finite_stay_in_their_row(M):
    x, sx, w, sw = linear_problem(M, 200, 528)
    clean = run_linear(x, sx, w, sw)
    x[3, 77] = NAN_BYTE
    sx[5, 2] = float("inf")
    sx[6, 4] = float("nan")
    w[11, 300] = NAN_BYTE
    got = run_linear(x, sx, w, sw)
    assert bool(got[3].isnan().all()) and bool(got[6].isnan().all()) and bool(got[:, 11].isnan().all())
    keep = torch.ones(M, dtype=torch.bool, device="cuda")
    keep[[3, 5, 6]] = False
    cols = torch.ones(200, dtype=torch.bool, device="cuda")
    cols[11] = False
    assert bool(same(got[keep][:, cols], clean[keep][:, cols]).all())
    assert not bool(got[5, cols].isfinite().any())


@pytest.mark.parametrize("M,N,K", [(8, 4096, 4096), (700, 1500, 2000)])
def test_linear_same_call_same_bits(M, N, K):
    x, sx, w, sw = linear_problem(M, N, K)
    assert bool(same(run_linear(x, sx, w, sw), run_linear(x, sx, w, sw)).all())


def test_linear_of_no_rows():
    x, sx, w, sw = linear_problem(1, 64, 64)
    p = F.make_scaled_gemm_params(M=0, N=64, K=64)
    ws, y = F.alloc_scaled_gemm_workspace(p), torch.full((1, 64), 3.0, device="cuda", dtype=torch.bfloat16)
    F.fdpp_scaled_gemm(x, sx, w, sw, p, ws, y)
    assert F.fdpp_read_error(ws) == 0 and bool((y == 3.0).all())


def test_norm_into_linear_on_another_stream_and_in_a_graph():
    """A norm's bytes and scales feed the linear layer as they are, K not a multiple of 128; captured, then
    replayed on new inputs."""
    T, dim, N = 37, 272, 500
    gen = torch.Generator("cuda").manual_seed(1)
    x = torch.randn(T, dim, generator=gen, device="cuda").bfloat16()
    res = torch.randn(T, dim, generator=gen, device="cuda").bfloat16()
    _, _, w, sw = linear_problem(1, N, dim, 2)
    pn = F.make_norm_params(num_tokens=T, dim=dim, dtype=F.FDPP_BF16, out_dtype=F.FDPP_E4M3)
    q, s = torch.empty(T, pn.out_stride, device="cuda", dtype=torch.uint8), torch.empty(T, pn.scale_stride, device="cuda")
    pg = F.make_scaled_gemm_params(M=T, N=N, K=dim, out_dtype=F.FDPP_F32, x_stride=pn.out_stride, x_scale_stride=pn.scale_stride)
    ws, y = F.alloc_scaled_gemm_workspace(pg), torch.empty(T, N, device="cuda")
    stream = torch.cuda.Stream()

    def step():
        F.fdpp_rms_norm(x, res, None, pn, q, s, None)
        F.fdpp_scaled_gemm(q, s, w, sw, pg, ws, y)

    def check():
        _, normed = norm_reference(x, res, None, 1e-6, 0.0)
        each = s.double().repeat_interleave(128, 1)[:, :dim]
        wd = e4m3(w).double() * sw.double().repeat_interleave(128, 0)[:N].repeat_interleave(128, 1)[:, :dim]
        want = (e4m3(q).double() * each) @ wd.T
        size = (e4m3(q).double() * each).abs() @ wd.abs().T
        assert bool(((y.double() - want).abs() <= 2.0 ** -24 * want.abs() + 2.0 ** -15 * size).all())
        # and the whole chain: each normed value is off by its rounding to e4m3
        off = ((2.0 ** -4 + 2.0 ** -16) * normed.abs() + 2.0 ** -10 * each) @ wd.abs().T
        assert bool(((y.double() - normed @ wd.T).abs() <= off + 2.0 ** -15 * size).all())

    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        step()
    stream.synchronize()
    check()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        step()
    x.copy_(torch.randn(T, dim, generator=gen, device="cuda"))
    graph.replay()
    torch.cuda.synchronize()
    check()
    assert F.fdpp_read_error(ws) == 0


def test_linear_two_streams_with_one_workspace():
    """The workspace holds the error word alone: calls at once may share it."""
    problems = [linear_problem(M, 1500, 2048, seed) for M, seed in ((8, 1), (300, 2))]
    want = [run_linear(*p, out="f32") for p in problems]
    params = [F.make_scaled_gemm_params(M=p[0].shape[0], N=1500, K=2048, out_dtype=F.FDPP_F32) for p in problems]
    ws = F.alloc_scaled_gemm_workspace(params[0])
    y = [torch.zeros_like(w) for w in want]
    streams = [torch.cuda.Stream() for _ in problems]
    torch.cuda.synchronize()
    for _ in range(20):
        for p, q, o, s in zip(problems, params, y, streams):
            F.fdpp_scaled_gemm(*p, q, ws, o, stream=s)
    assert F.fdpp_read_error(ws) == 0
    assert all(bool(same(a, b).all()) for a, b in zip(y, want))


@pytest.mark.parametrize("M,N", [(70000, 32768), (40, (1 << 31) // 40 + 128)])
def test_linear_outputs_beyond_32_bits(M, N):
    x, sx, w, sw = linear_problem(M, N, 16)
    y = torch.full((M, N), 7.0, dtype=torch.bfloat16, device="cuda")
    p = F.make_scaled_gemm_params(M=M, N=N, K=16)
    ws = F.alloc_scaled_gemm_workspace(p)
    F.fdpp_scaled_gemm(x, sx, w, sw, p, ws, y)
    assert F.fdpp_read_error(ws) == 0
    for rows in (slice(0, 3), slice(M - 3, M)):
        for cols in (slice(0, 256), slice(N // 256 * 256 - 256, N)):
            first = cols.start // 128
            want, size = linear_reference(x[rows], sx[rows], w[cols], sw[first:])
            got = y[rows, cols].double()
            assert torch.equal(got.isnan(), want.isnan())
            assert bool(((got - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -15 * size).nan_to_num(1).logical_or(want.isnan()).all())


def test_norm_of_more_than_32_bits_of_elements():
    T, dim = 70000, 32768
    x = torch.randn(T, 1, device="cuda").bfloat16().expand(T, dim).contiguous()
    x[:, ::3] *= -2
    p = F.make_norm_params(num_tokens=T, dim=dim, dtype=F.FDPP_BF16, out_dtype=F.FDPP_E4M3)
    out, scales = torch.zeros(T, dim, device="cuda", dtype=torch.uint8), torch.zeros(T, dim // 128, device="cuda")
    F.fdpp_rms_norm(x, None, None, p, out, scales)
    torch.cuda.synchronize()
    for rows in (slice(0, 5), slice(T - 5, T)):
        _, y = norm_reference(x[rows], None, None, 1e-6, 0.0)
        each = scales[rows].double().repeat_interleave(128, 1)
        got = e4m3(out[rows]).double() * each
        assert bool(((got - y).abs() <= (2.0 ** -4 + 2.0 ** -16) * y.abs() + 2.0 ** -10 * each).all())


@pytest.mark.parametrize("dtype", [F.FDPP_F32, F.FDPP_E4M3])
def test_empty_tensors(dtype):
    """Tensors of no rows, whose address is NULL, through both calls."""
    t = torch.bfloat16 if dtype == F.FDPP_E4M3 else torch.float32
    x = torch.empty(0, 256, device="cuda", dtype=t)
    out = torch.empty(0, 256, device="cuda", dtype=torch.uint8 if dtype == F.FDPP_E4M3 else t)
    scales = torch.empty(0, 2, device="cuda") if dtype == F.FDPP_E4M3 else None
    F.fdpp_rms_norm(x, None, None, F.make_norm_params(num_tokens=0, dim=256, dtype=F.FDPP_BF16 if dtype == F.FDPP_E4M3 else dtype,
                                                      out_dtype=dtype), out, scales)
    _, _, w, sw = linear_problem(1, 64, 256)
    p = F.make_scaled_gemm_params(M=0, N=64, K=256)
    ws = F.alloc_scaled_gemm_workspace(p)
    e = torch.empty(0, 256, device="cuda", dtype=torch.uint8)
    F.fdpp_scaled_gemm(e, torch.empty(0, 2, device="cuda"), w, sw, p, ws, torch.empty(0, 64, device="cuda", dtype=torch.bfloat16))
    assert F.fdpp_read_error(ws) == 0
