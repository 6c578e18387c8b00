"""The RMS norm and the 8-bit linear layer without a GPU: argument errors come back before any CUDA call
with the documented status, and the binding's structures have the header's fields."""
import os
import re

import pytest

import split_kv_async_gb300 as F
from fdpp_harness import no_fake_pointer_calls_on_a_gpu

HEADER = os.path.join(os.path.dirname(os.path.dirname(__file__)), "include", "fdpp_linear.h")
FAKE = 1 << 20                 # an aligned address that nothing dereferences


@pytest.mark.parametrize("struct", ["fdpp_norm_params", "fdpp_scaled_gemm_params"])
def test_structures_match_the_header(struct):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    body = re.search(r"typedef struct %s \{(.*?)\} %s;" % (struct, struct), text, re.S).group(1)
    assert re.findall(r"\b(\w+)\s*[;,]", body) == [n for n, _ in getattr(F, struct)._fields_]


def test_constants_match_the_header():
    found = re.findall(r"#define (FDPP_[A-Z0-9_]+) (\d+)", open(HEADER).read())
    assert len(found) == 3
    for name, value in found:
        assert getattr(F, name) == int(value), name


# ---- RMS norm ----------------------------------------------------------------------------------

def _norm(x=FAKE, residual=2 * FAKE, weight=3 * FAKE, out=4 * FAKE, scales=None, total=5 * FAKE, **kw):
    no_fake_pointer_calls_on_a_gpu()
    p = F.make_norm_params(**{**dict(num_tokens=3, dim=256, dtype=F.FDPP_BF16), **kw})
    return F.lib.fdpp_rms_norm(x, residual, weight, p, out, scales, total, None)


E4M3 = dict(out_dtype=F.FDPP_E4M3, scales=6 * FAKE)


@pytest.mark.parametrize("kw", [
    dict(num_tokens=-1), dict(dim=0), dict(dim=12), dict(dtype=F.FDPP_E4M3), dict(dtype=7), dict(out_dtype=F.FDPP_F32),
    dict(eps=-1.0), dict(eps=float("inf")), dict(eps=float("nan")), dict(weight_offset=float("nan")), dict(x_stride=248),
    dict(x_stride=260), dict(residual_stride=0), dict(out_stride=255), dict(sum_stride=8), dict(x=None), dict(out=None),
    dict(x=FAKE + 8), dict(residual=FAKE + 4), dict(weight=FAKE + 2), dict(out=FAKE + 8), dict(total=FAKE + 8),
    dict(scales=6 * FAKE), dict(out_dtype=F.FDPP_E4M3), {**E4M3, "scales": 6 * FAKE + 2}, {**E4M3, "scale_stride": 1},
    {**E4M3, "dim": 264, "out_stride": 268}, {**E4M3, "out": FAKE}, dict(out=FAKE, x_stride=512), dict(total=FAKE, x_stride=512),
    dict(total=2 * FAKE, sum_stride=512), dict(out=2 * FAKE), dict(out=5 * FAKE), dict(x_stride=1 << 50),
])
def test_norm_rejects(kw):
    assert _norm(**kw) == F.FDPP_ERR_INVALID_ARG
    assert F.fdpp_last_error()


def test_norm_rejects_rows_beyond_registers():
    assert _norm(dim=F.FDPP_NORM_MAX_DIM + 8) == F.FDPP_ERR_UNSUPPORTED


@pytest.mark.parametrize("kw", [
    {}, dict(residual=None, weight=None, total=None), dict(out=FAKE), dict(total=FAKE), dict(total=2 * FAKE), dict(num_tokens=0),
    E4M3, {**E4M3, "dim": 264}, {**E4M3, "dtype": F.FDPP_F32}, dict(x_stride=264, residual_stride=512, out_stride=304, sum_stride=256),
    dict(dim=F.FDPP_NORM_MAX_DIM),
])
def test_norm_calls_that_pass_the_checks(kw):
    assert _norm(**kw) == F.FDPP_ERR_CUDA          # as far as the device query


# ---- linear layer ------------------------------------------------------------------------------

def _gemm(x=FAKE, sx=2 * FAKE, w=3 * FAKE, sw=4 * FAKE, ws=1 << 28, ws_bytes=256, y=5 * FAKE, **kw):
    no_fake_pointer_calls_on_a_gpu()
    p = F.make_scaled_gemm_params(**{**dict(M=8, N=100, K=272), **kw})
    return F.lib.fdpp_scaled_gemm(x, sx, w, sw, p, ws, ws_bytes, y, None)


BAD_SHAPES = [dict(M=-1), dict(N=0), dict(K=0), dict(K=24), dict(N=(1 << 30) + 1), dict(out_dtype=F.FDPP_E4M3), dict(out_dtype=5),
              dict(x_stride=256), dict(x_stride=280), dict(w_stride=0), dict(w_stride=1 << 40), dict(y_stride=99),
              dict(x_scale_stride=2), dict(split_k=-1), dict(split_k=4), dict(K=16384, split_k=9)]


@pytest.mark.parametrize("kw", BAD_SHAPES)
def test_gemm_rejects_bad_shapes(kw):
    p = F.make_scaled_gemm_params(**{**dict(M=8, N=100, K=272), **kw})
    assert F.fdpp_scaled_gemm_workspace_size(p) == 0
    with pytest.raises(F.FdppError):
        F.alloc_scaled_gemm_workspace(p, device="cpu")
    assert _gemm(**kw) == F.FDPP_ERR_INVALID_ARG
    assert F.fdpp_last_error()


@pytest.mark.parametrize("kw", [dict(x=None), dict(sx=None), dict(w=None), dict(sw=None), dict(y=None), dict(x=FAKE + 8),
                                dict(w=FAKE + 8), dict(sx=FAKE + 2), dict(sw=FAKE + 2), dict(y=FAKE + 1),
                                dict(y=FAKE + 2, out_dtype=F.FDPP_F32)])
def test_gemm_rejects_bad_pointers(kw):
    assert _gemm(**kw) == F.FDPP_ERR_INVALID_ARG


def test_gemm_workspace_errors_and_calls_that_pass():
    assert F.fdpp_scaled_gemm_workspace_size(F.make_scaled_gemm_params(M=8, N=100, K=272)) == 256
    assert _gemm(ws=None) == F.FDPP_ERR_WORKSPACE
    assert _gemm(ws=(1 << 28) + 128) == F.FDPP_ERR_WORKSPACE
    assert _gemm(ws_bytes=255) == F.FDPP_ERR_WORKSPACE
    for kw in ({}, dict(M=0), dict(M=5000), dict(split_k=3), dict(y=FAKE + 2), dict(y_stride=1001), dict(x_stride=1024, w_stride=288),
               dict(K=16)):
        assert _gemm(**kw) == F.FDPP_ERR_CUDA      # as far as the device query


def test_calls_on_empty_tensors_pass_without_addresses():
    assert _norm(num_tokens=0, x=None, residual=None, out=None, total=None) == F.FDPP_ERR_CUDA
    assert _norm(num_tokens=0, x=None, residual=None, out=None, total=None, out_dtype=F.FDPP_E4M3) == F.FDPP_ERR_CUDA
    assert _gemm(M=0, x=None, sx=None, y=None) == F.FDPP_ERR_CUDA
    assert _gemm(M=0, w=None) == F.FDPP_ERR_INVALID_ARG
