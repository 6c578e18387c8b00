"""The block map, the rotary append and the rows attention without a GPU: argument errors come back
before any CUDA call with the documented status, sizes and the rotation's angles are right, and the
binding's structures have the headers' fields."""
import ctypes
import math
import os
import re

import numpy as np
import pytest

import rows_reference as R
import split_kv_async_gb300 as F
from fdpp_harness import no_fake_pointer_calls_on_a_gpu

INCLUDE = os.path.join(os.path.dirname(os.path.dirname(__file__)), "include")
FAKE = 1 << 20                 # an aligned address that nothing dereferences


@pytest.mark.parametrize("header,struct", [("fdpp_cache.h", "fdpp_block_params"), ("fdpp_cache.h", "fdpp_rope_params"),
                                           ("fdpp_rows.h", "fdpp_rows_params")])
def test_structures_match_the_headers(header, struct):
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(INCLUDE, header)).read(), flags=re.S)
    body = re.search(r"typedef struct %s \{(.*?)\} %s;" % (struct, struct), text, re.S).group(1)
    names = re.findall(r"\b(\w+)\s*[;,]", body)
    assert names == [n for n, _ in getattr(F, struct)._fields_]


def test_constants_match_the_headers():
    text = open(os.path.join(INCLUDE, "fdpp_cache.h")).read() + open(os.path.join(INCLUDE, "fdpp_rows.h")).read()
    for name, value in re.findall(r"\b(FDPP_(?:ERRBIT|ROPE)_\w+) = (\d+)", text):
        assert getattr(F, name) == int(value), name
    assert F.FDPP_ROWS_MAX_GROUP == int(re.search(r"#define FDPP_ROWS_MAX_GROUP (\d+)", text).group(1))
    assert F.FDPP_ROWS_MAX_SOFTCAP == float(re.search(r"#define FDPP_ROWS_MAX_SOFTCAP ([\d.]+)f", text).group(1))


# ---- block map ---------------------------------------------------------------------------------

def _block(**kw):
    return F.make_block_params(**{**dict(batch=4, block_size=16, max_blocks_per_seq=8, num_kv_blocks=32, max_tokens=64), **kw})


def _map(p, ws=1 << 28, ws_bytes=1 << 20, **kw):
    no_fake_pointer_calls_on_a_gpu()
    names = ("held", "want", "pool_in", "table", "queue", "lens", "pool_out", "cu", "seq", "pos", "slots")
    a = {n: FAKE * (i + 1) for i, n in enumerate(names)}
    a.update(kw)
    v = [a[n] for n in names]
    return F.lib.fdpp_block_map(v[0], v[1], v[2], p, *v[3:], ws, ws_bytes, None)


@pytest.mark.parametrize("kw", [dict(batch=0), dict(block_size=8), dict(block_size=24), dict(block_size=512),
                                dict(max_blocks_per_seq=0), dict(num_kv_blocks=0), dict(max_tokens=-1),
                                dict(batch=1 << 16, max_blocks_per_seq=1 << 16)])
def test_block_map_rejects_bad_parameters(kw):
    p = _block(**kw)
    assert F.fdpp_block_map_workspace_size(p) == 0
    with pytest.raises(F.FdppError):
        F.alloc_block_workspace(p, device="cpu")
    assert _map(p) == F.FDPP_ERR_INVALID_ARG
    assert F.fdpp_last_error()


@pytest.mark.parametrize("kw", [dict(held=None), dict(want=None), dict(pool_in=None), dict(table=None), dict(queue=None),
                                dict(lens=None), dict(pool_out=None), dict(cu=None), dict(seq=None), dict(pos=None),
                                dict(slots=None), dict(held=FAKE + 2), dict(slots=FAKE + 4), dict(lens=2 * FAKE)])
def test_block_map_rejects_bad_pointers(kw):
    # (lens = want: the wanted lengths would be overwritten while they are read)
    assert _map(_block(), **kw) == F.FDPP_ERR_INVALID_ARG


def test_block_map_workspace_errors_and_calls_that_pass():
    p = _block()
    n = F.fdpp_block_map_workspace_size(p)
    assert 256 < n <= 1024
    assert _map(p, ws=None) == F.FDPP_ERR_WORKSPACE
    assert _map(p, ws=(1 << 28) + 128) == F.FDPP_ERR_WORKSPACE
    assert _map(p, ws_bytes=300) == F.FDPP_ERR_WORKSPACE
    # in place, and without rows: accepted as far as the device query
    assert _map(p, ws_bytes=n, lens=FAKE, pool_out=3 * FAKE) == F.FDPP_ERR_CUDA
    assert _map(_block(max_tokens=0), ws_bytes=n, seq=None, pos=None, slots=None) == F.FDPP_ERR_CUDA


# ---- rotary append -----------------------------------------------------------------------------

@pytest.mark.parametrize("rot", [16, 64, 96, 128])
@pytest.mark.parametrize("kind,kw", [
    ("plain", {}), ("linear", dict(factor=4.0)), ("ntk", dict(factor=2.5)), ("parts", dict(factor=8.0, context=4096)),
    ("parts", dict(factor=32.0, context=8192, low=2.0, high=5.0)),
])
def test_rope_table_holds_the_angles(rot, kind, kw):
    scaling = dict(plain=F.FDPP_ROPE_PLAIN, linear=F.FDPP_ROPE_LINEAR, ntk=F.FDPP_ROPE_NTK, parts=F.FDPP_ROPE_PARTS)[kind]
    t = F.fdpp_rope_table(rot, 500000.0, scaling=scaling, factor=kw.get("factor", 1.0), context=kw.get("context", 0),
                          low_turns=kw.get("low", 1.0), high_turns=kw.get("high", 32.0))
    theta = R.rope_theta(rot, 500000.0, kind, **kw)
    turns = t[:, 0].astype(np.float64) + t[:, 1].astype(np.float64)
    # two floats: 2^-49 of the angle; the powers are computed in 64 bits on both sides, a few 2^-52 apart
    assert np.all(np.abs(turns * 2 * math.pi - theta) <= (2.0 ** -49 + 2.0 ** -48) * theta)
    assert np.all(np.abs(t[:, 1]) <= 2.0 ** -24 * np.abs(t[:, 0]))


@pytest.mark.parametrize("kw", [dict(rot_dim=0), dict(rot_dim=24), dict(rot_dim=144), dict(base=1.0), dict(base=float("nan")),
                                dict(scaling=9), dict(scaling=1, factor=0.5), dict(scaling=2, factor=float("inf")),
                                dict(scaling=3, factor=2.0, context=0), dict(scaling=3, factor=2.0, context=64, low_turns=3.0, high_turns=3.0)])
def test_rope_table_rejects(kw):
    kw = {**dict(rot_dim=64, base=10000.0), **kw}
    with pytest.raises(F.FdppError) as e:
        F.fdpp_rope_table(kw.pop("rot_dim"), kw.pop("base"), **kw)
    assert e.value.status == F.FDPP_ERR_INVALID_ARG


def _rope(**kw):
    return F.make_rope_params(**{**dict(num_tokens=5, num_q_heads=8, num_kv_heads=2, head_dim=128, rot_dim=128,
                                        dtype=F.FDPP_BF16, num_slots=64), **kw})


def _append(p, ws=1 << 28, ws_bytes=256, **kw):
    no_fake_pointer_calls_on_a_gpu()
    names = ("q", "k", "v", "pos", "slots", "table", "q_out", "k_cache", "v_cache")
    a = {n: FAKE * (i + 1) for i, n in enumerate(names)}
    a.update(kw)
    v = [a[n] for n in names]
    return F.lib.fdpp_rope_append(*v[:6], p, *v[6:], ws, ws_bytes, None)


@pytest.mark.parametrize("kw,status", [
    (dict(num_tokens=-1), 1), (dict(num_q_heads=0), 1), (dict(num_kv_heads=0), 1), (dict(head_dim=96), 2), (dict(dtype=5), 1),
    (dict(rot_dim=0), 1), (dict(rot_dim=40), 1), (dict(head_dim=64), 1),          # rot_dim 128 > 64
    (dict(interleaved=2), 1), (dict(magnitude=float("nan")), 1), (dict(num_slots=-1), 1), (dict(num_slots=1 << 60), 1),
    (dict(q_stride=1000), 1), (dict(q_stride=1028), 1), (dict(k_stride=128), 1), (dict(v_stride=260), 1),
])
def test_rope_append_rejects_bad_parameters(kw, status):
    assert _append(_rope(**kw)) == status
    assert F.fdpp_last_error()


@pytest.mark.parametrize("kw", [dict(q=None), dict(k=None), dict(v=None), dict(pos=None), dict(slots=None), dict(table=None),
                                dict(q_out=None), dict(k_cache=None), dict(v_cache=None), dict(q=FAKE + 8),
                                dict(k_cache=FAKE + 8), dict(pos=FAKE + 2), dict(slots=FAKE + 4), dict(table=FAKE + 4)])
def test_rope_append_rejects_bad_pointers(kw):
    assert _append(_rope(), **kw) == F.FDPP_ERR_INVALID_ARG


def test_rope_append_in_place_and_workspace():
    assert _append(_rope(q_stride=2048), q_out=FAKE) == F.FDPP_ERR_INVALID_ARG     # q itself, with another stride
    assert _append(_rope(), q_out=FAKE) == F.FDPP_ERR_CUDA
    assert _append(_rope(), ws=None) == F.FDPP_ERR_WORKSPACE
    assert _append(_rope(), ws=(1 << 28) + 16) == F.FDPP_ERR_WORKSPACE
    assert _append(_rope(), ws_bytes=255) == F.FDPP_ERR_WORKSPACE
    # fp32 rows may be multiples of 4 elements apart
    assert _append(_rope(dtype=F.FDPP_F32, q_stride=1028)) == F.FDPP_ERR_CUDA


# ---- rows attention ----------------------------------------------------------------------------

def _rows(**kw):
    return F.make_rows_params(**{**dict(batch=4, num_q_heads=8, num_kv_heads=2, head_dim=128, dtype=F.FDPP_BF16,
                                        num_tokens=12, max_seq_len=1000, scale=0.1), **kw})


def _attend(p, ws=1 << 32, ws_bytes=1 << 32, prefix=False, **kw):
    no_fake_pointer_calls_on_a_gpu()
    a = dict(q=FAKE, k=FAKE, v=FAKE, table=None, lens=FAKE, cu=FAKE, out=FAKE, pk=FAKE, pv=FAKE, pt=None, pl=FAKE)
    a.update(kw)
    if prefix:
        return F.lib.fdpp_prefix_attn(a["q"], a["pk"], a["pv"], a["pt"], a["pl"], a["k"], a["v"], a["table"], a["lens"],
                                      a["cu"], p, ws, ws_bytes, a["out"], None)
    return F.lib.fdpp_rows_attn(a["q"], a["k"], a["v"], a["table"], a["lens"], a["cu"], p, ws, ws_bytes, a["out"], None)


@pytest.mark.parametrize("field,value,status", [
    ("batch", 0, 1), ("num_q_heads", 0, 1), ("num_q_heads", 9, 1), ("num_kv_heads", 0, 1), ("head_dim", 96, 2), ("dtype", 3, 1),
    ("num_q_heads", 2 * 129, 2), ("num_tokens", 0, 1), ("max_seq_len", 0, 1), ("max_seq_len", (1 << 30) + 1, 1),
    ("max_prefix_len", -1, 1), ("scale", 0.0, 1), ("scale", float("inf"), 1), ("softcap", -1.0, 1),
    ("softcap", float("nan"), 1), ("kernel", 7, 1), ("slopes", 2, 1), ("key_begin", 1, 1), ("key_end", 3, 1),
    ("num_tokens", 1 << 28, 1), ("softcap", 4097.0, 2), ("softcap", 1e-40, 1),
])
def test_rows_reject_bad_parameters(field, value, status):
    p = _rows()
    setattr(p, field, value)
    n = ctypes.c_size_t(0)
    assert F.lib.fdpp_rows_workspace_size(ctypes.byref(p), ctypes.byref(n)) == status
    assert F.fdpp_last_error()
    for prefix in (False, True):
        assert _attend(p, prefix=prefix) == status


def test_rows_tensor_kernel_needs_bf16():
    p = _rows(dtype=F.FDPP_F32, kernel=F.FDPP_KERNEL_TENSOR)
    assert _attend(p) == F.FDPP_ERR_UNSUPPORTED


@pytest.mark.parametrize("kw", [dict(q=None), dict(k=None), dict(v=None), dict(lens=None), dict(out=None), dict(q=FAKE + 8),
                                dict(out=FAKE + 2), dict(lens=FAKE + 1), dict(cu=FAKE + 2), dict(k=FAKE + 4)])
def test_rows_reject_bad_pointers(kw):
    assert _attend(_rows(), **kw) == F.FDPP_ERR_INVALID_ARG


def test_rows_without_cu_tokens_need_whole_shares():
    assert _attend(_rows(num_tokens=13), cu=None) == F.FDPP_ERR_INVALID_ARG
    assert _attend(_rows(num_tokens=12), cu=None) == F.FDPP_ERR_CUDA


def test_rows_paged_contract():
    paged = dict(block_size=16, max_blocks_per_seq=64, num_kv_blocks=10)
    for bad in (dict(block_size=20), dict(block_size=512), dict(max_blocks_per_seq=0), dict(max_blocks_per_seq=62),
                dict(num_kv_blocks=0)):
        assert _attend(_rows(**{**paged, **bad}), table=FAKE) == F.FDPP_ERR_INVALID_ARG
    assert _attend(_rows(**paged), table=FAKE) == F.FDPP_ERR_CUDA
    assert _attend(_rows(**paged), table=FAKE + 2) == F.FDPP_ERR_INVALID_ARG


def test_prefix_contract():
    paged = dict(block_size=16, max_blocks_per_seq=64, num_kv_blocks=10)
    assert _attend(_rows(), prefix=True) == F.FDPP_ERR_INVALID_ARG                                # max_prefix_len 0
    p = _rows(max_prefix_len=100)
    assert _attend(p, prefix=True) == F.FDPP_ERR_CUDA
    assert _attend(p, prefix=True, pl=None) == F.FDPP_ERR_INVALID_ARG
    assert _attend(p, prefix=True, pk=None) == F.FDPP_ERR_INVALID_ARG
    assert _attend(p, prefix=True, pv=FAKE + 8) == F.FDPP_ERR_INVALID_ARG
    assert _attend(p, prefix=True, pt=FAKE) == F.FDPP_ERR_INVALID_ARG                             # contiguous takes none
    p = _rows(max_prefix_len=100, **paged)
    assert _attend(p, prefix=True, table=FAKE, pk=None, pv=None, pt=FAKE) == F.FDPP_ERR_CUDA
    assert _attend(p, prefix=True, table=FAKE, pk=None, pv=None, pt=None) == F.FDPP_ERR_INVALID_ARG
    assert _attend(p, prefix=True, table=FAKE, pt=FAKE) == F.FDPP_ERR_INVALID_ARG                 # and no prefix_k, prefix_v


def test_rows_workspace():
    p = _rows()
    n = F.fdpp_rows_workspace_size(p)
    assert n % 256 == 0
    assert _attend(p, ws=None) == F.FDPP_ERR_WORKSPACE
    assert _attend(p, ws=(1 << 32) + 128) == F.FDPP_ERR_WORKSPACE
    assert _attend(p, ws_bytes=n - 1) == F.FDPP_ERR_WORKSPACE
    assert "needed" in F.fdpp_last_error()
    # a prefix adds two partials of fp32 for each row, and row tiles over all rows
    more = F.fdpp_rows_workspace_size(_rows(max_prefix_len=10)) - n
    assert 2 * 12 * 8 * (128 + 2) * 4 <= more <= 2 * 12 * 8 * (128 + 2) * 4 + 4096
    # fp32: one partial for each split of a row, and none where the rows alone fill the GPU
    few = F.fdpp_rows_workspace_size(_rows(dtype=F.FDPP_F32, batch=1, num_tokens=1, max_seq_len=4096))
    many = F.fdpp_rows_workspace_size(_rows(dtype=F.FDPP_F32, num_tokens=1000))
    assert few > 8 * 32 * 130 * 4 and many < 8192


def test_read_error_rejects_null():
    assert F.lib.fdpp_read_error(None, None) == F.FDPP_ERR_INVALID_ARG


def test_rows_softcap_limit_is_the_tensor_kernels():
    big = 8.0 * F.FDPP_ROWS_MAX_SOFTCAP
    assert F.fdpp_rows_workspace_size(_rows(softcap=F.FDPP_ROWS_MAX_SOFTCAP)) > 0
    assert F.fdpp_rows_workspace_size(_rows(softcap=big, dtype=F.FDPP_F32)) > 0
    assert F.fdpp_rows_workspace_size(_rows(softcap=big, kernel=F.FDPP_KERNEL_SIMT)) > 0
    with pytest.raises(F.FdppError) as e:
        F.fdpp_rows_workspace_size(_rows(softcap=big))
    assert e.value.status == F.FDPP_ERR_UNSUPPORTED


@pytest.mark.parametrize("field", ["scale", "softcap"])
def test_rows_reject_factors_that_overflow(field):
    # the kernels work in units of log2: a factor times log2(e) beyond fp32 would make NaN of a score of 0
    for dtype in (F.FDPP_F32, F.FDPP_BF16):
        p = _rows(dtype=dtype, **{"scale": 0.1, field: 3e38})
        n = ctypes.c_size_t(0)
        assert F.lib.fdpp_rows_workspace_size(ctypes.byref(p), ctypes.byref(n)) == F.FDPP_ERR_INVALID_ARG
        assert _attend(p) == F.FDPP_ERR_INVALID_ARG
    assert F.fdpp_rows_workspace_size(_rows(**{"scale": 0.1, "dtype": F.FDPP_F32, field: 2e38})) > 0
