"""Tree attention and the tree's commit without a GPU: argument errors come back before any CUDA call with
the documented status, and the binding's structure has the header's fields."""
import ctypes
import os
import re

import pytest

import split_kv_async_gb300 as F
from fdpp_harness import no_fake_pointer_calls_on_a_gpu

HEADER = os.path.join(os.path.dirname(os.path.dirname(__file__)), "include", "fdpp_tree.h")
FAKE = 1 << 20                 # an aligned address that nothing dereferences


def test_structure_and_constants_match_the_header():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    body = re.search(r"typedef struct fdpp_commit_params \{(.*?)\} fdpp_commit_params;", text, re.S).group(1)
    assert re.findall(r"\b(\w+)\s*[;,]", body) == [n for n, _ in F.fdpp_commit_params._fields_]
    found = re.findall(r"\b(FDPP_\w+)(?: =)? (\d+)", text)
    assert len(found) == 3
    for name, value in found:
        assert getattr(F, name) == int(value), name


# ---- tree attention ----------------------------------------------------------------------------

def _params(**kw):
    return F.make_rows_params(**{**dict(batch=2, num_q_heads=8, num_kv_heads=2, head_dim=128, dtype=F.FDPP_BF16, num_tokens=10,
                                        max_seq_len=100, scale=0.1), **kw})


def _tree(p, q=FAKE, k=FAKE, v=FAKE, table=None, lens=FAKE, cu=FAKE, parents=FAKE, ws=1 << 28, ws_bytes=1 << 40, out=FAKE):
    no_fake_pointer_calls_on_a_gpu()
    return F.lib.fdpp_tree_attn(q, k, v, table, lens, cu, parents, p, ws, ws_bytes, out, None)


def test_tree_rejects_masks_that_the_tree_replaces():
    p = _params()
    p.key_end = FAKE
    assert _tree(p) == F.FDPP_ERR_INVALID_ARG
    p = _params()
    p.slopes = FAKE
    assert _tree(p) == F.FDPP_ERR_UNSUPPORTED
    with pytest.raises(F.FdppError):
        F.fdpp_tree_workspace_size(p)


@pytest.mark.parametrize("kw", [dict(parents=None), dict(parents=FAKE + 2), dict(q=None), dict(out=FAKE + 8), dict(lens=None)])
def test_tree_rejects_bad_pointers(kw):
    assert _tree(_params(), **kw) == F.FDPP_ERR_INVALID_ARG


@pytest.mark.parametrize("kw", [dict(batch=0), dict(num_tokens=0), dict(scale=0.0), dict(dtype=F.FDPP_E4M3), dict(softcap=-1.0)])
def test_tree_rejects_bad_parameters(kw):
    assert _tree(_params(**kw)) == F.FDPP_ERR_INVALID_ARG


@pytest.mark.parametrize("dtype", [F.FDPP_BF16, F.FDPP_F32])
def test_tree_workspace(dtype):
    p = _params(dtype=dtype)
    n = F.fdpp_tree_workspace_size(p)
    p.kernel = F.FDPP_KERNEL_SIMT
    assert n == F.fdpp_tree_workspace_size(p)                          # (few keys: the CUDA cores by themselves)
    p.max_seq_len = 100000
    if dtype == F.FDPP_BF16:
        p.kernel = F.FDPP_KERNEL_TENSOR
    large = F.fdpp_tree_workspace_size(p)
    # (the tensor kernel keeps each token's line of ancestors and descendants)
    assert large >= F.fdpp_rows_workspace_size(p) + (10 * 4 * (1 + 2 * F.FDPP_TREE_MAX_TOKENS // 32) if dtype == F.FDPP_BF16 else 0)
    p.kernel = F.FDPP_KERNEL_AUTO
    assert F.fdpp_tree_workspace_size(p) == large
    p.max_seq_len = 100
    assert _tree(p, ws_bytes=n - 1) == F.FDPP_ERR_WORKSPACE
    assert _tree(p, ws=None) == F.FDPP_ERR_WORKSPACE
    assert _tree(p, ws_bytes=n) == F.FDPP_ERR_CUDA                     # as far as the device query
    p.key_begin = FAKE
    assert _tree(p, cu=None, ws_bytes=n) == F.FDPP_ERR_CUDA


# ---- commit ------------------------------------------------------------------------------------

def _commit(parents=FAKE, tokens=2 * FAKE, choices=3 * FAKE, lens=4 * FAKE, cu=5 * FAKE, table=None, caches=(FAKE, 2 * FAKE),
            ws=1 << 28, ws_bytes=256, new_lens=6 * FAKE, accepted=7 * FAKE, path=8 * FAKE, chosen=9 * FAKE, count=None, **kw):
    no_fake_pointer_calls_on_a_gpu()
    p = F.make_commit_params(**{**dict(batch=2, num_tokens=10, max_seq_len=100, row_bytes=256), **kw})
    array = None if caches is None else (ctypes.c_void_p * max(1, len(caches)))(*caches)
    return F.lib.fdpp_tree_commit(parents, tokens, choices, lens, cu, table, array, len(caches or ()) if count is None else count, p,
                                  ws, ws_bytes, new_lens, accepted, path, chosen, None)


PAGED = dict(table=FAKE, block_size=16, max_blocks_per_seq=8, num_kv_blocks=20)


@pytest.mark.parametrize("kw", [
    dict(batch=0), dict(batch=65536), dict(num_tokens=-1), dict(max_seq_len=0), dict(row_bytes=0), dict(row_bytes=24),
    dict(row_bytes=1 << 25), dict(cu=None, num_tokens=11), dict(parents=None), dict(tokens=None), dict(choices=None), dict(lens=None),
    dict(new_lens=None), dict(accepted=None), dict(path=None), dict(chosen=None), dict(parents=FAKE + 2), dict(chosen=9 * FAKE + 1),
    dict(new_lens=4 * FAKE), dict(accepted=4 * FAKE), dict(accepted=6 * FAKE), dict(path=9 * FAKE), dict(path=FAKE),
    dict(chosen=3 * FAKE), dict(caches=None, count=1), dict(count=-1), dict(caches=[FAKE * (i + 1) for i in range(257)]),
    dict(caches=(FAKE, None)), dict(caches=(FAKE, 2 * FAKE + 8)), dict(caches=(FAKE, FAKE)), dict(caches=(3 * FAKE, FAKE, 2 * FAKE, FAKE)),
    {**PAGED, "block_size": 8}, {**PAGED, "block_size": 48}, {**PAGED, "max_blocks_per_seq": 0}, {**PAGED, "num_kv_blocks": 0},
    {**PAGED, "max_seq_len": 129},
])
def test_commit_rejects(kw):
    assert _commit(**kw) == F.FDPP_ERR_INVALID_ARG
    assert F.fdpp_last_error()


def test_commit_workspace_errors_and_calls_that_pass():
    assert _commit(ws=None) == F.FDPP_ERR_WORKSPACE
    assert _commit(ws=(1 << 28) + 128) == F.FDPP_ERR_WORKSPACE
    assert _commit(ws_bytes=255) == F.FDPP_ERR_WORKSPACE
    with pytest.raises(F.FdppError):
        F.alloc_commit_workspace(F.make_commit_params(batch=1, num_tokens=1, max_seq_len=1, row_bytes=8), device="cpu")
    for kw in ({}, PAGED, dict(cu=None), dict(caches=()), dict(caches=None), dict(caches=(3 * FAKE, FAKE, 2 * FAKE)),
               dict(num_tokens=0, parents=None, tokens=None, choices=None, path=None, chosen=None)):
        assert _commit(**kw) == F.FDPP_ERR_CUDA    # as far as the device query
