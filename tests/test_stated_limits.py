"""Limits that the headers state, on both sides, without a GPU."""
import os
import re

import pytest

import split_kv_async_gb300 as F
from fdpp_harness import no_fake_pointer_calls_on_a_gpu

FAKE = 1 << 20                 # an aligned address that nothing dereferences
INCLUDE = os.path.join(os.path.dirname(os.path.dirname(__file__)), "include")


@pytest.mark.parametrize("kw,good", [
    (dict(batch=1), True), (dict(batch=65535), True), (dict(batch=65536), False), (dict(batch=0), False),
    (dict(row_bytes=16), True), (dict(row_bytes=1 << 24), True), (dict(row_bytes=(1 << 24) + 16), False), (dict(row_bytes=0), False),
])
def test_commit(kw, good):
    no_fake_pointer_calls_on_a_gpu()
    p = F.make_commit_params(**{**dict(batch=2, num_tokens=10, max_seq_len=100, row_bytes=256), **kw})
    assert bool(F.lib.fdpp_commit_workspace_size(p)) == good
    args = [FAKE * (i + 1) for i in range(5)]
    status = F.lib.fdpp_tree_commit(*args, None, None, 0, p, 1 << 28, 256, 6 * FAKE, 7 * FAKE, 8 * FAKE, 9 * FAKE, None)
    assert status == (F.FDPP_ERR_CUDA if good else F.FDPP_ERR_INVALID_ARG)       # (as far as the device query)
    text = open(os.path.join(INCLUDE, "fdpp_tree.h")).read()
    assert re.search(r"int batch;\s+/\* B sequences: 1 \.\. 65535 \*/", text) and "multiple of 16, at most 2^24" in text
