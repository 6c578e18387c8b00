"""split_k of the 8-bit linear: what is asked for is followed, but by pairs of CTAs, whose tiles fill the GPU."""
import pytest
import torch

from test_linear_gpu import check_linear

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("split_k", [1, 3, 8])
def test_pairs_do_not_split(split_k):
    """1200 x 4000 takes pairs: the bits do not depend on split_k."""
    a, b = (check_linear(1200, 4000, 1168, "f32", split_k=s) for s in (0, split_k))
    assert bool(((a == b) | (a.isnan() & b.isnan())).all())


@pytest.mark.parametrize("M,N", [(8, 40000), (70, 40000), (300, 6000)])
@pytest.mark.parametrize("split_k", [1, 2, 8])
def test_tiles_beyond_one_for_an_sm_split_where_asked(M, N, split_k):
    got = check_linear(M, N, 1168, "f32", split_k=split_k)
    if split_k > 1:                       # another order of the sums: other bits somewhere in so many
        assert not torch.equal(got, check_linear(M, N, 1168, "f32", split_k=1))
