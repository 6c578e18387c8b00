"""The block map at lengths and row counts next to 2^31."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import split_kv_async_gb300 as F
    from rows_harness import ints

TOP = 2 ** 31 - 1


def _map(held, want, table, blocks, room, block, in_place=False):
    B, width = table.shape
    p = F.make_block_params(batch=B, block_size=block, max_blocks_per_seq=width, num_kv_blocks=blocks, max_tokens=room)
    d = dict(held=ints(held), pool=ints([0, blocks]), table=table, queue=ints(np.arange(blocks)), lens=ints([-1] * B),
             pool_out=ints([-1, -1]), cu=ints([-1] * (B + 1)), seq=torch.empty(room, dtype=torch.int32, device="cuda"),
             pos=torch.empty(room, dtype=torch.int32, device="cuda"), slots=torch.empty(room, dtype=torch.int64, device="cuda"))
    ws = F.alloc_block_workspace(p)
    F.fdpp_block_map(d["held"], ints(want), d["pool"], p, table, d["queue"], d["held"] if in_place else d["lens"],
                     d["pool"] if in_place else d["pool_out"], d["cu"], d["seq"], d["pos"], d["slots"], ws)
    assert F.fdpp_read_error(ws) == 0
    return d


@pytest.mark.parametrize("held,want", [(TOP - 3, TOP), (TOP - 300, TOP - 100), (TOP - 255, TOP)])
def test_lengths_next_to_the_limit(held, want):
    # a sequence of nearly 2^31 tokens in blocks of 256, its last block held already or taken now
    block, width = 256, 2 ** 23
    table = torch.zeros((1, width), dtype=torch.int32, device="cuda")
    table[0, (held - 1) // block] = 3
    new = -(-want // block) - -(-held // block)
    d = _map([held], [want], table, 5, 512, block)
    n = want - held
    pos = np.arange(held, want)
    last_held = (held - 1) // block
    blk = np.where(pos // block <= last_held, 3, 0)              # (the queue's first block is 0)
    assert new in (0, 1) and d["lens"].item() == want
    np.testing.assert_array_equal(d["pos"][:n].cpu().numpy(), pos)
    np.testing.assert_array_equal(d["slots"][:n].cpu().numpy(), blk * block + pos % block)
    assert (d["slots"][n:] == -1).all() and d["pool_out"].tolist() == [new, 5 - new]


@pytest.mark.parametrize("in_place", [False, True])
def test_rows_next_to_the_limit(in_place):
    # 2^31 - 1 token rows (34 GB), most of them padding
    table = torch.zeros((3, 4), dtype=torch.int32, device="cuda")
    d = _map([0, 5, 0], [20, 7, 0], table, 9, TOP, 16, in_place)
    assert d["cu"].tolist() == [0, 20, 22, 22]
    assert d["seq"][:23].tolist() == [0] * 20 + [1, 1, -1] and d["pos"][:23].tolist() == list(range(20)) + [5, 6, 0]
    assert d["slots"][:23].tolist() == list(range(20)) + [5, 6, -1]
    for x, pad in ((d["seq"], -1), (d["pos"], 0), (d["slots"], -1)):
        assert all(bool((x[i:i + 2 ** 28] == pad).all()) for i in range(22, TOP, 2 ** 28))
