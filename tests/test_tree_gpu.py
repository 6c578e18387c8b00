"""Tree attention and the tree's commit on the GPU: against 64 bits and plain Python (tree_harness), at the
sizes and masks where a tree can go wrong."""
import numpy as np
import pytest
import torch

import split_kv_async_gb300 as F
from rows_harness import ints
from tree_harness import TreeProblem, commit, line, random_tree

pytestmark = pytest.mark.gpu

SIMT = F.FDPP_KERNEL_SIMT


def trees_of(seed, sizes, width=3, roots=0):
    rng = np.random.default_rng(seed)
    return [random_tree(rng, n, width, roots) for n in sizes]


# ---- attention ---------------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("block", [0, 16, 128])
@pytest.mark.parametrize("hq,hkv,d", [(4, 4, 64), (8, 1, 128), (6, 2, 128)])
@pytest.mark.parametrize("sizes,old", [((1,), (0,)), ((5, 1, 9), (0, 127, 300)), ((33, 16), (95, 1)), ((64,), (128,))])
def test_attention_sizes(dtype, block, hq, hkv, d, sizes, old):
    TreeProblem(trees_of(1, sizes), old, hq=hq, hkv=hkv, d=d, dtype=dtype, block=block).check()


@pytest.mark.parametrize("width", [1, 2, 300])
@pytest.mark.parametrize("n", [2, 31, 32, 33, 64, 65, 200, 256])
def test_attention_chains_and_bushes(width, n):
    # drafts that begin anywhere in a tile of keys and run over several; further roots
    for old in (0, 31, 120, 129, 700):
        TreeProblem(trees_of(n, (n,), width, roots=9), (old,), hq=4, hkv=2, d=64 if n % 2 else 128, seed=n + old).check()


@pytest.mark.parametrize("G", [1, 3, 8, 16, 40, 128])
def test_attention_heads_per_kv_head(G):
    TreeProblem(trees_of(G, (7, 3, 12)), (250, 5, 64), hq=2 * G, hkv=2, d=128, block=32).check()


@pytest.mark.parametrize("dtype,cap", [("bf16", 2.0), ("bf16", 50.0), ("f32", 3.0)])
@pytest.mark.parametrize("d", [64, 128])
def test_attention_capped(dtype, cap, d):
    TreeProblem(trees_of(3, (20, 6)), (300, 90), hq=8, hkv=2, d=d, dtype=dtype, cap=cap, q_gain=3.0).check()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("window", [1, 3, 40, 128, 100000])
def test_attention_window(dtype, window):
    TreeProblem(trees_of(4, (17, 40, 2)), (200, 0, 385), begin=lambda row, pos: pos + 1 - window, hq=8, hkv=2, d=64,
                dtype=dtype, block=16).check()


@pytest.mark.parametrize("hq,hkv,d", [(16, 2, 128), (8, 4, 64)])
@pytest.mark.parametrize("sizes,old", [
    ((61,), (5000,)),                                      # few units, each cut in many parts
    ((1,), (9000,)), ((0, 40, 0), (700, 3000, 0)), ((256,), (1000,)), ((7, 90), (1, 2500)),
    ((2,) * 12 + (61,), (10,) * 12 + (5000,)),             # many units, one of them long
])
def test_attention_cut_in_many_parts(hq, hkv, d, sizes, old):
    x = TreeProblem(trees_of(9, sizes), old, hq=hq, hkv=hkv, d=d, block=64)
    x.check()
    first = x.out.clone()
    x.out.fill_(float("nan"))
    x.check()
    assert bool((x.out[x.rows[0]:x.rows[1]] == first[x.rows[0]:x.rows[1]]).all())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_attention_leaves_rows_of_no_sequence(dtype):
    TreeProblem(trees_of(5, (3, 8)), (40, 77), lead=4, tail=5, spare_len=30, dtype=dtype).check()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_attention_uniform_without_offsets(dtype):
    TreeProblem(trees_of(6, (6, 6, 6)), (10, 300, 64), uniform=True, dtype=dtype, block=64).check()


def test_attention_bf16_on_the_cuda_cores():
    TreeProblem(trees_of(7, (11, 4)), (130, 20), kernel=SIMT, hq=8, hkv=2, d=128, block=16).check()


@pytest.mark.parametrize("old", [20, 2000])
def test_attention_kernel_chosen_by_the_library(old):
    """Small problems on the CUDA cores, larger ones on the tensor cores: the same bits as when asked for, and a
    workspace that fits either way."""
    for kernel in (SIMT, F.FDPP_KERNEL_TENSOR):
        x = TreeProblem(trees_of(15, (11, 4)), (old, 7), kernel=kernel, hq=8, hkv=2, d=128, block=16)
        got = x.call().clone()
        x.p.kernel = F.FDPP_KERNEL_AUTO
        x.ws, x.simt = F.alloc_tree_workspace(x.p), old == 20          # (the bound of the kernel that is taken)
        x.check()
        same = torch.equal(x.call(), got)
        torch.cuda.synchronize()
        assert same == ((kernel == SIMT) == (old == 20))


@pytest.mark.parametrize("hq", [2, 16])
@pytest.mark.parametrize("what", ["k", "v"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_attention_other_branches_may_hold_anything(hq, what, dtype):
    """A node's K or V is NaN or infinite: its descendants have the formula's effect, the others none."""
    for node, value in ((1, float("nan")), (5, float("inf")), (20, float("-inf"))):
        x = TreeProblem(trees_of(8, (30,), 4), (150,), hq=hq, hkv=1, d=128, dtype=dtype)
        key = 150 + node
        for host, dev in ((x.host.k, x.k_d),) if what == "k" else ((x.host.v, x.v_d),):
            host[0][key, 0, 3] = value
            dev[0, key, 0, 3] = value
        got = x.call().double().cpu().numpy()
        assert F.fdpp_read_error(x.ws) == 0
        # (scores of +-inf: rows that see such a K end NaN or without it, by the signs; looked at for V alone)
        rows = [i for i in range(30) if node not in line(x.trees[0], i)]
        clean = TreeProblem(trees_of(8, (30,), 4), (150,), hq=hq, hkv=1, d=128, dtype=dtype)
        want = clean.call().double().cpu().numpy()
        torch.cuda.synchronize()
        assert np.isfinite(got[rows]).all()
        step = float(torch.finfo({"bf16": torch.bfloat16, "f32": torch.float32}[dtype]).eps)
        # the same keys; a row's columns that are computed again add the same weights unrounded, in another order
        np.testing.assert_allclose(got[rows], want[rows], rtol=step, atol=2.0 ** -7 if dtype == "bf16" else 2.0 ** -18)
        if what == "v":
            seen = [i for i in range(30) if node in line(x.trees[0], i)]
            assert not np.isfinite(got[seen][:, :, 3]).any()
            others = np.delete(got[seen], 3, axis=2)
            assert np.isfinite(others).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_attention_reports_bad_parents(dtype):
    trees = trees_of(9, (6, 9))
    trees[1][4], trees[1][7], trees[0][0] = 4, -2, 3
    x = TreeProblem(trees, (50, 33), dtype=dtype)
    x.check(errors=F.FDPP_ERRBIT_TREE)             # (counted as roots, in the reference too)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_attention_of_a_tree_that_is_too_large(dtype):
    x = TreeProblem(trees_of(10, (5, 257, 4)), (50, 20, 3), dtype=dtype, hq=2, hkv=1, d=64)
    x.check(errors=F.FDPP_ERRBIT_TREE)


def test_attention_of_keys_that_are_fewer_than_the_tokens():
    """seq_lens below the number of tokens: the nodes that have no key see nothing."""
    for dtype in ("bf16", "f32"):
        x = TreeProblem(trees_of(11, (9,), 1), (30,), dtype=dtype)
        x.lens_d.fill_(6)
        x.host.lens = np.array([6])
        x.host.k[0], x.host.v[0] = x.host.k[0][:6], x.host.v[0][:6]
        x.check()


def test_attention_rows_and_tree_agree_on_a_chain():
    """A chain is the causal mask: the same bits as fdpp_rows_attn."""
    x = TreeProblem(trees_of(12, (40, 3), 1), (300, 129), hq=8, hkv=2, block=16)
    got = x.call().clone()
    ws, out = F.alloc_rows_workspace(x.p), torch.full_like(x.out, 9.0)
    F.fdpp_rows_attn(x.q_d, x.k_d, x.v_d, x.table, x.lens_d, x.cu_d, x.p, ws, out)
    torch.cuda.synchronize()
    assert torch.equal(got, out)


def test_attention_many_sequences():
    """More sequences than the plan keeps in shared memory, and a plan of several CTAs."""
    for B, n in ((1100, 2), (300, 9)):
        TreeProblem(trees_of(B, [n] * B, 2), [b % 70 for b in range(B)], hq=2, hkv=1, d=64).check()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_attention_captured_on_another_stream(dtype):
    """A captured call follows lengths and trees that change between replays."""
    trees = trees_of(13, (8, 20), 3)
    x = TreeProblem(trees, (100, 40), dtype=dtype, block=16)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    x.call(stream=stream)
    stream.synchronize()
    x.check(x.out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        x.call(stream=stream)
    x.trees = trees_of(14, (8, 20), 5)
    x.parents_d.copy_(ints([p for t in x.trees for p in t]))
    x.lens_d.copy_(ints([101, 57]))
    x.host.lens = np.array([101, 57])
    x.out.fill_(9.0)
    graph.replay()
    torch.cuda.synchronize()
    assert F.fdpp_read_error(x.ws) == 0
    x.check(x.out)


# ---- commit ------------------------------------------------------------------------------------

class Commit:
    """caches of random rows, and what is expected of them."""

    def __init__(self, trees, old, block=0, caches=3, row=64, dtype=torch.bfloat16, match=0.8, seed=0, lead=0, tail=0, few=50):
        rng = np.random.default_rng(seed)
        B, n = len(trees), [len(t) for t in trees]
        self.trees, self.n, self.lens = trees, n, [a + o for a, o in zip(n, old)]
        self.tokens = [[int(rng.integers(few)) for _ in t] for t in trees]
        self.choices = []
        for t, k in zip(trees, self.tokens):
            c = []
            for i in range(len(t)):
                after = [j for j in range(len(t)) if t[j] == i]
                c.append(k[int(rng.choice(after))] if after and rng.random() < match else -5)
            self.choices.append(c)
        T = lead + sum(n) + tail
        self.cu = lead + np.concatenate([[0], np.cumsum(n)])
        flat = lambda x: ints([99] * lead + [v for y in x for v in y] + [99] * tail)  # noqa: E731
        self.d = dict(parents=flat(trees), tokens=flat(self.tokens), choices=flat(self.choices), lens=ints(self.lens), cu=ints(self.cu))
        Lmax = max(max(self.lens), 1)
        self.table = self.table_d = None
        self.block = block
        kw = {}
        size = (B, Lmax, row)
        if block:
            used = [-(-L // block) for L in self.lens]
            ids = rng.permutation(sum(used) + 2)
            width = max(1, -(-Lmax // block))
            self.table = np.full((B, width), 2 ** 30, np.int64)
            at = 0
            for b, u in enumerate(used):
                self.table[b, :u] = ids[at:at + u]
                at += u
            self.table_d = ints(self.table)
            size = (sum(used) + 2, block, row)
            kw = dict(block_size=block, max_blocks_per_seq=width, num_kv_blocks=sum(used) + 2)
        gen = torch.Generator().manual_seed(seed)
        self.host = [torch.randn(size, generator=gen).to(dtype) for _ in range(caches)]
        self.dev = [c.cuda() for c in self.host]
        self.list = F.make_cache_list(self.dev)
        self.p = F.make_commit_params(batch=B, num_tokens=T, max_seq_len=Lmax, row_bytes=row * self.host[0].element_size() if caches
                                      else 16, **kw)
        self.ws = F.alloc_commit_workspace(self.p)
        self.out = dict(new_lens=ints([77] * B), accepted=ints([77] * B), path=ints([77] * T), chosen=ints([77] * T))
        self.lead = lead

    def call(self, stream=None, uniform=False):
        table = self.table_d
        F.fdpp_tree_commit(self.d["parents"], self.d["tokens"], self.d["choices"], self.d["lens"], None if uniform else self.d["cu"],
                           table, self.list, self.p, self.ws, self.out["new_lens"], self.out["accepted"], self.out["path"],
                           self.out["chosen"], stream=stream)

    def slot(self, b, pos):
        if self.table is None:
            return b, pos
        return int(self.table[b, pos // self.block]), pos % self.block

    def check(self, paths=None, errors=0, refused=()):
        torch.cuda.synchronize()
        assert F.fdpp_read_error(self.ws) == errors
        paths = commit(self.trees, self.tokens, self.choices) if paths is None else paths
        want = {k: v.cpu().numpy().copy() for k, v in self.out.items()}
        for b, path in enumerate(paths):
            base, c0 = self.lens[b] - self.n[b], int(self.cu[b])
            if b in refused:
                path = []
            want["accepted"][b], want["new_lens"][b] = len(path), self.lens[b] if b in refused else base + len(path)
            rows = np.arange(c0, c0 + self.n[b])
            want["path"][rows] = path + [-1] * (self.n[b] - len(path))
            want["chosen"][rows] = [self.choices[b][i] for i in path] + [-1] * (self.n[b] - len(path))
            for c in self.host:
                moved = [c[self.slot(b, base + i)].clone() for i in path]
                for k, row in enumerate(moved):
                    c[self.slot(b, base + k)] = row
        for k, v in self.out.items():
            np.testing.assert_array_equal(v.cpu().numpy(), want[k], err_msg=k)
        assert (self.out["path"].cpu().numpy()[:self.lead] == 77).all()
        for c, d in zip(self.host, self.dev):
            assert torch.equal(c.view(torch.uint8), d.cpu().view(torch.uint8))


@pytest.mark.parametrize("block", [0, 16, 64])
@pytest.mark.parametrize("sizes,old", [((1,), (0,)), ((0, 3), (5, 0)), ((16, 2, 9, 40), (15, 100, 0, 33)), ((256,), (200,))])
@pytest.mark.parametrize("match", [0.0, 0.8, 1.0])
def test_commit_sizes(block, sizes, old, match):
    for width in (1, 3, 30):
        x = Commit(trees_of(20 + width, sizes, width, roots=12), old, block=block, match=match, seed=width)
        x.call()
        x.check()


@pytest.mark.parametrize("row,dtype", [(8, torch.bfloat16), (4, torch.float32), (1000, torch.bfloat16), (1024, torch.bfloat16),
                                       (16, torch.float32)])
@pytest.mark.parametrize("caches", [0, 1, 2, 7, 256])
def test_commit_rows_and_caches(row, dtype, caches):
    x = Commit(trees_of(30, (14, 7, 30), 4), (9, 20, 3), block=16, caches=caches, row=row, dtype=dtype)
    x.call()
    x.check()


def test_commit_long_paths():
    """Paths of up to 256 nodes, each place but the first written after it is read: a chain with a gap behind
    every so many nodes."""
    for gap in (2, 3, 50):
        parents, on_path = [-1], [0]
        while len(parents) < 256:
            parents.append(on_path[-1])
            if len(parents) % gap:
                on_path.append(len(parents) - 1)
        x = Commit([parents], [13], block=16, row=72)
        x.tokens = [[1 if i in on_path else 2 for i in range(256)]]
        x.choices = [[1] * 256]
        x.d["tokens"], x.d["choices"] = ints(x.tokens[0]), ints(x.choices[0])
        x.call()
        x.check([on_path])


def test_commit_the_first_of_children_with_one_token():
    parents = [-1, 0, 0, 0, 2, 3, -1]
    x = Commit([parents], [4])
    x.tokens, x.choices = [[0, 5, 6, 6, 7, 7, 6]], [[6, 1, 7, 7, 9, 9, 9]]
    x.d["tokens"], x.d["choices"] = ints(x.tokens[0]), ints(x.choices[0])
    x.call()
    x.check([[0, 2, 4]])


def test_commit_leaves_rows_of_no_sequence_and_takes_uniform_batches():
    x = Commit(trees_of(31, (6, 4), 2), (3, 8), lead=3, tail=4)
    x.call()
    x.check()
    x = Commit(trees_of(32, (6, 6, 6), 2), (3, 8, 0), block=32)
    x.call(uniform=True)
    x.check()


def test_commit_reports_bad_parents_lengths_and_trees():
    trees = trees_of(33, (6, 9), 2)
    trees[1][4], trees[1][7] = 4, -2
    x = Commit(trees, (5, 3))
    x.call()
    x.check(errors=F.FDPP_ERRBIT_TREE)
    x = Commit(trees_of(34, (5, 257, 4)), (5, 2, 3))
    x.call()
    x.check(errors=F.FDPP_ERRBIT_TREE, refused=(1,))
    x = Commit(trees_of(35, (5, 8, 4), 1), (5, 2, 3))
    x.lens[1] = 7                                  # fewer keys than tokens
    x.d["lens"].copy_(ints(x.lens))
    x.call()
    x.check(errors=F.FDPP_ERRBIT_SEQ_LEN, refused=(1,))


def test_commit_skips_blocks_outside_the_pool():
    """A path that moves from node 2 to place 1, whose block is bad: nothing is moved, the rest is reported."""
    x = Commit([[-1, 0, 0]], [15], block=16)
    x.tokens, x.choices = [[0, 1, 2]], [[2, 0, 0]]
    x.d["tokens"], x.d["choices"] = ints(x.tokens[0]), ints(x.choices[0])
    before = [c.clone() for c in x.host]
    x.table_d[0, 1] = 2 ** 30
    x.call()
    torch.cuda.synchronize()
    assert F.fdpp_read_error(x.ws) == F.FDPP_ERRBIT_BLOCK_TABLE
    assert x.out["accepted"].item() == 2 and x.out["new_lens"].item() == 17
    assert all(torch.equal(a, b.cpu()) for a, b in zip(before, x.dev))


def test_commit_captured_on_another_stream():
    x = Commit(trees_of(36, (12, 5), 3), (30, 8), block=16)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    x.call(stream=stream)
    x.check()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        x.call(stream=stream)
    x.d["choices"].copy_(ints([v for c in x.choices for v in c[::-1]]))
    x.choices = [v for v in np.split(x.d["choices"].cpu().numpy(), [12])]
    x.choices = [list(map(int, c)) for c in x.choices]
    graph.replay()
    x.check()


@pytest.mark.parametrize("paged", [False, True])
def test_commit_in_caches_beyond_32_bits(paged):
    """Rows that lie more than 2^32 bytes into a cache."""
    row, keys = 1024, (1 << 32) // 2048 + 4096
    kw = dict(block_size=256, max_blocks_per_seq=1, num_kv_blocks=keys // 256) if paged else {}
    cache = torch.zeros(keys, row, dtype=torch.bfloat16, device="cuda")
    n, parents, path = 6, [-1, 0, 0, 2, 2, 4], [0, 2, 4, 5]
    L = 250 if paged else keys - 3
    base = (keys // 256 - 1) * 256 + L - n if paged else L - n          # the last block, or the end of the one sequence
    cache[base:base + n] = torch.arange(1, n + 1, device="cuda")[:, None].to(torch.bfloat16)
    p = F.make_commit_params(batch=1, num_tokens=n, max_seq_len=256 if paged else keys, row_bytes=2 * row, **kw)
    ws, out = F.alloc_commit_workspace(p), [ints([0]), ints([0]), ints([0] * n), ints([0] * n)]
    tokens = ints([1 if i in path else 2 for i in range(n)])
    F.fdpp_tree_commit(ints(parents), tokens, ints([1] * n), ints([L]), None, ints([[keys // 256 - 1]]) if paged else None,
                       F.make_cache_list([cache]), p, ws, *out)
    torch.cuda.synchronize()
    assert F.fdpp_read_error(ws) == 0 and out[1].item() == 4 and out[2].tolist() == path + [-1, -1]
    assert cache[base:base + n, ::97].float().mean(1).tolist() == [1, 3, 5, 6, 5, 6]
    assert int(torch.count_nonzero(cache[:4096])) == 0


def test_attention_two_streams():
    xs = [TreeProblem(trees_of(40 + i, (9, 30), 3), (200, 77), hq=8, hkv=2, d=64 * (i + 1), block=16) for i in range(2)]
    streams = [torch.cuda.Stream() for _ in xs]
    torch.cuda.synchronize()
    for _ in range(10):
        for x, s in zip(xs, streams):
            x.call(stream=s)
    torch.cuda.synchronize()
    for x in xs:
        assert F.fdpp_read_error(x.ws) == 0
        x.check(x.out)
