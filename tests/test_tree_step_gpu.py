"""Steps of tree drafting on a paged cache of two layers, every call on the GPU as a serving loop makes them: the
block map makes room for the trees, hidden states are normed into 8 bits and projected, rotated and appended,
the trees attend, the next projection follows, the accepted paths are committed in all caches, and the
block map takes the blocks behind them back. Each call is checked against 64 bits of its own inputs, and the caches
against a host copy over all steps; then the same step captured and replayed with other trees."""
import numpy as np
import pytest
import torch

import tree_harness as T
import split_kv_async_gb300 as F
from rows_harness import ints

pytestmark = pytest.mark.gpu

B, HQ, HKV, D, DIM, BLOCK, WIDTH, BLOCKS, LAYERS = 3, 8, 2, 64, 400, 16, 12, 40, 2
ROOM = 48                       # token rows of a step
ROW = (HQ + 2 * HKV) * D
FP8 = torch.float8_e4m3fn


def bf16(*shape, gen):
    return torch.randn(*shape, generator=gen, device="cuda").bfloat16()


class Loop:
    def __init__(self, seed=0):
        gen = self.gen = torch.Generator("cuda").manual_seed(seed)
        self.rng = np.random.default_rng(seed)
        zeros = lambda *s, t=torch.int32: torch.zeros(*s, dtype=t, device="cuda")  # noqa: E731
        self.k, self.v = ([torch.full((BLOCKS, BLOCK, HKV, D), float("nan"), dtype=torch.bfloat16, device="cuda")
                           for _ in range(LAYERS)] for _ in range(2))
        self.caches = F.make_cache_list(self.k + self.v)
        # the block map's state, and the step's arrays
        self.lens, self.want, self.new_lens, self.accepted = (zeros(B) for _ in range(4))
        self.pool, self.queue = ints([0, BLOCKS]), ints(np.arange(BLOCKS))
        self.table = ints(np.full((B, WIDTH), -1))
        self.cu, self.none_cu = zeros(B + 1), zeros(B + 1)
        self.seq, self.pos, self.slots = zeros(ROOM), zeros(ROOM), zeros(ROOM, t=torch.int64)
        self.parents, self.tokens, self.choices, self.path, self.chosen, self.rotary = (zeros(ROOM) for _ in range(6))
        self.bp = F.make_block_params(batch=B, block_size=BLOCK, max_blocks_per_seq=WIDTH, num_kv_blocks=BLOCKS, max_tokens=ROOM)
        self.x, self.res = bf16(ROOM, DIM, gen=gen), bf16(ROOM, DIM, gen=gen)
        self.gain = bf16(DIM, gen=gen)
        self.np = F.make_norm_params(num_tokens=ROOM, dim=DIM, dtype=F.FDPP_BF16, out_dtype=F.FDPP_E4M3)
        self.q8, self.qs = zeros(ROOM, DIM, t=torch.uint8), zeros(ROOM, self.np.scale_stride, t=torch.float32)
        self.w = [(torch.randn(ROW, DIM, generator=gen, device="cuda") * 40).clamp(-448, 448).to(FP8).view(torch.uint8)
                  for _ in range(LAYERS)]
        self.ws = [0.002 * torch.rand(-(-ROW // 128), -(-DIM // 128), generator=gen, device="cuda") for _ in range(LAYERS)]
        self.gp = F.make_scaled_gemm_params(M=ROOM, N=ROW, K=DIM)
        self.qkv = [zeros(ROOM, ROW, t=torch.bfloat16) for _ in range(LAYERS)]
        self.rp = F.make_rope_params(num_tokens=ROOM, num_q_heads=HQ, num_kv_heads=HKV, head_dim=D, rot_dim=D, dtype=F.FDPP_BF16,
                                     num_slots=BLOCKS * BLOCK, q_stride=ROW, k_stride=ROW, v_stride=ROW)
        self.rope = torch.as_tensor(F.fdpp_rope_table(D, 10000.0)).cuda()
        self.ap = F.make_rows_params(batch=B, num_q_heads=HQ, num_kv_heads=HKV, head_dim=D, dtype=F.FDPP_BF16, num_tokens=ROOM,
                                     max_seq_len=WIDTH * BLOCK, scale=D ** -0.5, block_size=BLOCK, max_blocks_per_seq=WIDTH,
                                     num_kv_blocks=BLOCKS, kernel=F.FDPP_KERNEL_TENSOR)
        self.cp = F.make_commit_params(batch=B, num_tokens=ROOM, max_seq_len=WIDTH * BLOCK, row_bytes=HKV * D * 2, block_size=BLOCK,
                                       max_blocks_per_seq=WIDTH, num_kv_blocks=BLOCKS)
        self.q, self.out = ([torch.full((ROOM, HQ, D), 9.0, dtype=torch.bfloat16, device="cuda") for _ in range(LAYERS)]
                            for _ in range(2))
        self.spaces = dict(block=F.alloc_block_workspace(self.bp), rope=F.alloc_rope_workspace(), gemm=F.alloc_scaled_gemm_workspace(self.gp),
                           attn=F.alloc_tree_workspace(self.ap), commit=F.alloc_commit_workspace(self.cp))
        self.host = [[[np.zeros((0, HKV, D)) for _ in range(B)] for _ in range(2)] for _ in range(LAYERS)]
        self.held = [0] * B

    def draft(self, first=False):
        """New trees, their tokens, the target's choices, and rotary positions by depth."""
        n = [int(self.rng.integers(5, 9)) if first else int(self.rng.integers(1, 13)) for _ in range(B)]
        self.trees = [T.random_tree(self.rng, x, 1 if first else 3) for x in n]
        self.tok = [[int(self.rng.integers(4)) for _ in t] for t in self.trees]
        self.cho = [[int(self.rng.integers(4)) for _ in t] for t in self.trees]
        depth = [[len(T.line(t, i)) - 1 for i in range(len(t))] for t in self.trees]
        self.where = [h + np.array(d) for h, d in zip(self.held, depth)]
        pad = lambda rows: ints([v for r in rows for v in r] + [0] * (ROOM - sum(n)))  # noqa: E731
        self.n, self.rows = n, sum(n)
        for to, rows in ((self.parents, self.trees), (self.tokens, self.tok), (self.choices, self.cho), (self.rotary, self.where)):
            to.copy_(pad(rows))
        self.want.copy_(ints([h + x for h, x in zip(self.held, n)]))
        self.x.copy_(bf16(ROOM, DIM, gen=self.gen))
        for o in self.out:
            o.fill_(9.0)                       # (rows of no sequence are left as they were)

    def calls(self):
        s = self.spaces
        F.fdpp_block_map(self.lens, self.want, self.pool, self.bp, self.table, self.queue, self.lens, self.pool, self.cu, self.seq,
                         self.pos, self.slots, s["block"])
        for i in range(LAYERS):
            F.fdpp_rms_norm(self.x, self.res, self.gain, self.np, self.q8, self.qs)
            F.fdpp_scaled_gemm(self.q8, self.qs, self.w[i], self.ws[i], self.gp, s["gemm"], self.qkv[i])
            y = self.qkv[i]
            F.fdpp_rope_append(y[:, :HQ * D], y[:, HQ * D:(HQ + HKV) * D], y[:, (HQ + HKV) * D:], self.rotary, self.slots, self.rope,
                               self.rp, self.q[i], self.k[i], self.v[i], s["rope"])
            F.fdpp_tree_attn(self.q[i], self.k[i], self.v[i], self.table, self.lens, self.cu, self.parents, self.ap, s["attn"], self.out[i])
        F.fdpp_tree_commit(self.parents, self.tokens, self.choices, self.lens, self.cu, self.table, self.caches, self.cp, s["commit"],
                           self.new_lens, self.accepted, self.path, self.chosen)
        F.fdpp_block_map(self.lens, self.new_lens, self.pool, self.bp, self.table, self.queue, self.lens, self.pool, self.none_cu,
                         self.seq, self.pos, self.slots, s["block"])

    def step(self, graph=None, first=False):
        self.draft(first)
        if graph is None:
            self.calls()
        else:
            graph.replay()
        torch.cuda.synchronize()
        assert {k: F.fdpp_read_error(w) for k, w in self.spaces.items()} == {k: 0 for k in self.spaces}
        cu = np.concatenate([[0], np.cumsum(self.n)])
        assert self.cu.tolist() == cu.tolist()
        f64 = lambda t: t.double().cpu().numpy()  # noqa: E731
        R = self.rows
        # norm and projection
        r = self.x.double() + self.res.double()
        y = r / torch.sqrt((r * r).mean(-1, keepdim=True) + 1e-6) * self.gain.double()
        each = self.qs.double().repeat_interleave(128, 1)[:, :DIM]
        got8 = self.q8.view(FP8).double() * each
        assert bool(((got8 - y).abs() <= (2.0 ** -4 + 2.0 ** -16) * y.abs() + 2.0 ** -10 * each).all())
        paths = T.commit(self.trees, self.tok, self.cho)
        for i in range(LAYERS):
            wd = self.w[i].view(FP8).double() * self.ws[i].double().repeat_interleave(128, 0)[:ROW].repeat_interleave(128, 1)[:, :DIM]
            want = got8 @ wd.T
            assert bool(((self.qkv[i].double() - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -15 * (got8.abs() @ wd.abs().T)).all())
            # rotation (fp32 angles, good to 2^-23 turns, one rounding)
            h = f64(self.qkv[i]).reshape(ROOM, HQ + 2 * HKV, D)[:R]
            turned = T.R.rope(h, np.concatenate(self.where), T.R.rope_theta(D, 10000.0), False, 1.0)
            close = lambda a, b: (np.abs(a - b) <= 2.0 ** -8 * np.abs(b) + 2.0 ** -18 * np.abs(h).max()).all()  # noqa: E731
            q = f64(self.q[i])[:R]
            assert close(q, turned[:, :HQ])
            # the trees' keys as the cache had them before the commit: as the append rounds them
            keys, vals = [], []
            for b in range(B):
                rows = slice(int(cu[b]), int(cu[b + 1]))
                new_k = torch.as_tensor(turned[rows, HQ:HQ + HKV]).bfloat16().double().numpy()
                keys.append(np.concatenate([self.host[i][0][b], new_k]))
                vals.append(np.concatenate([self.host[i][1][b], h[rows, HQ + HKV:]]))
            x = T.R.Rows(q=q, k=keys, v=vals, pk=np.zeros((0, HKV, D)), pv=np.zeros((0, HKV, D)), cu=cu,
                         lens=np.array([len(k) for k in keys]), scale=D ** -0.5)
            ref, spread = T.attention(x, self.trees)
            got = f64(self.out[i])
            # besides the attention's own bounds: a rotated key within 2^-18 of a rounding border may be the
            # neighbour, 2^-7 of one element; a score then moves by up to 2^-7 |q k| / 8, the weights by 2^-6 of themselves
            bound = 2.0 ** -8 * np.abs(ref) + (2.0 ** -8 + 2.0 ** -12 + 2.0 ** -6 * max(1.0, np.abs(q).max() ** 2 / 16)) * spread
            assert (np.abs(got[:R] - ref) <= bound).all(), np.abs(got[:R] - ref).max()
            assert (got[R:] == 9.0).all()
            # the committed cache: the path's rows, bit for bit what the append wrote of them
            tab = self.table.cpu().numpy()
            for b, path in enumerate(paths):
                length = self.held[b] + len(path)
                at = np.arange(length)
                for which, cache, mine in ((0, self.k[i], keys), (1, self.v[i], vals)):
                    rows = f64(cache)[tab[b, at // BLOCK], at % BLOCK]
                    expect = np.concatenate([self.host[i][which][b], mine[b][self.held[b]:][path]])
                    assert (rows[:self.held[b]] == expect[:self.held[b]]).all()
                    assert close(rows, expect) if which == 0 else (rows == expect).all()
                    self.host[i][which][b] = rows
        new = [h + len(p) for h, p in zip(self.held, paths)]
        assert self.accepted.tolist() == [len(p) for p in paths] and self.new_lens.tolist() == new == self.lens.tolist()
        flat = [v for p, n in zip(paths, self.n) for v in p + [-1] * (n - len(p))]
        assert self.path[:R].tolist() == flat
        self.held = new
        # the blocks behind the committed lengths are back in the pool
        assert self.pool.tolist()[1] == BLOCKS - sum(-(-x // BLOCK) for x in new)


def test_steps():
    s = Loop()
    s.step(first=True)
    for _ in range(8):
        s.step()


def test_captured_step_follows_new_trees():
    s = Loop(seed=3)
    s.step(first=True)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        s.calls()
    for _ in range(5):
        s.step(graph)
