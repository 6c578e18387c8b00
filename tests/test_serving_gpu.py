"""The cache upkeep and the attention calls as a serving loop makes them, one after another on one
stream: prompts join, sequences grow by a token or a few, some end and give their blocks back, one batch
runs behind a shared prefix; and calls under conditions that single tests do not make (many mixed runs,
two streams at once, caches beyond 2^32 elements)."""
import numpy as np
import pytest

import rows_reference as R

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import split_kv_async_gb300 as F
    from rows_harness import Problem, ints


class Server:
    """A paged cache of `blocks` blocks, the block map's state, and a host copy of every key and value."""

    def __init__(self, slots, blocks, width, block=16, hq=4, hkv=2, d=64, room=512, rot=64, seed=0):
        self.B, self.block, self.hq, self.hkv, self.d, self.room, self.rot = slots, block, hq, hkv, d, room, rot
        self.gen = torch.Generator().manual_seed(seed)
        dev = "cuda"
        self.k, self.v = (torch.full((blocks, block, hkv, d), float("nan"), dtype=torch.bfloat16, device=dev) for _ in range(2))
        self.held, self.want = ints([0] * slots), ints([0] * slots)
        self.pool, self.queue = ints([0, blocks]), ints(np.arange(blocks))
        self.table = ints(np.full((slots, width), -1))
        self.cu, self.seq, self.pos = ints([0] * (slots + 1)), ints([0] * room), ints([0] * room)
        self.slots = torch.zeros(room, dtype=torch.int64, device=dev)
        self.bp = F.make_block_params(batch=slots, block_size=block, max_blocks_per_seq=width, num_kv_blocks=blocks, max_tokens=room)
        self.bws = F.alloc_block_workspace(self.bp)
        row = (hq + 2 * hkv) * d
        self.rp = F.make_rope_params(num_tokens=room, num_q_heads=hq, num_kv_heads=hkv, head_dim=d, rot_dim=rot,
                                     dtype=F.FDPP_BF16, num_slots=blocks * block, q_stride=row, k_stride=row, v_stride=row)
        self.rope = torch.as_tensor(F.fdpp_rope_table(rot, 10000.0)).cuda()
        self.rws = F.alloc_rope_workspace()
        self.ap = F.make_rows_params(batch=slots, num_q_heads=hq, num_kv_heads=hkv, head_dim=d, dtype=F.FDPP_BF16,
                                     num_tokens=room, max_seq_len=width * block, scale=d ** -0.5, softcap=25.0,
                                     block_size=block, max_blocks_per_seq=width, num_kv_blocks=blocks)
        self.aws = F.alloc_rows_workspace(self.ap)
        self.q_out = torch.zeros(room, hq, d, dtype=torch.bfloat16, device=dev)
        self.out = torch.full_like(self.q_out, 9.0)
        self.qkv = torch.zeros(room, row, dtype=torch.bfloat16, device=dev)
        self.hk, self.hv, self.lens = [np.zeros((0, hkv, d))] * slots, [np.zeros((0, hkv, d))] * slots, [0] * slots

    def calls(self):
        hq, hkv, d = self.hq, self.hkv, self.d
        F.fdpp_block_map(self.held, self.want, self.pool, self.bp, self.table, self.queue, self.held, self.pool, self.cu,
                         self.seq, self.pos, self.slots, self.bws)
        F.fdpp_rope_append(self.qkv[:, :hq * d], self.qkv[:, hq * d:(hq + hkv) * d], self.qkv[:, (hq + hkv) * d:], self.pos,
                           self.slots, self.rope, self.rp, self.q_out, self.k, self.v, self.rws)
        F.fdpp_rows_attn(self.q_out, self.k, self.v, self.table, self.held, self.cu, self.ap, self.aws, self.out)

    def step(self, want, graph=None):
        """One step to `want` tokens; checks the attention of every new token."""
        hq, hkv, d = self.hq, self.hkv, self.d
        self.want.copy_(ints(want))
        qkv = torch.randn(self.room, (hq + 2 * hkv) * d, generator=self.gen).bfloat16()
        self.qkv.copy_(qkv)
        self.out.fill_(9.0)
        if graph is None:
            self.calls()
        else:
            graph.replay()
        torch.cuda.synchronize()
        assert F.fdpp_read_error(self.bws) == F.fdpp_read_error(self.rws) == F.fdpp_read_error(self.aws) == 0
        h = qkv.double().numpy().reshape(self.room, hq + 2 * hkv, d)
        theta = R.rope_theta(self.rot, 10000.0)
        n = [max(0, w - x) for w, x in zip(want, self.lens)]
        cu = np.concatenate([[0], np.cumsum(n)])
        T = int(cu[-1])
        pos = np.concatenate([np.arange(x, w) for w, x in zip(want, self.lens) if w > x] or [np.zeros(0)])
        bf16 = lambda x: torch.as_tensor(x).bfloat16().double().numpy()  # noqa: E731  (one rounding, as the cache's)
        k_new = bf16(R.rope(h[:T, hq:hq + hkv], pos, theta, False, 1.0))
        for b, w in enumerate(want):
            rows = slice(int(cu[b]), int(cu[b + 1]))
            self.hk[b] = np.concatenate([self.hk[b][:w], k_new[rows]])
            self.hv[b] = np.concatenate([self.hv[b][:w], h[rows, hq + hkv:]])
            self.lens[b] = w
        if not T:
            return
        x = R.Rows(q=bf16(R.rope(h[:T, :hq], pos, theta, False, 1.0)), k=self.hk, v=self.hv, pk=np.zeros((0, hkv, d)),
                   pv=np.zeros((0, hkv, d)), cu=cu, lens=np.asarray(self.lens), scale=d ** -0.5, cap=25.0)
        ref, spread = R.attention(x)
        got = self.out[:T].double().cpu().numpy()
        # besides the attention's own bounds: q and k are rounded after the rotation, and where the fp32
        # rotation lies within 2^-19 of a rounding border the two sides round to neighbours, 2^-7 of one
        # element apart. A score then moves by up to 2^-7 |q_i k_i| scale, at most about 2^-7 x 16 / 8: the
        # weights by 2^-6 of themselves.
        bound = 2.0 ** -8 * np.abs(ref) + (2.0 ** -8 + 2.0 ** -6) * spread
        assert (np.abs(got - ref) <= bound).all(), np.abs(got - ref).max()
        assert (self.out[T:] == 9.0).all()


def test_serving_loop():
    rng = np.random.default_rng(5)
    s = Server(slots=6, blocks=90, width=20)
    lens = [0] * 6
    s.step([40, 0, 3, 0, 100, 17])
    lens = [40, 0, 3, 0, 100, 17]
    for step in range(12):
        want = []
        for b, x in enumerate(lens):
            r = rng.random()
            want.append(0 if x and r < 0.1 else int(rng.integers(20, 120)) if not x and r < 0.5 else x if not x or r > 0.9
                        else min(300, x + int(rng.integers(1, 4))))
        s.step(want)
        lens = want


def test_captured_serving_step():
    s = Server(slots=5, blocks=120, width=20, room=64)
    s.step([15, 16, 17, 0, 9])
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=stream):
        s.calls()
    lens = [15, 16, 17, 0, 9]
    for step in range(20):
        lens = [x + (1 if b != 3 else 0) + (step % 3 == 0 and b == 1) for b, x in enumerate(lens)]
        if step == 10:
            lens[0], lens[3] = 0, 12
        s.step(lens, graph=g)


def test_many_runs_of_every_kind_again_and_again():
    # CTAs whose parts hold prefix pairs, single row tiles, key-major runs of one tile and of many, with the
    # streams at any distance from one another: a hundred calls without a wait that runs out
    rng = np.random.default_rng(7)
    for seed, (prefix, G, d) in enumerate(((2000, 8, 128), (0, 8, 128), (700, 4, 64))):
        seqs = [(int(rng.choice([1, 1, 1, 2, 5, 20, 70])), int(rng.integers(1, 700))) for _ in range(40)]
        x = Problem(seqs, hq=2 * G, hkv=2, d=d, block=16, prefix=prefix, seed=seed)
        first = x.call().clone()
        for _ in range(100):
            x.call()
        torch.cuda.synchronize()
        assert F.fdpp_read_error(x.ws) == 0
        assert torch.equal(x.out.view(torch.int16), first.view(torch.int16))
        x.check()


def test_two_streams_at_once():
    a = Problem([(1, 900)] * 20, hq=8, hkv=2, prefix=500, block=16, seed=1)
    b = Problem([(200, 300)], hq=8, hkv=2, seed=2)
    s, t = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(10):
        a.call(stream=s)
        b.call(stream=t)
    torch.cuda.synchronize()
    a.check(got=a.out)
    b.check(got=b.out)
    assert F.fdpp_read_error(a.ws) == F.fdpp_read_error(b.ws) == 0


def test_caches_beyond_32_bit_offsets():
    # 280000 blocks of 16 tokens: 4.6e9 elements in each pool; the sequence's blocks lie at both ends
    hkv, d, block, blocks = 8, 128, 16, 280000
    hq, L, n = 16, 130, 3
    gen = torch.Generator().manual_seed(3)
    k, v = torch.randn(L, hkv, d, generator=gen).bfloat16(), torch.randn(L, hkv, d, generator=gen).bfloat16()
    kp, vp = (torch.empty((blocks, block, hkv, d), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    ids = [blocks - 1, 0, blocks - 2, 262144, 262143, 1, blocks - 7, 131072, 5]
    table = ints([ids])
    q = torch.randn(n, hq, d, generator=gen).bfloat16()
    slots = torch.as_tensor([ids[t // block] * block + t % block for t in range(L)]).cuda()
    # k and v get there by the append, at position 0 (no rotation)
    p = F.make_rope_params(num_tokens=L, num_q_heads=hkv, num_kv_heads=hkv, head_dim=d, rot_dim=d, dtype=F.FDPP_BF16,
                           num_slots=blocks * block)
    ws = F.alloc_rope_workspace()
    kd = k.cuda()
    F.fdpp_rope_append(kd, kd, v.cuda(), ints([0] * L), slots, torch.as_tensor(F.fdpp_rope_table(d, 1e4)).cuda(), p,
                       torch.empty_like(kd), kp, vp, ws)
    out = torch.zeros(n, hq, d, dtype=torch.bfloat16, device="cuda")
    for kernel in (F.FDPP_KERNEL_TENSOR, F.FDPP_KERNEL_SIMT):
        ap = F.make_rows_params(batch=1, num_q_heads=hq, num_kv_heads=hkv, head_dim=d, dtype=F.FDPP_BF16, num_tokens=n,
                                max_seq_len=block * len(ids), scale=d ** -0.5, block_size=block, max_blocks_per_seq=len(ids),
                                num_kv_blocks=blocks, kernel=kernel)
        aws = F.alloc_rows_workspace(ap)
        out.zero_()
        F.fdpp_rows_attn(q.cuda(), kp, vp, table, ints([L]), ints([0, n]), ap, aws, out)
        torch.cuda.synchronize()
        assert F.fdpp_read_error(aws) == F.fdpp_read_error(ws) == 0
        f64 = lambda t: t.double().numpy()  # noqa: E731
        ref, spread = R.attention(R.Rows(q=f64(q), k=[f64(k)], v=[f64(v)], pk=np.zeros((0, hkv, d)), pv=np.zeros((0, hkv, d)),
                                         cu=np.array([0, n]), lens=np.array([L]), scale=d ** -0.5))
        assert (np.abs(out.double().cpu().numpy() - ref) <= 2.0 ** -8 * np.abs(ref) + (2.0 ** -8 + 2.0 ** -12) * spread).all()


def test_the_largest_plan():
    # more sequences than a small plan holds (and than the block map's shared memory): the general plan
    rng = np.random.default_rng(11)
    seqs = [(1, int(rng.integers(1, 40))) for _ in range(1500)]
    Problem(seqs, hq=2, hkv=1, d=64, block=16, seed=3).check()
    Problem(seqs[:1300], hq=2, hkv=1, d=64, prefix=130, seed=3, mask=lambda row, pos, total: (max(0, pos - 25), pos + 1)).check()


def test_a_layer_between_two_linears():
    # flat GEMM -> append -> attention -> flat GEMM in one graph: each call reads what the one before it wrote
    hq, hkv, d, block, B, L = 8, 2, 128, 16, 24, 200
    E, row = 512, (8 + 2 * 2) * 128
    gen = torch.Generator().manual_seed(17)
    x = torch.randn(B, E, generator=gen).bfloat16().cuda()
    w_qkv = (torch.randn(row, E, generator=gen) * E ** -0.5).bfloat16().cuda()
    w_o = (torch.randn(E, hq * d, generator=gen) * (hq * d) ** -0.5).bfloat16().cuda()
    per = (L + block) // block + 1
    blocks = B * per
    k, v = (torch.randn(blocks, block, hkv, d, generator=gen).bfloat16().cuda() for _ in range(2))
    table = ints(np.arange(blocks).reshape(B, per))
    lens, pos = ints([L + 1] * B), ints([L] * B)
    slots = (table[:, L // block].long() * block + L % block).contiguous()
    cu = ints(np.arange(B + 1))
    qkv = torch.zeros(B, row, dtype=torch.bfloat16, device="cuda")
    q_out, out = torch.zeros(B, hq, d, dtype=torch.bfloat16, device="cuda"), torch.zeros(B, hq, d, dtype=torch.bfloat16, device="cuda")
    y = torch.zeros(B, E, dtype=torch.bfloat16, device="cuda")
    rp = F.make_rope_params(num_tokens=B, num_q_heads=hq, num_kv_heads=hkv, head_dim=d, rot_dim=d, dtype=F.FDPP_BF16,
                            num_slots=blocks * block, q_stride=row, k_stride=row, v_stride=row)
    ap = F.make_rows_params(batch=B, num_q_heads=hq, num_kv_heads=hkv, head_dim=d, dtype=F.FDPP_BF16, num_tokens=B,
                            max_seq_len=per * block, scale=d ** -0.5, block_size=block, max_blocks_per_seq=per,
                            num_kv_blocks=blocks)
    rope = torch.as_tensor(F.fdpp_rope_table(d, 1e4)).cuda()
    rws, aws = F.alloc_rope_workspace(), F.alloc_rows_workspace(ap)
    g1, g2 = F.alloc_flat_gemm_workspace(B, row, E), F.alloc_flat_gemm_workspace(B, E, hq * d)

    def calls():
        F.fdpp_flat_gemm(x, w_qkv, qkv, g1)
        F.fdpp_rope_append(qkv[:, :hq * d], qkv[:, hq * d:(hq + hkv) * d], qkv[:, (hq + hkv) * d:], pos, slots, rope, rp,
                           q_out, k, v, rws)
        F.fdpp_rows_attn(q_out, k, v, table, lens, cu, ap, aws, out)
        F.fdpp_flat_gemm(out.view(B, hq * d), w_o, y, g2)

    # every call alone, with a wait between them
    for f in (lambda: F.fdpp_flat_gemm(x, w_qkv, qkv, g1),
              lambda: F.fdpp_rope_append(qkv[:, :hq * d], qkv[:, hq * d:(hq + hkv) * d], qkv[:, (hq + hkv) * d:], pos, slots,
                                         rope, rp, q_out, k, v, rws),
              lambda: F.fdpp_rows_attn(q_out, k, v, table, lens, cu, ap, aws, out),
              lambda: F.fdpp_flat_gemm(out.view(B, hq * d), w_o, y, g2)):
        f()
        torch.cuda.synchronize()
    apart = y.clone()
    ref = out.double().view(B, -1) @ w_o.double().T
    assert (y.double() - ref).abs().max() <= 2.0 ** -8 * ref.abs().max() + 1e-4
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=stream):
        calls()
    for again in range(5):
        for t in (qkv, q_out, out, y):
            t.fill_(3.0)
        k.view(-1, hkv, d)[slots] = 1.0
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, apart)


@pytest.mark.parametrize("block", [0, 16])
@pytest.mark.parametrize("n,G", [(300, 4), (3, 4), (1, 1)])
def test_visible_values_that_are_not_finite(n, G, block):
    # an inf (a NaN) among the values that rows see: inf (NaN) in its column, every other column as without
    L = 300
    x = Problem([(n, L), (2, 40)], hq=G, hkv=1, d=128, block=block, seed=4)
    x.call()
    torch.cuda.synchronize()
    plain = x.out.clone()
    at = (int(x.table[0, 0]), 3) if block else (0, 3)
    for value in (float("inf"), float("nan")):
        x.v_d[at[0], at[1], 0, 5] = value
        x.out.fill_(9.0)
        x.call()
        torch.cuda.synchronize()
        assert F.fdpp_read_error(x.ws) == 0
        first = L - n                                     # position of the first row
        sees = torch.arange(n + 2, device="cuda") + first >= 3
        sees[n:] = False
        col = x.out[:, :, 5].float()
        assert (torch.isinf(col[sees]) & (col[sees] > 0)).all() if value == float("inf") else torch.isnan(col[sees]).all()
        # rows that do not see it are computed again in another order: the bounds of the operator
        same = x.out.clone()
        same[:, :, 5][sees] = plain[:, :, 5][sees]
        x.check(got=same)
        other = torch.arange(128, device="cuda") != 5
        assert torch.equal(same[sees][:, :, other], plain[sees][:, :, other])


@pytest.mark.parametrize("many", [False, True])
def test_token_offsets_out_of_order_behind_a_prefix(many):
    # (the large plan, too): whatever the workspace held before, the error is reported and the call returns
    seqs = [(1, 20)] * (1300 if many else 4) + [(90, 90)]
    x = Problem(seqs, hq=4, hkv=1, d=64, prefix=150, seed=6)
    x.ws[4096:].fill_(0x9d)
    x.check()
    cu = x.cu_d.clone()
    for at, value in ((len(seqs), 3), (2, 60), (len(seqs) - 1, 0)):
        x.ws[4096:].fill_(0x9d)
        x.cu_d.copy_(cu)
        x.cu_d[at] = value
        x.call()
        torch.cuda.synchronize()
        bits = F.fdpp_read_error(x.ws)
        assert bits & F.FDPP_ERRBIT_TOKENS and not bits & F.FDPP_ERRBIT_TIMEOUT
        F.fdpp_workspace_init(x.ws)
    x.cu_d.copy_(cu)
    x.check()
