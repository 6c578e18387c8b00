"""Rows attention where a unit is cut between CTAs, where tiles hold lanes without a row, where tables and
offsets are wrong, and at the ends of the parameters' ranges (bounds in rows_harness)."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import split_kv_async_gb300 as F
    from rows_harness import Problem, ints


def _hide(x, b, t, value):
    """V of key t of sequence b (-1: the prefix) of problem x becomes `value` in every column."""
    block = x.p.block_size
    if b < 0:
        x.host.pv[t] = value
        if block:
            x.v_d[int(x.prefix_table[t // block]), t % block] = value
        else:
            x.pv[t] = value
    else:
        x.host.v[b][t] = value
        if block:
            x.v_d[int(x.table[b, t // block]), t % block] = value
        else:
            x.v_d[b, t] = value


def _ends(row, pos, total):        # even rows see the last 60 keys, odd ones the first 60
    return (0, 60) if row % 2 else (total - 60, total)


def _begin_or_end(row, pos, total):
    return (0, 90) if row % 2 else (300, total)


def _begin_or_all(row, pos, total):
    return (0, 90) if row % 2 else (0, total)


def _name(x):
    return "-".join(f"{k}={getattr(v, '__name__', v)}".replace(" ", "") for k, v in x.items()) if isinstance(x, dict) else str(x)


@pytest.mark.parametrize("value", [float("nan"), float("inf")])
@pytest.mark.parametrize("block", [0, 16])
@pytest.mark.parametrize("kw,b,t", [
    # positions on both sides of key 128, and a key that only the later ones see: with so few key tiles each is
    # a part of its own, and the second tile's part holds rows that see none of its keys
    (dict(seqs=[(5, 131)], hq=4, hkv=2), 0, 130),
    (dict(seqs=[(9, 133)], hq=2, hkv=2), 0, 132),
    (dict(seqs=[(20, 140)], hq=4, hkv=2), 0, 139),
    (dict(seqs=[(40, 290)], hq=4, hkv=1), 0, 270),
    (dict(seqs=[(150, 150)], hq=4, hkv=1), 0, 140),
    # keys that no row sees between the two ranges that the rows see
    (dict(seqs=[(6, 400)], hq=4, hkv=2, mask=_ends), 0, 200),
    (dict(seqs=[(60, 400)], hq=4, hkv=2, mask=_ends), 0, 200),
    (dict(seqs=[(60, 700)], hq=2, hkv=1, mask=_ends), 0, 300),
    # the same in a prefix, which rows see the beginning or the end of
    (dict(seqs=[(6, 20), (50, 50)], hq=4, hkv=2, prefix=420, mask=_begin_or_end), -1, 200),
    (dict(seqs=[(3, 20), (2, 70)], hq=4, hkv=2, prefix=300, mask=_begin_or_all), -1, 299),
], ids=_name)
def test_hidden_values_in_cut_units(kw, b, t, block, value):
    for d in (128, 64):
        x = Problem(**kw, block=block, d=d, seed=21)
        _hide(x, b, t, value)
        x.check()


def _same_bits(x, between):
    """x's output is the same, bit for bit, after each of the calls in `between`."""
    outs = []
    for f in between:
        f()
        x.out.fill_(x.fill)
        outs.append(x.call().clone())
    torch.cuda.synchronize()
    assert F.fdpp_read_error(x.ws) == 0
    for o in outs[1:]:
        assert torch.equal(o.view(torch.int16), outs[0].view(torch.int16))
    x.check()


@pytest.mark.parametrize("kw", [dict(), dict(cap=20.0), dict(cap=6.0, bias=True), dict(bias=True)], ids=_name)
@pytest.mark.parametrize("hq,hkv,block", [(14, 2, 0), (3, 1, 16), (5, 1, 0), (6, 2, 16)])
def test_bits_do_not_depend_on_what_shared_memory_held(hq, hkv, block, kw):
    # 3, 5, 6 and 7 heads do not divide 128: a tile's last lanes hold no row, and their operand is what the SM's
    # shared memory held before: here queries of next to no size, or of a size that grows a maximum by far more
    # than the frames' lag from tile to tile; and keys past a sequence's end likewise
    others = [Problem([(64, 600)] * 8, hq=32, hkv=8, d=128, block=block, q_gain=g, seed=31) for g in (1e-3, 60.0, 0.0)]
    x = Problem([(90, 907), (40, 333), (7, 1001), (130, 130)], hq=hq, hkv=hkv, d=128, block=block, seed=32, **kw)
    _same_bits(x, [o.call for o in others] * 2)


@pytest.mark.parametrize("kw", [dict(), dict(cap=20.0)], ids=_name)
@pytest.mark.parametrize("prefix", [0, 700])
def test_bits_do_not_depend_on_rows_of_no_sequence(prefix, kw):
    # (a tile's lanes past a sequence's last token hold the rows that follow)
    x = Problem([(10, 907), (37, 611)], hq=4, hkv=1, d=128, prefix=prefix, lead=9, tail=30, seed=33, **kw)

    def fill(gain):
        gen = torch.Generator().manual_seed(5)
        rows = (gain * torch.randn(39, 4, 128, generator=gen)).bfloat16().cuda()
        x.q_d[:9], x.q_d[-30:] = rows[:9], rows[9:]

    _same_bits(x, [lambda: fill(1e-3), lambda: fill(60.0), lambda: fill(float("nan"))])


@pytest.mark.parametrize("dtype,kernel", [("f32", "AUTO"), ("bf16", "SIMT"), ("bf16", "TENSOR")])
@pytest.mark.parametrize("kw,entry", [
    # one key of the bad block is seen, or few, and not by the lanes that hold the first key of every sixteen
    (dict(seqs=[(1, 17), (1, 50)], mask=lambda row, pos, total: (5 if total == 17 else 0, total)), 1),
    (dict(seqs=[(1, 3), (1, 50)], prefix=500), 0),
    (dict(seqs=[(1, 1000), (1, 50)], spare_len=1048), 62),
    (dict(seqs=[(3, 33), (2, 50)]), 2),
], ids=["begin", "prefix", "split", "tokens"])
def test_bad_blocks_are_reported_by_every_kernel(kw, entry, dtype, kernel):
    for bad in (-5, 1 << 20):
        x = Problem(hq=4, hkv=2, d=64, block=16, dtype=dtype, kernel=getattr(F, "FDPP_KERNEL_" + kernel), seed=41, **kw)
        x.check()
        x.table[0, entry] = bad
        got = x.call().clone()
        torch.cuda.synchronize()
        assert F.fdpp_read_error(x.ws) == F.FDPP_ERRBIT_BLOCK_TABLE
        # the other sequence's rows are what they were
        n = x.host.cu[1]
        x.table[0, entry] = 0
        assert torch.equal(got[n:], x.call()[n:])


@pytest.mark.parametrize("kernel", ["TENSOR", "SIMT"])
def test_bad_offsets_and_lengths_are_reported_by_every_kernel(kernel):
    kernel = getattr(F, "FDPP_KERNEL_" + kernel)
    for cu in ([0, 2, 1], [-4, 1, 2], [0, 9, 2], [0, 1, 9], [2, 1, 0], [0, 0, -1], [5, 2, 2]):
        x = Problem([(1, 40), (1, 50)], hq=2, hkv=1, seed=1, kernel=kernel)
        x.cu_d.copy_(ints(cu))
        x.call()
        torch.cuda.synchronize()
        assert F.fdpp_read_error(x.ws) == F.FDPP_ERRBIT_TOKENS, cu
    # lengths of sequences with tokens and without
    for at in (0, 1, 170):
        x = Problem([(1, 40)] + [(0, 50)] * 180, hq=2, hkv=1, seed=1, kernel=kernel)
        x.check()
        x.lens_d[at] = 51 if at else -3
        x.call()
        torch.cuda.synchronize()
        assert F.fdpp_read_error(x.ws) == F.FDPP_ERRBIT_SEQ_LEN, at
    # a batch in which no sequence has tokens
    x = Problem([(0, 40), (0, 50)], hq=2, hkv=1, seed=1, kernel=kernel, tail=1, prefix=20)
    x.check()
    x.plen_d.fill_(21)
    x.call()
    torch.cuda.synchronize()
    assert F.fdpp_read_error(x.ws) == F.FDPP_ERRBIT_PREFIX


@pytest.mark.parametrize("scale,cap", [(10.0, 1e-6), (1.0, 1e-9), (3.0, 1e-5), (1e-6, 4000.0), (4e8, 4000.0)])
def test_caps_far_from_their_scale(scale, cap):
    # 64 tokens with queries of size zero before the others (whole tiles of them): their scores are 0 whatever the
    # ratio of scale and cap
    for d, seqs in ((128, [(100, 300), (1, 200)]), (64, [(150, 400)])):
        x = Problem(seqs, hq=4, hkv=1, d=d, scale=scale, cap=cap, seed=51)
        for t in (x.q_d, x.q, x.host.q):
            t[:64] = 0
        if cap < 1:
            x.check()
            continue
        # scores far below their cap, or at it (the scores of a row are equal then): finite, and the rows of
        # zeros the mean of their values
        got = x.call()
        torch.cuda.synchronize()
        assert F.fdpp_read_error(x.ws) == 0 and torch.isfinite(got.float()).all()
        ref, spread = __import__("rows_reference").attention(x.host)
        err = np.abs(got.double().cpu().numpy() - ref)
        assert (err <= 2.0 ** -8 * np.abs(ref) + (2.0 ** -8 + 2.0 ** -12) * spread)[:64].all()


def test_rows_computed_again_may_take_longer_than_a_wait():
    # the newest token of every sequence holds a NaN, 160000 keys behind it: the rows that do not see it are
    # computed again, for some seconds, while the warps that feed the next unit wait
    B, L, n, G, hkv, d, pool, block = 24, 160000, 16, 8, 8, 64, 64, 256
    width = L // block
    gen = torch.Generator("cuda").manual_seed(61)
    k, v = (torch.randn(pool, block, hkv, d, generator=gen, device="cuda").bfloat16() for _ in range(2))
    table = np.random.default_rng(61).integers(0, pool - 1, (B, width))
    table[:, -1] = pool - 1                                  # the block with the NaN, nowhere else
    q = torch.randn(B * n, G * hkv, d, generator=gen, device="cuda").bfloat16()
    p = F.make_rows_params(batch=B, num_q_heads=G * hkv, num_kv_heads=hkv, head_dim=d, dtype=F.FDPP_BF16, num_tokens=B * n,
                           max_seq_len=L, scale=d ** -0.5, block_size=block, max_blocks_per_seq=width, num_kv_blocks=pool)
    ws, table, lens = F.alloc_rows_workspace(p), ints(table), ints([L] * B)

    def call(values):
        out = torch.empty_like(q)
        F.fdpp_rows_attn(q, k, values, table, lens, None, p, ws, out)
        torch.cuda.synchronize()
        assert F.fdpp_read_error(ws) == 0
        return out.double().view(B, n, G * hkv, d)

    clean, spread = call(v), call(v.abs())                   # (spread: sum_t p_t |v_t|, 2^-7 of itself off)
    v[pool - 1, block - 1] = float("nan")
    got = call(v)
    assert torch.isnan(got[:, -1]).all()
    # both calls are within the operator's bounds of the formula
    bound = 2.0 ** -8 * 2 * clean.abs() + 2 * (2.0 ** -8 + 2.0 ** -12) * (1 + 2.0 ** -6) * spread
    assert ((got - clean).abs() <= bound)[:, :-1].all()


@pytest.mark.parametrize("kw", [dict(), dict(prefix=140), dict(mask=_begin_or_all)], ids=_name)
@pytest.mark.parametrize("uniform", [False, True])
def test_plans_of_more_sequences_than_their_shared_memory_holds(kw, uniform):
    # 2100 sequences and more: lengths, offsets and the row tiles' starts are read from global memory
    rng = np.random.default_rng(71)
    seqs = [(2 if uniform else int(rng.integers(0, 4)), int(rng.integers(0, 150))) for _ in range(2100)]
    Problem(seqs, hq=2, hkv=1, d=64, block=16, seed=71, uniform=uniform, **kw).check()
