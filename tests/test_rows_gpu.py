"""Rows attention and shared-prefix attention on the GPU against the 64-bit reference (bounds in
rows_harness). Caches hold NaN wherever no sequence has a key."""
import numpy as np
import pytest

import rows_reference as R

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import split_kv_async_gb300 as F
    from rows_harness import Problem, ints


def _window(w):
    return lambda row, pos, total: (max(0, pos + 1 - w), pos + 1)


def _ahead(m):
    return lambda row, pos, total: (0, min(total, max(pos + 1, m)))


def _documents(row, pos, total):
    return (pos // 37 * 37, pos + 1)


def _some_nothing(row, pos, total):
    return (5, 5) if row % 3 == 0 else ((7, 2) if row % 3 == 1 else (0, pos + 1))


def _odd(row, pos, total):       # ranges that reach out of the keys on either side
    return (-9, total + 50) if row % 2 else (pos - 3, pos + 130)


SHAPES = [
    # one sequence, one token; every side of a key tile
    dict(seqs=[(1, 1)]),
    dict(seqs=[(1, 127)]),
    dict(seqs=[(1, 128)], hq=8, hkv=1),
    dict(seqs=[(1, 129)], hq=3, hkv=3),
    dict(seqs=[(1, 5000)], hq=7, hkv=1),
    # a ragged batch of single tokens, one sequence without keys, one without tokens
    dict(seqs=[(1, 300), (1, 0), (0, 50), (1, 77), (1, 1024)], hq=8, hkv=2),
    # prompts: fewer rows than a tile, one tile and a bit, a pair and a bit
    dict(seqs=[(5, 5)], hq=4, hkv=4),
    dict(seqs=[(33, 33)], hq=4, hkv=1),
    dict(seqs=[(70, 200), (3, 3), (129, 129)], hq=4, hkv=2),
    dict(seqs=[(300, 300)], hq=2, hkv=2),
    dict(seqs=[(257, 700), (1, 900)], hq=6, hkv=2),
    # fewer keys than tokens: the first tokens see nothing
    dict(seqs=[(9, 4), (40, 10)], hq=4, hkv=2),
    # heads that do not divide a tile
    dict(seqs=[(50, 260)], hq=7, hkv=1),
    dict(seqs=[(3, 260)], hq=96, hkv=1),
    dict(seqs=[(4, 130)], hq=128, hkv=1),
    # rows before the first sequence and behind the last
    dict(seqs=[(4, 40), (2, 140)], lead=3, tail=5, spare_len=30),
    # T / B tokens each, without cu_tokens
    dict(seqs=[(3, 40), (3, 140), (3, 3)], uniform=True),
]
MODS = [
    dict(),
    dict(cap=20.0),
    dict(bias=True),
    dict(cap=5.0, bias=True, q_gain=3.0),
    dict(mask=_window(20)),
    dict(mask=_documents, bias=True),
    dict(mask=_ahead(150)),
    dict(mask=_some_nothing, cap=10.0),
    dict(mask=_odd),
]


def _name(x):
    return "-".join(f"{k}={getattr(v, '__name__', v)}".replace(" ", "") for k, v in x.items()) or "plain"


@pytest.mark.parametrize("d", [128, 64])
@pytest.mark.parametrize("block", [0, 16, 256])
@pytest.mark.parametrize("shape", SHAPES, ids=_name)
def test_shapes(shape, block, d):
    Problem(**shape, block=block, d=d, seed=len(str(shape))).check()


@pytest.mark.parametrize("prefix", [0, 150])
@pytest.mark.parametrize("mod", MODS, ids=_name)
def test_scores_and_masks(mod, prefix):
    for d, block, seqs in ((128, 32, [(1, 260), (40, 200), (150, 150)]), (64, 0, [(300, 300), (2, 9)])):
        Problem(seqs, hq=4, hkv=2, d=d, block=block, prefix=prefix, seed=3, **mod).check()


PREFIXES = [
    dict(seqs=[(1, 1)], prefix=1),
    dict(seqs=[(1, 0), (1, 5)], prefix=128, hq=8, hkv=2),
    dict(seqs=[(1, 40)] * 9, prefix=1000, hq=16, hkv=2),
    dict(seqs=[(1, 3), (2, 300), (0, 7), (3, 3), (1, 200)], prefix=333, hq=8, hkv=2),
    dict(seqs=[(1, 17)] * 40, prefix=2050, hq=8, hkv=1),         # more rows than a pair of tiles
    dict(seqs=[(90, 90), (1, 1), (20, 60)], prefix=260, hq=7, hkv=1),
    dict(seqs=[(4, 0), (9, 2)], prefix=5, hq=4, hkv=2),          # positions inside the prefix and before it
    dict(seqs=[(1, 12)] * 3, prefix=0, spare_prefix=64),         # an empty prefix
    dict(seqs=[(1, 12)] * 3, prefix=70, spare_prefix=64, lead=2, tail=4),
]


@pytest.mark.parametrize("d", [128, 64])
@pytest.mark.parametrize("block", [0, 16, 128])
@pytest.mark.parametrize("shape", PREFIXES, ids=_name)
def test_prefix(shape, block, d):
    Problem(**shape, block=block, d=d, seed=5).check()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape", [
    dict(seqs=[(1, 256)], hq=4, hkv=4, d=64, bias=True),
    dict(seqs=[(1, 3), (2, 300), (0, 7), (5, 5)], hq=7, hkv=1, d=128, prefix=90, cap=9.0),
    dict(seqs=[(1, 1), (1, 0)], hq=2, hkv=2, d=64, block=16),
    dict(seqs=[(60, 300), (3, 100)], hq=6, hkv=2, d=128, block=64, mask=_documents),
    dict(seqs=[(9, 4)], hq=4, hkv=1, d=64, mask=_some_nothing),
    dict(seqs=[(1, 3000)], hq=1, hkv=1, d=128, lead=1, tail=2),
    dict(seqs=[(2, 30), (2, 70)], hq=9, hkv=1, d=64, uniform=True, prefix=130, block=32),
], ids=_name)
def test_cuda_core_kernel(shape, dtype):
    x = Problem(**shape, dtype=dtype, kernel=F.FDPP_KERNEL_SIMT, seed=8)
    x.check()
    x.check()              # the split counters are back at zero


@pytest.mark.parametrize("seed", range(24))
def test_random(seed):
    rng = np.random.default_rng(1000 + seed)
    hkv = int(rng.choice([1, 2, 3]))
    G = int(rng.choice([1, 2, 3, 5, 8, 16]))
    kind = seed % 3
    B = int(rng.integers(1, 12))
    seqs = []
    for _ in range(B):
        n = int(rng.integers(0, 4)) if kind == 0 else int(rng.integers(0, 200 // G + 2))
        seqs.append((n, int(rng.integers(0, 600)) if rng.random() < 0.8 else n))
    seqs[0] = (max(1, seqs[0][0]), seqs[0][1])
    mods = MODS[int(rng.integers(0, len(MODS)))]
    Problem(seqs, hq=hkv * G, hkv=hkv, d=int(rng.choice([64, 128])), block=int(rng.choice([0, 16, 32, 64, 128, 256])),
            prefix=int(rng.integers(1, 700)) if kind == 2 else 0, seed=seed, **mods).check()


def test_many_small_units():
    # far more row tiles than CTAs, most of them a single key tile
    rng = np.random.default_rng(2)
    seqs = [(int(rng.integers(0, 3)), int(rng.integers(0, 140))) for _ in range(700)]
    Problem(seqs, hq=4, hkv=2, d=64, block=16, seed=2).check()
    Problem(seqs[:300], hq=4, hkv=2, d=128, prefix=64, seed=2).check()


def test_repeated_calls_are_bitwise_equal():
    for kw in (dict(seqs=[(1, 900), (30, 400)], hq=8, hkv=2), dict(seqs=[(1, 50)] * 30, hq=8, hkv=2, prefix=900)):
        x = Problem(**kw, seed=6)
        first = x.call().clone()
        for _ in range(5):
            x.out.fill_(x.fill)
            assert torch.equal(x.call().view(torch.int16), first.view(torch.int16))
        x.check()


def test_nan_and_infinity():
    # a key's NaN or infinity reaches the rows that see it, and no other, in any mix of tiles
    for hidden in (float("nan"), float("inf")):
        for seqs, at in (([(40, 200)], 190), ([(150, 150)], 64), ([(3, 130)], 129)):
            x = Problem(seqs, hq=4, hkv=2, seed=9)
            x.v_d[0, at] = hidden
            x.host.v[0][at] = hidden
            x.check()
    x = Problem([(40, 200)], hq=4, hkv=2, seed=9)
    x.k_d[0, 180, 1] = float("nan")
    x.host.k[0][180, 1] = np.nan
    x.check()
    x = Problem([(1, 300), (4, 80)], hq=4, hkv=2, seed=9, prefix=140)
    x.pv[100, 0, 5] = float("nan")
    x.host.pv[100, 0, 5] = np.nan
    x.check()


def test_hidden_keys_may_hold_anything():
    # keys that a sliding window has left behind, in the same tile as ones still seen
    x = Problem([(1, 300), (5, 260)], hq=4, hkv=2, mask=_window(30), block=16, seed=4)
    for b, L in enumerate((300, 260)):
        n = (1, 5)[b]
        for t in range(L - n + 1 - 30):
            blk = int(x.table[b, t // 16])
            x.k_d[blk, t % 16] = float("nan")
            x.v_d[blk, t % 16] = float("nan")
    x.check()


def test_large_and_far_apart_scores():
    # maxima that grow by far more than the frame's lag from tile to tile, and rows of one key's weight
    x = Problem([(5, 700)], hq=4, hkv=2, q_gain=8.0, scale=1.0, seed=7)
    ramp = torch.linspace(0.1, 3.0, 700).cuda()[:, None, None]
    x.k_d[0, :700] = (x.k_d[0, :700].float() * ramp).bfloat16()
    x.host.k[0] = x.k_d[0, :700].double().cpu().numpy()
    # the scores reach some thousands: their fp32 rounding, 2^-24 of sum |q k| <= 2^13 each way, moves a
    # weight by up to 2^-10 of itself, within what the weights' own rounding allows twice
    x.check()


def test_bad_lengths_tables_and_rows_set_bits():
    x = Problem([(1, 40), (1, 50)], hq=2, hkv=1, block=16, seed=1)
    x.table[0, 1] = -5
    x.call()
    torch.cuda.synchronize()
    assert F.fdpp_read_error(x.ws) == F.FDPP_ERRBIT_BLOCK_TABLE
    ref, _ = __import__("rows_reference").attention(x.host)
    assert np.abs(x.out[1].double().cpu().numpy() - ref[1]).max() < 0.05      # the other row is right
    x = Problem([(1, 40), (1, 50)], hq=2, hkv=1, seed=1)
    x.lens_d.copy_(ints([-3, 51]))
    x.call()
    torch.cuda.synchronize()
    assert F.fdpp_read_error(x.ws) == F.FDPP_ERRBIT_SEQ_LEN
    assert (x.out[0] == 0).all()
    for cu in ([0, 2, 1], [-4, 1, 2], [0, 9, 2], [0, 1, 9], [2, 1, 0]):
        for kernel in (F.FDPP_KERNEL_TENSOR, F.FDPP_KERNEL_SIMT):
            x = Problem([(1, 40), (1, 50)], hq=2, hkv=1, seed=1, kernel=kernel)
            x.cu_d.copy_(ints(cu))
            x.call()
            torch.cuda.synchronize()
            bits = F.fdpp_read_error(x.ws)
            assert bits in (0, F.FDPP_ERRBIT_TOKENS) and (kernel == F.FDPP_KERNEL_SIMT or bits)
    x = Problem([(1, 40)], hq=2, hkv=1, seed=1, prefix=20)
    x.plen_d.fill_(21)
    x.call()
    torch.cuda.synchronize()
    assert F.fdpp_read_error(x.ws) == F.FDPP_ERRBIT_PREFIX


def test_one_workspace_for_calls_of_different_shapes():
    big = Problem([(1, 100)] * 6 + [(60, 300)], hq=8, hkv=2, prefix=300, seed=1)
    others = [Problem([(1, 256)], hq=4, hkv=4, d=64, dtype="f32", seed=2), Problem([(90, 90)], hq=2, hkv=1, d=64, seed=3),
              Problem([(1, 30)] * 4, hq=4, hkv=1, seed=4)]
    for _ in range(2):
        for x in [big] + others:
            x.out.fill_(x.fill)
            x.call(ws=big.ws)
            torch.cuda.synchronize()
            x.check(got=x.out)
    assert F.fdpp_read_error(big.ws) == 0


def test_captured_and_on_another_stream():
    x = Problem([(1, 300), (3, 90)], hq=8, hkv=2, block=16, prefix=200, seed=1)
    y = Problem([(70, 200)], hq=4, hkv=2, seed=2)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    x.call(stream=s)
    y.call(stream=s)
    torch.cuda.synchronize()
    x.check(got=x.out)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        x.call()
        y.call()
        x.call()
    for _ in range(3):
        x.out.fill_(x.fill)
        y.out.fill_(y.fill)
        g.replay()
        torch.cuda.synchronize()
        x.check(got=x.out)
        y.check(got=y.out)


@pytest.mark.parametrize("rows", [1025, 2100, 9000])
@pytest.mark.parametrize("kw", [dict(), dict(prefix=90), dict(cap=20.0, prefix=200),
                                dict(mask=lambda row, pos, total: (pos // 64 * 64 if row % 5 else pos, pos + 1 + (row % 3 == 0)))],
                         ids=["plain", "prefix", "cap", "mask"])
def test_plans_of_many_tokens(rows, kw):
    # one to nine rounds of 1024 tokens: a plan made by several CTAs, the last one with few tokens or none
    rng = np.random.default_rng(rows)
    seqs, left = [], rows
    while left:
        n = min(left, int(rng.choice([1, 1, 7, 200, 700])))
        seqs.append((n, n + int(rng.integers(0, 60))))
        left -= n
    Problem(seqs, hq=4, hkv=1, d=64, block=16, seed=rows, lead=3, tail=5, **kw).check()


def test_uniform_tokens_of_many_sequences():
    Problem([(3, 40)] * 1000, hq=2, hkv=2, d=64, seed=2, uniform=True).check()
    Problem([(9, 9)] * 1100, hq=2, hkv=1, d=64, seed=2, uniform=True).check()


@pytest.mark.parametrize("cap", [2.0, 50.0, 1000.0])
def test_capped_scores_in_fp32_keep_its_accuracy(cap):
    # a score: each of eight lanes adds 16 products and three additions join them, 19 x 2^-24 scale sum |q k|,
    # below 2^-16 (scale 0.09, sum |q k| about 82, up to 115); the cap: two units in the last place of a value
    # below 5, 2^-20; the exponent's product with log2(e), 2^-21. A weight is off by as much of itself, the
    # sums by 2^-22
    x = Problem([(2, 130), (1, 700)], hq=8, hkv=2, dtype="f32", cap=cap, seed=8)
    got = x.call()
    torch.cuda.synchronize()
    ref, spread = R.attention(x.host)
    err = np.abs(got.double().cpu().numpy() - ref)
    assert (err <= 2.0 ** -24 * np.abs(ref) + (2.0 ** -16 + 2.0 ** -19) * spread).all(), (err / spread).max()


@pytest.mark.parametrize("gain", [0.5, 2.0, 8.0])
@pytest.mark.parametrize("bias", [False, True])
def test_caps_near_and_far(gain, bias):
    # scores below half their cap, some above it, most above it: both forms of the cap, in one tile and in turn
    seqs = [(300, 300), (150, 400)]
    Problem(seqs, hq=4, hkv=1, d=128, block=16, cap=6.0, bias=bias, q_gain=gain, seed=12).check()
    Problem(seqs, hq=4, hkv=2, d=64, cap=6.0, bias=bias, q_gain=gain, seed=13, prefix=140).check()
