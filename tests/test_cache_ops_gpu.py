"""The block map and the rotary append on the GPU against plain implementations.

The block map is whole numbers: equal. The rotary append computes in fp32 with angles to about 2^-23
turns (2^-20 rad, which is 2^-20 of the pair's length at most) and rounds once; the products and the sum
of a pair add a few 2^-24 of the same length. So an element is off by at most half a step of its type
(eps / 2 of the value) and 2^-19 of its pair's length times the magnitude; and by the angle that the
table is off: theta is held as two floats, hi with 24 bits and lo with the 24 bits that follow, so it is
off by 2^-49 of itself, and the angle at position pos by 2^-49 |pos| theta <= 2^-49 |pos| rad (2^-29 at
2^20, 2^-18 at 2^31)."""
import numpy as np
import pytest

import rows_reference as R

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import split_kv_async_gb300 as F

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def _dev(a, dtype=np.int32):
    return torch.as_tensor(np.asarray(a, dtype)).cuda()


class Map:
    """A pool and the tables of `held` tokens, on the host and on the device."""

    def __init__(self, held, block, free, width, seed=0, room=64):
        rng = np.random.default_rng(seed)
        used = [-(-h // block) for h in held]
        pool = sum(used) + free
        ids = rng.permutation(pool).astype(np.int32)
        self.block, self.room, self.cap = block, room, pool
        self.table = np.full((len(held), width), -7, np.int32)
        at = 0
        for b, u in enumerate(used):
            self.table[b, :u] = ids[at:at + u]
            at += u
        head = int(rng.integers(pool))
        self.queue = np.full(pool, -9, np.int32)
        self.queue[(head + np.arange(free)) % pool] = ids[at:]
        self.pool, self.held = (head, free), list(held)
        self.p = F.make_block_params(batch=len(held), block_size=block, max_blocks_per_seq=width, num_kv_blocks=pool,
                                     max_tokens=room)
        self.ws = F.alloc_block_workspace(self.p)
        self.d = dict(held=_dev(held), pool=_dev(self.pool), table=_dev(self.table), queue=_dev(self.queue),
                      lens=_dev([-1] * len(held)), pool_out=_dev([-1, -1]), cu=_dev([-1] * (len(held) + 1)),
                      seq=_dev([-5] * room), pos=_dev([-5] * room), slots=_dev([-5] * room, np.int64))

    def call(self, want, in_place=False, stream=None):
        d = self.d
        self.want_d = _dev(want)
        F.fdpp_block_map(d["held"], self.want_d, d["pool"], self.p, d["table"], d["queue"],
                         d["held"] if in_place else d["lens"], d["pool"] if in_place else d["pool_out"], d["cu"],
                         d["seq"], d["pos"], d["slots"], self.ws, stream=stream)
        return [x.cpu().numpy() for x in (d["held"] if in_place else d["lens"], d["table"], d["queue"],
                                          d["pool"] if in_place else d["pool_out"], d["cu"], d["seq"], d["pos"],
                                          d["slots"])]

    def check(self, want, in_place=False):
        got = self.call(want, in_place)
        ref = R.block_map(self.held, want, self.pool, self.table, self.queue, self.block, self.room)
        for name, x, y in zip(("lens", "table", "queue", "pool", "cu", "seq", "pos", "slots"), got, ref):
            np.testing.assert_array_equal(x, np.asarray(y), err_msg=name)
        bits = (F.FDPP_ERRBIT_POOL if any(r[0] for r in ref[8].values()) else 0) | \
            (F.FDPP_ERRBIT_ROOM if any(r[1] for r in ref[8].values()) else 0)
        assert F.fdpp_read_error(self.ws) == bits
        return ref


MAPS = [
    # held, want, block, free blocks, room
    ([0], [1], 16, 1, 1),
    ([15, 16, 17], [16, 17, 18], 16, 3, 8),
    ([5], [5], 16, 0, 4),                                  # nothing to do
    ([40, 0, 33, 256], [0, 70, 33, 255], 32, 9, 100),      # one ends, one begins, one loses a token
    ([100, 3, 64], [130, 300, 65], 16, 5, 512),            # too few blocks: the later ones wait
    ([10, 20, 30], [15, 25, 31], 16, 5, 7),                # too few rows
    ([16, 16, 16], [17, 16, 30], 16, 1, 64),               # the third needs the block the first took
    ([300] * 5, [0] * 5, 256, 0, 0),                       # all end, no rows at all
]


@pytest.mark.parametrize("held,want,block,free,room", MAPS)
@pytest.mark.parametrize("in_place", [False, True])
def test_block_map(held, want, block, free, room, in_place):
    m = Map(held, block, free, width=-(-max(held + want) // block) + 1, room=room)
    m.check(want, in_place)


@pytest.mark.parametrize("batch,block,room", [(33, 16, 4096), (1025, 64, 3000), (2500, 16, 4096), (700, 32, 60001)])
def test_block_map_large(batch, block, room):
    # more sequences than the CTA has threads, rows on both sides of the one-launch limit, some refused
    rng = np.random.default_rng(batch)
    held = rng.integers(0, 500, batch).tolist()
    want = [0 if rng.random() < 0.2 else h + int(rng.integers(0, 2 * room // batch + 2)) for h in held]
    need = sum(max(0, -(-w // block) - -(-h // block)) for h, w in zip(held, want))
    m = Map(held, block, free=max(1, int(need * 0.9)), width=-(-max(held + want) // block) + 2, room=room, seed=batch)
    m.check(want)


@pytest.mark.parametrize("batch,block,room,in_place", [(1500, 16, 9000, False), (1024, 16, 4097, True),
                                                       (40, 64, 20000, True), (1025, 16, 5000, True),
                                                       (3, 16, 100000, False), (1024, 128, 70000, False)])
def test_block_map_in_two_launches_or_many_ctas(batch, block, room, in_place):
    # sequences that end, grow and stay; with and without refusals; blocks given back while others are taken
    rng = np.random.default_rng(batch + room)
    held = rng.integers(0, 300, batch).tolist()
    want = [0 if rng.random() < 0.3 else h + int(rng.integers(0, 2 * room // batch + 2)) for h in held]
    need = sum(max(0, -(-w // block) - -(-h // block)) for h, w in zip(held, want))
    for share in (1.0, 0.5):
        m = Map(held, block, free=max(1, int(need * share)), width=-(-max(held + want) // block) + 1, room=room, seed=7)
        m.check(want, in_place)


def test_block_map_many_steps_give_and_take():
    # forty steps of one pool, its state carried on the device; the queue wraps around several times
    rng = np.random.default_rng(4)
    m = Map([0] * 12, 16, free=30, width=12, room=256)
    for _ in range(40):
        want = [0 if rng.random() < 0.15 else min(180, h + int(rng.integers(0, 30))) for h in m.held]
        m.ws.zero_()
        ref = m.check(want, in_place=True)
        m.held, m.table, m.queue, m.pool = ref[0].tolist(), ref[1], ref[2], tuple(ref[3])
    # every block is in the queue or in one table, once
    owned = [int(m.table[b, j]) for b, h in enumerate(m.held) for j in range(-(-h // 16))]
    free = [int(m.queue[(m.pool[0] + i) % m.cap]) for i in range(m.pool[1])]
    assert sorted(owned + free) == list(range(m.cap))


def test_block_map_clamps_and_reports_what_is_out_of_range():
    m = Map([16, 16], 16, free=2, width=3, room=64)
    got = m.call([1000, -4])                  # wants 48 at most, and 0 at least
    assert got[0].tolist() == [48, 0]
    assert F.fdpp_read_error(m.ws) == F.FDPP_ERRBIT_SEQ_LEN
    m = Map([16], 16, free=2, width=3, room=64)
    m.d["pool"].copy_(_dev([-3, 1000]))
    m.call([17])
    assert F.fdpp_read_error(m.ws) & F.FDPP_ERRBIT_POOL
    m = Map([16], 16, free=2, width=3, room=64)
    m.d["table"][0, 0] = 99                   # an entry outside the pool, freed and used
    got = m.call([20])
    assert F.fdpp_read_error(m.ws) == 0       # the new tokens lie in the block granted
    m.d["held"].fill_(10)
    got = m.call([14])
    assert got[7][:4].tolist() == [-1] * 4 and F.fdpp_read_error(m.ws) == F.FDPP_ERRBIT_BLOCK_TABLE


def test_block_map_in_a_graph():
    m = Map([100, 7, 31], 16, free=20, width=20, room=32)
    want = [101, 8, 32]
    want_d = _dev(want)
    d = m.d
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    args = (d["held"], want_d, d["pool"], m.p, d["table"], d["queue"], d["held"], d["pool"], d["cu"], d["seq"], d["pos"],
            d["slots"], m.ws)
    with torch.cuda.stream(s):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            F.fdpp_block_map(*args)
    torch.cuda.synchronize()
    held, table, queue, pool = m.held, m.table, m.queue, m.pool
    for step in range(20):
        want_d.copy_(_dev([h + 1 for h in held]))
        g.replay()
        ref = R.block_map(held, [h + 1 for h in held], pool, table, queue, 16, 32)
        held, table, queue, pool = ref[0].tolist(), ref[1], ref[2], tuple(ref[3])
        np.testing.assert_array_equal(d["slots"].cpu().numpy(), ref[7])
        np.testing.assert_array_equal(d["table"].cpu().numpy(), table)
    assert F.fdpp_read_error(m.ws) == 0


# ---- rotary append -----------------------------------------------------------------------------

def _rope_case(T, hq, hkv, d, dtype, rot, inter, scaling="plain", factor=1.0, context=0, magnitude=1.0, far=4096, pad=0,
               base=10000.0, seed=1, joint=True, positions=None):
    rng = np.random.default_rng(seed)
    gen = torch.Generator().manual_seed(seed)
    row = (hq + 2 * hkv) * d
    qkv = torch.randn(T, row, generator=gen).to(TYPES[dtype])
    slots_n = T + 11
    slots = rng.permutation(slots_n)[:T].astype(np.int64)
    if pad:
        slots[rng.permutation(T)[:pad]] = -1
    pos = rng.integers(0, far, T).astype(np.int32) if positions is None else np.asarray(positions, np.int32)
    x = qkv.cuda()
    parts = [x[:, :hq * d], x[:, hq * d:(hq + hkv) * d], x[:, (hq + hkv) * d:]]
    strides = [row] * 3
    if not joint:
        parts, strides = [y.contiguous() for y in parts], [hq * d, hkv * d, hkv * d]
    fill = 7.0
    q_out = torch.full((T, hq, d), fill, dtype=TYPES[dtype], device="cuda")
    kc, vc = (torch.full((slots_n, hkv, d), fill, dtype=TYPES[dtype], device="cuda") for _ in range(2))
    kinds = dict(plain=F.FDPP_ROPE_PLAIN, linear=F.FDPP_ROPE_LINEAR, ntk=F.FDPP_ROPE_NTK, parts=F.FDPP_ROPE_PARTS)
    table = torch.as_tensor(F.fdpp_rope_table(rot, base, scaling=kinds[scaling], factor=factor, context=context)).cuda()
    p = F.make_rope_params(num_tokens=T, num_q_heads=hq, num_kv_heads=hkv, head_dim=d, rot_dim=rot, interleaved=inter,
                           dtype=F.FDPP_BF16 if dtype == "bf16" else F.FDPP_F32, num_slots=slots_n, q_stride=strides[0],
                           k_stride=strides[1], v_stride=strides[2], magnitude=magnitude)
    ws = F.alloc_rope_workspace()
    F.fdpp_rope_append(parts[0], parts[1], parts[2], _dev(pos), _dev(slots, np.int64), table, p, q_out, kc, vc, ws)
    torch.cuda.synchronize()
    assert F.fdpp_read_error(ws) == 0
    theta = R.rope_theta(rot, base, scaling, factor, context)
    h = qkv.double().numpy().reshape(T, hq + 2 * hkv, d)
    q, k, v = h[:, :hq], h[:, hq:hq + hkv], h[:, hq + hkv:]
    live = slots >= 0
    eps = float(torch.finfo(TYPES[dtype]).eps)

    def close(got, ref, src, what):
        half = rot // 2
        a, b = (np.arange(0, rot, 2), np.arange(1, rot, 2)) if inter else (np.arange(half), half + np.arange(half))
        pair = np.zeros_like(src)
        pair[:, :, a] = pair[:, :, b] = np.hypot(src[:, :, a], src[:, :, b])
        err = np.abs(got - ref)
        angle = 2.0 ** -49 * np.abs(pos.astype(np.float64))[live, None, None]
        bound = eps / 2 * np.abs(ref) + (2.0 ** -19 + angle) * magnitude * pair
        assert (err <= bound).all(), f"{what}: {(err - bound).max():.3e} over"

    got_q, got_k, got_v = (t.double().cpu().numpy() for t in (q_out, kc, vc))
    close(got_q[live], R.rope(q, pos, theta, inter, magnitude)[live], q[live], "q")
    close(got_k[slots[live]], R.rope(k, pos, theta, inter, magnitude)[live], k[live], "k")
    np.testing.assert_array_equal(got_v[slots[live]], v[live])
    # nothing else is written
    rest = np.ones(slots_n, bool)
    rest[slots[live]] = False
    assert (got_k[rest] == fill).all() and (got_v[rest] == fill).all() and (got_q[~live] == fill).all()


ROPES = [
    dict(T=1, hq=1, hkv=1, d=64, dtype="bf16", rot=64, inter=False),
    dict(T=5, hq=8, hkv=2, d=128, dtype="bf16", rot=128, inter=False, pad=2),
    dict(T=5, hq=8, hkv=2, d=128, dtype="bf16", rot=128, inter=True, pad=1),
    dict(T=9, hq=7, hkv=1, d=128, dtype="bf16", rot=32, inter=False, joint=False),
    dict(T=9, hq=7, hkv=7, d=64, dtype="bf16", rot=48, inter=True, scaling="linear", factor=4.0),
    dict(T=3, hq=4, hkv=4, d=64, dtype="f32", rot=16, inter=True, scaling="ntk", factor=3.0),
    dict(T=17, hq=6, hkv=3, d=128, dtype="f32", rot=96, inter=False, scaling="parts", factor=8.0, context=2048,
         magnitude=1.2, far=20000, pad=5),
    dict(T=2500, hq=3, hkv=1, d=128, dtype="bf16", rot=128, inter=False, far=1000000, pad=100),
    dict(T=700, hq=64, hkv=8, d=128, dtype="bf16", rot=112, inter=True, scaling="parts", factor=2.0, context=8192),
]


@pytest.mark.parametrize("case", ROPES, ids=lambda c: f"T{c['T']}-{c['hq']}q{c['hkv']}-d{c['d']}-{c['dtype']}-r{c['rot']}"
                         f"-{'inter' if c['inter'] else 'half'}-{c.get('scaling', 'plain')}")
def test_rope_append(case):
    case = dict(case)
    pad = case.pop("pad", 0)
    _rope_case(pad=pad, **case)


def test_rope_far_and_negative_positions():
    # angles at the ends of int32 are off by no more than the table is
    _rope_case(T=8, hq=2, hkv=2, d=64, dtype="f32", rot=64, inter=False,
               positions=[0, 1, 4095, 4096, 16777217, 2 ** 31 - 1, -1, -2 ** 31])


def test_rope_in_place_and_slots_out_of_range():
    T, h, d = 6, 4, 64
    gen = torch.Generator().manual_seed(3)
    q = torch.randn(T, h, d, generator=gen).cuda()
    k, v = torch.randn(T, h, d, generator=gen).cuda(), torch.randn(T, h, d, generator=gen).cuda()
    table = torch.as_tensor(F.fdpp_rope_table(64, 10000.0)).cuda()
    p = F.make_rope_params(num_tokens=T, num_q_heads=h, num_kv_heads=h, head_dim=d, rot_dim=64, dtype=F.FDPP_F32,
                           num_slots=4)
    pos = np.arange(T)
    kc, vc = torch.zeros(5, h, d).cuda(), torch.zeros(5, h, d).cuda()
    ws = F.alloc_rope_workspace()
    q0 = q.double().cpu().numpy()
    F.fdpp_rope_append(q, k, v, _dev(pos), _dev([0, 1, 2, 3, 4, 2 ** 40], np.int64), table, p, q, kc, vc, ws)
    torch.cuda.synchronize()
    assert F.fdpp_read_error(ws) == F.FDPP_ERRBIT_SLOT
    assert (kc[4] == 0).all() and (vc[4] == 0).all()
    ref = R.rope(q0, pos, R.rope_theta(64, 10000.0), False, 1.0)
    assert np.abs(q.double().cpu().numpy() - ref).max() < 2.0 ** -18 * np.abs(q0).max() * 2


def test_rope_without_tokens_does_nothing():
    p = F.make_rope_params(num_tokens=0, num_q_heads=1, num_kv_heads=1, head_dim=64, rot_dim=64, dtype=F.FDPP_F32,
                           num_slots=1)
    x = torch.zeros(1, 1, 64).cuda()
    i = _dev([0])
    F.fdpp_rope_append(x, x, x, i, _dev([0], np.int64), torch.zeros(32, 2).cuda(), p, x.clone(), x.clone(), x.clone(),
                       F.alloc_rope_workspace())
    torch.cuda.synchronize()
