"""What is measured of the operators around the attention step, and their plain forms.

Four operators that a serving step needs next to decode attention: the block map (block tables and
slot maps from request lengths), rotary positions with the append to the cache, attention of any
number of query tokens with capped or biased scores and key ranges, and attention for a batch that
shares a long prefix. ``run`` computes one of them, in plain torch operations in 32 bits (angles in
64) or, where ``own`` is true, through the library's entry points. ``exact`` computes the same from
the definitions in 64 bits.

A case is a dict of plain values; ``shape`` seeds the lengths, document borders and other sizes of
a case, so that they belong to the case, while ``prepare``'s seed makes the values.
"""
import math
import random

import numpy as np
import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---- cases -------------------------------------------------------------------------------------

def listed():
    cases = [
        # one tick of a paged continuous batch: every sequence grows by one token
        dict(name="map tick", op="map", batch=64, block=16, lo=512, hi=16384, new_lo=1, new_hi=1,
             stop=0, spare=64, room=64, shape=1),
        # a scheduler's mixed step: prompts of any length join, some sequences end, the pool and
        # the token rows are padded to fixed sizes as a captured step has them
        dict(name="map prompts", op="map", batch=512, block=16, lo=0, hi=2048, new_lo=1, new_hi=255,
             stop=20, spare=4096, room=81920, shape=2),
        # the decode step of the paged batch: 64 tokens, three of them padding rows
        dict(name="rope tick", op="rope", tokens=64, live=61, hq=64, hkv=8, d=128, type="bf16",
             rot=128, inter=False, scaling="plain", base=10000.0, factor=1.0, context=0,
             magnitude=1.0, far=16384),
        # a long prompt's keys and values on their way into the cache, positions stretched for a
        # context beyond the one trained on
        dict(name="rope prompt", op="rope", tokens=16384, live=16384, hq=32, hkv=8, d=128,
             type="bf16", rot=128, inter=False, scaling="parts", base=500000.0, factor=8.0,
             context=8192, magnitude=1.2079, far=131072),
        # small fp32 model, half of each head rotated, neighbouring elements paired
        dict(name="rope f32 part", op="rope", tokens=777, live=777, hq=4, hkv=4, d=64, type="f32",
             rot=32, inter=True, scaling="linear", base=10000.0, factor=4.0, context=0,
             magnitude=1.0, far=4096),
        # the paged continuous batch's decode step with capped scores
        dict(name="rows tick cap", op="rows", batch=64, hq=64, hkv=8, d=128, type="bf16", block=16,
             new_lo=1, new_hi=1, old_lo=511, old_hi=16383, cap=30.0, bias=False, mask="causal",
             prefix=0, shape=3),
        # one long prompt with a penalty on distance
        dict(name="rows prompt bias", op="rows", batch=1, hq=32, hkv=8, d=128, type="bf16",
             block=16, new_lo=8192, new_hi=8192, old_lo=0, old_hi=0, cap=0.0, bias=True,
             mask="causal", prefix=0, shape=4),
        # a ragged batch of packed documents: a token sees its own document only
        dict(name="rows documents", op="rows", batch=5, hq=16, hkv=2, d=64, type="bf16", block=0,
             new_lo=333, new_hi=1500, old_lo=0, old_hi=77, cap=0.0, bias=False, mask="document",
             prefix=0, shape=5),
        # the smallest attention call: four heads, fp32, 256 keys, distance bias
        dict(name="rows f32 tiny", op="rows", batch=1, hq=4, hkv=4, d=64, type="f32", block=0,
             new_lo=1, new_hi=1, old_lo=255, old_hi=255, cap=0.0, bias=True, mask="causal",
             prefix=0, shape=6),
        # a batch behind one long shared prompt, each with its own short continuation
        dict(name="prefix tick", op="rows", batch=64, hq=64, hkv=8, d=128, type="bf16", block=16,
             new_lo=1, new_hi=1, old_lo=0, old_hi=511, cap=0.0, bias=False, mask="causal",
             prefix=16384, shape=7),
        # eight sequences, a shared prompt of odd length, contiguous caches, a few tokens each as
        # speculative decoding has them
        dict(name="prefix tokens", op="rows", batch=8, hq=32, hkv=8, d=128, type="bf16", block=0,
             new_lo=2, new_hi=4, old_lo=1, old_hi=200, cap=50.0, bias=False, mask="causal",
             prefix=4001, shape=8),
        # the same in fp32, small
        dict(name="prefix f32", op="rows", batch=4, hq=8, hkv=4, d=64, type="f32", block=0,
             new_lo=1, new_hi=1, old_lo=0, old_hi=63, cap=0.0, bias=True, mask="causal",
             prefix=500, shape=9),
    ]
    return cases


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(("map", "rope", "rows", "rows", "prefix", "prefix"))
    shape = rng.randrange(1 << 30)
    if kind == "map":
        batch = _log(rng, 1, 1024)
        hi = _log(rng, 1, 16384)
        new_hi = min(_log(rng, 1, 2048), max(1, 65536 // batch))
        return dict(op="map", batch=batch, block=rng.choice((16, 32, 64, 128, 256)),
                    lo=rng.randrange(0, hi + 1), hi=hi, new_lo=rng.randrange(0, 2), new_hi=new_hi,
                    stop=rng.choice((0, 10, 50)), spare=_log(rng, 1, 4096),
                    room=_log(rng, max(1, batch * new_hi // 4), 2 * batch * new_hi + 16), shape=shape)
    d = rng.choice((64, 128))
    kind_type = "bf16" if rng.random() < 0.8 else "f32"
    hkv = rng.choice((1, 2, 4, 8))
    group = rng.choice((1, 2, 3, 4, 7, 8))
    if kind == "rope":
        tokens = _log(rng, 1, 12000)
        scaling = rng.choice(("plain", "linear", "ntk", "parts"))
        return dict(op="rope", tokens=tokens, live=tokens - rng.randrange(0, 1 + tokens // 8),
                    hq=hkv * group, hkv=hkv, d=d, type=kind_type,
                    rot=rng.choice((16, 32, 48, 64) if d == 64 else (32, 64, 96, 128)),
                    inter=rng.random() < 0.5, scaling=scaling, base=rng.choice((10000.0, 500000.0)),
                    factor=1.0 if scaling == "plain" else rng.choice((2.0, 4.0, 8.0)),
                    context=rng.choice((2048, 8192)), magnitude=rng.choice((1.0, 1.1386)),
                    far=_log(rng, 1024, 1000000))
    prefix = _log(rng, 64, 16384) if kind == "prefix" else 0
    mask = rng.choice(("causal", "causal", "document", "prefix", "window"))
    cap = rng.choice((0.0, 0.0, 20.0, 50.0))
    bias = rng.random() < 0.35
    block = rng.choice((0, 16, 32, 64, 128, 256))
    if kind_type == "f32":      # the CUDA-core kernel: short contexts
        batch, new_hi, old_hi, prefix = _log(rng, 1, 8), rng.choice((1, 1, 3)), _log(rng, 1, 2048), min(prefix, 2048)
    elif rng.random() < 0.5:    # decode and speculative steps
        batch, new_hi, old_hi = _log(rng, 1, 64), rng.choice((1, 1, 1, 2, 4, 9)), _log(rng, 1, 8192)
    else:                       # prompts
        batch, new_hi, old_hi = _log(rng, 1, 6), _log(rng, 16, 3000), _log(rng, 1, 2000)
        prefix = min(prefix, 4096)
    return dict(op="rows", batch=batch, hq=hkv * group, hkv=hkv, d=d, type=kind_type, block=block,
                new_lo=rng.randrange(1, new_hi + 1), new_hi=new_hi, old_lo=rng.randrange(0, old_hi + 1),
                old_hi=old_hi, cap=cap, bias=bias, mask=mask, prefix=prefix, shape=shape)


# ---- sizes that belong to a case ---------------------------------------------------------------

def _map_shape(case):
    """(tokens held, tokens wanted) of each sequence."""
    r = random.Random(case["shape"])
    held = [r.randint(case["lo"], case["hi"]) for _ in range(case["batch"])]
    want = [0 if r.randrange(100) < case["stop"] else h + r.randint(case["new_lo"], case["new_hi"]) for h in held]
    return held, want


def _blocks(n, block):
    return -(-n // block)


def _rows_shape(case):
    """(new tokens, own keys) of each sequence, and each token's key range [begin, end), its
    position and its sequence. Positions count the shared prefix first."""
    r = random.Random(case["shape"])
    n = [r.randint(case["new_lo"], case["new_hi"]) for _ in range(case["batch"])]
    keys = [x + r.randint(case["old_lo"], case["old_hi"]) for x in n]
    P = case["prefix"]
    begin, end, pos, seq = [], [], [], []
    for b, (x, L) in enumerate(zip(n, keys)):
        total = P + L
        p = np.arange(total - x, total)
        lo, hi = np.zeros(x, np.int64), p + 1
        if case["mask"] == "document":      # borders anywhere; now and then a token of no document
            borders = sorted({0} | {r.randrange(total) for _ in range(1 + total // 700)})
            lo = np.asarray(borders)[np.searchsorted(borders, p, side="right") - 1]
            nothing = np.asarray([r.randrange(40) == 0 for _ in range(x)])
            lo, hi = np.where(nothing, 3, lo), np.where(nothing, 3, hi)
        elif case["mask"] == "prefix":      # the first part of the new tokens sees itself whole
            hi = np.maximum(hi, min(total, total - x + r.randint(1, x)))
        elif case["mask"] == "window":
            lo = np.maximum(0, p + 1 - r.choice((16, 100, 512, 1024)))
        begin.append(lo), end.append(hi), pos.append(p), seq.append(np.full(x, b))
    return n, keys, np.concatenate(begin), np.concatenate(end), np.concatenate(pos), np.concatenate(seq)


def _frequencies(case):
    """Angle per position of each pair, in 64 bits."""
    rot, base, f = case["rot"], case["base"], case["factor"]
    if case["scaling"] == "ntk":
        base = base * f ** (rot / (rot - 2))
    theta = base ** (-2.0 * np.arange(rot // 2, dtype=np.float64) / rot)
    if case["scaling"] == "linear":
        theta = theta / f
    if case["scaling"] == "parts":      # pairs that turn often in the context keep their angle
        turns = case["context"] * theta / (2 * math.pi)
        keep = np.clip((turns - 1.0) / (32.0 - 1.0), 0.0, 1.0)
        theta = theta * (keep + (1 - keep) / f)
    return theta


def work(case):
    if case["op"] == "map":
        held, want = _map_shape(case)
        new = sum(max(0, w - h) for h, w in zip(held, want))
        moved = sum(abs(_blocks(w, case["block"]) - _blocks(h, case["block"])) for h, w in zip(held, want))
        return dict(bytes=4 * (4 * case["batch"] + 5) + 8 * moved + 16 * max(case["room"], min(new, case["room"])), flops=0)
    size = 2 if case["type"] == "bf16" else 4
    if case["op"] == "rope":
        rows = case["hq"] + 2 * case["hkv"]
        turned = case["live"] * (case["hq"] + case["hkv"]) * case["rot"]
        return dict(bytes=case["live"] * (2 * rows * case["d"] * size + 12), flops=3 * turned)
    n, keys, begin, end, _, seq = _rows_shape(case)
    visible = int(np.maximum(0, end - begin).sum())
    P, tokens = case["prefix"], int(sum(n))
    # a key is read once for each kv head if any of its sequence's tokens sees it
    first = np.full(len(n), 1 << 40, np.int64)
    last = np.zeros(len(n), np.int64)
    some = end > begin
    np.minimum.at(first, seq[some], begin[some])
    np.maximum.at(last, seq[some], end[some])
    own_keys = int(np.maximum(0, last - np.maximum(first, P)).sum())
    shared = max(0, min(P, int(last.max(initial=0))) - int(min(first.min(initial=1 << 40), P)))
    row = case["d"] * size
    return dict(bytes=2 * tokens * case["hq"] * row + 2 * (own_keys + shared) * case["hkv"] * row,
                flops=4 * visible * case["hq"] * case["d"])


# ---- inputs ------------------------------------------------------------------------------------

def _randn(gen, *size, type="bf16"):
    return torch.randn(size, generator=gen, device="cuda", dtype=TYPES[type])


def _int32(a):
    return torch.as_tensor(np.asarray(a, dtype=np.int32)).cuda()


def prepare(case, seed):
    gen = torch.Generator("cuda").manual_seed(seed)
    perm = np.random.default_rng(seed)
    return {"map": _prepare_map, "rope": _prepare_rope, "rows": _prepare_rows}[case["op"]](case, gen, perm)


def _prepare_map(case, gen, perm):
    held, want = _map_shape(case)
    block, B = case["block"], case["batch"]
    used = [_blocks(h, block) for h in held]
    need = sum(max(0, _blocks(w, block) - u) for w, u in zip(want, used))
    # the pool is sometimes short: `spare` blocks are free besides half of what is asked for
    free = case["spare"] + need // 2
    pool = sum(used) + free
    width = max(max(used), max(_blocks(w, block) for w in want)) + 1
    ids = perm.permutation(pool).astype(np.int32)
    table = np.full((B, width), -1, np.int32)
    at = 0
    for b, u in enumerate(used):
        table[b, :u] = ids[at:at + u]
        at += u
    head = int(perm.integers(pool))
    queue = np.full(pool, -1, np.int32)
    queue[(head + np.arange(free)) % pool] = ids[at:]
    s = dict(case=case, held=_int32(held), want=_int32(want), table=_int32(table), queue=_int32(queue),
             pool=_int32([head, free]), lens=_int32(held), pool_out=_int32([0, 0]),
             cu=_int32(np.zeros(B + 1)), seq=_int32(np.zeros(case["room"])), pos=_int32(np.zeros(case["room"])),
             slots=torch.zeros(case["room"], dtype=torch.int64, device="cuda"))
    if own:
        import split_kv_async_gb300 as F
        s["p"] = F.make_block_params(batch=B, block_size=block, max_blocks_per_seq=width,
                                     num_kv_blocks=pool, max_tokens=case["room"])
        s["ws"] = F.alloc_block_workspace(s["p"])
    return s


def _prepare_rope(case, gen, perm):
    T, hq, hkv, d = case["tokens"], case["hq"], case["hkv"], case["d"]
    qkv = _randn(gen, T, (hq + 2 * hkv) * d, type=case["type"])      # one projection's output
    slots_n = T + 37
    slots = perm.permutation(slots_n)[:T].astype(np.int64)
    slots[case["live"]:] = -1                                         # rows of padding
    s = dict(case=case, qkv=qkv, q=qkv[:, :hq * d].unflatten(1, (hq, d)),
             k=qkv[:, hq * d:(hq + hkv) * d].unflatten(1, (hkv, d)),
             v=qkv[:, (hq + hkv) * d:].unflatten(1, (hkv, d)),
             pos=_int32(perm.integers(0, case["far"], T)), slots=torch.as_tensor(slots).cuda(),
             q_out=torch.zeros(T, hq, d, dtype=TYPES[case["type"]], device="cuda"),
             k_cache=torch.zeros(slots_n, hkv, d, dtype=TYPES[case["type"]], device="cuda"),
             v_cache=torch.zeros(slots_n, hkv, d, dtype=TYPES[case["type"]], device="cuda"))
    if own:
        import split_kv_async_gb300 as F
        scaling = dict(plain=F.FDPP_ROPE_PLAIN, linear=F.FDPP_ROPE_LINEAR, ntk=F.FDPP_ROPE_NTK,
                       parts=F.FDPP_ROPE_PARTS)[case["scaling"]]
        s["table"] = torch.as_tensor(F.fdpp_rope_table(case["rot"], case["base"], scaling=scaling,
                                                       factor=case["factor"], context=case["context"],
                                                       low_turns=1.0, high_turns=32.0)).cuda()
        row = (hq + 2 * hkv) * d
        s["p"] = F.make_rope_params(num_tokens=T, num_q_heads=hq, num_kv_heads=hkv, head_dim=d,
                                    rot_dim=case["rot"], interleaved=case["inter"],
                                    dtype=F.FDPP_BF16 if case["type"] == "bf16" else F.FDPP_F32,
                                    q_stride=row, k_stride=row, v_stride=row, num_slots=slots_n,
                                    magnitude=case["magnitude"])
        s["ws"] = F.alloc_rope_workspace()
    else:
        s["theta"] = torch.as_tensor(_frequencies(case)).cuda()
    return s


def _prepare_rows(case, gen, perm):
    n, keys, begin, end, pos, seq = _rows_shape(case)
    B, hq, hkv, d, P, block = (case[x] for x in ("batch", "hq", "hkv", "d", "prefix", "block"))
    T, longest = int(sum(n)), max(keys)
    cu = np.concatenate([[0], np.cumsum(n)])
    s = dict(case=case, n_max=max(n), longest=longest, q=_randn(gen, T, hq, d, type=case["type"]),
             out=torch.zeros(T, hq, d, dtype=TYPES[case["type"]], device="cuda"),
             cu=_int32(cu), lens=_int32(keys), plen=_int32([P]), begin=None, end=None, slopes=None,
             table=None, prefix_table=None, prefix_k=None, prefix_v=None)
    if case["mask"] != "causal":
        s["begin"], s["end"] = _int32(begin), _int32(end)
    if case["bias"]:
        s["slopes"] = torch.as_tensor(np.asarray([2.0 ** (-8.0 * (h + 1) / hq) for h in range(hq)], np.float32)).cuda()
    if block:
        used, shared = [_blocks(L, block) for L in keys], _blocks(P, block)
        blocks = sum(used) + shared
        ids = perm.permutation(blocks).astype(np.int32)
        table = np.full((B, max(used)), -1, np.int32)
        at = shared
        for b, u in enumerate(used):
            table[b, :u] = ids[at:at + u]
            at += u
        s["table"], s["blocks"] = _int32(table), blocks
        if P:
            s["prefix_table"] = _int32(ids[:shared])
        size = (blocks, block, hkv, d)
    else:
        size = (B, longest, hkv, d)
        if P:
            s["prefix_k"] = _randn(gen, P, hkv, d, type=case["type"])
            s["prefix_v"] = _randn(gen, P, hkv, d, type=case["type"])
    s["k"], s["v"] = _randn(gen, *size, type=case["type"]), _randn(gen, *size, type=case["type"])
    # rows of a padded batch, for the plain form: token (b, i), or the first one where there is none
    b, i = np.divmod(np.arange(B * max(n)), max(n))
    s["row"] = torch.as_tensor(np.where(i < np.asarray(n)[b], cu[b] + i, 0)).cuda()
    s["flat"] = torch.as_tensor(seq * max(n) + np.arange(T) - cu[seq]).cuda()
    s["pos"] = torch.as_tensor(pos).cuda()
    if own:
        import split_kv_async_gb300 as F
        s["p"] = F.make_rows_params(batch=B, num_q_heads=hq, num_kv_heads=hkv, head_dim=d,
                                    dtype=F.FDPP_BF16 if case["type"] == "bf16" else F.FDPP_F32,
                                    num_tokens=T, max_seq_len=longest, scale=d ** -0.5, softcap=case["cap"],
                                    slopes=s["slopes"], key_begin=s["begin"], key_end=s["end"],
                                    block_size=block, max_blocks_per_seq=s["table"].shape[1] if block else 0,
                                    num_kv_blocks=s["blocks"] if block else 0, max_prefix_len=P)
        s["ws"] = F.alloc_rows_workspace(s["p"])
    return s


# ---- one pass ----------------------------------------------------------------------------------

def run(s):
    return {"map": _run_map, "rope": _run_rope, "rows": _run_rows}[s["case"]["op"]](s)


def _run_map(s):
    if own:
        import split_kv_async_gb300 as F
        F.fdpp_block_map(s["held"], s["want"], s["pool"], s["p"], s["table"], s["queue"], s["lens"], s["pool_out"],
                         s["cu"], s["seq"], s["pos"], s["slots"], s["ws"])
        return s["lens"], s["table"], s["queue"], s["pool_out"], s["cu"], s["seq"], s["pos"], s["slots"]
    case = s["case"]
    block, room, cap = case["block"], case["room"], s["queue"].numel()
    held, want = s["held"].long(), s["want"].long()
    head, count = s["pool"][0].long(), s["pool"][1].long()
    old, new = (held + block - 1) // block, (want + block - 1) // block
    need, back, tokens = (new - old).clamp(min=0), (old - new).clamp(min=0), (want - held).clamp(min=0)
    # in order: a sequence is served if the blocks and the rows asked for up to it are there
    served = ((need.cumsum(0) <= count) | (need == 0)) & ((tokens.cumsum(0) <= room) | (tokens == 0))
    lens, need, tokens = torch.where(served, want, held), need * served, tokens * served
    col = torch.arange(s["table"].shape[1], device="cuda")[None]
    first = (need.cumsum(0) - need)[:, None]
    grown = (col >= old[:, None]) & (col < (old + need)[:, None])
    table = torch.where(grown, s["queue"][(head + first + col - old[:, None]) % cap], s["table"])
    freed = (col >= new[:, None]) & (col < old[:, None])
    to = head + count + (back.cumsum(0) - back)[:, None] + col - new[:, None]
    queue = torch.cat([s["queue"], s["queue"][:1]])
    queue.scatter_(0, torch.where(freed, to % cap, cap).reshape(-1), s["table"].reshape(-1))
    taken, given = need.sum(), back.sum()
    pool = torch.stack([(head + taken) % cap, count - taken + given]).int()
    cu = torch.cat([tokens.new_zeros(1), tokens.cumsum(0)])
    r = torch.arange(room, device="cuda")
    seq = torch.searchsorted(cu[1:].contiguous(), r, right=True)
    live = r < cu[-1]
    b = seq.clamp(max=held.numel() - 1)
    pos = held[b] + r - cu[b]
    at = (pos // block).clamp(0, table.shape[1] - 1)
    slots = table[b, at].long() * block + pos % block
    return (lens.int(), table, queue[:-1], pool, cu.int(), torch.where(live, seq, -1).int(),
            torch.where(live, pos, 0).int(), torch.where(live, slots, -1))


def _turn(x, cos, sin, rot, inter):
    """x [T][heads][d] with its first `rot` elements turned in pairs."""
    x = x.float()
    a, b = (x[..., :rot:2], x[..., 1:rot:2]) if inter else (x[..., :rot // 2], x[..., rot // 2:rot])
    a, b = a * cos - b * sin, a * sin + b * cos
    turned = torch.stack([a, b], -1).flatten(-2) if inter else torch.cat([a, b], -1)
    return torch.cat([turned, x[..., rot:]], -1)


def _run_rope(s):
    if own:
        import split_kv_async_gb300 as F
        F.fdpp_rope_append(s["q"], s["k"], s["v"], s["pos"], s["slots"], s["table"], s["p"], s["q_out"], s["k_cache"],
                           s["v_cache"], s["ws"])
        return s["q_out"], s["k_cache"], s["v_cache"]
    case = s["case"]
    angle = s["pos"].double()[:, None, None] * s["theta"]
    cos = (angle.cos() * case["magnitude"]).float()
    sin = (angle.sin() * case["magnitude"]).float()
    live = case["live"]
    to = s["slots"][:live]
    s["q_out"][:live] = _turn(s["q"], cos, sin, case["rot"], case["inter"])[:live].to(s["q_out"].dtype)
    s["k_cache"][to] = _turn(s["k"], cos, sin, case["rot"], case["inter"])[:live].to(s["k_cache"].dtype)
    s["v_cache"][to] = s["v"][:live]
    return s["q_out"], s["k_cache"], s["v_cache"]


def _run_rows(s):
    case = s["case"]
    if own:
        import split_kv_async_gb300 as F
        if case["prefix"]:
            F.fdpp_prefix_attn(s["q"], s["prefix_k"], s["prefix_v"], s["prefix_table"], s["plen"], s["k"], s["v"],
                               s["table"], s["lens"], s["cu"], s["p"], s["ws"], s["out"])
        else:
            F.fdpp_rows_attn(s["q"], s["k"], s["v"], s["table"], s["lens"], s["cu"], s["p"], s["ws"], s["out"])
        return s["out"]
    B, hq, hkv, d, P = (case[x] for x in ("batch", "hq", "hkv", "d", "prefix"))
    n, L, G = s["n_max"], s["longest"], hq // hkv
    if s["table"] is not None:
        k = s["k"][s["table"].long()].flatten(1, 2)[:, :L]
        v = s["v"][s["table"].long()].flatten(1, 2)[:, :L]
    else:
        k, v = s["k"], s["v"]
    k, v = k.float().permute(0, 2, 1, 3), v.float().permute(0, 2, 1, 3)           # [B][hkv][L][d]
    q = s["q"][s["row"]].float().reshape(B, n, hkv, G, d).permute(0, 2, 1, 3, 4)   # [B][hkv][n][G][d]
    scores = (q.reshape(B, hkv, n * G, d) @ k.transpose(2, 3)).reshape(B, hkv, n, G, L)
    if P:       # the shared keys against every row of the batch at once
        pk = s["prefix_k"] if s["table"] is None else s["k"][s["prefix_table"].long()].flatten(0, 1)[:P]
        pv = s["prefix_v"] if s["table"] is None else s["v"][s["prefix_table"].long()].flatten(0, 1)[:P]
        pk, pv = pk.float().transpose(0, 1), pv.float().transpose(0, 1)            # [hkv][P][d]
        rows = q.transpose(0, 1).reshape(hkv, B * n * G, d)
        shared = (rows @ pk.transpose(1, 2)).reshape(hkv, B, n, G, P).transpose(0, 1)
        scores = torch.cat([shared, scores], -1)
    scores = scores * d ** -0.5
    if case["cap"]:
        scores = case["cap"] * torch.tanh(scores / case["cap"])
    t = torch.arange(P + L, device="cuda")
    pos = s["pos"][s["row"]].reshape(B, n, 1)
    if s["slopes"] is not None:
        distance = (pos - t).abs().float()
        scores = scores - s["slopes"].reshape(hkv, 1, G, 1) * distance[:, None, :, None]
    if s["begin"] is not None:
        seen = (t >= s["begin"][s["row"]].reshape(B, n, 1)) & (t < s["end"][s["row"]].reshape(B, n, 1))
    else:
        seen = t <= pos
    seen = (seen & (t < P + s["lens"].long().reshape(B, 1, 1)))[:, None, :, None]
    scores = torch.where(seen, scores, float("-inf"))
    most = scores.amax(-1, keepdim=True)
    p = torch.exp(scores - torch.where(most == float("-inf"), 0.0, most))
    total = p.sum(-1, keepdim=True)
    o = (p[..., P:].reshape(B, hkv, n * G, L) @ v).reshape(B, hkv, n, G, d)
    if P:
        o = o + (p[..., :P].transpose(0, 1).reshape(hkv, B * n * G, P) @ pv).reshape(hkv, B, n, G, d).transpose(0, 1)
    o = torch.where(total > 0, o / total, 0.0)
    o = o.permute(0, 2, 1, 3, 4).reshape(B * n, hq, d)
    return o[s["flat"]].to(s["q"].dtype)


# ---- the definitions, in 64 bits ---------------------------------------------------------------

def exact(case, seed):
    if case["op"] == "map":
        return None             # whole numbers only
    s = prepare(case, seed)
    return _exact_rope(case, s) if case["op"] == "rope" else _exact_rows(case, s)


def _exact_rope(case, s):
    """Each pair is a complex number; a position multiplies it by magnitude exp(i angle)."""
    rot, half, live = case["rot"], case["rot"] // 2, case["live"]
    i = torch.arange(half, device="cuda")
    first, second = (2 * i, 2 * i + 1) if case["inter"] else (i, i + half)
    angle = torch.outer(s["pos"].double(), torch.as_tensor(_frequencies(case)).cuda())[:live]
    factor = torch.polar(torch.full_like(angle, case["magnitude"]), angle)[:, None, :]

    def turned(x):
        x = x[:live].double()
        z = torch.complex(x[..., first], x[..., second]) * factor
        x[..., first], x[..., second] = z.real, z.imag
        return x

    q_out, k_cache, v_cache = s["q_out"].double(), s["k_cache"].double(), s["v_cache"].double()
    slots = s["slots"][:live]
    q_out[:live] = turned(s["q"])
    k_cache[slots] = turned(s["k"])
    v_cache[slots] = s["v"][:live].double()
    return q_out, k_cache, v_cache


def _exact_rows(case, s):
    """Sequence by sequence and kv head by kv head: all keys of the sequence in a row."""
    hq, hkv, d, P = case["hq"], case["hkv"], case["d"], case["prefix"]
    G, block = hq // hkv, case["block"]
    n, keys, begin, end, pos, _ = _rows_shape(case)
    if int(np.maximum(end - begin, 0).sum()) * hq * d > 3e12:
        return None
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    begin, end, pos = (torch.as_tensor(x).cuda() for x in (begin, end, pos))
    at = 0
    for b, (x, L) in enumerate(zip(n, keys)):
        rows = slice(at, at + x)
        at += x
        t = torch.arange(P + L, device="cuda")
        if block:
            own_slots = s["table"][b].long()[torch.arange(L, device="cuda") // block] * block + torch.arange(L, device="cuda") % block
            slots = own_slots
            if P:
                u = torch.arange(P, device="cuda")
                slots = torch.cat([s["prefix_table"].long()[u // block] * block + u % block, own_slots])
            k_all, v_all = s["k"].reshape(-1, hkv, d)[slots], s["v"].reshape(-1, hkv, d)[slots]
        else:
            k_all, v_all = s["k"][b, :L], s["v"][b, :L]
            if P:
                k_all, v_all = torch.cat([s["prefix_k"], k_all]), torch.cat([s["prefix_v"], v_all])
        hidden = (t[None] < begin[rows][:, None]) | (t[None] >= end[rows][:, None])
        gap = (pos[rows][:, None] - t[None]).abs().double()
        for g in range(hkv):
            kg, vg = k_all[:, g].double(), v_all[:, g].double()
            for h in range(g * G, (g + 1) * G):
                z = s["q"][rows, h].double() @ kg.T / math.sqrt(d)
                if case["cap"]:
                    z = torch.tanh(z / case["cap"]) * case["cap"]
                if case["bias"]:
                    z = z - s["slopes"][h].double() * gap
                z = z.masked_fill(hidden, -math.inf)
                weight = torch.exp(z - torch.logsumexp(z, 1, keepdim=True))
                weight = weight.masked_fill(hidden, 0.0)
                out[rows, h] = weight @ vg
    return out
