"""What is measured of the operators that a step with drafted trees and 8-bit linears needs, and
their plain forms.

Four operators: the RMS norm with the residual's addition (output in the input's type, or in 8 bits
with a scale for every 128 channels), the linear layer in 8 bits with block scales, attention of a
tree of drafted tokens to a cache, and the commit of the tree's accepted path (its tokens' cache rows
move together in every layer). ``run`` computes one of them, in plain torch operations in 32 bits or,
where ``own`` is true, through the library's entry points. ``exact`` computes the same from the
definitions in 64 bits.

A case is a dict of plain values; ``shape`` seeds the trees, lengths and drafted tokens of a case, so
that they belong to the case, while ``prepare``'s seed makes the values.
"""
import math
import random

import numpy as np
import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32, "e4m3": torch.float8_e4m3fn}
GROUP = 128             # channels that share a scale
LARGEST = 448.0         # of e4m3
LEAST_SCALE = 2.0 ** -126


# ---- cases -------------------------------------------------------------------------------------

def listed():
    return [
        # one token on its way into an 8-bit linear: the smallest call of a decode step
        dict(name="norm token 8 bits", op="norm", tokens=1, dim=4096, type="bf16", out="e4m3", residual=True),
        # a long prompt's hidden states, residual added and written back
        dict(name="norm prompt 8 bits", op="norm", tokens=16384, dim=8192, type="bf16", out="e4m3", residual=True),
        # an fp32 model's last norm, an odd number of rows, channels that are no multiple of 128
        dict(name="norm f32 odd", op="norm", tokens=777, dim=1000, type="f32", out="f32", residual=False),
        # a decode step's attention output projection for eight sequences
        dict(name="linear 8 rows", op="linear", M=8, N=4096, K=4096, out="bf16"),
        # the wide projection of the MLP for the 64 tokens of a paged batch's step
        dict(name="linear 64 rows", op="linear", M=64, N=28672, K=4096, out="bf16"),
        # the same for a long prompt: bound by the tensor cores
        dict(name="linear prompt", op="linear", M=8192, N=28672, K=4096, out="bf16"),
        # a mixed step's odd number of rows into an fp32 output, ragged in every direction
        dict(name="linear odd", op="linear", M=333, N=1000, K=1040, out="f32"),
        # a paged continuous batch verifies a tree of 16 drafted tokens for each of 64 sequences
        dict(name="tree batch", op="tree", batch=64, hq=64, hkv=8, d=128, type="bf16", block=16, nodes_lo=16,
             nodes_hi=16, old_lo=512, old_hi=16384, cap=0.0, window=0, shape=11),
        # one sequence, a wide tree, capped scores
        dict(name="tree one", op="tree", batch=1, hq=32, hkv=8, d=128, type="bf16", block=0, nodes_lo=61,
             nodes_hi=61, old_lo=8000, old_hi=8000, cap=50.0, window=0, shape=12),
        # a small fp32 model with ragged trees
        dict(name="tree f32", op="tree", batch=3, hq=4, hkv=4, d=64, type="f32", block=16, nodes_lo=2, nodes_hi=9,
             old_lo=1, old_hi=300, cap=0.0, window=0, shape=13),
        # the batch's trees committed in the caches of 32 layers
        dict(name="commit batch", op="commit", batch=64, caches=64, hkv=8, d=128, type="bf16", block=16,
             nodes_lo=16, nodes_hi=16, old_lo=16, old_hi=160, match=85, shape=14),
        # one sequence of a small model
        dict(name="commit one", op="commit", batch=1, caches=4, hkv=2, d=64, type="bf16", block=0, nodes_lo=13,
             nodes_hi=13, old_lo=200, old_hi=200, match=90, shape=15),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("norm", "linear", "linear", "tree", "tree", "commit"))
    shape = rng.randrange(1 << 30)
    if op == "norm":
        dim = 8 * _log(rng, 8, 2048)
        kind = rng.choice(("bf16", "bf16", "f32"))
        return dict(op="norm", tokens=_log(rng, 1, max(1, min(32768, (1 << 26) // dim))), dim=dim, type=kind,
                    out=rng.choice((kind, "e4m3", "e4m3")), residual=rng.random() < 0.7)
    if op == "linear":
        K = 16 * _log(rng, 1, 896)
        N = _log(rng, 1, 28672)
        M = _log(rng, 1, max(1, min(8192, int(3e11) // (N * K)))) if rng.random() < 0.5 else _log(rng, 1, 128)
        return dict(op="linear", M=M, N=N, K=K, out=rng.choice(("bf16", "bf16", "f32")))
    d = rng.choice((64, 128))
    hkv = rng.choice((1, 2, 4, 8))
    kind = "bf16" if rng.random() < 0.8 else "f32"
    block = rng.choice((0, 16, 32, 64, 128, 256))
    hi = rng.choice((1, 4, 8, 16, 26, 64)) if rng.random() < 0.7 else _log(rng, 1, 256)
    lo = rng.randrange(1, hi + 1)
    if op == "tree":
        if kind == "f32":       # the CUDA-core kernel: short contexts
            batch, hi, old_hi = _log(rng, 1, 6), min(hi, 26), _log(rng, 1, 1500)
            lo = min(lo, hi)
        else:
            batch, old_hi = _log(rng, 1, max(1, min(64, 2048 // hi))), _log(rng, 1, 8192)
        return dict(op="tree", batch=batch, hq=hkv * rng.choice((1, 2, 3, 4, 7, 8)), hkv=hkv, d=d, type=kind,
                    block=block, nodes_lo=lo, nodes_hi=hi, old_lo=rng.randrange(0, old_hi + 1), old_hi=old_hi,
                    cap=rng.choice((0.0, 0.0, 30.0)), window=rng.choice((0, 0, 0, 128, 700)), shape=shape)
    return dict(op="commit", batch=_log(rng, 1, max(1, min(64, 1024 // hi))), caches=2 * _log(rng, 1, 32), hkv=hkv, d=d,
                type=kind, block=block, nodes_lo=lo, nodes_hi=hi, old_lo=0, old_hi=_log(rng, 1, 160),
                match=rng.choice((30, 70, 90, 100)), shape=shape)


# ---- sizes that belong to a case ---------------------------------------------------------------

def _blocks(n, block):
    return -(-n // block)


def _trees(case):
    """(nodes, keys) of each sequence, and each token row's parent: an index among its sequence's
    nodes, before its own; -1 for the first."""
    r = random.Random(case["shape"])
    n = [r.randint(case["nodes_lo"], case["nodes_hi"]) for _ in range(case["batch"])]
    keys = [x + r.randint(case["old_lo"], case["old_hi"]) for x in n]
    parents = []
    for x in n:
        width = r.choice((1, 3, 8, 64))         # from chains to bushes
        parents.append([-1] + [r.randint(max(0, i - width), i - 1) for i in range(1, x)])
    return n, keys, parents


def _choices(case, parents):
    """Drafted tokens, and the target model's token behind each node: often one of the node's children."""
    r = random.Random(case["shape"] + 1)
    tokens, choices = [], []
    for p in parents:
        t = [r.randrange(50) if r.randrange(8) == 0 else r.randrange(32000) for _ in p]
        c = []
        for i in range(len(p)):
            children = [j for j in range(i + 1, len(p)) if p[j] == i]
            c.append(t[r.choice(children)] if children and r.randrange(100) < case["match"] else r.randrange(32000))
        tokens.append(t), choices.append(c)
    return tokens, choices


def _paths(parents, tokens, choices):
    """The nodes of each sequence's accepted path."""
    paths = []
    for p, t, c in zip(parents, tokens, choices):
        path = [0]
        while True:
            after = [j for j in range(len(p)) if p[j] == path[-1] and t[j] == c[path[-1]]]
            if not after:
                break
            path.append(after[0])
        paths.append(path)
    return paths


def _bytes(kind):
    return {"bf16": 2, "f32": 4, "e4m3": 1}[kind]


def work(case):
    if case["op"] == "norm":
        size, n = _bytes(case["type"]), case["tokens"] * case["dim"]
        total = n * (size * (3 if case["residual"] else 1) + _bytes(case["out"])) + case["dim"] * size
        if case["out"] == "e4m3":
            total += 4 * case["tokens"] * _blocks(case["dim"], GROUP)
        return dict(bytes=total, flops=4 * n)
    if case["op"] == "linear":
        M, N, K = case["M"], case["N"], case["K"]
        scales = 4 * (M + _blocks(N, GROUP)) * _blocks(K, GROUP)
        return dict(bytes=M * K + N * K + scales + M * N * _bytes(case["out"]), flops=2 * M * N * K)
    n, keys, parents = _trees(case)
    row = case["d"] * _bytes(case["type"])
    if case["op"] == "tree":
        seen = read = 0
        for x, L, p in zip(n, keys, parents):
            old, depth = L - x, [0] * x
            for i in range(1, x):
                depth[i] = depth[p[i]] + 1
            window = case["window"] or L
            seen += sum(min(old, window) + k + 1 for k in depth)
            read += min(old, window) + x
        return dict(bytes=2 * sum(n) * case["hq"] * row + 2 * read * case["hkv"] * row, flops=4 * seen * case["hq"] * case["d"])
    moved = sum(sum(a != j for j, a in enumerate(path)) for path in _paths(parents, *_choices(case, parents)))
    return dict(bytes=2 * moved * case["caches"] * case["hkv"] * row + 20 * sum(n) + 12 * case["batch"], flops=0)


# ---- inputs ------------------------------------------------------------------------------------

def _int32(a):
    return torch.as_tensor(np.asarray(a, dtype=np.int32)).cuda()


def _hidden(gen, rows, dim):
    """Hidden states: normal, with a few channels that are much larger."""
    x = torch.randn(rows, dim, generator=gen, device="cuda")
    far = torch.rand(dim, generator=gen, device="cuda") < 0.01
    return torch.where(far, 12.0 * x, x)


def _code(kind):
    import split_kv_async_gb300 as F
    return {"bf16": F.FDPP_BF16, "f32": F.FDPP_F32, "e4m3": F.FDPP_E4M3}[kind]


def prepare(case, seed):
    gen = torch.Generator("cuda").manual_seed(seed)
    perm = np.random.default_rng(seed)
    return {"norm": _prepare_norm, "linear": _prepare_linear, "tree": _prepare_tree,
            "commit": _prepare_commit}[case["op"]](case, gen, perm)


def _prepare_norm(case, gen, perm):
    T, dim = case["tokens"], case["dim"]
    kind = TYPES[case["type"]]
    s = dict(case=case, x=_hidden(gen, T, dim).to(kind), residual=None, total=None, scales=None,
             weight=(1.0 + 0.2 * torch.randn(dim, generator=gen, device="cuda")).to(kind),
             out=torch.zeros(T, dim, device="cuda", dtype=torch.bfloat16).to(TYPES[case["out"]]))
    if case["residual"]:
        s["residual"] = (4.0 * _hidden(gen, T, dim)).to(kind)
        s["total"] = torch.zeros(T, dim, device="cuda", dtype=kind)
    if case["out"] == "e4m3":
        s["scales"] = torch.zeros(T, _blocks(dim, GROUP), device="cuda")
    if own:
        import split_kv_async_gb300 as F
        s["p"] = F.make_norm_params(num_tokens=T, dim=dim, dtype=_code(case["type"]), out_dtype=_code(case["out"]), eps=1e-6)
    return s


def _prepare_linear(case, gen, perm):
    M, N, K = case["M"], case["N"], case["K"]
    pad = _blocks(K, GROUP) * GROUP - K
    x = torch.nn.functional.pad(_hidden(gen, M, K), (0, pad)).reshape(M, -1, GROUP)
    sx = (x.abs().amax(-1) / LARGEST).clamp(min=LEAST_SCALE)
    x = (x / sx[..., None]).reshape(M, -1)[:, :K].to(TYPES["e4m3"]).contiguous()
    w = torch.randn(N, K, generator=gen, device="cuda") * 0.02
    w = torch.nn.functional.pad(w, (0, pad, 0, -N % GROUP)).reshape(_blocks(N, GROUP), GROUP, -1, GROUP)
    sw = (w.abs().amax((1, 3)) / LARGEST).clamp(min=LEAST_SCALE)
    w = (w / sw[:, None, :, None]).reshape(-1, K + pad)[:N, :K].to(TYPES["e4m3"]).contiguous()
    s = dict(case=case, x=x, sx=sx, w=w, sw=sw, y=torch.zeros(M, N, device="cuda", dtype=TYPES[case["out"]]))
    if own:
        import split_kv_async_gb300 as F
        s["p"] = F.make_scaled_gemm_params(M=M, N=N, K=K, out_dtype=_code(case["out"]))
        s["ws"] = F.alloc_scaled_gemm_workspace(s["p"])
    return s


def _table(case, keys, perm):
    """(block table, blocks of the pool) of a paged cache, with a few blocks that belong to nobody."""
    used = [_blocks(L, case["block"]) for L in keys]
    ids = perm.permutation(sum(used) + 3).astype(np.int32)
    table = np.full((case["batch"], max(used)), -1, np.int32)
    at = 0
    for b, u in enumerate(used):
        table[b, :u] = ids[at:at + u]
        at += u
    return _int32(table), sum(used) + 3


def _prepare_tree(case, gen, perm):
    n, keys, parents = _trees(case)
    B, hq, hkv, d, block = (case[x] for x in ("batch", "hq", "hkv", "d", "block"))
    T, longest, kind = sum(n), max(keys), TYPES[case["type"]]
    cu = np.concatenate([[0], np.cumsum(n)])
    randn = lambda *size: torch.randn(size, generator=gen, device="cuda", dtype=kind)  # noqa: E731
    s = dict(case=case, n_max=max(n), longest=longest, q=randn(T, hq, d), parents=_int32(np.concatenate(parents)),
             lens=_int32(keys), cu=_int32(cu), begin=None, table=None, out=torch.zeros(T, hq, d, device="cuda", dtype=kind))
    if case["window"]:          # the window's first key, by a token's depth in its tree
        first = []
        for x, L, p in zip(n, keys, parents):
            depth = [0] * x
            for i in range(1, x):
                depth[i] = depth[p[i]] + 1
            first += [max(0, L - x + k + 1 - case["window"]) for k in depth]
        s["begin"] = _int32(first)
    size = (B, longest, hkv, d)
    if block:
        s["table"], s["blocks"] = _table(case, keys, perm)
        size = (s["blocks"], block, hkv, d)
    s["k"], s["v"] = randn(*size), randn(*size)
    # rows of a padded batch, for the plain form: token (b, i), or the first one where there is none
    b, i = np.divmod(np.arange(B * max(n)), max(n))
    s["row"] = torch.as_tensor(np.where(i < np.asarray(n)[b], cu[b] + i, 0)).cuda()
    seq = np.repeat(np.arange(B), n)
    s["flat"] = torch.as_tensor(seq * max(n) + np.arange(T) - cu[seq]).cuda()
    s["n"] = _int32(n).long()
    if own:
        import split_kv_async_gb300 as F
        s["p"] = F.make_rows_params(batch=B, num_q_heads=hq, num_kv_heads=hkv, head_dim=d, dtype=_code(case["type"]),
                                    num_tokens=T, max_seq_len=longest, scale=d ** -0.5, softcap=case["cap"],
                                    key_begin=s["begin"], block_size=block,
                                    max_blocks_per_seq=s["table"].shape[1] if block else 0,
                                    num_kv_blocks=s["blocks"] if block else 0)
        s["ws"] = F.alloc_tree_workspace(s["p"])
    return s


def _prepare_commit(case, gen, perm):
    n, keys, parents = _trees(case)
    tokens, choices = _choices(case, parents)
    B, block, T, longest = case["batch"], case["block"], sum(n), max(keys)
    cu = np.concatenate([[0], np.cumsum(n)])
    s = dict(case=case, n_max=max(n), longest=longest, parents=_int32(np.concatenate(parents)),
             tokens=_int32(np.concatenate(tokens)), choices=_int32(np.concatenate(choices)), lens=_int32(keys), cu=_int32(cu),
             table=None, new_lens=_int32(np.zeros(B)), accepted=_int32(np.zeros(B)), path=_int32(np.zeros(T)),
             chosen=_int32(np.zeros(T)))
    size = (B, longest)
    if block:
        s["table"], s["blocks"] = _table(case, keys, perm)
        size = (s["blocks"], block)
    s["caches"] = torch.randn((case["caches"],) + size + (case["hkv"], case["d"]), generator=gen, device="cuda",
                              dtype=TYPES[case["type"]])
    b, i = np.divmod(np.arange(B * max(n)), max(n))
    s["row"] = torch.as_tensor(np.where(i < np.asarray(n)[b], cu[b] + i, 0)).cuda()
    seq = np.repeat(np.arange(B), n)
    s["flat"] = torch.as_tensor(seq * max(n) + np.arange(T) - cu[seq]).cuda()
    s["n"] = _int32(n).long()
    if own:
        import split_kv_async_gb300 as F
        s["p"] = F.make_commit_params(batch=B, num_tokens=T, max_seq_len=longest,
                                      row_bytes=case["hkv"] * case["d"] * _bytes(case["type"]), block_size=block,
                                      max_blocks_per_seq=s["table"].shape[1] if block else 0,
                                      num_kv_blocks=s["blocks"] if block else 0)
        s["list"] = F.make_cache_list(s["caches"].unbind(0))
        s["ws"] = F.alloc_commit_workspace(s["p"])
    return s


# ---- one pass ----------------------------------------------------------------------------------

def run(s):
    return {"norm": _run_norm, "linear": _run_linear, "tree": _run_tree, "commit": _run_commit}[s["case"]["op"]](s)


def _run_norm(s):
    outputs = [s[k] for k in ("out", "scales", "total") if s[k] is not None]
    if own:
        import split_kv_async_gb300 as F
        F.fdpp_rms_norm(s["x"], s["residual"], s["weight"], s["p"], s["out"], s["scales"], s["total"])
        return outputs
    r = s["x"].float()
    if s["residual"] is not None:
        r = r + s["residual"].float()
        s["total"].copy_(r)
    y = r * torch.rsqrt(r.square().mean(-1, keepdim=True) + 1e-6) * s["weight"].float()
    if s["scales"] is not None:
        T, dim = y.shape
        y = torch.nn.functional.pad(y, (0, -dim % GROUP)).reshape(T, -1, GROUP)
        s["scales"].copy_((y.abs().amax(-1) / LARGEST).clamp(min=LEAST_SCALE))
        y = (y / s["scales"][..., None]).reshape(T, -1)[:, :dim]
    s["out"].copy_(y)
    return outputs


def _run_linear(s):
    if own:
        import split_kv_async_gb300 as F
        F.fdpp_scaled_gemm(s["x"], s["sx"], s["w"], s["sw"], s["p"], s["ws"], s["y"])
        return s["y"]
    M, N, K = (s["case"][x] for x in "MNK")
    x = s["x"].float() * s["sx"].repeat_interleave(GROUP, 1)[:, :K]
    w = s["w"].float() * s["sw"].repeat_interleave(GROUP, 0)[:N].repeat_interleave(GROUP, 1)[:, :K]
    s["y"].copy_(x @ w.T)
    return s["y"]


def _lineage(parents):
    """[B][n][n]: whether node j is node i itself or one of its ancestors, from the parents [B][n]."""
    n = parents.shape[1]
    at = torch.arange(n, device="cuda")
    seen = (parents[..., None] == at) | (at[:, None] == at)
    for _ in range(max(1, (n - 1).bit_length())):       # lines of 2, 4, 8, .. generations
        seen = seen.float() @ seen.float() > 0
    return seen


def _run_tree(s):
    case = s["case"]
    if own:
        import split_kv_async_gb300 as F
        F.fdpp_tree_attn(s["q"], s["k"], s["v"], s["table"], s["lens"], s["cu"], s["parents"], s["p"], s["ws"], s["out"])
        return s["out"]
    B, hq, hkv, d = (case[x] for x in ("batch", "hq", "hkv", "d"))
    n, L, G = s["n_max"], s["longest"], hq // hkv
    k, v = s["k"], s["v"]
    if s["table"] is not None:
        k = k[s["table"].long()].flatten(1, 2)[:, :L]
        v = v[s["table"].long()].flatten(1, 2)[:, :L]
    k, v = k.float().permute(0, 2, 1, 3), v.float().permute(0, 2, 1, 3)           # [B][hkv][L][d]
    q = s["q"][s["row"]].float().reshape(B, n, hkv, G, d).permute(0, 2, 1, 3, 4)   # [B][hkv][n][G][d]
    scores = (q.reshape(B, hkv, n * G, d) @ k.transpose(2, 3)).reshape(B, hkv, n, G, L) * d ** -0.5
    if case["cap"]:
        scores = case["cap"] * torch.tanh(scores / case["cap"])
    lens = s["lens"].long()
    old = (lens - s["n"])[:, None, None]
    t = torch.arange(L, device="cuda")
    node = (t - old).clamp(0, n - 1).expand(B, n, L)
    line = _lineage(s["parents"][s["row"]].reshape(B, n)).gather(2, node)
    seen = ((t < old) | line) & (t < lens[:, None, None])
    if s["begin"] is not None:
        seen = seen & (t >= s["begin"][s["row"]].reshape(B, n, 1))
    scores = torch.where(seen[:, None, :, None], scores, float("-inf"))
    most = scores.amax(-1, keepdim=True)
    p = torch.exp(scores - torch.where(most == float("-inf"), 0.0, most))
    total = p.sum(-1, keepdim=True)
    o = (p.reshape(B, hkv, n * G, L) @ v).reshape(B, hkv, n, G, d)
    o = torch.where(total > 0, o / total, 0.0).permute(0, 2, 1, 3, 4).reshape(B * n, hq, d)
    return o[s["flat"]].to(s["q"].dtype)


def _run_commit(s):
    outputs = [s[k] for k in ("accepted", "new_lens", "path", "chosen", "caches")]
    if own:
        import split_kv_async_gb300 as F
        F.fdpp_tree_commit(s["parents"], s["tokens"], s["choices"], s["lens"], s["cu"], s["table"], s["list"], s["p"], s["ws"],
                           s["new_lens"], s["accepted"], s["path"], s["chosen"])
        return outputs
    case, n = s["case"], s["n_max"]
    B = case["batch"]
    at = torch.arange(n, device="cuda")
    live = at < s["n"][:, None]
    parents, tokens, choices = (s[k][s["row"]].reshape(B, n).long() for k in ("parents", "tokens", "choices"))
    up = parents.clamp(min=0)
    fits = live & (at > 0) & (parents >= 0) & (tokens == choices.gather(1, up))
    # of a node's children with the chosen token the first one counts
    first = torch.full((B, n), n, device="cuda").scatter_reduce(1, up, torch.where(fits, at, n), "amin")
    good = (at == 0) | (fits & (first.gather(1, up) == at))
    line = _lineage(parents)
    taken = live & ~(line & ~good[:, None]).any(-1)
    depth = (line & (at > 0)).sum(-1)
    accepted = taken.sum(-1)
    # the path's nodes in order: node i at place depth(i)
    path = torch.full((B, n + 1), -1, device="cuda").scatter(1, torch.where(taken, depth, n), at.expand(B, n))[:, :n]
    chosen = torch.where(path >= 0, choices.gather(1, path.clamp(min=0)), -1)
    old = s["lens"].long() - s["n"]
    s["accepted"].copy_(accepted)
    s["new_lens"].copy_(old + accepted)
    s["path"].copy_(path.reshape(-1)[s["flat"]])
    s["chosen"].copy_(chosen.reshape(-1)[s["flat"]])
    to = torch.where(live, old[:, None] + at, 0).reshape(-1)[s["flat"]]
    come = (old[:, None] + torch.where(path >= 0, path, at)).reshape(-1)[s["flat"]]
    b = torch.div(s["flat"], n, rounding_mode="floor")
    if s["table"] is not None:
        block = case["block"]
        to = s["table"][b, to // block].long() * block + to % block
        come = s["table"][b, come // block].long() * block + come % block
    else:
        to, come = b * s["longest"] + to, b * s["longest"] + come
    rows = s["caches"].flatten(1, 2)
    rows[:, to] = rows[:, come]
    return outputs


# ---- the definitions, in 64 bits ---------------------------------------------------------------

def exact(case, seed):
    if case["op"] == "commit":
        return None             # whole numbers and copies only
    s = prepare(case, seed)
    return {"norm": _exact_norm, "linear": _exact_linear, "tree": _exact_tree}[case["op"]](case, s)


def _exact_norm(case, s):
    r = s["x"].double()
    if s["residual"] is not None:
        r += s["residual"].double()
    size = (torch.linalg.vector_norm(r, dim=1).square() / case["dim"] + 1e-6).sqrt()
    y = r * s["weight"].double() / size[:, None]
    outputs = [y]
    if s["scales"] is not None:
        scales = torch.stack([part.abs().amax(1) for part in y.split(GROUP, 1)], 1) / LARGEST
        scales = scales.clamp(min=LEAST_SCALE)
        outputs = [torch.cat([part / scales[:, i:i + 1] for i, part in enumerate(y.split(GROUP, 1))], 1), scales]
    if s["total"] is not None:
        outputs.append(r)
    return outputs


def _exact_linear(case, s):
    if 2.0 * case["M"] * case["N"] * case["K"] > 4e12:
        return None
    y = torch.zeros(case["M"], case["N"], dtype=torch.float64, device="cuda")
    for n0 in range(0, case["N"], 4096):        # rows of w at a time, block of K by block
        w = s["w"][n0:n0 + 4096].double()
        of = (torch.arange(w.shape[0], device="cuda") + n0) // GROUP
        for i, k0 in enumerate(range(0, case["K"], GROUP)):
            part = s["x"][:, k0:k0 + GROUP].double() @ w[:, k0:k0 + GROUP].T
            y[:, n0:n0 + 4096] += part * s["sx"][:, i:i + 1].double() * s["sw"][of, i].double()
    return y


def _exact_tree(case, s):
    """Token by token of the tree: its keys are listed by walking up to the root."""
    n, keys, parents = _trees(case)
    hq, hkv, d, block = (case[x] for x in ("hq", "hkv", "d", "block"))
    G = hq // hkv
    if sum(x * L for x, L in zip(n, keys)) * hq * d > 4e12:
        return None
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    row = 0
    for b, (x, L, p) in enumerate(zip(n, keys, parents)):
        t = torch.arange(L, device="cuda")
        if block:
            slots = s["table"][b].long()[t // block] * block + t % block
            k, v = s["k"].reshape(-1, hkv, d)[slots], s["v"].reshape(-1, hkv, d)[slots]
        else:
            k, v = s["k"][b, :L], s["v"][b, :L]
        hidden = np.zeros((x, L), bool)
        for i in range(x):
            hidden[i, L - x:] = True
            j = i
            while j >= 0:
                hidden[i, L - x + j] = False
                j = p[j]
        hidden = torch.as_tensor(hidden).cuda()
        if s["begin"] is not None:
            hidden |= t < s["begin"][row:row + x].long()[:, None]
        q = s["q"][row:row + x].double().reshape(x, hkv, G, d)
        z = torch.einsum("xhgd,thd->hgxt", q, k.double()) / math.sqrt(d)
        if case["cap"]:
            z = torch.tanh(z / case["cap"]) * case["cap"]
        weight = torch.softmax(z.masked_fill(hidden, -math.inf), -1)
        out[row:row + x] = torch.einsum("hgxt,thd->xhgd", weight, v.double()).reshape(x, hq, d)
        row += x
    return out
