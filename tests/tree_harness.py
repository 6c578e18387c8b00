"""Trees of drafted tokens for the tests: random ones of any width, the reference of tree attention and of
the commit in plain Python and 64 bits, and the problems on the device. Bounds as in rows_harness."""
from __future__ import annotations

import numpy as np
import torch

import rows_harness as H
import rows_reference as R
import split_kv_async_gb300 as F


def random_tree(rng, n, width, roots=0):
    """Parents of n nodes, each among the `width` nodes before it; `roots`: about one in so many is a root."""
    return [-1] + [-1 if roots and rng.integers(roots) == 0 else int(rng.integers(max(0, i - width), i)) for i in range(1, n)]


def line(parents, i):
    nodes = []
    while i >= 0:
        nodes.append(i)
        i = parents[i] if -1 <= parents[i] < i else -1
    return nodes


def attention(x: R.Rows, trees):
    """(out, spread) as rows_reference.attention, masked by the trees."""
    T, Hq, d = x.q.shape
    Hkv = x.pk.shape[1]
    G = Hq // Hkv
    out, spread = np.full((T, Hq, d), np.nan), np.zeros((T, Hq, d))
    for b, parents in enumerate(trees):
        L, n = int(x.lens[b]), len(parents)
        for i in range(n):
            row = int(x.cu[b]) + i
            t = np.array(list(range(max(0, L - n))) + sorted(L - n + j for j in line(parents, i) if L - n + j >= 0), np.int64)
            if x.begin is not None:
                t = t[t >= x.begin[row]]
            if n > F.FDPP_TREE_MAX_TOKENS or len(t) == 0 or L - n + i < 0:
                out[row] = 0.0
                continue
            for g in range(Hkv):
                k, v = x.k[b][t, g], x.v[b][t, g]
                s = x.scale * (x.q[row, g * G:(g + 1) * G] @ k.T)
                if x.cap:
                    s = x.cap * np.tanh(s / x.cap)
                with np.errstate(invalid="ignore", over="ignore"):
                    p = np.exp(s - s.max(-1, keepdims=True))
                    p = p / p.sum(-1, keepdims=True)
                    out[row, g * G:(g + 1) * G] = p @ v
                    spread[row, g * G:(g + 1) * G] = p @ np.abs(v)
    return out, spread


class TreeProblem(H.Problem):
    """trees: parents of each sequence; old: keys before them; begin: first keys by row, or None. bf16 takes the tensor
    kernel unless another is asked for (left to itself the library takes the CUDA cores for small problems)."""

    def __init__(self, trees, old, begin=None, **kw):
        if kw.get("kernel") is None and kw.get("dtype", "bf16") == "bf16":
            kw["kernel"] = F.FDPP_KERNEL_TENSOR
        mask = None
        if begin is not None:
            mask = lambda row, pos, total: (begin(row, pos), 0)  # noqa: E731
        super().__init__([(len(t), len(t) + o) for t, o in zip(trees, old)], mask=mask, **kw)
        self.trees = trees
        self.p.key_end = None
        self.ws = F.alloc_tree_workspace(self.p)
        lead, tail = self.rows[0], self.q.shape[0] - self.rows[1]
        # (parents of rows of no sequence are never looked at)
        self.parents_d = H.ints([7] * lead + [x for t in trees for x in t] + [7] * tail)

    def call(self, stream=None, ws=None, out=None):
        ws, out = self.ws if ws is None else ws, self.out if out is None else out
        F.fdpp_tree_attn(self.q_d, self.k_d, self.v_d, self.table, self.lens_d, self.cu_d, self.parents_d, self.p, ws, out,
                         stream=stream)
        return out

    def check(self, got=None, errors=0):
        if got is None:
            got = self.call()
            torch.cuda.synchronize()
            assert F.fdpp_read_error(self.ws) == errors
        ref, spread = attention(self.host, self.trees)
        got = got.double().cpu().numpy()
        a, z = self.rows
        assert (got[:a] == self.fill).all() and (got[z:] == self.fill).all(), "rows of no sequence were written"
        got, ref, spread = got[a:z], ref[a:z], spread[a:z]
        np.testing.assert_array_equal(np.isnan(got), np.isnan(ref))
        step = float(torch.finfo(H.TYPES[self.dtype]).eps) / 2
        bound = step * np.abs(ref) + ((0.0 if self.simt else 2.0 ** -8) + 2.0 ** -12) * spread
        err = np.abs(got - ref)
        ok = (err <= bound) | np.isnan(ref) | (got == ref)
        assert ok.all(), f"max err {np.nanmax(err):.3e}, {(~ok).sum()} of {ok.size} over the bound, at {np.argwhere(~ok)[:3]}"


# ---- commit ------------------------------------------------------------------------------------

def commit(trees, tokens, choices):
    """The accepted nodes of each sequence."""
    paths = []
    for p, t, c in zip(trees, tokens, choices):
        path = [0] if p else []
        while path:
            i = path[-1]
            after = [j for j in range(i + 1, len(p)) if p[j] == i and t[j] == c[i]]
            if not after:
                break
            path.append(after[0])
        paths.append(path)
    return paths
