"""Builds rows attention problems on the device (caches poisoned with NaN wherever no sequence has a
key), runs them through the library and compares with the 64-bit reference.

Bounds, from the arithmetic, per element. bf16 on the tensor cores: the output's rounding, half a step,
2^-8 |out|; each weight p_t is rounded to bf16 before the product with V, half a step, 2^-8 of
sum_t p_t |v_t|; and fp32 for the rest: a score's dot product is off by at most d 2^-24 scale sum |q k|
(below 2^-13 for the values here), its cap by a few 2^-23 of the cap and its bias by 2^-24 of itself, the
exponentials by 2^-22: together below 2^-12 of sum_t p_t |v_t|, as are the sums. fp32, and bf16 on the
CUDA cores (weights stay in fp32): the last part and the output's rounding."""
from __future__ import annotations

import numpy as np
import torch

import rows_reference as R
import split_kv_async_gb300 as F

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def ints(a):
    return torch.as_tensor(np.asarray(a, np.int32)).cuda()


class Problem:
    """seqs: (new tokens, own keys) of each sequence. lead: token rows before the first sequence, tail:
    behind the last. mask: None, or a function (row, pos, total) -> (begin, end)."""

    def __init__(self, seqs, hq=4, hkv=2, d=128, dtype="bf16", block=0, prefix=0, cap=0.0, bias=False, mask=None,
                 kernel=None, seed=0, lead=0, tail=0, spare_len=0, spare_prefix=0, scale=None, uniform=False, q_gain=1.0):
        rng = np.random.default_rng(seed)
        gen = torch.Generator().manual_seed(seed)
        tdt = TYPES[dtype]
        rand = lambda *s: torch.randn(*s, generator=gen).to(tdt)  # noqa: E731
        n, lens = [s[0] for s in seqs], [s[1] for s in seqs]
        B, P = len(seqs), prefix
        cu = lead + np.concatenate([[0], np.cumsum(n)]).astype(np.int64)
        T = int(cu[-1]) + tail
        Lmax = max(max(lens), 1) + spare_len
        Pmax = P + spare_prefix
        self.q = (q_gain * rand(T, hq, d).float()).to(tdt)
        k, v = [rand(L, hkv, d) for L in lens], [rand(L, hkv, d) for L in lens]
        pk, pv = rand(P, hkv, d), rand(P, hkv, d)
        nan = float("nan")
        self.table = self.prefix_table = self.pk = self.pv = None
        blocks = width = 0
        if block:
            used, shared = [-(-L // block) for L in lens], -(-P // block)
            blocks = sum(used) + shared + 2
            width = max(1, -(-Lmax // block))
            ids = rng.permutation(blocks)
            kc, vc = (torch.full((blocks, block, hkv, d), nan, dtype=tdt) for _ in range(2))
            table = np.full((B, width), 2 ** 30, np.int32)       # entries past the end are never read
            at = 0

            def fill(x, y, L, row):
                nonlocal at
                for j in range(-(-L // block)):
                    row[j] = ids[at]
                    m = min(block, L - j * block)
                    kc[ids[at], :m] = x[j * block:j * block + m]
                    vc[ids[at], :m] = y[j * block:j * block + m]
                    at += 1

            for b in range(B):
                fill(k[b], v[b], lens[b], table[b])
            self.table = ints(table)
            if Pmax:
                ptable = np.full(-(-Pmax // block), 2 ** 30, np.int32)
                fill(pk, pv, P, ptable)
                self.prefix_table = ints(ptable)
        else:
            kc, vc = (torch.full((B, Lmax, hkv, d), nan, dtype=tdt) for _ in range(2))
            for b in range(B):
                kc[b, :lens[b]], vc[b, :lens[b]] = k[b], v[b]
            if Pmax:
                pkc, pvc = (torch.full((Pmax, hkv, d), nan, dtype=tdt) for _ in range(2))
                pkc[:P], pvc[:P] = pk, pv
                self.pk, self.pv = pkc.cuda(), pvc.cuda()
        self.slopes = np.array([2.0 ** (-6.0 * (h + 1) / hq) for h in range(hq)], np.float32) if bias else None
        self.begin = self.end = None
        if mask is not None:
            self.begin, self.end = np.zeros(T, np.int64), np.zeros(T, np.int64)
            for b in range(B):
                for i in range(n[b]):
                    row, total = int(cu[b]) + i, P + lens[b]
                    self.begin[row], self.end[row] = mask(row, total - n[b] + i, total)
        self.scale = float(np.float32(d ** -0.5)) if scale is None else scale
        f64 = lambda t: t.double().numpy()  # noqa: E731
        self.host = R.Rows(q=f64(self.q), k=[f64(x) for x in k], v=[f64(x) for x in v], pk=f64(pk), pv=f64(pv), cu=cu,
                           lens=np.asarray(lens), scale=self.scale, cap=cap, slopes=self.slopes, begin=self.begin,
                           end=self.end)
        self.prefix, self.dtype, self.rows = bool(Pmax), dtype, (lead, int(cu[-1]))
        self.q_d, self.k_d, self.v_d = self.q.cuda(), kc.cuda(), vc.cuda()
        self.cu_d = None if uniform else ints(cu)
        self.lens_d, self.plen_d = ints(lens), ints([P])
        self.slopes_d = None if self.slopes is None else torch.as_tensor(self.slopes).cuda()
        self.begin_d, self.end_d = (None if x is None else ints(x) for x in (self.begin, self.end))
        self.simt = kernel == F.FDPP_KERNEL_SIMT or dtype == "f32"
        self.p = F.make_rows_params(batch=B, num_q_heads=hq, num_kv_heads=hkv, head_dim=d,
                                    dtype=F.FDPP_BF16 if dtype == "bf16" else F.FDPP_F32, num_tokens=T, max_seq_len=Lmax,
                                    scale=self.scale, softcap=cap, slopes=self.slopes_d, key_begin=self.begin_d,
                                    key_end=self.end_d, block_size=block, max_blocks_per_seq=width, num_kv_blocks=blocks,
                                    max_prefix_len=Pmax, kernel=F.FDPP_KERNEL_AUTO if kernel is None else kernel)
        self.ws = F.alloc_rows_workspace(self.p)
        self.fill = 9.0
        self.out = torch.full_like(self.q_d, self.fill)

    def call(self, stream=None, ws=None, out=None):
        ws, out = self.ws if ws is None else ws, self.out if out is None else out
        if self.prefix:
            F.fdpp_prefix_attn(self.q_d, self.pk, self.pv, self.prefix_table, self.plen_d, self.k_d, self.v_d, self.table,
                               self.lens_d, self.cu_d, self.p, ws, out, stream=stream)
        else:
            F.fdpp_rows_attn(self.q_d, self.k_d, self.v_d, self.table, self.lens_d, self.cu_d, self.p, ws, out,
                             stream=stream)
        return out

    def check(self, got=None, errors=0):
        """`got` (default: a call's output) against the reference; returns the largest share of the bound."""
        if got is None:
            got = self.call()
            torch.cuda.synchronize()
            assert F.fdpp_read_error(self.ws) == errors
        ref, spread = R.attention(self.host)
        got = got.double().cpu().numpy()
        a, z = self.rows
        assert (got[:a] == self.fill).all() and (got[z:] == self.fill).all(), "rows of no sequence were written"
        got, ref, spread = got[a:z], ref[a:z], spread[a:z]
        np.testing.assert_array_equal(np.isnan(got), np.isnan(ref))
        step = float(torch.finfo(TYPES[self.dtype]).eps) / 2
        weights = 0.0 if self.simt else 2.0 ** -8
        bound = step * np.abs(ref) + (weights + 2.0 ** -12) * spread
        err = np.abs(got - ref)
        ok = (err <= bound) | np.isnan(ref) | (got == ref)
        assert ok.all(), f"max err {np.nanmax(err):.3e}, {(~ok).sum()} of {ok.size} over the bound, at {np.argwhere(~ok)[:3]}"
        return float(np.nanmax(err / np.maximum(bound, 1e-30), initial=0.0))
