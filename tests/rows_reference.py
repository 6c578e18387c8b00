"""Plain 64-bit implementations of the block map, the rotary append and the rows attention, written
from their definitions (loops over sequences, tokens and heads), and the inputs of their tests."""
from __future__ import annotations

import dataclasses
import math

import numpy as np


# ---- block map ---------------------------------------------------------------------------------

def block_map(held, want, pool, table, queue, block, room):
    """(lens, table, queue, pool, cu, seq, pos, slots, refused) as the library leaves them; refused: the
    sequences that were not served, with the reason."""
    table, queue = table.copy(), queue.copy()
    cap, (head, count) = len(queue), pool
    lens, cu, rows, refused = [], [0], [], {}
    asked_blocks = asked_rows = taken = given = 0
    up = lambda n: -(-n // block)  # noqa: E731
    freed = []
    for b, (h, w) in enumerate(zip(held, want)):
        need, ask = max(0, up(w) - up(h)), max(0, w - h)
        asked_blocks += need
        asked_rows += ask
        short_blocks, short_rows = need > 0 and asked_blocks > count, ask > 0 and asked_rows > room
        if short_blocks or short_rows:
            refused[b] = (short_blocks, short_rows)
            lens.append(h)
            cu.append(len(rows))
            continue
        for j in range(up(h), up(h) + need):
            table[b, j] = queue[(head + taken) % cap]
            taken += 1
        for pos in range(h, w):
            rows.append((b, pos, int(table[b, pos // block]) * block + pos % block))
        freed += [int(table[b, j]) for j in range(up(w), up(h))]
        lens.append(w)
        cu.append(len(rows))
    for blk in freed:
        queue[(head + count + given) % cap] = blk
        given += 1
    rows += [(-1, 0, -1)] * (room - len(rows))
    seq, pos, slots = (np.array([r[i] for r in rows], np.int64) for i in range(3)) if rows else (np.zeros(0, np.int64),) * 3
    return (np.array(lens), table, queue, ((head + taken) % cap, count - taken + given), np.array(cu), seq, pos, slots,
            refused)


# ---- rotary append -----------------------------------------------------------------------------

def rope_theta(rot, base, scaling="plain", factor=1.0, context=0, low=1.0, high=32.0):
    if scaling == "ntk":
        base = base * factor ** (rot / (rot - 2))
    out = []
    for i in range(rot // 2):
        theta = base ** (-2.0 * i / rot)
        if scaling == "linear":
            theta /= factor
        if scaling == "parts":
            k = min(1.0, max(0.0, (context * theta / (2 * math.pi) - low) / (high - low)))
            theta *= k + (1 - k) / factor
        out.append(theta)
    return np.array(out)


def rope(x, positions, theta, inter, magnitude):
    """x float64 [T][heads][d] with its first 2 len(theta) elements turned."""
    y = x.copy()
    half = len(theta)
    for i, th in enumerate(theta):
        a, b = (2 * i, 2 * i + 1) if inter else (i, i + half)
        w = positions.astype(np.float64) * th
        c, s = (magnitude * f(w)[:, None] for f in (np.cos, np.sin))
        y[:, :, a], y[:, :, b] = x[:, :, a] * c - x[:, :, b] * s, x[:, :, a] * s + x[:, :, b] * c
    return y


# ---- rows attention ----------------------------------------------------------------------------

@dataclasses.dataclass
class Rows:
    """A rows attention problem on the host: values as float64 of what the device holds."""
    q: np.ndarray              # [T][Hq][d]
    k: list                    # per sequence [L][Hkv][d]
    v: list
    pk: np.ndarray             # [P][Hkv][d]
    pv: np.ndarray
    cu: np.ndarray
    lens: np.ndarray
    scale: float
    cap: float = 0.0
    slopes: np.ndarray = None
    begin: np.ndarray = None
    end: np.ndarray = None


def attention(x: Rows):
    """(out [T][Hq][d], spread): spread[row] = sum_t p_t |v_t|, the size that the rounding of the weights
    p is relative to. Rows of no sequence are NaN."""
    T, Hq, d = x.q.shape
    Hkv, P = x.pk.shape[1], x.pk.shape[0]
    G = Hq // Hkv
    out, spread = np.full((T, Hq, d), np.nan), np.zeros((T, Hq, d))
    for b in range(len(x.lens)):
        L, n = int(x.lens[b]), int(x.cu[b + 1] - x.cu[b])
        k, v = np.concatenate([x.pk, x.k[b][:L]]), np.concatenate([x.pv, x.v[b][:L]])
        for i in range(n):
            row, pos = int(x.cu[b]) + i, P + L - n + i
            lo = 0 if x.begin is None else max(0, int(x.begin[row]))
            hi = min(P + L, pos + 1 if x.end is None else int(x.end[row]))
            if hi <= lo:
                out[row] = 0.0
                continue
            t = np.arange(lo, hi)
            for g in range(Hkv):
                for h in range(g * G, (g + 1) * G):
                    s = x.scale * (k[lo:hi, g] @ x.q[row, h])
                    if x.cap:
                        s = x.cap * np.tanh(s / x.cap)
                    if x.slopes is not None:
                        s = s - float(x.slopes[h]) * np.abs(pos - t)
                    with np.errstate(invalid="ignore", over="ignore"):
                        p = np.exp(s - s.max())
                        p = p / p.sum()
                        out[row, h] = p @ v[lo:hi, g]
                        spread[row, h] = p @ np.abs(v[lo:hi, g])
    return out, spread
