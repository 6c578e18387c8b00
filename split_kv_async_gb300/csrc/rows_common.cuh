// rows_common.cuh -- what the rows attention's kernels share: the tokens of a sequence, the keys a
// row sees, cache addresses and the scores' cap and bias.
#pragma once

#include "device_common.cuh"
#include "rows_internal.h"

namespace fdpp {
namespace {

constexpr float LOG2E = 1.4426950408889634f;

__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ float rcp(float x)
{
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ void rows_error(const RowsArgs& a, unsigned bits)
{
    if (bits) atomicOr(a.err, bits);
}

// Token rows [c0, c0 + n) of sequence b.
__device__ __forceinline__ int seq_rows(const RowsArgs& a, int b, int& c0, unsigned& bad)
{
    if (!a.cu) {
        c0 = b * a.per_seq;
        return a.per_seq;
    }
    const int x = a.cu[b], y = a.cu[b + 1];
    c0 = clamp_len(x, a.T);
    const int c1 = max(c0, clamp_len(y, a.T));
    if (x != c0 || y != c1) bad |= FDPP_ERRBIT_TOKENS;
    return c1 - c0;
}

__device__ __forceinline__ int own_len(const RowsArgs& a, int b, unsigned& bad)
{
    const int L = a.seq_lens[b], c = clamp_len(L, a.max_seq_len);
    if (L != c) bad |= FDPP_ERRBIT_SEQ_LEN;
    return c;
}

__device__ __forceinline__ int prefix_keys(const RowsArgs& a, unsigned& bad)
{
    if (!a.prefix_len) return 0;
    const int P = a.prefix_len[0], c = clamp_len(P, a.max_prefix);
    if (P != c) bad |= FDPP_ERRBIT_PREFIX;
    return c;
}

// Keys [lo, hi) that row `row` at position `pos` sees of `total`.
__device__ __forceinline__ void row_keys(const RowsArgs& a, int row, int pos, int total, int& lo, int& hi)
{
    lo = a.key_begin ? max(a.key_begin[row], 0) : 0;
    hi = min(a.key_end ? a.key_end[row] : pos + 1, total);
    if (hi <= lo) lo = hi = 0;
}

// A sequence of n tokens whose tree is too large: its tokens see nothing.
__device__ __forceinline__ bool tree_too_large(const RowsArgs& a, int n) { return a.parents && n > FDPP_TREE_MAX_TOKENS; }

// Whether a token with this lineage, of a tree whose node 0 is key tree0, sees key t of its key range.
__device__ __forceinline__ bool line_sees(const uint32_t* line, int tree0, int t)
{
    const int node = t - tree0;
    return node < 0 || (node < FDPP_TREE_MAX_TOKENS && (line[LINE_UP + (node >> 5)] >> (node & 31) & 1u));
}

// Bits [at, at + 32) of LINE_BITS words, zeros behind them.
__device__ __forceinline__ uint32_t line_bits(const uint32_t* words, int at)
{
    const int w = at >> 5;
    const uint32_t lo = w < LINE_BITS ? words[w] : 0u, hi = w + 1 < LINE_BITS ? words[w + 1] : 0u;
    return __funnelshift_r(lo, hi, at & 31);
}

// Element offset of key t (local to its source) of kv head g; -1: its block lies outside the pool.
__device__ __forceinline__ long long key_offset(const RowsArgs& a, int b, int t, int g)
{
    long long slot;
    if (!a.block_table) {
        slot = b < 0 ? t : (long long)b * a.max_seq_len + t;
    } else {
        const int j = t / a.block_size;
        const int blk = b < 0 ? a.prefix_blocks[j] : a.block_table[(long long)b * a.max_blocks + j];
        if (blk < 0 || blk >= a.num_blocks) return -1;
        slot = (long long)blk * a.block_size + (t - j * a.block_size);
    }
    return (slot * a.Hkv + g) * a.D;
}

// The score in units of log2, to the accuracy of bf16 weights: cap, then the bias -slope |pos - t|. tanh(x) = 1 - 2 / (e^2x + 1): two
// MUFU operations, absolute error a few 2^-23 of the cap (tanh.approx would be 2^-11 off). cap_rate: 2
// scale log2(e) / cap.
__device__ __forceinline__ float mod_score(float qk, float scale, float cap, float cap_rate, float slope2, float dist)
{
    float s = qk * (scale * LOG2E);
    if (cap > 0.f) s = fmaf(-2.f * LOG2E * cap, rcp(ex2(qk * cap_rate) + 1.f), LOG2E * cap);
    return fmaf(-slope2, fabsf(dist), s);
}

// Two scores capped at once (top: log2(e) cap), with one reciprocal of the product of their denominators:
// a reciprocal takes the MUFU twice as long as an exponential. The exponents are cut at 60, where the tanh
// is 1 in fp32, so that the product stays finite; NaN stays NaN.
__device__ __forceinline__ void cap_pair(float& x0, float& x1, float cap_rate, float top)
{
    float t0, t1;
    asm("min.NaN.f32 %0, %1, 0f42700000;" : "=f"(t0) : "f"(x0 * cap_rate));
    asm("min.NaN.f32 %0, %1, 0f42700000;" : "=f"(t1) : "f"(x1 * cap_rate));
    const float e0 = ex2(t0) + 1.f, e1 = ex2(t1) + 1.f, r = rcp(e0 * e1);
    x0 = fmaf(-2.f * top, r * e1, top);
    x1 = fmaf(-2.f * top, r * e0, top);
}

}  // namespace
}  // namespace fdpp
