// rows_internal.h -- types shared by the rows attention's host API and kernels (not installed).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include "fdpp_internal.h"
#include "fdpp_rows.h"

namespace fdpp {

// The tensor kernel: 128 query rows per tile (one per tensor-memory lane), two tiles in a pair, 128
// keys per K/V tile.
constexpr int ROWS_TILE = 128;
constexpr int ROWS_PAIR = 2 * ROWS_TILE;
constexpr int ROWS_KEYS = 128;
// Most rows of a key-major run (scores with the keys on the tensor-memory lanes).
constexpr int ROWS_NARROW = 32;
// Parts that the key tiles of all units are cut into, at most (one per CTA, one CTA per SM).
constexpr int ROWS_MAX_PARTS = 160;
// Counters of the CUDA-core kernel's splits (zero between calls): it splits only calls with fewer
// (token, kv head, head chunk) triples than this.
constexpr int ROWS_COUNTERS = 1024;
// Heads of one kv head that a CTA of the CUDA-core kernel takes, and its splits at most.
constexpr int ROWS_SIMT_HEADS = 4;
constexpr int ROWS_SIMT_MAX_SPLITS = 64;

// A token row: its position and the keys [lo, hi) it sees, prefix keys first; lo >= hi: none. rt: its
// own row tile, -1: a row of no sequence.
struct RowToken {
    int pos, lo, hi, rt;
};

// A row tile: `ntok` tokens from row tok0 on, in one 128-row tile (ntok <= tokens per tile) or a pair,
// against the keys of sequence b (b < 0: the prefix). Key tiles [a0, a1) of the first 128 rows and
// [b0, b1) of the second, local to that source; the tile's units (one per kv head) stream the union
// [k0, k0 + nt), and begin at tile `start` + g nt of the order that is cut into parts.
struct RowTileRec {
    int b, tok0, ntok, len;
    int a0, a1, b0, b1;
    int k0, nt, start, pad;
};

// Workspace: byte offsets. The counters and the error word lie at fixed places, so that one
// workspace may serve calls of different parameters.
struct RowsLayout {
    size_t counters, plan, tok, seq_rt, rec, slot_o, slot_ml, row_o, row_ml, total;
    int max_rt, slot_rows;
};
constexpr size_t ROWS_OFF_COUNTERS = 256;
constexpr size_t ROWS_OFF_PLAN = ROWS_OFF_COUNTERS + ROWS_COUNTERS * 4;

// Plan header words, then the first row tile of each part.
enum { RP_NRT = 0, RP_NPRE = 1, RP_TILES = 2, RP_PREFIX = 3, RP_WORDS = 16 };

struct RowsArgs {
    const void* q;
    const void* k;
    const void* v;
    const void* pk;                 // contiguous prefix, or nullptr
    const void* pv;
    const int32_t* block_table;     // nullptr: contiguous caches
    const int32_t* prefix_blocks;
    const int32_t* prefix_len;      // nullptr: no prefix
    const int32_t* seq_lens;
    const int32_t* cu;              // nullptr: T / B tokens each
    const float* slopes;
    const int32_t* key_begin;
    const int32_t* key_end;
    void* out;
    unsigned* err;
    int* counters;
    int* plan;
    RowToken* tok;
    int* seq_rt;                    // [B + 1] first own row tile of each sequence
    RowTileRec* rec;
    float* slot_o;                  // [2 parts][slot_rows][D]: a unit cut in two or more
    float2* slot_ml;                // [2 parts][slot_rows]
    float* row_o;                   // [2][T][Hq][D]: whole units of a call with a prefix (prefix, own)
    float2* row_ml;                 // [2][T][Hq]
    int B, Hq, Hkv, G, D, T, per_seq;
    int max_seq_len, block_size, max_blocks, num_blocks, max_prefix;
    int tpt, tpn;                   // tokens per 128-row tile and per key-major run: floor(128 / G), floor(32 / G)
    int max_rt, slot_rows, parts, splits, stages;
    float scale, cap;
};

RowsLayout rows_layout(const fdpp_rows_params& p);

cudaError_t launch_rows_simt(const RowsArgs& a, int dtype, cudaStream_t s);
// Plan, tile kernel and join.
struct RowsMaps {
    CUtensorMap q, qn;     // q as {d, Hq, T}: boxes of a 128-row tile, and of a key-major run's 32 rows
    CUtensorMap k, v;      // the caches
    CUtensorMap pk, pv;    // the prefix (the pools again for paged caches)
};
cudaError_t launch_rows_tc(const RowsArgs& a, const RowsMaps& m, cudaStream_t s);
// K/V stages that fit the device's shared memory per block.
int rows_tc_stages(int head_dim, int smem_per_block);

}  // namespace fdpp
