// rows_tc.cu -- rows attention (fdpp_rows.h) on the tcgen05 tensor cores: bf16, d = 64 or 128.
//
// What it computes. For the rows of a kv head (its G query heads of some tokens) and a range of keys
//     v_t = log2(e) score_t, M = max v_t, l = sum 2^(v_t - M), o = sum 2^(v_t - M) v_t
// by one pass over the keys with a running max; the frame is moved only when a row's max has grown by
// more than 2^8 since it was set (until then the weights stay below 2^8, and the sums are exact in
// the same frame), so that the accumulator is hardly ever rescaled.
//
// How. One CTA per SM, fourteen warps at work, two streams:
//   warps 12, 13  load: the first walks this CTA's part of the key tiles (128 keys each), writes a header
//            for each run (the part's share of one unit = (row tile, kv head)) and brings Q, by one 3-D
//            TMA load per 64 of d, and the K tiles; the second brings the V tiles, into the other stages
//            of one ring (128-byte swizzle). Blocks of 16 tokens take 16 loads per tile and operand: with
//            one warp for both, issuing them took longer than HBM takes for the tile (438 us against 344
//            for the contiguous cache, 64 sequences of 512 to 16384 keys, 8 kv heads, d = 128).
//   warps 8, 9   issue Q K^T of streams 0 and 1 (one thread each): S, M = 128 rows, N = 64 keys, half a tile;
//   warps 10, 11 issue P V: O += P V with P from tensor memory and V MN-major from the TMA-landed tile. A
//            stream has two score buffers: while the softmax works on one half, the tensor cores finish
//            the other (its P V, then the next Q K^T into its place). With whole tiles P lay over the only
//            scores, and a stream's softmax and MMAs took turns; and with one warp for both products its
//            own instructions, between those of two busy softmax warps, set the pace.
//   warps 0-3, 4-7   the softmax of streams 0 and 1: a thread owns a row (tensor-memory lane), reads its
//            64 scores, and writes P as bf16 over them. P's rounding (up to half a step, 2^-8 of each weight,
//            independent) leaves at most as much of sum_t p_t |v_t|, and an error of the order of the output's own
//            rounding on average (its two bf16 parts, which the decode kernels keep, would take a second P V: half
//            as many MMAs again in what bounds prompts); l sums the unrounded weights.
// With more than 128 rows a unit is a pair: two row tiles, one per stream, share every K/V tile. With
// fewer, both streams take the same rows, alternate key tiles and are joined at the run's end.
//
// Few rows (32 at most): the same with the operands exchanged, the keys on the tensor-memory lanes. A
// row per lane would leave one warp of four with all the work; a key per lane shares it evenly.
//
// What bounds it. Many rows: the tensor pipe (4 x 128 keys x 128 rows x d FLOP per row tile and key tile, 1024
// cycles for d = 128; a half tile's Q K^T, N = 64, runs at two thirds of the rate, which makes them 1280) with the
// softmax beside it (512 cycles of the MUFU units for the exponentials, and its other instructions). A prompt of
// 8192 tokens, 32 heads, 8 kv heads, d = 128: 426 us, 1.29 PFLOP/s of the 1.87 that a plain matrix product was
// measured at; with a bias 485; with a cap 631 (scores near it 838: an exponential and half a reciprocal more for each).
// Few rows: HBM (K and V of a kv head are read once, at 512 bytes
// per key for d = 128): 64 sequences of 512 to 16384 keys, 64 heads, 8 kv heads, with a cap: 338.5 us, 6.50 TB/s,
// 0.95 of a measured copy. Short calls: latency, of which the plan takes 3 to 8 us, a first tile with cold
// instruction caches 5, the join 4 to 8.
//
// Cut. The key tiles of all units are laid end to end and cut into one equal part per CTA. A unit that
// lies in one part is written whole; of one cut in two or more, every part leaves its partial (o, M, l)
// in one of its two slots, and a second kernel joins them. With a prefix every row has two units (the
// prefix's and its own), and rows are joined from both.
//
// Masks. A key outside a row's range gets the score -inf by selection, so no value of it enters the max
// or the sums; V of keys past the source's length is zeroed in shared memory (the products with weight 0
// would be NaN otherwise). Keys that some rows of a tile see and others do not can still carry a
// non-finite V: a row that ends non-finite with finite l, and that saw such a tile, has its non-finite
// columns computed again from the keys that it sees.
//
// Every wait is bounded; a wait that runs out sets FDPP_ERRBIT_TIMEOUT, and the CTA lets its copies and
// MMAs land, frees its tensor memory and exits. Rows that are computed again can hold the others up for longer
// (128 rows of 16384 keys, d = 128: 0.3 s), so a wait begins anew as long as their warps show signs of life.
#include <cuda_bf16.h>

#include "rows_common.cuh"
#include "tcgen05.cuh"

namespace fdpp {
namespace {

constexpr int RW_MMA_WARP = 8;           // Q K^T of either stream, then P V of either
constexpr int RW_LOAD_WARP = 12;         // K (with the headers and Q), and V
constexpr int RW_THREADS = 16 * 32;      // the last two warps idle: register shares go by four warps
// Registers of a softmax warp and of the others: 2 x (176 + 80) x 128 = 65536 = 512 x 128, the launch's.
constexpr int RW_SOFT_REGS = 176;
constexpr int RW_HELP_REGS = 80;
constexpr int RW_HDRS = 4;               // run headers in flight
constexpr int RW_HDR_BYTES = 64;
constexpr float RW_LAG = 8.f;            // log2 of the growth of a row's max that moves its frame

enum { RH_KIND = 0, RH_G, RH_B, RH_TOK0, RH_NTOK, RH_LEN, RH_A0, RH_A1, RH_B0, RH_B1, RH_T0, RH_T1, RH_DEST,
       RH_FLAGS, RH_BASE, RH_WORDS };
enum { RUN_ROWS = 0, RUN_END = 1 };
// two row tiles; few rows (key-major); the first key tile goes to stream 1; all of them do (else: to stream 0)
enum { RF_PAIR = 1, RF_NARROW = 2, RF_START = 4, RF_SOLO = 8 };
// A key-major run of at most this many key tiles that another run follows is one stream's alone, so that the
// other begins the next meanwhile: a run's beginning and end take as long as two tiles. 64 single tokens with up
// to 512 own keys behind a prefix: 1 us of 77 less; runs of five tiles, which both streams share, 1.5 of 61 more.
constexpr int RW_SOLO_TILES = 4;
enum { DEST_OUT = -1, DEST_ROWS = -2 };  // else a slot
static_assert(RH_WORDS * 4 <= RW_HDR_BYTES, "header fits its slot");

// What the key-major runs share between warps (in the second Q buffer, which they leave free).
struct NarrowShared {
    float wmax[2][4][ROWS_NARROW];       // per stream and warp: rows' maxima of a tile
    float lsum[2][4][ROWS_NARROW];       // sums of a run
    float frame[2][ROWS_NARROW];
    int flag[2][2][4];                   // per stream, tile parity and warp: a score beyond its row's frame
};

// Shared memory. Each softmax warp has 4 kB through which it turns its accumulator rows into whole
// 128-byte lines on their way out. A key-major run keeps to the Q buffers: two slots of 32 query rows and
// the weights of both streams ([32 rows][128 keys] bf16) in the first, two slots more and NarrowShared in
// the second; the load warp lets all runs of one kind end before it starts one of the other.
template <int D>
struct RowsSmem {
    static constexpr int QB = ROWS_TILE * D * 2;           // a row tile's Q
    static constexpr int SB = ROWS_KEYS * D * 2;           // a K or V tile
    static constexpr int HALF = ROWS_KEYS * 128;           // one 64-wide half of either
    static constexpr int TURN = 32 * 128;                  // a warp's rows, 128 bytes of each
    static constexpr int NSLOTS = 4;
    static constexpr int NQ = ROWS_NARROW * D * 2;         // a key-major run's Q
    static constexpr int NQ_HALF = ROWS_NARROW * 128;
    static constexpr int NP = ROWS_NARROW * ROWS_KEYS * 2; // its weights, per stream
    // d = 64: the weights fill the first buffer, the slots the second, and NarrowShared lies at the end
    static constexpr int FIRST_SLOTS = (QB - 2 * NP) / NQ;
    static constexpr int NP_OFF = QB - 2 * NP;
    __host__ __device__ static constexpr int slot(int i) { return i < FIRST_SLOTS ? i * NQ : QB + (i - FIRST_SLOTS) * NQ; }
    static constexpr int SLOTS_END = QB + (NSLOTS - FIRST_SLOTS) * NQ;
    static constexpr bool NSH_IN_Q = SLOTS_END + (int)sizeof(NarrowShared) <= 2 * QB;
    int q, stages, turn, hdr, ml, bars, misc, tslot, nsh, total;
    __host__ __device__ explicit RowsSmem(int nst)
        : q(0), stages(2 * QB), turn(stages + nst * SB), hdr(turn + 8 * TURN), ml(hdr + RW_HDRS * RW_HDR_BYTES),
          bars(ml + 2 * ROWS_TILE * 8), misc(bars + (2 * nst + 2 * (2 + NSLOTS) + 2 * RW_HDRS + 3 * 4 + 4 * 2 + 1) * 8),
          tslot(misc + 64), nsh(NSH_IN_Q ? SLOTS_END : tslot + 16),
          total(tslot + 16 + (NSH_IN_Q ? 0 : (int)sizeof(NarrowShared)))
    {
        static_assert(QB >= 2 * NP && SLOTS_END <= 2 * QB, "a key-major run fits the Q buffers");
    }
};

struct RowsBars {
    uint32_t kvfull, kvempty;     // [stages]
    uint32_t qfull, qempty;       // [2]
    uint32_t nqfull, nqempty;     // [4] the key-major runs' slots
    uint32_t hfull, hempty;       // [RW_HDRS] run headers: read by the V loader, the MMA and the softmax warps
    uint32_t sfull, pready;       // [2][2] scores written; weights written (per stream and score buffer: either
                                  //     side may be one buffer ahead)
    uint32_t pvdone;              // [2][2] the P V complete: the buffer is free
    uint32_t ofull, ofree;        // [2] accumulator complete; read out
    uint32_t mlfree;              // [2] a stream's maxima and sums have been read
    uint32_t vote;                // [2] the warps of a stream meet (key-major runs)
    uint32_t drain;
    __device__ __forceinline__ RowsBars(uint32_t base, int nst)
    {
        kvfull = base;
        kvempty = kvfull + 8 * nst;
        qfull = kvempty + 8 * nst;
        qempty = qfull + 16;
        nqfull = qempty + 16;
        nqempty = nqfull + 32;
        hfull = nqempty + 32;
        hempty = hfull + 8 * RW_HDRS;
        sfull = hempty + 8 * RW_HDRS;
        pready = sfull + 32;
        pvdone = pready + 32;
        ofull = pvdone + 32;
        ofree = ofull + 16;
        mlfree = ofree + 16;
        vote = mlfree + 16;
        drain = vote + 16;
    }
};

// Shared words besides the barriers: the CTA gives up; signs of life of warps that compute rows again (which can
// take seconds: every key of a long context, for each row); runs whose sums a warp has told.
enum { MISC_ABORT = 0, MISC_BEAT = 1, MISC_TOLD = 4 };

__device__ __forceinline__ void beat(volatile int* misc)
{
    if ((threadIdx.x & 31) == 0) atomicAdd(const_cast<int*>(misc) + MISC_BEAT, 1);
}

// Whether a wait that began at t0 has run out: no sign of life for FDPP_WAIT_NS. last: beats at the check before.
__device__ __forceinline__ bool run_out(volatile int* misc, uint64_t& t0, int& last)
{
    if (global_ns() - t0 <= FDPP_WAIT_NS) return false;
    const int now = misc[MISC_BEAT];
    if (now == last) return true;
    last = now;
    t0 = global_ns();
    return false;
}

// All lanes wait. A wait that is over when asked for costs two instructions; otherwise it is bounded, and
// one that runs out aborts the CTA (warp-uniform result).
__device__ __forceinline__ bool rwait_slow(uint32_t bar, uint32_t parity, volatile int* misc, unsigned* err)
{
    bool ok = misc[MISC_ABORT] == 0;
    if (ok) {
        uint64_t t0 = global_ns();
        int last = 0;
        for (uint32_t it = 1; !mbar_try_wait(bar, parity); ++it) {
            if ((it & 63u) == 0 && run_out(misc, t0, last)) { ok = false; break; }
        }
    }
    ok = __all_sync(0xffffffffu, ok);
    if (!ok && (threadIdx.x & 31) == 0) {
        misc[MISC_ABORT] = 1;
        atomicOr(err, FDPP_ERRBIT_TIMEOUT);
    }
    return ok;
}

__device__ __forceinline__ bool rwait(uint32_t bar, uint32_t parity, volatile int* misc, const RowsArgs& a)
{
    if (__builtin_expect(__all_sync(0xffffffffu, mbar_try_wait(bar, parity & 1u)), 1)) return true;
    return rwait_slow(bar, parity & 1u, misc, a.err);
}

// First tile of part c of the `total` tiles.
__device__ __forceinline__ int part_begin(int c, int total, int parts) { return (int)((long long)c * total / parts); }

// A unit takes its key tiles and some more in the order that is cut: the time of a run's beginning and
// end, in key tiles, so that a part with many short runs holds fewer tiles. With one tile for every run a
// prompt of 8192 tokens takes 637 us, with two 532, with three 443, with four 443, with five 445 (32 heads,
// 8 kv heads, d = 128), ragged prompts of 333 to 1500 tokens 57, 55, 57, 61 and 62; 64 single-token rows
// behind a shared prefix, whose own units are key-major, take 89 us with one, 81 with two and 86 with three.
constexpr int RW_GAP = 3, RW_NARROW_GAP = 2;
__device__ __forceinline__ int unit_span(const RowsArgs& a, const RowTileRec& r)
{
    return r.nt > 0 ? r.nt + (r.ntok <= a.tpn ? RW_NARROW_GAP : RW_GAP) : 0;
}

// ------------------------------------------------------------------------------------------
// plan
// ------------------------------------------------------------------------------------------
constexpr int PLAN_THREADS = 1024;
constexpr int PLAN_SMEM_SEQS = 2048;

__device__ __forceinline__ int warp_min(int x)
{
    return __reduce_min_sync(0xffffffffu, x);
}
__device__ __forceinline__ int warp_max(int x)
{
    return __reduce_max_sync(0xffffffffu, x);
}

// Inclusive scan of x over the CTA and its total.
__device__ __forceinline__ long long plan_scan(long long x, long long& total, long long* red)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    __syncthreads();
    if (lane == 31) red[warp] = x;
    __syncthreads();
    long long add = 0;
    total = 0;
    for (int w = 0; w < nw; ++w) {
        const long long y = red[w];
        if (w < warp) add += y;
        total += y;
    }
    return x + add;
}

// Key tiles of the two halves of a row tile from the key ranges (local to the source) of their rows.
__device__ __forceinline__ void set_tiles(RowTileRec& r, int loA, int hiA, int loB, int hiB)
{
    r.a0 = r.a1 = r.b0 = r.b1 = 0;
    hiA = min(hiA, r.len);
    hiB = min(hiB, r.len);
    if (hiA > loA) { r.a0 = loA / ROWS_KEYS; r.a1 = ceil_div_i(hiA, ROWS_KEYS); }
    if (hiB > loB) { r.b0 = loB / ROWS_KEYS; r.b1 = ceil_div_i(hiB, ROWS_KEYS); }
    int k0 = r.a0, k1 = r.a1;
    if (r.b1 > r.b0) {
        k0 = k1 > k0 ? min(k0, r.b0) : r.b0;
        k1 = max(k1, r.b1);
    }
    r.k0 = k0;
    r.nt = k1 - k0;
}

// The plan of calls with at most PLAN_SMALL sequences and row tiles: everything in shared memory, each
// token looked at once. It is on every call's critical path, so it has few steps and little code (a kernel
// starts with cold instruction caches): one row of loads per sequence, a scan, one pass over the tokens
// that leaves the row tiles' key ranges in shared memory, a scan. With more than 1024 tokens it is a
// cluster of up to PLAN_CLUSTER CTAs that share out the tokens; the ranges gather in the first one's
// shared memory (5 rounds of 1024 tokens took 16 us in one CTA).
constexpr int PLAN_SMALL = 1024;
constexpr int PLAN_CLUSTER = 8;

__device__ __forceinline__ void cluster_meet()
{
    asm volatile("barrier.cluster.arrive.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
}

// The first CTA's copy of a shared variable.
template <typename T>
__device__ __forceinline__ T* in_first(T* p)
{
    uint64_t q;
    asm("mapa.u64 %0, %1, 0;" : "=l"(q) : "l"(p));
    return reinterpret_cast<T*>(q);
}

// Inclusive scan of x over the CTA's 1024 threads, and the total.
__device__ __forceinline__ int scan_1024(int x, int& total, int* red)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    if (lane == 31) red[warp] = x;
    __syncthreads();
    int y = red[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int z = __shfl_up_sync(0xffffffffu, y, o);
        if (lane >= o) y += z;
    }
    total = __shfl_sync(0xffffffffu, y, 31);
    const int before = __shfl_sync(0xffffffffu, y, (warp + 31) & 31);
    __syncthreads();
    return x + (warp ? before : 0);
}

// The last i in [0, n) with v[i] <= x (v[0] <= x).
__device__ __forceinline__ int last_at_most(const int* v, int n, int x)
{
    int lo = 0, hi = n;
#pragma unroll 1
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (v[mid] <= x) lo = mid; else hi = mid;
    }
    return lo;
}

__global__ void __launch_bounds__(PLAN_SMALL) rows_plan_small_kernel(RowsArgs a)
{
    __shared__ int red[32];
    __shared__ int rt0[PLAN_SMALL + 1], c0[PLAN_SMALL], cnt[PLAN_SMALL], len[PLAN_SMALL];
    __shared__ int low[2][PLAN_SMALL], high[2][PLAN_SMALL];      // key ranges of the row tiles' halves; later: starts
    const int t = threadIdx.x, rank = blockIdx.x, ranks = gridDim.x;      // (the grid is one cluster)
    grid_dependency_wait();
    grid_launch_dependents();
    unsigned bad = 0;
    int first = 0, n = 0, L = 0;
    if (t < a.B) {
        n = seq_rows(a, t, first, bad);
        L = own_len(a, t, bad);
    }
    const int P = prefix_keys(a, bad);
    const int last = a.cu ? clamp_len(a.cu[a.B], a.T) : a.T;
    const int pair = 2 * a.tpt, npre = P > 0 ? ceil_div_i(last, pair) : 0;
    low[0][t] = low[1][t] = INT32_MAX;
    high[0][t] = high[1][t] = 0;
    int total;
    const int mine = min(ceil_div_i(n, pair), PLAN_SMALL), incl = scan_1024(mine, total, red);
    const int nrt = min(npre + total, a.max_rt);
    if (npre + total > a.max_rt) bad |= FDPP_ERRBIT_TOKENS;      // sequences whose rows overlap
    if (t < a.B) {
        rt0[t] = min(npre + incl - mine, a.max_rt);
        c0[t] = first;
        cnt[t] = n;
        len[t] = L;
    }
    if (ranks > 1) cluster_meet(); else __syncthreads();
    int* const low0 = ranks > 1 ? in_first(&low[0][0]) : &low[0][0];
    int* const high0 = ranks > 1 ? in_first(&high[0][0]) : &high[0][0];
    // the least and greatest key of each half of a row tile: one shared-memory operation for all the lanes of
    // a warp that belong to it where these are few (a reduction for each set of lanes, one after another),
    // and one for each lane where they are many (a row tile per token: 2.5 us less for 64 tokens)
    auto widen = [&](int key, int from, int to) {
        const unsigned m = __match_any_sync(0xffffffffu, key);
        bool speaks = (t & 31) == __ffs(m) - 1;
        if (__popc(__ballot_sync(0xffffffffu, speaks)) <= 4) {
            from = __reduce_min_sync(m, from);
            to = __reduce_max_sync(m, to);
        } else {
            speaks = true;
        }
        if (key >= 0 && speaks) {
            atomicMin(low0 + (key & 1) * PLAN_SMALL + (key >> 1), from);
            atomicMax(high0 + (key & 1) * PLAN_SMALL + (key >> 1), to);
        }
    };
    // key ranges are read a round ahead
    const int row0 = rank * PLAN_SMALL + t, step = ranks * PLAN_SMALL;
    int kb = a.key_begin && row0 < a.T ? a.key_begin[row0] : 0, ke = a.key_end && row0 < a.T ? a.key_end[row0] : 0;
    for (int base = rank * PLAN_SMALL; base < a.T; base += step) {
        const int row = base + t, after = row + step;
        const int nb = a.key_begin && after < a.T ? a.key_begin[after] : 0;
        const int ne = a.key_end && after < a.T ? a.key_end[after] : 0;
        const int b = last_at_most(c0, a.B, row), i = row - c0[b], rt = rt0[b] + i / pair;
        RowToken k{0, 0, 0, -1};
        int own = -1, pre = -1;
        if (row < a.T && i >= 0 && i < cnt[b] && rt < nrt) {
            k.pos = P + len[b] - cnt[b] + i;
            k.rt = rt;
            k.lo = max(kb, 0);
            k.hi = min(a.key_end ? ke : k.pos + 1, P + len[b]);
            if (k.hi <= k.lo) k.lo = k.hi = 0;
            if (k.hi > max(k.lo, P)) own = rt * 2 + (i % pair >= a.tpt);
            if (row < last && k.lo < min(k.hi, P)) pre = row / pair * 2 + (row % pair >= a.tpt);
            if (k.lo >= k.hi && !a.prefix_len) {                 // no unit may come by this row
                uint4* o = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.out) + (long long)row * a.Hq * a.D);
                for (int x = 0; x < a.Hq * a.D / 8; ++x) o[x] = make_uint4(0, 0, 0, 0);
            }
        }
        widen(own, max(k.lo - P, 0), k.hi - P);
        if (P > 0) widen(pre, k.lo, min(k.hi, P));
        if (row < a.T) a.tok[row] = k;
        kb = nb;
        ke = ne;
    }
    rows_error(a, bad);
    if (ranks > 1) cluster_meet(); else __syncthreads();
    if (rank) return;
    RowTileRec r{};
    if (t < nrt) {
        if (t < npre) {
            r.b = -1;
            r.tok0 = t * pair;
            r.ntok = min(pair, last - r.tok0);
            r.len = P;
        } else {
            r.b = last_at_most(rt0, a.B, t);
            const int i0 = (t - rt0[r.b]) * pair;
            r.tok0 = c0[r.b] + i0;
            r.ntok = max(0, min(pair, cnt[r.b] - i0));
            r.len = len[r.b];
        }
        set_tiles(r, low[0][t], high[0][t], low[1][t], high[1][t]);
    }
    const int span = t < nrt ? unit_span(a, r) * a.Hkv : 0;
    int tiles;
    r.start = scan_1024(span, tiles, red) - span;
    if (t < nrt) {
        a.rec[t] = r;
        low[0][t] = r.start;
    }
    __syncthreads();
    if (t < a.parts) a.plan[RP_WORDS + t] = nrt ? last_at_most(low[0], nrt, part_begin(t, tiles, a.parts)) : 0;
    if (t == 0) {
        a.plan[RP_NRT] = nrt;
        a.plan[RP_NPRE] = npre;
        a.plan[RP_TILES] = tiles;
        a.plan[RP_PREFIX] = P;
    }
}

// The plan of larger calls.
__global__ void __launch_bounds__(PLAN_THREADS) rows_plan_kernel(RowsArgs a)
{
    __shared__ long long red[32];
    __shared__ int srt[PLAN_SMEM_SEQS + 1];              // first row tile of each sequence
    __shared__ int sc0[PLAN_SMEM_SEQS], sn[PLAN_SMEM_SEQS], sl[PLAN_SMEM_SEQS];
    __shared__ int sstart[PLAN_SMEM_SEQS];               // first tile of each row tile
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
    grid_dependency_wait();
    grid_launch_dependents();
    unsigned bad = 0;
    const bool in_smem = a.B <= PLAN_SMEM_SEQS;
    int* first_rt = in_smem ? srt : a.seq_rt;
    const int pair = 2 * a.tpt;
    int last = a.T;
    if (a.cu) last = clamp_len(a.cu[a.B], a.T);
    const int P = prefix_keys(a, bad);
    // prefix row tiles first, over all rows up to the last sequence's end
    const int npre = P > 0 ? ceil_div_i(last, pair) : 0;
    long long run = npre;
    for (int base = 0; base < a.B; base += blockDim.x) {
        const int b = base + threadIdx.x;
        int c0 = 0, n = 0, L = 0;
        if (b < a.B) {
            n = seq_rows(a, b, c0, bad);
            L = own_len(a, b, bad);
            if (in_smem) { sc0[b] = c0; sn[b] = n; sl[b] = L; }
        }
        const long long mine = ceil_div_i(n, pair);
        long long total;
        const long long incl = plan_scan(mine, total, red);
        if (b < a.B) first_rt[b] = (int)min(run + incl - mine, (long long)a.max_rt);
        run += total;
    }
    const int nrt = (int)min(run, (long long)a.max_rt);
    if (run > a.max_rt) bad |= FDPP_ERRBIT_TOKENS;      // sequences whose rows overlap
    if (threadIdx.x == 0) first_rt[a.B] = nrt;
    __syncthreads();
    auto sequence = [&](int b, int& c0, int& n, int& L) {
        if (in_smem) {
            c0 = sc0[b]; n = sn[b]; L = sl[b];
        } else {
            unsigned again = 0;
            n = seq_rows(a, b, c0, again);
            L = own_len(a, b, again);
        }
    };
    auto of_rt = [&](int rt) {                          // first_rt[b] <= rt < first_rt[b + 1]
        int lo = 0, hi = a.B;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (first_rt[mid] <= rt) lo = mid; else hi = mid;
        }
        return lo;
    };
    // rows of no sequence: outside [cu_tokens[0], cu_tokens[B]), and anywhere if cu_tokens is not in order
    const int first_row = a.cu ? clamp_len(a.cu[0], a.T) : 0;
    const bool disorder = __syncthreads_or((int)(bad & FDPP_ERRBIT_TOKENS));
    for (int t = threadIdx.x; t < a.T; t += blockDim.x)
        if (disorder || t < first_row || t >= last) a.tok[t] = RowToken{0, 0, 0, -1};
    if (disorder) __syncthreads();

    // own row tiles: the tokens' positions and key ranges, and the tiles' key tiles
    const bool arrays = a.key_begin || a.key_end;
    const int per = !arrays && pair <= 8 ? 1 : (arrays || pair > 32 ? 32 : 8);      // lanes of a row tile
    const int sub = threadIdx.x % per;
    for (int rt0 = npre + (int)threadIdx.x / per; rt0 - (int)threadIdx.x / per < nrt; rt0 += blockDim.x / per) {
        const bool on = rt0 < nrt;
        const int rt = on ? rt0 : nrt - 1;
        int loA = INT32_MAX, hiA = 0, loB = INT32_MAX, hiB = 0, c0 = 0, n = 0, L = 0, i0 = 0, nt = 0, b = 0;
        if (on) {
            b = of_rt(rt);
            sequence(b, c0, n, L);
            i0 = (rt - first_rt[b]) * pair;
            nt = max(0, min(pair, n - i0));
            for (int i = sub; i < nt; i += per) {
                RowToken k;
                const int row = c0 + i0 + i;
                k.pos = P + L - n + i0 + i;
                k.rt = rt;
                row_keys(a, row, k.pos, P + L, k.lo, k.hi);
                a.tok[row] = k;
                const int x = max(k.lo - P, 0), y = k.hi - P;
                if (y > x) {
                    if (i < a.tpt) { loA = min(loA, x); hiA = max(hiA, y); }
                    else { loB = min(loB, x); hiB = max(hiB, y); }
                }
            }
        }
        for (int o = per >> 1; o > 0; o >>= 1) {
            loA = min(loA, __shfl_xor_sync(0xffffffffu, loA, o));
            hiA = max(hiA, __shfl_xor_sync(0xffffffffu, hiA, o));
            loB = min(loB, __shfl_xor_sync(0xffffffffu, loB, o));
            hiB = max(hiB, __shfl_xor_sync(0xffffffffu, hiB, o));
        }
        if (!on) continue;
        RowTileRec r{};
        r.b = b;
        r.tok0 = c0 + i0;
        r.ntok = nt;
        r.len = L;
        set_tiles(r, loA, hiA, loB, hiB);
        if (sub == 0) a.rec[rt] = r;
        if (r.nt == 0 && !a.prefix_len) {               // rows that see nothing, and no unit writes
            uint32_t* o = reinterpret_cast<uint32_t*>(static_cast<__nv_bfloat16*>(a.out) + (long long)r.tok0 * a.Hq * a.D);
            const long long words = (long long)nt * a.Hq * a.D / 2;
            for (long long i = sub; i < words; i += per) o[i] = 0u;
        }
    }
    __syncthreads();
    for (int rt = warp; rt < npre; rt += nw) {
        const int tok0 = rt * pair, nt = min(pair, last - tok0);
        int loA = INT32_MAX, hiA = 0, loB = INT32_MAX, hiB = 0;
        for (int i = lane; i < nt; i += 32) {
            const RowToken k = a.tok[tok0 + i];
            const int y = min(k.hi, P);
            if (k.rt >= 0 && y > k.lo) {
                if (i < a.tpt) { loA = min(loA, k.lo); hiA = max(hiA, y); }
                else { loB = min(loB, k.lo); hiB = max(hiB, y); }
            }
        }
        RowTileRec r{};
        r.b = -1;
        r.tok0 = tok0;
        r.ntok = nt;
        r.len = P;
        set_tiles(r, warp_min(loA), warp_max(hiA), warp_min(loB), warp_max(hiB));
        if (lane == 0) a.rec[rt] = r;
    }
    if (npre) __syncthreads();
    const bool starts_in_smem = nrt <= PLAN_SMEM_SEQS;
    long long tiles = 0;
    for (int base = 0; base < nrt; base += blockDim.x) {
        const int rt = base + threadIdx.x;
        const long long mine = rt < nrt ? (long long)unit_span(a, a.rec[rt]) * a.Hkv : 0;
        long long total;
        const long long incl = plan_scan(mine, total, red);
        if (rt < nrt) {
            const int start = (int)(tiles + incl - mine);
            a.rec[rt].start = start;
            if (starts_in_smem) sstart[rt] = start;
        }
        tiles += total;
    }
    __syncthreads();
    // the row tile that each part begins in
    for (int c = threadIdx.x; c < a.parts; c += blockDim.x) {
        const int x = part_begin(c, (int)tiles, a.parts);
        int lo = 0, hi = nrt;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if ((starts_in_smem ? sstart[mid] : a.rec[mid].start) <= x) lo = mid; else hi = mid;
        }
        a.plan[RP_WORDS + c] = lo;
    }
    if (threadIdx.x == 0) {
        a.plan[RP_NRT] = nrt;
        a.plan[RP_NPRE] = npre;
        a.plan[RP_TILES] = (int)tiles;
        a.plan[RP_PREFIX] = P;
    }
    rows_error(a, bad);
}

// ------------------------------------------------------------------------------------------
// load warp
// ------------------------------------------------------------------------------------------
template <int D>
struct RowsLoader {
    const RowsArgs& a;
    const RowsSmem<D>& lay;
    const RowsBars& bars;
    uint8_t* sm;
    uint32_t sbase;
    volatile int* misc;
    uint32_t stage = 0, phase = 0, nq = 0, nqn = 0, nh = 0;      // Q buffers and key-major slots filled, headers
    unsigned bad = 0;

    // Block of key tile t that this lane answers for (-1: none): entry t's first block + lane.
    __device__ __forceinline__ int entry(int b, int len, int t)
    {
        const int lane = threadIdx.x & 31;
        const int bs = a.block_size, first = t * ROWS_KEYS / bs, nv = min(ROWS_KEYS, len - t * ROWS_KEYS);
        const int nb = bs >= ROWS_KEYS ? 1 : ceil_div_i(nv, bs);
        if (nv <= 0 || lane >= nb) return -1;
        return b < 0 ? a.prefix_blocks[first + lane] : a.block_table[(long long)b * a.max_blocks + first + lane];
    }

    // One K or V tile into the next stage.
    __device__ __forceinline__ bool tile(const CUtensorMap* map, int b, int len, int g, int t, int ent)
    {
        constexpr int HALVES = D / 64;
        const int lane = threadIdx.x & 31;
        if (!rwait(bars.kvempty + 8 * stage, phase ^ 1u, misc, a)) return false;
        const uint32_t dst = sbase + lay.stages + stage * RowsSmem<D>::SB, bar = bars.kvfull + 8 * stage;
        if (!a.block_table) {
            if (lane == 0) mbar_arrive_expect_tx(bar, RowsSmem<D>::SB);
            __syncwarp();
            if (lane < HALVES)
                tma_load(dst + lane * RowsSmem<D>::HALF, map, g * D + lane * 64, t * ROWS_KEYS, max(b, 0), bar);
        } else {
            const int bs = a.block_size, box = min(bs, ROWS_KEYS), nv = min(ROWS_KEYS, len - t * ROWS_KEYS);
            const int nb = ceil_div_i(nv, box);
            const int blk = lane / HALVES, half = lane % HALVES;
            const int e = __shfl_sync(0xffffffffu, ent, blk);
            const bool in = blk < nb, ok = in && e >= 0 && e < a.num_blocks;
            if (in && !ok) bad |= FDPP_ERRBIT_BLOCK_TABLE;
            const int n = __popc(__ballot_sync(0xffffffffu, ok));
            if (lane == 0) {
                if (n) mbar_arrive_expect_tx(bar, (uint32_t)(n * box * 128)); else mbar_arrive(bar);
            }
            __syncwarp();
            if (ok)
                tma_load(dst + half * RowsSmem<D>::HALF + blk * box * 128, map, g * D + half * 64,
                         bs > ROWS_KEYS ? (t * ROWS_KEYS) % bs : 0, e, bar);
        }
        __syncwarp();
        stage += 2;                                      // the stage between is the other loader's
        if (stage >= (uint32_t)a.stages) { stage -= (uint32_t)a.stages; phase ^= 1u; }
        return true;
    }

    __device__ __forceinline__ void tma_load(uint32_t dst, const CUtensorMap* map, int x, int y, int z, uint32_t bar)
    {
        asm volatile(
            "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
            " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
            "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar)
            : "memory");
    }

    // Query rows into the next Q buffer, or the next slot of the key-major runs.
    __device__ __forceinline__ bool query(const CUtensorMap* map, int g, int tok0)
    {
        const int lane = threadIdx.x & 31;
        const uint32_t qb = nq & 1u, bar = bars.qfull + 8 * qb;
        if (!rwait(bars.qempty + 8 * qb, ((nq >> 1) & 1u) ^ 1u, misc, a)) return false;
        if (lane == 0) mbar_arrive_expect_tx(bar, (uint32_t)(a.tpt * a.G * 128 * (D / 64)));
        __syncwarp();
        if (lane < D / 64)
            tma_load(sbase + lay.q + qb * RowsSmem<D>::QB + lane * RowsSmem<D>::HALF, map, lane * 64, g * a.G, tok0, bar);
        __syncwarp();
        ++nq;
        return true;
    }
    __device__ __forceinline__ bool query_narrow(const CUtensorMap* map, int g, int tok0)
    {
        const int lane = threadIdx.x & 31;
        const uint32_t i = nqn & 3u, bar = bars.nqfull + 8 * i;
        if (!rwait(bars.nqempty + 8 * i, ((nqn >> 2) & 1u) ^ 1u, misc, a)) return false;
        if (lane == 0) mbar_arrive_expect_tx(bar, (uint32_t)(a.tpn * a.G * 128 * (D / 64)));
        __syncwarp();
        if (lane < D / 64)
            tma_load(sbase + lay.q + RowsSmem<D>::slot(i) + lane * RowsSmem<D>::NQ_HALF, map, lane * 64, g * a.G, tok0, bar);
        __syncwarp();
        ++nqn;
        return true;
    }

    // The runs so far have left everything that the two kinds of runs share.
    __device__ __forceinline__ bool settle_queries()
    {
        for (uint32_t k = 0; k < 2 && k < nq; ++k) {
            const uint32_t i = nq - 1 - k;
            if (!rwait(bars.qempty + 8 * (i & 1u), (i >> 1) & 1u, misc, a)) return false;
        }
        for (uint32_t k = 0; k < 4 && k < nqn; ++k) {
            const uint32_t i = nqn - 1 - k;
            if (!rwait(bars.nqempty + 8 * (i & 3u), (i >> 2) & 1u, misc, a)) return false;
        }
        return true;
    }

    __device__ __forceinline__ int* header()
    {
        const uint32_t s = nh % RW_HDRS;
        if (!rwait(bars.hempty + 8 * s, ((nh / RW_HDRS) & 1u) ^ 1u, misc, a)) return nullptr;
        return reinterpret_cast<int*>(sm + lay.hdr + s * RW_HDR_BYTES);
    }
    __device__ __forceinline__ void publish()
    {
        __syncwarp();
        if ((threadIdx.x & 31) == 0) mbar_arrive(bars.hfull + 8 * (nh % RW_HDRS));
        ++nh;
    }

    __device__ __forceinline__ bool run_k(const CUtensorMap* tq, const CUtensorMap* tqn, const CUtensorMap* tk,
                                          const CUtensorMap* tpk)
    {
        const int lane = threadIdx.x & 31;
        const int c = blockIdx.x, parts = gridDim.x;
        const int total = a.plan[RP_TILES], P = a.plan[RP_PREFIX];
        int rt = a.plan[RP_WORDS + c];                   // the row tile that the part begins in
        int pos = part_begin(c, total, parts);
        const int end = part_begin(c + 1, total, parts);
        uint32_t toggle = 0;
        bool was_narrow = false;
        while (pos < end && rt < a.max_rt) {
            const RowTileRec r = a.rec[rt];
            const bool narrow = r.ntok <= a.tpn;
            if (narrow != was_narrow && !settle_queries()) return false;
            was_narrow = narrow;
            const int span = unit_span(a, r), past = r.start + span * a.Hkv;
            while (pos < end && pos < past) {
                const int g = (pos - r.start) / span, ta = (pos - r.start) - g * span, tb = min(r.nt, ta + end - pos);
                const int next_pos = r.start + (g + 1) * span;
                if (ta >= r.nt) {                        // between two units
                    pos = next_pos;
                    continue;
                }
                const int t0 = r.k0 + ta, t1 = r.k0 + tb;
                const bool pair = r.ntok > a.tpt, whole = ta == 0 && tb == r.nt;
                const bool solo = narrow && tb == r.nt && next_pos < end && t1 - t0 <= RW_SOLO_TILES;
                int* h = header();
                if (!h) return false;
                if (lane == 0) {
                    h[RH_KIND] = RUN_ROWS;
                    h[RH_G] = g;
                    h[RH_B] = r.b;
                    h[RH_TOK0] = r.tok0;
                    h[RH_NTOK] = r.ntok;
                    h[RH_LEN] = r.len;
                    h[RH_A0] = max(r.a0, t0);
                    h[RH_A1] = max(min(r.a1, t1), max(r.a0, t0));
                    h[RH_B0] = max(r.b0, t0);
                    h[RH_B1] = max(min(r.b1, t1), max(r.b0, t0));
                    h[RH_T0] = t0;
                    h[RH_T1] = t1;
                    h[RH_DEST] = whole ? (a.prefix_len ? DEST_ROWS : DEST_OUT) : 2 * c + (ta == 0 ? 1 : 0);
                    h[RH_FLAGS] = (pair ? RF_PAIR : (toggle ? RF_START : 0)) | (narrow ? RF_NARROW : 0) | (solo ? RF_SOLO : 0);
                    h[RH_BASE] = r.b < 0 ? 0 : P;
                }
                publish();
                if (!pair) toggle = (toggle + (solo ? 1u : (uint32_t)(t1 - t0))) & 1u;
                int ent = a.block_table ? entry(r.b, r.len, t1 - 1) : 0;
                if (narrow ? !query_narrow(tqn, g, r.tok0) : !query(tq, g, r.tok0)) return false;
                if (pair && !query(tq, g, r.tok0 + a.tpt)) return false;
                for (int t = t1 - 1; t >= t0; --t) {
                    const int next = a.block_table && t > t0 ? entry(r.b, r.len, t - 1) : 0;
                    if (!tile(r.b < 0 ? tpk : tk, r.b, r.len, g, t, ent)) return false;
                    ent = next;
                }
                pos = tb < r.nt ? end : next_pos;
            }
            ++rt;
        }
        int* h = header();
        if (!h) return false;
        if (lane == 0) h[RH_KIND] = RUN_END;
        publish();
        return true;
    }

    __device__ __forceinline__ bool run_v(const CUtensorMap* tv, const CUtensorMap* tpv)
    {
        const int lane = threadIdx.x & 31;
        stage = 1;
        for (;; ++nh) {
            const uint32_t hs = nh % RW_HDRS;
            if (!rwait(bars.hfull + 8 * hs, (nh / RW_HDRS) & 1u, misc, a)) return false;
            const int* h = reinterpret_cast<const int*>(sm + lay.hdr + hs * RW_HDR_BYTES);
            const int kind = h[RH_KIND], g = h[RH_G], b = h[RH_B], len = h[RH_LEN], t0 = h[RH_T0], t1 = h[RH_T1];
            __syncwarp();
            if (lane == 0) mbar_arrive(bars.hempty + 8 * hs);
            if (kind == RUN_END) return true;
            int ent = a.block_table ? entry(b, len, t1 - 1) : 0;
            for (int t = t1 - 1; t >= t0; --t) {
                const int next = a.block_table && t > t0 ? entry(b, len, t - 1) : 0;
                if (!tile(b < 0 ? tpv : tv, b, len, g, t, ent)) return false;
                ent = next;
            }
        }
    }

    // After an abort: every copy issued lands before the CTA exits (bounded waits). `first`: this loader's
    // first stage.
    __device__ __forceinline__ void settle(int first)
    {
        if ((threadIdx.x & 31) == 0) {
            for (int s = first; s < a.stages; s += 2) {
                const uint32_t par = (uint32_t)s < stage ? phase : (phase ^ 1u);
                const uint64_t t0 = global_ns();
                while (!mbar_try_wait(bars.kvfull + 8 * s, par) && global_ns() - t0 < 100000000ull) {
                }
            }
            for (uint32_t k = 0; k < 2 && k < nq; ++k) {
                const uint32_t i = nq - 1 - k;
                const uint64_t t0 = global_ns();
                while (!mbar_try_wait(bars.qfull + 8 * (i & 1u), (i >> 1) & 1u) && global_ns() - t0 < 100000000ull) {
                }
            }
            for (uint32_t k = 0; k < 4 && k < nqn; ++k) {
                const uint32_t i = nqn - 1 - k;
                const uint64_t t0 = global_ns();
                while (!mbar_try_wait(bars.nqfull + 8 * (i & 3u), (i >> 2) & 1u) && global_ns() - t0 < 100000000ull) {
                }
            }
        }
        __syncwarp();
    }
};

// ------------------------------------------------------------------------------------------
// MMA warp
// ------------------------------------------------------------------------------------------
// Tensor memory: the scores of streams 0 and 1 (128 columns each: two buffers of 64, the first 32 columns of
// which P takes over; a key-major run's S^T has the first 16 or 32 of the 128), then their accumulators (D
// columns each; O^T of a key-major run takes 16 or 32).
constexpr uint32_t TM_S = ROWS_KEYS;

// A value that is the same in all lanes, told to the compiler.
__device__ __forceinline__ int uniform(int x) { return __shfl_sync(0xffffffffu, x, 0); }

__device__ __forceinline__ uint32_t narrow_cols(int rows) { return rows <= 16 ? 16u : 32u; }

// What the MMA warps take from a run's header: whose tiles are theirs, counted from the run's last.
struct MmaRun {
    int kind, len, t1, n, j0, j1, last;
    bool every;                                  // all of j0 .. j1, not every other
    bool pair;
    uint32_t ncols;                              // of a key-major run, else 0

    __device__ __forceinline__ void read(const int* h, uint32_t S, int G)
    {
        kind = uniform(h[RH_KIND]);
        len = uniform(h[RH_LEN]);
        const int flags = uniform(h[RH_FLAGS]), t0 = uniform(h[RH_T0]);
        t1 = uniform(h[RH_T1]);
        const int s0 = uniform(S ? h[RH_B0] : h[RH_A0]), s1 = uniform(S ? h[RH_B1] : h[RH_A1]);
        ncols = (flags & RF_NARROW) ? narrow_cols(uniform(h[RH_NTOK]) * G) : 0u;
        pair = flags & RF_PAIR;
        const uint32_t start = (flags & RF_START) ? 1u : 0u;
        n = t1 - t0;
        const bool solo = flags & RF_SOLO;
        every = pair || solo;
        j0 = pair ? t1 - s1 : solo ? (S == start ? 0 : n) : (int)(S ^ start);
        j1 = pair ? t1 - s0 : n;
        last = j0 >= j1 ? -1 : (every ? j1 - 1 : j1 - 1 - ((j1 - 1 - j0) & 1));
    }
    __device__ __forceinline__ bool mine(int j) const { return j >= j0 && j < j1 && (every || ((uint32_t)(j - j0) & 1u) == 0u); }
};

// Q K^T of stream S: every half tile (a key-major run: tile) as soon as its keys are there and its score
// buffer is free.
template <int D>
struct RowsQk {
    const RowsArgs& a;
    const RowsSmem<D>& lay;
    const RowsBars& bars;
    uint32_t sbase, tmem;
    volatile int* misc;
    uint32_t S;

    __device__ __forceinline__ bool run(uint8_t* sm)
    {
        constexpr uint32_t IDESC = umma_idesc_bf16(128, 64, false);
        const int lane = threadIdx.x & 31;
        const uint32_t sd = tmem + S * TM_S;
        uint32_t stage = 0, phase = 0, nq = 0, nqn = 0, use0 = 0, use1 = 0;
        for (uint32_t nh = 0;; ++nh) {
            const uint32_t hs = nh % RW_HDRS;
            if (!rwait(bars.hfull + 8 * hs, (nh / RW_HDRS) & 1u, misc, a)) return false;
            MmaRun r;
            r.read(reinterpret_cast<const int*>(sm + lay.hdr + hs * RW_HDR_BYTES), S, a.G);
            __syncwarp();
            if (lane == 0) mbar_arrive(bars.hempty + 8 * hs);
            if (r.kind == RUN_END) return true;
            // Q: of a pair, the buffer that is not this stream's goes back at once, as one without tiles does
            uint32_t qd = 0, qbar = 0;
            if (r.ncols) {
                const uint32_t i = nqn & 3u;
                // (without tiles of its own the slot may be refilled before this stream has looked)
                if (r.last >= 0 && !rwait(bars.nqfull + 8 * i, (nqn >> 2) & 1u, misc, a)) return false;
                qd = sw128_kmajor_lo(sbase + lay.q + RowsSmem<D>::slot(i));
                ++nqn;
            } else {
                for (uint32_t k = 0; k < (r.pair ? 2u : 1u); ++k, ++nq) {
                    const uint32_t qb = nq & 1u;
                    if (!rwait(bars.qfull + 8 * qb, (nq >> 1) & 1u, misc, a)) return false;
                    if (r.last >= 0 && (!r.pair || k == S)) {
                        qd = sw128_kmajor_lo(sbase + lay.q + qb * RowsSmem<D>::QB);
                        qbar = bars.qempty + 8 * qb;
                    } else if (lane == 0) {
                        mbar_arrive(bars.qempty + 8 * qb);
                    }
                }
            }
            for (int j = 0; j < r.n; ++j) {
                if (!rwait(bars.kvfull + 8 * stage, phase, misc, a)) return false;
                if (!r.mine(j)) {                  // a tile of the other stream, or of neither
                    if (lane == 0) mbar_arrive(bars.kvempty + 8 * stage);
                } else {
                    const uint32_t kd = sw128_kmajor_lo(sbase + lay.stages + stage * RowsSmem<D>::SB);
                    if (r.ncols == 0) {
#pragma unroll 1
                        for (uint32_t o = 0; o < 2; ++o) {       // the upper 64 keys, then the lower
                            if (!rwait(bars.pvdone + 16 * S + 8 * o, (o ? use1 : use0) ^ 1u, misc, a)) return false;
                            tc_fence_after();
                            const bool lead = elect_one();
                            const uint32_t kh = kd + (o ^ 1u) * (64 * 128 >> 4);
#pragma unroll
                            for (int k = 0; k < D / 16; ++k) {
                                const uint32_t off = (uint32_t)(k >> 2) * (RowsSmem<D>::HALF >> 4) + (uint32_t)(k & 3) * 2u;
                                umma_bf16_lo(lead, sd + 64 * o, qd + off, kh + off, IDESC, k > 0 ? 1u : 0u);
                            }
                            umma_commit(lead, bars.sfull + 16 * S + 8 * o);
                            if (o == 1) {
                                umma_commit(lead, bars.kvempty + 8 * stage);
                                if (j == r.last) umma_commit(lead, qbar);
                            }
                            __syncwarp();
                        }
                        ++use1;
                    } else {
                        if (!rwait(bars.pvdone + 16 * S, use0 ^ 1u, misc, a)) return false;
                        tc_fence_after();
                        const bool lead = elect_one();
                        // S^T = K Q^T: the keys on M, the rows on N
                        const uint32_t idesc = umma_idesc_bf16(128, 16, false) + ((r.ncols - 16) >> 3 << 17);
#pragma unroll
                        for (int k = 0; k < D / 16; ++k)
                            umma_bf16_lo(lead, sd, kd + (uint32_t)(k >> 2) * (RowsSmem<D>::HALF >> 4) + (uint32_t)(k & 3) * 2u,
                                         qd + (uint32_t)(k >> 2) * (RowsSmem<D>::NQ_HALF >> 4) + (uint32_t)(k & 3) * 2u, idesc,
                                         k > 0 ? 1u : 0u);
                        umma_commit(lead, bars.sfull + 16 * S);
                        umma_commit(lead, bars.kvempty + 8 * stage);
                        __syncwarp();
                    }
                    ++use0;
                }
                stage += 2;
                if (stage == (uint32_t)a.stages) { stage = 0; phase ^= 1u; }
            }
        }
    }
};

// P V of stream S: as soon as the weights are there.
template <int D>
struct RowsPv {
    const RowsArgs& a;
    const RowsSmem<D>& lay;
    const RowsBars& bars;
    uint32_t sbase, tmem;
    volatile int* misc;
    uint32_t S;

    __device__ __forceinline__ bool run(uint8_t* sm)
    {
        constexpr uint32_t IDESC = umma_idesc_bf16(128, D, false) | (1u << 16);     // V: MN-major B
        const int lane = threadIdx.x & 31;
        const uint32_t od = tmem + 2 * TM_S + S * D;
        uint32_t stage = 1, phase = 0, use0 = 0, use1 = 0, nacc = 0;
        for (uint32_t nh = 0;; ++nh) {
            const uint32_t hs = nh % RW_HDRS;
            if (!rwait(bars.hfull + 8 * hs, (nh / RW_HDRS) & 1u, misc, a)) return false;
            MmaRun r;
            r.read(reinterpret_cast<const int*>(sm + lay.hdr + hs * RW_HDR_BYTES), S, a.G);
            __syncwarp();
            if (lane == 0) mbar_arrive(bars.hempty + 8 * hs);
            if (r.kind == RUN_END) return true;
            for (int j = 0; j < r.n; ++j) {
                if (!rwait(bars.kvfull + 8 * stage, phase, misc, a)) return false;
                if (!r.mine(j)) {
                    if (lane == 0) mbar_arrive(bars.kvempty + 8 * stage);
                } else {
                    const int nv = r.len - (r.t1 - 1 - j) * ROWS_KEYS;
                    if (nv < ROWS_KEYS) {          // V past the source's end: zeros
                        uint8_t* v = sm + lay.stages + stage * RowsSmem<D>::SB;
                        const int chunks = (ROWS_KEYS - nv) * 8;
                        for (int i = lane; i < chunks * (D / 64); i += 32) {
                            const int half = i / chunks, x = i - half * chunks;
                            *reinterpret_cast<uint4*>(v + half * RowsSmem<D>::HALF + nv * 128 + x * 16) =
                                make_uint4(0, 0, 0, 0);
                        }
                        fence_proxy_async_smem();
                        __syncwarp();
                    }
                    if (j == r.j0) {               // the run's first: the accumulator has been read out
                        if (!rwait(bars.ofree + 8 * S, (nacc & 1u) ^ 1u, misc, a)) return false;
                        ++nacc;
                    }
                    const uint32_t vd = sw128_mnmajor_lo(sbase + lay.stages + stage * RowsSmem<D>::SB, RowsSmem<D>::HALF);
                    uint32_t more = j == r.j0 ? 0u : 1u;
                    if (r.ncols == 0) {
#pragma unroll 1
                        for (uint32_t o = 0; o < 2; ++o) {       // the upper 64 keys, then the lower
                            if (!rwait(bars.pready + 16 * S + 8 * o, o ? use1 : use0, misc, a)) return false;
                            tc_fence_after();
                            const bool lead = elect_one();
                            const uint32_t pd = tmem + S * TM_S + 64 * o, vh = vd + (o ^ 1u) * (64 * 128 >> 4);
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                umma_bf16_ta_lo(lead, od, pd + 8 * k, vh + k * (2048 >> 4), IDESC, k == 0 ? more : 1u);
                            umma_commit(lead, bars.pvdone + 16 * S + 8 * o);
                            if (o == 1) {
                                umma_commit(lead, bars.kvempty + 8 * stage);
                                if (j == r.last) umma_commit(lead, bars.ofull + 8 * S);
                            }
                            more = 1u;
                            __syncwarp();
                        }
                        ++use1;
                    } else {
                        if (!rwait(bars.pready + 16 * S, use0, misc, a)) return false;
                        tc_fence_after();
                        const bool lead = elect_one();
                        // O^T += V^T P^T: d on M, the rows on N, 64 keys per half of P^T
                        const uint32_t idesc = umma_idesc_bf16(D, 16, true) + ((r.ncols - 16) >> 3 << 17);
                        const uint32_t pd = sw128_kmajor_lo(sbase + lay.q + RowsSmem<D>::NP_OFF + S * RowsSmem<D>::NP);
#pragma unroll
                        for (int k = 0; k < ROWS_KEYS / 16; ++k)
                            umma_bf16_lo(lead, od, vd + k * (2048 >> 4),
                                         pd + (k >> 2) * (RowsSmem<D>::NQ_HALF >> 4) + (k & 3) * 2, idesc, k == 0 ? more : 1u);
                        umma_commit(lead, bars.pvdone + 16 * S);
                        umma_commit(lead, bars.kvempty + 8 * stage);
                        if (j == r.last) umma_commit(lead, bars.ofull + 8 * S);
                        __syncwarp();
                    }
                    ++use0;
                }
                stage += 2;
                if (stage >= (uint32_t)a.stages) { stage -= (uint32_t)a.stages; phase ^= 1u; }
            }
        }
    }
};

// ------------------------------------------------------------------------------------------
// softmax warps
// ------------------------------------------------------------------------------------------
// Whether V of a key of [k0, k1) that a row does not see, outside [lo, hi), is not finite in this warp's columns
// col + 32 i, or is not known (its block lies outside the pool). If not, a row that is not finite got there
// by the keys that it sees. (Any lo and hi: t only grows.)
template <int D, int NC>
__device__ __noinline__ bool unseen_values(const RowsArgs& a, int b, int g, int k0, int lo, int hi, int k1, int col,
                                           volatile int* misc)
{
    const __nv_bfloat16* vc = static_cast<const __nv_bfloat16*>(b < 0 && a.pv ? a.pv : a.v);
    bool found = false;
    for (int t = k0; t < k1; ++t) {
        if (t >= lo && t < hi) t = hi;
        if (t >= k1) break;
        if (((t - k0) & 1023) == 0) beat(misc);
        const long long off = key_offset(a, b, t, g);
        found = found || off < 0;
        if (off >= 0)
#pragma unroll
            for (int i = 0; i < NC; ++i) found = found || !(fabsf(__bfloat162float(vc[off + col + 32 * i])) < INFINITY);
    }
    return __any_sync(0xffffffffu, found);
}

// The keys [k0, k1) of a row again, for columns of its sums that are not finite: sums over the keys it
// sees alone, in the frame M. By one warp, four keys at a time (their loads and sums over the lanes overlap);
// o: its columns col + 32 i of each lane.
template <int D, int NC>
__device__ __noinline__ void redo_row(const RowsArgs& a, int b, int g, int h, int row, int pos, int k0, int k1, int base,
                                      float M, int col, float (&o)[NC], volatile int* misc)
{
    const int lane = threadIdx.x & 31;
    const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(a.q) + ((long long)row * a.Hq + h) * D;
    const __nv_bfloat16* kc = static_cast<const __nv_bfloat16*>(b < 0 && a.pk ? a.pk : a.k);
    const __nv_bfloat16* vc = static_cast<const __nv_bfloat16*>(b < 0 && a.pv ? a.pv : a.v);
    const float slope = a.slopes ? a.slopes[h] * LOG2E : 0.f, cap_rate = a.cap > 0.f ? 2.f * LOG2E * a.scale / a.cap : 0.f;
    float qr[D / 32];
#pragma unroll
    for (int i = 0; i < D / 32; ++i) qr[i] = __bfloat162float(q[lane + 32 * i]);
#pragma unroll
    for (int i = 0; i < NC; ++i) o[i] = 0.f;
    for (int t = k0; t < k1; t += 4) {
        if (((t - k0) & 4095) == 0) beat(misc);
        long long off[4];
        float s[4], v[4][NC];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            off[k] = t + k < k1 ? key_offset(a, b, t + k, g) : -1;      // (a block outside the pool: reported)
            s[k] = 0.f;
#pragma unroll
            for (int i = 0; i < D / 32; ++i)
                s[k] = fmaf(qr[i], off[k] < 0 ? 0.f : __bfloat162float(kc[off[k] + lane + 32 * i]), s[k]);
#pragma unroll
            for (int i = 0; i < NC; ++i) v[k][i] = off[k] < 0 ? 0.f : __bfloat162float(vc[off[k] + col + 32 * i]);
        }
#pragma unroll
        for (int w = 16; w > 0; w >>= 1)
#pragma unroll
            for (int k = 0; k < 4; ++k) s[k] += __shfl_xor_sync(0xffffffffu, s[k], w);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            if (off[k] < 0) continue;
            const float p = ex2(mod_score(s[k], a.scale, a.cap, cap_rate, slope, (float)(base + t + k - pos)) - M);
#pragma unroll
            for (int i = 0; i < NC; ++i) o[i] = fmaf(p, v[k][i], o[i]);
        }
        bool done = true;
#pragma unroll
        for (int i = 0; i < NC; ++i) done = done && o[i] != o[i];
        if (__all_sync(0xffffffffu, done)) break;       // NaN stays NaN
    }
}

__device__ __forceinline__ float max3(float a, float b, float c)
{
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

__device__ __forceinline__ float max32(const uint32_t* y)
{
    float m[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) m[k] = fmaxf(__uint_as_float(y[k]), __uint_as_float(y[k + 4]));
#pragma unroll
    for (int i = 8; i < 32; i += 8)
#pragma unroll
        for (int k = 0; k < 4; ++k) m[k] = max3(m[k], __uint_as_float(y[i + k]), __uint_as_float(y[i + 4 + k]));
    return max3(fmaxf(m[0], m[1]), m[2], m[3]);
}

// Two fp32 operations in one instruction.
__device__ __forceinline__ uint64_t pair2(float x, float y)
{
    uint64_t d;
    asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(x), "f"(y));
    return d;
}
__device__ __forceinline__ void unpair2(uint64_t d, float& x, float& y)
{
    asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(d));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c)
{
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b)
{
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b)
{
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}

// v[0 .. NR) of every lane, each combined over the warp: row lane / (32 / NR)'s in every lane. Each step hands half
// of the rows to the lane across, so that all rows together take NR + 1 exchanges at most (5 NR one by one).
template <int NR, typename Op>
__device__ __forceinline__ float warp_rows(float (&v)[NR], Op op)
{
    const int lane = threadIdx.x & 31;
    int bit = 16;
#pragma unroll
    for (int k = NR / 2; k > 0; k >>= 1, bit >>= 1) {
        const bool up = lane & bit;
#pragma unroll
        for (int i = 0; i < k; ++i) {
            const float keep = up ? v[i + k] : v[i], give = up ? v[i] : v[i + k];
            v[i] = op(keep, __shfl_xor_sync(0xffffffffu, give, bit));
        }
    }
    float x = v[0];
#pragma unroll
    for (int b = 16 / NR; b > 0; b >>= 1) x = op(x, __shfl_xor_sync(0xffffffffu, x, b));
    return x;
}

template <int NR>
__device__ __forceinline__ void tmem_ld_rows(uint32_t taddr, uint32_t (&r)[NR])
{
    if constexpr (NR == 32) {
        tmem_ld32_async(taddr, r);
    } else if constexpr (NR == 16) {
        tmem_ld16_async(taddr, r);
    } else {
        asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                     : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                     : "r"(taddr));
    }
}

__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t* r)
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, "
        "%13, %14, %15};" ::"r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
        "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(taddr)
        : "memory");
}

template <int NR>
__device__ __forceinline__ void tmem_st_rows(uint32_t taddr, const uint32_t (&r)[NR])
{
#pragma unroll
    for (int i = 0; i < NR; i += 8)
        asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%8], {%0, %1, %2, %3, %4, %5, %6, %7};" ::"r"(r[i]),
                     "r"(r[i + 1]), "r"(r[i + 2]), "r"(r[i + 3]), "r"(r[i + 4]), "r"(r[i + 5]), "r"(r[i + 6]),
                     "r"(r[i + 7]), "r"(taddr + i)
                     : "memory");
}

__device__ __forceinline__ float abs_max64(const uint32_t* y)
{
    float m[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < 64; i += 8)
#pragma unroll
        for (int k = 0; k < 4; ++k)
            asm("max.abs.f32 %0, %0, %1, %2;" : "+f"(m[k]) : "f"(__uint_as_float(y[i + k])), "f"(__uint_as_float(y[i + 4 + k])));
    return fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3]));
}

// Scores up to CAP_NEAR of their cap (most are far below it) are capped by tanh(z) / z as a polynomial in z^2,
// interpolated at the Chebyshev points: 2^-23 of itself off. It takes five operations of the FMA pipe where the exact
// form takes four and a half and two and a half of the MUFU: a prompt of 8192 tokens 631 us where all
// scores are near (a cap of 30), and 838 where few half tiles have none beyond (a cap of 2).
constexpr float CAP_NEAR = 0.35f;

// Ties the registers to the tcgen05.wait::ld before it.
template <int NR>
__device__ __forceinline__ void reg_fence(uint32_t (&r)[NR])
{
#pragma unroll
    for (int i = 0; i < NR; ++i) asm volatile("" : "+r"(r[i]) : : "memory");
}

// How scores become v, in units of log2: scale alone; scale and bias; cap, scale and bias.
enum { MODE_PLAIN = 0, MODE_BIAS = 1, MODE_CAP = 2 };

template <int D, int MODE>
struct Softmax {
    const RowsArgs& a;
    const RowsSmem<D>& lay;
    const RowsBars& bars;
    uint8_t* sm;
    uint32_t tmem;
    volatile int* misc;
    int S;                   // the stream
    // phases passed: headers, this stream's tiles, and the lower halves of those in 128-row runs, runs of either
    // stream's accumulator, its own hand-overs, meetings of this stream's warps, Q buffers
    uint32_t nh = 0, ntile = 0, nlow = 0, nacc = 0, nacc_o = 0, nml = 0, nvote = 0, nqn = 0;

    struct Run {
        int g, b, tok0, ntok, len, t0, t1, dest, flags, base, s0, s1;
        bool other_tiles;
    };

    __device__ __forceinline__ bool run()
    {
        const int lane = threadIdx.x & 31;
        bool ok = true;
        for (;; ++nh) {
            const uint32_t hs = nh % RW_HDRS;
            if (!rwait(bars.hfull + 8 * hs, (nh / RW_HDRS) & 1u, misc, a)) { ok = false; break; }
            const int* h = reinterpret_cast<const int*>(sm + lay.hdr + hs * RW_HDR_BYTES);
            const int kind = h[RH_KIND];
            Run r;
            r.g = h[RH_G]; r.b = h[RH_B]; r.tok0 = h[RH_TOK0]; r.ntok = h[RH_NTOK]; r.len = h[RH_LEN];
            r.t0 = h[RH_T0]; r.t1 = h[RH_T1]; r.dest = h[RH_DEST]; r.flags = h[RH_FLAGS]; r.base = h[RH_BASE];
            r.s0 = S ? h[RH_B0] : h[RH_A0];
            r.s1 = S ? h[RH_B1] : h[RH_A1];
            r.other_tiles = S ? h[RH_A1] > h[RH_A0] : h[RH_B1] > h[RH_B0];      // (pairs)
            __syncwarp();
            if (lane == 0) mbar_arrive(bars.hempty + 8 * hs);
            if (kind == RUN_END) break;
            if (r.flags & RF_NARROW) {
                const int rows = r.ntok * a.G;
                ok = rows <= 8 ? narrow<8>(r) : rows <= 16 ? narrow<16>(r) : narrow<32>(r);
            } else {
                ok = wide(r);
            }
            if (!ok) break;
        }
        return ok;
    }

    // ---- 128 rows on the lanes ----
    __device__ __forceinline__ bool wide(const Run& run)
    {
        const int lane = threadIdx.x & 31, r = threadIdx.x & (ROWS_TILE - 1);
        const uint32_t lane_base = (uint32_t)(r & ~31) << 16;
        const uint32_t ts = tmem + lane_base + S * TM_S, to = tmem + lane_base + 2 * TM_S;
        float2* ml = reinterpret_cast<float2*>(sm + lay.ml);
        const bool pair = run.flags & RF_PAIR;
        const int start = (run.flags & RF_START) ? 1 : 0, t0 = run.t0, t1 = run.t1, base = run.base;
        // this stream's tiles, from the last key on (the bias grows towards the row's own position, so a
        // row's largest scores tend to come first): first, first - step, .. down to `least`
        const int first = pair ? run.s1 - 1 : t1 - 1 - (S ^ start), least = pair ? run.s0 : t0, step = pair ? 1 : 2;
        const int ti = r / a.G, hh = r - ti * a.G;
        const int tok = run.tok0 + (pair ? S * a.tpt : 0) + ti;
        const bool live = ti < a.tpt && tok < run.tok0 + run.ntok;
        const bool warp_live = __any_sync(0xffffffffu, live);
        RowToken tk{0, 0, 0, -1};
        if (live) tk = a.tok[tok];
        const bool mine = live && tk.rt >= 0;
        // keys of this source that the row sees; a lane without a row masks nothing, is not written, and has no say in
        // what the warp does for its rows (its scores may come from what shared memory held before the call)
        int lo = mine ? max(tk.lo - base, 0) : 0, hi = mine ? min(tk.hi - base, run.len) : INT32_MAX;
        if (mine && hi <= lo) lo = hi = 0;
        const bool empty = hi <= lo;
        float slope = 0.f;
        if (MODE != MODE_PLAIN && a.slopes && live) slope = a.slopes[run.g * a.G + hh] * LOG2E;
        const int spos = tk.pos - base;                  // the position in this source's indexes
        const float rate = a.scale * LOG2E;
        const float cap_rate = MODE == MODE_CAP ? 2.f * LOG2E * a.scale / a.cap : 0.f;
        // every visible key is at or before the position: the bias is linear in the key
        const bool linear = __all_sync(0xffffffffu, !mine || hi <= spos + 1);
        // (a mask for ballots: with the predicate in votes, a prompt of 8192 tokens took 646 to 716 us under a cap, this
        // way 631; without a cap 423 to 431 both ways)
        const unsigned rows = __ballot_sync(0xffffffffu, mine);
        float m = -INFINITY, l = 0.f;                    // frame (log2 units) and sum
        int count = 0;
        for (int t = first; t >= least; t -= step) {
#pragma unroll 1
          for (int half = 1; half >= 0; --half, ++count) {
            const uint32_t buf = half ? 0u : 1u;
            if (!rwait(bars.sfull + 16 * S + 8 * buf, half ? ntile : nlow, misc, a)) return false;
            tc_fence_after();
            if (warp_live) {
                const int k0 = t * ROWS_KEYS + 64 * half;
                const uint32_t tb = ts + 64 * buf;
                // Half tiles with masked scores, or a bias that is not linear in the key: v (masked: -inf) back
                // to tensor memory first, by a rolled loop, since code that few tiles need costs more to fetch
                // than it saves.
                const bool open = __all_sync(0xffffffffu, lo <= k0 && hi >= k0 + 64);
                const bool ready_v = MODE == MODE_PLAIN || (open && (linear || !a.slopes));
                if (!open || !ready_v) {
#pragma unroll 1
                    for (int c = 0; c < 2; ++c) {
                        uint32_t y[32];
                        tmem_ld32_async(tb + 32 * c, y);
                        tmem_wait_ld();
                        reg_fence32(y);
                        const int kc = k0 + 32 * c, c0 = lo - kc, c1 = hi - kc;
                        const float d0 = (float)(kc - spos);
#pragma unroll
                        for (int i = 0; i < 32; i += 2) {
                            // a masked score may be anything, and one that is NaN would take its neighbour along
                            const bool in0 = i >= c0 && i < c1, in1 = i + 1 >= c0 && i + 1 < c1;
                            float v0 = in0 ? __uint_as_float(y[i]) : 0.f, v1 = in1 ? __uint_as_float(y[i + 1]) : 0.f;
                            if (MODE == MODE_CAP) {
                                cap_pair(v0, v1, cap_rate, LOG2E * a.cap);
                                v0 = fmaf(-slope, fabsf(d0 + (float)i), v0);
                                v1 = fmaf(-slope, fabsf(d0 + (float)(i + 1)), v1);
                            } else if (MODE == MODE_BIAS) {
                                v0 = mod_score(v0, a.scale, 0.f, 0.f, slope, d0 + (float)i);
                                v1 = mod_score(v1, a.scale, 0.f, 0.f, slope, d0 + (float)(i + 1));
                            }
                            y[i] = __float_as_uint(in0 ? v0 : -INFINITY);
                            y[i + 1] = __float_as_uint(in1 ? v1 : -INFINITY);
                        }
                        tmem_st32(tb + 32 * c, y);
                    }
                    tmem_wait_st();
                }
                uint32_t x[64];
                tmem_ld32_async(tb, x);
                tmem_ld32_async(tb + 32, x + 32);
                tmem_wait_ld();
                reg_fence32(x);
                reg_fence32(x + 32);
                if (MODE == MODE_CAP && ready_v) {
                    // (between these ratios the polynomial's coefficients are normal numbers: (scale / cap)^6 and the
                    // largest cap leave them below 2^125)
                    const unsigned far = __ballot_sync(0xffffffffu, abs_max64(x) * a.scale > CAP_NEAR * a.cap) & rows;
                    if (a.scale >= 1e-5f * a.cap && a.scale <= 1e5f * a.cap && !far) {
                        // v = y (rate p(z^2)), the coefficients taken with their powers of z / y
                        const float zz = (a.scale / a.cap) * (a.scale / a.cap);
                        const float k0_ = rate, k1_ = -0.333324194f * zz * rate, k2_ = 0.132957518f * zz * zz * rate,
                                    k3_ = -0.048955638f * zz * zz * zz * rate;
#pragma unroll
                        for (int i = 0; i < 64; i += 2) {
                            const uint64_t y = pair2(__uint_as_float(x[i]), __uint_as_float(x[i + 1])), u = mul2(y, y);
                            uint64_t p = fma2(u, pair2(k3_, k3_), pair2(k2_, k2_));
                            p = fma2(p, u, pair2(k1_, k1_));
                            p = fma2(p, u, pair2(k0_, k0_));
                            float v0, v1;
                            unpair2(mul2(y, p), v0, v1);
                            x[i] = __float_as_uint(v0);
                            x[i + 1] = __float_as_uint(v1);
                        }
                    } else {                             // (as cap_pair, two operations at a time)
                        const float top = LOG2E * a.cap;
                        const uint64_t cr2 = pair2(cap_rate, cap_rate), one2 = pair2(1.f, 1.f), top2 = pair2(top, top),
                                       slope_top2 = pair2(-2.f * top, -2.f * top);
#pragma unroll
                        for (int i = 0; i < 64; i += 2) {
                            float t0, t1, e0, e1, v0, v1;
                            unpair2(mul2(pair2(__uint_as_float(x[i]), __uint_as_float(x[i + 1])), cr2), t0, t1);
                            asm("min.NaN.f32 %0, %0, 0f42700000;" : "+f"(t0));
                            asm("min.NaN.f32 %0, %0, 0f42700000;" : "+f"(t1));
                            unpair2(add2(pair2(ex2(t0), ex2(t1)), one2), e0, e1);
                            const float r = rcp(e0 * e1);
                            unpair2(fma2(mul2(pair2(e1, e0), pair2(r, r)), slope_top2, top2), v0, v1);
                            x[i] = __float_as_uint(v0);
                            x[i + 1] = __float_as_uint(v1);
                        }
                    }
                    if (a.slopes) {
                        const float b0 = slope * (float)(k0 - spos);
#pragma unroll
                        for (int i = 0; i < 64; ++i)
                            x[i] = __float_as_uint(__uint_as_float(x[i]) + fmaf(slope, (float)i, b0));
                    }
                }
                if (MODE == MODE_BIAS && ready_v) {
                    const float b0 = slope * (float)(k0 - spos);
                    const uint64_t rate2 = pair2(rate, rate);
#pragma unroll
                    for (int i = 0; i < 64; i += 2) {
                        float v0, v1;
                        unpair2(fma2(pair2(__uint_as_float(x[i]), __uint_as_float(x[i + 1])), rate2,
                                     pair2(fmaf(slope, (float)i, b0), fmaf(slope, (float)(i + 1), b0))), v0, v1);
                        x[i] = __float_as_uint(v0);
                        x[i + 1] = __float_as_uint(v1);
                    }
                }
                float top = fmaxf(max32(x), max32(x + 32));
                if (MODE == MODE_PLAIN) top *= rate;
                if (count == 0) {
                    m = top;
                } else if (__ballot_sync(0xffffffffu, top > (m == -INFINITY ? -INFINITY : m + RW_LAG)) & rows) {
                    // move the frame, once the P V of the half before is complete (the one before that is: its
                    // buffer has held these scores since)
                    if (!rwait(bars.pvdone + 16 * S + 8 * (buf ^ 1u), (half ? nlow : ntile) - 1u, misc, a)) return false;
                    tc_fence_after();
                    const float f = fmaxf(m, top), wt = m == f ? 1.f : ex2(m - f);
                    m = f;
                    l *= wt;
#pragma unroll 1
                    for (int i = 0; i < D; i += 16) {
                        uint32_t o[16];
                        tmem_ld16_async(to + S * D + i, o);
                        tmem_wait_ld();
                        reg_fence16(o);
#pragma unroll
                        for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * wt);
                        tmem_st16(to + S * D + i, o);
                    }
                }
                // the weights, two to a register
                const float mu = m == -INFINITY ? 0.f : m;
                const uint64_t nmu = pair2(-mu, -mu), rate2 = pair2(rate, rate);
                uint64_t s0 = pair2(0.f, 0.f), s1 = s0;
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    uint32_t* y = x + 32 * c;
#pragma unroll
                    for (int i = 0; i < 32; i += 4) {
                        uint64_t v0 = pair2(__uint_as_float(y[i]), __uint_as_float(y[i + 1]));
                        uint64_t v1 = pair2(__uint_as_float(y[i + 2]), __uint_as_float(y[i + 3]));
                        if (MODE == MODE_PLAIN) { v0 = fma2(v0, rate2, nmu); v1 = fma2(v1, rate2, nmu); }
                        else { v0 = add2(v0, nmu); v1 = add2(v1, nmu); }
                        float p0, p1, p2, p3;
                        unpair2(v0, p0, p1);
                        unpair2(v1, p2, p3);
                        p0 = ex2(p0); p1 = ex2(p1); p2 = ex2(p2); p3 = ex2(p3);
                        s0 = add2(s0, pair2(p0, p1));
                        s1 = add2(s1, pair2(p2, p3));
                        y[i / 2] = pack_bf16x2(p0, p1);
                        y[i / 2 + 1] = pack_bf16x2(p2, p3);
                    }
                    tmem_st16(tb + 16 * c, y);
                }
                float p0, p1;
                unpair2(add2(s0, s1), p0, p1);
                l += p0 + p1;
                tmem_wait_st();
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bars.pready + 16 * S + 8 * buf);
            if (half) ++ntile; else ++nlow;
          }
        }

        // ---- the run's end ----
        const int O = S ^ 1;
        if (!pair && S != start) {                       // hand over to the other stream
            if (count > 0) {
                if (!rwait(bars.mlfree + 8 * S, (nml & 1u) ^ 1u, misc, a)) return false;
                ml[S * ROWS_TILE + r] = make_float2(m, l);
                tell();
                ++nml;
                ++nacc;
            }
            ++nacc_o;
            return true;
        }
        const bool other = !pair && t1 - t0 > 1;         // the other stream had tiles of these rows
        float wo = 0.f, ws = 1.f;                        // the streams' weights
        if (count > 0 && !rwait(bars.ofull + 8 * S, nacc & 1u, misc, a)) return false;
        if (other) {
            if (!told(O)) return false;
            const float2 x = ml[O * ROWS_TILE + r];
            __syncwarp();
            if (lane == 0) mbar_arrive(bars.mlfree + 8 * O);
            if (!rwait(bars.ofull + 8 * O, nacc_o & 1u, misc, a)) return false;
            const float f = fmaxf(m, x.x);
            ws = m == f ? 1.f : ex2(m - f);
            wo = x.x == f ? 1.f : ex2(x.x - f);
            l = l * ws + x.y * wo;
            m = f;
        }
        tc_fence_after();
        const int head = run.g * a.G + hh;
        const bool direct = run.dest == DEST_OUT;
        // the row's place in out, in a slot or in the whole-unit arrays
        long long at = -1;
        if (mine) {
            if (direct) at = (long long)tok * a.Hq + head;
            else if (run.dest == DEST_ROWS) at = ((run.b < 0 ? 0ll : (long long)a.T) + tok) * a.Hq + head;
            else at = (long long)run.dest * a.slot_rows + (tok - run.tok0) * a.G + hh;
            if (!direct) (run.dest == DEST_ROWS ? a.row_ml : a.slot_ml)[at] = make_float2(count > 0 ? m : -INFINITY, l);
        }
        float* pbase = run.dest == DEST_ROWS ? a.row_o : a.slot_o;
        bool fine = true;
        if (warp_live && (count > 0 || direct)) {
            const float inv = direct ? 1.f / l : 1.f;
            // 128 bytes of every row at a time: turned through shared memory (16-byte pieces of row r at
            // piece ^ (r & 7)), so that a store instruction writes four whole lines
            uint8_t* turn = sm + lay.turn + (threadIdx.x >> 5) * RowsSmem<D>::TURN;
            const int cols = direct ? 64 : 32;
#pragma unroll 1
            for (int i = 0; i < D; i += cols) {
#pragma unroll 1
                for (int c = 0; c < cols; c += 32) {
                    uint32_t x[32];
#pragma unroll
                    for (int k = 0; k < 32; ++k) x[k] = 0u;
                    if (count > 0) {
                        tmem_ld32_async(to + S * D + i + c, x);
                        if (other) {
                            uint32_t y[32];
                            tmem_ld32_async(to + O * D + i + c, y);
                            tmem_wait_ld();
                            reg_fence32(x);
                            reg_fence32(y);
#pragma unroll
                            for (int k = 0; k < 32; ++k)
                                x[k] = __float_as_uint(__uint_as_float(x[k]) * ws + __uint_as_float(y[k]) * wo);
                        } else {
                            tmem_wait_ld();
                            reg_fence32(x);
                        }
                    }
#pragma unroll
                    for (int k = 0; k < 32; ++k) fine = fine && fabsf(__uint_as_float(x[k])) < INFINITY;
                    if (direct) {
#pragma unroll
                        for (int k = 0; k < 32; k += 8) {
                            uint4 v = make_uint4(0, 0, 0, 0);
                            if (!empty)
                                v = make_uint4(pack_bf16x2(__uint_as_float(x[k]) * inv, __uint_as_float(x[k + 1]) * inv),
                                               pack_bf16x2(__uint_as_float(x[k + 2]) * inv, __uint_as_float(x[k + 3]) * inv),
                                               pack_bf16x2(__uint_as_float(x[k + 4]) * inv, __uint_as_float(x[k + 5]) * inv),
                                               pack_bf16x2(__uint_as_float(x[k + 6]) * inv, __uint_as_float(x[k + 7]) * inv));
                            *reinterpret_cast<uint4*>(turn + lane * 128 + ((((c + k) >> 3) ^ (lane & 7)) << 4)) = v;
                        }
                    } else {
#pragma unroll
                        for (int k = 0; k < 32; k += 4)
                            *reinterpret_cast<uint4*>(turn + lane * 128 + (((k >> 2) ^ (lane & 7)) << 4)) =
                                make_uint4(x[k], x[k + 1], x[k + 2], x[k + 3]);
                    }
                }
                __syncwarp();
#pragma unroll
                for (int k = 0; k < 32; k += 4) {
                    const int row = k + (lane >> 3), piece = lane & 7;
                    const long long rat = __shfl_sync(0xffffffffu, at, row);
                    const uint4 v = *reinterpret_cast<const uint4*>(turn + row * 128 + ((piece ^ (row & 7)) << 4));
                    if (rat >= 0) {
                        if (direct) *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.out) + rat * D + i + 8 * piece) = v;
                        else *reinterpret_cast<uint4*>(pbase + rat * D + i + 4 * piece) = v;
                    }
                }
                __syncwarp();
            }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
            if (count > 0) mbar_arrive(bars.ofree + 8 * S);
            if (other) mbar_arrive(bars.ofree + 8 * O);
        }
        // Rows that may have met a non-finite V of a key they do not see
        const int seen0 = (pair ? run.s0 : t0) * ROWS_KEYS, seen1 = min((pair ? run.s1 : t1) * ROWS_KEYS, run.len);
        // (one that sees none of the run's keys leaves an empty partial, which the join passes over)
        const bool again = mine && count > 0 && !fine && max(lo, seen0) < min(hi, seen1) && fabsf(l) < INFINITY &&
                           (lo > seen0 || hi < seen1);
        unsigned todo = __ballot_sync(0xffffffffu, again);
        while (todo) {
            beat(misc);
            const int j = __ffs(todo) - 1;
            todo &= todo - 1;
            const int jtok = __shfl_sync(0xffffffffu, tok, j), jhead = __shfl_sync(0xffffffffu, head, j);
            const int jpos = __shfl_sync(0xffffffffu, tk.pos, j);
            const int jlo = max(__shfl_sync(0xffffffffu, lo, j), seen0), jhi = min(__shfl_sync(0xffffffffu, hi, j), seen1);
            const float jm = __shfl_sync(0xffffffffu, m, j), jl = __shfl_sync(0xffffffffu, l, j);
            const long long jat = __shfl_sync(0xffffffffu, at, j);
            if (!unseen_values<D, D / 32>(a, run.b, run.g, seen0, jlo, jhi, seen1, lane, misc)) continue;
            float o[D / 32];
            redo_row<D, D / 32>(a, run.b, run.g, jhead, jtok, jpos, jlo, jhi, base, jm == -INFINITY ? 0.f : jm, lane, o, misc);
#pragma unroll
            for (int i = 0; i < D / 32; ++i) {
                if (direct) static_cast<__nv_bfloat16*>(a.out)[jat * D + lane + 32 * i] = __float2bfloat16_rn(o[i] / jl);
                else pbase[jat * D + lane + 32 * i] = o[i];
            }
        }
        if (count > 0) ++nacc;
        if (pair ? run.other_tiles : other) ++nacc_o;
        return true;
    }

    // A stream's maxima and sums of run nh, for whichever stream joins the two. Neither stream waits for
    // the other's runs in general, so either may be some runs ahead: a run number per warp, which a
    // barrier's one bit of phase could not tell apart.
    __device__ __forceinline__ void tell() const
    {
        __syncwarp();
        if ((threadIdx.x & 31) == 0) {
            __threadfence_block();
            misc[MISC_TOLD + (threadIdx.x >> 5)] = (int)nh + 1;
        }
        __syncwarp();
    }
    __device__ __forceinline__ bool told(int s) const
    {
        const int lane = threadIdx.x & 31;
        uint64_t t0 = global_ns();
        int last = 0;
        for (uint32_t it = 1;; ++it) {
            const int v = lane < 4 ? misc[MISC_TOLD + 4 * s + lane] : INT32_MAX;
            if (__all_sync(0xffffffffu, v > (int)nh)) break;
            if ((it & 63u) == 0) {
                const bool late = misc[MISC_ABORT] != 0 || run_out(misc, t0, last);
                if (__any_sync(0xffffffffu, late)) {
                    if (lane == 0) {
                        misc[MISC_ABORT] = 1;
                        rows_error(a, FDPP_ERRBIT_TIMEOUT);
                    }
                    return false;
                }
            }
        }
        __threadfence_block();
        return true;
    }

    // The four warps of this stream meet (bounded).
    __device__ __forceinline__ bool meet()
    {
        __syncwarp();
        if ((threadIdx.x & 31) == 0) mbar_arrive(bars.vote + 8 * S);
        const bool ok = rwait(bars.vote + 8 * S, nvote & 1u, misc, a);
        ++nvote;
        return ok;
    }

    // ---- up to 32 rows, the keys on the lanes ----
    // A thread holds one key of each tile for all NR rows: S^T comes from tensor memory as NR columns,
    // the weights go to shared memory as the K-major operand P^T, and O^T has d on its lanes. The rows'
    // frames are the same in all threads: the warps meet once a tile to see whether a score is beyond its
    // row's frame by more than the lag, and exchange maxima only then.
    template <int NR>
    __device__ __forceinline__ bool narrow(const Run& run)
    {
        constexpr int CH = NR < 16 ? NR : 16;
        const int O = S ^ 1;
        const int lane = threadIdx.x & 31, w = (threadIdx.x >> 5) & 3;
        const uint32_t lane_base = (uint32_t)(32 * w) << 16;
        const uint32_t ts = tmem + lane_base + S * TM_S, to = tmem + lane_base + 2 * TM_S;
        volatile NarrowShared& sh = *reinterpret_cast<volatile NarrowShared*>(sm + lay.nsh);
        uint8_t* prow = sm + lay.q + RowsSmem<D>::NP_OFF + S * RowsSmem<D>::NP + (w >> 1) * RowsSmem<D>::NQ_HALF;
        const int pcol = ((w & 1) * 32 + lane) * 2;
        const int start = (run.flags & RF_START) ? 1 : 0, base = run.base, R = run.ntok * a.G;
        // row `lane` (of the rows < R): token, head, keys
        const int ti = lane / a.G, hh = lane - ti * a.G, tok = run.tok0 + ti, head = run.g * a.G + hh;
        RowToken tk{0, 0, 0, -1};
        if (lane < R) tk = a.tok[tok];
        const bool mine = lane < R && tk.rt >= 0;
        int lo = 0, hi = 0;
        if (mine) {
            lo = max(tk.lo - base, 0);
            hi = min(tk.hi - base, run.len);
            if (hi <= lo) lo = hi = 0;
        }
        const int all_lo = warp_max(mine ? lo : 0), all_hi = warp_min(mine ? hi : INT32_MAX);
        float slope_l = 0.f;
        if (MODE != MODE_PLAIN && a.slopes && lane < R) slope_l = a.slopes[head] * LOG2E;
        const int spos_l = tk.pos - base;
        float fr[NR], l[NR];
#pragma unroll
        for (int r = 0; r < NR; ++r) {
            fr[r] = -INFINITY;
            l[r] = 0.f;
        }
        const float rate = a.scale * LOG2E;
        const float cap_rate = MODE == MODE_CAP ? 2.f * LOG2E * a.scale / a.cap : 0.f;
        const bool solo = run.flags & RF_SOLO;
        const int step = solo ? 1 : 2, top = solo ? (S == start ? run.t1 - 1 : run.t0 - 1) : run.t1 - 1 - (S ^ start);
        int count = 0;
        for (int t = top; t >= run.t0; t -= step, ++ntile, ++count) {
            if (!rwait(bars.sfull + 16 * S, ntile, misc, a)) return false;
            tc_fence_after();
            const int k0 = t * ROWS_KEYS, key = k0 + 32 * w + lane;
            const bool open = all_lo <= k0 && all_hi >= k0 + ROWS_KEYS;
            // v of CH rows from row c on. Sixteen rows at most are held at a time: with 32 their scores are
            // read from tensor memory again for each step.
            auto load = [&](int c, float (&v)[CH]) {
                uint32_t x[CH];
                tmem_ld_rows<CH>(ts + c, x);
                tmem_wait_ld();
                reg_fence<CH>(x);
#pragma unroll
                for (int i = 0; i < CH; ++i) {
                    if (MODE == MODE_PLAIN) {
                        v[i] = __uint_as_float(x[i]) * rate;
                    } else {
                        const float slope = __shfl_sync(0xffffffffu, slope_l, c + i);
                        const int spos = __shfl_sync(0xffffffffu, spos_l, c + i);
                        v[i] = mod_score(__uint_as_float(x[i]), a.scale, MODE == MODE_CAP ? a.cap : 0.f, cap_rate, slope,
                                         (float)(key - spos));
                    }
                    if (c + i >= R) v[i] = -INFINITY;
                }
                if (!open) {
#pragma unroll
                    for (int i = 0; i < CH; ++i) {
                        const int rlo = __shfl_sync(0xffffffffu, lo, c + i), rhi = __shfl_sync(0xffffffffu, hi, c + i);
                        if (key < rlo || key >= rhi) v[i] = -INFINITY;
                    }
                }
            };
            float v[CH];
            bool move = count == 0;                      // a run's first tile sets the frames
            if (CH < NR || !move) {
                bool beyond = false;
#pragma unroll
                for (int c = 0; c < NR; c += CH) {
                    load(c, v);
#pragma unroll
                    for (int i = 0; i < CH; ++i) beyond = beyond || v[i] > fr[c + i] + RW_LAG;
                }
                if (!move) {
                    beyond = __any_sync(0xffffffffu, beyond);
                    const uint32_t par = nvote & 1u;
                    if (lane == 0) sh.flag[S][par][w] = beyond;
                    if (!meet()) return false;
                    move = (sh.flag[S][par][0] | sh.flag[S][par][1] | sh.flag[S][par][2] | sh.flag[S][par][3]) != 0;
                }
            } else {
                load(0, v);
            }
            if (move) {
#pragma unroll
                for (int c = 0; c < NR; c += CH) {
                    if (CH < NR) load(c, v);
                    float x[CH];
#pragma unroll
                    for (int i = 0; i < CH; ++i) x[i] = v[i];
                    const float top = warp_rows(x, [](float p, float q) { return fmaxf(p, q); });
                    if (lane % (32 / CH) == 0) sh.wmax[S][w][c + lane / (32 / CH)] = top;
                }
                if (!meet()) return false;
#pragma unroll
                for (int c = 0; c < NR; c += 8) {
                    uint32_t o[8];
                    if (count > 0) {
                        tmem_ld_rows<8>(to + S * D + c, o);
                        tmem_wait_ld();
                        reg_fence<8>(o);
                    }
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const int r = c + i;
                        const float f = fmaxf(fmaxf(fr[r], fmaxf(sh.wmax[S][0][r], sh.wmax[S][1][r])),
                                              fmaxf(sh.wmax[S][2][r], sh.wmax[S][3][r]));
                        const float wt = fr[r] == f ? 1.f : ex2(fr[r] - f);
                        fr[r] = f;
                        l[r] *= wt;
                        if (count > 0) o[i] = __float_as_uint(__uint_as_float(o[i]) * wt);
                    }
                    if (count > 0) tmem_st_rows<8>(to + S * D + c, o);
                }
                tmem_wait_st();
            }
#pragma unroll
            for (int c = 0; c < NR; c += CH) {
                if (CH < NR) load(c, v);
#pragma unroll
                for (int i = 0; i < CH; ++i) {
                    const int r = c + i;
                    const float p = ex2(v[i] - (fr[r] == -INFINITY ? 0.f : fr[r]));
                    l[r] += p;
                    *reinterpret_cast<__nv_bfloat16*>(prow + r * 128 + (pcol ^ ((r & 7) << 4))) = __float2bfloat16_rn(p);
                }
            }
            fence_proxy_async_smem();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bars.pready + 16 * S);
        }

        // ---- the run's end ----
        if (count > 0) {
            if (!rwait(bars.mlfree + 8 * S, (nml & 1u) ^ 1u, misc, a)) return false;
            if (w == 0 && lane == 0) {
#pragma unroll
                for (int r = 0; r < NR; ++r) sh.frame[S][r] = fr[r];
            }
            const float x = warp_rows(l, [](float p, float q) { return p + q; });
            if (lane % (32 / NR) == 0) sh.lsum[S][w][lane / (32 / NR)] = x;
            tell();
            ++nml;
        }
        const bool other = !solo && run.t1 - run.t0 > 1; // both streams had tiles
        if (S != start) {
            if (count > 0) ++nacc;
            ++nacc_o;
            ++nqn;
            return true;
        }
        if (!told(S)) return false;
        if (!rwait(bars.ofull + 8 * S, nacc & 1u, misc, a)) return false;
        if (other) {
            if (!told(O)) return false;                  // (and so the accumulator's phase is this run's)
            if (!rwait(bars.ofull + 8 * O, nacc_o & 1u, misc, a)) return false;
        }
        tc_fence_after();
        // row `lane`: both streams' frames and sums joined
        float m = -INFINITY, lt = 0.f, ws = 1.f, wo = 0.f;
        if (lane < NR) {
            m = sh.frame[S][lane];
            lt = (sh.lsum[S][0][lane] + sh.lsum[S][1][lane]) + (sh.lsum[S][2][lane] + sh.lsum[S][3][lane]);
            if (other) {
                const float mo = sh.frame[O][lane], f = fmaxf(m, mo);
                const float lo_ = (sh.lsum[O][0][lane] + sh.lsum[O][1][lane]) + (sh.lsum[O][2][lane] + sh.lsum[O][3][lane]);
                ws = m == f ? 1.f : ex2(m - f);
                wo = mo == f ? 1.f : ex2(mo - f);
                lt = lt * ws + lo_ * wo;
                m = f;
            }
        }
        const bool direct = run.dest == DEST_OUT;
        const bool has = D == 128 || lane < 16;           // a 64-row accumulator leaves lanes 16-31 out
        const int d = D == 128 ? 32 * w + lane : 16 * w + (lane & 15);
        long long at = 0;                                 // the row's place: out, a slot or the whole-unit arrays
        if (direct) at = (long long)tok * a.Hq + head;
        else if (run.dest == DEST_ROWS) at = ((run.b < 0 ? 0ll : (long long)a.T) + tok) * a.Hq + head;
        else at = (long long)run.dest * a.slot_rows + lane;
        float* pbase = run.dest == DEST_ROWS ? a.row_o : a.slot_o;
        if (!direct && mine && w == 0) (run.dest == DEST_ROWS ? a.row_ml : a.slot_ml)[at] = make_float2(m, lt);
        const float inv_l = 1.f / lt;
        const bool empty_l = hi <= lo;
        unsigned todo = 0;
#pragma unroll 1
        for (int c = 0; c < NR; c += 8) {
            uint32_t x[8], y[8] = {0, 0, 0, 0, 0, 0, 0, 0};
            tmem_ld_rows<8>(to + S * D + c, x);
            if (other) tmem_ld_rows<8>(to + O * D + c, y);
            tmem_wait_ld();
            reg_fence<8>(x);
            reg_fence<8>(y);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int r = c + i;
                const float rws = __shfl_sync(0xffffffffu, ws, r), rwo = __shfl_sync(0xffffffffu, wo, r);
                const float inv = __shfl_sync(0xffffffffu, inv_l, r);
                const long long rat = __shfl_sync(0xffffffffu, at, r);
                const bool rmine = __shfl_sync(0xffffffffu, (int)mine, r), rempty = __shfl_sync(0xffffffffu, (int)empty_l, r);
                float val = __uint_as_float(x[i]);
                if (other) val = val * rws + __uint_as_float(y[i]) * rwo;
                if (__any_sync(0xffffffffu, has && !(fabsf(val) < INFINITY))) todo |= 1u << r;
                if (!rmine || !has) continue;
                if (direct) static_cast<__nv_bfloat16*>(a.out)[rat * D + d] = __float2bfloat16_rn(rempty ? 0.f : val * inv);
                else pbase[rat * D + d] = val;
            }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
            mbar_arrive(bars.ofree + 8 * S);
            mbar_arrive(bars.mlfree + 8 * S);
            if (other) {
                mbar_arrive(bars.ofree + 8 * O);
                mbar_arrive(bars.mlfree + 8 * O);
            }
        }
        // Rows that may have met a non-finite V of a key they do not see: this warp's columns again
        const int seen0 = run.t0 * ROWS_KEYS, seen1 = min(run.t1 * ROWS_KEYS, run.len);
        todo &= __ballot_sync(0xffffffffu, mine && max(lo, seen0) < min(hi, seen1) && fabsf(lt) < INFINITY &&
                                               (lo > seen0 || hi < seen1));
        __syncwarp();
        while (todo) {
            beat(misc);
            const int j = __ffs(todo) - 1;
            todo &= todo - 1;
            const int jtok = __shfl_sync(0xffffffffu, tok, j), jhead = __shfl_sync(0xffffffffu, head, j);
            const int jpos = __shfl_sync(0xffffffffu, tk.pos, j);
            const int jlo = max(__shfl_sync(0xffffffffu, lo, j), seen0), jhi = min(__shfl_sync(0xffffffffu, hi, j), seen1);
            const float jm = __shfl_sync(0xffffffffu, m, j), inv = __shfl_sync(0xffffffffu, inv_l, j);
            const long long jat = __shfl_sync(0xffffffffu, at, j);
            if (!unseen_values<D, 1>(a, run.b, run.g, seen0, jlo, jhi, seen1, d, misc)) continue;
            float o[1];
            redo_row<D, 1>(a, run.b, run.g, jhead, jtok, jpos, jlo, jhi, base, jm == -INFINITY ? 0.f : jm, d, o, misc);
            if (has) {
                if (direct) static_cast<__nv_bfloat16*>(a.out)[jat * D + d] = __float2bfloat16_rn(o[0] * inv);
                else pbase[jat * D + d] = o[0];
            }
        }
        ++nacc;
        if (other) ++nacc_o;
        // the run's Q slot, weights and shared words are free
        if (!meet()) return false;
        if (w == 0 && lane == 0) mbar_arrive(bars.nqempty + 8 * (nqn & 3u));
        ++nqn;
        return true;
    }
};

// ------------------------------------------------------------------------------------------
// tile kernel
// ------------------------------------------------------------------------------------------
template <int D, int MODE>
__global__ void __launch_bounds__(RW_THREADS, 1)
    rows_tile_kernel(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tqn,
                     const __grid_constant__ CUtensorMap tk, const __grid_constant__ CUtensorMap tv,
                     const __grid_constant__ CUtensorMap tpk, const __grid_constant__ CUtensorMap tpv,
                     const __grid_constant__ RowsArgs a)
{
    extern __shared__ __align__(1024) uint8_t sm[];
    constexpr uint32_t NCOLS = 512;              // 2 x 128 of scores, 2 x D of sums
    const RowsSmem<D> lay(a.stages);
    const uint32_t sbase = smem_u32(sm);
    const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    volatile int* misc = reinterpret_cast<volatile int*>(sm + lay.misc);
    uint32_t* tslot = reinterpret_cast<uint32_t*>(sm + lay.tslot);
    const RowsBars bars(sbase + lay.bars, a.stages);
    if (sbase & 1023u) {                         // 128-byte swizzle needs 1024-byte aligned tiles
        if (threadIdx.x == 0) rows_error(a, FDPP_ERRBIT_TIMEOUT);
        return;
    }
    if (threadIdx.x == 0) {
        for (int i = 0; i < a.stages; ++i) {
            mbar_init(bars.kvfull + 8 * i, 1);
            mbar_init(bars.kvempty + 8 * i, 2);      // both streams
        }
        for (int i = 0; i < RW_HDRS; ++i) {
            mbar_init(bars.hfull + 8 * i, 1);
            mbar_init(bars.hempty + 8 * i, 13);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(bars.qfull + 8 * i, 1);
            mbar_init(bars.qempty + 8 * i, 2);       // both streams
            for (int k = 0; k < 2; ++k) {
                mbar_init(bars.sfull + 16 * i + 8 * k, 1);
                mbar_init(bars.pready + 16 * i + 8 * k, 4);
                mbar_init(bars.pvdone + 16 * i + 8 * k, 1);
            }
            mbar_init(bars.ofull + 8 * i, 1);
            mbar_init(bars.ofree + 8 * i, 4);
            mbar_init(bars.mlfree + 8 * i, 4);
            mbar_init(bars.vote + 8 * i, 4);
        }
        for (int i = 0; i < RowsSmem<D>::NSLOTS; ++i) {
            mbar_init(bars.nqfull + 8 * i, 1);
            mbar_init(bars.nqempty + 8 * i, 1);
        }
        mbar_init(bars.drain, 4);
        for (int i = 0; i < 16; ++i) misc[i] = 0;
        fence_mbar_init();
    }
    if (warp == RW_MMA_WARP) tmem_alloc(smem_u32(tslot), NCOLS);
    if (warp == RW_LOAD_WARP && lane == 0) {
        prefetch_tensormap(&tq);
        prefetch_tensormap(&tqn);
        prefetch_tensormap(&tk);
        prefetch_tensormap(&tv);
        prefetch_tensormap(&tpk);
        prefetch_tensormap(&tpv);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = __shfl_sync(0xffffffffu, *tslot, 0);
    grid_dependency_wait();
    grid_launch_dependents();
    if (warp >= RW_MMA_WARP) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(RW_HELP_REGS));
        if (warp >= RW_LOAD_WARP) {
            RowsLoader<D> ld{a, lay, bars, sm, sbase, misc};
            if (warp == RW_LOAD_WARP) {
                if (!ld.run_k(&tq, &tqn, &tk, &tpk)) ld.settle(0);
            } else if (warp == RW_LOAD_WARP + 1) {
                if (!ld.run_v(&tv, &tpv)) ld.settle(1);
            }
            if (ld.bad) rows_error(a, ld.bad);
        } else {
            const uint32_t stream = (uint32_t)warp & 1u;
            if (warp < RW_MMA_WARP + 2) {
                RowsQk<D> qk{a, lay, bars, sbase, tmem, misc, stream};
                qk.run(sm);
            } else {
                RowsPv<D> pv{a, lay, bars, sbase, tmem, misc, stream};
                pv.run(sm);
            }
            // every MMA issued has landed before the tensor memory and the stages go
            umma_commit(elect_one(), bars.drain);
            __syncwarp();
            if (!mbar_wait(bars.drain, 0u) && lane == 0) rows_error(a, FDPP_ERRBIT_TIMEOUT);
            __syncwarp();
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(RW_SOFT_REGS));
        Softmax<D, MODE> sx{a, lay, bars, sm, tmem, misc, warp >> 2};
        sx.run();
        tc_fence_before();
    }
    __syncthreads();
    if (warp == RW_MMA_WARP) {
        tc_fence_after();
        tmem_dealloc(tmem, NCOLS);
    }
}

// ------------------------------------------------------------------------------------------
// joins
// ------------------------------------------------------------------------------------------
// Sums of one row in the frame of their largest max: a lane's D / 32 neighbouring columns.
template <int E>
struct RowSum {
    float m = -INFINITY, l = 0.f;
    float o[E];
    __device__ __forceinline__ RowSum()
    {
#pragma unroll
        for (int i = 0; i < E; ++i) o[i] = 0.f;
    }
    __device__ __forceinline__ static void fetch(const float* po, float (&v)[E])
    {
        if constexpr (E == 4) {
            const float4 t = __ldcg(reinterpret_cast<const float4*>(po) + (threadIdx.x & 31));
            v[0] = t.x; v[1] = t.y; v[2] = t.z; v[3] = t.w;
        } else {
            const float2 t = __ldcg(reinterpret_cast<const float2*>(po) + (threadIdx.x & 31));
            v[0] = t.x; v[1] = t.y;
        }
    }
    __device__ __forceinline__ void add(float2 ml, const float (&v)[E])
    {
        if (ml.x == -INFINITY && ml.y == 0.f) return;        // no key seen: its columns were not written
        const float f = fmaxf(m, ml.x), wa = m == f ? 1.f : ex2(m - f), wb = ml.x == f ? 1.f : ex2(ml.x - f);
        l = l * wa + ml.y * wb;
#pragma unroll
        for (int i = 0; i < E; ++i) o[i] = o[i] * wa + v[i] * wb;
        m = f;
    }
    __device__ __forceinline__ void store(__nv_bfloat16* out, bool empty) const
    {
        uint32_t w[E / 2];
#pragma unroll
        for (int i = 0; i < E / 2; ++i) w[i] = empty ? 0u : pack_bf16x2(o[2 * i] / l, o[2 * i + 1] / l);
        uint32_t* p = reinterpret_cast<uint32_t*>(out) + (threadIdx.x & 31) * (E / 2);
#pragma unroll
        for (int i = 0; i < E / 2; ++i) p[i] = w[i];
    }
};

// The partials of a unit cut in two or more, tiles [start, start + nt): the part of its first tile left
// its own in slot 2 c + 1, every later one in slot 2 c. Four are read at a time; the first `done` are left out.
template <int E>
__device__ __forceinline__ void add_cut(const RowsArgs& a, const int* begins, RowSum<E>& x, int start, int nt, int first,
                                        long long row, int done = 0)
{
    for (int c0 = first + done; c0 < a.parts && begins[c0] < start + nt; c0 += 4) {
        float2 ml[4];
        float v[4][E];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int c = min(c0 + k, a.parts - 1);
            const long long at = (long long)(2 * c + (c == first ? 1 : 0)) * a.slot_rows + row;
            ml[k] = make_float2(-INFINITY, 0.f);
            if (c0 + k < a.parts && begins[c] < start + nt && (c == first || begins[c] < begins[c + 1])) {
                ml[k] = __ldcg(a.slot_ml + at);
                RowSum<E>::fetch(a.slot_o + at * (E * 32), v[k]);
            }
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) x.add(ml[k], v[k]);
    }
}

constexpr int JOIN_WARPS = 8;

// The parts' first tiles, into shared memory.
__device__ __forceinline__ void load_begins(const RowsArgs& a, int total, int* begins)
{
    for (int c = threadIdx.x; c <= a.parts; c += blockDim.x) begins[c] = part_begin(c, total, a.parts);
    __syncthreads();
}

// Without a prefix: the units that a part boundary cuts, found from the boundaries (one grid column
// each; the first boundary inside a unit does it). A warp per row, and at most JOIN_ROWS CTAs for a unit so
// that all are resident at once. Ragged prompts of 333 to 1500 tokens, 16 heads, 2 kv heads, d = 64, in all:
// with 4 CTAs for a unit 58.5 us, with 8 52.8, with 16 53.7, with 32 (a CTA for every eight rows) 55.3.
constexpr int JOIN_ROWS = 8;
template <int D>
__global__ void __launch_bounds__(JOIN_WARPS * 32) rows_join_cut_kernel(RowsArgs a)
{
    __shared__ int begins[ROWS_MAX_PARTS + 1];
    grid_dependency_wait();
    grid_launch_dependents();
    const int c = blockIdx.x + 1, total = a.plan[RP_TILES];
    const RowTileRec r = a.rec[a.plan[RP_WORDS + c]];      // the row tile that part c begins in
    const int x = part_begin(c, total, a.parts), before = part_begin(c - 1, total, a.parts);
    if (x <= 0 || x >= total) return;
    const int span = unit_span(a, r), g = (x - r.start) / span, start = r.start + g * span;
    if (x == start || x >= start + r.nt || before > start) return;
    if (blockIdx.y * JOIN_WARPS >= r.ntok * a.G) return;
    load_begins(a, total, begins);
    for (int row = blockIdx.y * JOIN_WARPS + (threadIdx.x >> 5); row < r.ntok * a.G; row += gridDim.y * JOIN_WARPS) {
        const int i = row / a.G, tok = r.tok0 + i;
        const RowToken tk = a.tok[tok];
        RowSum<D / 32> s;
        add_cut(a, begins, s, start, r.nt, c - 1, row);
        s.store(static_cast<__nv_bfloat16*>(a.out) + ((long long)tok * a.Hq + g * a.G + (row - i * a.G)) * D, tk.hi <= tk.lo);
    }
}

// With a prefix: every row from its two units. A warp per row. Latency is all there is to it, so what can be
// read at once is: the token with both row tiles' records, then the first two partials of both units.
template <int D>
__global__ void __launch_bounds__(JOIN_WARPS * 32) rows_join_prefix_kernel(RowsArgs a)
{
    constexpr int E = D / 32;
    __shared__ int begins[ROWS_MAX_PARTS + 1];
    const long long w = (long long)blockIdx.x * JOIN_WARPS + (threadIdx.x >> 5);
    const int tok = min((int)(w / a.Hq), a.T - 1), head = (int)(w % a.Hq), g = head / a.G;
    grid_dependency_wait();
    grid_launch_dependents();
    const int total = a.plan[RP_TILES], npre = a.plan[RP_NPRE];
    const RowToken tk = a.tok[tok];
    RowTileRec rec[2];
    rec[0] = a.rec[min(tok / (2 * a.tpt), a.max_rt - 1)];
    rec[1] = a.rec[max(tk.rt, 0)];
    load_begins(a, total, begins);
    if (w >= (long long)a.T * a.Hq || tk.rt < 0) return;
    // per source: the partials are first, first + 1, .. (cut), or one (whole), or none
    int start[2], first[2], pieces[2];
    float2 ml[2][2];
    float v[2][2][E];
#pragma unroll
    for (int src = 0; src < 2; ++src) {
        const RowTileRec& r = rec[src];
        pieces[src] = 0;
        ml[src][0] = ml[src][1] = make_float2(-INFINITY, 0.f);
        // (the row is not one of the tile's where sequences overlap)
        if ((src == 0 && npre == 0) || r.nt == 0 || tok < r.tok0 || tok >= r.tok0 + r.ntok) continue;
        start[src] = r.start + g * unit_span(a, r);
        // the part of the unit's first tile: the last c with c total / parts < start + 1
        first[src] = (int)(((start[src] + 1ll) * a.parts - 1) / total);
        pieces[src] = begins[first[src] + 1] >= start[src] + r.nt ? 1 : 2;
        if (pieces[src] == 1) {
            const long long at = ((long long)src * a.T + tok) * a.Hq + head;
            ml[src][0] = __ldcg(a.row_ml + at);
            RowSum<E>::fetch(a.row_o + at * D, v[src][0]);
        } else {
            const long long row = (long long)(tok - r.tok0) * a.G + (head - g * a.G);
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const int c = first[src] + k;
                if (k == 1 && begins[c] >= begins[c + 1]) continue;
                const long long at = (long long)(2 * c + (k == 0)) * a.slot_rows + row;
                ml[src][k] = __ldcg(a.slot_ml + at);
                RowSum<E>::fetch(a.slot_o + at * D, v[src][k]);
            }
        }
    }
    RowSum<E> s;
#pragma unroll
    for (int src = 0; src < 2; ++src) {
        s.add(ml[src][0], v[src][0]);
        s.add(ml[src][1], v[src][1]);
        if (pieces[src] == 2)
            add_cut(a, begins, s, start[src], rec[src].nt, first[src], (long long)(tok - rec[src].tok0) * a.G + (head - g * a.G), 2);
    }
    s.store(static_cast<__nv_bfloat16*>(a.out) + ((long long)tok * a.Hq + head) * D, tk.hi <= tk.lo);
}

struct PdlConfig {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    PdlConfig(dim3 grid, int threads, size_t smem, cudaStream_t s, int cluster = 1)
    {
        cfg.gridDim = grid;
        cfg.blockDim = dim3((unsigned)threads);
        cfg.dynamicSmemBytes = smem;
        cfg.stream = s;
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        attr[1].id = cudaLaunchAttributeClusterDimension;
        attr[1].val.clusterDim.x = (unsigned)cluster;
        attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = cluster > 1 ? 2 : 1;
    }
};

template <int D, int MODE>
cudaError_t launch_d(const RowsArgs& a, const RowsMaps& m, cudaStream_t s)
{
    const bool small = a.B <= PLAN_SMALL && a.max_rt <= PLAN_SMALL;
    const int rounds = (a.T + PLAN_SMALL - 1) / PLAN_SMALL, ranks = !small || rounds == 1 ? 1 : (rounds < PLAN_CLUSTER ? rounds : PLAN_CLUSTER);
    PdlConfig plan(dim3((unsigned)ranks), small ? PLAN_SMALL : PLAN_THREADS, 0, s, ranks);
    cudaError_t e = cudaLaunchKernelEx(&plan.cfg, small ? rows_plan_small_kernel : rows_plan_kernel, a);
    if (e != cudaSuccess) return e;
    auto kern = rows_tile_kernel<D, MODE>;
    const int smem = RowsSmem<D>(a.stages).total;
    if ((e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem)) != cudaSuccess) return e;
    PdlConfig tile(dim3((unsigned)a.parts), RW_THREADS, (size_t)smem, s);
    if ((e = cudaLaunchKernelEx(&tile.cfg, kern, m.q, m.qn, m.k, m.v, m.pk, m.pv, a)) != cudaSuccess) return e;
    if (a.prefix_len) {
        const long long rows = (long long)a.T * a.Hq;
        PdlConfig join(dim3((unsigned)((rows + JOIN_WARPS - 1) / JOIN_WARPS)), JOIN_WARPS * 32, 0, s);
        e = cudaLaunchKernelEx(&join.cfg, rows_join_prefix_kernel<D>, a);
    } else if (a.parts > 1) {
        PdlConfig join(dim3((unsigned)(a.parts - 1), (unsigned)min(JOIN_ROWS, (a.slot_rows + JOIN_WARPS - 1) / JOIN_WARPS)), JOIN_WARPS * 32, 0, s);
        e = cudaLaunchKernelEx(&join.cfg, rows_join_cut_kernel<D>, a);
    }
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

int rows_tc_stages(int head_dim, int smem_per_block)
{
    int n = 0;
    while (n < 16 && (head_dim == 128 ? RowsSmem<128>(n + 2).total : RowsSmem<64>(n + 2).total) <= smem_per_block) n += 2;
    return n;                                            // even: K and V tiles take turns
}

cudaError_t launch_rows_tc(const RowsArgs& a, const RowsMaps& m, cudaStream_t s)
{
    const int mode = a.cap > 0.f ? MODE_CAP : (a.slopes ? MODE_BIAS : MODE_PLAIN);
    if (a.D == 128)
        return mode == MODE_CAP    ? launch_d<128, MODE_CAP>(a, m, s)
               : mode == MODE_BIAS ? launch_d<128, MODE_BIAS>(a, m, s)
                                   : launch_d<128, MODE_PLAIN>(a, m, s);
    return mode == MODE_CAP    ? launch_d<64, MODE_CAP>(a, m, s)
           : mode == MODE_BIAS ? launch_d<64, MODE_BIAS>(a, m, s)
                               : launch_d<64, MODE_PLAIN>(a, m, s);
}

}  // namespace fdpp
