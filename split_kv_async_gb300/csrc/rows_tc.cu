// rows_tc.cu -- rows attention (fdpp_rows.h) on the tcgen05 tensor cores: bf16, d = 64 or 128.
//
// What it computes. For the rows of a kv head (its G query heads of some tokens) and a range of keys
//     v_t = log2(e) score_t, M = max v_t, l = sum 2^(v_t - M), o = sum 2^(v_t - M) v_t
// by one pass over the keys with a running max; the frame is moved only when a row's max has grown by
// more than 2^8 since it was set (until then the weights stay below 2^8, and the sums are exact in
// the same frame), so that the accumulator is hardly ever rescaled.
//
// How. One CTA per SM, ten warps, two streams:
//   warp 9   loads: walks this CTA's part of the key tiles (128 keys each), writes a header for each run
//            (the part's share of one unit = (row tile, kv head)), brings Q by one 3-D TMA load per 64
//            of d and the K and V tiles into a ring of stages (128-byte swizzle).
//   warp 8   issues the MMAs of both streams (one thread): S = Q K^T (M = 128 rows, N = 128 keys), and
//            O += P V with P from tensor memory and V MN-major from the TMA-landed tile. A stream's P V
//            of one tile is issued right before its next Q K^T, so while one stream's softmax runs the
//            tensor cores work on the other's tile.
//   warps 0-3, 4-7   the softmax of streams 0 and 1: a thread owns a row (tensor-memory lane), reads its
//            128 scores, and writes P as bf16 over them. P's rounding (2^-9 of each weight, independent)
//            leaves an error of the order of the output's own rounding; l sums the unrounded weights.
// With more than 128 rows a unit is a pair: two row tiles, one per stream, share every K/V tile. With
// fewer, both streams take the same rows, alternate key tiles and are joined at the run's end.
//
// What bounds it. Many rows: the tensor pipe (4 x 128 keys x 128 rows x d FLOP per row tile and key tile)
// with the softmax's 128 x 128 exponentials on the MUFU units beside it. Few rows: HBM (K and V of a kv
// head are read once, at 512 bytes per key for d = 128).
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
// MMAs land, frees its tensor memory and exits.
#include <cuda_bf16.h>

#include "rows_common.cuh"
#include "tcgen05.cuh"

namespace fdpp {
namespace {

constexpr int RW_MMA_WARP = 8;
constexpr int RW_LOAD_WARP = 9;
constexpr int RW_THREADS = 10 * 32;
constexpr int RW_HDRS = 4;               // run headers in flight
constexpr int RW_HDR_BYTES = 64;
constexpr float RW_LAG = 8.f;            // log2 of the growth of a row's max that moves its frame

enum { RH_KIND = 0, RH_G, RH_B, RH_TOK0, RH_NTOK, RH_LEN, RH_A0, RH_A1, RH_B0, RH_B1, RH_T0, RH_T1, RH_DEST,
       RH_FLAGS, RH_BASE, RH_WORDS };
enum { RUN_ROWS = 0, RUN_END = 1 };
enum { RF_PAIR = 1, RF_START = 2 };      // two row tiles; the first key tile goes to stream 1
enum { DEST_OUT = -1, DEST_ROWS = -2 };  // else a slot
static_assert(RH_WORDS * 4 <= RW_HDR_BYTES, "header fits its slot");

template <int D>
struct RowsSmem {
    static constexpr int QB = ROWS_TILE * D * 2;           // a row tile's Q
    static constexpr int SB = ROWS_KEYS * D * 2;           // a K or V tile
    static constexpr int HALF = ROWS_KEYS * 128;           // one 64-wide half of either
    int q, stages, hdr, ml, bars, misc, tslot, total;
    __host__ __device__ explicit RowsSmem(int nst)
        : q(0), stages(2 * QB), hdr(stages + nst * SB), ml(hdr + RW_HDRS * RW_HDR_BYTES), bars(ml + 2 * ROWS_TILE * 8),
          misc(bars + (2 * nst + 2 * 2 + 2 * RW_HDRS + 6 * 2 + 1) * 8), tslot(misc + 16), total(tslot + 16)
    {
    }
};

struct RowsBars {
    uint32_t kvfull, kvempty;     // [stages]
    uint32_t qfull, qempty;       // [2]
    uint32_t hfull, hempty;       // [RW_HDRS] run headers: read by the MMA warp and the eight softmax warps
    uint32_t sfull, pready;       // [2] scores written; weights written over them
    uint32_t ofull, ofree;        // [2] accumulator complete; read out
    uint32_t mlready, mlfree;     // [2] the second stream's maxima and sums for the joined epilogue
    uint32_t drain;
    __device__ __forceinline__ RowsBars(uint32_t base, int nst)
    {
        kvfull = base;
        kvempty = kvfull + 8 * nst;
        qfull = kvempty + 8 * nst;
        qempty = qfull + 16;
        hfull = qempty + 16;
        hempty = hfull + 8 * RW_HDRS;
        sfull = hempty + 8 * RW_HDRS;
        pready = sfull + 16;
        ofull = pready + 16;
        ofree = ofull + 16;
        mlready = ofree + 16;
        mlfree = mlready + 16;
        drain = mlfree + 16;
    }
};

// All lanes wait; a wait that runs out aborts the CTA (warp-uniform result).
__device__ __forceinline__ bool rwait(uint32_t bar, uint32_t parity, volatile int* misc, const RowsArgs& a)
{
    bool ok = (misc[0] == 0) && mbar_wait(bar, parity & 1u);
    ok = __all_sync(0xffffffffu, ok);
    if (!ok && (threadIdx.x & 31) == 0) {
        misc[0] = 1;
        rows_error(a, FDPP_ERRBIT_TIMEOUT);
    }
    return ok;
}

// First tile of part c of the `total` tiles.
__device__ __forceinline__ int part_begin(int c, int total, int parts) { return (int)((long long)c * total / parts); }

// The part that holds tile x.
__device__ __forceinline__ int part_of(int x, int total, int parts)
{
    return (int)((((long long)x + 1) * parts - 1) / total);
}

// The row tile whose units hold tile x (x < total): the last that starts at or before it.
__device__ __forceinline__ int find_rt(const RowTileRec* rec, int n, int x)
{
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (rec[mid].start <= x) lo = mid; else hi = mid;
    }
    return lo;
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

__global__ void __launch_bounds__(PLAN_THREADS) rows_plan_kernel(RowsArgs a)
{
    __shared__ long long red[32];
    __shared__ int srt[PLAN_SMEM_SEQS + 1];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
    grid_dependency_wait();
    grid_launch_dependents();
    unsigned bad = 0;
    const int P = prefix_keys(a, bad);
    const int pair = 2 * a.tpt;
    int last = a.T;
    if (a.cu) last = clamp_len(a.cu[a.B], a.T);
    // prefix row tiles first, over all rows up to the last sequence's end
    const int npre = P > 0 ? ceil_div_i(last, pair) : 0;
    for (int t = threadIdx.x; t < a.T; t += blockDim.x) a.tok[t] = RowToken{0, 0, 0, -1};
    const bool in_smem = a.B <= PLAN_SMEM_SEQS;
    int* first_rt = in_smem ? srt : a.seq_rt;
    long long run = npre;
    for (int base = 0; base < a.B; base += blockDim.x) {
        const int b = base + threadIdx.x;
        int c0 = 0, n = 0;
        if (b < a.B) n = seq_rows(a, b, c0, bad);
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

    // own row tiles: the tokens' positions and key ranges, and the tiles' key tiles
    for (int rt = npre + warp; rt < nrt; rt += nw) {
        int lo = 0, hi = a.B;                           // first_rt[lo] <= rt < first_rt[hi]
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (first_rt[mid] <= rt) lo = mid; else hi = mid;
        }
        const int b = lo;
        int c0;
        const int n = seq_rows(a, b, c0, bad), L = own_len(a, b, bad);
        const int i0 = (rt - first_rt[b]) * pair, nt = min(pair, n - i0);
        int loA = INT32_MAX, hiA = 0, loB = INT32_MAX, hiB = 0;
        for (int i = lane; i < nt; i += 32) {
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
        RowTileRec r{};
        r.b = b;
        r.tok0 = c0 + i0;
        r.ntok = nt;
        r.len = L;
        set_tiles(r, warp_min(loA), warp_max(hiA), warp_min(loB), warp_max(hiB));
        if (lane == 0) a.rec[rt] = r;
        if (r.nt == 0 && !a.prefix_len) {               // rows that see nothing, and no unit writes
            uint32_t* o = reinterpret_cast<uint32_t*>(static_cast<__nv_bfloat16*>(a.out) + (long long)r.tok0 * a.Hq * a.D);
            const long long words = (long long)nt * a.Hq * a.D / 2;
            for (long long i = lane; i < words; i += 32) o[i] = 0u;
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
    __syncthreads();
    long long tiles = 0;
    for (int base = 0; base < nrt; base += blockDim.x) {
        const int rt = base + threadIdx.x;
        const long long mine = rt < nrt ? (long long)a.rec[rt].nt * a.Hkv : 0;
        long long total;
        const long long incl = plan_scan(mine, total, red);
        if (rt < nrt) a.rec[rt].start = (int)(tiles + incl - mine);
        tiles += total;
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
    uint32_t stage = 0, phase = 0, nq = 0, nh = 0;
    unsigned bad = 0;

    // Block of key tile t that this lane answers for (-1: none): entry t's first block + lane.
    __device__ __forceinline__ int entry(const RowTileRec& r, int t)
    {
        const int lane = threadIdx.x & 31;
        const int bs = a.block_size, first = t * ROWS_KEYS / bs, nv = min(ROWS_KEYS, r.len - t * ROWS_KEYS);
        const int nb = bs >= ROWS_KEYS ? 1 : ceil_div_i(nv, bs);
        if (nv <= 0 || lane >= nb) return -1;
        return r.b < 0 ? a.prefix_blocks[first + lane] : a.block_table[(long long)r.b * a.max_blocks + first + lane];
    }

    // One K or V tile into the next stage.
    __device__ __forceinline__ bool tile(const CUtensorMap* map, const RowTileRec& r, int g, int t, int ent)
    {
        constexpr int HALVES = D / 64;
        const int lane = threadIdx.x & 31;
        if (!rwait(bars.kvempty + 8 * stage, phase ^ 1u, misc, a)) return false;
        const uint32_t dst = sbase + lay.stages + stage * RowsSmem<D>::SB, bar = bars.kvfull + 8 * stage;
        if (!a.block_table) {
            if (lane == 0) mbar_arrive_expect_tx(bar, RowsSmem<D>::SB);
            __syncwarp();
            if (lane < HALVES)
                tma_load(dst + lane * RowsSmem<D>::HALF, map, g * D + lane * 64, t * ROWS_KEYS, r.b < 0 ? 0 : r.b, bar);
        } else {
            const int bs = a.block_size, box = min(bs, ROWS_KEYS), nv = min(ROWS_KEYS, r.len - t * ROWS_KEYS);
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
        if (++stage == (uint32_t)a.stages) { stage = 0; phase ^= 1u; }
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

    __device__ __forceinline__ bool run(const CUtensorMap* tq, const CUtensorMap* tk, const CUtensorMap* tv,
                                        const CUtensorMap* tpk, const CUtensorMap* tpv)
    {
        const int lane = threadIdx.x & 31;
        const int total = a.plan[RP_TILES], nrt = a.plan[RP_NRT], P = a.plan[RP_PREFIX];
        const int c = blockIdx.x, parts = gridDim.x;
        int pos = part_begin(c, total, parts);
        const int end = part_begin(c + 1, total, parts);
        int rt = pos < end ? find_rt(a.rec, nrt, pos) : 0;
        uint32_t toggle = 0;
        while (pos < end) {
            const RowTileRec r = a.rec[rt];
            const int past = r.start + r.nt * a.Hkv;
            while (pos < end && pos < past) {
                const int g = (pos - r.start) / r.nt, ta = (pos - r.start) - g * r.nt, tb = min(r.nt, ta + end - pos);
                const int t0 = r.k0 + ta, t1 = r.k0 + tb;
                const bool pair = r.ntok > a.tpt, whole = ta == 0 && tb == r.nt;
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
                    h[RH_FLAGS] = pair ? RF_PAIR : (toggle ? RF_START : 0);
                    h[RH_BASE] = r.b < 0 ? 0 : P;
                }
                publish();
                if (!pair) toggle = (toggle + (uint32_t)(t1 - t0)) & 1u;
                int ent = a.block_table ? entry(r, t0) : 0;
                if (!query(tq, g, r.tok0)) return false;
                if (pair && !query(tq, g, r.tok0 + a.tpt)) return false;
                for (int t = t0; t < t1; ++t) {
                    const int next = a.block_table && t + 1 < t1 ? entry(r, t + 1) : 0;
                    if (!tile(r.b < 0 ? tpk : tk, r, g, t, ent)) return false;
                    if (!tile(r.b < 0 ? tpv : tv, r, g, t, ent)) return false;
                    ent = next;
                }
                pos += tb - ta;
            }
            ++rt;
        }
        int* h = header();
        if (!h) return false;
        if (lane == 0) h[RH_KIND] = RUN_END;
        publish();
        return true;
    }

    // After an abort: every copy issued lands before the CTA exits (bounded waits).
    __device__ __forceinline__ void settle()
    {
        if ((threadIdx.x & 31) == 0) {
            for (int s = 0; s < a.stages; ++s) {
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
        }
        __syncwarp();
    }
};

// ------------------------------------------------------------------------------------------
// MMA warp
// ------------------------------------------------------------------------------------------
// Tensor memory: the scores of streams 0 and 1 (128 columns each; P takes the first 64 of them), then
// their accumulators (D columns each).
constexpr uint32_t TM_S = ROWS_KEYS;

template <int D>
struct RowsMma {
    const RowsArgs& a;
    const RowsSmem<D>& lay;
    const RowsBars& bars;
    uint8_t* sm;
    uint32_t sbase, tmem;
    volatile int* misc;
    // a stream's tile whose P V is still to be issued
    struct Pending {
        bool on;
        uint32_t tile, stage, phase;
        bool first, last, release;
    } pend[2];
    uint32_t np[2], nacc[2];       // P V issued, runs begun, per stream

    // Issues the P V that stream s owes, after one that the other stream owes from before it (of the
    // same tile: stream 0's first): the joined epilogue waits for both accumulators, and a tile's last
    // P V gives its stage back.
    __device__ __forceinline__ bool flush(int s)
    {
        const Pending& o = pend[s ^ 1];
        if (!pend[s].on) return true;
        if (o.on && (o.tile < pend[s].tile || (o.tile == pend[s].tile && s == 1)) && !issue(s ^ 1)) return false;
        return issue(s);
    }

    __device__ __forceinline__ bool issue(int s)
    {
        constexpr uint32_t IDESC = umma_idesc_bf16(128, D, false) | (1u << 16);     // V: MN-major
        Pending& p = pend[s];
        if (!rwait(bars.pready + 8 * s, np[s] & 1u, misc, a)) return false;
        if (!rwait(bars.kvfull + 8 * p.stage, p.phase, misc, a)) return false;
        if (p.first && !rwait(bars.ofree + 8 * s, (nacc[s] & 1u) ^ 1u, misc, a)) return false;
        tc_fence_after();
        if ((threadIdx.x & 31) == 0) {
            const uint64_t vd =
                sw128_mnmajor_desc(sbase + lay.stages + p.stage * RowsSmem<D>::SB, RowsSmem<D>::HALF, 1024);
            const uint32_t pd = tmem + s * TM_S, od = tmem + 2 * TM_S + s * D;
#pragma unroll
            for (int k = 0; k < ROWS_KEYS / 16; ++k)
                umma_bf16_ta(od, pd + 8 * k, vd + k * (2048 >> 4), IDESC, (p.first && k == 0) ? 0u : 1u);
            if (p.release) umma_commit(bars.kvempty + 8 * p.stage);
            if (p.last) umma_commit(bars.ofull + 8 * s);
        }
        __syncwarp();
        ++np[s];
        if (p.first) ++nacc[s];
        p.on = false;
        return true;
    }

    __device__ __forceinline__ bool run()
    {
        constexpr uint32_t IDESC = umma_idesc_bf16(128, ROWS_KEYS, false);
        const int lane = threadIdx.x & 31;
        uint32_t stage = 0, phase = 0, nq = 0, nh = 0, tile = 0;
        pend[0].on = pend[1].on = false;
        np[0] = np[1] = nacc[0] = nacc[1] = 0;
        for (;; ++nh) {
            const uint32_t hs = nh % RW_HDRS;
            if (!rwait(bars.hfull + 8 * hs, (nh / RW_HDRS) & 1u, misc, a)) return false;
            const int* h = reinterpret_cast<const int*>(sm + lay.hdr + hs * RW_HDR_BYTES);
            const int kind = h[RH_KIND], len = h[RH_LEN], t0 = h[RH_T0], t1 = h[RH_T1], flags = h[RH_FLAGS];
            const int a0 = h[RH_A0], a1 = h[RH_A1], b0 = h[RH_B0], b1 = h[RH_B1];
            __syncwarp();
            if (lane == 0) mbar_arrive(bars.hempty + 8 * hs);
            if (kind == RUN_END) break;
            const bool pair = flags & RF_PAIR;
            const uint32_t qb0 = nq & 1u;
            for (uint32_t k = 0; k < (pair ? 2u : 1u); ++k, ++nq)
                if (!rwait(bars.qfull + 8 * (nq & 1u), (nq >> 1) & 1u, misc, a)) return false;
            bool begun[2] = {false, false};
            for (int t = t0; t < t1; ++t, ++tile) {
                // a P V left behind by a stream that is not in turn holds a stage: issue it first
                for (int s = 0; s < 2; ++s)
                    if (pend[s].on && pend[s].tile + 1 < tile && !flush(s)) return false;
                uint32_t vstage = stage + 1, vphase = phase;
                if (vstage == (uint32_t)a.stages) { vstage = 0; vphase ^= 1u; }
                bool act[2], lst[2];
                if (pair) {
                    act[0] = t >= a0 && t < a1;
                    act[1] = t >= b0 && t < b1;
                    lst[0] = t + 1 == a1;
                    lst[1] = t + 1 == b1;
                } else {
                    const int s = ((t - t0) + ((flags & RF_START) ? 1 : 0)) & 1;
                    act[s] = true;
                    act[s ^ 1] = false;
                    lst[0] = lst[1] = t + 2 >= t1;
                }
                if (!rwait(bars.kvfull + 8 * stage, phase, misc, a)) return false;
                const int nv = len - t * ROWS_KEYS;
                if (nv < ROWS_KEYS || !(act[0] || act[1])) {
                    if (!rwait(bars.kvfull + 8 * vstage, vphase, misc, a)) return false;
                }
                if (nv < ROWS_KEYS) {              // V past the source's end: zeros
                    uint8_t* v = sm + lay.stages + vstage * RowsSmem<D>::SB;
                    const int chunks = (ROWS_KEYS - nv) * 8;
                    for (int i = lane; i < chunks * (D / 64); i += 32) {
                        const int half = i / chunks, x = i - half * chunks;
                        *reinterpret_cast<uint4*>(v + half * RowsSmem<D>::HALF + nv * 128 + x * 16) = make_uint4(0, 0, 0, 0);
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                }
                for (int s = 0; s < 2; ++s) {
                    if (!act[s]) continue;
                    if (!flush(s)) return false;
                    const uint32_t qb = pair ? (qb0 + (uint32_t)s) & 1u : qb0;
                    const bool release = s == 1 || !act[1];
                    tc_fence_after();
                    if (lane == 0) {
                        const uint64_t qd = sw128_kmajor_desc(sbase + lay.q + qb * RowsSmem<D>::QB);
                        const uint64_t kd = sw128_kmajor_desc(sbase + lay.stages + stage * RowsSmem<D>::SB);
#pragma unroll
                        for (int k = 0; k < D / 16; ++k) {
                            const uint32_t off = (uint32_t)(k >> 2) * (RowsSmem<D>::HALF >> 4) + (uint32_t)(k & 3) * 2u;
                            umma_bf16(tmem + s * TM_S, qd + off, kd + off, IDESC, k > 0 ? 1u : 0u);
                        }
                        umma_commit(bars.sfull + 8 * s);
                        if (release) umma_commit(bars.kvempty + 8 * stage);
                        // a row tile's Q is free after its last tile of the run
                        if (pair ? lst[s] : t + 1 == t1) umma_commit(bars.qempty + 8 * qb);
                    }
                    __syncwarp();
                    pend[s] = Pending{true, tile, vstage, vphase, !begun[s], lst[s], release};
                    begun[s] = true;
                }
                if (!(act[0] || act[1]) && lane == 0) {     // a tile that neither half sees
                    mbar_arrive(bars.kvempty + 8 * stage);
                    mbar_arrive(bars.kvempty + 8 * vstage);
                }
                __syncwarp();
                for (int k = 0; k < 2; ++k)
                    if (++stage == (uint32_t)a.stages) { stage = 0; phase ^= 1u; }
            }
            // a half without tiles in this run gives its Q back here
            if (pair && lane == 0) {
                if (a1 <= a0) mbar_arrive(bars.qempty + 8 * qb0);
                if (b1 <= b0) mbar_arrive(bars.qempty + 8 * (qb0 ^ 1u));
            }
            __syncwarp();
        }
        return flush(0) && flush(1);
    }
};

// ------------------------------------------------------------------------------------------
// softmax warps
// ------------------------------------------------------------------------------------------
// The keys [k0, k1) of a row again, for columns of its sums that are not finite: sums over the keys it
// sees alone, in the frame M. By one warp; o: this lane's D / 32 columns (lane + 32 i).
template <int D>
__device__ __noinline__ void redo_row(const RowsArgs& a, int b, int g, int h, int row, int pos, int k0, int k1, int base,
                                      float M, float cap_rate, float (&o)[D / 32], unsigned& bad)
{
    const int lane = threadIdx.x & 31;
    const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(a.q) + ((long long)row * a.Hq + h) * D;
    const __nv_bfloat16* kc = static_cast<const __nv_bfloat16*>(b < 0 && a.pk ? a.pk : a.k);
    const __nv_bfloat16* vc = static_cast<const __nv_bfloat16*>(b < 0 && a.pv ? a.pv : a.v);
    const float slope = a.slopes ? a.slopes[h] * LOG2E : 0.f;
    float qr[D / 32];
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
        qr[i] = __bfloat162float(q[lane + 32 * i]);
        o[i] = 0.f;
    }
    for (int t = k0; t < k1; ++t) {
        const long long off = key_offset(a, b, t, g);
        if (off < 0) { bad |= FDPP_ERRBIT_BLOCK_TABLE; continue; }
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < D / 32; ++i) s = fmaf(qr[i], __bfloat162float(kc[off + lane + 32 * i]), s);
        s = warp_sum(s);
        const float p = ex2(mod_score(s, a.scale, a.cap, cap_rate, slope, (float)(base + t - pos)) - M);
        bool done = true;
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {
            o[i] = fmaf(p, __bfloat162float(vc[off + lane + 32 * i]), o[i]);
            done = done && o[i] != o[i];
        }
        if (__all_sync(0xffffffffu, done)) break;       // NaN stays NaN
    }
}

__device__ __forceinline__ float max3(float a, float b, float c)
{
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

template <int D, bool MOD>
__device__ __forceinline__ bool softmax_stream(const RowsArgs& a, const RowsSmem<D>& lay, const RowsBars& bars,
                                               uint8_t* sm, uint32_t tmem, int s, volatile int* misc)
{
    const int lane = threadIdx.x & 31, r = threadIdx.x & (ROWS_TILE - 1);
    const uint32_t lane_base = (uint32_t)(r & ~31) << 16;
    const uint32_t ts = tmem + lane_base + s * TM_S, to = tmem + lane_base + 2 * TM_S;
    float2* ml = reinterpret_cast<float2*>(sm + lay.ml);
    const float rate = MOD ? 1.f : a.scale * LOG2E;      // log2 units per unit of v
    const float cap_rate = a.cap > 0.f ? 2.f * LOG2E / a.cap : 0.f;
    const int live_rows = a.tpt * a.G;
    uint32_t nh = 0, ntile = 0, nacc[2] = {0, 0}, nml[2] = {0, 0};
    unsigned bad = 0;
    for (;; ++nh) {
        const uint32_t hs = nh % RW_HDRS;
        if (!rwait(bars.hfull + 8 * hs, (nh / RW_HDRS) & 1u, misc, a)) return false;
        const int* h = reinterpret_cast<const int*>(sm + lay.hdr + hs * RW_HDR_BYTES);
        const int kind = h[RH_KIND], g = h[RH_G], b = h[RH_B], tok0 = h[RH_TOK0], ntok = h[RH_NTOK], len = h[RH_LEN];
        const int t0 = h[RH_T0], t1 = h[RH_T1], dest = h[RH_DEST], flags = h[RH_FLAGS], base = h[RH_BASE];
        const int s0 = s ? h[RH_B0] : h[RH_A0], s1 = s ? h[RH_B1] : h[RH_A1];
        const bool other_tiles = s ? h[RH_A1] > h[RH_A0] : h[RH_B1] > h[RH_B0];      // (pairs)
        __syncwarp();
        if (lane == 0) mbar_arrive(bars.hempty + 8 * hs);
        if (kind == RUN_END) break;
        const bool pair = flags & RF_PAIR;
        // this stream's tiles: first, first + step, .. below past
        const int start = (flags & RF_START) ? 1 : 0;
        const int first = pair ? s0 : t0 + (s ^ start), past = pair ? s1 : t1, step = pair ? 1 : 2;
        const int ti = r / a.G, hh = r - ti * a.G;
        const int tok = tok0 + (pair ? s * a.tpt : 0) + ti;
        const bool live = r < live_rows && tok < tok0 + ntok;
        const bool warp_live = __any_sync(0xffffffffu, live);
        RowToken tk{0, 0, 0, -1};
        if (live) tk = a.tok[tok];
        const bool mine = live && tk.rt >= 0;
        // keys of this source that the row sees; a row that is not one masks nothing and is not written
        int lo = mine ? max(tk.lo - base, 0) : 0, hi = mine ? min(tk.hi - base, len) : INT32_MAX;
        if (mine && hi <= lo) lo = hi = 0;
        float slope = 0.f;
        if (MOD && a.slopes && live) slope = a.slopes[g * a.G + hh] * LOG2E;
        const float fpos = (float)(tk.pos - base);       // the position in this source's indexes
        float m = -INFINITY, l = 0.f;                    // frame (log2 units) and sum
        int count = 0;
        for (int t = first; t < past; t += step, ++ntile, ++count) {
            if (!rwait(bars.sfull + 8 * s, ntile & 1u, misc, a)) return false;
            tc_fence_after();
            if (warp_live) {
                uint32_t x[ROWS_KEYS];
#pragma unroll
                for (int i = 0; i < 4; ++i) tmem_ld32_async(ts + 32 * i, x + 32 * i);
                tmem_wait_ld();
#pragma unroll
                for (int i = 0; i < 4; ++i) reg_fence32(x + 32 * i);
                const int k0 = t * ROWS_KEYS;
                if (MOD) {
                    const float d0 = (float)k0 - fpos;
#pragma unroll
                    for (int i = 0; i < ROWS_KEYS; ++i)
                        x[i] = __float_as_uint(mod_score(__uint_as_float(x[i]), a.scale, a.cap, cap_rate, slope, d0 + (float)i));
                }
                if (!__all_sync(0xffffffffu, lo <= k0 && hi >= k0 + ROWS_KEYS)) {
                    const int c0 = lo - k0, c1 = hi - k0;
#pragma unroll
                    for (int i = 0; i < ROWS_KEYS; ++i)
                        if (i < c0 || i >= c1) x[i] = __float_as_uint(-INFINITY);
                }
                float mx[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) mx[i] = fmaxf(__uint_as_float(x[i]), __uint_as_float(x[i + 4]));
#pragma unroll
                for (int i = 8; i < ROWS_KEYS; i += 8)
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        mx[k] = max3(mx[k], __uint_as_float(x[i + k]), __uint_as_float(x[i + 4 + k]));
                const float top = max3(fmaxf(mx[0], mx[1]), mx[2], mx[3]) * rate;
                if (count == 0) {
                    m = top;
                } else if (__any_sync(0xffffffffu, top > m + RW_LAG)) {
                    // move the frame: the accumulator's P V of the tile before has completed (the
                    // scores' barrier counts every MMA issued before them)
                    const float f = fmaxf(m, top), w = m == f ? 1.f : ex2(m - f);
                    m = f;
                    l *= w;
#pragma unroll
                    for (int i = 0; i < D / 32; ++i) {
                        uint32_t o[32];
                        tmem_ld32_async(to + s * D + 32 * i, o);
                        tmem_wait_ld();
                        reg_fence32(o);
#pragma unroll
                        for (int k = 0; k < 32; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * w);
                        tmem_st32(to + s * D + 32 * i, o);
                    }
                }
                const float mu = m == -INFINITY ? 0.f : m;
                float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int i = 0; i < ROWS_KEYS; i += 4) {
                    float p[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        p[k] = ex2(fmaf(__uint_as_float(x[i + k]), rate, -mu));
                        sum[k] += p[k];
                    }
                    x[i / 2] = pack_bf16x2(p[0], p[1]);
                    x[i / 2 + 1] = pack_bf16x2(p[2], p[3]);
                }
                l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
                tmem_st32(ts, x);
                tmem_st32(ts + 32, x + 32);
                tmem_wait_st();
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bars.pready + 8 * s);
        }

        // ---- the run's end ----
        const int other = s ^ 1;
        const int n_other = pair ? 0 : max(0, (t1 - t0 + (other == start ? 1 : 0)) / 2);
        if (!pair && s != start) {                       // hand over to the other stream
            if (count > 0) {
                if (!rwait(bars.mlfree + 8 * s, (nml[s] & 1u) ^ 1u, misc, a)) return false;
                ml[s * ROWS_TILE + r] = make_float2(m, l);
                __syncwarp();
                if (lane == 0) mbar_arrive(bars.mlready + 8 * s);
                ++nml[s];
                ++nacc[s];
            }
            ++nacc[other];
            continue;
        }
        float mo = -INFINITY, wo = 0.f, ws = 1.f;        // the other stream's frame and weights
        if (count > 0 && !rwait(bars.ofull + 8 * s, nacc[s] & 1u, misc, a)) return false;
        if (n_other > 0) {
            if (!rwait(bars.mlready + 8 * other, nml[other] & 1u, misc, a)) return false;
            const float2 x = ml[other * ROWS_TILE + r];
            __syncwarp();
            if (lane == 0) mbar_arrive(bars.mlfree + 8 * other);
            if (!rwait(bars.ofull + 8 * other, nacc[other] & 1u, misc, a)) return false;
            mo = x.x;
            const float f = fmaxf(m, mo);
            ws = m == f ? 1.f : ex2(m - f);
            wo = mo == f ? 1.f : ex2(mo - f);
            l = l * ws + x.y * wo;
            m = f;
        }
        tc_fence_after();
        const int head = g * a.G + hh;
        const bool direct = dest == DEST_OUT;
        const bool empty = hi <= lo;
        __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.out) + ((long long)tok * a.Hq + head) * D;
        float* po = nullptr;
        if (!direct && mine) {
            long long at;
            float2* pml;
            if (dest == DEST_ROWS) {
                at = ((b < 0 ? 0ll : (long long)a.T) + tok) * a.Hq + head;
                po = a.row_o + at * D;
                pml = a.row_ml + at;
            } else {
                at = (long long)dest * a.slot_rows + (tok - tok0) * a.G + hh;
                po = a.slot_o + at * D;
                pml = a.slot_ml + at;
            }
            *pml = make_float2(count > 0 ? m : -INFINITY, l);
        }
        bool fine = true;
        if (warp_live && (count > 0 || direct)) {
            const float inv = direct ? 1.f / l : 1.f;
#pragma unroll
            for (int i = 0; i < D / 32; ++i) {
                uint32_t x[32];
                if (count > 0) {
                    tmem_ld32_async(to + s * D + 32 * i, x);
                    if (n_other > 0) {
                        uint32_t y[32];
                        tmem_ld32_async(to + other * D + 32 * i, y);
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
                if (!mine) continue;
                if (direct) {
#pragma unroll
                    for (int k = 0; k < 32; k += 8) {
                        uint4 v = make_uint4(0, 0, 0, 0);
                        if (!empty)
                            v = make_uint4(pack_bf16x2(__uint_as_float(x[k]) * inv, __uint_as_float(x[k + 1]) * inv),
                                           pack_bf16x2(__uint_as_float(x[k + 2]) * inv, __uint_as_float(x[k + 3]) * inv),
                                           pack_bf16x2(__uint_as_float(x[k + 4]) * inv, __uint_as_float(x[k + 5]) * inv),
                                           pack_bf16x2(__uint_as_float(x[k + 6]) * inv, __uint_as_float(x[k + 7]) * inv));
                        *reinterpret_cast<uint4*>(out + 32 * i + k) = v;
                    }
                } else {
#pragma unroll
                    for (int k = 0; k < 32; k += 4)
                        *reinterpret_cast<uint4*>(po + 32 * i + k) = make_uint4(x[k], x[k + 1], x[k + 2], x[k + 3]);
                }
            }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
            if (count > 0) mbar_arrive(bars.ofree + 8 * s);
            if (n_other > 0) mbar_arrive(bars.ofree + 8 * other);
        }
        // Rows that may have met a non-finite V of a key they do not see
        const int seen0 = (pair ? s0 : t0) * ROWS_KEYS, seen1 = min((pair ? s1 : t1) * ROWS_KEYS, len);
        const bool again = mine && count > 0 && !fine && !empty && fabsf(l) < INFINITY && (lo > seen0 || hi < seen1);
        unsigned todo = __ballot_sync(0xffffffffu, again);
        while (todo) {
            const int j = __ffs(todo) - 1;
            todo &= todo - 1;
            const int jtok = __shfl_sync(0xffffffffu, tok, j), jhead = __shfl_sync(0xffffffffu, head, j);
            const int jpos = __shfl_sync(0xffffffffu, tk.pos, j);
            const int jlo = max(__shfl_sync(0xffffffffu, lo, j), seen0), jhi = min(__shfl_sync(0xffffffffu, hi, j), seen1);
            const float jm = __shfl_sync(0xffffffffu, m, j), jl = __shfl_sync(0xffffffffu, l, j);
            float* jpo = reinterpret_cast<float*>(__shfl_sync(0xffffffffu, (unsigned long long)po, j));
            float o[D / 32];
            redo_row<D>(a, b, g, jhead, jtok, jpos, jlo, jhi, base, jm == -INFINITY ? 0.f : jm, cap_rate, o, bad);
            __nv_bfloat16* jout = static_cast<__nv_bfloat16*>(a.out) + ((long long)jtok * a.Hq + jhead) * D;
#pragma unroll
            for (int i = 0; i < D / 32; ++i) {
                if (direct) jout[lane + 32 * i] = __float2bfloat16_rn(o[i] / jl);
                else jpo[lane + 32 * i] = o[i];
            }
        }
        if (count > 0) ++nacc[s];
        if (n_other > 0) { ++nacc[other]; ++nml[other]; }
        if (pair && other_tiles) ++nacc[other];
    }
    rows_error(a, bad);
    return true;
}

// ------------------------------------------------------------------------------------------
// tile kernel
// ------------------------------------------------------------------------------------------
template <int D, bool MOD>
__global__ void __launch_bounds__(RW_THREADS, 1)
    rows_tile_kernel(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tk,
                     const __grid_constant__ CUtensorMap tv, const __grid_constant__ CUtensorMap tpk,
                     const __grid_constant__ CUtensorMap tpv, const RowsArgs a)
{
    extern __shared__ __align__(1024) uint8_t sm[];
    constexpr uint32_t NCOLS = 512;              // 2 x 128 of scores, 2 x D of sums
    const RowsSmem<D> lay(a.stages);
    const uint32_t sbase = smem_u32(sm);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
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
            mbar_init(bars.kvempty + 8 * i, 1);
        }
        for (int i = 0; i < RW_HDRS; ++i) {
            mbar_init(bars.hfull + 8 * i, 1);
            mbar_init(bars.hempty + 8 * i, 9);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(bars.qfull + 8 * i, 1);
            mbar_init(bars.qempty + 8 * i, 1);
            mbar_init(bars.sfull + 8 * i, 1);
            mbar_init(bars.pready + 8 * i, 4);
            mbar_init(bars.ofull + 8 * i, 1);
            mbar_init(bars.ofree + 8 * i, 4);
            mbar_init(bars.mlready + 8 * i, 4);
            mbar_init(bars.mlfree + 8 * i, 4);
        }
        mbar_init(bars.drain, 1);
        misc[0] = 0;
        fence_mbar_init();
    }
    if (warp == RW_MMA_WARP) tmem_alloc(smem_u32(tslot), NCOLS);
    if (warp == RW_LOAD_WARP && lane == 0) {
        prefetch_tensormap(&tq);
        prefetch_tensormap(&tk);
        prefetch_tensormap(&tv);
        prefetch_tensormap(&tpk);
        prefetch_tensormap(&tpv);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tslot;
    grid_dependency_wait();
    grid_launch_dependents();
    if (warp == RW_LOAD_WARP) {
        RowsLoader<D> ld{a, lay, bars, sm, sbase, misc};
        if (!ld.run(&tq, &tk, &tv, &tpk, &tpv)) ld.settle();
        if (ld.bad) rows_error(a, ld.bad);
    } else if (warp == RW_MMA_WARP) {
        RowsMma<D> mma{a, lay, bars, sm, sbase, tmem, misc};
        mma.run();
        // every MMA issued has landed before the tensor memory and the stages go
        if (lane == 0) umma_commit(bars.drain);
        __syncwarp();
        if (!mbar_wait(bars.drain, 0u) && lane == 0) rows_error(a, FDPP_ERRBIT_TIMEOUT);
        __syncwarp();
    } else {
        softmax_stream<D, MOD>(a, lay, bars, sm, tmem, warp >> 2, misc);
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
// Sums of one row in the frame of their largest max: lane's D / 32 columns (D / 32 lane ..).
template <int E>
struct RowSum {
    float m = -INFINITY, l = 0.f;
    float o[E];
    __device__ __forceinline__ RowSum()
    {
#pragma unroll
        for (int i = 0; i < E; ++i) o[i] = 0.f;
    }
    __device__ __forceinline__ void add(float2 ml, const float* po)
    {
        if (ml.x == -INFINITY && ml.y == 0.f) return;        // no key seen: its columns were not written
        float v[E];
        if constexpr (E == 4) {
            const float4 t = __ldcg(reinterpret_cast<const float4*>(po) + (threadIdx.x & 31));
            v[0] = t.x; v[1] = t.y; v[2] = t.z; v[3] = t.w;
        } else {
            const float2 t = __ldcg(reinterpret_cast<const float2*>(po) + (threadIdx.x & 31));
            v[0] = t.x; v[1] = t.y;
        }
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

// The partials of a unit cut in two or more: the part of its first tile left its own in slot 2 c + 1,
// every later one in slot 2 c.
template <int E>
__device__ __forceinline__ void add_cut(const RowsArgs& a, RowSum<E>& x, int start, int nt, int total, int first, long long row)
{
    for (int c = first; c < a.parts; ++c) {
        const int p0 = part_begin(c, total, a.parts);
        if (p0 >= start + nt) break;
        if (c > first && p0 == part_begin(c + 1, total, a.parts)) continue;      // an empty part
        const long long at = (long long)(2 * c + (c == first ? 1 : 0)) * a.slot_rows + row;
        x.add(__ldcg(a.slot_ml + at), a.slot_o + at * (E * 32));
    }
}

constexpr int JOIN_WARPS = 8;
constexpr int JOIN_ROWS = 32;       // rows of a cut unit per CTA

// Without a prefix: the units that a part boundary cuts, found from the boundaries (one grid column
// each; the first boundary inside a unit does it).
template <int D>
__global__ void __launch_bounds__(JOIN_WARPS * 32) rows_join_cut_kernel(RowsArgs a)
{
    grid_dependency_wait();
    grid_launch_dependents();
    const int c = blockIdx.x + 1, total = a.plan[RP_TILES];
    const int x = part_begin(c, total, a.parts);
    if (x <= 0 || x >= total) return;
    const RowTileRec r = a.rec[find_rt(a.rec, a.plan[RP_NRT], x)];
    const int g = (x - r.start) / r.nt, start = r.start + g * r.nt;
    if (x == start || part_begin(c - 1, total, a.parts) > start) return;
    const int rows = r.ntok * a.G, y0 = blockIdx.y * JOIN_ROWS;
    for (int row = y0 + (threadIdx.x >> 5); row < min(rows, y0 + JOIN_ROWS); row += JOIN_WARPS) {
        const int i = row / a.G, tok = r.tok0 + i;
        const RowToken tk = a.tok[tok];
        RowSum<D / 32> s;
        add_cut(a, s, start, r.nt, total, c - 1, row);
        s.store(static_cast<__nv_bfloat16*>(a.out) + ((long long)tok * a.Hq + g * a.G + (row - i * a.G)) * D, tk.hi <= tk.lo);
    }
}

// With a prefix: every row from its two units.
template <int D>
__global__ void __launch_bounds__(JOIN_WARPS * 32) rows_join_prefix_kernel(RowsArgs a)
{
    grid_dependency_wait();
    grid_launch_dependents();
    const long long w = (long long)blockIdx.x * JOIN_WARPS + (threadIdx.x >> 5);
    const int tok = (int)(w / a.Hq), head = (int)(w - (long long)tok * a.Hq);
    if (tok >= a.T) return;
    const RowToken tk = a.tok[tok];
    if (tk.rt < 0) return;
    const int total = a.plan[RP_TILES], npre = a.plan[RP_NPRE], g = head / a.G;
    RowSum<D / 32> s;
#pragma unroll
    for (int src = 0; src < 2; ++src) {
        if (src == 0 && npre == 0) continue;
        const RowTileRec r = a.rec[src ? tk.rt : tok / (2 * a.tpt)];
        if (r.nt == 0) continue;
        const int start = r.start + g * r.nt, first = part_of(start, total, a.parts);
        if (part_of(start + r.nt - 1, total, a.parts) == first) {
            const long long at = ((long long)src * a.T + tok) * a.Hq + head;
            s.add(__ldcg(a.row_ml + at), a.row_o + at * D);
        } else {
            add_cut(a, s, start, r.nt, total, first, (long long)(tok - r.tok0) * a.G + (head - g * a.G));
        }
    }
    s.store(static_cast<__nv_bfloat16*>(a.out) + ((long long)tok * a.Hq + head) * D, tk.hi <= tk.lo);
}

struct PdlConfig {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    PdlConfig(dim3 grid, int threads, size_t smem, cudaStream_t s)
    {
        cfg.gridDim = grid;
        cfg.blockDim = dim3((unsigned)threads);
        cfg.dynamicSmemBytes = smem;
        cfg.stream = s;
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
    }
};

template <int D, bool MOD>
cudaError_t launch_d(const RowsArgs& a, const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                     const CUtensorMap& tpk, const CUtensorMap& tpv, cudaStream_t s)
{
    PdlConfig plan(dim3(1), PLAN_THREADS, 0, s);
    cudaError_t e = cudaLaunchKernelEx(&plan.cfg, rows_plan_kernel, a);
    if (e != cudaSuccess) return e;
    auto kern = rows_tile_kernel<D, MOD>;
    const int smem = RowsSmem<D>(a.stages).total;
    if ((e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem)) != cudaSuccess) return e;
    PdlConfig tile(dim3((unsigned)a.parts), RW_THREADS, (size_t)smem, s);
    if ((e = cudaLaunchKernelEx(&tile.cfg, kern, tq, tk, tv, tpk, tpv, a)) != cudaSuccess) return e;
    if (a.prefix_len) {
        const long long rows = (long long)a.T * a.Hq;
        PdlConfig join(dim3((unsigned)((rows + JOIN_WARPS - 1) / JOIN_WARPS)), JOIN_WARPS * 32, 0, s);
        e = cudaLaunchKernelEx(&join.cfg, rows_join_prefix_kernel<D>, a);
    } else if (a.parts > 1) {
        PdlConfig join(dim3((unsigned)(a.parts - 1), (unsigned)((a.slot_rows + JOIN_ROWS - 1) / JOIN_ROWS)), JOIN_WARPS * 32, 0, s);
        e = cudaLaunchKernelEx(&join.cfg, rows_join_cut_kernel<D>, a);
    }
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

int rows_tc_stages(int head_dim, int smem_per_block)
{
    int n = 0;
    while (n < 16 && (head_dim == 128 ? RowsSmem<128>(n + 1).total : RowsSmem<64>(n + 1).total) <= smem_per_block) ++n;
    return n;
}

cudaError_t launch_rows_tc(const RowsArgs& a, const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                           const CUtensorMap& tpk, const CUtensorMap& tpv, cudaStream_t s)
{
    const bool mod = a.cap > 0.f || a.slopes;
    if (a.D == 128)
        return mod ? launch_d<128, true>(a, tq, tk, tv, tpk, tpv, s) : launch_d<128, false>(a, tq, tk, tv, tpk, tpv, s);
    return mod ? launch_d<64, true>(a, tq, tk, tv, tpk, tpv, s) : launch_d<64, false>(a, tq, tk, tv, tpk, tpv, s);
}

}  // namespace fdpp
