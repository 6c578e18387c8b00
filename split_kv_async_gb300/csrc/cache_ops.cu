// cache_ops.cu -- cache upkeep of a serving step (fdpp_cache.h): the block map (block tables, slot
// maps and token rows from request lengths) and rotary positions with the append to the cache.
#include <algorithm>
#include <cmath>

#include "device_common.cuh"
#include "fdpp_cache.h"

namespace fdpp {
namespace {

__device__ __forceinline__ void raise(unsigned* err, unsigned bits)
{
    if (bits) atomicOr(err, bits);
}

// ------------------------------------------------------------------------------------------
// block map
// ------------------------------------------------------------------------------------------
// Three running sums over the sequences decide everything: blocks asked for (who is served, and
// which queue entry a new block takes), tokens asked for (who is served), and tokens of the served
// (the token rows). A block asked for by a served sequence has only served ones before it: where an
// earlier one was refused for lack of blocks the sum stays above the count, and where it was refused
// for lack of rows every later one that has tokens is. So the sum over all that ask is also the
// place in the queue.
//
// Every new block holds a new token at its first position, so the row of that token writes the
// table entry, and a row whose block is new takes it from the queue itself: nothing waits for the
// table. What bounds this is latency, not bytes (a tick of 64 sequences moves 2 kB). So it is one
// launch wherever it can be: up to MAP_SMEM_SEQS sequences every CTA makes the whole plan for itself in
// shared memory (a few microseconds less than a launch that waits for another: 512 sequences with 81920
// rows 8.5 us in two launches) and takes its share of the rows; with one CTA that also serves calls in
// place and, with the plan in the workspace, any number of sequences. Only what needs more than one CTA
// and cannot plan apart (in place, where a CTA would read lengths that another has already replaced, or
// more sequences) takes a second launch over the rows.
struct MapArgs {
    const int32_t* held;
    const int32_t* want;
    const int32_t* pool_in;
    int32_t* table;
    int32_t* queue;
    int32_t* lens;
    int32_t* pool_out;
    int32_t* cu;
    int32_t* seq;
    int32_t* pos;
    int64_t* slots;
    unsigned* err;
    // plan (workspace or shared memory), for the rows: first row of each sequence, tokens held before,
    // first queue entry of the new blocks, freed blocks of the sequences up to each one, blocks kept
    int32_t* p_cu;     // [B + 1]
    int32_t* p_held;   // [B]
    int32_t* p_first;  // [B]
    int32_t* p_back;   // [B + 1]
    int32_t* p_kept;   // [B]
    int32_t* p_pool;   // [2] head, count, clamped
    int B, shift, width, cap, room;
};

constexpr int MAP_THREADS = 1024;

struct MapSums {
    long long need, ask;       // blocks and tokens asked for
    long long rows, back;      // tokens of the served, blocks freed
};

// Inclusive sums of two values over the threads of a CTA, and their totals. `red`: 2 x 32 words.
__device__ __forceinline__ void block_scan2(long long& x, long long& y, long long& tx, long long& ty,
                                            long long* red)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long a = __shfl_up_sync(0xffffffffu, x, o), b = __shfl_up_sync(0xffffffffu, y, o);
        if (lane >= o) { x += a; y += b; }
    }
    if (lane == 31) { red[warp] = x; red[32 + warp] = y; }
    __syncthreads();
    long long sx = lane < nw ? red[lane] : 0, sy = lane < nw ? red[32 + lane] : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long a = __shfl_up_sync(0xffffffffu, sx, o), b = __shfl_up_sync(0xffffffffu, sy, o);
        if (lane >= o) { sx += a; sy += b; }
    }
    tx = __shfl_sync(0xffffffffu, sx, 31);
    ty = __shfl_sync(0xffffffffu, sy, 31);
    const long long bx = __shfl_sync(0xffffffffu, sx, (warp + 31) & 31), by = __shfl_sync(0xffffffffu, sy, (warp + 31) & 31);
    if (warp) { x += bx; y += by; }
    __syncthreads();
}

// Queue entry i past the first (both below 2^31, so that the sum fits 32 bits unsigned).
__device__ __forceinline__ int wrap(long long i, int cap) { return (int)((unsigned)i % (unsigned)cap); }

// Rows r = first, first + step, ..: the sequence of a row is the last one that starts at or before
// it among those with rows (cu is non-decreasing).
__device__ __forceinline__ unsigned map_rows(const MapArgs& a, int first, int step)
{
    unsigned bad = 0;
    const int total = a.p_cu[a.B], bs = 1 << a.shift;
    const int head = a.p_pool[0];
    for (unsigned r0 = first; r0 < (unsigned)a.room; r0 += step) {       // (unsigned: room may be 2^31 - 1)
        const int r = (int)r0;
        int b = -1, pos = 0;
        long long slot = -1;
        if (r < total) {
            int lo = 0, hi = a.B;          // p_cu[lo] <= r < p_cu[hi]
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (a.p_cu[mid] <= r) lo = mid; else hi = mid;
            }
            b = lo;
            pos = a.p_held[b] + (r - a.p_cu[b]);
            const int j = pos >> a.shift, had = (int)(((long long)a.p_held[b] + bs - 1) >> a.shift);
            int block;
            if (j < had) {
                block = a.table[(long long)b * a.width + j];
            } else {
                block = a.queue[wrap((long long)head + a.p_first[b] + (j - had), a.cap)];
                if ((pos & (bs - 1)) == 0) a.table[(long long)b * a.width + j] = block;
            }
            if (block >= 0 && block < a.cap) slot = (long long)block * bs + (pos & (bs - 1));
            else bad = FDPP_ERRBIT_BLOCK_TABLE;
        }
        a.seq[r] = b;
        a.pos[r] = pos;
        a.slots[r] = slot;
    }
    // freed blocks, behind the free ones: the queue entries written are none of those read above
    const int freed = a.p_back[a.B], tail = wrap((long long)head + a.p_pool[1], a.cap);
    for (unsigned i0 = first; i0 < (unsigned)freed; i0 += step) {
        const int i = (int)i0;
        int lo = 0, hi = a.B;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (a.p_back[mid] <= i) lo = mid; else hi = mid;
        }
        const int block = a.table[(long long)lo * a.width + a.p_kept[lo] + (i - a.p_back[lo])];
        if (block < 0 || block >= a.cap) bad |= FDPP_ERRBIT_BLOCK_TABLE;
        a.queue[wrap((long long)tail + i, a.cap)] = block;
    }
    return bad;
}

constexpr int MAP_SMEM_SEQS = 1024;

// ROWS: the rows as well, in the same launch. SMEM: the plan in shared memory, so that any number of CTAs
// may make it; the first one writes what the caller gets of it.
template <bool ROWS, bool SMEM>
__global__ void __launch_bounds__(MAP_THREADS) block_map_kernel(MapArgs a)
{
    __shared__ long long red[64];
    __shared__ int32_t plan[SMEM ? 5 * MAP_SMEM_SEQS + 4 : 4];
    unsigned bad = 0;
    const int bs = 1 << a.shift;
    const int most = (int)min((long long)a.width << a.shift, (long long)INT32_MAX);
    const bool publish = blockIdx.x == 0;
    if (SMEM) {
        a.p_pool = plan;
        a.p_held = plan + 2;
        a.p_first = a.p_held + MAP_SMEM_SEQS;
        a.p_kept = a.p_first + MAP_SMEM_SEQS;
        a.p_back = a.p_kept + MAP_SMEM_SEQS;
        a.p_cu = a.p_back + MAP_SMEM_SEQS + 1;
    }
    grid_dependency_wait();
    int head = a.pool_in[0], count = a.pool_in[1];
    if (head < 0 || head >= a.cap || count < 0 || count > a.cap) {
        bad |= FDPP_ERRBIT_POOL;
        head = head < 0 || head >= a.cap ? 0 : head;
        count = count < 0 ? 0 : min(count, a.cap);
    }
    MapSums run{0, 0, 0, 0};
    long long taken = 0;
    for (int base = 0; base < a.B; base += blockDim.x) {
        const int b = base + threadIdx.x;
        int held = 0, want = 0;
        if (b < a.B) {
            const int h = a.held[b], w = a.want[b];
            held = clamp_len(h, most);
            want = clamp_len(w, most);
            if (held != h || want != w) bad |= FDPP_ERRBIT_SEQ_LEN;
        }
        const int old_blocks = (int)(((long long)held + bs - 1) >> a.shift);
        const int new_blocks = (int)(((long long)want + bs - 1) >> a.shift);
        const int need = max(0, new_blocks - old_blocks), ask = max(0, want - held);
        long long need_i = need, ask_i = ask, need_t, ask_t;
        block_scan2(need_i, ask_i, need_t, ask_t, red);
        const bool short_blocks = need > 0 && run.need + need_i > count;
        const bool short_rows = ask > 0 && run.ask + ask_i > a.room;
        const bool served = !short_blocks && !short_rows;
        if (short_blocks) bad |= FDPP_ERRBIT_POOL;
        if (short_rows) bad |= FDPP_ERRBIT_ROOM;
        // rows and blocks of the served, both below 2^31, in one word
        const int rows = served ? ask : 0, back = max(0, old_blocks - new_blocks);
        long long both_i = (long long)rows | ((long long)(served ? need : 0) << 32), back_i = back, both_t, back_t;
        block_scan2(both_i, back_i, both_t, back_t, red);
        const long long rows_i = both_i & 0xffffffffll, rows_t = both_t & 0xffffffffll;
        if (b < a.B) {
            const int cu = (int)(run.rows + rows_i - rows);
            a.p_cu[b] = cu;
            a.p_held[b] = held;
            a.p_first[b] = (int)min(run.need + need_i - need, (long long)INT32_MAX);
            a.p_back[b] = (int)(run.back + back_i - back);
            a.p_kept[b] = new_blocks;
            if (publish) {
                a.lens[b] = served ? want : held;
                a.cu[b] = cu;
            }
        }
        run.need += need_t;
        run.ask += ask_t;
        run.rows += rows_t;
        run.back += back_t;
        taken += both_t >> 32;
    }
    if (threadIdx.x == 0) {
        a.p_cu[a.B] = (int)run.rows;
        a.p_back[a.B] = (int)run.back;
        a.p_pool[0] = head;
        a.p_pool[1] = count;
        const long long now = (long long)count - taken + run.back;
        if (now > a.cap) bad |= FDPP_ERRBIT_POOL;      // more freed than the pool has
        if (publish) {
            a.cu[a.B] = (int)run.rows;
            a.pool_out[0] = wrap((long long)head + taken, a.cap);
            a.pool_out[1] = (int)min(now, (long long)a.cap);
        }
    }
    if (ROWS) {
        __syncthreads();
        bad |= map_rows(a, blockIdx.x * blockDim.x + threadIdx.x, gridDim.x * blockDim.x);
    }
    raise(a.err, bad);
}

__global__ void __launch_bounds__(256) block_map_rows_kernel(MapArgs a)
{
    grid_dependency_wait();
    raise(a.err, map_rows(a, blockIdx.x * blockDim.x + threadIdx.x, gridDim.x * blockDim.x));
}

// Rows that the planning CTA takes itself.
constexpr int MAP_ONE_CTA_ROWS = 4096;

bool block_params_ok(const fdpp_block_params* p)
{
    return p && p->batch >= 1 && p->block_size >= 16 && p->block_size <= 256 &&
           (p->block_size & (p->block_size - 1)) == 0 && p->max_blocks_per_seq >= 1 && p->num_kv_blocks >= 1 &&
           p->max_tokens >= 0 && (long long)p->batch * p->max_blocks_per_seq < (1ll << 31);
}

size_t block_ws_bytes(const fdpp_block_params& p) { return 256 + ((size_t)p.batch * 5 + 4) * 4; }

// ------------------------------------------------------------------------------------------
// rotary positions and append
// ------------------------------------------------------------------------------------------
// A row of q, k or v (one head of one token) is d / (2 VEC) items of two 16-byte vectors. In the
// half layout a rotated item is the vectors at i and i + rot / 2, so that a thread holds both
// halves of its pairs; interleaved it is two neighbouring vectors. Each lane keeps one item
// position for all the heads that its warp takes, so it needs its VEC angles once: the warp
// computes the token's angles (each pair once) into shared memory, and the lanes read theirs.
// The loads of the first heads are issued before the angles, which hide behind them.
//
// Bounded by HBM: every element is read once and written once: 403 MB of a prompt of 16384 tokens, 32 + 2 x 8
// heads of 128 in bf16, in 64.6 us, 6.24 TB/s (0.92 of a copy's measured rate); 64 tokens of 64 + 2 x 8 heads,
// 2.5 MB, 4.7 us launched from the host, 2.8 in a graph: latency.
struct RopeArgs {
    const void* q;
    const void* k;
    const void* v;
    const int32_t* pos;
    const int64_t* slots;
    const float2* table;
    void* q_out;
    void* k_cache;
    void* v_cache;
    unsigned* err;
    long long q_stride, k_stride, v_stride, num_slots;
    int T, Hq, Hkv, rot;
    float mag;
    int warps;             // warps per token
};

// (cos, sin) 2 pi pos (hi + lo). The product is reduced to a fraction of a turn before anything is
// rounded: pos is cut in two parts of at most 19 and 12 bits, a part times hi is the sum of two
// floats (product and FMA remainder), and whole turns are dropped from each exactly. For fp32 results what
// the sum of the fractions loses (2^-25 turns, 2e-7 rad, each time) is kept and turned by to first order: of
// 3.6e-8 off in the mean it leaves 2.8e-8, their own rounding (bf16's is 2^15 times that; 0.5 us of 65 for
// the prompt below).
template <bool KEEP>
__device__ __forceinline__ void add_kept(float& s, float& lost, float x)
{
    const float t = s + x, y = t - s;
    if (KEEP) lost += (s - (t - y)) + (x - y);
    s = t;
}

template <bool KEEP>
__device__ __forceinline__ float2 turn_of(int pos, float2 theta, float mag)
{
    const int low = pos & 4095;
    const float p1 = (float)(pos - low), p2 = (float)low;
    const float t1 = p1 * theta.x, t2 = p2 * theta.x;
    const float e1 = fmaf(p1, theta.x, -t1), e2 = fmaf(p2, theta.x, -t2);
    // p1 lo may pass one turn at positions beyond 2^24: reduced like the others
    const float l1 = p1 * theta.y;
    float r = t1 - rintf(t1), lost = fmaf(p1, theta.y, -l1);
    add_kept<KEEP>(r, lost, t2 - rintf(t2));
    add_kept<KEEP>(r, lost, l1 - rintf(l1));
    add_kept<KEEP>(r, lost, e1 - rintf(e1));
    add_kept<KEEP>(r, lost, e2 + p2 * theta.y + (KEEP ? 0.f : lost));
    float s, c;
    sincospif(2.f * r, &s, &c);
    const float d = KEEP ? 6.2831853f * lost : 0.f;
    return make_float2(fmaf(-s, d, c) * mag, fmaf(c, d, s) * mag);
}

template <typename T>
struct Vec16;

template <>
struct Vec16<float> {
    static constexpr int N = 4;
    __device__ static __forceinline__ void get(const uint4& v, float (&x)[4])
    {
        x[0] = __uint_as_float(v.x); x[1] = __uint_as_float(v.y);
        x[2] = __uint_as_float(v.z); x[3] = __uint_as_float(v.w);
    }
    __device__ static __forceinline__ uint4 put(const float (&x)[4])
    {
        return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
    }
};

template <>
struct Vec16<__nv_bfloat16> {
    static constexpr int N = 8;
    __device__ static __forceinline__ void get(const uint4& v, float (&x)[8])
    {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = __uint_as_float(w[i] << 16);
            x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
    __device__ static __forceinline__ uint4 put(const float (&x)[8])
    {
        return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                          pack_bf16x2(x[6], x[7]));
    }
};

constexpr int ROPE_WARPS = 8;      // per CTA
constexpr int ROPE_UNROLL = 4;

template <typename T, int D, bool INTER>
__global__ void __launch_bounds__(ROPE_WARPS * 32) rope_append_kernel(RopeArgs a)
{
    constexpr int N = Vec16<T>::N;
    constexpr int ITEMS = D / (2 * N);        // items of a head: 4, 8 or 16
    constexpr int HPW = 32 / ITEMS;           // heads a warp takes at a time
    __shared__ float2 cs_all[ROPE_WARPS][D / 2];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    float2* cs = cs_all[warp];
    grid_dependency_wait();
    const long long gw = (long long)blockIdx.x * ROPE_WARPS + warp;
    const long long t = gw / a.warps;
    const int part = (int)(gw - t * a.warps);
    if (t >= a.T) return;
    const long long slot = a.slots[t];
    if (slot < 0) return;
    const bool keep = slot < a.num_slots;
    if (!keep && lane == 0 && part == 0) raise(a.err, FDPP_ERRBIT_SLOT);
    const int heads = a.Hq + 2 * a.Hkv;
    const int p = lane % ITEMS, sub = lane / ITEMS;
    const int turned = a.rot / (2 * N);       // items that are rotated
    // offsets of the item's two vectors in a rotated head (q, k); v's are the plain ones
    int oa = 2 * N * p, ob = oa + N;
    if (!INTER && p < turned) { oa = N * p; ob = oa + a.rot / 2; }
    const T* q = static_cast<const T*>(a.q) + t * a.q_stride;
    const T* k = static_cast<const T*>(a.k) + t * a.k_stride;
    const T* v = static_cast<const T*>(a.v) + t * a.v_stride;
    T* qo = static_cast<T*>(a.q_out) + t * a.Hq * D;
    T* ko = static_cast<T*>(a.k_cache) + slot * a.Hkv * D;
    T* vo = static_cast<T*>(a.v_cache) + slot * a.Hkv * D;

    uint4 xa[ROPE_UNROLL], xb[ROPE_UNROLL];
    const int step = a.warps * HPW;
    auto load = [&](int h, uint4& va, uint4& vb) {
        if (h < a.Hq) {
            va = *reinterpret_cast<const uint4*>(q + h * D + oa);
            vb = *reinterpret_cast<const uint4*>(q + h * D + ob);
        } else if (h < a.Hq + a.Hkv) {
            va = *reinterpret_cast<const uint4*>(k + (h - a.Hq) * D + oa);
            vb = *reinterpret_cast<const uint4*>(k + (h - a.Hq) * D + ob);
        } else if (h < heads) {
            va = *reinterpret_cast<const uint4*>(v + (h - a.Hq - a.Hkv) * D + 2 * N * p);
            vb = *reinterpret_cast<const uint4*>(v + (h - a.Hq - a.Hkv) * D + 2 * N * p + N);
        }
    };
    int h0 = part * HPW + sub;
#pragma unroll
    for (int u = 0; u < ROPE_UNROLL; ++u) load(h0 + u * step, xa[u], xb[u]);

    const int pos = a.pos[t];
    for (int i = lane; i < a.rot / 2; i += 32) cs[i] = turn_of<sizeof(T) == 4>(pos, a.table[i], a.mag);
    __syncwarp();
    float2 w[N];
#pragma unroll
    for (int i = 0; i < N; ++i) w[i] = p < turned ? cs[p * N + i] : make_float2(1.f, 0.f);

    for (; h0 < heads; h0 += ROPE_UNROLL * step) {
#pragma unroll
        for (int u = 0; u < ROPE_UNROLL; ++u) {
            const int h = h0 + u * step;
            if (h >= heads) break;
            uint4 ya = xa[u], yb = xb[u];
            const bool is_v = h >= a.Hq + a.Hkv;
            if (!is_v && p < turned) {
                float fa[N], fb[N];
                Vec16<T>::get(ya, fa);
                Vec16<T>::get(yb, fb);
                if (INTER) {
#pragma unroll
                    for (int i = 0; i < N / 2; ++i) {
                        const float a0 = fa[2 * i], b0 = fa[2 * i + 1], a1 = fb[2 * i], b1 = fb[2 * i + 1];
                        fa[2 * i] = a0 * w[i].x - b0 * w[i].y;
                        fa[2 * i + 1] = a0 * w[i].y + b0 * w[i].x;
                        fb[2 * i] = a1 * w[N / 2 + i].x - b1 * w[N / 2 + i].y;
                        fb[2 * i + 1] = a1 * w[N / 2 + i].y + b1 * w[N / 2 + i].x;
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < N; ++i) {
                        const float x = fa[i], y = fb[i];
                        fa[i] = x * w[i].x - y * w[i].y;
                        fb[i] = x * w[i].y + y * w[i].x;
                    }
                }
                ya = Vec16<T>::put(fa);
                yb = Vec16<T>::put(fb);
            }
            if (h < a.Hq) {
                *reinterpret_cast<uint4*>(qo + h * D + oa) = ya;
                *reinterpret_cast<uint4*>(qo + h * D + ob) = yb;
            } else if (keep) {
                T* o = is_v ? vo + (h - a.Hq - a.Hkv) * D : ko + (h - a.Hq) * D;
                *reinterpret_cast<uint4*>(o + (is_v ? 2 * N * p : oa)) = ya;
                *reinterpret_cast<uint4*>(o + (is_v ? 2 * N * p + N : ob)) = yb;
            }
        }
#pragma unroll
        for (int u = 0; u < ROPE_UNROLL; ++u) load(h0 + (ROPE_UNROLL + u) * step, xa[u], xb[u]);
    }
}

}  // namespace
}  // namespace fdpp

using namespace fdpp;

extern "C" {

size_t fdpp_block_map_workspace_size(const fdpp_block_params* p)
{
    return block_params_ok(p) ? (block_ws_bytes(*p) + 255) / 256 * 256 : 0;
}

fdpp_status fdpp_block_map(const int32_t* held_lens, const int32_t* want_lens, const int32_t* pool_in,
                           const fdpp_block_params* p, int32_t* block_table, int32_t* pool_queue,
                           int32_t* seq_lens, int32_t* pool_out, int32_t* cu_tokens, int32_t* token_seq,
                           int32_t* positions, int64_t* slots, void* workspace, size_t workspace_bytes,
                           fdpp_stream stream)
{
    if (!p) return fail(FDPP_ERR_INVALID_ARG, "params is NULL");
    if (!block_params_ok(p))
        return fail(FDPP_ERR_INVALID_ARG,
                     "block map of batch %d, block_size %d (a power of two in [16, 256]), %d blocks per sequence, "
                     "%d blocks, %d rows (batch x blocks per sequence below 2^31)",
                     p->batch, p->block_size, p->max_blocks_per_seq, p->num_kv_blocks, p->max_tokens);
    if (!held_lens || !want_lens || !pool_in || !block_table || !pool_queue || !seq_lens || !pool_out || !cu_tokens)
        return fail(FDPP_ERR_INVALID_ARG, "lengths, pool state, block_table, pool_queue and cu_tokens must be non-NULL");
    if (p->max_tokens > 0 && (!token_seq || !positions || !slots))
        return fail(FDPP_ERR_INVALID_ARG, "token_seq, positions and slots must be non-NULL");
    if (want_lens == seq_lens) return fail(FDPP_ERR_INVALID_ARG, "seq_lens must not be want_lens");
    if ((((uintptr_t)held_lens | (uintptr_t)want_lens | (uintptr_t)pool_in | (uintptr_t)block_table |
          (uintptr_t)pool_queue | (uintptr_t)seq_lens | (uintptr_t)pool_out | (uintptr_t)cu_tokens |
          (uintptr_t)token_seq | (uintptr_t)positions) % 4) != 0 || ((uintptr_t)slots % 8) != 0)
        return fail(FDPP_ERR_INVALID_ARG, "int32 arrays must be 4-byte aligned, slots 8-byte aligned");
    if (!workspace) return fail(FDPP_ERR_WORKSPACE, "workspace is NULL");
    if ((uintptr_t)workspace % 256 != 0) return fail(FDPP_ERR_WORKSPACE, "workspace must be 256-byte aligned");
    if (workspace_bytes < block_ws_bytes(*p))
        return fail(FDPP_ERR_WORKSPACE, "workspace has %zu bytes, %zu needed", workspace_bytes, block_ws_bytes(*p));
    int sms = 0, unused = 0;
    const fdpp_status st = query_device(&sms, &unused, &unused);
    if (st != FDPP_OK) return st;

    MapArgs a{};
    a.held = held_lens;
    a.want = want_lens;
    a.pool_in = pool_in;
    a.table = block_table;
    a.queue = pool_queue;
    a.lens = seq_lens;
    a.pool_out = pool_out;
    a.cu = cu_tokens;
    a.seq = token_seq;
    a.pos = positions;
    a.slots = slots;
    a.B = p->batch;
    a.width = p->max_blocks_per_seq;
    a.cap = p->num_kv_blocks;
    a.room = p->max_tokens;
    while ((1 << a.shift) < p->block_size) ++a.shift;
    a.err = static_cast<unsigned*>(workspace);
    a.p_pool = reinterpret_cast<int32_t*>(static_cast<uint8_t*>(workspace) + 256);
    a.p_held = a.p_pool + 2;
    a.p_first = a.p_held + a.B;
    a.p_kept = a.p_first + a.B;
    a.p_back = a.p_kept + a.B;
    a.p_cu = a.p_back + a.B + 1;
    cudaStream_t s = (cudaStream_t)stream;
    cudaError_t e;
    const bool in_place = held_lens == seq_lens || pool_in == pool_out;
    if (a.B <= MAP_SMEM_SEQS && (a.room <= MAP_ONE_CTA_ROWS || !in_place)) {
        // several CTAs: just threads for the sequences, since each makes the plan, and a row a thread
        const bool one = a.room <= MAP_ONE_CTA_ROWS;
        const int work = one ? std::max(a.B, a.room) : std::max(a.B, 256);
        const int threads = std::min(MAP_THREADS, std::max(64, (work + 31) / 32 * 32));
        const int grid = one ? 1 : (int)std::min<long long>(2 * sms, ((long long)a.room + threads - 1) / threads);
        e = launch_pdl(block_map_kernel<true, true>, dim3((unsigned)grid), threads, s, a);
    } else if (a.room <= MAP_ONE_CTA_ROWS) {
        e = launch_pdl(block_map_kernel<true, false>, dim3(1), MAP_THREADS, s, a);
    } else {
        e = launch_pdl(block_map_kernel<false, false>, dim3(1), MAP_THREADS, s, a);
        if (e == cudaSuccess) {
            const int grid = (int)std::min<long long>(((long long)a.room + 255) / 256, sms * 8);
            e = launch_pdl(block_map_rows_kernel, dim3((unsigned)grid), 256, s, a);
        }
    }
    if (e != cudaSuccess) return fail(FDPP_ERR_CUDA, "block map launch: %s", cudaGetErrorString(e));
    return FDPP_OK;
}

fdpp_status fdpp_rope_table(int rot_dim, double base, int scaling, double factor, int context, double low_turns,
                            double high_turns, float* table)
{
    if (!table) return fail(FDPP_ERR_INVALID_ARG, "table is NULL");
    if (rot_dim < 16 || rot_dim > 128 || rot_dim % 16)
        return fail(FDPP_ERR_INVALID_ARG, "rot_dim must be a multiple of 16 in [16, 128] (got %d)", rot_dim);
    if (!(base > 1.0) || !std::isfinite(base)) return fail(FDPP_ERR_INVALID_ARG, "base must be finite and above 1");
    if (scaling < FDPP_ROPE_PLAIN || scaling > FDPP_ROPE_PARTS)
        return fail(FDPP_ERR_INVALID_ARG, "unknown scaling %d", scaling);
    if (scaling != FDPP_ROPE_PLAIN && (!(factor >= 1.0) || !std::isfinite(factor)))
        return fail(FDPP_ERR_INVALID_ARG, "factor must be finite and at least 1");
    if (scaling == FDPP_ROPE_PARTS && (context < 1 || !(low_turns < high_turns) || !std::isfinite(low_turns) ||
                                       !std::isfinite(high_turns)))
        return fail(FDPP_ERR_INVALID_ARG, "PARTS needs context >= 1 and finite low_turns < high_turns");
    const double two_pi = 6.283185307179586476925286766559;
    if (scaling == FDPP_ROPE_NTK) base *= std::pow(factor, (double)rot_dim / (rot_dim - 2));
    for (int i = 0; i < rot_dim / 2; ++i) {
        double theta = std::pow(base, -2.0 * i / rot_dim);
        if (scaling == FDPP_ROPE_LINEAR) theta /= factor;
        if (scaling == FDPP_ROPE_PARTS) {
            double k = (context * theta / two_pi - low_turns) / (high_turns - low_turns);
            k = k < 0.0 ? 0.0 : (k > 1.0 ? 1.0 : k);
            theta *= k + (1.0 - k) / factor;
        }
        const double turns = theta / two_pi;
        table[2 * i] = (float)turns;
        table[2 * i + 1] = (float)(turns - (double)table[2 * i]);
    }
    return FDPP_OK;
}

fdpp_status fdpp_rope_append(const void* q, const void* k, const void* v, const int32_t* positions,
                             const int64_t* slots, const float* table, const fdpp_rope_params* p, void* q_out,
                             void* k_cache, void* v_cache, void* workspace, size_t workspace_bytes,
                             fdpp_stream stream)
{
    if (!p) return fail(FDPP_ERR_INVALID_ARG, "params is NULL");
    if (p->num_tokens < 0 || p->num_q_heads < 1 || p->num_kv_heads < 1)
        return fail(FDPP_ERR_INVALID_ARG, "num_tokens must be >= 0 and head counts >= 1");
    if (p->dtype != FDPP_F32 && p->dtype != FDPP_BF16)
        return fail(FDPP_ERR_INVALID_ARG, "dtype must be FDPP_F32 or FDPP_BF16 (got %d)", p->dtype);
    if (p->head_dim != 64 && p->head_dim != 128)
        return fail(FDPP_ERR_UNSUPPORTED, "head_dim %d: only 64 and 128 are built", p->head_dim);
    if (p->rot_dim < 16 || p->rot_dim > p->head_dim || p->rot_dim % 16)
        return fail(FDPP_ERR_INVALID_ARG, "rot_dim must be a multiple of 16 in [16, %d] (got %d)", p->head_dim,
                     p->rot_dim);
    if (p->interleaved != 0 && p->interleaved != 1)
        return fail(FDPP_ERR_INVALID_ARG, "interleaved must be 0 or 1 (got %d)", p->interleaved);
    if (!std::isfinite(p->magnitude)) return fail(FDPP_ERR_INVALID_ARG, "magnitude must be finite");
    if (p->num_slots < 0) return fail(FDPP_ERR_INVALID_ARG, "num_slots must be >= 0");
    const int vec = p->dtype == FDPP_F32 ? 4 : 8;
    const long long q_row = (long long)p->num_q_heads * p->head_dim, k_row = (long long)p->num_kv_heads * p->head_dim;
    if (q_row > (1ll << 30) || k_row > (1ll << 30)) return fail(FDPP_ERR_INVALID_ARG, "too many heads");
    if (p->num_slots > (1ll << 62) / k_row) return fail(FDPP_ERR_INVALID_ARG, "num_slots is too large");
    if (p->q_stride < q_row || p->k_stride < k_row || p->v_stride < k_row || p->q_stride % vec || p->k_stride % vec ||
        p->v_stride % vec)
        return fail(FDPP_ERR_INVALID_ARG, "q, k and v strides must cover a row and be multiples of 16 bytes");
    if (!q || !k || !v || !positions || !slots || !table || !q_out || !k_cache || !v_cache)
        return fail(FDPP_ERR_INVALID_ARG, "q, k, v, positions, slots, table, q_out and the caches must be non-NULL");
    if ((((uintptr_t)q | (uintptr_t)k | (uintptr_t)v | (uintptr_t)q_out | (uintptr_t)k_cache | (uintptr_t)v_cache) % 16) != 0)
        return fail(FDPP_ERR_INVALID_ARG, "q, k, v, q_out and the caches must be 16-byte aligned");
    if ((uintptr_t)positions % 4 != 0 || (uintptr_t)slots % 8 != 0 || (uintptr_t)table % 8 != 0)
        return fail(FDPP_ERR_INVALID_ARG, "positions must be 4-byte, slots and table 8-byte aligned");
    if (q == q_out && p->q_stride != q_row)
        return fail(FDPP_ERR_INVALID_ARG, "q_out may be q only where q_stride is num_q_heads * head_dim");
    if (!workspace) return fail(FDPP_ERR_WORKSPACE, "workspace is NULL");
    if ((uintptr_t)workspace % 256 != 0) return fail(FDPP_ERR_WORKSPACE, "workspace must be 256-byte aligned");
    if (workspace_bytes < 256) return fail(FDPP_ERR_WORKSPACE, "workspace has %zu bytes, 256 needed", workspace_bytes);
    int sms = 0, unused = 0;
    const fdpp_status st = query_device(&sms, &unused, &unused);
    if (st != FDPP_OK) return st;
    if (p->num_tokens == 0) return FDPP_OK;

    RopeArgs a{};
    a.q = q;
    a.k = k;
    a.v = v;
    a.pos = positions;
    a.slots = slots;
    a.table = reinterpret_cast<const float2*>(table);
    a.q_out = q_out;
    a.k_cache = k_cache;
    a.v_cache = v_cache;
    a.err = static_cast<unsigned*>(workspace);
    a.q_stride = p->q_stride;
    a.k_stride = p->k_stride;
    a.v_stride = p->v_stride;
    a.num_slots = p->num_slots;
    a.T = p->num_tokens;
    a.Hq = p->num_q_heads;
    a.Hkv = p->num_kv_heads;
    a.rot = p->rot_dim;
    a.mag = p->magnitude;
    // warps per token: one where the tokens alone fill the GPU (64 warps per SM), else as many as its
    // heads have work for, so that a decode step's few tokens are spread too
    const int per_warp = 32 / (p->head_dim / (2 * vec));
    const int most = (a.Hq + 2 * a.Hkv + per_warp - 1) / per_warp;
    const long long fill = ((long long)sms * 64 + a.T - 1) / a.T;
    a.warps = (int)std::max(1ll, std::min<long long>(most, fill));
    const long long grid = ((long long)a.T * a.warps + ROPE_WARPS - 1) / ROPE_WARPS;
    if (grid > INT32_MAX) return fail(FDPP_ERR_INVALID_ARG, "too many tokens");
    void (*kern)(RopeArgs) = nullptr;
    const bool il = p->interleaved == 1, wide = p->head_dim == 128;
    if (p->dtype == FDPP_F32)
        kern = wide ? (il ? rope_append_kernel<float, 128, true> : rope_append_kernel<float, 128, false>)
                    : (il ? rope_append_kernel<float, 64, true> : rope_append_kernel<float, 64, false>);
    else
        kern = wide ? (il ? rope_append_kernel<__nv_bfloat16, 128, true> : rope_append_kernel<__nv_bfloat16, 128, false>)
                    : (il ? rope_append_kernel<__nv_bfloat16, 64, true> : rope_append_kernel<__nv_bfloat16, 64, false>);
    const cudaError_t e = launch_pdl(kern, dim3((unsigned)grid), ROPE_WARPS * 32, (cudaStream_t)stream, a);
    if (e != cudaSuccess) return fail(FDPP_ERR_CUDA, "rope append launch: %s", cudaGetErrorString(e));
    return FDPP_OK;
}

fdpp_status fdpp_read_error(const void* workspace, uint32_t* error_bits)
{
    if (!workspace || !error_bits) return fail(FDPP_ERR_INVALID_ARG, "null pointer");
    // the copy waits for the legacy stream alone, not for non-blocking streams
    cudaError_t e = cudaDeviceSynchronize();
    if (e != cudaSuccess) return fail(FDPP_ERR_CUDA, "cudaDeviceSynchronize: %s", cudaGetErrorString(e));
    if ((e = cudaMemcpy(error_bits, workspace, 4, cudaMemcpyDeviceToHost)) != cudaSuccess)
        return fail(FDPP_ERR_CUDA, "cudaMemcpy: %s", cudaGetErrorString(e));
    return FDPP_OK;
}

}  // extern "C"
