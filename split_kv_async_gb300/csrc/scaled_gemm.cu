// scaled_gemm.cu -- the linear layer on 8-bit operands with block scales (fdpp_linear.h), on tcgen05
// tensor cores:
//
//     y[m][n] = sum_b sx[m][b] sw[n / 128][b] sum_{k in block b} x[m][k] w[n][k]
//
// Both kernels stream blocks of 128 channels (128-byte rows, 128-byte swizzle) of x and w through a TMA
// ring; a block is four MMAs of K = 32 into a tensor-memory buffer of its own, which other warps read,
// scale by sx sw and add to fp32 sums in registers while the tensor cores work on the next block's buffer.
// The scales are fp32 numbers, so they cannot be left to the tensor cores (whose block scales are
// powers of two); sx sw is one product in fp32 for each row, block of w and block of K.
//
//   rows kernel (few rows): y^T = w x^T. 128 weight rows on the tensor-memory lanes, the rows of x on N, padded to the
//     next 16 only; two CTAs per SM.
//   tile kernel: 128 rows of x on the lanes, 128 or 256 weight rows on N, one persistent CTA per SM, or two as a pair.
// Where the tiles are too few for the GPU, K is cut into ranges whose CTAs form a cluster and add their sums through
// distributed shared memory, in range order.
//
// What bounds it. Few rows: HBM (28672 x 4096 weights: 8 rows 19.9 us, 0.88 of a measured copy, 64 rows 22.3), and for small
// weights the start and the end of a CTA (4096 x 4096, 8 rows: 5.8 us in a graph, of which the bytes take 2.5). Many rows: 8192 x
// 28672 x 4096 takes 680 to 700 us in ten calls after a rest, 2.8 PFLOP/s, and 740 to 770 one call after the other, when the
// power limit holds the clock at 1650 to 1740 MHz: 823 cycles for a block of K, a 32nd of a tile's stores among them. Two buffers of 256
// columns are all the tensor memory, so a block's sums have the 512 cycles of the next block's MMAs from the commit to the
// release. Neither is the bound by itself: the MMAs alone run at 4.6 PFLOP/s on data that lies there, at 3.5 to 3.7 with the
// loads (128 bytes of shared memory a cycle, written and read), and one CTA's hand-over alone, with its sums, takes 465 cycles
// a block; what they add to one another and the stores add was not measured apart. Tried: 192 columns and twelve warps
// of sums 782 us, sixteen warps of 64 columns 915, a buffer released before its last 64 sums 674 (673 to 684 without).
//
// Every wait is bounded: on a timeout the CTA records FDPP_ERRBIT_TIMEOUT, lets its copies and MMAs land,
// frees its tensor memory and exits.
#include <cuda_bf16.h>

#include <algorithm>
#include <map>
#include <mutex>

#include "device_common.cuh"
#include "fdpp_linear.h"
#include "gemm_common.cuh"
#include "tcgen05.cuh"

namespace fdpp {
namespace {

constexpr int SB = FDPP_SCALE_BLOCK;     // channels of a block: one 128-byte swizzle row
constexpr int SG_N = 128;                // weight rows that share a scale; the rows kernel's weight tile
constexpr int SG_ROWS = 128;             // the tile kernel's rows of x in a CTA
constexpr int SG_GROUP = 64;             // most rows of x that the rows kernel takes
constexpr int SG_MAX_SPLIT = 8;          // K ranges per weight tile (a portable cluster)
constexpr int SG_MAX_STAGES = 8;

struct ScaledArgs {
    const float* sx;
    const float* sw;
    void* y;
    unsigned* err;                       // sticky FDPP_ERRBIT_*
    long long y_stride, sx_stride;
    int M, N, kb;                        // kb: blocks of K
    int Mp, split_k, nstage;             // rows kernel: rows of x, padded; K ranges of a tile
    int m_tiles, n_tiles;                // tile kernel
};

// D (+)= A B^T of 32 channels, issued by the lane where `lead` is set: the whole warp runs the code around it, so
// that the operands stay in uniform registers. A and B: the descriptors' low words. PAIR: two CTAs as one operand
// (cta_group::2), issued by the first.
template <bool PAIR>
__device__ __forceinline__ void umma_e4m3(bool lead, uint32_t d_tmem, uint32_t alo, uint32_t blo, uint32_t idesc, uint32_t accumulate)
{
    if constexpr (PAIR)
        asm volatile(
            "{\n\t.reg .pred p, q;\n\t.reg .b64 da, db;\n\t"
            "setp.ne.b32 p, %4, 0;\n\t"
            "setp.ne.b32 q, %6, 0;\n\t"
            "mov.b64 da, {%1, %5};\n\t"
            "mov.b64 db, {%2, %5};\n\t"
            "@q tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], da, db, %3, p;\n\t}" ::"r"(d_tmem),
            "r"(alo), "r"(blo), "r"(idesc), "r"(accumulate), "n"(SW128_DESC_HI), "r"((uint32_t)lead)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p, q;\n\t.reg .b64 da, db;\n\t"
            "setp.ne.b32 p, %4, 0;\n\t"
            "setp.ne.b32 q, %6, 0;\n\t"
            "mov.b64 da, {%1, %5};\n\t"
            "mov.b64 db, {%2, %5};\n\t"
            "@q tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], da, db, %3, p;\n\t}" ::"r"(d_tmem),
            "r"(alo), "r"(blo), "r"(idesc), "r"(accumulate), "n"(SW128_DESC_HI), "r"((uint32_t)lead)
            : "memory");
}

// An arrival at the barrier, of both CTAs of a pair, when the MMAs issued so far have completed.
template <bool PAIR>
__device__ __forceinline__ void umma_done(bool lead, uint32_t bar)
{
    if constexpr (PAIR)
        asm volatile(
            "{\n\t.reg .pred q;\n\t"
            "setp.ne.b32 q, %2, 0;\n\t"
            "@q tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;\n\t}" ::"r"(bar),
            "h"((uint16_t)3), "r"((uint32_t)lead)
            : "memory");
    else
        umma_commit(lead, bar);
}

__device__ __forceinline__ void tmem_alloc_pair(uint32_t dst_smem, uint32_t ncols)
{
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(dst_smem), "r"(ncols) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}

__device__ __forceinline__ void tmem_dealloc_pair(uint32_t taddr, uint32_t ncols)
{
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}

// A load into this CTA's shared memory that completes on a barrier of either CTA of the pair.
__device__ __forceinline__ void tma_load_2d_pair(uint32_t dst, const CUtensorMap* map, int x, int y, uint32_t bar)
{
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar)
        : "memory");
}

// An arrival at a barrier of either CTA. (Released to the CTA only, as what it tells of is not memory but that the
// tensor-memory loads before it have completed; a release to the cluster waits a microsecond for the L2.)
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t bar)
{
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}

// Instruction descriptor of kind f8f6f4 with e4m3 A and B (types 0), both K-major, fp32 sums, M x N.
__host__ __device__ constexpr uint32_t umma_idesc_e4m3(int M, int N)
{
    return (1u << 4) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

// A block of 128 channels: four MMAs of 32.
template <bool PAIR>
__device__ __forceinline__ void umma_block(bool lead, uint32_t d_tmem, uint32_t a0, uint32_t b0, uint32_t idesc)
{
    const uint32_t alo = sw128_kmajor_lo(a0), blo = sw128_kmajor_lo(b0);
#pragma unroll
    for (int k = 0; k < 4; ++k) umma_e4m3<PAIR>(lead, d_tmem, alo + 2 * k, blo + 2 * k, idesc, k > 0 ? 1u : 0u);
}

__device__ __forceinline__ uint64_t pack2(float x, float y)
{
    uint64_t d;
    asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(x), "f"(y));
    return d;
}
__device__ __forceinline__ float2 unpack2(uint64_t d)
{
    float2 v;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(v.x), "=f"(v.y) : "l"(d));
    return v;
}
// acc += s v for the 64 consecutive columns v of this thread's tensor-memory lane, two columns to an operation (s2: s
// twice). One statement from the load to the sums: with the columns handed to C++ in between, a third of the
// instructions were moves from register to register, and two loads of 32 columns wait for tensor memory twice as often.
#define SUM2(acc, lo, hi) "mov.b64 d, {t" #lo ", t" #hi "};\n\tfma.rn.f32x2 %" #acc ", d, %32, %" #acc ";\n\t"
#define SUM8(a0, a1, a2, a3, c0, c1, c2, c3, c4, c5, c6, c7) SUM2(a0, c0, c1) SUM2(a1, c2, c3) SUM2(a2, c4, c5) SUM2(a3, c6, c7)
__device__ __forceinline__ void tmem_sum64(uint32_t taddr, uint64_t s2, uint64_t* a)
{
    asm volatile(
        "{\n\t.reg .b32 t<64>;\n\t.reg .b64 d;\n\t"
        "tcgen05.ld.sync.aligned.32x32b.x64.b32 {"
        "t0, t1, t2, t3, t4, t5, t6, t7, t8, t9, t10, t11, t12, t13, t14, t15, "
        "t16, t17, t18, t19, t20, t21, t22, t23, t24, t25, t26, t27, t28, t29, t30, t31, "
        "t32, t33, t34, t35, t36, t37, t38, t39, t40, t41, t42, t43, t44, t45, t46, t47, "
        "t48, t49, t50, t51, t52, t53, t54, t55, t56, t57, t58, t59, t60, t61, t62, t63}, [%33];\n\t"
        "tcgen05.wait::ld.sync.aligned;\n\t"
        SUM8(0, 1, 2, 3, 0, 1, 2, 3, 4, 5, 6, 7)
        SUM8(4, 5, 6, 7, 8, 9, 10, 11, 12, 13, 14, 15)
        SUM8(8, 9, 10, 11, 16, 17, 18, 19, 20, 21, 22, 23)
        SUM8(12, 13, 14, 15, 24, 25, 26, 27, 28, 29, 30, 31)
        SUM8(16, 17, 18, 19, 32, 33, 34, 35, 36, 37, 38, 39)
        SUM8(20, 21, 22, 23, 40, 41, 42, 43, 44, 45, 46, 47)
        SUM8(24, 25, 26, 27, 48, 49, 50, 51, 52, 53, 54, 55)
        SUM8(28, 29, 30, 31, 56, 57, 58, 59, 60, 61, 62, 63)
        "}"
        : "+l"(a[0]), "+l"(a[1]), "+l"(a[2]), "+l"(a[3]), "+l"(a[4]), "+l"(a[5]), "+l"(a[6]), "+l"(a[7]),
          "+l"(a[8]), "+l"(a[9]), "+l"(a[10]), "+l"(a[11]), "+l"(a[12]), "+l"(a[13]), "+l"(a[14]), "+l"(a[15]),
          "+l"(a[16]), "+l"(a[17]), "+l"(a[18]), "+l"(a[19]), "+l"(a[20]), "+l"(a[21]), "+l"(a[22]), "+l"(a[23]),
          "+l"(a[24]), "+l"(a[25]), "+l"(a[26]), "+l"(a[27]), "+l"(a[28]), "+l"(a[29]), "+l"(a[30]), "+l"(a[31])
        : "l"(s2), "r"(taddr)
        : "memory");
}
#undef SUM8
#undef SUM2

// 16 consecutive fp32 columns of this thread's TMEM lane, the wait in the same statement (see above).
__device__ __forceinline__ void tmem_ld16w(uint32_t taddr, float (&v)[16])
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]),
          "=f"(v[8]), "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15])
        : "r"(taddr)
        : "memory");
}

// Every lane waits; one that runs out aborts the CTA (warp-uniform result).
__device__ __forceinline__ bool gwait(uint32_t bar, uint32_t parity, volatile int* abort_, unsigned* err)
{
    if (__builtin_expect(__all_sync(0xffffffffu, mbar_try_wait(bar, parity & 1u)), 1)) return true;
    bool ok = *abort_ == 0 && mbar_wait_short(bar, parity & 1u);
    ok = __all_sync(0xffffffffu, ok);
    if (!ok && (threadIdx.x & 31) == 0) {
        *abort_ = 1;
        atomicOr(err, FDPP_ERRBIT_TIMEOUT);
    }
    return ok;
}

__device__ __forceinline__ void store_y(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }
__device__ __forceinline__ void store_y(float* p, float v) { *p = v; }

// The sums of g.split_k ranges, added in order, into y[m][n .. n + 3].
template <typename T>
__device__ __forceinline__ void store_sum4(const ScaledArgs& g, const float4 (&t)[SG_MAX_SPLIT], int m, int n, T* y)
{
    float4 s = t[0];
#pragma unroll
    for (int r = 1; r < SG_MAX_SPLIT; ++r)
        if (r < g.split_k) {
            s.x += t[r].x; s.y += t[r].y; s.z += t[r].z; s.w += t[r].w;
        }
    T* yp = y + (long long)m * g.y_stride + n;
    const float v[4] = {s.x, s.y, s.z, s.w};
    if (n + 3 < g.N && (reinterpret_cast<uintptr_t>(yp) & (4 * sizeof(T) - 1)) == 0) {
        if constexpr (sizeof(T) == 4) *reinterpret_cast<float4*>(yp) = s;
        else *reinterpret_cast<uint2*>(yp) = make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
    } else {
#pragma unroll
        for (int u = 0; u < 4; ++u)
            if (n + u < g.N) store_y(yp + u, v[u]);
    }
}

// ---- rows kernel --------------------------------------------------------------------------

constexpr int R_THREADS = 64;            // producer warp, MMA warp; then 128 threads that scale and add for every R_COLS rows of x
// (A block's sums follow one another, 64 rows of x in four warps at 700 ns a block: 64 rows of 20480 x 4096 took 24.2 us,
// of 28672 x 4096 24.7; with eight warps 20.8 and 22.3, with sixteen, which 56 registers leave spilling, 28.1 and 29.7. Half as many readings
// of x, by CTAs of 256 weight rows, saved nothing: 25.5.)
constexpr int R_COLS = 32;
__host__ __device__ constexpr int rows_sets(int nr) { return nr < R_COLS ? 1 : nr / R_COLS; }
constexpr int R_SCALES = 8;              // blocks of K whose scales are loaded together
constexpr int RW_BYTES = SG_N * SB;      // weight slice of a stage

// Shared memory (dynamic, 1024-byte aligned base): nstage stages of [w slice 16 KB | x slice Mp x 128 B],
// then the scales of 16 blocks, the barriers, the TMEM address and the abort flag. Once every MMA has
// completed, the stages hold this CTA's fp32 sums [M][128] for the cluster's reduction.
template <typename T, int NR>
__global__ void __launch_bounds__(R_THREADS + 128 * rows_sets(NR), 2)
    scaled_rows_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX,
                       const ScaledArgs g)
{
    extern __shared__ uint8_t smem_raw[];
    uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sbase = smem_u32(sm);
    constexpr int SETS = rows_sets(NR), C = NR / SETS;     // C: rows of x whose sums a warp has (Mp is above NR - C)
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int stage_bytes = RW_BYTES + g.Mp * SB;
    float* scale = reinterpret_cast<float*>(sm + g.nstage * stage_bytes);        // [2 R_SCALES][SG_GROUP]
    const int bar_off = g.nstage * stage_bytes + 2 * R_SCALES * SG_GROUP * 4;
    const uint32_t bars = sbase + bar_off;
    const uint32_t full = bars, empty = bars + 8 * g.nstage, accf = bars + 16 * g.nstage, acce = accf + 16;
    volatile uint32_t* tslot = reinterpret_cast<volatile uint32_t*>(sm + bar_off + 16 * g.nstage + 32);
    volatile int* abort_ = reinterpret_cast<volatile int*>(sm + bar_off + 16 * g.nstage + 40);
    volatile int* blocks_ = abort_ + 1;  // blocks whose MMAs were issued

    const int tile = blockIdx.x / g.split_k;
    const int ks = g.split_k > 1 ? (int)cluster_rank() : 0;
    const int n0 = tile * SG_N;
    const int kb0 = (int)((long long)ks * g.kb / g.split_k), kb1 = (int)((long long)(ks + 1) * g.kb / g.split_k);
    const int nkb = kb1 - kb0;
    uint32_t ncols = 32;                 // two buffers of Mp columns
    while ((int)ncols < 2 * g.Mp) ncols <<= 1;

    if (threadIdx.x == 0) {
        for (int s = 0; s < g.nstage; ++s) {
            mbar_init(full + 8 * s, 1);
            mbar_init(empty + 8 * s, 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(accf + 8 * b, 1);
            mbar_init(acce + 8 * b, 4 * SETS);
        }
        *abort_ = 0;
        fence_mbar_init();
        prefetch_tensormap(&tmW);
        prefetch_tensormap(&tmX);
    }
    if (warp == 1) tmem_alloc(smem_u32((const void*)tslot), ncols);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tslot;

    int issued = 0;                      // producer: slices issued
    if (warp == 0) {
        if (lane == 0) {
            // w is not written by the kernel before this one on the stream: the first ring's worth of it
            // streams while that kernel finishes
            const int pre = nkb < g.nstage ? nkb : g.nstage;
            for (int i = 0; i < pre; ++i) {
                mbar_arrive_expect_tx(full + 8 * i, (uint32_t)stage_bytes);
                tma_load_2d(sbase + i * stage_bytes, &tmW, (kb0 + i) * SB, n0, full + 8 * i);
            }
            grid_dependency_wait();
            for (int i = 0; i < pre; ++i)
                tma_load_2d(sbase + i * stage_bytes + RW_BYTES, &tmX, (kb0 + i) * SB, 0, full + 8 * i);
            issued = pre;
            for (int i = pre; i < nkb; ++i) {
                const int s = i % g.nstage;
                const uint32_t par = (uint32_t)(i / g.nstage) & 1u;
                if (*abort_ || !mbar_wait_short(empty + 8 * s, par ^ 1u)) {
                    atomicOr(g.err, FDPP_ERRBIT_TIMEOUT);
                    *abort_ = 1;
                    break;
                }
                const uint32_t dst = sbase + s * stage_bytes;
                const int k = (kb0 + i) * SB;
                mbar_arrive_expect_tx(full + 8 * s, (uint32_t)stage_bytes);
                tma_load_2d(dst, &tmW, k, n0, full + 8 * s);
                tma_load_2d(dst + RW_BYTES, &tmX, k, 0, full + 8 * s);
                ++issued;
            }
            grid_launch_dependents();
            if (!*abort_ && !ring_used(empty, (uint32_t)issued, (uint32_t)g.nstage)) {
                atomicOr(g.err, FDPP_ERRBIT_TIMEOUT);
                *abort_ = 1;
            }
        } else {
            grid_dependency_wait();
        }
    } else if (warp == 1) {
        grid_dependency_wait();
        const uint32_t idesc = umma_idesc_e4m3(SG_N, g.Mp);
        int done = 0;
        for (; done < nkb; ++done) {
            const int s = done % g.nstage, b = done & 1;
            if (!gwait(acce + 8 * b, ((uint32_t)(done >> 1) & 1u) ^ 1u, abort_, g.err) ||
                !gwait(full + 8 * s, (uint32_t)(done / g.nstage), abort_, g.err))
                break;
            tc_fence_after();
            const bool lead = elect_one();
            const uint32_t a0 = sbase + s * stage_bytes;
            umma_block<false>(lead, tmem + b * g.Mp, a0, a0 + RW_BYTES, idesc);
            umma_commit(lead, empty + 8 * s);
            umma_commit(lead, accf + 8 * b);
            __syncwarp();
        }
        if (lane == 0) *blocks_ = done;
        __syncwarp();
    } else {
        grid_dependency_wait();
        // ---- TMEM lanes 32 (warp % 4) .. hold weight rows n0 + that lane ----
        const int q = warp & 3, t = threadIdx.x - R_THREADS, c0 = C * (t >> 7);
        const int n = n0 + 32 * q + lane;
        const uint32_t trow = tmem + ((uint32_t)(32 * q) << 16) + c0;
        // the scales of R_SCALES blocks at a time, loaded as many blocks ahead, since a load takes longer than a block's MMAs
        // while the ring keeps the memory busy: this thread's are those of rows
        // t / R_SCALES, + APART in block t % R_SCALES
        constexpr int PER = C / 16, APART = 128 * SETS / R_SCALES;
        const int row = t / R_SCALES, j0 = t % R_SCALES;
        const float* sx = g.sx + (long long)row * g.sx_stride + kb0 + j0;
        const float* sw = g.sw + (long long)tile * g.kb + kb0 + j0;
        float acc[C];
#pragma unroll
        for (int j = 0; j < C; ++j) acc[j] = 0.f;
        float next[PER];
        auto load = [&](int k) {
#pragma unroll
            for (int u = 0; u < PER; ++u)
                next[u] = row + APART * u < g.M && k + j0 < nkb ? sx[APART * u * g.sx_stride + k] * sw[k] : 0.f;
        };
        load(0);
        bool ok = true;
        for (int i = 0; i < nkb; ++i) {
            const int b = i & 1;
            if (i % R_SCALES == 0) {
                float* to = scale + (i / R_SCALES & 1) * R_SCALES * SG_GROUP + j0 * SG_GROUP + row;
#pragma unroll
                for (int u = 0; u < PER; ++u) to[APART * u] = next[u];
                named_bar_sync(1, 128 * SETS);   // (this half was last read before the barrier R_SCALES blocks ago)
                load(i + R_SCALES);
            }
            const float* sc = scale + (i % (2 * R_SCALES)) * SG_GROUP + c0;
            ok = gwait(accf + 8 * b, (uint32_t)(i >> 1), abort_, g.err) && ok;
            if (ok) {
                tc_fence_after();
#pragma unroll
                for (int c = 0; c < C; c += 16) {
                    if (c0 + c >= g.Mp) break;
                    float v[16];
                    tmem_ld16w(trow + b * g.Mp + c, v);
                    if (c + 16 == C || c0 + c + 16 >= g.Mp) {    // the buffer is read out
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(acce + 8 * b);
                    }
#pragma unroll
                    for (int j = 0; j < 16; j += 4) {
                        const float4 s = *reinterpret_cast<const float4*>(sc + c + j);
                        acc[c + j] = fmaf(v[j], s.x, acc[c + j]);
                        acc[c + j + 1] = fmaf(v[j + 1], s.y, acc[c + j + 1]);
                        acc[c + j + 2] = fmaf(v[j + 2], s.z, acc[c + j + 2]);
                        acc[c + j + 3] = fmaf(v[j + 3], s.w, acc[c + j + 3]);
                    }
                }
            }
        }
        // the tensor cores' reads of the stages are complete (the last block's barrier); the sums of a
        // split tile reuse that memory
        fence_proxy_async_smem();
        float* red = reinterpret_cast<float*>(sm);
        T* y = static_cast<T*>(g.y);
        if (ok) {
#pragma unroll
            for (int j = 0; j < C; ++j) {
                const float v = acc[j];
                if (c0 + j < g.M) {
                    if (g.split_k > 1) red[(c0 + j) * SG_N + 32 * q + lane] = v;
                    else if (n < g.N) store_y(y + (long long)(c0 + j) * g.y_stride + n, v);
                }
            }
        }
    }

    // ---- split tile: every member adds its share of the outputs from all members' sums ----
    __syncthreads();
    if (g.split_k > 1) {
        // every thread of every member passes both cluster barriers, whatever happened before
        cluster_sync_all();
        if (!*abort_) {
            const int P = g.M * (SG_N / 4);
            const int p0 = (int)((long long)ks * P / g.split_k), p1 = (int)((long long)(ks + 1) * P / g.split_k);
            for (int i = p0 + (int)threadIdx.x; i < p1; i += R_THREADS + 128 * SETS) {
                const int m = i / (SG_N / 4), c = 4 * (i - m * (SG_N / 4)), n = n0 + c;
                if (n >= g.N) continue;
                const uint32_t off = sbase + (uint32_t)((m * SG_N + c) * 4);
                float4 t[SG_MAX_SPLIT];
#pragma unroll
                for (int r = 0; r < SG_MAX_SPLIT; ++r)
                    if (r < g.split_k) t[r] = ld_dsmem_f4(dsmem_addr(off, (uint32_t)r));
                store_sum4(g, t, m, n, static_cast<T*>(g.y));
            }
        }
        // no member leaves (releasing its shared memory) while another still reads it
        cluster_sync_all();
    }

    // ---- teardown: copies and MMAs landed (without an abort they have), tensor memory freed ----
    if (*abort_ && warp < 2) {
        RingBarriers slices{full, (uint32_t)stage_bytes};
        if (warp == 0 && lane == 0) land_ring(slices, (uint32_t)issued, (uint32_t)issued, (uint32_t)g.nstage);
        if (warp == 1) {
            RingBarriers{empty, 0u}.arrived((uint32_t)*blocks_, (uint32_t)g.nstage);
            RingBarriers{accf, 0u}.arrived((uint32_t)*blocks_, 2u);
        }
        __syncwarp();
    }
    tc_fence_after();
    if (warp == 1) tmem_dealloc(tmem, ncols);
}

// ---- tile kernel --------------------------------------------------------------------------
// PAIR: two CTAs (a cluster, on neighbouring SMs) work on 256 rows as one tensor-core operand. Each holds its
// 128 rows of x and half of the BN weight rows; the first one's MMA thread issues for both, each half's sums lie in its
// own CTA's tensor memory. What this saves is shared-memory bandwidth: a block of 128 x 256 sums takes 512
// cycles of the tensor cores, and 48 kB written and read again alone would be 768 at 128 bytes a cycle; with
// half of w it is 32 kB, 512 cycles.

// Warps: one loads, one issues the MMAs, two load scales; eight scale and add, each 32 rows and half of the columns.
constexpr int T_SCALES = 4;              // blocks of K whose scales are loaded together
constexpr int T_GROUP = 16;              // row tiles that a run of weight tiles is shared by (see tile_at)

template <int BN, bool PAIR>
struct TileSmem {
    static constexpr int COLS = BN / 2;                  // columns of a warp's sums
    static constexpr int SUM_WARPS = 8;
    static constexpr int THREADS = 128 + 32 * SUM_WARPS;
    // 128 x 56 + 256 x 224 = 64512, the launch's 384 x 168 registers; 128 x 80 + 256 x 200 = 61440 of them. (A spill in either part
    // shows: shared memory and the L1 cache are busy, and what should take 40 cycles takes hundreds. With 28 bytes of
    // them the largest prompt took 835 us instead of 696.)
    static constexpr int HELP_REGS = BN == 256 ? 56 : 80, SUM_REGS = BN == 256 ? 224 : 200;
    static constexpr int W_ROWS = PAIR ? BN / 2 : BN;    // weight rows that a CTA holds
    static constexpr int STAGE = (SG_ROWS + W_ROWS) * SB;
    static constexpr int TURN = 32 * 64;                 // a warp's rows, 64 bytes of each
    static constexpr int NBUF = 512 / BN;                // tensor-memory buffers of BN columns
    static constexpr int W_SCALES = (BN + SG_N - 1) / SG_N;          // blocks of 128 weight rows that a tile lies in
    static constexpr int SCALES = T_SCALES * W_SCALES * SG_ROWS;     // of T_SCALES blocks: sx sw by [block][128 of w][row]
    static constexpr int STAGES = 196608 / STAGE < SG_MAX_STAGES ? 196608 / STAGE : SG_MAX_STAGES;
    static constexpr int SCALES_OFF = STAGES * STAGE + SUM_WARPS * TURN;
    static constexpr int BARS = SCALES_OFF + 2 * SCALES * 4;
    static constexpr int TOTAL = BARS + (2 * STAGES + 2 * NBUF + 4) * 8 + 32 + 1024;
};

// Tile i of the order: T_GROUP row tiles at a time, the weight tiles outside, so that the CTAs at work
// together read few of either.
__device__ __forceinline__ void tile_at(const ScaledArgs& g, int i, int& mt, int& nt)
{
    const int per = T_GROUP * g.n_tiles, group = i / per, first = group * T_GROUP;
    const int rows = min(T_GROUP, g.m_tiles - first), r = i - group * per;
    nt = r / rows;
    mt = first + r - nt * rows;
}

// SPLIT: the g.split_k CTAs of a cluster share a tile's blocks of K and add their sums through distributed shared
// memory, in the order of their ranges.
template <typename T, int BN, bool PAIR, bool SPLIT>
__global__ void __launch_bounds__(TileSmem<BN, PAIR>::THREADS, 1)
    scaled_tile_kernel(const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmW, const ScaledArgs g)
{
    using L = TileSmem<BN, PAIR>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sbase = smem_u32(sm);
    const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const uint32_t full = sbase + L::BARS, empty = full + 8 * L::STAGES, accf = empty + 8 * L::STAGES, acce = accf + 8 * L::NBUF;
    const uint32_t scf = acce + 8 * L::NBUF, sce = scf + 16;
    volatile uint32_t* tslot = reinterpret_cast<volatile uint32_t*>(sm + L::BARS + (2 * L::STAGES + 2 * L::NBUF + 4) * 8);
    float* scales = reinterpret_cast<float*>(sm + L::SCALES_OFF);
    volatile int* abort_ = reinterpret_cast<volatile int*>(tslot + 2);
    volatile uint32_t* slices_ = tslot + 3;              // slices that this CTA issued, blocks whose MMAs were issued
    volatile uint32_t* blocks_ = tslot + 4;
    const int rank = PAIR ? (int)cluster_rank() : 0;
    // (both CTAs' loads complete on the first one's barriers, which its MMA thread waits for)
    const uint32_t full0 = PAIR ? dsmem_addr(full, 0) : full, acce0 = PAIR ? dsmem_addr(acce, 0) : acce;

    if (threadIdx.x == 0) {
        for (int s = 0; s < L::STAGES; ++s) {
            mbar_init(full + 8 * s, 1);
            mbar_init(empty + 8 * s, 1);
        }
        for (int b = 0; b < L::NBUF; ++b) {
            mbar_init(accf + 8 * b, 1);
            mbar_init(acce + 8 * b, (PAIR ? 2 : 1) * L::SUM_WARPS);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(scf + 8 * b, 2);
            mbar_init(sce + 8 * b, L::SUM_WARPS);
        }
        *abort_ = 0;
        fence_mbar_init();
        prefetch_tensormap(&tmW);
        prefetch_tensormap(&tmX);
    }
    if (warp == 1) {
        if (PAIR) tmem_alloc_pair(smem_u32((const void*)tslot), 512);
        else tmem_alloc(smem_u32((const void*)tslot), 512);
    }
    tc_fence_before();
    __syncthreads();
    if (PAIR) cluster_sync_all();
    tc_fence_after();
    const uint32_t tmem = *tslot;
    grid_dependency_wait();
    grid_launch_dependents();
    static_assert(!(PAIR && SPLIT), "a cluster is a pair or shares out K");
    static_assert(!SPLIT || SG_ROWS * BN * 4 <= L::STAGES * L::STAGE, "a split tile's sums take the place of the stages");
    const int tiles = g.m_tiles * g.n_tiles;
    // (with shared K a cluster has one tile: its sums take the place of the ring's stages)
    const int first = PAIR ? blockIdx.x >> 1 : SPLIT ? blockIdx.x / g.split_k : blockIdx.x;
    const int step = PAIR ? gridDim.x >> 1 : SPLIT ? tiles : gridDim.x;
    const int ks = SPLIT ? (int)cluster_rank() : 0;
    const int kb0 = SPLIT ? (int)((long long)ks * g.kb / g.split_k) : 0;
    const int nkb = (SPLIT ? (int)((long long)(ks + 1) * g.kb / g.split_k) : g.kb) - kb0;

    // Behind it no warp issues anything; whether one gave up, in either CTA of a pair. (Each part of the warps passes it and ends for
    // itself, in its own registers. Neither CTA's shared or tensor memory goes while the other uses it.)
    auto meet = [&]() -> bool {
        __syncthreads();
        if (PAIR) {
            if (threadIdx.x == 0 && *abort_) st_dsmem_u32(dsmem_addr(smem_u32((const void*)abort_), rank ^ 1u), 1u);
            cluster_sync_all();
        }
        return *abort_ != 0;
    };

    if (warp < 4) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(L::HELP_REGS));
        if (warp == 0 && lane == 0) {
            uint32_t i = 0;              // blocks issued
            bool ok = true;
            for (int t = first; t < tiles && ok; t += step) {
                int mt, nt;
                tile_at(g, t, mt, nt);
                const int m0 = (PAIR ? 2 * mt + rank : mt) * SG_ROWS, n0 = nt * BN + rank * L::W_ROWS;
                for (int k = kb0; k < kb0 + nkb; ++k, ++i) {
                    const uint32_t s = i % L::STAGES, par = (i / L::STAGES) & 1u;
                    if (*abort_ || !mbar_wait_short(empty + 8 * s, par ^ 1u)) {
                        atomicOr(g.err, FDPP_ERRBIT_TIMEOUT);
                        *abort_ = 1;
                        ok = false;
                        break;
                    }
                    const uint32_t dst = sbase + s * L::STAGE;
                    if (rank == 0) mbar_arrive_expect_tx(full + 8 * s, (uint32_t)((PAIR ? 2 : 1) * L::STAGE));
                    if (PAIR) {
                        tma_load_2d_pair(dst, &tmX, k * SB, m0, full0 + 8 * s);
                        tma_load_2d_pair(dst + SG_ROWS * SB, &tmW, k * SB, n0, full0 + 8 * s);
                    } else {
                        tma_load_2d(dst, &tmX, k * SB, m0, full + 8 * s);
                        tma_load_2d(dst + SG_ROWS * SB, &tmW, k * SB, n0, full + 8 * s);
                    }
                }
            }
            *slices_ = i;
            if (ok && !*abort_ && !ring_used(empty, i, L::STAGES)) {
                atomicOr(g.err, FDPP_ERRBIT_TIMEOUT);
                *abort_ = 1;
            }
        } else if (warp == 1 && rank == 0) {
            constexpr uint32_t IDESC = umma_idesc_e4m3(PAIR ? 2 * SG_ROWS : SG_ROWS, BN);
            uint32_t st = 0, sp = 0, b = 0, bp = 0, i = 0;       // stage and buffer, with their phases; blocks issued
            bool ok = true;
            for (int t = first; t < tiles && ok; t += step) {
                for (int k = 0; k < nkb; ++k, ++i) {
                    if (!gwait(full + 8 * st, sp, abort_, g.err) || !gwait(acce + 8 * b, bp ^ 1u, abort_, g.err)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const bool lead = elect_one();
                    const uint32_t a0 = sbase + st * L::STAGE;
                    umma_block<PAIR>(lead, tmem + b * BN, a0, a0 + SG_ROWS * SB, IDESC);
                    umma_done<PAIR>(lead, accf + 8 * b);
                    umma_done<PAIR>(lead, empty + 8 * st);
                    __syncwarp();
                    if (++st == (uint32_t)L::STAGES) { st = 0; sp ^= 1u; }
                    if (++b == (uint32_t)L::NBUF) { b = 0; bp ^= 1u; }
                }
            }
            if (lane == 0) *blocks_ = i;
        } else if (warp >= 2) {
            // ---- the scales, T_SCALES blocks of K at a time, well ahead of the sums: a load takes longer
            // than a block's MMAs while the ring keeps the memory busy ----
            const int r0 = threadIdx.x - 64;             // rows r0 and r0 + 64
            uint32_t c = 0;
            bool ok = true;
            for (int t = first; t < tiles && ok; t += step) {
                int mt, nt;
                tile_at(g, t, mt, nt);
                const int m0 = (PAIR ? 2 * mt + rank : mt) * SG_ROWS;
                const float* sx[2];
#pragma unroll
                for (int h = 0; h < 2; ++h) sx[h] = g.sx + (long long)(m0 + r0 + 64 * h < g.M ? m0 + r0 + 64 * h : 0) * g.sx_stride;
                for (int k0 = 0; k0 < nkb; k0 += T_SCALES, ++c) {
                    float v[2][T_SCALES], w[L::W_SCALES][T_SCALES];
#pragma unroll
                    for (int j = 0; j < T_SCALES; ++j) {
                        const int k = kb0 + min(k0 + j, nkb - 1);
#pragma unroll
                        for (int h = 0; h < 2; ++h) v[h][j] = sx[h][k];
                        // (weight rows past the last block have no scale of their own and are not stored)
#pragma unroll
                        for (int n = 0; n < L::W_SCALES; ++n)
                            w[n][j] = g.sw[(long long)min(nt * BN / SG_N + n, (g.N - 1) / SG_N) * g.kb + k];
                    }
                    float* to = scales + (c & 1) * L::SCALES;
                    if (!gwait(sce + 8 * (c & 1), (c >> 1) ^ 1u, abort_, g.err)) {
                        ok = false;
                        break;
                    }
#pragma unroll
                    for (int j = 0; j < T_SCALES; ++j)
#pragma unroll
                        for (int n = 0; n < L::W_SCALES; ++n)
#pragma unroll
                            for (int h = 0; h < 2; ++h) to[(j * L::W_SCALES + n) * SG_ROWS + r0 + 64 * h] = v[h][j] * w[n][j];
                    __syncwarp();
                    if (lane == 0) mbar_arrive(scf + 8 * (c & 1));
                }
            }
        }
        __syncwarp();
        if (meet()) {                    // copies and MMAs land before the CTAs end (without an abort they have)
            if (warp == 0 && lane == 0 && rank == 0) {
                RingBarriers slices{full, (uint32_t)L::STAGE};
                land_ring(slices, *slices_, PAIR ? ld_dsmem_u32(dsmem_addr(smem_u32((const void*)slices_), 1u)) : *slices_,
                          (uint32_t)L::STAGES);
            }
            if (warp == 1) {             // (of a pair each CTA gets the first one's arrivals)
                const uint32_t n = PAIR ? ld_dsmem_u32(dsmem_addr(smem_u32((const void*)blocks_), 0u)) : *blocks_;
                RingBarriers{empty, 0u}.arrived(n, L::STAGES);
                RingBarriers{accf, 0u}.arrived(n, L::NBUF);
            }
            __syncwarp();
            if (PAIR) cluster_sync_all();
        }
        if (SPLIT) {
            cluster_sync_all();
            cluster_sync_all();
        }
        if (warp == 1) {
            tc_fence_after();
            if (PAIR) tmem_dealloc_pair(tmem, 512);
            else tmem_dealloc(tmem, 512);
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(L::SUM_REGS));
        constexpr int COLS = L::COLS;
        const int w = warp - 4, q = w & 3, part = w >> 2;        // lanes 32 q .., columns COLS part ..
        const uint32_t trow = tmem + ((uint32_t)(32 * q) << 16) + part * COLS;
        uint8_t* turn = sm + L::STAGES * L::STAGE + w * L::TURN;
        T* y = static_cast<T*>(g.y);
        // 16-byte stores where y and its rows allow them
        const bool wide = ((reinterpret_cast<uintptr_t>(y) | (uintptr_t)(g.y_stride * (long long)sizeof(T))) & 15u) == 0;
        uint32_t b = 0, bp = 0, c = 0;   // buffer and its phase, sets of scales
        bool ok = true;
        for (int t = first; t < tiles; t += step) {
            int mt, nt;
            tile_at(g, t, mt, nt);
            const int m0 = (PAIR ? 2 * mt + rank : mt) * SG_ROWS + 32 * q, n0 = nt * BN + part * COLS;
            uint64_t acc[COLS / 2];
#pragma unroll
            for (int j = 0; j < COLS / 2; ++j) acc[j] = 0ull;
            // (One way through these loops, whatever a wait says: with a way out of them the sums move to other registers.)
#pragma unroll 1
            for (int k0 = 0; k0 < nkb; k0 += T_SCALES, ++c) {
                ok = gwait(scf + 8 * (c & 1), c >> 1, abort_, g.err) && ok;
                const float* sc = scales + (c & 1) * L::SCALES + (n0 / SG_N - nt * BN / SG_N) * SG_ROWS + 32 * q + lane;
                float s = *sc;
#pragma unroll 1
                for (int k = min(T_SCALES, nkb - k0); k > 0; --k) {
                    ok = gwait(accf + 8 * b, bp, abort_, g.err) && ok;
                    tc_fence_after();
                    const uint64_t s2 = pack2(s, s);
                    sc += L::W_SCALES * SG_ROWS;
                    if (k > 1) s = *sc;                  // (the next block's: an answer of shared memory takes long)
#pragma unroll
                    for (int h = 0; h < COLS / 64; ++h) tmem_sum64(trow + b * BN + 64 * h, s2, acc + 32 * h);
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) {                     // the buffer is read out
                        if (PAIR) mbar_arrive_cluster(acce0 + 8 * b);
                        else mbar_arrive(acce + 8 * b);
                    }
                    if (++b == (uint32_t)L::NBUF) { b = 0; bp ^= 1u; }
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(sce + 8 * (c & 1));
            }
            if (!ok) break;
            if constexpr (SPLIT) {
                // the tensor cores' reads of the stages are complete (the last block's barrier). Row r's 16-byte pieces lie
                // at piece ^ (r & 7)
                fence_proxy_async_smem();
                const int row = 32 * q + lane;
                float* to = reinterpret_cast<float*>(sm) + row * BN;
#pragma unroll
                for (int j = 0; j < COLS / 4; ++j) {
                    const float2 p0 = unpack2(acc[2 * j]), p1 = unpack2(acc[2 * j + 1]);
                    *reinterpret_cast<float4*>(to + (((part * COLS / 4 + j) ^ (row & 7)) << 2)) = make_float4(p0.x, p0.y, p1.x, p1.y);
                }
                continue;
            }
            // 64 bytes of every row at a time, turned through shared memory (16-byte pieces of row r at piece
            // ^ (r / 2 % 4)), so that a store instruction writes whole sectors
            constexpr int PC = 64 / (int)sizeof(T), PIECE = 16 / (int)sizeof(T);         // columns of 64 and of 16 bytes
#pragma unroll
            for (int col = 0; col < COLS; col += PC) {
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    uint4 v;
                    const uint64_t* x = acc + (col + k * PIECE) / 2;
                    const float2 p0 = unpack2(x[0]), p1 = unpack2(x[1]);
                    if constexpr (sizeof(T) == 4) {
                        v = make_uint4(__float_as_uint(p0.x), __float_as_uint(p0.y), __float_as_uint(p1.x), __float_as_uint(p1.y));
                    } else {
                        const float2 p2 = unpack2(x[2]), p3 = unpack2(x[3]);
                        v = make_uint4(pack_bf16x2(p0.x, p0.y), pack_bf16x2(p1.x, p1.y), pack_bf16x2(p2.x, p2.y), pack_bf16x2(p3.x, p3.y));
                    }
                    *reinterpret_cast<uint4*>(turn + lane * 64 + ((k ^ (lane >> 1 & 3)) << 4)) = v;
                }
                __syncwarp();
                const int n1 = n0 + col;
                if (wide && n1 + PC <= g.N) {
#pragma unroll
                    for (int k = 0; k < 32; k += 8) {
                        const int row = k + (lane >> 2), piece = lane & 3;
                        const uint4 v = *reinterpret_cast<const uint4*>(turn + row * 64 + ((piece ^ (row >> 1 & 3)) << 4));
                        if (m0 + row < g.M) *reinterpret_cast<uint4*>(y + (long long)(m0 + row) * g.y_stride + n1 + piece * PIECE) = v;
                    }
                } else {                 // element by element, neighbours on neighbouring lanes
                    for (int e = lane; e < 32 * PC; e += 32) {
                        const int row = e / PC, x = e % PC;
                        const T v = *reinterpret_cast<const T*>(turn + row * 64 + (((x / PIECE) ^ (row >> 1 & 3)) << 4) + (x % PIECE) * (int)sizeof(T));
                        if (m0 + row < g.M && n1 + x < g.N) y[(long long)(m0 + row) * g.y_stride + n1 + x] = v;
                    }
                }
                __syncwarp();
            }
        }
        tc_fence_before();
        const bool gave_up = meet();
        if (PAIR && gave_up) cluster_sync_all();
        if constexpr (SPLIT) {
            // every thread of every member passes both cluster barriers, whatever happened before
            cluster_sync_all();
            if (!gave_up) {
                int mt, nt;
                tile_at(g, first, mt, nt);
                const int r0 = ks * SG_ROWS / g.split_k, r1 = (ks + 1) * SG_ROWS / g.split_k;
                for (int i = r0 * (BN / 4) + (int)threadIdx.x - 128; i < r1 * (BN / 4); i += L::THREADS - 128) {
                    const int row = i / (BN / 4), piece = i % (BN / 4), m = mt * SG_ROWS + row, n = nt * BN + 4 * piece;
                    if (m >= g.M || n >= g.N) continue;
                    const uint32_t off = sbase + (uint32_t)((row * BN + ((piece ^ (row & 7)) << 2)) * 4);
                    float4 t[SG_MAX_SPLIT];
#pragma unroll
                    for (int r = 0; r < SG_MAX_SPLIT; ++r)
                        if (r < g.split_k) t[r] = ld_dsmem_f4(dsmem_addr(off, (uint32_t)r));
                    store_sum4(g, t, m, n, static_cast<T*>(g.y));
                }
            }
            cluster_sync_all();
        }
    }
}

// ---- host ---------------------------------------------------------------------------------

int blocks_of(int K) { return (K + SB - 1) / SB; }

fdpp_status check_params(const fdpp_scaled_gemm_params* p)
{
    if (!p) return fail(FDPP_ERR_INVALID_ARG, "params is NULL");
    if (p->M < 0 || p->N < 1 || p->K < 16 || p->K % 16)
        return fail(FDPP_ERR_INVALID_ARG, "scaled GEMM shape M=%d N=%d K=%d (M >= 0, N >= 1, K >= 16, K %% 16 == 0)", p->M,
                     p->N, p->K);
    if (p->N > (1 << 30) || p->K > (1 << 30) || p->M > (1 << 30)) return fail(FDPP_ERR_INVALID_ARG, "problem too large for one call");
    if (p->out_dtype != FDPP_F32 && p->out_dtype != FDPP_BF16)
        return fail(FDPP_ERR_INVALID_ARG, "out_dtype must be FDPP_F32 or FDPP_BF16 (got %d)", p->out_dtype);
    const long long most = 1ll << 39;    // of a tensor map's strides
    if (p->x_stride < p->K || p->w_stride < p->K || p->x_stride % 16 || p->w_stride % 16 || p->x_stride > most || p->w_stride > most)
        return fail(FDPP_ERR_INVALID_ARG, "x_stride and w_stride must cover a row and be multiples of 16 bytes");
    if (p->y_stride < p->N || p->y_stride > most) return fail(FDPP_ERR_INVALID_ARG, "y_stride must cover a row");
    if (p->x_scale_stride < blocks_of(p->K) || p->x_scale_stride > most)
        return fail(FDPP_ERR_INVALID_ARG, "x_scale_stride must cover a row's scales");
    if (p->split_k < 0 || p->split_k > std::min(blocks_of(p->K), SG_MAX_SPLIT))
        return fail(FDPP_ERR_INVALID_ARG, "split_k %d outside 0 .. %d", p->split_k, std::min(blocks_of(p->K), SG_MAX_SPLIT));
    return FDPP_OK;
}

fdpp_status encode_rows(CUtensorMap* map, const void* base, int rows, int K, long long stride, int box_rows)
{
    PFN_cuTensorMapEncodeTiled_v12000 enc = nullptr;
    const fdpp_status st = get_tensor_map_encoder(&enc);
    if (st != FDPP_OK) return st;
    cuuint64_t dims[2] = {(cuuint64_t)K, (cuuint64_t)rows};
    cuuint64_t strides[1] = {(cuuint64_t)stride};
    cuuint32_t box[2] = {SB, (cuuint32_t)box_rows};
    cuuint32_t estr[2] = {1, 1};
    const CUresult r = enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box, estr,
                           CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                           CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) return fail(FDPP_ERR_CUDA, "cuTensorMapEncodeTiled failed (%d)", (int)r);
    return FDPP_OK;
}

using SgKernel = void (*)(const CUtensorMap, const CUtensorMap, const ScaledArgs);

template <typename T>
SgKernel rows_kernel(int Mp)
{
    return Mp <= 16 ? scaled_rows_kernel<T, 16> : Mp <= 32 ? scaled_rows_kernel<T, 32> : scaled_rows_kernel<T, 64>;
}

int rows_smem(int Mp, int nstage) { return nstage * (RW_BYTES + Mp * SB) + 2 * R_SCALES * SG_GROUP * 4 + 16 * nstage + 64 + 1024; }

// Ring depth for two CTAs per SM.
int rows_stages(int Mp, int smem_per_sm, int smem_per_block)
{
    const int budget = std::min(smem_per_sm / 2 - 1024, smem_per_block) - rows_smem(Mp, 0) - 16 * SG_MAX_STAGES;
    return std::max(2, std::min(SG_MAX_STAGES, budget / (RW_BYTES + Mp * SB)));
}

// Clusters of `split` CTAs that the GPU holds at once; cached (0 if the query fails, which is not).
int max_clusters(SgKernel kern, int split, int threads, int smem)
{
    static std::mutex mu;
    static std::map<std::pair<SgKernel, std::pair<int, long long>>, int> cache;
    int dev = 0;
    cudaGetDevice(&dev);
    const auto key = std::make_pair(kern, std::make_pair(dev, ((long long)split << 32) | smem));
    std::lock_guard<std::mutex> lk(mu);
    const auto it = cache.find(key);
    if (it != cache.end()) return it->second;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)split);
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = (size_t)smem;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)split;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, kern, &cfg) == cudaSuccess) return cache[key] = n;
    cudaGetLastError();
    return 0;
}

// Ranges of K for `tiles` output tiles: as many as keep all clusters on the GPU at once. The query for resident
// clusters takes a kernel with tensor memory for one CTA per SM; of the rows kernel, whose CTAs share an SM by two, twice
// as many fit, and as many as there are places for clusters of half the size. (8 rows, us in a graph: 4096 x 4096, 32 tiles, in
// 2 ranges 8.3, in 4 6.0, in 8 5.8; 6144 x 4096, 48 tiles, in 4 or 5 7.6, in 6, which do not fit, 12.4; 4096 x 14336 in 4 15.3,
// in 8 12.4. The rule does not look at the rows: 64 of 4096 x 4096 take 7.3 in 4 ranges and 8.6 in the 8 that it gives.)
int choose_split(SgKernel kern, long long tiles, int kb, int threads, int smem, int ctas_per_sm, int sms)
{
    for (int n = std::min(SG_MAX_SPLIT, kb); n > 1; --n) {
        if (tiles * n > (long long)ctas_per_sm * sms) continue;
        int fit = max_clusters(kern, n, threads, smem);
        if (ctas_per_sm == 2) fit = std::max(2 * fit, n > 2 ? max_clusters(kern, (n + 1) / 2, threads, smem) : 0);
        if (tiles <= fit) return n;
    }
    return 1;
}

fdpp_status launch_rows(const fdpp_scaled_gemm_params& p, ScaledArgs& g, const void* x, const void* w, int sms, int smem_sm,
                        int smem_blk, cudaStream_t s)
{
    g.Mp = (p.M + 15) / 16 * 16;
    g.nstage = rows_stages(g.Mp, smem_sm, smem_blk);
    const int smem = rows_smem(g.Mp, g.nstage), tiles = (p.N + SG_N - 1) / SG_N;
    const int nr = g.Mp <= 16 ? 16 : g.Mp <= 32 ? 32 : 64, threads = R_THREADS + 128 * rows_sets(nr);
    const SgKernel kern = p.out_dtype == FDPP_F32 ? rows_kernel<float>(g.Mp) : rows_kernel<__nv_bfloat16>(g.Mp);
    cudaError_t e = allow_dynamic_smem((const void*)kern);
    if (e != cudaSuccess) return fail(FDPP_ERR_CUDA, "cudaFuncSetAttribute: %s", cudaGetErrorString(e));
    g.split_k = p.split_k ? p.split_k : choose_split(kern, tiles, g.kb, threads, smem, 2, sms);
    CUtensorMap tw, tx;
    fdpp_status st;
    if ((st = encode_rows(&tw, w, p.N, p.K, p.w_stride, SG_N)) != FDPP_OK) return st;
    if ((st = encode_rows(&tx, x, p.M, p.K, p.x_stride, g.Mp)) != FDPP_OK) return st;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(tiles * g.split_k));
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = (size_t)smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)g.split_k;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    e = cudaLaunchKernelEx(&cfg, kern, tw, tx, g);
    if (e == cudaSuccess) e = cudaGetLastError();
    if (e != cudaSuccess) return fail(FDPP_ERR_CUDA, "scaled GEMM launch: %s", cudaGetErrorString(e));
    return FDPP_OK;
}

template <typename T, int BN, bool PAIR>
fdpp_status launch_tile(const fdpp_scaled_gemm_params& p, ScaledArgs& g, const void* x, const void* w, int sms, int smem_blk,
                        cudaStream_t s)
{
    constexpr int smem = TileSmem<BN, PAIR>::TOTAL, rows = PAIR ? 2 * SG_ROWS : SG_ROWS, threads = TileSmem<BN, PAIR>::THREADS;
    if (smem > smem_blk) return fail(FDPP_ERR_UNSUPPORTED, "too little shared memory for the tile kernel");
    const long long m_tiles = ((long long)p.M + rows - 1) / rows, n_tiles = ((long long)p.N + BN - 1) / BN;
    if (m_tiles * n_tiles >= (1ll << 31) - sms || T_GROUP * n_tiles >= (1ll << 31))
        return fail(FDPP_ERR_INVALID_ARG, "problem too large for one call");
    g.m_tiles = (int)m_tiles;
    g.n_tiles = (int)n_tiles;
    CUtensorMap tw, tx;
    fdpp_status st;
    if ((st = encode_rows(&tw, w, p.N, p.K, p.w_stride, TileSmem<BN, PAIR>::W_ROWS)) != FDPP_OK) return st;
    if ((st = encode_rows(&tx, x, p.M, p.K, p.x_stride, SG_ROWS)) != FDPP_OK) return st;
    SgKernel kern = scaled_tile_kernel<T, BN, PAIR, false>;
    g.split_k = 1;
    cudaError_t e;
    if constexpr (!PAIR) {
        const SgKernel split = scaled_tile_kernel<T, BN, PAIR, true>;
        if ((e = allow_dynamic_smem((const void*)split)) != cudaSuccess)
            return fail(FDPP_ERR_CUDA, "cudaFuncSetAttribute: %s", cudaGetErrorString(e));
        g.split_k = p.split_k ? p.split_k : choose_split(split, m_tiles * n_tiles, g.kb, threads, smem, 1, sms);
        if (g.split_k > 1) kern = split;
    }
    if ((e = allow_dynamic_smem((const void*)kern)) != cudaSuccess)
        return fail(FDPP_ERR_CUDA, "cudaFuncSetAttribute: %s", cudaGetErrorString(e));
    const int cluster = PAIR ? 2 : g.split_k;
    const long long tiles = m_tiles * n_tiles;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(cluster * (g.split_k > 1 ? tiles : std::min<long long>(sms / cluster, tiles))));
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = (size_t)smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    e = cudaLaunchKernelEx(&cfg, kern, tx, tw, g);
    if (e == cudaSuccess) e = cudaGetLastError();
    if (e != cudaSuccess) return fail(FDPP_ERR_CUDA, "scaled GEMM launch: %s", cudaGetErrorString(e));
    return FDPP_OK;
}

}  // namespace
}  // namespace fdpp

using namespace fdpp;

extern "C" {

size_t fdpp_scaled_gemm_workspace_size(const fdpp_scaled_gemm_params* p) { return check_params(p) == FDPP_OK ? 256 : 0; }

fdpp_status fdpp_scaled_gemm(const void* x, const float* x_scales, const void* w, const float* w_scales,
                             const fdpp_scaled_gemm_params* p, void* workspace, size_t workspace_bytes, void* y,
                             fdpp_stream stream)
try {
    fdpp_status st = check_params(p);
    if (st != FDPP_OK) return st;
    if (!w || !w_scales || (p->M > 0 && (!x || !x_scales || !y)))    // (an empty tensor's address may be NULL)
        return fail(FDPP_ERR_INVALID_ARG, "x, w, their scales and y must be non-NULL");
    if (((uintptr_t)x | (uintptr_t)w) % 16 != 0) return fail(FDPP_ERR_INVALID_ARG, "x and w must be 16-byte aligned");
    if (((uintptr_t)x_scales | (uintptr_t)w_scales) % 4 != 0) return fail(FDPP_ERR_INVALID_ARG, "scales must be 4-byte aligned");
    if ((uintptr_t)y % (p->out_dtype == FDPP_F32 ? 4 : 2) != 0) return fail(FDPP_ERR_INVALID_ARG, "y must be aligned to its elements");
    if (!workspace) return fail(FDPP_ERR_WORKSPACE, "workspace is NULL");
    if ((uintptr_t)workspace % 256 != 0) return fail(FDPP_ERR_WORKSPACE, "workspace must be 256-byte aligned");
    if (workspace_bytes < 256) return fail(FDPP_ERR_WORKSPACE, "workspace has %zu bytes, 256 needed", workspace_bytes);
    int sms = 0, smem_sm = 0, smem_blk = 0;
    if ((st = query_device(&sms, &smem_sm, &smem_blk)) != FDPP_OK) return st;
    if (p->M == 0) return FDPP_OK;

    ScaledArgs g{};
    g.sx = x_scales;
    g.sw = w_scales;
    g.y = y;
    g.err = static_cast<unsigned*>(workspace);
    g.y_stride = p->y_stride;
    g.sx_stride = p->x_scale_stride;
    g.M = p->M;
    g.N = p->N;
    g.kb = blocks_of(p->K);
    cudaStream_t s = (cudaStream_t)stream;
    // Few rows: the rows kernel pads them least, and two of its CTAs share an SM. us a call at 64 rows, rows kernel against
    // tile kernel: 2048 x 2048 6.7 and 7.1, 6144 x 4096 9.9 and 11.2, 8192 x 8192 14.4 and 15.5, 28672 x 4096 22.3 and 31.6;
    // but 4096 x 4096 8.9 and 8.4, 4096 x 14336 14.2 and 13.6.
    if (p->M <= SG_GROUP) return launch_rows(*p, g, x, w, sms, smem_sm, smem_blk, s);
    // Tiles of 128 x 128 (whose sums join soonest where K is split) while each SM has one at most and K is short, then of
    // 128 x 256, for which less is read; pairs of CTAs on 256 x 256 where those would be more than one for an SM too, unless
    // the pairs' larger tiles take more turns. us a call in a graph, 128 x 128, 128 x 256 (four buffers of sums become two) and
    // pairs: 512 x 4096 x 4096 14.2, 16.6, 16.2; 512 x 4096 x 8192 24.7, 22.5, 27.1; 512 x 4096 x 14336 40.0, 31.3, 43.2;
    // 640 x 4096 x 14336 76.0, 44.9, 43.7; 1000 x 4096 x 4096 25.4, 16.9, 17.0; 1100 x 4096 x 4096 25.4, 17.0, 29.3;
    // 256 x 14336 x 4096 25.4, 19.0, 17.7; 128 x 28672 x 4096 28.4, 25.4, 32.3; 256 x 28672 x 4096 37.0, 35.8, 33.3;
    // 128 x 128256 x 4096 92.3, 96.2, 106.2; 2048 x 14336 x 4096 141, 88.1, 85.0. With one 128 x 256 tile for an SM
    // at most, pairs take 3 to 7 % less where they are full (640 and 256 rows), and 20 to 38 % more where the single tiles split K.
    const long long m_tiles = (p->M + 127ll) / 128, tiles = m_tiles * ((p->N + 127ll) / 128);
    const long long wide_tiles = m_tiles * ((p->N + 255ll) / 256), pair_tiles = (m_tiles + 1) / 2 * ((p->N + 255ll) / 256);
    const bool pairs = wide_tiles > sms && (pair_tiles - 1) / std::max(1, sms / 2) <= (wide_tiles - 1) / sms;
    const bool wide = tiles > sms || (2 * tiles > sms && g.kb >= 64);
    auto launch = [&](auto type) {
        using T = decltype(type);
        return pairs ? launch_tile<T, 256, true>(*p, g, x, w, sms, smem_blk, s)
               : wide ? launch_tile<T, 256, false>(*p, g, x, w, sms, smem_blk, s)
                      : launch_tile<T, 128, false>(*p, g, x, w, sms, smem_blk, s);
    };
    return p->out_dtype == FDPP_F32 ? launch(float{}) : launch(__nv_bfloat16{});
} catch (...) {                          // (the cache of cluster counts allocates)
    return fail(FDPP_ERR_CUDA, "out of host memory");
}

}  // extern "C"
