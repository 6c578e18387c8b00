// rows_simt.cu -- rows attention on the CUDA cores: fp32 caches (which the tensor cores would round),
// and bf16 when asked for.
//
// One CTA of four warps takes one token, up to four heads of one kv head and one split of the keys
// that the token sees. Eight lanes share a key (each holds d / 8 of its elements for all four heads,
// so K and V are read once for the four), sixteen keys are in flight per CTA, and each eight-lane
// group keeps its own running max, sum and accumulator (the online softmax of every sixteenth key);
// they are joined in a fixed order at the end. With few rows the keys are split over CTAs, and the
// last CTA of a row to finish joins the splits, again in a fixed order. One CTA more checks the offsets
// and lengths of all sequences (in the others it would cost them latency). Bounded by latency on short
// contexts (one token on 256 keys, 4 heads of 64: 6.5 us, two dependent passes over L2) and by the L2's rate on
// long ones: the four-head chunks of a wide group, and the tokens of a prompt or behind a prefix, each read the
// keys again.
#include <cuda_bf16.h>

#include "rows_common.cuh"

namespace fdpp {
namespace {

constexpr int SW = 4;                  // warps per CTA
constexpr int SH = ROWS_SIMT_HEADS;    // heads per CTA
constexpr int LANES = 8;               // lanes per key
constexpr int GROUPS = SW * 32 / LANES;

template <typename T, int N>
__device__ __forceinline__ void load_vec(const T* p, float (&x)[N]);

template <>
__device__ __forceinline__ void load_vec<float, 4>(const float* p, float (&x)[4])
{
    const float4 v = *reinterpret_cast<const float4*>(p);
    x[0] = v.x; x[1] = v.y; x[2] = v.z; x[3] = v.w;
}

template <>
__device__ __forceinline__ void load_vec<__nv_bfloat16, 4>(const __nv_bfloat16* p, float (&x)[4])
{
    const uint2 v = *reinterpret_cast<const uint2*>(p);
    x[0] = __uint_as_float(v.x << 16); x[1] = __uint_as_float(v.x & 0xffff0000u);
    x[2] = __uint_as_float(v.y << 16); x[3] = __uint_as_float(v.y & 0xffff0000u);
}

__device__ __forceinline__ void store_one(float* p, float x) { *p = x; }
__device__ __forceinline__ void store_one(__nv_bfloat16* p, float x) { *p = __float2bfloat16_rn(x); }

// Weight of a partial with max m in the frame M (M = -inf: no key yet).
__device__ __forceinline__ float join_weight(float m, float M) { return m == M ? 1.f : ex2(m - M); }

template <typename T, int D, bool TREE>
__global__ void __launch_bounds__(SW * 32) rows_simt_kernel(RowsArgs a)
{
    constexpr int NV = D / (LANES * 4);        // 4-element pieces per lane
    constexpr int E = NV * 4;
    __shared__ float sm_m[GROUPS][SH], sm_l[GROUPS][SH];
    __shared__ float sm_o[SW][SH][D];
    __shared__ float sm_w[SH][ROWS_SIMT_MAX_SPLITS];
    __shared__ int last;
    __shared__ int up[TREE ? FDPP_TREE_MAX_TOKENS : 1];
    __shared__ uint32_t seen[LINE_BITS];       // with trees: the token itself and its ancestors
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, grp = threadIdx.x / LANES, j = lane % LANES;
    const int chunks = (a.G + SH - 1) / SH;
    grid_dependency_wait();
    if (blockIdx.x == gridDim.x - 1) {           // looks at all offsets and lengths, those without rows too
        unsigned bad = 0;
        if (blockIdx.y == 0) {
            prefix_keys(a, bad);
            for (int b = threadIdx.x; b < a.B; b += SW * 32) {
                int c0;
                seq_rows(a, b, c0, bad);
                own_len(a, b, bad);
            }
        }
        rows_error(a, bad);
        return;
    }
    long long unit = blockIdx.x;
    const int chunk = (int)(unit % chunks);
    unit /= chunks;
    const int g = (int)(unit % a.Hkv), row = (int)(unit / a.Hkv), split = blockIdx.y;
    const int h0 = g * a.G + chunk * SH, nh = min(SH, a.G - chunk * SH);

    // the row's sequence: the last one that starts at or before it and has rows
    unsigned bad = 0;                            // (reported by the last CTA)
    int b = 0, c0 = 0, n = 0;
    if (a.cu) {
        int lo = 0, hi = a.B;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (a.cu[mid] <= row) lo = mid; else hi = mid;
        }
        b = lo;
    } else {
        b = row / a.per_seq;
    }
    n = seq_rows(a, b, c0, bad);
    if (row < c0 || row >= c0 + n) return;       // a row of no sequence: left as it was
    const int P = prefix_keys(a, bad), L = own_len(a, b, bad);
    const int pos = P + L - n + (row - c0);
    int lo, hi;
    row_keys(a, row, pos, P + L, lo, hi);
    const int tree0 = L - n;
    if (TREE) {
        // the token's walk up to the root, through shared memory (each CTA its own: a launch that does it for all
        // tokens before takes longer)
        const bool large = tree_too_large(a, n);
        if (large) lo = hi = 0;
        unsigned wrong = large ? FDPP_ERRBIT_TREE : 0;
        for (int i = threadIdx.x; i < n && !large; i += SW * 32) {
            const int p = a.parents[c0 + i];
            const bool ok = p >= -1 && p < i;
            up[i] = ok ? p : -1;
            if (!ok && i == row - c0) wrong = FDPP_ERRBIT_TREE;
        }
        if (threadIdx.x < LINE_BITS) seen[threadIdx.x] = 0u;
        rows_error(a, wrong);
        __syncthreads();
        if (threadIdx.x == 0 && !large)
            for (int i = row - c0; i >= 0; i = up[i]) seen[i >> 5] |= 1u << (i & 31);
        __syncthreads();
    }
    const int len = hi - lo;
    const int k0 = lo + (int)((long long)len * split / a.splits), k1 = lo + (int)((long long)len * (split + 1) / a.splits);

    const T* q = static_cast<const T*>(a.q) + ((long long)row * a.Hq + h0) * D;
    float qr[SH][E], o[SH][E], m[SH], l[SH], slope[SH];
#pragma unroll
    for (int h = 0; h < SH; ++h) {
        m[h] = -INFINITY;
        l[h] = 0.f;
        slope[h] = a.slopes && h < nh ? a.slopes[h0 + h] * LOG2E : 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            float x[4] = {0.f, 0.f, 0.f, 0.f};
            if (h < nh) load_vec<T, 4>(q + h * D + (i * LANES + j) * 4, x);
#pragma unroll
            for (int e = 0; e < 4; ++e) { qr[h][4 * i + e] = x[e]; o[h][4 * i + e] = 0.f; }
        }
    }
    const float cap_rate = a.cap > 0.f ? a.scale / a.cap : 0.f;
    const unsigned gmask = 0xffu << (lane & ~(LANES - 1));
    unsigned bad_block = 0;

#pragma unroll 2
    for (int t = k0 + grp; t < k1; t += GROUPS) {
        if (TREE && t >= tree0 && !(seen[(t - tree0) >> 5] >> ((t - tree0) & 31) & 1u)) continue;
        const bool pre = t < P;
        const long long off = key_offset(a, pre ? -1 : b, pre ? t : t - P, g);
        if (off < 0) {
            bad_block = FDPP_ERRBIT_BLOCK_TABLE;
            continue;
        }
        const T* kp = static_cast<const T*>(pre && a.pk ? a.pk : a.k) + off;
        const T* vp = static_cast<const T*>(pre && a.pv ? a.pv : a.v) + off;
        float kx[E], vx[E], s[SH];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            float x[4], y[4];
            load_vec<T, 4>(kp + (i * LANES + j) * 4, x);
            load_vec<T, 4>(vp + (i * LANES + j) * 4, y);
#pragma unroll
            for (int e = 0; e < 4; ++e) { kx[4 * i + e] = x[e]; vx[4 * i + e] = y[e]; }
        }
#pragma unroll
        for (int h = 0; h < SH; ++h) {
            float acc = 0.f;
#pragma unroll
            for (int e = 0; e < E; ++e) acc = fmaf(qr[h][e], kx[e], acc);
#pragma unroll
            for (int x = LANES / 2; x > 0; x >>= 1) acc += __shfl_xor_sync(gmask, acc, x);
            s[h] = acc;
        }
        // fp32 results need tanh to fp32's accuracy (1 - 2 / (e^2x + 1) is a few 2^-23 of the cap off: with a
        // cap of 50 ten times the error of the rest). All eight lanes hold all scores: each takes one head's.
        if (a.cap > 0.f) {
            float x = s[0];
#pragma unroll
            for (int h = 1; h < SH; ++h)
                if (j % SH == h) x = s[h];
            x = a.cap * tanhf(x * cap_rate);
#pragma unroll
            for (int h = 0; h < SH; ++h) s[h] = __shfl_sync(gmask, x, h, LANES);
        }
#pragma unroll
        for (int h = 0; h < SH; ++h)
            s[h] = fmaf(-slope[h], fabsf((float)(t - pos)), s[h] * (a.cap > 0.f ? LOG2E : a.scale * LOG2E));
#pragma unroll
        for (int h = 0; h < SH; ++h) {
            if (s[h] > m[h]) {
                const float w = ex2(m[h] - s[h]);
                l[h] *= w;
#pragma unroll
                for (int e = 0; e < E; ++e) o[h][e] *= w;
                m[h] = s[h];
            }
            // a score of -inf before any other: exp(-inf - M) is 0 for every finite M
            const float p = s[h] == -INFINITY ? 0.f : ex2(s[h] - m[h]);
            l[h] += p;
#pragma unroll
            for (int e = 0; e < E; ++e) o[h][e] = fmaf(p, vx[e], o[h][e]);
        }
    }
    // a bad block is known to the groups that came by it alone
    if (j == 0) rows_error(a, bad_block);
    __syncwarp();

    // join the groups: all of a head's maxima first, then sums in the common frame
    if (j == 0) {
#pragma unroll
        for (int h = 0; h < SH; ++h) { sm_m[grp][h] = m[h]; sm_l[grp][h] = l[h]; }
    }
    __syncthreads();
#pragma unroll
    for (int h = 0; h < SH; ++h) {
        float M = -INFINITY;
#pragma unroll
        for (int x = 0; x < GROUPS; ++x) M = fmaxf(M, sm_m[x][h]);
        const float w = join_weight(m[h], M);
#pragma unroll
        for (int e = 0; e < E; ++e) {
            float x = o[h][e] * w;
            x += __shfl_xor_sync(0xffffffffu, x, 8);
            x += __shfl_xor_sync(0xffffffffu, x, 16);
            o[h][e] = x;
        }
        m[h] = M;
        float lt = 0.f;
        for (int x = 0; x < GROUPS; ++x) lt += sm_l[x][h] * join_weight(sm_m[x][h], M);
        l[h] = lt;
        if (lane < LANES) {
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) sm_o[warp][h][(i * LANES + j) * 4 + e] = o[h][4 * i + e];
        }
    }
    __syncthreads();
    T* out = static_cast<T*>(a.out) + ((long long)row * a.Hq + h0) * D;
    const long long slot0 = ((long long)row * a.Hq + h0) * a.splits;
#pragma unroll
    for (int h = 0; h < SH; ++h) {
        if (h >= nh) break;
        for (int d = threadIdx.x; d < D; d += SW * 32) {
            float x = 0.f;
#pragma unroll
            for (int w = 0; w < SW; ++w) x += sm_o[w][h][d];
            if (a.splits == 1) store_one(out + h * D + d, len == 0 ? 0.f : x / l[h]);
            else a.row_o[(slot0 + h * a.splits + split) * D + d] = x;
        }
        if (a.splits > 1 && threadIdx.x == 0) a.row_ml[slot0 + h * a.splits + split] = make_float2(m[h], l[h]);
    }
    if (a.splits == 1) return;

    // the last CTA of the row joins its splits
    __threadfence();
    __syncthreads();
    if (threadIdx.x == 0) {
        const int done = atom_add_acq_rel_gpu(a.counters + blockIdx.x, 1);
        last = done == a.splits - 1;
        if (last) a.counters[blockIdx.x] = 0;
    }
    __syncthreads();
    if (!last) return;
    __threadfence();
    // a warp per head: the splits' maxima and sums over its lanes, their weights into shared memory
    if (warp < nh) {
        const float2* ml = a.row_ml + slot0 + warp * a.splits;
        float2 x[ROWS_SIMT_MAX_SPLITS / 32];
        float M = -INFINITY, lt = 0.f;
#pragma unroll
        for (int i = 0; i < ROWS_SIMT_MAX_SPLITS / 32; ++i) {
            x[i] = lane + 32 * i < a.splits ? __ldcg(ml + lane + 32 * i) : make_float2(-INFINITY, 0.f);
            M = fmaxf(M, x[i].x);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
#pragma unroll
        for (int i = 0; i < ROWS_SIMT_MAX_SPLITS / 32; ++i) {
            const float w = join_weight(x[i].x, M);
            if (lane + 32 * i < a.splits) {
                sm_w[warp][lane + 32 * i] = w;
                lt += x[i].y * w;
            }
        }
        lt = warp_sum(lt);
        if (lane == 0) sm_l[0][warp] = lt;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < nh * D; i += SW * 32) {
        const int h = i / D, d = i - h * D;
        const float* po = a.row_o + (slot0 + h * a.splits) * D + d;
        float x = 0.f;
#pragma unroll 8
        for (int s = 0; s < a.splits; ++s) x += __ldcg(po + (long long)s * D) * sm_w[h][s];
        store_one(out + i, len == 0 ? 0.f : x / sm_l[0][h]);
    }
}

}  // namespace

cudaError_t launch_rows_simt(const RowsArgs& a, int dtype, cudaStream_t s)
{
    void (*kern)(RowsArgs);
    if (a.parents)
        kern = dtype == FDPP_F32 ? (a.D == 128 ? rows_simt_kernel<float, 128, true> : rows_simt_kernel<float, 64, true>)
                                 : (a.D == 128 ? rows_simt_kernel<__nv_bfloat16, 128, true>
                                               : rows_simt_kernel<__nv_bfloat16, 64, true>);
    else
        kern = dtype == FDPP_F32 ? (a.D == 128 ? rows_simt_kernel<float, 128, false> : rows_simt_kernel<float, 64, false>)
                                 : (a.D == 128 ? rows_simt_kernel<__nv_bfloat16, 128, false>
                                               : rows_simt_kernel<__nv_bfloat16, 64, false>);
    const int chunks = (a.G + ROWS_SIMT_HEADS - 1) / ROWS_SIMT_HEADS;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((long long)a.T * a.Hkv * chunks + 1), (unsigned)a.splits);      // (the last one checks)
    cfg.blockDim = dim3(SW * 32);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, a);
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace fdpp
