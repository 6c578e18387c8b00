// norm.cu -- RMS norm with the residual's addition (fdpp_linear.h), output in the input's type or in
// e4m3 with a scale for every 128 channels.
//
//     r = x + residual,  y = r (mean(r^2) + eps)^(-1/2) w,  scale_g = max |y| of block g / 448
//
// A row is read once and stays in registers: each thread holds V vectors of 8 channels, thread i of the
// row's R takes vectors i, i + R, .. so that a warp reads whole lines, and the 16 lanes of a half warp hold
// a block of 128 channels, whose largest |y| takes four exchanges. The sum of squares is the only thing
// that the row's threads have to wait for; the row after is on its way meanwhile.
//
// What bounds it: HBM. 16384 rows of 8192 bf16 channels with a residual, its sum written back and the output in e4m3:
// 145 us, 6.47 TB/s, 0.97 of a measured copy (a CTA for each row, without the row ahead: 209). One row of 4096: the
// launch (2.2 us in a graph).
#include <algorithm>
#include <cmath>

#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include "device_common.cuh"
#include "fdpp_linear.h"

namespace fdpp {
namespace {

constexpr float E4M3_MAX = 448.f;
constexpr float LEAST_SCALE = 1.17549435e-38f;       // 2^-126: its reciprocal is finite
// With an epsilon below EPS_SMALL a row's mean square may come from squares that fp32 does not hold: below 2^-126 they lose
// bits, at most 2^-150 each, which shows where mean and epsilon stay below 2^-100. Such a row (of values below 2^-42) is
// taken times 2^100: then its values lie in 2^-49 .. 2^58.
constexpr float EPS_SMALL = 7.8886091e-31f, SMALL_ROWS = 1.2676506e30f;      // 2^-100, 2^100
constexpr int NORM_THREADS = 512, NORM_MAX_THREADS = 1024;     // of a CTA
constexpr int NORM_RESIDENT = 2048;                  // threads of the grid for an SM: all at once with 32 registers, in two turns with 64
constexpr int NORM_WARP_ROWS = 8;                    // rows of a CTA where each is one warp's

struct NormArgs {
    const void* x;
    const void* residual;
    const void* weight;
    void* out;
    float* scales;
    void* sum_out;
    long long x_stride, residual_stride, out_stride, sum_stride, scale_stride;
    int T, dim;
    float eps, offset;
};

// Eight consecutive elements as they lie in memory, as fp32, and back.
template <typename T>
struct Raw8;

template <>
struct Raw8<float> {
    float4 a, b;
    __device__ __forceinline__ void load(const float* p)
    {
        a = __ldcs(reinterpret_cast<const float4*>(p));
        b = __ldcs(reinterpret_cast<const float4*>(p) + 1);
    }
    __device__ __forceinline__ void keep(const float* p)
    {
        a = __ldg(reinterpret_cast<const float4*>(p));
        b = __ldg(reinterpret_cast<const float4*>(p) + 1);
    }
    __device__ __forceinline__ void get(float (&v)[8]) const
    {
        v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
        v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    }
};

template <>
struct Raw8<__nv_bfloat16> {
    uint4 a;
    __device__ __forceinline__ void load(const __nv_bfloat16* p) { a = __ldcs(reinterpret_cast<const uint4*>(p)); }
    __device__ __forceinline__ void keep(const __nv_bfloat16* p) { a = __ldg(reinterpret_cast<const uint4*>(p)); }
    __device__ __forceinline__ void get(float (&v)[8]) const
    {
        const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = __uint_as_float(w[i] << 16);
            v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
};

__device__ __forceinline__ void store8(float* p, const float (&v)[8])
{
    reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}

__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&v)[8])
{
    *reinterpret_cast<uint4*>(p) =
        make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
}

__device__ __forceinline__ uint32_t pack_e4m3x4(float a, float b, float c, float d)
{
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
    return lo | (hi << 16);
}

__device__ __forceinline__ float max_nan(float a, float b)
{
    float d;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
    return d;
}

// WARP: a row is one warp's, NORM_WARP_ROWS rows to a CTA; otherwise a row is the CTA's, and the next one is loaded
// while this one is added up and written.
// SMALL: for an epsilon below EPS_SMALL, with a second sum of squares. (A build of its own: the second sum behind a flag
// of the call took single rows 0 to 8 % longer and many rows of 128 channels up to 13 %; rows summed again behind a branch
// up to 62 %, 65536 fp32 rows of 1024 into e4m3 138 to 224 us.)
template <typename T, bool E4M3, int V, bool WARP, bool SMALL, int MOST = WARP ? 32 * NORM_WARP_ROWS : NORM_THREADS>
__global__ void __launch_bounds__(MOST)
    rms_norm_kernel(const __grid_constant__ NormArgs a)
{
    __shared__ float part[2][SMALL ? 64 : 32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int R = WARP ? 32 : blockDim.x, me = WARP ? lane : threadIdx.x;
    const long long step = WARP ? (long long)gridDim.x * NORM_WARP_ROWS : gridDim.x;
    long long t = WARP ? (long long)blockIdx.x * NORM_WARP_ROWS + warp : blockIdx.x;
    grid_dependency_wait();
    grid_launch_dependents();
    const int vectors = a.dim / 8;
    // (four vectors a thread: as many registers as there are, without a row ahead)
    constexpr bool AHEAD = V < 4 || WARP;
    const T* w = static_cast<const T*>(a.weight);
    Raw8<T> x[V], res[V], g[V];
    auto load = [&](long long row) {
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (me + i * R < vectors) {
                x[i].load(static_cast<const T*>(a.x) + row * a.x_stride + (me + i * R) * 8);
                if (a.residual) res[i].load(static_cast<const T*>(a.residual) + row * a.residual_stride + (me + i * R) * 8);
            }
    };
    if (AHEAD && t < a.T) load(t);
    if (AHEAD && w)
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (me + i * R < vectors) g[i].keep(w + (me + i * R) * 8);
    for (int turn = 0; t < a.T; t += step, turn ^= 1) {
        if (!AHEAD) load(t);
        float r[V][8];
        float sum = 0.f, times = 0.f;
#pragma unroll
        for (int i = 0; i < V; ++i) {
#pragma unroll
            for (int k = 0; k < 8; ++k) r[i][k] = 0.f;
            if (me + i * R < vectors) {
                x[i].get(r[i]);
                if (a.residual) {
                    float s[8];
                    res[i].get(s);
#pragma unroll
                    for (int k = 0; k < 8; ++k) r[i][k] += s[k];
                }
            }
#pragma unroll
            for (int k = 0; k < 8; ++k) sum = fmaf(r[i][k], r[i][k], sum);
            if constexpr (SMALL)
#pragma unroll
                for (int k = 0; k < 8; ++k) times = fmaf(r[i][k] * SMALL_ROWS, r[i][k] * SMALL_ROWS, times);
        }
        if (AHEAD && t + step < a.T) load(t + step);
        sum = warp_sum(sum);
        if constexpr (SMALL) times = warp_sum(times);
        if (!WARP) {
            if (lane == 0) {
                part[turn][warp] = sum;
                if constexpr (SMALL) part[turn][32 + warp] = times;
            }
            __syncthreads();                             // (the other half is read before the next barrier)
            sum = lane < (R >> 5) ? part[turn][lane] : 0.f;
            sum = warp_sum(sum);
            if constexpr (SMALL) times = warp_sum(lane < (R >> 5) ? part[turn][32 + lane] : 0.f);
        }
        float mean = sum / (float)a.dim + a.eps, f = 1.f;
        if (SMALL && mean < EPS_SMALL) {
            f = SMALL_ROWS;
            mean = times / (float)a.dim + f * a.eps * f;
        }
        const float inv = 1.f / sqrtf(mean);
        if (a.sum_out) {
            T* so = static_cast<T*>(a.sum_out) + t * a.sum_stride;
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (me + i * R < vectors) store8(so + (me + i * R) * 8, r[i]);
        }
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int at = me + i * R;
            const bool in = at < vectors;
            float y[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) y[k] = (SMALL ? r[i][k] * f : r[i][k]) * inv;
            if (w && in) {
                float gain[8];
                if (!AHEAD) g[i].keep(w + at * 8);
                g[i].get(gain);
#pragma unroll
                for (int k = 0; k < 8; ++k) y[k] *= gain[k] + a.offset;
            }
            if constexpr (!E4M3) {
                if (in) store8(static_cast<T*>(a.out) + t * a.out_stride + at * 8, y);
            } else {
                // a block's 16 lanes (those past the row hold zeros)
                float top = 0.f;
#pragma unroll
                for (int k = 0; k < 8; ++k) top = max_nan(top, fabsf(y[k]));
#pragma unroll
                for (int o = 8; o > 0; o >>= 1) top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, o));
                const float scale = max_nan(top / E4M3_MAX, LEAST_SCALE), over = 1.f / scale;
                if (in) {
                    uint2 v;
                    v.x = pack_e4m3x4(y[0] * over, y[1] * over, y[2] * over, y[3] * over);
                    v.y = pack_e4m3x4(y[4] * over, y[5] * over, y[6] * over, y[7] * over);
                    *reinterpret_cast<uint2*>(static_cast<uint8_t*>(a.out) + t * a.out_stride + at * 8) = v;
                    if ((at & 15) == 0) a.scales[t * a.scale_stride + (at >> 4)] = scale;
                }
            }
        }
    }
}

template <typename T, bool E4M3, bool SMALL>
cudaError_t launch_norm(const NormArgs& a, int sms, cudaStream_t s)
{
    const int vectors = a.dim / 8;
    void (*kern)(NormArgs);
    unsigned grid, threads;
    if (vectors <= 128) {
        kern = vectors <= 32   ? rms_norm_kernel<T, E4M3, 1, true, SMALL>
               : vectors <= 64 ? rms_norm_kernel<T, E4M3, 2, true, SMALL>
                               : rms_norm_kernel<T, E4M3, 4, true, SMALL>;
        grid = (unsigned)std::min((a.T - 1) / NORM_WARP_ROWS + 1, 8 * sms);
        threads = 32 * NORM_WARP_ROWS;
    } else {
        // Channels a thread holds, by what was fastest on 2^27 bf16 elements into e4m3: rows of 4096 in 512 threads of 8
        // channels 79 us, in 256 of 16 75; of 8192 in 512 of 16 145, in 1024 of 8 159, in 256 of 32 235; of 16384 in 1024
        // of 16 144, of 32 253.
        const int v = vectors <= 256 ? 1 : vectors <= 2 * NORM_MAX_THREADS ? 2 : 4;
        kern = v == 1                         ? rms_norm_kernel<T, E4M3, 1, false, SMALL>
               : vectors <= 2 * NORM_THREADS  ? rms_norm_kernel<T, E4M3, 2, false, SMALL>
               : v == 2                       ? rms_norm_kernel<T, E4M3, 2, false, SMALL, NORM_MAX_THREADS>
                                              : rms_norm_kernel<T, E4M3, 4, false, SMALL, NORM_MAX_THREADS>;
        threads = (unsigned)((vectors + v - 1) / v + 31) / 32 * 32;
        grid = (unsigned)std::min(a.T, std::max(1, NORM_RESIDENT / (int)threads) * sms);
    }
    return launch_pdl(kern, dim3(grid), (int)threads, s, a);
}

}  // namespace
}  // namespace fdpp

using namespace fdpp;

extern "C" fdpp_status fdpp_rms_norm(const void* x, const void* residual, const void* weight, const fdpp_norm_params* p,
                                     void* out, float* scales, void* sum_out, fdpp_stream stream)
{
    if (!p) return fail(FDPP_ERR_INVALID_ARG, "params is NULL");
    if (p->num_tokens < 0) return fail(FDPP_ERR_INVALID_ARG, "num_tokens must be >= 0 (got %d)", p->num_tokens);
    if (p->dim < 8 || p->dim % 8) return fail(FDPP_ERR_INVALID_ARG, "dim must be a positive multiple of 8 (got %d)", p->dim);
    if (p->dim > FDPP_NORM_MAX_DIM)
        return fail(FDPP_ERR_UNSUPPORTED, "dim %d > %d", p->dim, FDPP_NORM_MAX_DIM);
    if (p->dtype != FDPP_F32 && p->dtype != FDPP_BF16)
        return fail(FDPP_ERR_INVALID_ARG, "dtype must be FDPP_F32 or FDPP_BF16 (got %d)", p->dtype);
    const bool e4m3 = p->out_dtype == FDPP_E4M3;
    if (!e4m3 && p->out_dtype != p->dtype)
        return fail(FDPP_ERR_INVALID_ARG, "out_dtype must be dtype or FDPP_E4M3 (got %d)", p->out_dtype);
    if (!(p->eps >= 0.f) || !std::isfinite(p->eps)) return fail(FDPP_ERR_INVALID_ARG, "eps must be finite and >= 0");
    if (!std::isfinite(p->weight_offset)) return fail(FDPP_ERR_INVALID_ARG, "weight_offset must be finite");
    const long long vec = p->dtype == FDPP_F32 ? 4 : 8, out_vec = e4m3 ? 8 : vec, most = 1ll << 40;
    auto stride_ok = [&](long long stride, long long v) { return stride >= p->dim && stride % v == 0 && stride <= most; };
    if (!stride_ok(p->x_stride, vec) || !stride_ok(p->out_stride, out_vec) ||
        (residual && !stride_ok(p->residual_stride, vec)) || (sum_out && !stride_ok(p->sum_stride, vec)))
        return fail(FDPP_ERR_INVALID_ARG, "strides must cover a row and be multiples of 16 bytes (an e4m3 output's: of 8)");
    const bool some = p->num_tokens > 0;     // (an empty tensor's address may be NULL)
    if (some && (!x || !out)) return fail(FDPP_ERR_INVALID_ARG, "x and out must be non-NULL");
    if (((uintptr_t)x | (uintptr_t)residual | (uintptr_t)weight | (uintptr_t)out | (uintptr_t)sum_out) % 16 != 0)
        return fail(FDPP_ERR_INVALID_ARG, "x, residual, weight, out and sum_out must be 16-byte aligned");
    if (e4m3) {
        if ((some && !scales) || (uintptr_t)scales % 4 != 0)
            return fail(FDPP_ERR_INVALID_ARG, "an e4m3 output needs scales, 4-byte aligned");
        if (p->scale_stride < (p->dim + FDPP_SCALE_BLOCK - 1) / FDPP_SCALE_BLOCK || p->scale_stride > most)
            return fail(FDPP_ERR_INVALID_ARG, "scale_stride must cover a row's scales");
    } else if (scales) {
        return fail(FDPP_ERR_INVALID_ARG, "scales are of an e4m3 output only");
    }
    if (some &&
        ((out == x && (e4m3 || p->out_stride != p->x_stride)) || (sum_out && sum_out == x && p->sum_stride != p->x_stride) ||
         (sum_out && sum_out == residual && p->sum_stride != p->residual_stride) || out == residual || out == sum_out))
        return fail(FDPP_ERR_INVALID_ARG, "out may be x, and sum_out residual or x, where types and strides are the same");
    int sms = 0, unused = 0;
    const fdpp_status st = query_device(&sms, &unused, &unused);
    if (st != FDPP_OK) return st;
    if (p->num_tokens == 0) return FDPP_OK;

    NormArgs a{};
    a.x = x;
    a.residual = residual;
    a.weight = weight;
    a.out = out;
    a.scales = scales;
    a.sum_out = sum_out;
    a.x_stride = p->x_stride;
    a.residual_stride = p->residual_stride;
    a.out_stride = p->out_stride;
    a.sum_stride = p->sum_stride;
    a.scale_stride = p->scale_stride;
    a.T = p->num_tokens;
    a.dim = p->dim;
    a.eps = p->eps;
    a.offset = p->weight_offset;
    cudaStream_t s = (cudaStream_t)stream;
    auto launch = [&](auto type) {
        using T = decltype(type);
        if (a.eps < EPS_SMALL) return e4m3 ? launch_norm<T, true, true>(a, sms, s) : launch_norm<T, false, true>(a, sms, s);
        return e4m3 ? launch_norm<T, true, false>(a, sms, s) : launch_norm<T, false, false>(a, sms, s);
    };
    const cudaError_t e = p->dtype == FDPP_F32 ? launch(float{}) : launch(__nv_bfloat16{});
    if (e != cudaSuccess) return fail(FDPP_ERR_CUDA, "RMS norm launch: %s", cudaGetErrorString(e));
    return FDPP_OK;
}
