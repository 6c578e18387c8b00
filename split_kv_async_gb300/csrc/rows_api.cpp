// rows_api.cpp -- the C ABI of the rows attention (fdpp_rows.h): argument checks, workspace layout,
// kernel choice and tensor maps.
#include <algorithm>
#include <cmath>
#include <cstdarg>
#include <cstdio>

#include "rows_internal.h"

using namespace fdpp;

namespace {

fdpp_status rfail(fdpp_status s, const char* fmt, ...)
{
    char buf[512];
    va_list ap;
    va_start(ap, fmt);
    std::vsnprintf(buf, sizeof buf, fmt, ap);
    va_end(ap);
    set_last_error(buf);
    return s;
}

bool aligned(const void* p, size_t a) { return (uintptr_t)p % a == 0; }
size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

bool tensor_kernel(const fdpp_rows_params& p) { return p.dtype == FDPP_BF16 && p.kernel != FDPP_KERNEL_SIMT; }

// CTAs of the CUDA-core kernel without splits, and the splits a call of this shape uses: enough
// CTAs for about four on each of 152 SMs, but at least 32 keys for each.
long long simt_units(const fdpp_rows_params& p)
{
    const int G = p.num_q_heads / p.num_kv_heads;
    return (long long)p.num_tokens * p.num_kv_heads * ((G + ROWS_SIMT_HEADS - 1) / ROWS_SIMT_HEADS);
}

int simt_splits(const fdpp_rows_params& p)
{
    const long long units = simt_units(p), keys = (long long)p.max_seq_len + p.max_prefix_len;
    if (units >= ROWS_COUNTERS) return 1;
    const long long want = std::min<long long>((608 + units - 1) / units, keys / 32);
    return (int)std::max(1ll, std::min<long long>(want, ROWS_SIMT_MAX_SPLITS));
}

fdpp_status check_params(const fdpp_rows_params* p)
{
    if (!p) return rfail(FDPP_ERR_INVALID_ARG, "params is NULL");
    if (p->batch < 1) return rfail(FDPP_ERR_INVALID_ARG, "batch must be >= 1 (got %d)", p->batch);
    if (p->num_q_heads < 1 || p->num_kv_heads < 1) return rfail(FDPP_ERR_INVALID_ARG, "head counts must be >= 1");
    if (p->num_q_heads % p->num_kv_heads)
        return rfail(FDPP_ERR_INVALID_ARG, "num_q_heads (%d) is not a multiple of num_kv_heads (%d)", p->num_q_heads,
                     p->num_kv_heads);
    if (p->dtype != FDPP_F32 && p->dtype != FDPP_BF16)
        return rfail(FDPP_ERR_INVALID_ARG, "dtype must be FDPP_F32 or FDPP_BF16 (got %d)", p->dtype);
    if (p->head_dim != 64 && p->head_dim != 128)
        return rfail(FDPP_ERR_UNSUPPORTED, "head_dim %d: only 64 and 128 are built", p->head_dim);
    if (p->num_q_heads / p->num_kv_heads > FDPP_ROWS_MAX_GROUP)
        return rfail(FDPP_ERR_UNSUPPORTED, "%d query heads per kv head > %d", p->num_q_heads / p->num_kv_heads,
                     FDPP_ROWS_MAX_GROUP);
    if (p->num_tokens < 1) return rfail(FDPP_ERR_INVALID_ARG, "num_tokens must be >= 1");
    if (p->max_seq_len < 1) return rfail(FDPP_ERR_INVALID_ARG, "max_seq_len must be >= 1");
    if (p->max_prefix_len < 0) return rfail(FDPP_ERR_INVALID_ARG, "max_prefix_len must be >= 0");
    // (both are turned into units of log2: an infinite factor would make NaN of a score of 0)
    if (!std::isfinite(p->scale * 1.4426950f) || !(p->scale > 0.f))
        return rfail(FDPP_ERR_INVALID_ARG, "scale must be positive, and scale * log2(e) finite (got %g)", (double)p->scale);
    if (!std::isfinite(p->softcap * 1.4426950f) || p->softcap < 0.f)
        return rfail(FDPP_ERR_INVALID_ARG, "softcap must be 0 or positive, and softcap * log2(e) finite (got %g)", (double)p->softcap);
    // the tensor kernel's tanh is off by a few 2^-23 softcap: above this limit by more than its weights are
    if (tensor_kernel(*p) && p->softcap > FDPP_ROWS_MAX_SOFTCAP)
        return rfail(FDPP_ERR_UNSUPPORTED, "softcap %g > %g", (double)p->softcap, (double)FDPP_ROWS_MAX_SOFTCAP);
    if (p->softcap > 0.f && !std::isfinite(2.f * p->scale * 1.4426950f / p->softcap))
        return rfail(FDPP_ERR_INVALID_ARG, "scale / softcap overflows");
    if (p->kernel < FDPP_KERNEL_AUTO || p->kernel > FDPP_KERNEL_SIMT)
        return rfail(FDPP_ERR_INVALID_ARG, "unknown kernel %d", p->kernel);
    if (p->kernel == FDPP_KERNEL_TENSOR && p->dtype != FDPP_BF16)
        return rfail(FDPP_ERR_UNSUPPORTED, "tensor kernel needs bf16");
    if (!aligned(p->slopes, 4) || !aligned(p->key_begin, 4) || !aligned(p->key_end, 4))
        return rfail(FDPP_ERR_INVALID_ARG, "slopes, key_begin and key_end must be 4-byte aligned");
    // positions, key tiles and row counts stay within 32 bits
    const long long keys = (long long)p->max_seq_len + p->max_prefix_len;
    const int G = p->num_q_heads / p->num_kv_heads, tpt = ROWS_TILE / G;
    const long long rt = p->batch + 2ll * ((p->num_tokens + 2ll * tpt - 1) / (2 * tpt)) + 1;
    if (keys > (1ll << 30) || rt * p->num_kv_heads > (1ll << 31) / (keys / ROWS_KEYS + 8) ||
        (long long)p->num_tokens * p->num_q_heads >= (1ll << 31) / 2 || simt_units(*p) >= (1ll << 31) - 1)
        return rfail(FDPP_ERR_INVALID_ARG, "problem too large for one call");
    return FDPP_OK;
}

fdpp_status check_paged(const fdpp_rows_params* p)
{
    if (p->block_size < 16 || p->block_size > 256 || (p->block_size & (p->block_size - 1)))
        return rfail(FDPP_ERR_INVALID_ARG, "block_size must be a power of two in [16, 256] (got %d)", p->block_size);
    if (p->max_blocks_per_seq < 1) return rfail(FDPP_ERR_INVALID_ARG, "max_blocks_per_seq must be >= 1");
    if (p->num_kv_blocks < 1) return rfail(FDPP_ERR_INVALID_ARG, "num_kv_blocks must be >= 1");
    if ((long long)p->max_seq_len > (long long)p->max_blocks_per_seq * p->block_size)
        return rfail(FDPP_ERR_INVALID_ARG, "max_seq_len exceeds max_blocks_per_seq * block_size");
    return FDPP_OK;
}

// bf16 cache as {Hkv d, rows, outer} in boxes of 64 elements by up to 128 rows, 128-byte swizzle.
fdpp_status encode_cache(CUtensorMap* map, const void* base, const fdpp_rows_params& p, long long rows, long long outer,
                         int box_rows)
{
    PFN_cuTensorMapEncodeTiled_v12000 enc = nullptr;
    const fdpp_status st = get_tensor_map_encoder(&enc);
    if (st != FDPP_OK) return st;
    const cuuint64_t row = (cuuint64_t)p.num_kv_heads * p.head_dim;
    cuuint64_t dims[3] = {row, (cuuint64_t)rows, (cuuint64_t)outer};
    cuuint64_t strides[2] = {row * 2, row * 2 * (cuuint64_t)rows};
    cuuint32_t box[3] = {64, (cuuint32_t)box_rows, 1};
    cuuint32_t estr[3] = {1, 1, 1};
    const CUresult r = enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, estr,
                           CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                           CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) return rfail(FDPP_ERR_CUDA, "cuTensorMapEncodeTiled failed (%d)", (int)r);
    return FDPP_OK;
}

// q as {d, Hq, T}, box {64, G, tokens}: one load lands a row tile's rows (token i, head h of the kv
// head in row i G + h) as rows of 128 bytes, 128-byte swizzled.
fdpp_status encode_q(CUtensorMap* map, const void* q, const fdpp_rows_params& p, int tokens)
{
    PFN_cuTensorMapEncodeTiled_v12000 enc = nullptr;
    const fdpp_status st = get_tensor_map_encoder(&enc);
    if (st != FDPP_OK) return st;
    const cuuint64_t D = (cuuint64_t)p.head_dim, Hq = (cuuint64_t)p.num_q_heads;
    const int G = p.num_q_heads / p.num_kv_heads;
    cuuint64_t dims[3] = {D, Hq, (cuuint64_t)p.num_tokens};
    cuuint64_t strides[2] = {D * 2, Hq * D * 2};
    cuuint32_t box[3] = {64, (cuuint32_t)G, (cuuint32_t)tokens};
    cuuint32_t estr[3] = {1, 1, 1};
    const CUresult r = enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(q), dims, strides, box, estr,
                           CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
                           CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) return rfail(FDPP_ERR_CUDA, "cuTensorMapEncodeTiled (q) failed (%d)", (int)r);
    return FDPP_OK;
}

fdpp_status attend(const void* q, const void* prefix_k, const void* prefix_v, const int32_t* prefix_blocks,
                   const int32_t* prefix_len, bool prefix, const void* k_cache, const void* v_cache,
                   const int32_t* block_table, const int32_t* seq_lens, const int32_t* cu_tokens,
                   const fdpp_rows_params* p, void* workspace, size_t workspace_bytes, void* out, fdpp_stream stream)
{
    fdpp_status st = check_params(p);
    if (st != FDPP_OK) return st;
    const bool paged = block_table != nullptr;
    if (paged && (st = check_paged(p)) != FDPP_OK) return st;
    if (!q || !k_cache || !v_cache || !seq_lens || !out)
        return rfail(FDPP_ERR_INVALID_ARG, "q, k_cache, v_cache, seq_lens and out must be non-NULL");
    if (!aligned(q, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(out, 16))
        return rfail(FDPP_ERR_INVALID_ARG, "q, k_cache, v_cache and out must be 16-byte aligned");
    if (!aligned(seq_lens, 4) || !aligned(block_table, 4) || !aligned(cu_tokens, 4))
        return rfail(FDPP_ERR_INVALID_ARG, "seq_lens, block_table and cu_tokens must be 4-byte aligned");
    if (!cu_tokens && p->num_tokens % p->batch)
        return rfail(FDPP_ERR_INVALID_ARG, "without cu_tokens num_tokens (%d) must be a multiple of batch (%d)",
                     p->num_tokens, p->batch);
    if (prefix) {
        if (p->max_prefix_len < 1) return rfail(FDPP_ERR_INVALID_ARG, "max_prefix_len must be >= 1");
        if (!prefix_len || !aligned(prefix_len, 4))
            return rfail(FDPP_ERR_INVALID_ARG, "prefix_len must be non-NULL and 4-byte aligned");
        if (paged && (!prefix_blocks || prefix_k || prefix_v))
            return rfail(FDPP_ERR_INVALID_ARG, "paged caches take prefix_blocks, and no prefix_k or prefix_v");
        if (!paged && (!prefix_k || !prefix_v || prefix_blocks))
            return rfail(FDPP_ERR_INVALID_ARG, "contiguous caches take prefix_k and prefix_v, and no prefix_blocks");
        if (!aligned(prefix_k, 16) || !aligned(prefix_v, 16) || !aligned(prefix_blocks, 4))
            return rfail(FDPP_ERR_INVALID_ARG, "prefix_k and prefix_v must be 16-byte, prefix_blocks 4-byte aligned");
    }
    if (!workspace) return rfail(FDPP_ERR_WORKSPACE, "workspace is NULL");
    if (!aligned(workspace, 256)) return rfail(FDPP_ERR_WORKSPACE, "workspace must be 256-byte aligned");
    const RowsLayout w = rows_layout(*p);
    if (workspace_bytes < w.total)
        return rfail(FDPP_ERR_WORKSPACE, "workspace has %zu bytes, %zu needed", workspace_bytes, w.total);
    int sms = 0, smem_sm = 0, smem_blk = 0;
    if ((st = query_device(&sms, &smem_sm, &smem_blk)) != FDPP_OK) return st;

    uint8_t* ws = static_cast<uint8_t*>(workspace);
    RowsArgs a{};
    a.q = q;
    a.k = k_cache;
    a.v = v_cache;
    a.pk = prefix_k;
    a.pv = prefix_v;
    a.block_table = block_table;
    a.prefix_blocks = prefix_blocks;
    a.prefix_len = prefix ? prefix_len : nullptr;
    a.seq_lens = seq_lens;
    a.cu = cu_tokens;
    a.slopes = p->slopes;
    a.key_begin = p->key_begin;
    a.key_end = p->key_end;
    a.out = out;
    a.err = reinterpret_cast<unsigned*>(ws);
    a.counters = reinterpret_cast<int*>(ws + w.counters);
    a.plan = reinterpret_cast<int*>(ws + w.plan);
    a.tok = reinterpret_cast<RowToken*>(ws + w.tok);
    a.seq_rt = reinterpret_cast<int*>(ws + w.seq_rt);
    a.rec = reinterpret_cast<RowTileRec*>(ws + w.rec);
    a.slot_o = reinterpret_cast<float*>(ws + w.slot_o);
    a.slot_ml = reinterpret_cast<float2*>(ws + w.slot_ml);
    a.row_o = reinterpret_cast<float*>(ws + w.row_o);
    a.row_ml = reinterpret_cast<float2*>(ws + w.row_ml);
    a.B = p->batch;
    a.Hq = p->num_q_heads;
    a.Hkv = p->num_kv_heads;
    a.G = a.Hq / a.Hkv;
    a.D = p->head_dim;
    a.T = p->num_tokens;
    a.per_seq = p->num_tokens / p->batch;
    a.max_seq_len = p->max_seq_len;
    a.block_size = paged ? p->block_size : 0;
    a.max_blocks = paged ? p->max_blocks_per_seq : 0;
    a.num_blocks = paged ? p->num_kv_blocks : 0;
    a.max_prefix = prefix ? p->max_prefix_len : 0;
    a.tpt = ROWS_TILE / a.G;
    a.tpn = ROWS_NARROW / a.G;
    a.max_rt = w.max_rt;
    a.slot_rows = w.slot_rows;
    a.scale = p->scale;
    a.cap = p->softcap;

    cudaStream_t s = (cudaStream_t)stream;
    if (!tensor_kernel(*p)) {
        a.splits = simt_splits(*p);
        const cudaError_t e = launch_rows_simt(a, p->dtype, s);
        if (e != cudaSuccess) return rfail(FDPP_ERR_CUDA, "rows kernel launch: %s", cudaGetErrorString(e));
        return FDPP_OK;
    }
    a.parts = std::min(sms, ROWS_MAX_PARTS);
    a.stages = rows_tc_stages(a.D, std::min(smem_blk, smem_sm - 1024));
    if (a.stages < 4) return rfail(FDPP_ERR_UNSUPPORTED, "too little shared memory for the tensor kernel");
    const int box = paged ? std::min(p->block_size, ROWS_KEYS) : ROWS_KEYS;
    const long long rows = paged ? p->block_size : p->max_seq_len, outer = paged ? p->num_kv_blocks : p->batch;
    RowsMaps m;
    if ((st = encode_q(&m.q, q, *p, a.tpt)) != FDPP_OK) return st;
    if ((st = encode_q(&m.qn, q, *p, std::max(1, a.tpn))) != FDPP_OK) return st;
    if ((st = encode_cache(&m.k, k_cache, *p, rows, outer, box)) != FDPP_OK) return st;
    if ((st = encode_cache(&m.v, v_cache, *p, rows, outer, box)) != FDPP_OK) return st;
    m.pk = m.k;
    m.pv = m.v;
    if (prefix && !paged) {
        if ((st = encode_cache(&m.pk, prefix_k, *p, p->max_prefix_len, 1, ROWS_KEYS)) != FDPP_OK) return st;
        if ((st = encode_cache(&m.pv, prefix_v, *p, p->max_prefix_len, 1, ROWS_KEYS)) != FDPP_OK) return st;
    }
    const cudaError_t e = launch_rows_tc(a, m, s);
    if (e != cudaSuccess) return rfail(FDPP_ERR_CUDA, "rows kernel launch: %s", cudaGetErrorString(e));
    return FDPP_OK;
}

}  // namespace

namespace fdpp {

RowsLayout rows_layout(const fdpp_rows_params& p)
{
    RowsLayout w{};
    const size_t T = (size_t)p.num_tokens, Hq = (size_t)p.num_q_heads, D = (size_t)p.head_dim;
    const int G = p.num_q_heads / p.num_kv_heads, pair = 2 * (ROWS_TILE / G);
    w.counters = ROWS_OFF_COUNTERS;
    w.plan = ROWS_OFF_PLAN;
    size_t off = align256(w.plan + (RP_WORDS + ROWS_MAX_PARTS) * 4);
    if (!tensor_kernel(p)) {
        const size_t splits = (size_t)simt_splits(p), rows = splits > 1 ? T * Hq * splits : 0;
        w.tok = w.seq_rt = w.rec = w.slot_o = w.slot_ml = off;
        w.row_o = off;   off = align256(off + rows * D * 4);
        w.row_ml = off;  off = align256(off + rows * 8);
        w.total = off;
        return w;
    }
    // a pair of row tiles for every `pair` tokens, one more for each sequence that starts anew; the
    // prefix's row tiles besides
    const long long tiles = (p.num_tokens + pair - 1) / pair;
    w.max_rt = (int)(p.batch + tiles + (p.max_prefix_len > 0 ? tiles : 0));
    const size_t rows = T * G;
    w.slot_rows = (int)std::min<size_t>(ROWS_PAIR, rows);
    w.tok = off;      off = align256(off + T * sizeof(RowToken));
    w.seq_rt = off;   off = align256(off + ((size_t)p.batch + 1) * 4);
    w.rec = off;      off = align256(off + (size_t)w.max_rt * sizeof(RowTileRec));
    const size_t slots = 2 * (size_t)ROWS_MAX_PARTS * w.slot_rows;
    w.slot_o = off;   off = align256(off + slots * D * 4);
    w.slot_ml = off;  off = align256(off + slots * 8);
    const size_t whole = p.max_prefix_len > 0 ? 2 * T * Hq : 0;
    w.row_o = off;    off = align256(off + whole * D * 4);
    w.row_ml = off;   off = align256(off + whole * 8);
    w.total = off;
    return w;
}

}  // namespace fdpp

extern "C" {

fdpp_status fdpp_rows_workspace_size(const fdpp_rows_params* p, size_t* bytes)
{
    const fdpp_status st = check_params(p);
    if (st != FDPP_OK) return st;
    if (!bytes) return rfail(FDPP_ERR_INVALID_ARG, "bytes is NULL");
    *bytes = rows_layout(*p).total;
    return FDPP_OK;
}

fdpp_status fdpp_rows_attn(const void* q, const void* k_cache, const void* v_cache, const int32_t* block_table,
                           const int32_t* seq_lens, const int32_t* cu_tokens, const fdpp_rows_params* p, void* workspace,
                           size_t workspace_bytes, void* out, fdpp_stream stream)
{
    return attend(q, nullptr, nullptr, nullptr, nullptr, false, k_cache, v_cache, block_table, seq_lens, cu_tokens, p,
                  workspace, workspace_bytes, out, stream);
}

fdpp_status fdpp_prefix_attn(const void* q, const void* prefix_k, const void* prefix_v, const int32_t* prefix_blocks,
                             const int32_t* prefix_len, const void* k_cache, const void* v_cache,
                             const int32_t* block_table, const int32_t* seq_lens, const int32_t* cu_tokens,
                             const fdpp_rows_params* p, void* workspace, size_t workspace_bytes, void* out,
                             fdpp_stream stream)
{
    return attend(q, prefix_k, prefix_v, prefix_blocks, prefix_len, true, k_cache, v_cache, block_table, seq_lens,
                  cu_tokens, p, workspace, workspace_bytes, out, stream);
}

}  // extern "C"
