// tree.cu -- trees of drafted tokens (fdpp_tree.h): the tokens' lineage, which the rows attention's kernels mask
// by, and the commit of an accepted path.
#include <algorithm>

#include "rows_common.cuh"

namespace fdpp {
namespace {

constexpr int TREE = FDPP_TREE_MAX_TOKENS;

// ---- lineage ------------------------------------------------------------------------------
// A CTA per sequence, a thread per node: it walks up to the root through shared memory, sets a bit for each
// node that it passes, and its own bit with each of them.
//
// It lies on the stream behind the plan, which starts it as soon as what came before the plan has completed. So it
// does its work first, beside the plan (its reads go past the L1 cache), and then waits for the plan: the kernel
// behind it waits for it alone. It adds nothing to most calls then (as a launch of its own before the plan 2 to 3 us).
__global__ void __launch_bounds__(TREE) lineage_kernel(const __grid_constant__ RowsArgs a)
{
    __shared__ int up[TREE];
    constexpr int ROW = 1 + 2 * LINE_BITS;               // (an odd number of words: no two rows in one bank)
    __shared__ uint32_t line[TREE * ROW];                // the tree's first key, ancestors, descendants
    const int b = blockIdx.x, i = threadIdx.x;
    grid_launch_dependents();
    int c0 = b * a.per_seq, n = a.per_seq;
    if (a.cu) {
        c0 = clamp_len(__ldcg(a.cu + b), a.T);
        n = max(c0, clamp_len(__ldcg(a.cu + b + 1), a.T)) - c0;
    }
    const int L = clamp_len(__ldcg(a.seq_lens + b), a.max_seq_len);
    // (the attention's kernels report what is wrong with offsets and lengths)
    unsigned bad = n > TREE ? FDPP_ERRBIT_TREE : 0;
    if (n <= TREE) {
        if (i < n) {
            int p = __ldcg(a.parents + c0 + i);
            if (p < -1 || p >= i) {
                bad = FDPP_ERRBIT_TREE;
                p = -1;
            }
            up[i] = p;
        }
        for (int w = i; w < n * ROW; w += TREE) line[w] = w % ROW == 0 ? (uint32_t)(L - n) : 0u;
        __syncthreads();
        if (i < n)
            for (int j = i; j >= 0; j = up[j]) {
                line[i * ROW + 1 + (j >> 5)] |= 1u << (j & 31);
                atomicOr(&line[j * ROW + 1 + LINE_BITS + (i >> 5)], 1u << (i & 31));
            }
        __syncthreads();
        uint32_t* to = a.lineage + (long long)c0 * LINE_WORDS;
        for (int w = i; w < n * ROW; w += TREE) {
            const int row = w / ROW, k = w - row * ROW;
            to[row * LINE_WORDS + (k <= LINE_BITS ? k : k - 1 - LINE_BITS + LINE_DOWN)] = line[w];
        }
    }
    rows_error(a, bad);
    grid_dependency_wait();
}

// ---- commit -------------------------------------------------------------------------------
// A CTA takes a sequence and some of the 16-byte columns of all caches' rows. Each finds the path for itself (a
// few hundred cycles through shared memory, less than a launch that waits for another): a node whose token
// is its parent's choice enters itself as the parent's next one, the first such child winning, and one
// thread follows the path. A thread then moves its column's rows in the order of the path. Node p_k >= k goes
// to place k: a place that is written has been read by then, or is of no later node, so eight rows at a time
// are read before the first of them is written, and no thread waits for another.
constexpr int COMMIT_THREADS = 256;
constexpr int COMMIT_AT_ONCE = 8;
constexpr int COMMIT_RESIDENT = 8;       // CTAs of an SM (64 trees of 16 in 64 caches, us: eight 6.4, four 7.3, two 8.8)
static_assert(COMMIT_THREADS >= TREE, "a thread per node");

// N: most caches (a launch with 2 kB of arguments takes the host a microsecond longer than one with 300 bytes).
template <int N>
struct CommitArgs {
    const int32_t* parents;
    const int32_t* tokens;
    const int32_t* choices;
    const int32_t* seq_lens;
    const int32_t* cu;
    const int32_t* table;
    int32_t* new_lens;
    int32_t* accepted;
    int32_t* path;
    int32_t* chosen;
    unsigned* err;
    long long row_bytes;
    int T, per_seq, max_seq_len, block_size, max_blocks, num_blocks;
    int columns, caches;                 // 16-byte columns of a row
    void* cache[N];
};

template <int N>
__global__ void __launch_bounds__(COMMIT_THREADS) tree_commit_kernel(const __grid_constant__ CommitArgs<N> a)
{
    __shared__ int choice[TREE], next[TREE], path[TREE];
    __shared__ long long slot[TREE];                     // each node's row in the caches, -1: its block is not in the pool
    __shared__ long long from[TREE], to[TREE];           // byte offsets of the path's rows, -1: not moved
    __shared__ int taken, first_moved;
    const int b = blockIdx.y, i = threadIdx.x;
    const bool tells = blockIdx.x == 0;
    grid_dependency_wait();
    grid_launch_dependents();
    unsigned bad = 0;
    int c0 = b * a.per_seq, n = a.per_seq;
    if (a.cu) {
        const int x = a.cu[b], y = a.cu[b + 1];
        c0 = clamp_len(x, a.T);
        const int c1 = max(c0, clamp_len(y, a.T));
        if (x != c0 || y != c1) bad |= FDPP_ERRBIT_TOKENS;
        n = c1 - c0;
    }
    const int L = a.seq_lens[b];
    if (L < n || L > a.max_seq_len) bad |= FDPP_ERRBIT_SEQ_LEN;
    if (n > TREE) bad |= FDPP_ERRBIT_TREE;
    if (n == 0 || (bad & (FDPP_ERRBIT_SEQ_LEN | FDPP_ERRBIT_TREE))) {
        if (tells) {
            if (i == 0) {
                a.accepted[b] = 0;
                a.new_lens[b] = clamp_len(L, a.max_seq_len);
                if (bad) atomicOr(a.err, bad);
            }
            for (int k = i; k < n; k += COMMIT_THREADS) a.path[c0 + k] = a.chosen[c0 + k] = -1;
        }
        return;
    }
    const int base = L - n;
    int up = -1, token = 0;
    if (i < n) {
        up = a.parents[c0 + i];
        token = a.tokens[c0 + i];
        choice[i] = a.choices[c0 + i];
        next[i] = TREE;
        // all nodes' blocks, not only the path's, so that their reading does not wait for the path (the eight's 6.4 us
        // above became 6.0)
        const int pos = base + i;
        long long at = (long long)b * a.max_seq_len + pos;
        if (a.table) {
            const int j = pos / a.block_size, blk = a.table[(long long)b * a.max_blocks + j];
            at = blk >= 0 && blk < a.num_blocks ? (long long)blk * a.block_size + (pos - j * a.block_size) : -1;
        }
        slot[i] = at;
        if (up < -1 || up >= i) {
            bad |= FDPP_ERRBIT_TREE;
            up = -1;
        }
    }
    __syncthreads();
    if (up >= 0 && token == choice[up]) atomicMin(&next[up], i);
    __syncthreads();
    if (i == 0) {
        int count = 0, moved = TREE;
        for (int k = 0; k < n; k = next[k]) {            // (next is a later node, or TREE)
            if (moved == TREE && k != count) moved = count;
            path[count++] = k;
        }
        taken = count;
        first_moved = moved;
    }
    __syncthreads();
    const int count = taken, start = min(first_moved, count);
    if (i < count && i >= start) {
        const long long source = slot[path[i]], place = slot[i];
        if (source < 0 || place < 0) bad |= FDPP_ERRBIT_BLOCK_TABLE;
        from[i] = source >= 0 && place >= 0 ? source * a.row_bytes : -1;
        to[i] = place * a.row_bytes;
    }
    if (tells) {
        if (i == 0) {
            a.accepted[b] = count;
            a.new_lens[b] = base + count;
        }
        if (i < n) {
            a.path[c0 + i] = i < count ? path[i] : -1;
            a.chosen[c0 + i] = i < count ? choice[path[i]] : -1;
        }
        if (bad) atomicOr(a.err, bad);
    }
    __syncthreads();
    const long long items = (long long)a.caches * a.columns;
    for (long long item = (long long)blockIdx.x * COMMIT_THREADS + i; item < items; item += (long long)gridDim.x * COMMIT_THREADS) {
        const int c = (int)(item / a.columns);
        char* cache = static_cast<char*>(a.cache[c]) + (item - (long long)c * a.columns) * 16;
        for (int k0 = start; k0 < count; k0 += COMMIT_AT_ONCE) {
            uint4 v[COMMIT_AT_ONCE];
#pragma unroll
            for (int k = 0; k < COMMIT_AT_ONCE; ++k)
                if (k0 + k < count && from[k0 + k] >= 0) v[k] = *reinterpret_cast<const uint4*>(cache + from[k0 + k]);
#pragma unroll
            for (int k = 0; k < COMMIT_AT_ONCE; ++k)
                if (k0 + k < count && from[k0 + k] >= 0) *reinterpret_cast<uint4*>(cache + to[k0 + k]) = v[k];
        }
    }
}

fdpp_status check_params(const fdpp_commit_params* p)
{
    if (!p) return fail(FDPP_ERR_INVALID_ARG, "params is NULL");
    if (p->batch < 1 || p->batch > 65535) return fail(FDPP_ERR_INVALID_ARG, "batch must be in [1, 65535] (got %d)", p->batch);
    if (p->num_tokens < 0) return fail(FDPP_ERR_INVALID_ARG, "num_tokens must be >= 0 (got %d)", p->num_tokens);
    if (p->max_seq_len < 1) return fail(FDPP_ERR_INVALID_ARG, "max_seq_len must be >= 1");
    if (p->row_bytes < 16 || p->row_bytes % 16 || p->row_bytes > (1ll << 24))
        return fail(FDPP_ERR_INVALID_ARG, "row_bytes must be a positive multiple of 16, at most 2^24 (got %lld)", p->row_bytes);
    return FDPP_OK;
}

// Whether two of the pointers are the same one (they usually come in order).
bool repeated(void* const* p, int n)
{
    bool rising = true;
    for (int i = 1; i < n; ++i) rising = rising && (uintptr_t)p[i - 1] < (uintptr_t)p[i];
    if (rising) return false;
    uintptr_t v[FDPP_TREE_MAX_CACHES];
    for (int i = 0; i < n; ++i) v[i] = (uintptr_t)p[i];
    std::sort(v, v + n);
    return std::adjacent_find(v, v + n) != v + n;
}

}  // namespace

cudaError_t launch_lineage(const RowsArgs& a, cudaStream_t s)
{
    return launch_pdl(lineage_kernel, dim3((unsigned)a.B), TREE, s, a);
}

}  // namespace fdpp

using namespace fdpp;

extern "C" {

size_t fdpp_commit_workspace_size(const fdpp_commit_params* p) { return check_params(p) == FDPP_OK ? 256 : 0; }

fdpp_status fdpp_tree_commit(const int32_t* parents, const int32_t* tokens, const int32_t* choices, const int32_t* seq_lens,
                             const int32_t* cu_tokens, const int32_t* block_table, void* const* caches, int num_caches,
                             const fdpp_commit_params* p, void* workspace, size_t workspace_bytes, int32_t* new_lens,
                             int32_t* accepted, int32_t* path, int32_t* chosen, fdpp_stream stream)
{
    fdpp_status st = check_params(p);
    if (st != FDPP_OK) return st;
    if (!cu_tokens && p->num_tokens % p->batch)
        return fail(FDPP_ERR_INVALID_ARG, "without cu_tokens num_tokens (%d) must be a multiple of batch (%d)", p->num_tokens,
                     p->batch);
    if (block_table) {
        if (p->block_size < 16 || p->block_size > 256 || (p->block_size & (p->block_size - 1)))
            return fail(FDPP_ERR_INVALID_ARG, "block_size must be a power of two in [16, 256] (got %d)", p->block_size);
        if (p->max_blocks_per_seq < 1 || p->num_kv_blocks < 1)
            return fail(FDPP_ERR_INVALID_ARG, "max_blocks_per_seq and num_kv_blocks must be >= 1");
        if ((long long)p->max_seq_len > (long long)p->max_blocks_per_seq * p->block_size)
            return fail(FDPP_ERR_INVALID_ARG, "max_seq_len exceeds max_blocks_per_seq * block_size");
    }
    if (!seq_lens || !new_lens || !accepted) return fail(FDPP_ERR_INVALID_ARG, "seq_lens, new_lens and accepted must be non-NULL");
    if (p->num_tokens > 0 && (!parents || !tokens || !choices || !path || !chosen))
        return fail(FDPP_ERR_INVALID_ARG, "parents, tokens, choices, path and chosen must be non-NULL");
    if ((((uintptr_t)parents | (uintptr_t)tokens | (uintptr_t)choices | (uintptr_t)seq_lens | (uintptr_t)cu_tokens |
          (uintptr_t)block_table | (uintptr_t)new_lens | (uintptr_t)accepted | (uintptr_t)path | (uintptr_t)chosen) % 4) != 0)
        return fail(FDPP_ERR_INVALID_ARG, "int32 arrays must be 4-byte aligned");
    if (new_lens == seq_lens || accepted == seq_lens || new_lens == accepted)
        return fail(FDPP_ERR_INVALID_ARG, "seq_lens, new_lens and accepted must be different arrays");
    for (const int32_t* in : {parents, tokens, choices})
        if (in && (in == path || in == chosen)) return fail(FDPP_ERR_INVALID_ARG, "path and chosen must not be an input");
    if (path && path == chosen) return fail(FDPP_ERR_INVALID_ARG, "path and chosen must be different arrays");
    if (num_caches < 0 || num_caches > FDPP_TREE_MAX_CACHES || (num_caches > 0 && !caches))
        return fail(FDPP_ERR_INVALID_ARG, "num_caches %d outside 0 .. %d, or caches is NULL", num_caches, FDPP_TREE_MAX_CACHES);
    for (int i = 0; i < num_caches; ++i)
        if (!caches[i] || (uintptr_t)caches[i] % 16 != 0)
            return fail(FDPP_ERR_INVALID_ARG, "cache %d must be non-NULL and 16-byte aligned", i);
    if (repeated(caches, num_caches)) return fail(FDPP_ERR_INVALID_ARG, "a cache is given twice");
    if (!workspace) return fail(FDPP_ERR_WORKSPACE, "workspace is NULL");
    if ((uintptr_t)workspace % 256 != 0) return fail(FDPP_ERR_WORKSPACE, "workspace must be 256-byte aligned");
    if (workspace_bytes < 256) return fail(FDPP_ERR_WORKSPACE, "workspace has %zu bytes, 256 needed", workspace_bytes);
    int sms = 0, unused = 0;
    if ((st = query_device(&sms, &unused, &unused)) != FDPP_OK) return st;

    auto launch = [&](auto a) {
        a.parents = parents;
        a.tokens = tokens;
        a.choices = choices;
        a.seq_lens = seq_lens;
        a.cu = cu_tokens;
        a.table = block_table;
        a.new_lens = new_lens;
        a.accepted = accepted;
        a.path = path;
        a.chosen = chosen;
        a.err = static_cast<unsigned*>(workspace);
        a.row_bytes = p->row_bytes;
        a.T = p->num_tokens;
        a.per_seq = p->num_tokens / p->batch;
        a.max_seq_len = p->max_seq_len;
        a.block_size = p->block_size;
        a.max_blocks = p->max_blocks_per_seq;
        a.num_blocks = p->num_kv_blocks;
        a.columns = (int)(p->row_bytes / 16);
        a.caches = num_caches;
        for (int i = 0; i < num_caches; ++i) a.cache[i] = caches[i];
        // a CTA for every 256 columns, but no more than are on the GPU at once: each finds the path for itself
        const long long all = ((long long)num_caches * a.columns + COMMIT_THREADS - 1) / COMMIT_THREADS;
        const long long grid = std::max(1ll, std::min(all, (COMMIT_RESIDENT * (long long)sms + p->batch - 1) / p->batch));
        return launch_pdl(tree_commit_kernel<sizeof a.cache / sizeof(void*)>, dim3((unsigned)grid, (unsigned)p->batch),
                          COMMIT_THREADS, (cudaStream_t)stream, a);
    };
    const cudaError_t e = num_caches <= 16   ? launch(CommitArgs<16>{})
                          : num_caches <= 64 ? launch(CommitArgs<64>{})
                                             : launch(CommitArgs<FDPP_TREE_MAX_CACHES>{});
    if (e != cudaSuccess) return fail(FDPP_ERR_CUDA, "tree commit launch: %s", cudaGetErrorString(e));
    return FDPP_OK;
}

}  // extern "C"
