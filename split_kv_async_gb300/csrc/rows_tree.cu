// rows_tree.cu -- the rows attention's kernels on the tensor cores (rows_tc.cuh), masked by trees of drafted
// tokens (fdpp_tree.h). A translation unit of their own, so that they compile beside the others.
#include "rows_tc.cuh"

namespace fdpp {

cudaError_t launch_rows_tree(const RowsArgs& a, const RowsMaps& m, cudaStream_t s)
{
    const bool cap = a.cap > 0.f;                        // (trees take no bias)
    if (a.D == 128) return cap ? launch_d<128, MODE_CAP, true>(a, m, s) : launch_d<128, MODE_PLAIN, true>(a, m, s);
    return cap ? launch_d<64, MODE_CAP, true>(a, m, s) : launch_d<64, MODE_PLAIN, true>(a, m, s);
}

}  // namespace fdpp
