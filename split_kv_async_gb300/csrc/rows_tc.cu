// rows_tc.cu -- the rows attention's kernels on the tensor cores (rows_tc.cuh), key ranges as masks.
#include "rows_tc.cuh"

namespace fdpp {

int rows_tc_stages(int head_dim, int smem_per_block)
{
    int n = 0;
    while (n < 16 && (head_dim == 128 ? RowsSmem<128>(n + 2).total : RowsSmem<64>(n + 2).total) <= smem_per_block) n += 2;
    return n;                                            // even: K and V tiles take turns
}

cudaError_t launch_rows_tc(const RowsArgs& a, const RowsMaps& m, cudaStream_t s)
{
    const int mode = a.cap > 0.f ? MODE_CAP : (a.slopes ? MODE_BIAS : MODE_PLAIN);
    if (a.parents) return launch_rows_tree(a, m, s);
    if (a.D == 128)
        return mode == MODE_CAP    ? launch_d<128, MODE_CAP>(a, m, s)
               : mode == MODE_BIAS ? launch_d<128, MODE_BIAS>(a, m, s)
                                   : launch_d<128, MODE_PLAIN>(a, m, s);
    return mode == MODE_CAP    ? launch_d<64, MODE_CAP>(a, m, s)
           : mode == MODE_BIAS ? launch_d<64, MODE_BIAS>(a, m, s)
                               : launch_d<64, MODE_PLAIN>(a, m, s);
}

}  // namespace fdpp
