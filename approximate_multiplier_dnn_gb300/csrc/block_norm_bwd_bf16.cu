// Block norm kernels, backward, with a bf16 residual stream.
#include "block_norm.cuh"

int amsim::bn::launch_bwd_bf16(int nv, Loads loads, Has has, int y_type, int n_type, const Params &p, unsigned grid,
                            cudaStream_t st)
{
    return launch_stream<true, bf16>(nv, loads, has, y_type, n_type, p, grid, st);
}
