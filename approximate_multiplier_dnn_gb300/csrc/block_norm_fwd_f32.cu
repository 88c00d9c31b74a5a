// Block norm kernels, forward, with an fp32 residual stream.
#include "block_norm.cuh"

int amsim::bn::launch_fwd_f32(int nv, Loads loads, Has has, int y_type, int n_type, const Params &p, unsigned grid,
                            cudaStream_t st)
{
    return launch_stream<false, float>(nv, loads, has, y_type, n_type, p, grid, st);
}
