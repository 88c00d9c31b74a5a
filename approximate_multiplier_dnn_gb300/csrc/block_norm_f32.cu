// Block norm kernels with an fp32 residual stream.
#include "block_norm.cuh"

int amsim::bn::launch_f32(bool bwd, int nv, Loads loads, int y_type, int n_type, const Params &p, unsigned grid,
                          cudaStream_t st)
{
    return launch_stream<float>(bwd, nv, loads, y_type, n_type, p, grid, st);
}
