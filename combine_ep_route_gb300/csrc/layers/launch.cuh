// launch.cuh -- launch helpers of the layer's operators.
#pragma once

#include "../ep_internal.cuh"

namespace ep {

// A launch whose set-up may overlap the end of the kernel before it on the stream; the
// kernel itself calls pdl_wait() before its first access to global memory.
template <class... Params, class... Args>
cudaError_t launch_after(void (*kernel)(Params...), dim3 grid, int block, cudaStream_t st, Args... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)block);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, static_cast<Params>(args)...);
}

// out[g][c] (+)= the sum over group g's rows in use of src[g][row][c] (bf16), n columns
cudaError_t launch_row_sums(const void *src, const int32_t *counts, int groups, int rows, int n, bool out_f32,
                            bool accumulate, void *out, cudaStream_t st);

}  // namespace ep
