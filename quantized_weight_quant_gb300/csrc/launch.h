// Launches that may begin while the kernel before them on the stream ends
// (programmatic dependent launch): such a kernel waits (griddepcontrol.wait) before
// it reads what another has written, and before it writes.
#pragma once

#include "qwq_internal.h"

namespace qwq {

template <class K, class... P>
cudaError_t launch_dependent(K kernel, dim3 grid, dim3 block, size_t smem, cudaStream_t st, const P &...p) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, p...);
    count_launch();
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace qwq
