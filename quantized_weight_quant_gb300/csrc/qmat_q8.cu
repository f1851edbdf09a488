// Which kernel a product on 8-bit rows runs on.
#include "qwq_internal.h"

namespace qwq {

cudaError_t launch_mat_q8(const MatQ8 &a, cudaStream_t st) {
    bool handled = false;
    cudaError_t e = launch_mv_q8(a, st, &handled);
    if (e != cudaSuccess || handled) return e;
    return launch_gemm_q8(a, st);
}

}  // namespace qwq
