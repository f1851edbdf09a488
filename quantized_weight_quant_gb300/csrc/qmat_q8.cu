// Which kernel a product on 8-bit rows runs on: up to 8 rows, the columns of one
// warp-level tensor instruction, the one that streams the weights; more rows,
// or rows too long for its shared memory, the tcgen05 kernel (int4, 6144 x
// 12288: 8 rows 15.3 us by the first; 9 rows 21.2 us by the second, which takes
// 16 at a time; the first in two calls, 8 rows and 1, 15.3 + 12.0 us).
#include "qwq_internal.h"

namespace qwq {

cudaError_t launch_mat_q8(const MatQ8 &a, cudaStream_t st) {
    bool handled = false;
    cudaError_t e = launch_mv_q8(a, st, &handled);
    if (e != cudaSuccess || handled) return e;
    return launch_gemm_q8(a, st);
}

}  // namespace qwq
