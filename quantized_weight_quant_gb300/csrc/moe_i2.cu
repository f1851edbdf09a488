// The experts' products on int2 codes.
#include "moe_kernels.h"

namespace qwq {

template cudaError_t moe_launch_stream<B200Q_I2>(const MoeStream &, const MoeWay &, int, cudaStream_t);
template cudaError_t moe_launch_prepare<B200Q_I2>(const MoeStream &, int, bool, uint8_t *, float *, cudaStream_t);
template <> MoeWay moe_way<B200Q_I2>(int kind, int pieces, int S, int lines) { return moe_way_of<B200Q_I2>(kind, pieces, S, lines); }

}  // namespace qwq
