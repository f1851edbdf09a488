// Shared by the files of the experts' layer.
#pragma once

#include "launch.h"
#include "qwq_internal.h"

namespace qwq {

constexpr int kMoePairs = 1024;               // slots of a launch at most
constexpr int kMoeTokens = 64;                // tokens of a launch at most
constexpr int kMoeFewColumns = 8;             // of a chunk, few columns

// One of the two products: gate and up of the tokens' rows, or down of h.
struct MoeStream {
    const Expert *table;
    const int *ids;
    const void *x;                            // gate and up: the tokens' rows
    const float *in;                          // down: h [P][ldh], or the slices' sums of gate and up [ns_in][P][2][ldh]
    float *out;                               // gate and up: what down reads; down: [ns][P][D]
    unsigned int *err;                        // where a wrong id is recorded
    long long ldx;                            // values
    int S, P, k, E, type, act;                // P = S * k
    int K, rows, ldh;                         // columns of the product's rows; its rows; F rounded up to 8
    int lines, ns, ns_in;                     // 128-byte lines of a row, slices of them
    int tiles, wk;                            // of the rows; 2^wk warps share one (few columns)
    Quotient by_tiles, by_grid, by_k, by_rounds;   // by_rounds: 16 tiles of a chunk each (many columns)
    int nc, held, pitch;                      // columns of a chunk, of those staged together, bytes of one in shared memory
    bool down, aligned, prepared;             // aligned: the tokens' rows start on 16 bytes
    // prepared: rows in pieces, their scales
    const uint8_t *cols;                      // as moe_prepare_kernel lays them out
    const float *info;                        // inverse scales
    unsigned long long wait_ns;               // limit of any wait for a copy
    int withheld;                             // bytes that prepared columns are waited for and do not come: 0, but in the self test
};

// How a product is launched: its kernel, columns of a chunk, slices, shared memory.
struct MoeWay {
    int kind;                                 // 0 few columns, 1 few and short ones (two blocks on an SM), 2 many columns
    int nc, held, ns, pitch;                  // columns of a chunk, of those staged together, slices, bytes of a column
    int warps, blocks;                        // warps of a block, blocks on an SM
    size_t smem;
};
template <int FMT> MoeWay moe_way(int kind, int pieces, int S, int lines);

template <int FMT> cudaError_t moe_launch_stream(const MoeStream &p, const MoeWay &w, int n_sms, cudaStream_t st);
// rows of the tokens, or of h, prepared for many columns
template <int FMT> cudaError_t moe_launch_prepare(const MoeStream &p, int rows, bool ordered, uint8_t *cols, float *info, cudaStream_t st);

// One translation unit per format has these.
#define MOE_FORMAT(F)                                                                                          \
    template <> MoeWay moe_way<F>(int kind, int pieces, int S, int lines);                                     \
    extern template cudaError_t moe_launch_stream<F>(const MoeStream &, const MoeWay &, int, cudaStream_t);    \
    extern template cudaError_t moe_launch_prepare<F>(const MoeStream &, int, bool, uint8_t *, float *, cudaStream_t)
MOE_FORMAT(B200Q_I8);
MOE_FORMAT(B200Q_I4);
MOE_FORMAT(B200Q_I2);
#undef MOE_FORMAT

// f16 pieces of a column.  One holds f16 rows exactly, of bf16 rows every value above 2^-32 of
// the largest (the others to 2^-40 of it).  f32 needs two for its 24 bits (to 2^-50 of
// the largest), and so does h of f16 rows, so that its rounding is below y's.  h of bf16
// rows has one, 11 bits beside the 8 of y: y is 1.66e-3 from 64 bits so and 1.65e-3 with two
// (8 tokens of 8 of 32 int4 experts of 6144 / 2048; 2-norms), which take 137 us instead of 125,
// and 286 instead of 242 for 64 tokens.
inline int moe_pieces(int type, bool down) { return type == B200Q_T_F32 || (down && type == B200Q_T_F16) ? 2 : 1; }

}  // namespace qwq
