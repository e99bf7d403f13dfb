// Decode attention that leaves its logits and softmax statistics, on a paged
// packed cache: the scoring paged instances of the decode kernel
// (decode_kernel.cuh; the score kernel is in decode_score.cu).
#include "decode_kernel.cuh"

namespace bgtq {

cudaError_t launch_decode_score_paged(const DecodeParams& p, dim3 grid, cudaStream_t s, int kind, int bk, int bv) {
    return launch_widths<true, kDecodeScore>(p, grid, s, kind, bk, bv);
}

}  // namespace bgtq
