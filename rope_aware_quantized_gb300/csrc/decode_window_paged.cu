// Decode attention with a sliding window and sinks on a paged packed cache:
// the windowed paged instances of the decode kernel (decode_kernel.cuh).  A
// page without a visible token is never read: its page-table entry may be
// unmapped and the page given to another sequence.
#include "decode_kernel.cuh"

namespace bgtq {

cudaError_t launch_decode_window_paged(const DecodeParams& p, dim3 grid, cudaStream_t s, int kind, int bk, int bv) {
    return launch_widths<true, kDecodeWindow>(p, grid, s, kind, bk, bv);
}

}  // namespace bgtq
