// Decode attention with a sliding window and sinks on a contiguous packed
// cache: the windowed instances of the decode kernel (decode_kernel.cuh).
// A row attends positions [0, sinks) and [seq - window, seq); only their
// records are read, so the launch is bound as the plain decode is, by the
// decode work of the visible tokens, and by the launch's fixed phases when
// they are few.
#include "decode_kernel.cuh"

namespace bgtq {

cudaError_t launch_decode_window(const DecodeParams& p, dim3 grid, cudaStream_t s, int kind, int bk, int bv) {
    return launch_widths<false, kDecodeWindow>(p, grid, s, kind, bk, bv);
}

}  // namespace bgtq
