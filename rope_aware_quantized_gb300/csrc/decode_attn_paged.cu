// Decode attention on a paged Block-GTQ cache (pools of P-token pages and a
// page table per sequence): the paged instances of the decode kernel.  The
// kernel, shared with contiguous caches, is in decode_kernel.cuh; only the
// staging addresses, the L2 prefetch and the fused append's record location
// differ (a 16-token tile never straddles a page).
#include "decode_kernel.cuh"

namespace bgtq {

cudaError_t launch_decode_paged(const DecodeParams& p, dim3 grid, cudaStream_t s, int kind, int bk, int bv) {
    return launch_widths<true, kDecodePlain>(p, grid, s, kind, bk, bv);
}

}  // namespace bgtq
