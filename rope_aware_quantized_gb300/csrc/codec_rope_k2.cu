// Bulk quantize-append kernels of keys rotated on the way, for 2-word K record slices (256 bits per key).
#include "codec_bulk.cuh"

namespace bgtq {

template <>
cudaError_t launch_bulk_bk<2, RQParams>(const RQParams& p, int bv, int batch, cudaStream_t s) {
    return launch_bulk_bk_impl<2, RQParams>(p, bv, batch, s);
}

}  // namespace bgtq
