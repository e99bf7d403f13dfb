// Bulk quantize-append kernels of keys rotated on the way, for 1-word K record slices (128 bits per key).
#include "codec_bulk.cuh"

namespace bgtq {

template <>
cudaError_t launch_bulk_bk<1, RQParams>(const RQParams& p, int bv, int batch, cudaStream_t s) {
    return launch_bulk_bk_impl<1, RQParams>(p, bv, batch, s);
}

}  // namespace bgtq
