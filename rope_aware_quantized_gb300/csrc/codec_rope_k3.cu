// Bulk quantize-append kernels of keys rotated on the way, for 3-word K record slices (384 bits per key).
#include "codec_bulk.cuh"

namespace bgtq {

template <>
cudaError_t launch_bulk_bk<3, RQParams>(const RQParams& p, int bv, int batch, cudaStream_t s) {
    return launch_bulk_bk_impl<3, RQParams>(p, bv, batch, s);
}

cudaError_t launch_quantize_append_bulk(const RQParams& p, int bk, int bv, int batch, cudaStream_t s) {
    switch (bk) {
        case 1: return launch_bulk_bk<1, RQParams>(p, bv, batch, s);
        case 2: return launch_bulk_bk<2, RQParams>(p, bv, batch, s);
        case 3: return launch_bulk_bk<3, RQParams>(p, bv, batch, s);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace bgtq
