// Packed queries over a float8_e4m3fn paged cache (TileOPs "Attention
// Operators", GQAPagedFwdOp over the FP8 caches of GQADenseFwdOp stage 2): as
// varlen_paged.cu, each key K * k_scale[b, r] and each value V * v_scale[b, r].
#include "onetile.cuh"

namespace gqa {

cudaError_t launch_varlen_paged_fp8(const CUtensorMap& tm_o, const PrefillArgs& a, long max_items,
                                    cudaStream_t stream) {
    // only the output goes by tensor map
    switch (a.D * 2 + (a.f16 ? 1 : 0)) {
        case 128 * 2: return ot::launch_onetile<128, ot::kPaged8, true, false>(tm_o, tm_o, tm_o, tm_o, a, max_items, 0, stream);
        case 128 * 2 + 1: return ot::launch_onetile<128, ot::kPaged8, true, true>(tm_o, tm_o, tm_o, tm_o, a, max_items, 0, stream);
        case 256 * 2: return ot::launch_onetile<256, ot::kPaged8, true, false>(tm_o, tm_o, tm_o, tm_o, a, max_items, 0, stream);
        case 256 * 2 + 1: return ot::launch_onetile<256, ot::kPaged8, true, true>(tm_o, tm_o, tm_o, tm_o, a, max_items, 0, stream);
        default: return cudaErrorInvalidValue;
    }
}

int varlen_paged_fp8_take_device_error() { return ot::take_error(); }

}  // namespace gqa
