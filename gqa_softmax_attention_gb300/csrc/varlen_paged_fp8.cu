// Packed queries over a float8_e4m3fn paged cache (TileOPs "Attention
// Operators", GQAPagedFwdOp over the FP8 caches of GQADenseFwdOp stage 2): as
// varlen_paged.cu, each key K * k_scale[b, r] and each value V * v_scale[b, r].
#include "onetile.cuh"

namespace gqa {
namespace {

// Joins the parts of every (row block, KV head): one warp per tile row, weights
// 2^(lse_p - max) over the parts' base-2 LSEs (MATE "QSA", Core Attention,
// SplitKV), the sink joining the denominator once.  A part's LSE of -inf means
// that it saw no key of the row; a NaN one (a query that is no number) makes the
// row NaN, as it is with its keys in one part.  A few hundred rows of D
// FP32 values a part: bound by the launch.  Ends at once when the plan cut
// nothing.  The whole call with its keys in parts, and in one: 4 queries over
// 32004 keys 37 and 270 us, over 2048 keys 23 and 29; 256 queries over 32256 keys
// 155 and 277, over 4096 keys 41 and 48 (32/8 heads, D = 128); 4 queries over 32004
// keys at 24/2, D = 256: 50 and 569 (cut_pays has the borders).
constexpr int JOIN_WARPS = 8;

template <int D, bool F16>
__global__ void __launch_bounds__(32 * JOIN_WARPS) join_parts_kernel(const PrefillArgs a) {
    const int parts = a.n_entries[3];
    if (parts <= 1) return;
    const int lane = threadIdx.x % 32;
    const long row = (long)blockIdx.x * JOIN_WARPS + threadIdx.x / 32;
    const long block = row / pf::BM;                          // entry * Hkv + KV head
    if (block >= (long)a.n_entries[0] * a.Hkv) return;
    const int r = (int)(row % pf::BM), rq = r / a.g, rh = r % a.g;
    const int32_t* e = a.entries + (size_t)(block / a.Hkv) * ot::ENTRY_INTS;
    const int q0 = e[1], qs = e[2], sq = e[3];
    if (rq >= a.qpb || q0 + rq >= sq) return;
    const int head = (int)(block % a.Hkv) * a.g + rh;
    const size_t orow = ((size_t)qs + q0 + rq) * a.Hq + head;
    const size_t p0 = (size_t)block * parts * pf::BM + r;     // row of part 0; parts are BM rows apart
    float top = -INFINITY;
    for (int p = lane; p < parts; p += 32) top = max_or_nan(top, a.part_lse[p0 + (size_t)p * pf::BM]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = max_or_nan(top, __shfl_xor_sync(0xffffffffu, top, o));
    constexpr int PER = D / 128;                              // float4 groups per lane
    uint16_t* out = static_cast<uint16_t*>(a.o) + orow * D;
    const float sink = a.x.sinks && top != -INFINITY ? a.x.sinks[head] * 1.4426950408889634f : -INFINITY;
    float acc[PER][4] = {}, den = 0.f, lse = -INFINITY;
    if (sink == INFINITY && !isnan(top)) {
        lse = INFINITY;
    } else if (top != -INFINITY) {
        const float M = max_or_nan(top, sink);
        den = sink == -INFINITY ? 0.f : exp2f(sink - M);
#pragma unroll 4
        for (int p = 0; p < parts; ++p) {
            const size_t pr = p0 + (size_t)p * pf::BM;
            const float w = exp2f(a.part_lse[pr] - M);
            if (w == 0.f) continue;                           // a part that saw no key of this row wrote no values
            den += w;
#pragma unroll
            for (int q = 0; q < PER; ++q) {
                const float4 v = *reinterpret_cast<const float4*>(a.part_o + pr * D + (q * 32 + lane) * 4);
                acc[q][0] += w * v.x; acc[q][1] += w * v.y; acc[q][2] += w * v.z; acc[q][3] += w * v.w;
            }
        }
        const float inv = 1.f / den;
#pragma unroll
        for (int q = 0; q < PER; ++q)
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[q][i] *= inv;
        lse = (M + log2f(den)) * pf::kLn2;
    }
#pragma unroll
    for (int q = 0; q < PER; ++q)
        *reinterpret_cast<uint2*>(out + (q * 32 + lane) * 4) =
            make_uint2(pack2<F16>(acc[q][0], acc[q][1]), pack2<F16>(acc[q][2], acc[q][3]));
    if (lane == 0 && a.lse) a.lse[orow] = lse;
}

template <int D, bool F16>
cudaError_t launch_t(const CUtensorMap& tm_o, const PrefillArgs& a, long max_items, cudaStream_t stream) {
    // parts may fill every SM, however few the items
    const long items = a.part_o ? a.num_sms : max_items;
    // only the output goes by tensor map
    const cudaError_t e = ot::launch_onetile<D, ot::kPaged8, true, F16>(
        tm_o, tm_o, tm_o, tm_o, a, items > max_items ? items : max_items, 0, stream);
    if (e != cudaSuccess || !a.part_o) return e;
    // blocks are cut only while there are at most num_sms / 2 of them
    const long blocks = max_items < a.num_sms / 2 ? max_items : a.num_sms / 2;
    const long rows = blocks * pf::BM;
    join_parts_kernel<D, F16><<<(unsigned)((rows + JOIN_WARPS - 1) / JOIN_WARPS), 32 * JOIN_WARPS, 0, stream>>>(a);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_varlen_paged_fp8(const CUtensorMap& tm_o, const PrefillArgs& a, long max_items,
                                    cudaStream_t stream) {
    switch (a.D * 2 + (a.f16 ? 1 : 0)) {
        case 128 * 2: return launch_t<128, false>(tm_o, a, max_items, stream);
        case 128 * 2 + 1: return launch_t<128, true>(tm_o, a, max_items, stream);
        case 256 * 2: return launch_t<256, false>(tm_o, a, max_items, stream);
        case 256 * 2 + 1: return launch_t<256, true>(tm_o, a, max_items, stream);
        default: return cudaErrorInvalidValue;
    }
}

int varlen_paged_fp8_take_device_error() { return ot::take_error(); }

}  // namespace gqa
