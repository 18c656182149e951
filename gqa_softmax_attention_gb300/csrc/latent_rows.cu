// Rows of a latent cache: norm, rotation and append of new ones, and the
// gathering of cached ones.
//
// Append: a token's projected row is a latent c of 512 values and 64 shared key
// dims; its cache row is [w * c * rsqrt(mean c^2 + eps), R(p) k_pe] with R(p) the
// rotation of the 32 pairs (j, j + 32), or (2j, 2j + 1) interleaved, by the angles
// of position p.  The rotated dims of the H query heads are turned alongside
// (from a slice of the projection, into any strided place: the last 64 dims of
// the absorbed queries).  FP32 throughout, rounded once.
//
// Gather: the cached rows of requests, one after the other, for the projection
// that expands them to keys and values per head.
//
// Both read and write every row once; HBM is the bound, and the launch at a few
// tokens.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "internal.h"
#include "ptx.cuh"

namespace gqa {
namespace {

constexpr int NT = 128;
constexpr int U = 4;                       // groups of four query heads a warp loads at once
constexpr int HEADS = 4 * U;               // query heads of a warp

template <bool F16>
__device__ __forceinline__ void widen(uint32_t w, float& lo, float& hi) {
    if constexpr (F16) {
        const float2 p = __half22float2(*reinterpret_cast<const __half2*>(&w));
        lo = p.x;
        hi = p.y;
    } else {
        lo = __uint_as_float(w << 16);
        hi = __uint_as_float(w & 0xffff0000u);
    }
}

// Eight lanes turn a row of 64 values: lane l holds dims 4l .. 4l + 3 (x) and 32
// + 4l .. 35 + 4l (y), which holds every pair of either kind whole.
struct Turn {
    float co[8], si[8];                    // of x and y's dims
    template <bool NEXT>
    __device__ __forceinline__ void load(const float* row, int l) {
        if constexpr (NEXT) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {  // pairs 2l, 2l + 1 and 16 + 2l, 17 + 2l
                const int j = (e / 2) * 16 + 2 * l + e % 2;
                co[2 * e] = co[2 * e + 1] = __ldg(row + j);
                si[2 * e] = si[2 * e + 1] = __ldg(row + kLatentRope / 2 + j);
            }
        } else {
            const float4 c = __ldg(reinterpret_cast<const float4*>(row + 4 * l));
            const float4 s = __ldg(reinterpret_cast<const float4*>(row + kLatentRope / 2 + 4 * l));
            co[0] = co[4] = c.x; co[1] = co[5] = c.y; co[2] = co[6] = c.z; co[3] = co[7] = c.w;
            si[0] = si[4] = s.x; si[1] = si[5] = s.y; si[2] = si[6] = s.z; si[3] = si[7] = s.w;
        }
    }
    template <bool F16, bool NEXT>
    __device__ __forceinline__ void turn(uint2& x, uint2& y) const {
        float v[8], r[8];
        widen<F16>(x.x, v[0], v[1]);
        widen<F16>(x.y, v[2], v[3]);
        widen<F16>(y.x, v[4], v[5]);
        widen<F16>(y.y, v[6], v[7]);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const bool second = NEXT ? (e & 1) : e >= 4;
            const float mate = NEXT ? v[e ^ 1] : v[e ^ 4];
            r[e] = second ? fmaf(v[e], co[e], mate * si[e]) : fmaf(v[e], co[e], -(mate * si[e]));
        }
        x = make_uint2(pack2<F16>(r[0], r[1]), pack2<F16>(r[2], r[3]));
        y = make_uint2(pack2<F16>(r[4], r[5]), pack2<F16>(r[6], r[7]));
    }
};

// A warp per task: a token's latent row, or up to 16 of its query heads, every load of
// a task under way before its first store (16384 tokens with 32 heads, rows to the
// cache and packed: 36.6 us, 5.3 TB/s; 32 heads a warp in two turns the same, 8192
// tokens with 128 heads 54.0 against 55.5 with 64 a warp; blocks of 64 or 256
// threads, 8 or 32 heads at once within 1 us).
template <bool F16, bool NEXT>
__global__ void __launch_bounds__(NT) latent_append_kernel(const LatentAppendArgs a, int q_parts) {
    const int lane = threadIdx.x % 32, l = lane % 8;
    long task = (long)blockIdx.x * (NT / 32) + threadIdx.x / 32;
    const bool is_kv = task < a.T;
    if (!is_kv) {
        task -= a.T;
        if (task >= (long)a.T * q_parts) return;
    }
    const long t = is_kv ? task : task / q_parts;
    const long slot = a.slots[t];
    const int pos = min(max(a.positions[t], 0), a.max_pos - 1);
    if (is_kv) {
        // lane: latents 8 lane .. and 256 + 8 lane ..; the first eight lanes turn the shared dims
        const uint16_t* src = static_cast<const uint16_t*>(a.kv) + t * a.kv_ts;
        uint4 c[2];
        c[0] = *reinterpret_cast<const uint4*>(src + 8 * lane);
        c[1] = *reinterpret_cast<const uint4*>(src + 256 + 8 * lane);
        uint2 x = *reinterpret_cast<const uint2*>(src + kLatentDim + 4 * l);
        uint2 y = *reinterpret_cast<const uint2*>(src + kLatentDim + kLatentRope / 2 + 4 * l);
        if (slot < 0 || slot >= a.num_slots) return;           // a padding row
        Turn tr;
        tr.load<NEXT>(a.cos_sin + (size_t)pos * kLatentRope, l);
        tr.turn<F16, NEXT>(x, y);
        if (a.weight) {
            float v[16], ss = 0.f;
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                widen<F16>(c[k].x, v[8 * k], v[8 * k + 1]);
                widen<F16>(c[k].y, v[8 * k + 2], v[8 * k + 3]);
                widen<F16>(c[k].z, v[8 * k + 4], v[8 * k + 5]);
                widen<F16>(c[k].w, v[8 * k + 6], v[8 * k + 7]);
            }
#pragma unroll
            for (int e = 0; e < 16; ++e) ss = fmaf(v[e], v[e], ss);
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
            const float r = rsqrtf(ss * (1.f / kLatentDim) + a.eps);
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const int d = 256 * k + 8 * lane;
                float w[8];
                if (a.weight_f32) {
#pragma unroll
                    for (int e = 0; e < 8; e += 4) {
                        const float4 q = __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(a.weight) + d + e));
                        w[e] = q.x; w[e + 1] = q.y; w[e + 2] = q.z; w[e + 3] = q.w;
                    }
                } else {
                    const uint4 q = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.weight) + d));
                    widen<F16>(q.x, w[0], w[1]);
                    widen<F16>(q.y, w[2], w[3]);
                    widen<F16>(q.z, w[4], w[5]);
                    widen<F16>(q.w, w[6], w[7]);
                }
                float* n = v + 8 * k;
#pragma unroll
                for (int e = 0; e < 8; ++e) n[e] = n[e] * r * w[e];
                c[k] = make_uint4(pack2<F16>(n[0], n[1]), pack2<F16>(n[2], n[3]), pack2<F16>(n[4], n[5]),
                                  pack2<F16>(n[6], n[7]));
            }
        }
        auto store = [&](uint16_t* dst) {
            *reinterpret_cast<uint4*>(dst + 8 * lane) = c[0];
            *reinterpret_cast<uint4*>(dst + 256 + 8 * lane) = c[1];
            if (lane < 8) {
                *reinterpret_cast<uint2*>(dst + kLatentDim + 4 * l) = x;
                *reinterpret_cast<uint2*>(dst + kLatentDim + kLatentRope / 2 + 4 * l) = y;
            }
        };
        store(static_cast<uint16_t*>(a.cache) + slot * kLatentRow);
        if (a.kv_out) store(static_cast<uint16_t*>(a.kv_out) + t * a.kvo_ts);
        return;
    }
    const int h0 = (int)(task % q_parts) * HEADS, n = a.H - h0, sub = lane / 8;
    const uint16_t* src = static_cast<const uint16_t*>(a.q) + t * a.q_ts + (h0 + sub) * a.q_hs;
    uint16_t* dst = static_cast<uint16_t*>(a.q_out) + t * a.qo_ts + (h0 + sub) * a.qo_hs;
    uint2 x[U], y[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        if (4 * u + sub < n) {
            const uint16_t* p = src + 4 * u * a.q_hs;
            x[u] = *reinterpret_cast<const uint2*>(p + 4 * l);
            y[u] = *reinterpret_cast<const uint2*>(p + kLatentRope / 2 + 4 * l);
        }
    }
    if (slot < 0 || slot >= a.num_slots) return;
    Turn tr;
    tr.load<NEXT>(a.cos_sin + (size_t)pos * kLatentRope, l);
#pragma unroll
    for (int u = 0; u < U; ++u) {
        if (4 * u + sub < n) {
            tr.turn<F16, NEXT>(x[u], y[u]);
            uint16_t* p = dst + 4 * u * a.qo_hs;
            *reinterpret_cast<uint2*>(p + 4 * l) = x[u];
            *reinterpret_cast<uint2*>(p + kLatentRope / 2 + 4 * l) = y[u];
        }
    }
}

// A block takes GROWS rows of the packed result: a warp finds the rows' requests
// and cache rows, then all threads copy 16 bytes at a time, every load of a
// thread issued before its first store (16 requests, 134K rows: 51 us, 90 % of the
// copy rate).  The search reads all offsets before the block's rows, 32 at a time: 1000
// requests of 100 rows 5.8 TB/s, 4000 of 30 4.4, 16384 of 10 1.8.
constexpr int GROWS = 32;
constexpr int CHUNKS = kLatentRow * 2 / 16;    // 72
constexpr int GT = 288;                        // GROWS * CHUNKS / GT = 8 chunks a thread
static_assert(GROWS * CHUNKS % GT == 0 && GT % CHUNKS == 0, "whole rows a step");

__global__ void __launch_bounds__(GT) latent_gather_kernel(const LatentGatherArgs a) {
    __shared__ long src_row[GROWS];            // cache row, -1: zeros, -2: of no request
    const int lane = threadIdx.x % 32;
    const int j0 = blockIdx.x * GROWS;
    if (threadIdx.x < 32) {
        const int j = j0 + lane;
        // the request of row j: how many of them end at or before it
        int b = 0;
        for (int b0 = 0; b0 < a.B; b0 += 32) {
            const int end = b0 + lane < a.B ? a.cu[b0 + lane + 1] : 0x7fffffff;
            const int n = min(32, a.B - b0);
            if (__shfl_sync(0xffffffffu, end, n - 1) <= j0) {      // all of these end before the block's rows
                b += n;
                continue;
            }
            for (int e = 0; e < n; ++e) b += __shfl_sync(0xffffffffu, end, e) <= j ? 1 : 0;
            if (__shfl_sync(0xffffffffu, end, n - 1) > j0 + GROWS - 1) break;
        }
        long row = -2;
        if (b < a.B && j < a.total) {
            const int t = j - a.cu[b];
            if (t >= 0) {
                const int lp = t / a.page_size;
                const int page = lp < a.max_pages ? a.table[(size_t)b * a.max_pages + lp] : -1;
                row = page >= 0 && page < a.num_pages ? (long)page * a.page_size + (t - lp * a.page_size) : -1;
            }
        }
        src_row[lane] = row;
    }
    __syncthreads();
    constexpr int N = GROWS * CHUNKS / GT, STEP = GT / CHUNKS;     // 8 chunks of rows STEP apart
    const int r0 = threadIdx.x / CHUNKS, c = threadIdx.x % CHUNKS;
    const uint4* src = static_cast<const uint4*>(a.cache);
    uint4* dst = static_cast<uint4*>(a.out) + (size_t)j0 * CHUNKS + c;
    uint4 v[N];
#pragma unroll
    for (int e = 0; e < N; ++e) {
        const long row = src_row[r0 + e * STEP];
        v[e] = make_uint4(0u, 0u, 0u, 0u);
        if (row >= 0) ldg16(reinterpret_cast<uint32_t*>(&v[e]), src + row * CHUNKS + c);
    }
#pragma unroll
    for (int e = 0; e < N; ++e)
        if (src_row[r0 + e * STEP] != -2) dst[(size_t)(r0 + e * STEP) * CHUNKS] = v[e];
}

}  // namespace

cudaError_t launch_latent_append(const LatentAppendArgs& a, bool f16, cudaStream_t stream) {
    const int parts = (a.H + HEADS - 1) / HEADS;
    const long blocks = ((long)a.T * (1 + parts) + NT / 32 - 1) / (NT / 32);
    if (blocks >= (1L << 31)) return cudaErrorInvalidValue;
    const unsigned g = (unsigned)blocks;
    if (f16) {
        if (a.interleaved) latent_append_kernel<true, true><<<g, NT, 0, stream>>>(a, parts);
        else latent_append_kernel<true, false><<<g, NT, 0, stream>>>(a, parts);
    } else {
        if (a.interleaved) latent_append_kernel<false, true><<<g, NT, 0, stream>>>(a, parts);
        else latent_append_kernel<false, false><<<g, NT, 0, stream>>>(a, parts);
    }
    return cudaGetLastError();
}

cudaError_t launch_latent_gather(const LatentGatherArgs& a, cudaStream_t stream) {
    const unsigned blocks = (unsigned)(((long)a.total + GROWS - 1) / GROWS);
    latent_gather_kernel<<<blocks, GT, 0, stream>>>(a);
    return cudaGetLastError();
}

}  // namespace gqa
