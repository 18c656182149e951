// Per-head RMS norm of queries and keys and the rotation by position in one
// pass, the results written as packed rows or, for keys and values, into a
// paged cache (16-bit or float8_e4m3fn) through a slot map.
//
// For head row x of D values, weight w (1 without a norm) and pair j of the
// first `rot` dims, (d0, d1) = (j, j + rot/2), or (2j, 2j + 1) interleaved:
//   n_d = x_d * r * w_d,  r = rsqrt(mean(x^2) + eps)   (r = 1 without a norm)
//   y_d0 = n_d0 cos - n_d1 sin,  y_d1 = n_d1 cos + n_d0 sin,  y_d = n_d past rot
// with cos, sin of the token's position on the pair's axis from an FP32 table.
// Each value is y = r * (x_d * A + x_mate * B) with A = w_d cos and
// B = -+ w_mate sin, so a warp forms A and B once per token and keeps them for
// its heads.  Sums and products are FP32, rounded once to the output's type.
//
// Bound by HBM: every head row is read once and written once.  D / 8 lanes
// share a row, 16 bytes each; a warp holds 32 / (D / 8) rows at a time and
// loads U of those ahead before it reduces the first.  A warp's rows are of one
// kind (queries, keys or values), so nothing diverges.  The mate of a lane's
// chunk sits rot / 16 lanes away (rot a multiple of 16) and comes by shuffle as
// packed 16-bit pairs, before the norm is applied.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "internal.h"
#include "ptx.cuh"

namespace gqa {
namespace {

constexpr int NT = 128;
constexpr int U = 4;               // row groups a warp loads ahead

enum Kind : int { kQ = 0, kK = 1, kV = 2 };

template <bool F16>
__device__ __forceinline__ void unpack8(const uint4& v, float* f) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (F16) {
            const float2 p = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
            f[2 * i] = p.x;
            f[2 * i + 1] = p.y;
        } else {
            f[2 * i] = __uint_as_float(w[i] << 16);
            f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
}

// Two FP32 values -> two e4m3fn codes (round to nearest even, +-448 beyond the
// range, NaN stays NaN), lo in the low byte.
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

template <bool F16>
__device__ __forceinline__ uint4 pack8(const float* f) {
    return make_uint4(pack2<F16>(f[0], f[1]), pack2<F16>(f[2], f[3]), pack2<F16>(f[4], f[5]), pack2<F16>(f[6], f[7]));
}

// Eight weights of dims d .. d + 7 (ones without a norm).
template <bool F16>
__device__ __forceinline__ void load_w(const void* w, int f32, int d, float* out) {
    if (!w) {
#pragma unroll
        for (int i = 0; i < 8; ++i) out[i] = 1.f;
    } else if (f32) {
        const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(w) + d);
        const float4 x = __ldg(p), y = __ldg(p + 1);
        out[0] = x.x; out[1] = x.y; out[2] = x.z; out[3] = x.w;
        out[4] = y.x; out[5] = y.y; out[6] = y.z; out[7] = y.w;
    } else {
        unpack8<F16>(__ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(w) + d)), out);
    }
}

template <int D, bool F16, bool PAGED>
__global__ void __launch_bounds__(NT) qk_norm_rope_kernel(const RopeArgs a, int nq, int nk, int rows_per_warp) {
    constexpr int LPH = D / 8;              // lanes per head row
    constexpr int HPW = 32 / LPH;           // rows of a warp at a time
    const int lane = threadIdx.x % 32;
    const int c = lane % LPH, sub = lane / LPH;
    const long task = (long)blockIdx.x * (NT / 32) + threadIdx.x / 32;
    const int per_token = nq + nk + (PAGED ? nk : 0);
    const long t = task / per_token;
    if (t >= a.T) return;
    const int part = (int)(task % per_token);
    const int kind = part < nq ? kQ : (part < nq + nk ? kK : kV);
    const int h0 = (kind == kQ ? part : (kind == kK ? part - nq : part - nq - nk)) * rows_per_warp;
    const int H = kind == kQ ? a.Hq : a.Hkv;
    const int h_end = min(H, h0 + rows_per_warp);

    long slot = 0;
    float kv_scale = 1.f;
    const float* scales = nullptr;
    int req = 0;
    if constexpr (PAGED) {
        slot = a.slots[t];
        if (slot < 0 || slot >= a.num_slots) return;       // a padding row
        if (a.k_scale || a.v_scale) {
            req = a.requests[t];
            if (req < 0 || req >= a.B) return;
            scales = kind == kQ ? nullptr : (kind == kK ? a.k_scale : a.v_scale);
        }
    }
    const uint16_t* src = static_cast<const uint16_t*>(kind == kQ ? a.q : (kind == kK ? a.k : a.v)) +
                          t * (kind == kQ ? a.q_ts : (kind == kK ? a.k_ts : a.v_ts)) + 8 * c;
    const long hs = kind == kQ ? a.q_hs : (kind == kK ? a.k_hs : a.v_hs);

    uint4 raw[U];
    auto load = [&](int h) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int hh = h + u * HPW + sub;
            raw[u] = hh < h_end ? *reinterpret_cast<const uint4*>(src + hh * hs) : make_uint4(0u, 0u, 0u, 0u);
        }
    };
    load(h0);

    // A and B of this lane's eight dims
    const bool normed = kind == kQ ? a.q_weight != nullptr : (kind == kK && a.k_weight != nullptr);
    float A[8], Bm[8];
    int mate = lane;
    if (kind != kV) {
        const void* w = kind == kQ ? a.q_weight : a.k_weight;
        load_w<F16>(w, a.weight_f32, 8 * c, A);
#pragma unroll
        for (int i = 0; i < 8; ++i) Bm[i] = 0.f;
        if (8 * c < a.rot) {
            const int half = a.rot / 2;
            int pos[4];
#pragma unroll
            for (int x = 0; x < 4; ++x) pos[x] = x < a.n_axes ? min(max(a.positions[(size_t)x * a.T + t], 0), a.max_pos - 1) : 0;
            // the table row of pair j
            auto row = [&](int j) -> const float* {
                if (a.n_axes == 1) return a.cos_sin + (size_t)pos[0] * a.rot;
                const int ax = (a.pair_axis[j >> 4] >> (2 * (j & 15))) & 3;
                const int p = ax == 0 ? pos[0] : (ax == 1 ? pos[1] : (ax == 2 ? pos[2] : pos[3]));
                return a.cos_sin + (size_t)p * a.rot;
            };
            if (a.interleaved) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int j = 4 * c + i;
                    const float* r = row(j);
                    const float co = __ldg(r + j), si = __ldg(r + half + j);
                    const float w0 = A[2 * i], w1 = A[2 * i + 1];
                    A[2 * i] = w0 * co;
                    Bm[2 * i] = -w1 * si;
                    A[2 * i + 1] = w1 * co;
                    Bm[2 * i + 1] = w0 * si;
                }
            } else {
                const int hc = a.rot / 16;                  // chunks of a half
                const bool low = c < hc;
                mate = low ? lane + hc : lane - hc;
                float wm[8];
                load_w<F16>(w, a.weight_f32, 8 * (low ? c + hc : c - hc), wm);
                const int j0 = 8 * (low ? c : c - hc);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float* r = row(j0 + i);
                    const float co = __ldg(r + j0 + i), si = __ldg(r + half + j0 + i);
                    A[i] *= co;
                    Bm[i] = low ? -wm[i] * si : wm[i] * si;
                }
            }
        }
    }
    const bool rotated = 8 * c < a.rot;

    for (int h = h0; h < h_end; h += U * HPW) {
        uint4 cur[U];
#pragma unroll
        for (int u = 0; u < U; ++u) cur[u] = raw[u];
        if (h + U * HPW < h_end) load(h + U * HPW);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int hh = h + u * HPW + sub;
            float y[8];
            unpack8<F16>(cur[u], y);
            if (kind != kV) {
                float r = 1.f;
                if (normed) {
                    float s = 0.f;
#pragma unroll
                    for (int i = 0; i < 8; ++i) s = fmaf(y[i], y[i], s);
#pragma unroll
                    for (int o = LPH / 2; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
                    r = rsqrtf(s * (1.f / D) + a.eps);
                }
                float m[8];
                if (a.interleaved) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) m[i] = y[i ^ 1];
                } else {
                    uint4 o;
                    o.x = __shfl_sync(0xffffffffu, cur[u].x, mate);
                    o.y = __shfl_sync(0xffffffffu, cur[u].y, mate);
                    o.z = __shfl_sync(0xffffffffu, cur[u].z, mate);
                    o.w = __shfl_sync(0xffffffffu, cur[u].w, mate);
                    unpack8<F16>(o, m);
                }
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    // an unrotated dim has no mate: inf * 0 would make it NaN
                    const float v = rotated ? fmaf(y[i], A[i], m[i] * Bm[i]) : y[i] * A[i];
                    y[i] = v * r;
                }
            }
            if (hh >= h_end) continue;
            if (kind == kQ) {
                reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.q_out) + ((size_t)t * a.Hq + hh) * D)[c] =
                    pack8<F16>(y);
            } else if (!PAGED) {
                reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.k_out) + ((size_t)t * a.Hkv + hh) * D)[c] =
                    pack8<F16>(y);
            } else {
                void* cache = kind == kK ? a.k_cache : a.v_cache;
                const size_t at = ((size_t)slot * a.Hkv + hh) * D;
                if (a.e4m3) {
                    if (scales) {
                        kv_scale = __ldg(scales + (size_t)req * a.Hkv + hh);
#pragma unroll
                        for (int i = 0; i < 8; ++i) y[i] = __fdiv_rn(y[i], kv_scale);
                    }
                    uint2 o;
                    o.x = e4m3x2(y[0], y[1]) | (e4m3x2(y[2], y[3]) << 16);
                    o.y = e4m3x2(y[4], y[5]) | (e4m3x2(y[6], y[7]) << 16);
                    reinterpret_cast<uint2*>(static_cast<uint8_t*>(cache) + at)[c] = o;
                } else {
                    reinterpret_cast<uint4*>(static_cast<uint16_t*>(cache) + at)[c] =
                        kind == kV ? cur[u] : pack8<F16>(y);
                }
            }
        }
    }
}

template <int D, bool F16, bool PAGED>
cudaError_t launch_t(const RopeArgs& a, int num_sms, cudaStream_t stream) {
    // Rows of one kind a warp takes: one load-ahead (U groups) while that
    // leaves SMs idle otherwise, all heads of a kind once there are warps
    // enough (A and B are then formed once per token and kind).
    constexpr int unit = U * (32 / (D / 8));
    const int most = a.Hq > a.Hkv ? a.Hq : a.Hkv;
    int rows = unit;
    auto parts = [&](int H) { return (H + rows - 1) / rows; };
    auto tasks = [&]() { return (long)a.T * (parts(a.Hq) + (PAGED ? 2 : 1) * parts(a.Hkv)); };
    const long enough = 32L * (num_sms > 0 ? num_sms : 148);
    while (rows < most && tasks() / 2 >= enough) rows *= 2;
    const long blocks = (tasks() + NT / 32 - 1) / (NT / 32);
    if (blocks >= (1L << 31)) return cudaErrorInvalidValue;
    qk_norm_rope_kernel<D, F16, PAGED><<<(unsigned)blocks, NT, 0, stream>>>(a, parts(a.Hq), parts(a.Hkv), rows);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_qk_norm_rope(const RopeArgs& a, int D, bool f16, bool paged, int num_sms, cudaStream_t stream) {
    switch (D * 4 + (f16 ? 2 : 0) + (paged ? 1 : 0)) {
        case 64 * 4: return launch_t<64, false, false>(a, num_sms, stream);
        case 64 * 4 + 1: return launch_t<64, false, true>(a, num_sms, stream);
        case 64 * 4 + 2: return launch_t<64, true, false>(a, num_sms, stream);
        case 64 * 4 + 3: return launch_t<64, true, true>(a, num_sms, stream);
        case 128 * 4: return launch_t<128, false, false>(a, num_sms, stream);
        case 128 * 4 + 1: return launch_t<128, false, true>(a, num_sms, stream);
        case 128 * 4 + 2: return launch_t<128, true, false>(a, num_sms, stream);
        case 128 * 4 + 3: return launch_t<128, true, true>(a, num_sms, stream);
        case 256 * 4: return launch_t<256, false, false>(a, num_sms, stream);
        case 256 * 4 + 1: return launch_t<256, false, true>(a, num_sms, stream);
        case 256 * 4 + 2: return launch_t<256, true, false>(a, num_sms, stream);
        case 256 * 4 + 3: return launch_t<256, true, true>(a, num_sms, stream);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace gqa
