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
// share a row; a lane holds two pieces of four values, chosen so that the mates
// of a piece lie in the lane itself: pieces 4l and rot/2 + 4l (mates in the
// other piece), or 4l and D/2 + 4l interleaved (mates in the same piece), so
// that only the sum of squares crosses lanes, and each load of a warp still
// covers whole 64-byte stretches.  A warp holds 32 / (D / 8) rows at a time
// and loads U of those before it works on them; its rows are of one kind
// (queries, keys or values), so nothing diverges.  Arithmetic goes in pairs
// (f32x2).  Measured, 16384 tokens at D = 128: 32/8 heads dense 57-59 us (86-89 %
// of the copy rate), 64/8 heads into e4m3 caches 107-109 us (88-89 %); a few tokens
// 3-4 us on the GPU.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "internal.h"
#include "ptx.cuh"

namespace gqa {
namespace {

constexpr int NT = 128;
constexpr int U = 4;               // row groups a warp loads at once

enum Kind : int { kQ = 0, kK = 1, kV = 2 };

// Two 16-bit values -> a pair of floats.
template <bool F16>
__device__ __forceinline__ uint64_t widen2(uint32_t w) {
    if constexpr (F16) {
        const float2 p = __half22float2(*reinterpret_cast<const __half2*>(&w));
        return f32x2(p.x, p.y);
    } else {
        return f32x2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
    }
}
__device__ __forceinline__ uint64_t swap2(uint64_t v) {
    float lo, hi;
    f32x2_split(v, lo, hi);
    return f32x2(hi, lo);
}

// Two FP32 values -> two e4m3fn codes (round to nearest even, +-448 beyond the
// range, NaN stays NaN), lo in the low byte.
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

// Pairs y / s given inv, the rounded 1 / s: the product corrected by its
// remainder (Markstein 1990), which is the rounded quotient where it matters;
// beyond the e4m3 range, where the remainder could overflow, the product alone.
__device__ __forceinline__ void quotient2(uint64_t y, float s, float inv, float& lo, float& hi) {
    const uint64_t inv2 = f32x2(inv, inv), q = fmul2(y, inv2);
    const uint64_t c = ffma2(ffma2(q, f32x2(-s, -s), y), inv2, q);
    float q0, q1;
    f32x2_split(q, q0, q1);
    f32x2_split(c, lo, hi);
    lo = fabsf(q0) < 1024.f ? lo : q0;
    hi = fabsf(q1) < 1024.f ? hi : q1;
}

// Four weights of dims d .. d + 3 (ones without a norm).
template <bool F16>
__device__ __forceinline__ void load_w(const void* w, int f32, int d, float* out) {
    if (!w) {
        out[0] = out[1] = out[2] = out[3] = 1.f;
    } else if (f32) {
        const float4 x = __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(w) + d));
        out[0] = x.x; out[1] = x.y; out[2] = x.z; out[3] = x.w;
    } else {
        const uint2 x = __ldg(reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(w) + d));
        f32x2_split(widen2<F16>(x.x), out[0], out[1]);
        f32x2_split(widen2<F16>(x.y), out[2], out[3]);
    }
}

// Rows h0 .. h_end - 1 of one kind of token t.
template <int D, bool F16, bool PAGED, bool NEXT, int KIND>
__device__ __forceinline__ void do_rows(const RopeArgs& a, long t, int h0, int h_end, int lane) {
    constexpr int LPH = D / 8;              // lanes per head row
    constexpr int HPW = 32 / LPH;           // rows of a warp at a time
    constexpr bool STORE8 = PAGED && KIND != kQ;
    const int l = lane % LPH, sub = lane / LPH;
    // this lane's two pieces
    const int pairs = a.rot / 8;            // lanes that hold rotated pieces (mates in halves)
    const int p0 = NEXT ? 4 * l : (l < pairs ? 4 * l : a.rot + 8 * (l - pairs));
    const int p1 = NEXT ? D / 2 + 4 * l : (l < pairs ? a.rot / 2 + 4 * l : p0 + 4);
    const bool rot0 = p0 < a.rot, rot1 = p1 < a.rot;

    const long hs = KIND == kQ ? a.q_hs : (KIND == kK ? a.k_hs : a.v_hs);
    const uint16_t* src = static_cast<const uint16_t*>(KIND == kQ ? a.q : (KIND == kK ? a.k : a.v)) +
                          t * (KIND == kQ ? a.q_ts : (KIND == kK ? a.k_ts : a.v_ts)) + (h0 + sub) * hs;
    const int n = h_end - h0;               // rows; this lane's are sub, sub + HPW, ...
    uint2 raw[U][2];
    auto load = [&](int i) {                // rows i .. of the task; past its end the last row this lane has
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const uint16_t* p = src + (i + u * HPW + sub < n ? i + u * HPW : (n - 1 - sub) / HPW * HPW) * hs;
            raw[u][0] = *reinterpret_cast<const uint2*>(p + p0);
            raw[u][1] = *reinterpret_cast<const uint2*>(p + p1);
        }
    };
    if (sub < n) load(0);                   // a lane without a row works on whatever its registers hold
    long slot = 0;
    int req = 0;
    if constexpr (PAGED) {
        slot = a.slots[t];
        if (a.k_scale || a.v_scale) req = a.requests[t];
    }
    int pos[4] = {0, 0, 0, 0};
    if (KIND != kV && a.rot > 0) {
#pragma unroll
        for (int x = 0; x < 4; ++x)
            if (x < a.n_axes) pos[x] = min(max(a.positions[(size_t)x * a.T + t], 0), a.max_pos - 1);
    }
    if constexpr (PAGED) {
        if (slot < 0 || slot >= a.num_slots) return;               // a padding row
        if ((a.k_scale || a.v_scale) && (req < 0 || req >= a.B)) return;
    }

    // A and B of the two pieces
    const void* w = KIND == kQ ? a.q_weight : a.k_weight;
    uint64_t A[2][2], B[2][2];
    if constexpr (KIND != kV) {
        const int half = a.rot / 2;
        float wp[2][4], co[2][4], si[2][4];
        load_w<F16>(w, a.weight_f32, p0, wp[0]);
        load_w<F16>(w, a.weight_f32, p1, wp[1]);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                co[k][i] = 1.f;
                si[k][i] = 0.f;
            }
        }
        // the table row of pair j
        auto row = [&](int j) -> const float* {
            int p = pos[0];
            if (a.n_axes > 1) {
                const int ax = (a.pair_axis[j >> 4] >> (2 * (j & 15))) & 3;
                p = ax == 0 ? pos[0] : (ax == 1 ? pos[1] : (ax == 2 ? pos[2] : pos[3]));
            }
            return a.cos_sin + (size_t)p * a.rot;
        };
        if constexpr (NEXT) {
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                if (k == 0 ? rot0 : rot1) {
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const int j = (k == 0 ? p0 : p1) / 2 + i;
                        const float* r = row(j);
                        co[k][2 * i] = co[k][2 * i + 1] = __ldg(r + j);
                        si[k][2 * i] = si[k][2 * i + 1] = __ldg(r + half + j);
                    }
                }
            }
        } else if (rot0 && a.n_axes == 1) {
            // rot is a multiple of 16, so four cosines or sines are 16 aligned bytes
            const float* r = row(0);
            const float4 c4 = __ldg(reinterpret_cast<const float4*>(r + p0));
            const float4 s4 = __ldg(reinterpret_cast<const float4*>(r + half + p0));
            co[0][0] = co[1][0] = c4.x; co[0][1] = co[1][1] = c4.y; co[0][2] = co[1][2] = c4.z; co[0][3] = co[1][3] = c4.w;
            si[0][0] = si[1][0] = s4.x; si[0][1] = si[1][1] = s4.y; si[0][2] = si[1][2] = s4.z; si[0][3] = si[1][3] = s4.w;
        } else if (rot0) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float* r = row(p0 + i);
                co[0][i] = co[1][i] = __ldg(r + p0 + i);
                si[0][i] = si[1][i] = __ldg(r + half + p0 + i);
            }
        }
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            float b[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                b[i] = NEXT ? (i & 1 ? wp[k][i ^ 1] * si[k][i] : -wp[k][i ^ 1] * si[k][i])
                            : (k == 1 ? wp[0][i] * si[k][i] : -wp[1][i] * si[k][i]);
            A[k][0] = f32x2(wp[k][0] * co[k][0], wp[k][1] * co[k][1]);
            A[k][1] = f32x2(wp[k][2] * co[k][2], wp[k][3] * co[k][3]);
            B[k][0] = f32x2(b[0], b[1]);
            B[k][1] = f32x2(b[2], b[3]);
        }
    }
    const bool normed = KIND != kV && w != nullptr;
    const bool partial = a.rot < D;
    const float* scale = nullptr;           // of this lane's first row
    if constexpr (STORE8) {
        scale = KIND == kK ? a.k_scale : a.v_scale;
        if (scale) scale += (size_t)req * a.Hkv + h0 + sub;
    }
    // this lane's first output row, in elements
    const size_t out = ((KIND != kQ && PAGED ? (size_t)slot : (size_t)t) * (KIND == kQ ? a.Hq : a.Hkv) + h0 + sub) * D;

    for (int i = 0; i < n; i += U * HPW) {
        if (i > 0 && sub < n) load(i);
        float sc[U];
        if constexpr (STORE8) {
#pragma unroll
            for (int u = 0; u < U; ++u)
                sc[u] = scale && i + u * HPW + sub < n ? __ldg(scale + i + u * HPW) : 1.f;
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int row = i + u * HPW;                           // + sub
            uint64_t y[2][2];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                y[k][0] = widen2<F16>(raw[u][k].x);
                y[k][1] = widen2<F16>(raw[u][k].y);
            }
            if constexpr (KIND != kV) {
                float r = 1.f;
                if (normed) {
                    uint64_t s2 = fmul2(y[0][0], y[0][0]);
                    s2 = ffma2(y[0][1], y[0][1], s2);
                    s2 = ffma2(y[1][0], y[1][0], s2);
                    s2 = ffma2(y[1][1], y[1][1], s2);
                    float s, s1;
                    f32x2_split(s2, s, s1);
                    s += s1;
#pragma unroll
                    for (int o = LPH / 2; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
                    r = rsqrtf(s * (1.f / D) + a.eps);
                }
                uint64_t m[2][2];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    m[0][e] = NEXT ? swap2(y[0][e]) : y[1][e];
                    m[1][e] = NEXT ? swap2(y[1][e]) : y[0][e];
                }
                if (partial) {                             // an unrotated value has no mate: inf * 0 would be NaN
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        m[0][e] = rot0 ? m[0][e] : 0ull;
                        m[1][e] = rot1 ? m[1][e] : 0ull;
                    }
                }
                const uint64_t r2 = f32x2(r, r);
#pragma unroll
                for (int k = 0; k < 2; ++k)
#pragma unroll
                    for (int e = 0; e < 2; ++e)
                        y[k][e] = fmul2(ffma2(y[k][e], A[k][e], fmul2(m[k][e], B[k][e])), r2);
            }
            if (row + sub >= n) continue;
            const size_t at = out + (size_t)row * D;
            float f[2][4];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                f32x2_split(y[k][0], f[k][0], f[k][1]);
                f32x2_split(y[k][1], f[k][2], f[k][3]);
            }
            if (STORE8 && a.e4m3) {
                if (scale) {
                    const float s = sc[u];
                    if (s > 0x1p-120f && s < 0x1p120f) {
                        const float inv = __frcp_rn(s);
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            quotient2(y[k][0], s, inv, f[k][0], f[k][1]);
                            quotient2(y[k][1], s, inv, f[k][2], f[k][3]);
                        }
                    } else {                               // no normal reciprocal
#pragma unroll
                        for (int k = 0; k < 2; ++k)
#pragma unroll
                            for (int e = 0; e < 4; ++e) f[k][e] = __fdiv_rn(f[k][e], s);
                    }
                }
                uint8_t* dst = static_cast<uint8_t*>(KIND == kK ? a.k_cache : a.v_cache) + at;
                *reinterpret_cast<uint32_t*>(dst + p0) = e4m3x2(f[0][0], f[0][1]) | (e4m3x2(f[0][2], f[0][3]) << 16);
                *reinterpret_cast<uint32_t*>(dst + p1) = e4m3x2(f[1][0], f[1][1]) | (e4m3x2(f[1][2], f[1][3]) << 16);
            } else {
                uint16_t* dst = static_cast<uint16_t*>(KIND == kQ ? a.q_out
                                                                  : (!PAGED ? a.k_out
                                                                            : (KIND == kK ? a.k_cache : a.v_cache))) + at;
                if constexpr (KIND == kV) {                        // values go as they came
                    *reinterpret_cast<uint2*>(dst + p0) = raw[u][0];
                    *reinterpret_cast<uint2*>(dst + p1) = raw[u][1];
                } else {
                    *reinterpret_cast<uint2*>(dst + p0) =
                        make_uint2(pack2<F16>(f[0][0], f[0][1]), pack2<F16>(f[0][2], f[0][3]));
                    *reinterpret_cast<uint2*>(dst + p1) =
                        make_uint2(pack2<F16>(f[1][0], f[1][1]), pack2<F16>(f[1][2], f[1][3]));
                }
            }
        }
    }
}

// A warp per task: up to rows_per_warp rows of one kind of one token.  All query
// tasks come before the key tasks and those before the value tasks, so that a
// block's warps take equally long (token by token, blocks held three warps of 8
// rows until one of 64 was done: 180 instead of 134 us at 16384 tokens, 64/8
// heads, D = 128, e4m3 caches).
template <int D, bool F16, bool PAGED, bool NEXT>
__global__ void __launch_bounds__(NT, 7) qk_norm_rope_kernel(const RopeArgs a, int nq, int nk, int rows_per_warp) {
    const int lane = threadIdx.x % 32;
    long task = (long)blockIdx.x * (NT / 32) + threadIdx.x / 32;
    if (task < (long)a.T * nq) {
        const int h0 = (int)(task % nq) * rows_per_warp;
        do_rows<D, F16, PAGED, NEXT, kQ>(a, task / nq, h0, min(a.Hq, h0 + rows_per_warp), lane);
        return;
    }
    task -= (long)a.T * nq;
    if (task < (long)a.T * nk) {
        const int h0 = (int)(task % nk) * rows_per_warp;
        do_rows<D, F16, PAGED, NEXT, kK>(a, task / nk, h0, min(a.Hkv, h0 + rows_per_warp), lane);
        return;
    }
    if constexpr (PAGED) {
        task -= (long)a.T * nk;
        if (task < (long)a.T * nk) {
            const int h0 = (int)(task % nk) * rows_per_warp;
            do_rows<D, F16, PAGED, NEXT, kV>(a, task / nk, h0, min(a.Hkv, h0 + rows_per_warp), lane);
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
    if (a.interleaved)
        qk_norm_rope_kernel<D, F16, PAGED, true><<<(unsigned)blocks, NT, 0, stream>>>(a, parts(a.Hq), parts(a.Hkv), rows);
    else
        qk_norm_rope_kernel<D, F16, PAGED, false><<<(unsigned)blocks, NT, 0, stream>>>(a, parts(a.Hq), parts(a.Hkv), rows);
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
