// Attention in the latent space over a paged cache: every token has one row of
// 576 numbers, a latent of 512 (value and first part of the key of every head)
// and 64 rotated dims that complete the key.  Queries are already projected
// into that space, so with q', row_j in R^576
//   s_j = scale * q' . row_j,   o' = sum_j softmax(s)_j * row_j[0:512]
// (TileOPs "Attention Operators", the decode with q, q_pe, k, k_pe).  All heads
// of a query read the same row: 1152 bytes and 2 * 1088 FLOP a head, so up to
// about 100 (head, query) rows a key the cache's bytes are the bound, and the
// tensor cores from there.
//
// Packed queries: request b owns queries [cu_q[b], cu_q[b + 1]), its rows are
// r = i * H + h (query i, head h), and query i sees the keys
// j <= i + L_b - Sq_b.  NR rows go to one CTA; a team of one or two CTAs takes
// the rows [seg * team * NR, ...) of a request and reads the same keys at the
// same time, so that the second reading comes from L2.
//
// The products are formed transposed, keys and dims on the MMAs' M side and the
// rows on N, because O of 512 dims by 64 rows then takes half of TMEM (as O
// itself it would take all of it, whatever the row count):
//   S^T [128 keys, NR]  = K [128, 576] Q^T            36 MMAs of K = 16
//   O^T [512 dims, NR] += V^T [512, 128 keys] P^T     4 x 8 MMAs
// A cache tile lies in shared memory once and is both operands: K-major for
// S^T, dims-major (transposed) for O^T.  Shared memory holds Q (72 KB at 64
// rows) and one tile (144 KB); so that loads keep running, the tile is four
// slots of 128 dims and one of the 64 shared dims, each released by itself as
// O^T has taken it, and P^T is written over the shared dims, which only S^T needs.
//
// A softmax thread owns a key: its S^T row holds the key's score with every
// row of queries.  The reference maximum of a row (column) is kept in shared
// memory and moves only when a score exceeds it by more than 2^8, which the
// threads vote on; the row sums are kept as per-thread parts and joined across
// the keys once per piece.
//
// Work is balanced: the row groups of all requests, laid end to end, form one
// sequence of 128-key tiles, and each team takes an equal range.  A row group
// that lies in one range is written out directly; of one that is cut, each
// piece leaves O, maximum and sum in FP32, at most two pieces a team, and
// latent_join_kernel adds them up.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cmath>

#include "internal.h"
#include "ptx.cuh"

namespace gqa {
namespace {

__device__ int g_latent_paged_error;

constexpr int BN = 128;                    // keys per tile
constexpr int DC = kLatentDim;             // 512: latent
constexpr int DR = kLatentRope;            // 64: shared rotated dims
constexpr int DK = DC + DR;
constexpr int ROW_BYTES = DK * 2;
constexpr int NJ = DC / 128;               // 128-dim blocks of O^T (pairs of 64-dim slices)
constexpr float kLn2 = 0.693147180559945309f;
constexpr float kRescaleThreshold = 8.f;
constexpr int WARP_MMA = 4;
constexpr int WARP_LOAD = 5;
constexpr int kSmBar = 1;                  // named barrier of the softmax warps

template <int NR, bool GATHER>
struct LCfg {
    static constexpr int NP = 4;                                   // slots of 128 dims
    static constexpr int PAIR = BN * 256;                          // bytes of a slot: [16 groups][2 slices][8 keys][128]
    static constexpr int ROPE = BN * 128;                          // shared dims, later P^T: [128 keys][128]
    static constexpr int Q_SLICE = NR * 128;                       // 64 dims of Q
    static constexpr int OFF_Q = 0;
    static constexpr int OFF_P = OFF_Q + (DK / 64) * Q_SLICE;
    static constexpr int OFF_KV = OFF_P + ROPE;
    static constexpr int OFF_COL = OFF_KV + NP * PAIR;             // per row: -reference, rescale, limit, sums [4]
    static constexpr int OFF_BAR = OFF_COL + 8 * NR * 4;
    // kv_full[NP], kv_empty[NP], pe_full, q_full, q_empty, s_full, p_full, o_done, drain
    static constexpr int NBAR = 2 * NP + 7;
    static constexpr int OFF_MISC = OFF_BAR + NBAR * 8;
    static constexpr int SMEM_BYTES = OFF_MISC + 64 + 1024;
    static constexpr int LOAD_WARPS = GATHER ? 2 : 1;      // 8 warps at most: 255 registers a thread
    static constexpr int THREADS = 32 * (5 + LOAD_WARPS);
    static constexpr uint32_t COL_S = NJ * NR;                     // TMEM: O^T blocks | S^T
    static constexpr uint32_t TMEM_COLS = 512;
    static_assert(COL_S + NR <= TMEM_COLS, "TMEM budget");
    static_assert(OFF_KV % 1024 == 0 && OFF_P % 1024 == 0, "swizzle atoms");
    static_assert(SMEM_BYTES <= 227 * 1024, "shared memory budget");
};

// Where this team's range of the tile sequence starts.
struct LRange {
    long g0, n, per;        // first tile, tiles, tiles per team
    int b, seg, lt, pad;    // request, row group and tile of the first one
};

__device__ __forceinline__ int request_len(const LatentArgs& a, int b) {
    return (int)min((long)max(a.lens[b], 0), (long)a.max_pages * a.page_size);
}
__device__ __forceinline__ void request_rows(const LatentArgs& a, int b, int& qs, int& sq) {
    qs = min(max(a.cu_q[b], 0), a.total_q);
    sq = min(max(a.cu_q[b + 1], qs), a.total_q) - qs;
}

// A stretch of one row group's tiles, and the walk over those of a range.
struct Piece {
    int b, seg, nseg, nt;    // request, row group, its groups, tiles of each
    int qs, sq, L;
    int lt0, lt1;            // tiles [lt0, lt1) of the row group
    long left;               // tiles of the range from lt0 on
    int row0, rows;          // this CTA's rows (of the request's sq * H)
    int n;                   // tiles from lt0 on with a key that one of its rows sees
    __device__ __forceinline__ void request(const LatentArgs& a, int rb, int group) {
        b = rb;
        request_rows(a, b, qs, sq);
        L = request_len(a, b);
        nseg = (sq * a.H + group - 1) / group;
        nt = max(1, (L + BN - 1) / BN);
    }
    __device__ __forceinline__ void fit(const LatentArgs& a, int group, int nr, int rank) {
        lt1 = (int)min((long)nt, lt0 + left);
        row0 = seg * group + rank * nr;
        rows = min(nr, sq * a.H - row0);
        n = 0;
        if (rows > 0) {
            const int i_last = (row0 + rows - 1) / a.H;
            const int lim = a.causal ? max(0, min(L, L - sq + i_last + 1)) : L;
            n = max(0, min(lt1, (lim + BN - 1) / BN) - lt0);
        }
    }
    __device__ __forceinline__ void first(const LatentArgs& a, const LRange& r, int group, int nr, int rank) {
        request(a, r.b, group);
        seg = r.seg;
        lt0 = r.lt;
        left = r.n;
        fit(a, group, nr, rank);
    }
    __device__ __forceinline__ bool next(const LatentArgs& a, int group, int nr, int rank) {
        left -= lt1 - lt0;
        if (left <= 0) return false;
        lt0 = 0;
        if (++seg >= nseg) {
            seg = 0;
            do {
                if (b + 1 >= a.B) return false;
                request(a, b + 1, group);
            } while (nseg == 0);
        }
        fit(a, group, nr, rank);
        return true;
    }
};

// Order-preserving integers of floats, for the warp-wide maximum (NaN ends up
// above +inf or below -inf; the row's weights are NaN either way).
__device__ __forceinline__ int ordered(float x) {
    const int i = __float_as_int(x);
    return i ^ ((i >> 31) & 0x7fffffff);
}
__device__ __forceinline__ float unordered(int i) { return __int_as_float(i ^ ((i >> 31) & 0x7fffffff)); }

// Sums of v[0 .. N) over the warp's lanes: lane l returns columns
// l * N / 32 .. of them in v[0 .. max(1, N / 32)).  Each step exchanges the
// half of the columns that the other half of the lanes keeps.
template <int N>
__device__ __forceinline__ void warp_column_sums(float* v, int lane) {
    static_assert(N == 64 || N == 32, "columns");
#pragma unroll
    for (int o = 16, w = N / 2; o >= 1; o >>= 1, w >>= 1) {
        const bool up = (lane & o) != 0;
#pragma unroll
        for (int i = 0; i < N / 2; ++i) {
            if (i < w) {
                const float mine = up ? v[i + w] : v[i], other = up ? v[i] : v[i + w];
                v[i] = mine + __shfl_xor_sync(0xffffffffu, other, o);
            }
        }
    }
}

// n / page_size for 0 <= n < 2^31
__device__ __forceinline__ int page_of(const LatentArgs& a, uint32_t n) {
    return (int)((__umulhi(n, a.ps_mul) + n) >> a.ps_shift);
}

template <int NR, bool F16, bool GATHER>
__global__ void __launch_bounds__((LCfg<NR, GATHER>::THREADS), 1)
latent_paged_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_kv,
                    const __grid_constant__ CUtensorMap tm_pe, const LatentArgs a) {
    using C = LCfg<NR, GATHER>;
    constexpr uint32_t IDESC_S = make_idesc_16<F16>(BN, NR, false, false);
    constexpr uint32_t IDESC_O = make_idesc_16<F16>(128, NR, true, true);
    griddep_launch_dependents();                 // the joining kernel may be scheduled (it waits for this grid)

    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    uint8_t* smem = smem_raw + ((1024 - (raw & 1023)) & 1023);
    const uint32_t sb = smem_u32(smem);
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int team = blockIdx.x / a.team, rank = blockIdx.x % a.team;
    const int group = a.team * NR;               // rows of a team

    const uint32_t bar0 = sb + C::OFF_BAR;
    auto kv_full = [&](int i) { return bar0 + 8u * i; };
    auto kv_empty = [&](int i) { return bar0 + 8u * (C::NP + i); };
    const uint32_t pe_full = bar0 + 8u * (2 * C::NP), q_full = pe_full + 8, q_empty = pe_full + 16,
                   s_full = pe_full + 24, p_full = pe_full + 32, o_done = pe_full + 40, drain = pe_full + 48;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::OFF_MISC);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::OFF_MISC + 4);
    LRange* range = reinterpret_cast<LRange*>(smem + C::OFF_MISC + 16);

    if (threadIdx.x == 0) {
        const int fills = GATHER ? 32 * C::LOAD_WARPS : 1;
        for (int i = 0; i < C::NP; ++i) { mbar_init(kv_full(i), fills); mbar_init(kv_empty(i), 1); }
        mbar_init(pe_full, fills);
        mbar_init(q_full, 1);
        mbar_init(q_empty, 1);
        mbar_init(s_full, 1);
        mbar_init(p_full, 128);
        mbar_init(o_done, 1);
        mbar_init(drain, 1);
        *abort_flag = 0;
        *range = LRange{0, 0, 0, 0, 0, 0, 0};
        fence_mbar_init();
        if (rank == 0) *reinterpret_cast<int4*>(a.join + 4 * team) = make_int4(0, 0, 0, 0);
    }
    {
        // The tiles before each request (the ring is free until the loads start),
        // their total, and the request that holds this team's first tile.
        long* pre = reinterpret_cast<long*>(smem + C::OFF_KV);
        long* part = reinterpret_cast<long*>(smem + C::OFF_Q);
        long base = 0;
        for (int b0 = 0; b0 < a.B; b0 += C::THREADS) {
            const int b = b0 + threadIdx.x;
            long x = 0;
            if (b < a.B) {
                Piece p;
                p.request(a, b, group);
                x = (long)p.nseg * p.nt;
            }
            const long own = x;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const long y = __shfl_up_sync(0xffffffffu, x, o);
                if (lane >= o) x += y;
            }
            if (lane == 31) part[warp] = x;
            __syncthreads();
            long before = base, all = 0;
            for (int w = 0; w < C::THREADS / 32; ++w) {
                if (w < warp) before += part[w];
                all += part[w];
            }
            if (b < a.B) pre[b] = before + x - own;
            base += all;
            __syncthreads();
        }
        long per = (base + a.teams - 1) / a.teams;
        if (per < a.min_tiles) per = a.min_tiles;
        const long g0 = team * per, n = max(0L, min(per, base - g0));
        if (n > 0) {
            for (int b = threadIdx.x; b < a.B; b += C::THREADS) {
                const long lo = pre[b], hi = b + 1 < a.B ? pre[b + 1] : base;
                if (lo <= g0 && g0 < hi) {
                    Piece p;
                    p.request(a, b, group);
                    *range = LRange{g0, n, per, b, (int)((g0 - lo) / p.nt), (int)((g0 - lo) % p.nt), 0};
                }
            }
        }
    }
    if (warp == WARP_MMA) {
        tmem_alloc(smem_u32(tmem_slot), C::TMEM_COLS);
        tmem_relinquish();
    }
    tc_fence_before();
    fence_proxy_async_smem();                    // the prefix sums were generic writes; the ring is TMA's now
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const LRange rg = *range;

    if (rg.n > 0) {
    if (warp >= WARP_LOAD) {
        // ------------------------------------------------------------ producer
        const int pw = warp - WARP_LOAD;
        int it = 0, nq = 0;                      // tiles and Q blocks loaded
        bool ok = true;
        if (lane == 0) {
            tma_prefetch_desc(&tm_q);
            if (!GATHER) {
                tma_prefetch_desc(&tm_kv);
                tma_prefetch_desc(&tm_pe);
            }
        }
        Piece p;
        p.first(a, rg, group, NR, rank);
        bool more = true;
        // Page id that holds token t of the piece's request, as the table has it
        // (-1 past the request's end).
        auto page_at = [&](const Piece& c, int t) {
            const int lp = page_of(a, (uint32_t)t);
            return t < c.L ? ldg_int(a.table + (size_t)c.b * a.max_pages + lp) : -1;
        };
        for (; more && ok; more = p.next(a, group, NR, rank)) {
            if (p.n == 0) continue;
            if (pw == 0) {
                // the piece's Q rows, once the last S^T of the piece before is done
                if (lane == 0) {
                    ok = mbar_wait(q_empty, (nq & 1) ^ 1, abort_flag);
                    if (ok) {
                        mbar_arrive_expect_tx(q_full, (DK / 64) * C::Q_SLICE);
                        tma_load_3d(sb + C::OFF_Q, &tm_q, q_full, 0, p.qs * a.H + p.row0, 0);
                    }
                }
                ok = __shfl_sync(0xffffffffu, ok, 0);
                if (!ok) break;
                ++nq;
            }
            if constexpr (!GATHER) {
                // Lane i loads page block i of the tile: 8-row groups of the cache as
                // one box of 128 dims each; a block past the request's end or of a
                // page outside the pool lies outside the map and comes as zeros.
                const int bt = a.box_tokens, nbox = BN / bt;
                const int outside = a.num_pages * (a.page_size / 8);
                auto token = [&](int k) { return (p.lt0 + k) * BN + lane * bt; };
                int page = lane < nbox ? page_at(p, token(0)) : -1;
                for (int k = 0; k < p.n && ok; ++k, ++it) {
                    const int t = token(k);
                    const int in_page = t - page_of(a, (uint32_t)t) * a.page_size;
                    const int grp = page >= 0 && page < a.num_pages
                                        ? (int)(((long)page * a.page_size + in_page) >> 3)
                                        : outside;
                    if (k + 1 < p.n) page = lane < nbox ? page_at(p, token(k + 1)) : -1;
                    for (int j = 0; j <= NJ && ok; ++j) {
                        const uint32_t full = j < NJ ? kv_full(j) : pe_full;
                        if (lane == 0) {
                            // P^T of the tile before lies where the shared dims go
                            ok = j < NJ ? mbar_wait(kv_empty(j), (it & 1) ^ 1, abort_flag)
                                        : mbar_wait(o_done, (it & 1) ^ 1, abort_flag);
                            if (ok) mbar_arrive_expect_tx(full, j < NJ ? C::PAIR : C::ROPE);
                        }
                        ok = __shfl_sync(0xffffffffu, ok, 0);
                        if (!ok) break;
                        __syncwarp();            // the expect-tx precedes every lane's copy
                        if (lane < nbox) {
                            if (j < NJ)
                                tma_load_4d(sb + C::OFF_KV + j * C::PAIR + lane * bt * 256, &tm_kv, full, 0, 0, 2 * j, grp);
                            else
                                tma_load_4d(sb + C::OFF_P + lane * bt * 128, &tm_pe, full, 0, 0, 2 * NJ, grp);
                        }
                    }
                }
            } else {
                // Rows one by one: a warp copies 64 of them, eight lanes a row's 128
                // bytes; a slot is announced once the copies of the next one are under
                // way, or at once where the next slot is not free yet.
                uint32_t pending = 0;
                auto announce = [&]() {
                    if (pending) {
                        fence_proxy_async_smem();
                        mbar_arrive(pending);
                        pending = 0;
                    }
                };
                auto row_of = [&](int k, int half) {   // cache row of one of this lane's keys of tile k, -1 for zeros
                    const int t = (p.lt0 + k) * BN + pw * 64 + half * 32 + lane;
                    const int page = page_at(p, t);
                    return page >= 0 && page < a.num_pages
                               ? page * a.page_size + (t - page_of(a, (uint32_t)t) * a.page_size)
                               : -1;
                };
                int row0 = row_of(0, 0), row1 = row_of(0, 1);
                for (int k = 0; k < p.n && ok; ++k, ++it) {
                    const int now0 = row0, now1 = row1;
                    if (k + 1 < p.n) {
                        row0 = row_of(k + 1, 0);
                        row1 = row_of(k + 1, 1);
                    }
                    for (int j = 0; j <= NJ && ok; ++j) {
                        const uint32_t empty = j < NJ ? kv_empty(j) : o_done;
                        if (!__all_sync(0xffffffffu, mbar_test_wait(empty, (it & 1) ^ 1))) {
                            cp_async_wait<0>();
                            announce();
                            ok = __all_sync(0xffffffffu, mbar_wait(empty, (it & 1) ^ 1, abort_flag));
                            if (!ok) break;
                        }
                        const uint32_t dst = sb + (j < NJ ? C::OFF_KV + j * C::PAIR : C::OFF_P);
                        const int stride = j < NJ ? 2048 : 1024, slices = j < NJ ? 2 : 1;
#pragma unroll 4
                        for (int e = 0; e < 16; ++e) {
                            const int key = pw * 64 + 4 * e + lane / 8, c = lane % 8;
                            const int r = __shfl_sync(0xffffffffu, e < 8 ? now0 : now1, (4 * e + lane / 8) & 31);
                            const char* src = static_cast<const char*>(a.cache) + (size_t)max(r, 0) * ROW_BYTES +
                                              j * 256 + c * 16;
                            for (int s = 0; s < slices; ++s)
                                cp_async16(dst + (key >> 3) * stride + s * 1024 + (key & 7) * 128 + ((c ^ (key & 7)) << 4),
                                           src + s * 128, r >= 0 ? 16 : 0);
                        }
                        cp_async_commit();
                        if (pending) {
                            cp_async_wait<1>();
                            announce();
                        }
                        pending = j < NJ ? kv_full(j) : pe_full;
                    }
                }
                cp_async_wait<0>();
                announce();
            }
        }
        if (*abort_flag && pw == 0 && lane == 0) {
            // let the copies in flight land: the last load of each slot
            if (!GATHER && it > 0) {
                for (int j = 0; j < C::NP; ++j) mbar_drain(kv_full(j), (it - 1) & 1);
                mbar_drain(pe_full, (it - 1) & 1);
            }
            if (nq > 0) mbar_drain(q_full, (nq - 1) & 1);
        }
    } else if (warp == WARP_MMA) {
        // ------------------------------------------------------------ MMA issuer (lane 0 issues)
        Piece p;
        p.first(a, rg, group, NR, rank);
        bool more = true, ok = true;
        int it = 0, nq = 0;
        const uint64_t qdesc = make_sdesc_sw128(sb + C::OFF_Q, 16, 1024);
        const uint64_t pdesc = make_sdesc_sw128(sb + C::OFF_P, 1024, 1024);
        for (; more && ok; more = p.next(a, group, NR, rank)) {
            for (int k = 0; k < p.n && ok; ++k, ++it) {
                // S^T of the tile: the slots as they land, the shared dims last
                if (k == 0) ok = __all_sync(0xffffffffu, mbar_wait(q_full, nq & 1, abort_flag));
                for (int j = 0; j <= NJ && ok; ++j) {
                    ok = __all_sync(0xffffffffu, mbar_wait(j < NJ ? kv_full(j) : pe_full, it & 1, abort_flag));
                    if (!ok) break;
                    tc_fence_after();
                    if (lane == 0) {
                        // K-major A: 8-key groups 2 KB apart (1 KB in the shared dims' slot)
                        const uint64_t kdesc = j < NJ ? make_sdesc_sw128(sb + C::OFF_KV + j * C::PAIR, 16, 2048)
                                                      : make_sdesc_sw128(sb + C::OFF_P, 16, 1024);
                        const uint64_t qd = qdesc + (uint64_t)((2 * j * C::Q_SLICE) >> 4);
#pragma unroll
                        for (int kk = 0; kk < 8; ++kk)
                            if (kk < 4 || j < NJ)
                                mma_bf16_ss(tmem + C::COL_S, kdesc + (uint64_t)(((kk / 4) * 1024 + (kk % 4) * 32) >> 4),
                                            qd + (uint64_t)(((kk / 4) * C::Q_SLICE + (kk % 4) * 32) >> 4), IDESC_S,
                                            (j > 0 || kk > 0) ? 1u : 0u);
                    }
                    __syncwarp();
                }
                if (!ok) break;
                if (lane == 0) {
                    mma_commit(s_full);
                    if (k == p.n - 1) mma_commit(q_empty);
                }
                if (k == p.n - 1) ++nq;
                __syncwarp();
                ok = __all_sync(0xffffffffu, mbar_wait(p_full, it & 1, abort_flag));
                if (!ok) break;
                tc_fence_after();
                if (lane == 0) {
#pragma unroll
                    for (int j = 0; j < NJ; ++j) {
                        // dims-major A: 64-dim slices 1 KB apart, 8-key groups 2 KB apart
                        const uint64_t vdesc = make_sdesc_sw128(sb + C::OFF_KV + j * C::PAIR, 1024, 2048);
#pragma unroll
                        for (int kk = 0; kk < BN / 16; ++kk)
                            mma_bf16_ss(tmem + j * NR, vdesc + (uint64_t)((kk * 4096) >> 4),
                                        pdesc + (uint64_t)((kk * 2048) >> 4), IDESC_O, (k > 0 || kk > 0) ? 1u : 0u);
                        mma_commit(kv_empty(j));
                    }
                    mma_commit(o_done);
                }
                __syncwarp();
            }
        }
        if (lane == 0) {
            mma_commit(drain);                   // every MMA issued above has completed once this arrives
            mbar_drain(drain, 0);
        }
        __syncwarp();
    } else {
        // ------------------------------------------------------------ softmax warps 0-3
        const int kk = threadIdx.x;              // this thread's key of a tile (TMEM lane), or its row where rows are meant
        const uint32_t lane_addr = (uint32_t)(warp * 32) << 16;
        float* neg_ref = reinterpret_cast<float*>(smem + C::OFF_COL);   // -reference maximum (0 while there is none)
        float* factor = neg_ref + NR;                                   // rescale factor of the last move; 1 / sum
        int* limit = reinterpret_cast<int*>(neg_ref + 2 * NR);          // keys that the row sees
        float* cross = neg_ref + 4 * NR;                                // [4][NR]: per warp
        float* ref = neg_ref + 3 * NR;                                  // reference maximum, -inf while there is none
        const float sl = a.scale_log2;
        Piece p;
        p.first(a, rg, group, NR, rank);
        bool more = true, ok = true, at_start = true;
        int it = 0;
        long at = rg.g0;                         // the piece's first tile in the sequence
        // A wait that gave up (ok false) ends the work but not the walk: all four
        // warps pass the same named barriers to the end.
        for (; more; more = p.next(a, group, NR, rank), at_start = false) {
            const bool whole = p.lt0 == 0 && p.lt1 == p.nt;
            int lim_all = 0;
            if (p.rows > 0) {
                // row r of the block is query (row0 + r) / H; blocks cut short see what their last row sees
                auto lim_of = [&](int r) {
                    const int i = (p.row0 + min(r, p.rows - 1)) / a.H;
                    return a.causal ? max(0, min(p.L, p.L - p.sq + i + 1)) : p.L;
                };
                lim_all = lim_of(0);             // every row sees the keys below
                if (kk < NR) {
                    limit[kk] = lim_of(kk);
                    neg_ref[kk] = 0.f;
                    ref[kk] = -INFINITY;
                }
            }
            named_bar_sync(kSmBar, 128);
            float sums[NR];
#pragma unroll
            for (int c = 0; c < NR; ++c) sums[c] = 0.f;
            for (int k = 0; k < p.n; ++k, ++it) {
                const int t = (p.lt0 + k) * BN + kk;
                const bool all_seen = (p.lt0 + k + 1) * BN <= lim_all;
                if (ok) ok = __all_sync(0xffffffffu, mbar_wait(s_full, it & 1, abort_flag));
                tc_fence_after();
                float s[NR];
                auto load = [&]() {              // scores in log2 units against the rows' references; hidden ones -inf
#pragma unroll
                    for (int c = 0; c < NR; c += 32) tmem_ld32(tmem + lane_addr + C::COL_S + c, s + c);
#pragma unroll
                    for (int c = 0; c < NR; c += 4) {
                        const float4 nr = *reinterpret_cast<const float4*>(neg_ref + c);
                        s[c] = fmaf(s[c], sl, nr.x);
                        s[c + 1] = fmaf(s[c + 1], sl, nr.y);
                        s[c + 2] = fmaf(s[c + 2], sl, nr.z);
                        s[c + 3] = fmaf(s[c + 3], sl, nr.w);
                    }
                    if (!all_seen) {
#pragma unroll
                        for (int c = 0; c < NR; c += 4) {
                            const int4 li = *reinterpret_cast<const int4*>(limit + c);
                            s[c] = t < li.x ? s[c] : -INFINITY;
                            s[c + 1] = t < li.y ? s[c + 1] : -INFINITY;
                            s[c + 2] = t < li.z ? s[c + 2] : -INFINITY;
                            s[c + 3] = t < li.w ? s[c + 3] : -INFINITY;
                        }
                    }
                };
                if (ok) {
                    load();
                } else {
#pragma unroll
                    for (int c = 0; c < NR; ++c) s[c] = -INFINITY;
                }
                float top = -INFINITY;
                {
#pragma unroll
                    for (int c = 0; c < NR; c += 2) top = fmax3(top, s[c], s[c + 1]);
                }
                // The first tile gives every row that sees a key its reference;
                // a row that sees none there sees none in later tiles either.
                const bool keep = named_bar_and(kSmBar, 128, ok && k > 0 && !(top > kRescaleThreshold));
                if (!keep) {
                    // column maxima over the 128 keys
#pragma unroll
                    for (int c = 0; c < NR; ++c) {
                        const int m = __reduce_max_sync(0xffffffffu, ordered(s[c]));
                        if (lane == c % 32) cross[warp * NR + c] = unordered(m);
                    }
                    named_bar_sync(kSmBar, 128);
                    if (kk < NR) {
                        const float d = fmaxf(fmaxf(cross[kk], cross[NR + kk]), fmaxf(cross[2 * NR + kk], cross[3 * NR + kk]));
                        const float old = ref[kk];
                        float f = 1.f;
                        if (old == -INFINITY || d > kRescaleThreshold) {
                            const float m = d - neg_ref[kk];          // neg_ref is 0 while there is no reference
                            f = old == -INFINITY ? 0.f : fast_exp2(old - m);
                            ref[kk] = m;
                            neg_ref[kk] = m == -INFINITY ? 0.f : -m;
                        }
                        factor[kk] = f;
                    }
                    named_bar_sync(kSmBar, 128);
                    if (ok) load();
                    if (k > 0 && ok) {
                        // O^T of the tiles before is complete (this S^T came after it)
#pragma unroll
                        for (int c = 0; c < NR; ++c) sums[c] *= factor[c];
#pragma unroll 1
                        for (int c = 0; c < NJ * NR; c += 32) {
                            float o[32];
                            tmem_ld32(tmem + lane_addr + c, o);
#pragma unroll
                            for (int e = 0; e < 32; ++e) o[e] *= factor[(c + e) % NR];
                            tmem_st32(tmem + lane_addr + c, reinterpret_cast<uint32_t*>(o));
                        }
                    }
                }
                if (!ok) continue;
                // P^T: row = key, 128 bytes with the 128-byte swizzle
                const uint32_t prow = sb + C::OFF_P + kk * 128;
#pragma unroll
                for (int c = 0; c < NR; c += 8) {
                    uint32_t w[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float p0 = fast_exp2(s[c + 2 * e]), p1 = fast_exp2(s[c + 2 * e + 1]);
                        sums[c + 2 * e] += p0;
                        sums[c + 2 * e + 1] += p1;
                        w[e] = pack2<F16>(p0, p1);
                    }
                    st_shared_v4(prow + (((c / 8) ^ (kk & 7)) << 4), w[0], w[1], w[2], w[3]);
                }
                if (t >= p.L) {
                    // a row past the request's end: whatever the page holds there must not reach O^T
                    for (int j = 0; j < NJ; ++j)
                        for (int c = 0; c < 16; ++c)
                            st_shared_v4(sb + C::OFF_KV + j * C::PAIR + (kk >> 3) * 2048 + (c >> 3) * 1024 + (kk & 7) * 128 +
                                             (c & 7) * 16, 0u, 0u, 0u, 0u);
                }
                fence_proxy_async_smem();
                tc_fence_before();
                mbar_arrive(p_full);
            }
            // ---- the piece's end
            __syncwarp();
            if (ok && p.n > 0) {
                ok = __all_sync(0xffffffffu, mbar_wait(o_done, (it - 1) & 1, abort_flag));
                tc_fence_after();
            }
            warp_column_sums<NR>(sums, lane);
#pragma unroll
            for (int e = 0; e < NR / 32; ++e) cross[warp * NR + lane * (NR / 32) + e] = sums[e];
            ok = named_bar_and(kSmBar, 128, ok);
            if (p.rows > 0) {
                const long orow = (long)p.qs * a.H + p.row0;       // first row of the block in [total_q * H]
                if (kk < NR) {
                    const float m = ref[kk];
                    const float l = (cross[kk] + cross[NR + kk]) + (cross[2 * NR + kk] + cross[3 * NR + kk]);
                    const bool some = p.n > 0 && l != 0.f;         // 0: no key; NaN goes on
                    if (whole) {
                        factor[kk] = some ? 1.f / l : 0.f;
                        if (kk < p.rows && a.lse) a.lse[orow + kk] = some ? (m + log2f(l)) * kLn2 : -INFINITY;
                    } else {
                        const int id = 2 * blockIdx.x + (at_start ? 0 : 1);
                        a.part_ml[(size_t)id * NR + kk] = some ? make_float2(m, l) : make_float2(-INFINITY, 0.f);
                    }
                }
                named_bar_sync(kSmBar, 128);
                if (whole) {
                    // O^T [dim, row] / sum -> [row, dim]: two lanes exchange so that each
                    // holds two neighbouring dims of one row
                    uint32_t* out = reinterpret_cast<uint32_t*>(a.o);
                    const bool odd = lane & 1;
#pragma unroll 1
                    for (int j = 0; j < NJ; ++j) {
#pragma unroll 1
                        for (int c = 0; c < NR; c += 32) {
                            float o[32];
                            if (p.n > 0) {
                                __syncwarp();
                                tmem_ld32(tmem + lane_addr + j * NR + c, o);
                            }
#pragma unroll
                            for (int e = 0; e < 32; e += 2) {
                                const float o0 = p.n > 0 ? o[e] * factor[c + e] : 0.f;
                                const float o1 = p.n > 0 ? o[e + 1] * factor[c + e + 1] : 0.f;
                                const float got = __shfl_xor_sync(0xffffffffu, odd ? o0 : o1, 1);
                                const int r = c + e + (odd ? 1 : 0);
                                if (r < p.rows)
                                    out[((orow + r) * DC + j * 128 + warp * 32 + (lane & ~1)) / 2] =
                                        odd ? pack2<F16>(got, o1) : pack2<F16>(o0, got);
                            }
                        }
                    }
                } else if (p.n > 0) {
                    // as it lies, [block][four rows][dim][4], for the joining kernel
                    const size_t id = 2 * (size_t)blockIdx.x + (at_start ? 0 : 1);
                    float4* dst = reinterpret_cast<float4*>(a.part_o) + id * (NJ * NR / 4) * 128 + kk;
#pragma unroll 1
                    for (int c = 0; c < NJ * NR; c += 32) {
                        float o[32];
                        __syncwarp();
                        tmem_ld32(tmem + lane_addr + c, o);
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            dst[(c / 4 + e) * 128] = make_float4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
                    }
                }
            }
            if (!whole && p.lt0 == 0 && kk == 0 && rank == 0) {
                // this team holds the row group's first tile: where its pieces lie
                const long last = (at + p.nt - 1) / rg.per;
                *reinterpret_cast<int4*>(a.join + 4 * team) =
                    make_int4((int)(last - team) + 1, (int)((long)p.qs * a.H) + p.seg * group,
                              min(group, p.sq * a.H - p.seg * group), at_start ? 0 : 1);
            }
            at += p.lt1 - p.lt0;
            tc_fence_before();
            named_bar_sync(kSmBar, 128);           // the rows' numbers may be written again
        }
    }
    }

    tc_fence_before();
    __syncthreads();
    if (warp == WARP_MMA) {
        tc_fence_after();
        tmem_dealloc(tmem, C::TMEM_COLS);
    }
    if (threadIdx.x == 0 && *abort_flag) atomicExch(&g_latent_paged_error, (int)kErrDecodeWait);
}

// Adds up the pieces of the row groups that were cut: o = sum_p w_p O_p / sum_p
// w_p l_p with w_p = 2^(m_p - M).  Block (CTA of the team's first piece, four
// rows of it); thread = dim, so a piece is read 512 x 16 bytes at a time.
template <int NR, bool F16>
__global__ void __launch_bounds__(512) latent_join_kernel(const LatentArgs a) {
    griddep_wait();
    const int team = blockIdx.x / a.team, rank = blockIdx.x % a.team, c4 = blockIdx.y;
    const int4 j = *reinterpret_cast<const int4*>(a.join + 4 * team);
    const int n = min(j.x, a.teams - team);
    const int r0 = rank * NR + 4 * c4;             // row of the group
    if (n <= 0 || r0 >= j.z) return;
    __shared__ float4 m_s[256], l_s[256];          // n <= teams <= 256
    __shared__ float inv[4];
    const int d = threadIdx.x;
    auto slot = [&](int p) { return 2 * ((team + p) * a.team + rank) + (p == 0 ? j.w : 0); };
    for (int p = d; p < n; p += 512) {
        const float2* ml = a.part_ml + (size_t)slot(p) * NR + 4 * c4;
        m_s[p] = make_float4(ml[0].x, ml[1].x, ml[2].x, ml[3].x);
        l_s[p] = make_float4(ml[0].y, ml[1].y, ml[2].y, ml[3].y);
    }
    __syncthreads();
    if (d < 4) {
        float* m = reinterpret_cast<float*>(m_s) + d;
        const float* l = reinterpret_cast<const float*>(l_s) + d;
        float M = -INFINITY, L = 0.f;
        for (int p = 0; p < n; ++p) M = fmaxf(M, m[4 * p]);
        for (int p = 0; p < n; ++p) {
            const float w = l[4 * p] == 0.f ? 0.f : fast_exp2(m[4 * p] - M);
            m[4 * p] = w;
            L += w * l[4 * p];
        }
        inv[d] = L != 0.f ? 1.f / L : 0.f;
        if (r0 + d < j.z && a.lse) a.lse[(size_t)j.y + r0 + d] = L != 0.f ? (M + log2f(L)) * kLn2 : -INFINITY;
    }
    __syncthreads();
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    const float4* src = reinterpret_cast<const float4*>(a.part_o) + ((d / 128) * (NR / 4) + c4) * 128 + d % 128;
#pragma unroll 4
    for (int p = 0; p < n; ++p) {
        const float4 w = m_s[p];
        const float4 o = src[(size_t)slot(p) * (NJ * NR / 4) * 128];
        // a piece with no key for a row has not written its O
        acc.x = w.x != 0.f ? fmaf(w.x, o.x, acc.x) : acc.x;
        acc.y = w.y != 0.f ? fmaf(w.y, o.y, acc.y) : acc.y;
        acc.z = w.z != 0.f ? fmaf(w.z, o.z, acc.z) : acc.z;
        acc.w = w.w != 0.f ? fmaf(w.w, o.w, acc.w) : acc.w;
    }
    uint16_t* out = static_cast<uint16_t*>(a.o) + ((size_t)j.y + r0) * DC + d;
    const float v[4] = {acc.x * inv[0], acc.y * inv[1], acc.z * inv[2], acc.w * inv[3]};
#pragma unroll
    for (int e = 0; e < 4; ++e)
        if (r0 + e < j.z) out[e * DC] = (uint16_t)pack2<F16>(v[e], 0.f);
}

template <int NR, bool F16, bool GATHER>
cudaError_t launch_t(const CUtensorMap& tm_q, const CUtensorMap& tm_kv, const CUtensorMap& tm_pe, const LatentArgs& a,
                     cudaStream_t stream) {
    using C = LCfg<NR, GATHER>;
    cudaError_t e = cudaFuncSetAttribute(latent_paged_kernel<NR, F16, GATHER>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM_BYTES);
    if (e != cudaSuccess) return e;
    const unsigned ctas = (unsigned)(a.teams * a.team);
    latent_paged_kernel<NR, F16, GATHER><<<ctas, C::THREADS, C::SMEM_BYTES, stream>>>(tm_q, tm_kv, tm_pe, a);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(ctas, NR / 4);
    cfg.blockDim = dim3(512);
    cfg.stream = stream;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, latent_join_kernel<NR, F16>, a);
}

}  // namespace

cudaError_t launch_latent_paged(const CUtensorMap& tm_q, const CUtensorMap& tm_kv, const CUtensorMap& tm_pe,
                                const LatentArgs& a, cudaStream_t stream) {
    const bool gather = a.box_tokens == 0;
    if (a.f16) return gather ? launch_t<kLatentRows, true, true>(tm_q, tm_kv, tm_pe, a, stream)
                             : launch_t<kLatentRows, true, false>(tm_q, tm_kv, tm_pe, a, stream);
    return gather ? launch_t<kLatentRows, false, true>(tm_q, tm_kv, tm_pe, a, stream)
                  : launch_t<kLatentRows, false, false>(tm_q, tm_kv, tm_pe, a, stream);
}

int latent_paged_take_device_error() {
    int v = 0;
    if (cudaMemcpyFromSymbol(&v, g_latent_paged_error, sizeof(int)) != cudaSuccess) return -1;
    if (v != 0) {
        const int zero = 0;
        cudaMemcpyToSymbol(g_latent_paged_error, &zero, sizeof(int));
    }
    return v;
}

}  // namespace gqa
