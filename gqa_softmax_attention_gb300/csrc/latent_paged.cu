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
// j <= i + L_b - Sq_b.  NR rows (16, 32 or 64) go to one CTA; a team of one or two
// CTAs takes the rows [seg * team * NR, ...) of a request and reads the same keys
// at the same time, so that the second reading comes from L2.
//
// The products are formed transposed, keys and dims on the MMAs' M side and the
// rows on N, because O of 512 dims by 64 rows then takes half of TMEM (as O
// itself it would take all of it, whatever the row count):
//   S^T [64 keys, NR]   = K [64, 576] Q^T            36 MMAs of K = 16
//   O^T [512 dims, NR] += V^T [512, 64 keys] P^T     4 x 4 MMAs
// A cache tile lies in shared memory once and is both operands: K-major for
// S^T, dims-major (transposed) for O^T.  MMAs with so few columns are bound by
// reading their A operand from shared memory (128 bytes a cycle: 33 and 49 cycles
// a step at 64 rows, 24 and 40 at 16; measured), 2000 or 1500 cycles a tile where
// HBM brings one every 3200.
//
// Shared memory holds Q (72 KB at 64 rows) and two to two and a half tiles of 72 KB: a
// ring of slots of 256 dims, two a tile, and one of the 64 shared dims.  P^T is
// written over the shared dims, which only S^T needs.  (Slots of 128 dims took the
// producer five hand-overs of 400 cycles a tile, 700 with pages of 16.)  With one tile of 128 keys at a
// time the loads of a tile could not run while the tile before was worked on, and
// all CTAs loaded and all computed at the same time (64 requests of 1K to 16K
// keys, 16 heads: 188 us).
//   warps 0-3  softmax; the output
//   warps 4, 5 MMA issuers of S^T, which runs up to a tile ahead, and of O^T, an elected
//              lane each: the tensor core takes whichever is ready
//   warp 6     producer (TMA), or warps 6-7 (rows gathered)
// A softmax thread owns a key and half of the rows.  The reference maximum of a row
// (column) is kept in shared memory and moves only when a score exceeds it by more
// than 2^8, which the threads vote on; the row sums are kept as per-thread parts
// and joined across the keys once per piece.
//
// Work is balanced: the row groups of all requests, laid end to end, form one
// sequence of 64-key tiles, and each team takes an equal range.  A row group
// that lies in one range is written out directly; of one that is cut, each
// piece leaves O, maximum and sum in FP32, at most two pieces a team, and
// latent_join_kernel adds them up.
//
// Measured (bf16, pages of 64, queries of one token): 64 requests of 1K to 16K keys
// take 104 to 112 us with 16 heads (625 MB once: 83 to 90 % of the copy rate) and 171 to 185 us
// with 128 heads (860 TFLOP/s), which the chain of a tile's loads, S^T, softmax and O^T through
// a ring two tiles deep bounds: 2450 cycles a tile where its MMAs read operands for 1970.
// Replayed from a graph: two requests of 300 to 700 keys 11 us; 64 of 1K to 16K, 16 heads, 91,
// and 176 in pages of one token, gathered.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cmath>
#include <type_traits>

#include "internal.h"
#include "ptx.cuh"

namespace gqa {
namespace {

__device__ int g_latent_paged_error;

constexpr int BN = 64;                     // keys per tile
constexpr int DC = kLatentDim;             // 512: latent
constexpr int DR = kLatentRope;            // 64: shared rotated dims
constexpr int DK = DC + DR;
constexpr int ROW_BYTES = DK * 2;
constexpr int NJ = DC / 128;               // 128-dim blocks of O^T (pairs of 64-dim slices)
constexpr int NU = 2;                      // slots of latents a tile takes: 256 dims, 4 slices, 2 blocks each
constexpr float kLn2 = 0.693147180559945309f;
constexpr float kRescaleThreshold = 8.f;
constexpr int WARP_S = 4, WARP_O = 5;      // MMA issuers of S^T and of O^T
constexpr int WARP_LOAD = 6;
constexpr int kSmBar = 1;                  // named barrier of the softmax warps

template <int NR, bool GATHER>
struct LCfg {
    static constexpr int NP = NR == 64 ? 4 : 5;                    // slots of 256 dims, NU a tile
    static constexpr int NT = NR == 64 ? 2 : 3;                    // slots of the shared dims, one a tile
    static constexpr int HALF = BN * 512;                          // [8 groups][4 slices][8 keys][128 bytes]
    static constexpr int ROPE = BN * 128;                          // shared dims, later P^T: [64 keys][128 bytes]
    static constexpr int Q_SLICE = NR * 128;                       // 64 dims of Q
    static constexpr int OFF_Q = 0;
    static constexpr int OFF_P = OFF_Q + (DK / 64) * Q_SLICE;
    static constexpr int OFF_KV = OFF_P + NT * ROPE;
    static constexpr int OFF_COL = OFF_KV + NP * HALF;             // per row: -reference, factor, limit, reference, [4] per warp
    static constexpr int OFF_BAR = OFF_COL + 8 * NR * 4;
    // kv_full[NP], kv_empty[NP], q_full, q_empty, drain[2], s_full[2], p_full[2]
    static constexpr int NBAR = 2 * NP + 8;
    static constexpr int OFF_MISC = OFF_BAR + NBAR * 8;
    static constexpr int SMEM_BYTES = OFF_MISC + 64 + 1024;
    static constexpr int LOAD_WARPS = GATHER ? 2 : 1;
    static constexpr int THREADS = 32 * (WARP_LOAD + LOAD_WARPS);
    static constexpr uint32_t COL_S = NJ * NR;                     // TMEM: O^T blocks | S^T of even, of odd tiles
    static constexpr uint32_t TMEM_COLS = 512;
    static_assert(COL_S + 2 * NR <= TMEM_COLS, "TMEM budget");
    // The shared dims' slot of a tile is free when its second slot of latents is: that one
    // was last used by a tile that came after the shared dims' last one, or with it.
    static_assert((NP == 4 && NT == 2) || (NP == 5 && NT == 3), "slots that come free together");
    static_assert(kLatentMaxB * 8 <= NP * HALF, "prefix sums over the ring");
    static_assert(OFF_KV % 1024 == 0 && OFF_P % 1024 == 0, "swizzle atoms");
    static_assert(SMEM_BYTES <= 227 * 1024, "shared memory budget");
};

// Where this team's range of the tile sequence starts.
struct LRange {
    long g0, n, per;        // first place, places, places per team (key and start tiles)
    int b, seg, off, pad;   // request and row group of the first one, and its place in that
};

__device__ __forceinline__ int request_len(const LatentArgs& a, int b) {
    return (int)min((long)max(a.lens[b], 0), (long)a.max_pages * a.page_size);
}
__device__ __forceinline__ void request_rows(const LatentArgs& a, int b, int& qs, int& sq) {
    qs = min(max(a.cu_q[b], 0), a.total_q);
    sq = min(max(a.cu_q[b + 1], qs), a.total_q) - qs;
}

// A row group counts kStartTiles tiles more than it has: a piece's start and end cost a
// team about as much (4 us at 64 rows a CTA, 2.6 at 16, where a tile takes 1.2 and 1.4),
// and a range of many short row groups would take longer than one of a single long one
// (64 requests of 1K to 16K keys, 128 heads, none counted: ranges of four pieces ended
// 24 us after those of one, of 155).  23 drafts and 9 steps of 40 heads: 73 us with 1, 68
// with 2, 65 with 3, 62 to 66 with 4; 24 chunks of 4 queries by 64 heads 91, 86 and 87
// with 2 to 4.
constexpr int kStartTiles = 3;

// A stretch of one row group's tiles, and the walk over those of a range.
struct Piece {
    int b, seg, nseg, nt;    // request, row group, its groups, tiles of each
    int qs, sq, L;
    int lt0, lt1;            // tiles [lt0, lt1) of the row group
    long at;                 // place of the row group's first tile in the sequence
    long pos, left;          // place of the next tile, tiles of the range from there on (start tiles included)
    int row0, rows;          // this CTA's rows (of the request's sq * H)
    int n;                   // tiles from lt0 on with a key that one of its rows sees
    __device__ __forceinline__ void request(const LatentArgs& a, int rb, int group) {
        b = rb;
        request_rows(a, b, qs, sq);
        L = request_len(a, b);
        nseg = (sq * a.H + group - 1) / group;
        nt = max(1, (L + BN - 1) / BN);
    }
    __device__ __forceinline__ bool whole() const { return lt0 == 0 && lt1 == nt; }
    // The stretch from place `off` of the row group on; false: none but start tiles.
    __device__ __forceinline__ bool fit(const LatentArgs& a, long off, int group, int nr, int rank) {
        const long end = min((long)nt + kStartTiles, off + left);
        at = pos - off + kStartTiles;
        pos += end - off;
        left -= end - off;
        lt0 = (int)max(0L, off - kStartTiles);
        lt1 = (int)max(0L, end - kStartTiles);
        row0 = seg * group + rank * nr;
        rows = min(nr, sq * a.H - row0);
        n = 0;
        if (rows > 0) {
            const int i_last = (row0 + rows - 1) / a.H;
            const int lim = a.causal ? max(0, min(L, L - sq + i_last + 1)) : L;
            n = max(0, min(lt1, (lim + BN - 1) / BN) - lt0);
        }
        return lt1 > lt0;
    }
    __device__ __forceinline__ bool first(const LatentArgs& a, const LRange& r, int group, int nr, int rank) {
        request(a, r.b, group);
        seg = r.seg;
        pos = r.g0;
        left = r.n;
        return fit(a, r.off, group, nr, rank);
    }
    __device__ __forceinline__ bool next(const LatentArgs& a, int group, int nr, int rank) {
        if (left <= 0) return false;
        if (++seg >= nseg) {
            seg = 0;
            do {
                if (b + 1 >= a.B) return false;
                request(a, b + 1, group);
            } while (nseg == 0);
        }
        return fit(a, 0, group, nr, rank);
    }
};

// Sums or maxima of v[0 .. N) over the 16 lanes of a half-warp: lane l returns the
// columns l * N / 16 .. of them in v[0 .. max(1, N / 16)) (N = 8: lanes 2c and 2c + 1
// column c).  Each step exchanges the half of the columns that the other lanes keep.
template <int N, bool MAX>
__device__ __forceinline__ void half_warp_columns(float* v, int lane) {
    static_assert(N == 32 || N == 16 || N == 8, "columns");
    auto both = [](float x, float y) { return MAX ? fmaxf(x, y) : x + y; };
#pragma unroll
    for (int o = 8, w = N / 2; o >= 1; o >>= 1, w >>= 1) {
        const bool up = (lane & o) != 0;
#pragma unroll
        for (int i = 0; i < N / 2; ++i) {
            if (i < w) {
                const float mine = up ? v[i + w] : v[i], other = up ? v[i] : v[i + w];
                v[i] = both(mine, __shfl_xor_sync(0xffffffffu, other, o));
            }
        }
        if (w == 0) v[0] = both(v[0], __shfl_xor_sync(0xffffffffu, v[0], o));
    }
}

// 16 lanes x 2 N columns of TMEM -> N registers per thread, lanes l and l + 16 of
// the warp reading columns 0 .. N - 1 and N .. 2 N - 1 of TMEM lane l (the rows
// of an M = 64 accumulator lie in the first 16 lanes of each warp's quarter).
// The caller waits.
template <int N>
__device__ __forceinline__ void tmem_ld_half(uint32_t taddr, float* v) {
    uint32_t* r = reinterpret_cast<uint32_t*>(v);
    if constexpr (N == 32) {
        asm volatile(
            "tcgen05.ld.sync.aligned.16x32bx2.x32.b32 "
            "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
            "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32], 32;"
            : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
              "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
              "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]),
              "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]),
              "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
            : "r"(taddr)
            : "memory");
    } else if constexpr (N == 16) {
        asm volatile(
            "tcgen05.ld.sync.aligned.16x32bx2.x16.b32 "
            "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16], 16;"
            : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
              "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
              "=r"(r[14]), "=r"(r[15])
            : "r"(taddr)
            : "memory");
    } else {
        asm volatile("tcgen05.ld.sync.aligned.16x32bx2.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8], 8;"
                     : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                     : "r"(taddr)
                     : "memory");
    }
}

// o / sum: exact zeros for a row without a key (whose O^T may hold anything)
__device__ __forceinline__ float scaled(float o, float factor) { return factor != 0.f ? o * factor : 0.f; }

// n / page_size for 0 <= n < 2^31
__device__ __forceinline__ int page_of(const LatentArgs& a, uint32_t n) {
    return (int)((__umulhi(n, a.ps_mul) + n) >> a.ps_shift);
}

template <int NR, bool F16, bool GATHER>
__global__ void __launch_bounds__((LCfg<NR, GATHER>::THREADS), 1)
latent_paged_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_kv,
                    const __grid_constant__ CUtensorMap tm_pe, const __grid_constant__ CUtensorMap tm_row, const LatentArgs a) {
    using C = LCfg<NR, GATHER>;
    constexpr uint32_t IDESC_S = make_idesc_16<F16>(BN, NR, false, false);
    constexpr uint32_t IDESC_O = make_idesc_16<F16>(128, NR, true, true);
    griddep_launch_dependents();                 // the joining kernel may be scheduled (it waits for this grid)

    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    uint8_t* smem = smem_raw + ((1024 - (raw & 1023)) & 1023);
    const uint32_t sb = smem_u32(smem);
    // through a shuffle, so that the compiler knows the roles' branches to be uniform
    // and keeps descriptors and addresses in uniform registers
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x / 32, 0), lane = threadIdx.x % 32;
    const int team = blockIdx.x / a.team, rank = blockIdx.x % a.team;
    const int group = a.team * NR;               // rows of a team

    const uint32_t bar0 = sb + C::OFF_BAR;
    auto kv_full = [&](int i) { return bar0 + 8u * i; };
    auto kv_empty = [&](int i) { return bar0 + 8u * (C::NP + i); };
    const uint32_t bar1 = bar0 + 8u * (2 * C::NP);
    const uint32_t q_full = bar1, q_empty = bar1 + 8;
    auto drain = [&](int i) { return bar1 + 16 + 8u * i; };
    auto s_full = [&](int i) { return bar1 + 32 + 8u * i; };
    auto p_full = [&](int i) { return bar1 + 48 + 8u * i; };
    // Tile it's latents are units u = NU it, NU it + 1 of the ring: use u / NP of slot
    // u % NP; its shared dims, and P^T later, lie in slot it % NT and are loaded with the
    // second unit.  A fill's parity is its use's.
    auto slot_addr = [&](int i) { return sb + C::OFF_KV + (uint32_t)i * C::HALF; };
    auto rope_addr = [&](int i) { return sb + C::OFF_P + (uint32_t)i * C::ROPE; };
    // Whether O^T holds tile it: its second unit's slot has been released.
    auto tile_done = [&](int it, volatile int* abort) {
        const uint32_t u = (uint32_t)(NU * it + 1);
        return mbar_wait(kv_empty((int)(u % C::NP)), u / C::NP & 1, abort);
    };
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::OFF_MISC);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::OFF_MISC + 4);
    LRange* range = reinterpret_cast<LRange*>(smem + C::OFF_MISC + 16);

    if (threadIdx.x == 0) {
        const int fills = GATHER ? 32 * C::LOAD_WARPS : 1;
        for (int i = 0; i < C::NP; ++i) { mbar_init(kv_full(i), fills); mbar_init(kv_empty(i), 1); }
        for (int i = 0; i < 2; ++i) { mbar_init(s_full(i), 1); mbar_init(p_full(i), 128); mbar_init(drain(i), 1); }
        mbar_init(q_full, 1);
        mbar_init(q_empty, 1);
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
                x = (long)p.nseg * (p.nt + kStartTiles);
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
        if (per < a.min_places) per = a.min_places;
        const long g0 = team * per, n = max(0L, min(per, base - g0));
        if (n > 0) {
            for (int b = threadIdx.x; b < a.B; b += C::THREADS) {
                const long lo = pre[b], hi = b + 1 < a.B ? pre[b + 1] : base;
                if (lo <= g0 && g0 < hi) {
                    Piece p;
                    p.request(a, b, group);
                    const int each = p.nt + kStartTiles;
                    *range = LRange{g0, n, per, b, (int)((g0 - lo) / each), (int)((g0 - lo) % each), 0};
                }
            }
        }
    }
    if (warp == WARP_S) {
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
        int nq = 0;                              // Q blocks loaded
        int ps = 0, ts = 0;                      // next slots, and the parity of the use of ps
        uint32_t pp = 0, units = 0;
        bool ok = true;
        Piece p;
        bool more = p.first(a, rg, group, NR, rank);
        auto step = [&](int u) {                 // past unit u of a tile
            ++units;
            if (++ps == C::NP) { ps = 0; pp ^= 1; }
            if (u == NU - 1 && ++ts == C::NT) ts = 0;
        };
        // The piece's Q rows, once the last S^T of the piece before is done (one lane).
        auto load_q = [&]() {
            if (!mbar_wait(q_empty, (nq & 1) ^ 1, abort_flag)) return false;
            mbar_arrive_expect_tx(q_full, (DK / 64) * C::Q_SLICE);
            tma_load_3d(sb + C::OFF_Q, &tm_q, q_full, 0, p.qs * a.H + p.row0, 0);
            return true;
        };
        if constexpr (!GATHER) {
            // Page blocks of a tile: 8-row groups of the cache as one box of 256 dims a
            // unit, and one of the shared dims; a block past the request's end or of a
            // page outside the pool lies outside the map and comes as zeros.  One elected
            // lane does it all: as a whole warp, which meets at every wait, it fell into a
            // slow state at some row groups' starts (800 cycles a copy for 200).
            // NB: blocks of a tile, or the most there can be.
            auto run = [&](auto blocks) {
                constexpr int NB = decltype(blocks)::value;
                const int bt = a.box_tokens, nbox = NB == 1 ? 1 : BN / bt;
                const int outside = a.num_pages * (a.page_size / 8);
                for (; more && ok; more = p.next(a, group, NR, rank)) {
                    if (p.n == 0) continue;
                    const int32_t* table = a.table + (size_t)p.b * a.max_pages;
                    // page ids of tile k's blocks as the table has them (-1 past the request's end)
                    auto pages = [&](int k, int (&pg)[NB]) {
#pragma unroll
                        for (int i = 0; i < NB; ++i) {
                            const int t = (p.lt0 + k) * BN + i * bt;
                            pg[i] = -1;
                            if (k < p.n && i < nbox && t < p.L) pg[i] = ldg_int(table + page_of(a, (uint32_t)t));
                        }
                    };
                    auto groups = [&](int k, const int (&pg)[NB], int (&gr)[NB]) {
#pragma unroll
                        for (int i = 0; i < NB; ++i) {
                            const int t = (p.lt0 + k) * BN + i * bt;
                            const int in_page = t - page_of(a, (uint32_t)t) * a.page_size;
                            gr[i] = pg[i] >= 0 && pg[i] < a.num_pages ? (int)(((long)pg[i] * a.page_size + in_page) >> 3)
                                                                      : outside;
                        }
                    };
                    // tiles k, k + 1, k + 2; a tile is brought to L2 two tiles before its slots come free
                    int g0[NB], g1[NB], g2[NB], pg[NB];
                    pages(0, pg);
                    pages(1, g1);
                    pages(2, g2);
                    if (!(ok = load_q())) break;
                    ++nq;
                    groups(0, pg, g0);
                    groups(1, g1, g1);
#pragma unroll
                    for (int i = 0; i < NB; ++i) pg[i] = g2[i];
                    for (int k = 0; k < p.n && ok; ++k) {
                        groups(k + 2, pg, g2);
                        pages(k + 3, pg);
#pragma unroll
                        for (int u = 0; u < NU; ++u) {
                            if (!(ok = mbar_wait(kv_empty(ps), pp ^ 1, abort_flag))) break;
                            const uint32_t full = kv_full(ps), dst = slot_addr(ps), dst_pe = rope_addr(ts);
                            mbar_arrive_expect_tx(full, C::HALF + (u == NU - 1 ? C::ROPE : 0));
#pragma unroll
                            for (int i = 0; i < NB; ++i) {
                                if (i < nbox) {
                                    tma_load_4d(dst + i * bt * 512, &tm_kv, full, 0, 0, 4 * u, g0[i]);
                                    if (u == NU - 1) tma_load_4d(dst_pe + i * bt * 128, &tm_pe, full, 0, 0, 4 * NU, g0[i]);
                                }
                            }
                            step(u);
                        }
                        if (rank == 0) {
#pragma unroll
                            for (int i = 0; i < NB; ++i)
                                if (i < nbox && g2[i] != outside) tma_prefetch_4d(&tm_row, 0, 0, 0, g2[i]);
                        }
#pragma unroll
                        for (int i = 0; i < NB; ++i) {
                            g0[i] = g1[i];
                            g1[i] = g2[i];
                        }
                    }
                }
                if (*abort_flag) {
                    // let the copies in flight land: the last fill of each slot
                    for (uint32_t u = units < C::NP ? 0 : units - C::NP; u != units; ++u)
                        mbar_drain(kv_full((int)(u % C::NP)), u / C::NP & 1);
                    if (nq > 0) mbar_drain(q_full, (nq - 1) & 1);
                }
            };
            if (elect_one()) {
                tma_prefetch_desc(&tm_q);
                tma_prefetch_desc(&tm_kv);
                tma_prefetch_desc(&tm_pe);
                tma_prefetch_desc(&tm_row);
                if (a.box_tokens == BN) run(std::integral_constant<int, 1>{});
                else run(std::integral_constant<int, BN / 8>{});
            }
            __syncwarp();
        } else {
            for (; more && ok; more = p.next(a, group, NR, rank)) {
                if (p.n == 0) continue;
                if (pw == 0) {
                    if (lane == 0) ok = load_q();
                    ok = __shfl_sync(0xffffffffu, ok, 0);
                    if (!ok) break;
                    ++nq;
                }
                // Rows one by one: a warp copies 32 of them, 512 bytes at a time; a slot is
                // announced once the copies of the next one are under way, or at once where
                // the next slot is not free yet.
                uint32_t pending = 0;
                auto announce = [&]() {
                    if (pending) {
                        fence_proxy_async_smem();
                        mbar_arrive(pending);
                        pending = 0;
                    }
                };
                auto row_of = [&](int k) {       // cache row of this lane's key of tile k, -1 for zeros
                    const int t = (p.lt0 + k) * BN + pw * 32 + lane;
                    const int lp = page_of(a, (uint32_t)t);
                    const int page = t < p.L ? ldg_int(a.table + (size_t)p.b * a.max_pages + lp) : -1;
                    return page >= 0 && page < a.num_pages ? page * a.page_size + (t - lp * a.page_size) : -1;
                };
                int row = row_of(0);
                for (int k = 0; k < p.n && ok; ++k) {
                    const int now = row;
                    if (k + 1 < p.n) row = row_of(k + 1);
#pragma unroll
                    for (int u = 0; u < NU; ++u) {
                        if (!__all_sync(0xffffffffu, mbar_test_wait(kv_empty(ps), pp ^ 1))) {
                            cp_async_wait<0>();
                            announce();
                            ok = __all_sync(0xffffffffu, mbar_wait(kv_empty(ps), pp ^ 1, abort_flag));
                            if (!ok) break;
                        }
                        const uint32_t dst = slot_addr(ps), dst_pe = rope_addr(ts);
#pragma unroll 4
                        for (int e = 0; e < 32; ++e) {
                            const int r = __shfl_sync(0xffffffffu, now, e), key = pw * 32 + e;
                            const char* src = static_cast<const char*>(a.cache) + (size_t)max(r, 0) * ROW_BYTES + u * 512 +
                                              lane * 16;
                            cp_async16(dst + (key >> 3) * 4096 + (lane / 8) * 1024 + (key & 7) * 128 +
                                           (((lane % 8) ^ (key & 7)) << 4), src, r >= 0 ? 16 : 0);
                        }
                        if (u == NU - 1) {
#pragma unroll 4
                            for (int e = 0; e < 8; ++e) {
                                const int r = __shfl_sync(0xffffffffu, now, 4 * e + lane / 8), key = pw * 32 + 4 * e + lane / 8;
                                const char* src = static_cast<const char*>(a.cache) + (size_t)max(r, 0) * ROW_BYTES +
                                                  NU * 512 + (lane % 8) * 16;
                                cp_async16(dst_pe + key * 128 + (((lane % 8) ^ (key & 7)) << 4), src, r >= 0 ? 16 : 0);
                            }
                        }
                        cp_async_commit();
                        if (pending) {
                            cp_async_wait<1>();
                            announce();
                        }
                        pending = kv_full(ps);
                        step(u);
                    }
                }
                cp_async_wait<0>();
                announce();
            }
            if (*abort_flag && pw == 0 && lane == 0 && nq > 0) mbar_drain(q_full, (nq - 1) & 1);
        }
    } else if (warp == WARP_S) {
        // ------------------------------------------------------------ S^T issuer (one elected lane)
        if (elect_one()) {
            Piece p;
            bool more = p.first(a, rg, group, NR, rank);
            int it = 0, nq = 0, ps = 0, ts = 0;  // tile, Q blocks taken, slots and the parity of the use of ps
            uint32_t pp = 0;
            bool ok = true;
            const uint64_t qdesc = make_sdesc_sw128(sb + C::OFF_Q, 16, 1024);
            // K-major A: 8-key groups 4 KB apart (1 KB in the shared dims' slot)
            const uint64_t kdesc0 = make_sdesc_sw128(sb + C::OFF_KV, 16, 4096), edesc0 = make_sdesc_sw128(sb + C::OFF_P, 16, 1024);
            for (; more && ok; more = p.next(a, group, NR, rank)) {
                for (int k = 0; k < p.n && ok; ++k, ++it) {
                    if (k == 0) ok = mbar_wait(q_full, nq & 1, abort_flag);
                    // at most one tile ahead of O^T, so that no barrier runs two phases ahead
                    // of who waits on it: the tile before the last is done, and its S^T read
                    if (ok && it > 1) ok = tile_done(it - 2, abort_flag);
                    const uint32_t d = tmem + C::COL_S + (it & 1) * NR;
                    tc_fence_after();
#pragma unroll
                    for (int u = 0; u < NU; ++u) {
                        if (ok) ok = mbar_wait(kv_full(ps), pp, abort_flag);
                        if (!ok) break;
                        const uint64_t kdesc = desc_at(kdesc0, ps * C::HALF);
#pragma unroll
                        for (int kk = 0; kk < 16; ++kk)
                            mma_bf16_ss(d, desc_at(kdesc, (kk / 4) * 1024 + (kk % 4) * 32),
                                        desc_at(qdesc, (4 * u + kk / 4) * C::Q_SLICE + (kk % 4) * 32), IDESC_S,
                                        (u > 0 || kk > 0) ? 1u : 0u);
                        if (++ps == C::NP) { ps = 0; pp ^= 1; }
                    }
                    if (!ok) break;
                    const uint64_t edesc = desc_at(edesc0, ts * C::ROPE);
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)
                        mma_bf16_ss(d, desc_at(edesc, kk * 32), desc_at(qdesc, 4 * NU * C::Q_SLICE + kk * 32), IDESC_S, 1u);
                    mma_commit(s_full(it & 1));
                    if (k == p.n - 1) {
                        mma_commit(q_empty);
                        ++nq;
                    }
                    if (++ts == C::NT) ts = 0;
                }
            }
            mma_commit(drain(0));                // every MMA issued above has completed once this arrives
            mbar_drain(drain(0), 0);
        }
        __syncwarp();
    } else if (warp == WARP_O) {
        // ------------------------------------------------------------ O^T issuer (one elected lane)
        if (elect_one()) {
            Piece p;
            bool more = p.first(a, rg, group, NR, rank);
            int it = 0, ps = 0, ts = 0;
            bool ok = true;
            // dims-major A: 64-dim slices 1 KB apart, 8-key groups 4 KB apart
            const uint64_t vdesc0 = make_sdesc_sw128(sb + C::OFF_KV, 1024, 4096), pdesc0 = make_sdesc_sw128(sb + C::OFF_P, 1024, 1024);
            for (; more && ok; more = p.next(a, group, NR, rank)) {
                for (int k = 0; k < p.n; ++k, ++it) {
                    ok = mbar_wait(p_full(it & 1), (it >> 1) & 1, abort_flag);
                    if (!ok) break;
                    tc_fence_after();
                    const uint64_t pdesc = desc_at(pdesc0, ts * C::ROPE);
#pragma unroll
                    for (int u = 0; u < NU; ++u) {
                        const uint64_t vdesc = desc_at(vdesc0, ps * C::HALF);
#pragma unroll
                        for (int j = 0; j < NJ / NU; ++j) {
#pragma unroll
                            for (int kk = 0; kk < BN / 16; ++kk)
                                mma_bf16_ss(tmem + (u * (NJ / NU) + j) * NR, desc_at(vdesc, j * 2048 + kk * 8192),
                                            desc_at(pdesc, kk * 2048), IDESC_O, (k > 0 || kk > 0) ? 1u : 0u);
                        }
                        mma_commit(kv_empty(ps));
                        if (++ps == C::NP) ps = 0;
                    }
                    if (++ts == C::NT) ts = 0;
                }
            }
            mma_commit(drain(1));
            mbar_drain(drain(1), 0);
        }
        __syncwarp();
    } else {
        // ------------------------------------------------------------ softmax warps 0-3
        constexpr int HC = NR / 2;               // rows (columns of S^T) of a thread
        // A float16 P below 2^-14 rounds to a multiple of 2^-24.  The reference stands six
        // binades below the maximum, so that a weight is off by 2^-31 of the strongest at most
        // (from the maximum itself 16383 keys 26 binades below one would lose their share).
        constexpr float kLead = F16 ? 6.f : 0.f, kMost = kRescaleThreshold + kLead;
        const int row = threadIdx.x;             // this thread's row, where rows are meant
        const int key = warp * 16 + lane % 16, c0 = (lane / 16) * HC;   // its key of a tile and first column
        const uint32_t lane_addr = (uint32_t)(warp * 32) << 16;
        float* neg_ref = reinterpret_cast<float*>(smem + C::OFF_COL);   // -reference maximum (0 while there is none)
        float* factor = neg_ref + NR;                                   // rescale factor of the last move; 1 / sum
        int* limit = reinterpret_cast<int*>(neg_ref + 2 * NR);          // keys that the row sees
        float* ref = neg_ref + 3 * NR;                                  // reference maximum, -inf while there is none
        float* cross = neg_ref + 4 * NR;                                // [4][NR]: per warp
        const float sl = a.scale_log2;
        Piece p;
        bool more = p.first(a, rg, group, NR, rank), ok = true, at_start = true;
        int it = 0, sv = 0, tv = 0;              // tile; its slots
        // Columns of a half-warp's result (half_warp_columns): this lane's first one, and how many.
        constexpr int OWN = HC >= 16 ? HC / 16 : 1;
        const int own = c0 + (HC >= 16 ? (lane % 16) * OWN : (lane % 16) / 2);
        // A wait that gave up (ok false) ends the work but not the walk: all four
        // warps pass the same named barriers to the end.
        while (more) {
            const bool whole = p.whole();
            int lim_all = 0;
            if (p.rows > 0) {
                // row r of the block is query (row0 + r) / H; blocks cut short see what their last row sees
                auto lim_of = [&](int r) {
                    const int i = (p.row0 + min(r, p.rows - 1)) / a.H;
                    return a.causal ? max(0, min(p.L, p.L - p.sq + i + 1)) : p.L;
                };
                lim_all = lim_of(0);             // every row sees the keys below
                if (row < NR) {
                    limit[row] = lim_of(row);
                    neg_ref[row] = 0.f;
                    ref[row] = -INFINITY;
                }
            }
            named_bar_sync(kSmBar, 128);
            bool unset = false;                  // this row has seen infinite scores alone so far
            float sums[HC];
#pragma unroll
            for (int c = 0; c < HC; ++c) sums[c] = 0.f;
            for (int k = 0; k < p.n; ++k, ++it) {
                const int t = (p.lt0 + k) * BN + key;
                const bool all_seen = (p.lt0 + k + 1) * BN <= lim_all;
                if (ok) ok = __all_sync(0xffffffffu, mbar_wait(s_full(it & 1), (it >> 1) & 1, abort_flag));
                tc_fence_after();
                float s[HC];
                auto load = [&]() {              // scores in log2 units against the rows' references; hidden ones -inf
                    tmem_ld_half<HC>(tmem + lane_addr + C::COL_S + (it & 1) * NR, s);
                    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
                    for (int c = 0; c < HC; c += 4) {
                        const float4 nr = *reinterpret_cast<const float4*>(neg_ref + c0 + c);
                        s[c] = fmaf(s[c], sl, nr.x);
                        s[c + 1] = fmaf(s[c + 1], sl, nr.y);
                        s[c + 2] = fmaf(s[c + 2], sl, nr.z);
                        s[c + 3] = fmaf(s[c + 3], sl, nr.w);
                    }
                    if (!all_seen) {
#pragma unroll
                        for (int c = 0; c < HC; c += 4) {
                            const int4 li = *reinterpret_cast<const int4*>(limit + c0 + c);
                            s[c] = t < li.x ? s[c] : -INFINITY;
                            s[c + 1] = t < li.y ? s[c + 1] : -INFINITY;
                            s[c + 2] = t < li.z ? s[c + 2] : -INFINITY;
                            s[c + 3] = t < li.w ? s[c + 3] : -INFINITY;
                        }
                    }
                };
                load();
                float top = -INFINITY;
#pragma unroll
                for (int c = 0; c < HC; c += 2) top = fmax3(top, s[c], s[c + 1]);
                // The first tile gives every row that sees a key its reference (unless all
                // its scores are -inf); a row that sees none there sees none in later tiles.
                const bool keep = named_bar_and(kSmBar, 128, ok && k > 0 && !unset && !(top > kMost));
                if (!keep) {
                    // column maxima over the tile's keys
                    half_warp_columns<HC, true>(s, lane);
#pragma unroll
                    for (int e = 0; e < OWN; ++e) cross[warp * NR + own + e] = s[e];
                    named_bar_sync(kSmBar, 128);
                    if (row < NR) {
                        const float d = fmaxf(fmaxf(cross[row], cross[NR + row]), fmaxf(cross[2 * NR + row], cross[3 * NR + row]));
                        const float old = ref[row];
                        float f = 1.f;
                        if (old == -INFINITY || d > kMost) {
                            const float m = d - neg_ref[row] - kLead;     // neg_ref is 0 while there is no reference
                            f = old == -INFINITY ? 0.f : fast_exp2(old - m);
                            ref[row] = m;
                            neg_ref[row] = m == -INFINITY ? 0.f : -m;
                            // (no reference, and the row sees keys of the next tile)
                            unset = m == -INFINITY && limit[row] > (p.lt0 + k + 1) * BN;
                        }
                        factor[row] = f;
                    }
                    named_bar_sync(kSmBar, 128);
                    load();
                    if (k > 0 && ok) {
                        // O^T has to hold the tile before
                        if (ok) ok = __all_sync(0xffffffffu, tile_done(it - 1, abort_flag));
                        tc_fence_after();
#pragma unroll
                        for (int c = 0; c < HC; ++c) sums[c] *= factor[c0 + c];
                        if (ok) {
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
                }
                // P^T: row = key, 128 bytes with the 128-byte swizzle
                const uint32_t prow = rope_addr(tv) + key * 128;
#pragma unroll
                for (int c = 0; c < HC; c += 8) {
                    uint32_t w[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float p0 = fast_exp2(s[c + 2 * e]), p1 = fast_exp2(s[c + 2 * e + 1]);
                        sums[c + 2 * e] += p0;
                        sums[c + 2 * e + 1] += p1;
                        w[e] = pack2<F16>(p0, p1);
                    }
                    if (ok) st_shared_v4(prow + ((((c0 + c) / 8) ^ (key & 7)) << 4), w[0], w[1], w[2], w[3]);
                }
                if (++tv == C::NT) tv = 0;
                for (int u = 0; u < NU; ++u) {
                    if (t >= p.L && ok) {
                        // a row past the request's end: whatever the page holds there must not
                        // reach O^T (two slices for each of the key's two threads)
                        const uint32_t v = slot_addr(sv) + (key >> 3) * 4096 + (lane / 16) * 2048 + (key & 7) * 128;
                        for (int c = 0; c < 256; c += 16) st_shared_v4(v + (c >> 7) * 1024 + (c & 127), 0u, 0u, 0u, 0u);
                    }
                    if (++sv == C::NP) sv = 0;
                }
                fence_proxy_async_smem();
                tc_fence_before();
                if (ok) mbar_arrive(p_full(it & 1));
            }
            // ---- the piece's end; the next one is looked up while O^T comes to an end
            __syncwarp();
            Piece nx = p;
            more = nx.next(a, group, NR, rank);
            if (ok && p.n > 0) {
                ok = __all_sync(0xffffffffu, tile_done(it - 1, abort_flag));
                tc_fence_after();
            }
            half_warp_columns<HC, false>(sums, lane);
#pragma unroll
            for (int e = 0; e < OWN; ++e) cross[warp * NR + own + e] = sums[e];
            ok = named_bar_and(kSmBar, 128, ok);
            if (p.rows > 0) {
                const long orow = (long)p.qs * a.H + p.row0;       // first row of the block in [total_q * H]
                if (row < NR) {
                    const float m = ref[row];
                    const float l = (cross[row] + cross[NR + row]) + (cross[2 * NR + row] + cross[3 * NR + row]);
                    const bool some = p.n > 0 && l != 0.f;         // 0: no key; NaN goes on
                    if (whole) {
                        factor[row] = some ? 1.f / l : 0.f;
                        if (row < p.rows && a.lse) a.lse[orow + row] = some ? (m + log2f(l)) * kLn2 : -INFINITY;
                    } else {
                        const size_t id = 2 * (size_t)blockIdx.x + (at_start ? 0 : 1);
                        a.part_ml[id * NR + row] = some ? make_float2(m, l) : make_float2(-INFINITY, 0.f);
                    }
                }
                named_bar_sync(kSmBar, 128);
                if (whole) {
                    // O^T [dim, row] / sum -> [row, dim].  A lane has one dim of 32 rows; in
                    // three exchanges eight lanes turn 8 dims x 32 rows of 16 bits so that
                    // each holds 8 dims of 4 rows, which go out 16 bytes at a time (4-byte
                    // stores after the first exchange took 6.6 us for 64 rows, 24 cycles each).
                    char* out = static_cast<char*>(a.o) + (orow * DC + warp * 32 + (lane & 24)) * 2;
#pragma unroll 1
                    for (int c = 0; c < NJ * NR; c += 32) {
                        float o[32];
                        __syncwarp();
                        if (p.n > 0) {
                            tmem_ld32(tmem + lane_addr + c, o);
                        } else {
#pragma unroll
                            for (int e = 0; e < 32; ++e) o[e] = 0.f;
                        }
                        uint32_t v[16];
#pragma unroll
                        for (int e = 0; e < 32; e += 4) {
                            const float4 f = *reinterpret_cast<const float4*>(factor + (c + e) % NR);
                            v[e / 2] = pack2<F16>(scaled(o[e], f.x), scaled(o[e + 1], f.y));
                            v[e / 2 + 1] = pack2<F16>(scaled(o[e + 2], f.z), scaled(o[e + 3], f.w));
                        }
                        const bool b0 = lane & 1, b1 = lane & 2, b2 = lane & 4;
#pragma unroll
                        for (int e = 0; e < 16; ++e) {       // (rows 2e, 2e + 1; dim) -> (row 2e + b0; two dims)
                            const uint32_t x = __shfl_xor_sync(0xffffffffu, v[e], 1);
                            v[e] = b0 ? __byte_perm(x, v[e], 0x7632) : __byte_perm(v[e], x, 0x5410);
                        }
                        uint2 w[8];
#pragma unroll
                        for (int e = 0; e < 8; ++e) {        // -> (row 4e + 2 b1 + b0; four dims)
                            const uint32_t x = __shfl_xor_sync(0xffffffffu, b1 ? v[2 * e] : v[2 * e + 1], 2);
                            w[e] = b1 ? make_uint2(x, v[2 * e + 1]) : make_uint2(v[2 * e], x);
                        }
#pragma unroll
                        for (int e = 0; e < 4; ++e) {        // -> (row 8e + 4 b2 + 2 b1 + b0; eight dims)
                            const uint2 mine = b2 ? w[2 * e + 1] : w[2 * e], other = b2 ? w[2 * e] : w[2 * e + 1];
                            const uint32_t x = __shfl_xor_sync(0xffffffffu, other.x, 4);
                            const uint32_t y = __shfl_xor_sync(0xffffffffu, other.y, 4);
                            const int i = c + 8 * e + (lane & 7), r = i % NR;
                            if (r < p.rows)
                                *reinterpret_cast<uint4*>(out + (size_t)r * DC * 2 + (i / NR) * 256) =
                                    b2 ? make_uint4(x, y, mine.x, mine.y) : make_uint4(mine.x, mine.y, x, y);
                        }
                    }
                } else if (p.n > 0) {
                    // as it lies, [block][four rows][dim][4], for the joining kernel
                    const size_t id = 2 * (size_t)blockIdx.x + (at_start ? 0 : 1);
                    float4* dst = reinterpret_cast<float4*>(a.part_o) + id * (NJ * NR / 4) * 128 + row;
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
            if (!whole && p.lt0 == 0 && row == 0 && rank == 0) {
                // this team holds the row group's first tile: where its pieces lie
                const long last = (p.at + p.nt - 1) / rg.per;
                *reinterpret_cast<int4*>(a.join + 4 * team) =
                    make_int4((int)(last - team) + 1, (int)((long)p.qs * a.H) + p.seg * group,
                              min(group, p.sq * a.H - p.seg * group), at_start ? 0 : 1);
            }
            tc_fence_before();
            named_bar_sync(kSmBar, 128);           // the rows' numbers may be written again
            p = nx;
            at_start = false;
        }
    }
    }

    tc_fence_before();
    __syncthreads();
    if (warp == WARP_S) {
        tc_fence_after();
        tmem_dealloc(tmem, C::TMEM_COLS);
    }
    if (threadIdx.x == 0 && *abort_flag) atomicExch(&g_latent_paged_error, (int)kErrDecodeWait);
}

// Adds up the pieces of the row groups that were cut: o = sum_p w_p O_p / sum_p
// w_p l_p with w_p = 2^(m_p - M).  Block (CTA of the team's first piece, JR rows of it,
// 128 dims): 128 / JR lanes per row for the weights, then thread = dim, U pieces at a
// time, the first of them on their way while the weights are formed (with a warp per row
// and four rows in turn the weights took 5 us of the kernel's 6).  JR is small where a
// group has few rows, because few groups of many pieces (one to four long requests)
// would leave all the reading to a few SMs.
template <int NR, bool F16>
__global__ void __launch_bounds__(128) latent_join_kernel(const LatentArgs a) {
    constexpr int JR = NR == 64 ? 16 : 4, U = 32 / JR, LR = 128 / JR;
    griddep_wait();
    const int team = blockIdx.x / a.team, rank = blockIdx.x % a.team, r_first = blockIdx.y * JR;
    const int4 j = *reinterpret_cast<const int4*>(a.join + 4 * team);
    const int n = min(j.x, a.teams - team);
    const int r0 = rank * NR + r_first;            // row of the group
    if (n <= 0 || r0 >= j.z) return;
    __shared__ float w_s[256][JR];                 // n <= teams <= 256
    __shared__ float inv[JR];
    const int d = threadIdx.x, lane = d % LR, r = d / LR;     // of the weights' row
    auto slot = [&](int p) { return 2 * ((team + p) * a.team + rank) + (p == 0 ? j.w : 0); };
    const float4* src = reinterpret_cast<const float4*>(a.part_o) + (blockIdx.z * (NR / 4) + r_first / 4) * 128 + d;
    float4 o[U][JR / 4];
    auto load = [&](int p0) {
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int g = 0; g < JR / 4; ++g)
                if (p0 + u < n) o[u][g] = src[(size_t)slot(p0 + u) * (NJ * NR / 4) * 128 + g * 128];
    };
    const float2* ml = a.part_ml + r_first + r;
    const float2 first = lane < n ? ml[(size_t)slot(lane) * NR] : make_float2(-INFINITY, 0.f);
    load(0);
    float M = first.x, L = 0.f;
    for (int p = lane + LR; p < n; p += LR) {
        w_s[p][r] = ml[(size_t)slot(p) * NR].x;
        M = fmaxf(M, w_s[p][r]);
    }
#pragma unroll
    for (int x = LR / 2; x > 0; x >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, x));
    for (int p = lane; p < n; p += LR) {
        const float l = p == lane ? first.y : ml[(size_t)slot(p) * NR].y;
        const float w = l == 0.f ? 0.f : fast_exp2((p == lane ? first.x : w_s[p][r]) - M);
        w_s[p][r] = w;
        L += w * l;
    }
#pragma unroll
    for (int x = LR / 2; x > 0; x >>= 1) L += __shfl_xor_sync(0xffffffffu, L, x);
    if (lane == 0) {
        inv[r] = L != 0.f ? 1.f / L : 0.f;
        if (blockIdx.z == 0 && r0 + r < j.z && a.lse)
            a.lse[(size_t)j.y + r0 + r] = L != 0.f ? (M + log2f(L)) * kLn2 : -INFINITY;
    }
    __syncthreads();
    float4 acc[JR / 4];
#pragma unroll
    for (int g = 0; g < JR / 4; ++g) acc[g] = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int p = 0; p < n; p += U) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
#pragma unroll
            for (int g = 0; g < JR / 4; ++g) {
                if (p + u < n) {
                    const float4 w = *reinterpret_cast<const float4*>(&w_s[p + u][4 * g]);
                    // a piece with no key for a row has not written its O
                    acc[g].x = w.x != 0.f ? fmaf(w.x, o[u][g].x, acc[g].x) : acc[g].x;
                    acc[g].y = w.y != 0.f ? fmaf(w.y, o[u][g].y, acc[g].y) : acc[g].y;
                    acc[g].z = w.z != 0.f ? fmaf(w.z, o[u][g].z, acc[g].z) : acc[g].z;
                    acc[g].w = w.w != 0.f ? fmaf(w.w, o[u][g].w, acc[g].w) : acc[g].w;
                }
            }
        }
        load(p + U);
    }
    uint16_t* out = static_cast<uint16_t*>(a.o) + ((size_t)j.y + r0) * DC + blockIdx.z * 128 + d;
#pragma unroll
    for (int g = 0; g < JR / 4; ++g) {
        const float v[4] = {acc[g].x, acc[g].y, acc[g].z, acc[g].w};
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (r0 + 4 * g + e < j.z) out[(4 * g + e) * DC] = (uint16_t)pack2<F16>(v[e] * inv[4 * g + e], 0.f);
    }
}

template <int NR, bool F16, bool GATHER>
cudaError_t launch_t(const CUtensorMap& tm_q, const CUtensorMap& tm_kv, const CUtensorMap& tm_pe,
                     const CUtensorMap& tm_row, const LatentArgs& a, cudaStream_t stream) {
    using C = LCfg<NR, GATHER>;
    static SmemLimit limit;
    cudaError_t e = limit.set(reinterpret_cast<const void*>(latent_paged_kernel<NR, F16, GATHER>), C::SMEM_BYTES);
    if (e != cudaSuccess) return e;
    const unsigned ctas = (unsigned)(a.teams * a.team);
    latent_paged_kernel<NR, F16, GATHER><<<ctas, C::THREADS, C::SMEM_BYTES, stream>>>(tm_q, tm_kv, tm_pe, tm_row, a);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(ctas, NR == 64 ? 4 : NR / 4, NJ);
    cfg.blockDim = dim3(128);
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
                                const CUtensorMap& tm_row, const LatentArgs& a, cudaStream_t stream) {
    const bool gather = a.box_tokens == 0;
    switch ((gather ? 64 : a.nr) * 4 + (a.f16 ? 2 : 0) + (gather ? 1 : 0)) {
        case 16 * 4: return launch_t<16, false, false>(tm_q, tm_kv, tm_pe, tm_row, a, stream);
        case 16 * 4 + 2: return launch_t<16, true, false>(tm_q, tm_kv, tm_pe, tm_row, a, stream);
        case 32 * 4: return launch_t<32, false, false>(tm_q, tm_kv, tm_pe, tm_row, a, stream);
        case 32 * 4 + 2: return launch_t<32, true, false>(tm_q, tm_kv, tm_pe, tm_row, a, stream);
        case 64 * 4: return launch_t<64, false, false>(tm_q, tm_kv, tm_pe, tm_row, a, stream);
        case 64 * 4 + 2: return launch_t<64, true, false>(tm_q, tm_kv, tm_pe, tm_row, a, stream);
        case 64 * 4 + 1: return launch_t<64, false, true>(tm_q, tm_kv, tm_pe, tm_row, a, stream);
        case 64 * 4 + 3: return launch_t<64, true, true>(tm_q, tm_kv, tm_pe, tm_row, a, stream);
        default: return cudaErrorInvalidValue;
    }
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
