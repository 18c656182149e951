// One-query-tile causal GQA attention forward on sm_103a: the kernel behind
// dense prefill at head dim 256 and behind every packed variable-length call.
//
// Computes what prefill.cu computes (TileOPs "Attention Operators",
// GQADenseFwdOp stages 1-7; RL-Kernel "Standard Softmax Attention", Tensor
// Contract; natural-log LSE per MATE "QSA", Core Attention) for three input
// layouts:
//   kBSHD    q [B, Sq, Hq, D], k / v [B, Skv, Hkv, D]; one item = one 128-row
//            query tile of one (b, h);
//   kPacked  packed rows (TileOPs GQAVarlenFwdOp): q [total_q, Hq, D],
//            k / v [total_kv, Hkv, D], request b owning the rows its
//            cu_seqlens name;
//   kPaged   packed queries over a paged cache (TileOPs GQAPagedFwdOp):
//            k / v [pages, page_size, Hkv, D] read through block_table, the
//            cache length of a request counting its query tokens;
//   kPaged8  kPaged over float8_e4m3fn caches with one scale per (request,
//            KV head): the products run in float16 on exactly widened keys
//            and values, and the scales join the softmax scale and 1 / l.
// In the packed layouts an item is a row block of one (request, KV
// head): the g = Hq / Hkv query heads of the group are packed into the tile
// rows (row r = query q0 + r / g, head hkv * g + r % g; floor(128 / g)
// queries per block), so every key and value a request reads serves all g
// heads at once: a decode request streams its cache once per KV head.
//
// TMEM holds S0 | S1 (128 columns each) | O (D columns): the tensor core
// computes S of key tile i+1 while the softmax warps work on tile i.
// Warp roles (384 threads, one CTA per SM, persistent over the items):
//   warps 0-3   softmax: thread t owns tile row t; reads its S row from TMEM,
//               folds the causal / window / padding mask, keeps the running
//               max and sum, writes P (16-bit) over its S row and rescales
//               its O row when the reference max moves;
//   warps 4-7   epilogue: once an item's last P V has completed, reads O,
//               frees it for the next item, and stores O / l and the LSE
//               (TMA through two alternating staging boxes for whole
//               blocks, row by row for a block cut by its request's end),
//               while the next item's first tiles already run;
//   warp 8      TMA producer: the Q block, then K and V through one ring of
//               32 KB slots in the order the MMAs consume them;
//   warp 9      MMA issuer: QK(0), QK(1), PV(0), QK(2), PV(1), ...; it also
//               zeroes the value rows of an item's last key tile that lie
//               past the request's end before P V reads them (packed and
//               paged layouts: those rows hold other requests' values or
//               stale cache slots, and 0 * NaN would not vanish);
//   warps 10-11 complete the third warpgroup (register limits are per
//               warpgroup).
// kPaged8 has 512 threads and no TMA loads: warps 8-10 widen keys and warps
// 12-15 values (fp8_item), each team filling a ring of its own; the epilogue warps
// write the next item's Q block (fill_q8); warp 11 issues QK(i + 1) before PV(i).  e4m3 halves what a key costs in
// HBM, but the tensor core takes A and B of one type and P needs more than e4m3's
// four bits, so every key is widened once per row block; that and the softmax,
// not the MMAs, set the pace.  Measured: a 2048-query chunk over 32768 keys, 64/8
// heads, D = 128: 1.86-1.88 ms, 1.14 PFLOP/s (the 16-bit call: 2.10 ms); about 2100
// cycles a tile, 1400 of them softmax and 1445 the issue of its MMAs (QK 681, PV
// 764), which overlap as far as two S buffers allow.  Between two items
// the MMA warp loses about 9000 cycles (the last P, the new Q, O's hand-over).
// Five ragged chunks at 24/2, D = 256: 0.33-0.41 ms with softcap over three draws, 0.31-0.38
// without (a draw that takes 0.43: the 16-bit call 0.56); 4200-4400 cycles a tile, in which the
// data pipe of shared memory and L1 carries 1536 wavefronts of MMA operands, 1366 of
// stores and 1435 of loads (ncu): 4337, if they share it, so the port is full.  The MMAs
// wait 1250 cycles a tile for keys (a ring of one tile: a slot is refilled only after
// the S before has read it).
// The MMA shapes stay M128 x N128 (QK) and M128 x N(D) (PV); at D = 256 K is
// split into two 128-column halves and V into two 64-key halves so that each
// half fills one ring slot.  Shared-memory operand layouts:
//   slice-major  (kBSHD, kPacked): a {64, rows} box per 64-column slice,
//                8-row atoms 1 KB apart, slices rows * 128 bytes apart;
//   group-major  (kPaged): one 5-D box per page block lands as
//                [8-key group][slice][8 keys][128 bytes], slices 1 KB apart.
// Both are described by a slice stride and an 8-key-group stride, which is
// all the MMA descriptors need.
//
// The lazy rescale is that of prefill.cu (kPaged8: from a reference below the max,
// kLead8).  Rescaling O before PV of tile i
// needs PV of tile i-1 complete (o_ready, waited for only by a warp that
// rescales): S of tile i having landed implies PV of tile i-2, so the phase
// waited for is never more than one behind.  Every wait is bounded; on a
// timeout the CTA stops issuing work, drains what is in flight, frees TMEM
// and returns.
#pragma once
#include <cmath>

#include "internal.h"
#include "prefill_tiles.cuh"
#include "ptx.cuh"

namespace gqa {
namespace {

__device__ int g_onetile_error;

namespace ot {

using namespace pf;

enum Mode : int { kBSHD = 0, kPacked = 1, kPaged = 2, kPaged8 = 3 };

constexpr int NUM_THREADS = 384;
constexpr int WARP_EPI0 = 4;
constexpr int WARP_LOAD = 8;
constexpr int WARP_MMA = 9;
// Registers: 168 per thread at launch (64,512 in all); the softmax warpgroup
// takes 208, the epilogue warpgroup (half a packed O row at a time) 152 and
// the producer/MMA warpgroup 144: (208 + 152 + 144) * 128.
constexpr int kRegsLaunch = 168;
constexpr int kRegsSoftmax = 208;
constexpr int kRegsEpi = 152;
constexpr int kRegsOther = 144;
static_assert((kRegsSoftmax + kRegsEpi + kRegsOther) * 128 <= kRegsLaunch * NUM_THREADS, "register split");
// kPaged8: warps 8-10 widen keys, 12-15 values, 11 issues the MMAs.  128
// registers per thread at launch (four warps on each SM sub-partition); softmax
// 208, epilogue 96, the other two warpgroups 104 each.  The values get the
// fourth warp: P V comes last in a tile (four warps on the keys instead: 0.46
// against 0.45 ms on five ragged chunks at 24/2, D = 256).
constexpr int NUM_THREADS8 = 512;
constexpr int WARP_V8 = 12;
constexpr int WARP_MMA8 = 11;
constexpr int TEAM_K8 = 3, TEAM_V8 = 4;        // warps of a widening team
constexpr int kRegsEpi8 = 96;
constexpr int kRegsOther8 = 104;
static_assert((kRegsSoftmax + kRegsEpi8 + 2 * kRegsOther8) * 128 <= 128 * NUM_THREADS8, "register split");
constexpr int num_threads(int mode) { return mode == kPaged8 ? NUM_THREADS8 : NUM_THREADS; }

constexpr int BOX = BM * 128;      // one 64-column box of 128 rows (16 KB)
constexpr int SLOT = 32768;        // one ring slot
constexpr int ENTRY_INTS = 8;      // a row block of a packed call: b, q0, qs, sq, ks, L, -, -

template <int D, int MODE>
struct Cfg {
    static constexpr int KSL = D / 64;                  // 64-column slices per row
    static constexpr int CK = D == 256 ? 2 : 1;         // ring chunks per K tile (halves along D)
    static constexpr int CV = D == 256 ? 2 : 1;         // ring chunks per V tile (halves along the keys)
    static constexpr int KSL_C = KSL / CK;              // slices per K chunk
    static constexpr int VKEYS = BN / CV;               // keys per V chunk
    static constexpr int K_CHUNK = BN * 128 * KSL_C;    // bytes
    static constexpr int V_CHUNK = VKEYS * 128 * KSL;
    static constexpr bool GROUPED = MODE == kPaged || MODE == kPaged8;
    static constexpr int K_SLICE = GROUPED ? 1024 : BN * 128;
    static constexpr int K_GROUP = GROUPED ? KSL_C * 1024 : 1024;
    static constexpr int V_SLICE = GROUPED ? 1024 : VKEYS * 128;
    static constexpr int V_GROUP = GROUPED ? KSL * 1024 : 1024;
    // kPaged8 at D = 128: Q lives in TMEM (64 columns beside S0, S1 and O), the A
    // operand of S = Q K^T; shared memory then carries 160 KB a tile instead of
    // 192 (K and V written by the wideners and read by the MMAs, and the loads
    // through L1, which share its 128 bytes a clock), and a sixth slot
    static constexpr bool TQ = MODE == kPaged8 && D == 128;
    // threads at the barrier before TMEM is freed: softmax, epilogue and MMA warps
    static constexpr int TMEM_USERS = 8 * 32 + 32;
    static constexpr int NS = TQ ? 6 : (D == 256 ? 4 : 5);         // ring slots
    // kPaged8: two rings, slots [0, NK8) for keys and [NK8, NS) for values, each
    // filled by one team: with one ring, a team could come to a slot whose use
    // before last was still to be released, and a parity would not tell.
    static constexpr int NK8 = NS / 2, NV8 = NS - NK8;
    static constexpr int OFF_Q = 0;
    static constexpr int OFF_RING = OFF_Q + (TQ ? 0 : KSL * BOX);
    static constexpr int OFF_STAGE = OFF_RING + NS * SLOT;   // 2 output boxes
    static constexpr int OFF_STATS = OFF_STAGE + 2 * BOX;    // m[128], l[128], visited-tile count
    static constexpr int OFF_BAR = OFF_STATS + 2 * BM * 4 + 16;
    // q_full, q_empty, r_full[NS], r_empty[NS], s_full[2], p_full[2], o_ready,
    // o_final, o_empty, stats_full, stats_empty, drain, item_full[2], item_empty[2]
    static constexpr int NBAR = 2 + 2 * NS + 4 + 6 + 4;
    static constexpr int OFF_MISC = OFF_BAR + NBAR * 8;
    static constexpr int SMEM_USED = OFF_MISC + 16;
    static constexpr int SMEM_BYTES = SMEM_USED + 1024;        // 1 KB alignment slack
    static_assert(K_CHUNK <= SLOT && V_CHUNK <= SLOT, "ring slot");
    static_assert(SMEM_BYTES <= 227 * 1024, "shared memory budget");
};
constexpr uint32_t COL_S0 = 0, COL_O = 256, COL_Q8 = 384, TMEM_COLS = 512;
// kPaged8: P is float16.  The reference stands kLead8 binades below the row's max,
// so that P = 2^kLead8 for the strongest key and weights down to 2^-20 of its keep
// float16's eleven bits; below that a weight is off by at most half a subnormal
// step, 2^-25 in P, 2^-31 of the strongest.  (With the reference at the max, weights
// below 2^-25 of it vanished from P V but not from the row sum: one strong key before
// 131071 equal ones took 3.8e-3 from a mean of 3.8e-3.)  Up to 2^(kLead8 + 8) between
// rescales and up to kSumLimit8 on a plain tile, P stays a finite float16.
constexpr float kLead8 = 6.f;
constexpr float kSumLimit8 = 65504.f;

// tanh of two values of magnitude at most 0.6: y times a polynomial of degree 4
// in y^2, the minimax one for the relative error there (Remez exchange in 40
// digits: 7.3e-08, with FP32 rounding 9.4e-08 absolute).
constexpr float kTanhSmall = 0.6f;
__device__ __forceinline__ uint64_t tanh2_small(uint64_t y) {
    auto both = [](float c) { return f32x2(c, c); };
    const uint64_t u = fmul2(y, y);
    uint64_t p = ffma2(u, both(0.01547542757f), both(-0.05210148018f));
    p = ffma2(u, p, both(0.1331017366f));
    p = ffma2(u, p, both(-0.3333230997f));
    p = ffma2(u, p, both(0.9999999269f));
    return fmul2(y, p);
}

// tanh(y) = 1 - 2 / (e^(2y) + 1)
__device__ __forceinline__ float tanh_mufu(float y) {
    return fmaf(-2.f, rcp_approx(fast_exp2(y * 2.8853900817779268f) + 1.f), 1.f);      // 2 log2(e)
}

// kPaged8: N raw scores -> tanh(to_y * s) (to_y = scale / softcap), in place.
// Scores up to 0.6 of the cap take a polynomial, 7 paired FP32 operations for
// two; a warp with a larger one takes 1 - 2 / (e^(2y) + 1).  Warp-collective.
template <int N>
__device__ __forceinline__ void tanh_cols(float* s, float to_y) {
    float am[2] = {0.f, 0.f};
#pragma unroll
    for (int c = 0; c < N; c += 2) am[(c >> 1) & 1] = fmax3(am[(c >> 1) & 1], fabsf(s[c]), fabsf(s[c + 1]));
    if (__all_sync(0xffffffffu, fmaxf(am[0], am[1]) * fabsf(to_y) <= kTanhSmall)) {
        const uint64_t k = f32x2(to_y, to_y);
#pragma unroll
        for (int c = 0; c < N; c += 2) f32x2_split(tanh2_small(fmul2(f32x2(s[c], s[c + 1]), k)), s[c], s[c + 1]);
    } else {
#pragma unroll
        for (int c = 0; c < N; ++c) s[c] = tanh_mufu(s[c] * to_y);
    }
}

// kPaged8: a row of raw scores in TMEM -> what the exponential scales, in
// place, 32 columns a turn: tanh(to_y * s) with a softcap, else s * factor; -inf
// outside [lo, lim).  Only tiles that need it take this pass (a mask, a scale
// that is not positive); all others go straight to the maximum, so that the
// code of the usual tile stays small: the roles of a CTA share one instruction
// cache, and with the masked and capped forms unrolled over 128 columns 4.5
// warps waited for instructions per issue (ncu, D = 256 with a softcap).
__device__ __forceinline__ void prepare_scores(uint32_t taddr, bool capped, float to_y, float factor, int lo, int lim) {
#pragma unroll 1
    for (int c0 = 0; c0 < BN; c0 += 32) {
        float s[32];
        __syncwarp();
        tmem_ld32(taddr + c0, s);
        if (capped) {
            tanh_cols<32>(s, to_y);
        } else {
#pragma unroll
            for (int c = 0; c < 32; ++c) s[c] *= factor;
        }
        const int l = lo - c0, h = lim - c0;
#pragma unroll
        for (int c = 0; c < 32; ++c) s[c] = c >= l && c < h ? s[c] : -INFINITY;
        __syncwarp();
        tmem_st32(taddr + c0, reinterpret_cast<uint32_t*>(s));
    }
}

// kPaged8: an unmasked row of raw scores in TMEM -> P = 2^(cap_out tanh(to_y s) - m)
// over its first 64 columns, 64 scores a turn; returns the row's sum.
__device__ __forceinline__ float capped_exp(uint32_t taddr, float to_y, float cap_out, float m) {
    float sum = 0.f;
#pragma unroll 1
    for (int k = 0; k < BN / 64; ++k) {
        float s[64];
        uint32_t pk[32];
        __syncwarp();
        tmem_ld32(taddr + 64 * k, s);
        tmem_ld32(taddr + 64 * k + 32, s + 32);
        tanh_cols<64>(s, to_y);
        sum += exp_row<true, 64>(s, cap_out, m, pk);
        __syncwarp();
        tmem_st32(taddr + 32 * k, pk);
    }
    return sum;
}

// kPaged8: one item's e4m3 key (V: value) rows, by a team of three (four)
// warps, as float16 tiles in the ring slots that hold its keys (values).  A
// 128-byte stretch of a cache row goes to eight lanes, 16 bytes each, so a
// warp's load covers 512 bytes, and a slot takes 32 of them.  The loads of the
// next slot are issued when this one's are widened and stored: their latency
// runs beside the wait for the slot.  The lane's 16 codes become two 16-byte chunks
// of the swizzled tile; which row and column a lane takes is chosen so that the
// eight lanes of a store cover eight different bank groups.  (One row to eight
// lanes, half of them storing their odd chunk first, needs selects instead: 2.50
// against 1.90 ms on a 2048-query chunk over 32768 keys, 64/8 heads, D = 128.)
// Nothing here
// may spill: the streaming loads evict local memory from the small L1 beside
// 227 KB of shared memory, and every reload then goes to L2 (10.6 ms instead of
// 3.8 on that chunk when it was found).
template <int D, class C, bool V>
__device__ __forceinline__ bool fp8_item(const PrefillArgs& a, uint8_t* smem, uint32_t full0, uint32_t empty0,
                                         volatile int* abort_flag, int b, int hkv, int skv, int kv_begin, int first,
                                         int n_tiles, int wid, int lane, int& nc) {
    constexpr int NCH = V ? C::CV : C::CK;        // slots per tile
    constexpr int NR = V ? C::NV8 : C::NK8;       // slots of this team's ring
    constexpr bool WIDE = D == 256 && V;          // a load covers two 256-byte rows, else four 128-byte stretches
    constexpr int LPR = WIDE ? 16 : 8;            // lanes per row
    constexpr int TEAM = V ? TEAM_V8 : TEAM_K8;
    constexpr int NL = (32 + TEAM - 1) / TEAM;    // a warp's loads of a slot
    constexpr int STEP = TEAM * (32 / LPR);       // rows between a warp's loads
    constexpr int GROUP = V ? C::V_GROUP : C::K_GROUP;
    // This lane's row and 16-byte column of the first load: eight lanes take half
    // a 128-byte slice of two neighbouring rows, so that their even (or odd)
    // chunks lie in eight different bank groups of the swizzled tile.
    const int row0 = wid * (32 / LPR) + (WIDE ? 0 : 2 * (lane >> 4)) + ((lane >> 2) & 1);
    const int col = (lane & 3) + 4 * (WIDE ? lane >> 3 : (lane >> 3) & 1);
    // where the first of its two chunks of row r goes (the second: bit 4 flipped)
    auto place = [&](int r) -> uint32_t {
        return (r / 8) * GROUP + (col >> 2) * 1024 + (r % 8) * 128 + (((2 * col) & 7) ^ (r % 8)) * 16;
    };
    constexpr int PER = STEP % 8 == 0 ? 1 : (STEP % 4 == 0 ? 2 : 4);      // loads after which r % 8 repeats
    uint32_t to[PER];
#pragma unroll
    for (int k = 0; k < PER; ++k) to[k] = place(k * STEP + row0);
    const uint8_t* cache = static_cast<const uint8_t*>(V ? a.v_cache : a.k_cache) + (size_t)hkv * D + 16 * col;
    const uint32_t row_bytes = (uint32_t)a.Hkv * D;
    const int32_t* table = a.table + (size_t)b * a.max_pages;
    // Keys of a tile, lane l holding l, l + 32, l + 64 and l + 96: their pages
    // and places in them; and, once the pages have arrived, their cache rows.  A
    // key past the request's end takes the last key's row (its score is masked
    // and its weight 0); one of a page outside the pool, or left of every window
    // of the block (its page may hold anything by now), row 0, marked to be
    // zeroed.  No load stands in a branch: what a branch loads may be moved to
    // its register at the branch's end, which waits out the load's latency.
    struct Pages {
        int page[4], off[4];
    };
    auto find_pages = [&](int tile) -> Pages {
        Pages p;
#pragma unroll
        for (int x = 0; x < 4; ++x) {
            const uint32_t key = (uint32_t)min(tile * BN + 32 * x + lane, skv - 1);
            const uint32_t n = (__umulhi(key, a.ps_mul) + key) >> a.ps_shift;       // key / page_size
            p.page[x] = ldg_int(table + n);
            p.off[x] = (int)(key - n * (uint32_t)a.page_size);
        }
        return p;
    };
    uint32_t bad[4];                               // keys of the tile (32 a word) to be zeroed
    auto find_rows = [&](int tile, const Pages& p) -> int4 {
        int r[4];
#pragma unroll
        for (int x = 0; x < 4; ++x) {
            const bool in = (uint32_t)p.page[x] < (uint32_t)a.num_pages && tile * BN + 32 * x + lane >= kv_begin;
            bad[x] = __ballot_sync(0xffffffffu, !in);
            r[x] = in ? p.page[x] * a.page_size + p.off[x] : 0;
        }
        return make_int4(r[0], r[1], r[2], r[3]);
    };
    uint32_t buf[NL][4];
    auto load = [&](int ch, const int4& all) {
        // a wide slot holds half a tile's keys
        const int4 rows = WIDE && ch ? make_int4(all.z, all.w, all.z, all.w) : all;
        auto part = [&](int x) { return x == 0 ? rows.x : (x == 1 ? rows.y : (x == 2 ? rows.z : rows.w)); };
        int src[NL];
#pragma unroll
        for (int j = 0; j < NL; ++j) {
            const int at = j * STEP;                                    // + row0 < STEP: the lane's row of the slot
            src[j] = __shfl_sync(0xffffffffu, part(at / 32), at % 32 + row0);
            if (at % 32 + STEP > 32 && at < (WIDE ? 32 : 96)) {                       // the warps' rows straddle two parts
                const int next = __shfl_sync(0xffffffffu, part(at / 32 + 1), at % 32 + row0);
                src[j] = at % 32 + row0 >= 32 ? next : src[j];
            }
        }
#pragma unroll
        for (int j = 0; j < NL; ++j)               // a team's surplus load repeats some row, and is not stored
            ldg16(buf[j], cache + (size_t)(uint32_t)src[j] * row_bytes + (D == 256 && !V ? 128 * ch : 0));
    };
    auto store = [&](int ch, uint8_t* dst) {
        if (bad[0] | bad[1] | bad[2] | bad[3]) {   // uniform; pages outside the pool
#pragma unroll
            for (int j = 0; j < NL; ++j) {
                const int r = (WIDE ? 64 * ch : 0) + j * STEP + row0, x = r / 32;
                const uint32_t w = x == 0 ? bad[0] : (x == 1 ? bad[1] : (x == 2 ? bad[2] : bad[3]));
                if ((w >> (r % 32)) & 1u) buf[j][0] = buf[j][1] = buf[j][2] = buf[j][3] = 0u;
            }
        }
#pragma unroll
        for (int j = 0; j < NL; ++j) {
            if (32 % TEAM && j == NL - 1 && wid + TEAM * j >= 32) break;
            uint32_t h[8];
#pragma unroll
            for (int e = 0; e < 4; ++e) e4m3x4_to_f16x4(buf[j][e], h[2 * e], h[2 * e + 1]);
            const uint32_t p = to[j % PER] + (j / PER) * (PER * STEP / 8) * GROUP;
            *reinterpret_cast<uint4*>(dst + p) = make_uint4(h[0], h[1], h[2], h[3]);
            *reinterpret_cast<uint4*>(dst + (p ^ 16)) = make_uint4(h[4], h[5], h[6], h[7]);
        }
    };

    const int c = n_tiles - first;
    int4 rows = find_rows(first, find_pages(first));
    load(0, rows);
    Pages pages = find_pages(first + 1);          // a tile ahead of their use
    for (int i = 0; i < c; ++i) {
#pragma unroll 1
        for (int ch = 0; ch < NCH; ++ch, ++nc) {
            const int s = nc % NR;
            if (!__all_sync(0xffffffffu, mbar_wait(empty0 + 8u * s, ((nc / NR) & 1) ^ 1, abort_flag))) return false;
            store(ch, smem + C::OFF_RING + ((V ? C::NK8 : 0) + s) * SLOT);
            fence_proxy_async_smem();             // the tensor core reads what the warp wrote
            __syncwarp();
            if (lane == 0) mbar_arrive(full0 + 8u * s);
            if (ch + 1 == NCH) rows = find_rows(first + i + 1, pages);
            load(ch + 1 < NCH ? ch + 1 : 0, rows);           // past the last tile: the last key's row again
        }
        pages = find_pages(first + i + 2);
    }
    return true;
}

// kPaged8: an item's Q block, by the four epilogue warps: n_rows rows (packed r =
// query * g + head, the block's first query in row q_row0 of the batch) as
// float16 (bfloat16 rounded), zeros past them, once the S MMAs that read the last
// block are complete.  The epilogue warps do it while they would wait for the
// item before to end, so that no widening team interrupts its stream of keys or
// values.  D / 4 registers of loads are in flight a thread.
template <int D, bool F16, class C>
__device__ __forceinline__ bool fill_q8(const PrefillArgs& a, uint8_t* smem, uint32_t q_full, uint32_t q_empty,
                                        volatile int* abort_flag, int q_row0, int n_rows, int hkv, int g, int wid,
                                        int lane, uint32_t tmem, int& nq) {
    constexpr int N = 16;                         // 16-byte pieces in flight
    const uint16_t* q = static_cast<const uint16_t*>(a.q) + ((size_t)q_row0 * a.Hq + hkv * g) * D;
    const uint32_t inv_g = (65535u + g) / g;      // r / g = r * inv_g >> 16 for r < 128, g <= 128
    auto piece = [&](int r, int c8, uint32_t* w) {          // dims 8 c8 .. of row r
        const bool ok = r < n_rows;
        const int rr = ok ? r : 0;
        // row rr / g of the batch, head rr % g of the group
        ldg16_or_zero(w, q + ((size_t)((rr * inv_g) >> 16) * (a.Hq - g) + rr) * D + 8 * c8, ok);
    };
    auto to_f16 = [&](uint32_t* w) {
        if constexpr (!F16) {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                w[e] = pack_f16x2(__uint_as_float(w[e] << 16), __uint_as_float(w[e] & 0xffff0000u));
        }
    };
#pragma unroll 1
    for (int k = 0; k < D / 8 / N; ++k) {
        uint32_t w[4 * N];
        // TMEM lane = row; shared memory: a warp's load covers a row (D = 256)
#pragma unroll
        for (int u = 0; u < N; ++u) {
            if constexpr (C::TQ) piece(wid * 32 + lane, u, w + 4 * u);
            else piece(4 * (k * N + u) + wid, lane, w + 4 * u);
        }
        if (k == 0) {
            if (!__all_sync(0xffffffffu, mbar_wait(q_empty, (nq & 1) ^ 1, abort_flag))) return false;
            tc_fence_after();
        }
#pragma unroll
        for (int u = 0; u < N; ++u) to_f16(w + 4 * u);
        if constexpr (C::TQ) {
            __syncwarp();
#pragma unroll
            for (int h = 0; h < 2; ++h)
                tmem_st32(tmem + ((uint32_t)(wid * 32) << 16) + COL_Q8 + 32 * h, w + 32 * h);
        } else {
#pragma unroll
            for (int u = 0; u < N; ++u) {
                const int r = 4 * (k * N + u) + wid;
                *reinterpret_cast<uint4*>(smem + C::OFF_Q + (lane >> 3) * BOX + r * 128 +
                                          (((lane & 7) ^ (r & 7)) << 4)) = make_uint4(w[4 * u], w[4 * u + 1], w[4 * u + 2],
                                                                                     w[4 * u + 3]);
            }
        }
    }
    if constexpr (C::TQ) tc_fence_before();
    else fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) mbar_arrive(q_full);
    ++nq;
    return true;
}

template <int D, int MODE, bool OPTS, bool F16>
__global__ void __launch_bounds__(num_threads(MODE), 1)
onetile_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
               const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_o,
               const PrefillArgs a, int n_qtiles) {
    // CTAs past the share the plan gave this launch leave their SMs to the
    // decode steps running beside it (uniform per CTA, before any set-up)
    if (a.g_eff != nullptr && (int)blockIdx.x >= *a.g_eff) return;
    using C = Cfg<D, MODE>;
    constexpr bool PACKED = MODE != kBSHD;
    constexpr bool KV8 = MODE == kPaged8;
    constexpr int WMMA = KV8 ? WARP_MMA8 : WARP_MMA;
    constexpr bool MF16 = KV8 || F16;            // the MMAs' operand type is float16 (F16: the call's type)
    constexpr uint32_t IDESC_QK = make_idesc_16<MF16>(BM, BN, false, false);
    constexpr uint32_t IDESC_PV = make_idesc_16<MF16>(BM, D, false, true);
    const int wl = OPTS ? a.x.wl : -1;
    const int wr = OPTS ? a.x.wr : -1;
    const float cap_in = OPTS ? a.x.cap_in : 0.f;
    const float cap_out = OPTS ? a.x.cap_out : 0.f;
    const float* sinks = OPTS ? a.x.sinks : nullptr;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw_base = smem_u32(smem_raw);
    uint8_t* smem = smem_raw + ((1024 - (raw_base & 1023)) & 1023);
    const uint32_t sb = smem_u32(smem);

    const int warp = threadIdx.x / 32;
    const int lane = threadIdx.x % 32;

    // rows per query in a tile (1, or the group size when heads are packed)
    const int g = PACKED ? a.g : 1;
    const int qpb = PACKED ? a.qpb : BM;         // queries per block
    const int n_e = PACKED ? *a.n_entries : 0;
    // Work items.  kBSHD: heaviest (last) query tiles first, adjacent items on
    // one KV head; round r takes item r * G + cta (even r) or r * G + G - 1 -
    // cta (odd r).  Packed: item w = (row block w / Hkv, KV head w % Hkv), the
    // requests ordered by estimated cost, heaviest first; items are claimed
    // in that order from a counter in the workspace (the plan kernel zeroes
    // it), so that a CTA whose items ran long takes fewer of them.
    // kPaged8: each such item may be cut into parts along the keys
    const int parts = KV8 && a.part_o != nullptr ? a.n_entries[3] : 1;
    const int n_items = PACKED ? n_e * a.Hkv * parts : n_qtiles * a.B * a.Hq;
    const int G = gridDim.x;
    const int cta = blockIdx.x;
    auto item_of = [&](int r) -> int {
        const long w = (long)r * G + ((r & 1) ? G - 1 - cta : cta);
        return w < n_items ? (int)w : -1;
    };
    struct Item {
        int b, hq, hkv;     // hq: the query head (kBSHD) or the group's first head
        int qs, ks;         // packed row of the request's first query / key
        int sq, skv;        // the request's queries and keys
        int first;          // first visited key tile
        TileInfo t;         // t.q0: first query of the block (within the request)
        const uint8_t* mrow;
    };
    auto describe = [&](int w) {
        Item it;
        const int part = KV8 ? w % parts : 0;
        if constexpr (KV8) w /= parts;
        if constexpr (PACKED) {
            const int4* e = reinterpret_cast<const int4*>(a.entries + (size_t)(w / a.Hkv) * ENTRY_INTS);
            const int4 e0 = e[0], e1 = e[1];
            it.b = e0.x;
            it.hkv = w % a.Hkv;
            it.hq = it.hkv * g;
            it.qs = e0.z;
            it.sq = e0.w;
            it.ks = e1.x;
            it.skv = e1.y;
            it.t = tile_info_n(e0.y, qpb, it.sq, it.skv, a.causal, wl, wr);
            it.mrow = nullptr;
        } else {
            const int bh = a.B * a.Hq;
            const int qt = n_qtiles - 1 - w / bh;
            const int rem = w % bh;
            it.hq = rem % a.Hq;
            it.b = rem / a.Hq;
            it.hkv = it.hq / (a.Hq / a.Hkv);
            it.qs = it.ks = 0;
            it.sq = a.Sq;
            it.skv = a.Skv;
            it.t = tile_info(qt * BM, a.Sq, a.Skv, a.causal, wl, wr);
            it.mrow = a.mask ? a.mask + (size_t)it.b * a.Skv : nullptr;
        }
        it.first = it.t.kv_begin / BN;
        if constexpr (KV8) {
            // equal parts, of kPartTiles tiles at least: a block with fewer tiles than
            // the longest fills only its first parts
            int per = (it.t.n_tiles - it.first + parts - 1) / parts;
            if (parts > 1) per = max(per, kPartTiles);
            it.first = min(it.first + part * per, it.t.n_tiles);
            it.t.n_tiles = min(it.first + per, it.t.n_tiles);
        }
        return it;
    };
    // Visited key tiles of an item (non-empty, in [first, n_tiles)).  Warp-collective.
    auto count_tiles = [&](const Item& it) {
        if (!it.mrow) return it.t.n_tiles - it.first;
        int c = 0;
        for (int chunk = it.first / 32; chunk * 32 < it.t.n_tiles; ++chunk)
            c += __popc(tile_flags(it.mrow, chunk, it.first, it.t.n_tiles, it.t.kv_end, lane));
        return c;
    };

    const uint32_t bar0 = sb + C::OFF_BAR;
    const uint32_t q_full = bar0, q_empty = bar0 + 8;
    auto r_full = [&](int s) { return bar0 + 8u * (2 + s); };
    auto r_empty = [&](int s) { return bar0 + 8u * (2 + C::NS + s); };
    auto s_full = [&](int k) { return bar0 + 8u * (2 + 2 * C::NS + k); };
    auto p_full = [&](int k) { return bar0 + 8u * (4 + 2 * C::NS + k); };
    const uint32_t o_ready = bar0 + 8u * (6 + 2 * C::NS);
    const uint32_t o_final = o_ready + 8, o_empty = o_ready + 16;
    const uint32_t stats_full = o_ready + 24, stats_empty = o_ready + 32, drain = o_ready + 40;
    auto item_full = [&](int k) { return o_ready + 48u + 8u * k; };
    auto item_empty = [&](int k) { return o_ready + 64u + 8u * k; };
    float* st_m = reinterpret_cast<float*>(smem + C::OFF_STATS);
    float* st_l = st_m + BM;
    volatile int* st_cnt = reinterpret_cast<volatile int*>(st_l + BM);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::OFF_MISC);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::OFF_MISC + 4);
    volatile int* item_rec = reinterpret_cast<volatile int*>(smem + C::OFF_MISC + 8);   // two claimed items
    // Packed: the producer claims items and hands each one's index to the
    // MMA warp and the eight softmax / epilogue warps through a two-slot
    // record; the last record it writes is -1.  Warp-collective.
    auto claim_item = [&](int r) -> int {
        if constexpr (!PACKED) {
            return item_of(r);
        } else {
            int w = -1;
            if (lane == 0) {
                const int slot = r & 1;
                if (mbar_wait(item_empty(slot), ((r >> 1) & 1) ^ 1, abort_flag)) {
                    w = atomicAdd(a.work, 1);
                    if (w >= n_items) w = -1;
                    item_rec[slot] = w;
                    mbar_arrive(item_full(slot));
                }
            }
            return __shfl_sync(0xffffffffu, w, 0);
        }
    };
    auto next_item = [&](int r) -> int {
        if constexpr (!PACKED) {
            return item_of(r);
        } else {
            const int slot = r & 1;
            const bool got = __all_sync(0xffffffffu, mbar_wait(item_full(slot), (r >> 1) & 1, abort_flag));
            const int w = got ? item_rec[slot] : -1;
            __syncwarp();
            if (lane == 0) mbar_arrive(item_empty(slot));
            return w;
        }
    };

    if (threadIdx.x == 0) {
        mbar_init(q_full, !KV8 ? 1 : 4);             // TMA, or the epilogue warps
        mbar_init(q_empty, 1);
        for (int s = 0; s < C::NS; ++s) {
            mbar_init(r_full(s), !KV8 ? 1 : (s < C::NK8 ? TEAM_K8 : TEAM_V8));     // TMA, or the widening team
            mbar_init(r_empty(s), 1);
        }
        for (int k = 0; k < 2; ++k) { mbar_init(s_full(k), 1); mbar_init(p_full(k), BM); }
        mbar_init(o_ready, 1);
        mbar_init(o_final, 1);
        mbar_init(o_empty, BM);
        mbar_init(stats_full, BM);
        mbar_init(stats_empty, BM);
        mbar_init(drain, 1);
        for (int k = 0; k < 2; ++k) {
            mbar_init(item_full(k), 1);
            // the MMA warp, the eight softmax / epilogue warps, and the widening warps but the claiming one
            mbar_init(item_empty(k), 1 + 8 + (KV8 ? TEAM_K8 + TEAM_V8 - 1 : 0));
        }
        *abort_flag = 0;
        fence_mbar_init();
    }
    if constexpr (PACKED && !KV8) {
        // Q rows past g * qpb are never loaded: zero them once (finite rows,
        // their results are never stored)
        const int rows = a.g * a.qpb;
        for (int idx = threadIdx.x; idx < (BM - rows) * 8 * C::KSL; idx += NUM_THREADS) {
            const int row = rows + idx / (8 * C::KSL), s = (idx / 8) % C::KSL, q = idx % 8;
            *reinterpret_cast<uint4*>(smem + C::OFF_Q + s * BOX + row * 128 + q * 16) = make_uint4(0u, 0u, 0u, 0u);
        }
        fence_proxy_async_smem();
    }
    if (warp == WMMA) {
        tmem_alloc(smem_u32(tmem_slot), TMEM_COLS);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;

    if (warp >= WARP_LOAD) {
        regs_dec<KV8 ? kRegsOther8 : kRegsOther>();
        if (KV8 && warp != WMMA) {
            if constexpr (KV8) {
                const bool team_v = warp >= WARP_V8;
                const int wid = warp % 4;
                int nc = 0;                         // slots of the team's ring filled
                for (int r = 0;; ++r) {
                    const int w = warp == WARP_LOAD ? claim_item(r) : next_item(r);
                    if (w < 0) break;
                    const Item it = describe(w);
                    if (it.t.n_tiles == it.first) continue;
                    const bool done =
                        team_v ? fp8_item<D, C, true>(a, smem, r_full(C::NK8), r_empty(C::NK8), abort_flag, it.b, it.hkv,
                                                      it.skv, it.t.kv_begin, it.first, it.t.n_tiles, wid, lane, nc)
                               : fp8_item<D, C, false>(a, smem, r_full(0), r_empty(0), abort_flag, it.b, it.hkv,
                                                       it.skv, it.t.kv_begin, it.first, it.t.n_tiles, wid, lane, nc);
                    if (!done) break;
                }
            }
        } else if (!KV8 && warp == WARP_LOAD) {
            // ------------------------------------------------------------ producer
            int nc = 0, nq = 0;                     // ring chunks and Q blocks issued (lane 0's count)
            bool ok = true;
            if (lane == 0) {
                tma_prefetch_desc(&tm_q);
                tma_prefetch_desc(&tm_k);
                tma_prefetch_desc(&tm_v);
            }
            // Waits for the next ring slot and arms its barrier for `bytes`.
            // TMA-tensor layouts: lane 0 alone (it issues every copy).  Paged:
            // warp-collective, every lane learning the slot (lanes copy one
            // page block each).
            // Paged caches whose page size is not a multiple of 8 are gathered
            // row by row with cp.async into the same layout the page-block
            // boxes give; a slot's full barrier then takes lane 0's plain
            // arrival once that slot's copies have landed.
            const bool gather = MODE == kPaged && a.bt_k == 0;
            auto take_slot = [&](uint32_t& dst, uint32_t& full, uint32_t bytes) -> bool {
                const int s = nc % C::NS;
                bool good = true;
                if (MODE != kPaged || lane == 0) {
                    good = mbar_wait(r_empty(s), ((nc / C::NS) & 1) ^ 1, abort_flag);
                    if (good && !gather) mbar_arrive_expect_tx(r_full(s), bytes);
                }
                if constexpr (MODE == kPaged) {
                    good = __shfl_sync(0xffffffffu, good, 0);
                    __syncwarp();                    // the expect-tx precedes every lane's copy
                }
                full = r_full(s);
                dst = sb + C::OFF_RING + s * SLOT;
                if (good) ++nc;
                return good;
            };
            // Paged: lane l < n copies block l (bt keys from key0 + l * bt) if it
            // starts below the request's end; returns the bytes of those copies.
            auto paged_blocks = [&](const Item& it, int key0, int bt, int n) -> int {
                const int key = key0 + lane * bt;
                return __popc(__ballot_sync(0xffffffffu, lane < n && key < it.skv)) * bt;
            };
            auto paged_copy = [&](const Item& it, const CUtensorMap* map, uint32_t dst, uint32_t full, int key0,
                                  int bt, int n, int group_stride, int slice0) {
                const int key = key0 + lane * bt;
                if (lane < n && key < it.skv) {
                    const int page = __ldg(a.table + (size_t)it.b * a.max_pages + key / a.page_size);
                    const long row = (long)page * a.page_size + key % a.page_size;
                    // a page id outside the pool reads as zeros (the coordinate is out of range)
                    tma_load_5d(dst + (lane * bt / 8) * group_stride, map, full, 0, 0, slice0, (int)(row / 8),
                                it.hkv);
                }
            };
            // Gathered rows: keys key0 .. key0 + nkeys - 1 (those below the
            // request's end), 64-column slices slice0 .. slice0 + nsl - 1, as
            // [8-key group][slice][8 keys][128 B] with the 128-byte swizzle; a
            // page id outside the pool reads as zeros.  The copies are
            // committed as one group; the previous slot's barrier is then
            // released once its group has landed (one slot stays in flight).
            uint32_t pend = 0;                      // full barrier of the slot still in flight
            auto release = [&](int keep) {
                if (pend == 0) return;
                if (keep) cp_async_wait<1>(); else cp_async_wait<0>();
                fence_proxy_async_smem();           // cp.async writes, read by the tensor core
                __syncwarp();
                if (lane == 0) mbar_arrive(pend);
                pend = 0;
            };
            auto gather_copy = [&](const Item& it, const void* cache, uint32_t dst, uint32_t full, int key0,
                                   int nkeys, int slice0, int nsl, int group_stride) {
                const uint16_t* base = static_cast<const uint16_t*>(cache);
                for (int idx = lane; idx < nkeys * nsl * 8; idx += 32) {
                    const int r = idx / (nsl * 8), s = (idx / 8) % nsl, q = idx % 8;
                    const int key = key0 + r;
                    if (key >= it.skv) continue;
                    const int page = __ldg(a.table + (size_t)it.b * a.max_pages + key / a.page_size);
                    const bool in_pool = page >= 0 && page < a.num_pages;
                    const long row = in_pool ? (long)page * a.page_size + key % a.page_size : 0;
                    const uint16_t* src = base + (row * a.Hkv + it.hkv) * D + 64 * (slice0 + s) + 8 * q;
                    cp_async16(dst + (r / 8) * group_stride + s * 1024 + (r % 8) * 128 + ((q ^ (r % 8)) << 4), src,
                               in_pool ? 16u : 0u);
                }
                cp_async_commit();
                release(1);
                pend = full;
            };
            auto load_k = [&](const Item& it, int j) -> bool {
                for (int c = 0; c < C::CK; ++c) {
                    uint32_t dst, full;
                    if (gather) {
                        if (!take_slot(dst, full, 0)) return false;
                        gather_copy(it, a.k_cache, dst, full, j * BN, BN, c * C::KSL_C, C::KSL_C, C::K_GROUP);
                    } else if constexpr (MODE == kPaged) {
                        const int n = BN / a.bt_k;
                        const int rows = paged_blocks(it, j * BN, a.bt_k, n);
                        if (!take_slot(dst, full, (uint32_t)(rows * 128 * C::KSL_C))) return false;
                        paged_copy(it, &tm_k, dst, full, j * BN, a.bt_k, n, C::K_GROUP, c * C::KSL_C);
                    } else {                        // lane 0 only
                        if (!take_slot(dst, full, C::K_CHUNK)) return false;
#pragma unroll
                        for (int s = 0; s < C::KSL_C; ++s) {
                            const int col = 64 * (c * C::KSL_C + s);
                            if constexpr (MODE == kPacked)
                                tma_load_3d(dst + s * C::K_SLICE, &tm_k, full, col, it.hkv, it.ks + j * BN);
                            else
                                tma_load_4d(dst + s * C::K_SLICE, &tm_k, full, col, j * BN, it.hkv, it.b);
                        }
                    }
                }
                return true;
            };
            auto load_v = [&](const Item& it, int j) -> bool {
                for (int c = 0; c < C::CV; ++c) {
                    uint32_t dst, full;
                    const int key0 = j * BN + c * C::VKEYS;
                    if (gather) {
                        if (!take_slot(dst, full, 0)) return false;
                        gather_copy(it, a.v_cache, dst, full, key0, C::VKEYS, 0, C::KSL, C::V_GROUP);
                    } else if constexpr (MODE == kPaged) {
                        const int n = C::VKEYS / a.bt_v;
                        const int rows = paged_blocks(it, key0, a.bt_v, n);
                        if (!take_slot(dst, full, (uint32_t)(rows * 128 * C::KSL))) return false;
                        paged_copy(it, &tm_v, dst, full, key0, a.bt_v, n, C::V_GROUP, 0);
                    } else {                        // lane 0 only
                        if (!take_slot(dst, full, C::V_CHUNK)) return false;
#pragma unroll
                        for (int s = 0; s < C::KSL; ++s) {
                            if constexpr (MODE == kPacked)
                                tma_load_3d(dst + s * C::V_SLICE, &tm_v, full, 64 * s, it.hkv, it.ks + key0);
                            else
                                tma_load_4d(dst + s * C::V_SLICE, &tm_v, full, 64 * s, key0, it.hkv, it.b);
                        }
                    }
                }
                return true;
            };
            for (int r = 0; ok; ++r) {
                const int w = claim_item(r);
                if (w < 0) break;
                const Item it = describe(w);
                const int c = count_tiles(it);
                if (c == 0) continue;
                if (lane == 0) {
                    ok = mbar_wait(q_empty, (nq & 1) ^ 1, abort_flag);
                    if (ok) {
                        if constexpr (PACKED) {
                            // {64, g, qpb} boxes: rows q * g + head of queries q0.. of the group
                            mbar_arrive_expect_tx(q_full, (uint32_t)(C::KSL * g * qpb * 128));
#pragma unroll
                            for (int s = 0; s < C::KSL; ++s)
                                tma_load_3d(sb + C::OFF_Q + s * BOX, &tm_q, q_full, 64 * s, it.hq, it.qs + it.t.q0);
                        } else {
                            mbar_arrive_expect_tx(q_full, C::KSL * BOX);
#pragma unroll
                            for (int s = 0; s < C::KSL; ++s)
                                tma_load_4d(sb + C::OFF_Q + s * BOX, &tm_q, q_full, 64 * s, it.t.q0, it.hq, it.b);
                        }
                        ++nq;
                    }
                }
                ok = __shfl_sync(0xffffffffu, ok, 0);
                if (!ok) break;
                // K of tile 0, then (K of tile i+1, V of tile i) for each tile i
                TileIter tiles(it.mrow, it.first, it.t.n_tiles, it.t.kv_end, lane);
                int j = tiles.next();
                if (MODE == kPaged || lane == 0) ok = load_k(it, j);
                if (MODE != kPaged) ok = __shfl_sync(0xffffffffu, ok, 0);
                while (ok && j >= 0) {
                    const int jn = tiles.next();
                    if (MODE == kPaged || lane == 0) {
                        if (jn >= 0) ok = load_k(it, jn);
                        if (ok) ok = load_v(it, j);
                    }
                    if (MODE != kPaged) ok = __shfl_sync(0xffffffffu, ok, 0);
                    j = jn;
                }
                // the item's last gathered slot, before the next item's waits
                // (its Q slot frees only once this item's MMAs have run)
                if (gather) release(0);
            }
            if (gather) cp_async_wait<0>();         // no copy outlives the loop
            if (lane == 0 && *abort_flag && !gather) {
                // let the copies in flight land: the last load of each slot
                for (int s = 0; s < C::NS && s < nc; ++s) {
                    const int last = nc - 1 - ((nc - 1 - s) % C::NS);
                    mbar_drain(r_full(s), (last / C::NS) & 1);
                }
                if (nq > 0) mbar_drain(q_full, (nq - 1) & 1);
            }
        } else if (warp == WMMA) {
            // ------------------------------------------------------------ MMA issuer
            // Lane 0 alone issues every MMA of an item but its last P V (a
            // single polling lane keeps the issue loop short); the whole warp
            // takes the last P V, whose value rows past the request's end it
            // zeroes first (packed layouts).
            int nc = 0, nq = 0;     // ring chunks (kPaged8: of the key ring) and Q blocks consumed
            int nv = 0;             // kPaged8: chunks of the value ring consumed
            int g_t = 0;            // visited tiles of earlier items (S buffer / p_full parity)
            int oe = 0;             // o_empty phases waited
            bool ok = true;
            // slot and phase of the k-th next chunk (v: of values)
            auto slot_of = [&](bool v, int k) -> int {
                if constexpr (KV8) return v ? C::NK8 + (nv + k) % C::NV8 : (nc + k) % C::NK8;
                else return (nc + k) % C::NS;
            };
            auto phase_of = [&](bool v, int k) -> uint32_t {
                if constexpr (KV8) return (v ? (nv + k) / C::NV8 : (nc + k) / C::NK8) & 1;
                else return ((nc + k) / C::NS) & 1;
            };
            auto chunk_addr = [&](bool v, int k) { return sb + C::OFF_RING + slot_of(v, k) * SLOT; };
            auto take = [&](bool v, int n) -> bool {        // lane 0: the next n ring chunks have landed
                for (int k = 0; k < n; ++k)
                    if (!mbar_wait(r_full(slot_of(v, k)), phase_of(v, k), abort_flag)) return false;
                tc_fence_after();
                return true;
            };
            // lane 0; kPaged8: the first of two chunks is released as soon as its
            // MMAs are issued (so that the wideners refill it meanwhile)
            auto release_half = [&](bool v) { mma_commit(r_empty(slot_of(v, 0))); };
            auto release = [&](bool v, int n) {             // lane 0
                for (int k = KV8 ? n - 1 : 0; k < n; ++k) mma_commit(r_empty(slot_of(v, k)));
                if (KV8 && v) nv += n;
                else nc += n;
            };
            // S of visited tile gi = Q K^T over D / 16 steps of 16 columns (lane 0)
            auto issue_qk = [&](int gi) -> bool {
                if (!take(false, C::CK)) return false;
                const uint32_t d = tmem + COL_S0 + (gi & 1) * BN;
                // descriptors of the Q tile and of each K chunk, advanced by
                // constant offsets (>> 4) per step
                const uint64_t qdesc = make_sdesc_sw128(sb + C::OFF_Q, 16, 1024);
                uint64_t kdesc[C::CK];
#pragma unroll
                for (int c = 0; c < C::CK; ++c) kdesc[c] = make_sdesc_sw128(chunk_addr(false, c), 16, C::K_GROUP);
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk) {
                    constexpr int PER = D / 16 / C::CK;       // steps per K chunk
                    const int kl = kk % PER;
                    const uint32_t qoff = (kk / 4) * BOX + (kk % 4) * 32;
                    const uint32_t koff = (kl / 4) * C::K_SLICE + (kl % 4) * 32;
                    if constexpr (C::TQ)
                        mma_bf16_ts(d, tmem + COL_Q8 + 8 * kk, kdesc[kk / PER] + (koff >> 4), IDESC_QK,
                                    kk > 0 ? 1u : 0u);
                    else
                        mma_bf16_ss(d, qdesc + (qoff >> 4), kdesc[kk / PER] + (koff >> 4), IDESC_QK,
                                    kk > 0 ? 1u : 0u);
                    if (KV8 && C::CK == 2 && kk == PER - 1) release_half(false);
                }
                mma_commit(s_full(gi & 1));
                release(false, C::CK);
                return true;
            };
            // O (+)= P V of visited tile gi: 8 steps of 16 keys (lane 0)
            auto mma_pv = [&](int gi, bool fresh) {
                const uint32_t p = tmem + COL_S0 + (gi & 1) * BN;
                uint64_t vdesc[C::CV];
#pragma unroll
                for (int c = 0; c < C::CV; ++c) vdesc[c] = make_sdesc_sw128(chunk_addr(true, c), C::V_SLICE, C::V_GROUP);
#pragma unroll
                for (int kk = 0; kk < BN / 16; ++kk) {
                    constexpr int PER = BN / 16 / C::CV;       // steps per V chunk
                    const int kc = (kk % PER) * 16;
                    mma_bf16_ts(tmem + COL_O, p + kk * 8, vdesc[kk / PER] + (((kc / 8) * C::V_GROUP) >> 4), IDESC_PV,
                                (!fresh || kk > 0) ? 1u : 0u);
                    if (KV8 && C::CV == 2 && kk == PER - 1) release_half(true);
                }
                release(true, C::CV);
                mma_commit(o_ready);
            };
            auto issue_pv = [&](int gi, bool fresh) -> bool {      // lane 0
                if (!mbar_wait(p_full(gi & 1), (gi >> 1) & 1, abort_flag)) return false;
                if (!take(true, C::CV)) return false;
                mma_pv(gi, fresh);
                return true;
            };
            // lane 0: the epilogue of every earlier item has read O
            auto wait_o_empty = [&](int n_item) -> bool {
                for (; oe < n_item; ++oe)
                    if (!mbar_wait(o_empty, oe & 1, abort_flag)) return false;
                return true;
            };
            if constexpr (KV8) {
                // the same order from two copies of each step (small code); the
                // next item is looked up while the last P is awaited
                auto tiles_of = [&](int w) { const Item it = describe(w); return it.t.n_tiles - it.first; };
                int w = next_item(0);
                int c = w >= 0 ? tiles_of(w) : 0;
                for (int r = 0; ok && w >= 0; ++r) {
                    if (lane == 0 && c > 0) {
                        ok = mbar_wait(q_full, nq++ & 1, abort_flag);
                        if (ok) ok = issue_qk(g_t);
                        for (int i = 0; i + 1 < c && ok; ++i) {
                            ok = issue_qk(g_t + i + 1) && wait_o_empty(r);
                            if (ok) ok = issue_pv(g_t + i, i == 0);
                        }
                        if (ok) mma_commit(q_empty);               // every S of the item is issued
                    }
                    ok = __shfl_sync(0xffffffffu, ok, 0);
                    if (!ok) break;
                    const int wn = next_item(r + 1);
                    const int cn = wn >= 0 ? tiles_of(wn) : 0;
                    if (lane == 0) {
                        ok = wait_o_empty(r);
                        if (ok && c > 0) ok = issue_pv(g_t + c - 1, c == 1);
                        // one phase per item: every MMA of the item has completed
                        if (ok) mma_commit(o_final);
                    }
                    ok = __shfl_sync(0xffffffffu, ok, 0);
                    g_t += c;
                    w = wn;
                    c = cn;
                }
            }
            for (int r = 0, n_item = 0; !KV8 && ok; ++r, ++n_item) {
                const int w = next_item(r);
                if (w < 0) break;
                const Item it = describe(w);
                const int c = count_tiles(it);
                if (lane == 0) {
                    if (c > 0) {
                        ok = mbar_wait(q_full, nq++ & 1, abort_flag);
                        if (ok) ok = issue_qk(g_t);
                        if (ok && c > 1) ok = issue_qk(g_t + 1);
                        if (ok) ok = wait_o_empty(n_item);
                        if (ok && c > 1) ok = issue_pv(g_t, true);
                        for (int i = 1; i + 1 < c && ok; ++i) {
                            ok = issue_qk(g_t + i + 1);
                            if (ok) ok = issue_pv(g_t + i, false);
                        }
                        if (ok) mma_commit(q_empty);               // every S of the item is issued
                        // BSHD: no value row to zero, lane 0 issues the last P V too
                        if (!PACKED && ok) ok = issue_pv(g_t + c - 1, c == 1);
                    } else {
                        ok = wait_o_empty(n_item);
                    }
                }
                ok = __shfl_sync(0xffffffffu, ok, 0);
                nc = __shfl_sync(0xffffffffu, nc, 0);
                nq = __shfl_sync(0xffffffffu, nq, 0);
                oe = __shfl_sync(0xffffffffu, oe, 0);
                if (PACKED && ok && c > 0) {
                    // the item's last P V, by the whole warp
                    const int gi = g_t + c - 1;
                    ok = __all_sync(0xffffffffu, mbar_wait(p_full(gi & 1), (gi >> 1) & 1, abort_flag));
                    for (int k = 0; k < C::CV && ok; ++k)
                        ok = __all_sync(0xffffffffu,
                                        mbar_wait(r_full((nc + k) % C::NS), ((nc + k) / C::NS) & 1, abort_flag));
                    if (ok) {
                        tc_fence_after();
                        const int nvalid = PACKED ? min(BN, it.skv - (it.t.n_tiles - 1) * BN) : BN;
                        if (PACKED && nvalid < BN) {
                            for (int idx = lane; idx < (BN - nvalid) * 8 * C::KSL; idx += 32) {
                                const int key = nvalid + idx / (8 * C::KSL);
                                const int s = (idx / 8) % C::KSL, q = idx % 8;
                                const int kc = key % C::VKEYS;
                                const uint32_t off = chunk_addr(true, key / C::VKEYS) - sb + s * C::V_SLICE +
                                                     (kc / 8) * C::V_GROUP + (kc % 8) * 128 + q * 16;
                                *reinterpret_cast<uint4*>(smem + off) = make_uint4(0u, 0u, 0u, 0u);
                            }
                            fence_proxy_async_smem();
                            __syncwarp();
                            tc_fence_after();
                        }
                        if (lane == 0) mma_pv(gi, c == 1);
                        nc = __shfl_sync(0xffffffffu, nc, 0);
                    }
                }
                g_t += c;
                // one phase per item: every MMA of the item has completed
                if (ok && lane == 0) mma_commit(o_final);
                __syncwarp();
            }
            if (lane == 0) {
                mma_commit(drain);
                mbar_drain(drain, 0);
            }
            __syncwarp();
            named_bar_sync(2, C::TMEM_USERS);        // softmax and epilogue warps are done with TMEM
            tc_fence_after();
            tmem_dealloc(tmem, TMEM_COLS);
        }
    } else if (warp < WARP_EPI0) {
        regs_inc<kRegsSoftmax>();
        // ------------------------------------------------------------ softmax warps 0-3
        const int r = warp * 32 + lane;                        // row of the tile == TMEM lane
        const uint32_t lane_addr = (uint32_t)(warp * 32) << 16;
        float sl = a.scale_log2, cap_i = cap_in;
        const int rq = r / g;                                  // query of this row within the block
        int gt = 0;                  // visited tiles so far
        int n = 0;                   // items finished
        bool ok = true;
        for (int rr = 0; ok; ++rr) {
            const int w = next_item(rr);
            if (w < 0) break;
            const Item itm = describe(w);
            const TileInfo ti = itm.t;
            const uint8_t* mrow = itm.mrow;
            if constexpr (KV8) {
                const float ks = a.k_scale ? a.k_scale[itm.b * a.Hkv + itm.hkv] : 1.f;
                sl = a.scale_log2 * ks;
                cap_i = cap_in * ks;
            }
            const long p_row = (long)ti.q0 + rq + itm.skv - itm.sq;
            const int lim = (int)key_hi(p_row, itm.skv, a.causal, wr);   // visible keys: [lo, lim)
            const int lo = (int)key_lo(p_row, itm.skv, wl);
            float m_ref = -INFINITY;
            float l_run = 0.f;
            bool has_ref = false;                      // kPaged8: every row of the warp has a reference max
            int it = 0;
            TileIter tiles(mrow, itm.first, ti.n_tiles, ti.kv_end, lane);
            auto fetch = [&](int j, uint8_t* mb) {
                if constexpr (!KV8) {                  // kPaged8 has no padding mask
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const int key = j * BN + q * 32 + lane;
                        mb[q] = (mrow && j >= 0 && key < ti.kv_end) ? mrow[key] : (uint8_t)(mrow ? 0 : 1);
                    }
                }
            };
            int j = tiles.next();
            uint8_t mb[4];
            fetch(j, mb);
            while (j >= 0) {
                const int jn = tiles.next();
                uint8_t mbn[4];
                fetch(jn, mbn);
                uint32_t mw[4];
                bool all_kept = true;
                if constexpr (!KV8) {
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        mw[q] = __ballot_sync(0xffffffffu, mb[q] != 0);
                        all_kept = all_kept && (mw[q] == 0xffffffffu);
                    }
                }
                const int kbase = j * BN;
                const bool need_mask = (kbase + BN > ti.lim_first) || kbase < ti.lo_last || !all_kept;
                const uint32_t col_s = COL_S0 + (gt & 1) * BN;

                ok = __all_sync(0xffffffffu, mbar_wait(s_full(gt & 1), (gt >> 1) & 1, abort_flag));
                if (!ok) break;
                tc_fence_after();
                const bool capped = cap_out != 0.f;
                // kPaged8 (need_mask is the same for the whole warp): masked tiles and
                // scales that are not positive are prepared in place; an unmasked
                // capped tile takes its maximum from the raw scores and applies the
                // cap with the exponential.  mul scales the row's values there.
                const float to_y = cap_i * 0.34657359027997264f;         // scale / cap: ln(2) / 2
                const bool prepare = KV8 && (need_mask || !(sl > 0.f));
                const bool late_cap = KV8 && capped && !prepare;
                const float mul = !KV8 ? sl : (capped ? cap_out : (sl > 0.f ? sl : 1.f));
                if (prepare)
                    prepare_scores(tmem + lane_addr + col_s, capped, to_y, sl > 0.f ? 1.f : sl, lo - kbase, lim - kbase);
                uint32_t sr[BN];
                tmem_ld128(tmem + lane_addr + col_s, sr);
                float* s = reinterpret_cast<float*>(sr);
                float most_lead = kLead8 + kRescaleThreshold;        // kPaged8: of the max over the reference
                if constexpr (KV8) {
                    // Once every row of the warp has a reference max, a plain tile
                    // is exponentiated against it without taking its own; a row
                    // sum past kSumLimit8 (no P of the row is larger than the sum, and
                    // float16 holds that) sends the warp to the full step, the scores
                    // being still in TMEM.
                    if (has_ref && !prepare && !capped) {
                        uint32_t pk[BN / 2];
                        const float rs = exp_row<true>(s, mul, m_ref, pk);
                        if (!__any_sync(0xffffffffu, rs > kSumLimit8)) {
                            tmem_st64(tmem + lane_addr + col_s, pk);
                            l_run += rs;
                            tc_fence_before();
                            mbar_arrive(p_full(gt & 1));
                            ++it;
                            ++gt;
                            j = jn;
                            continue;
                        }
                        tmem_ld128(tmem + lane_addr + col_s, sr);
                        // a row with such a sum has a score 9 binades or more above
                        // its reference: it takes a new one, so that the tiles after
                        // this one are plain again
                        most_lead = kLead8 + 2.f;
                    }
                }

                const bool fast = KV8 || (!need_mask && sl > 0.f && !capped);
                float mx8[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) mx8[e] = -INFINITY;
                if (fast) {
#pragma unroll
                    for (int c = 0; c < BN; c += 2) mx8[(c >> 1) & 7] = fmax3(mx8[(c >> 1) & 7], s[c], s[c + 1]);
                } else {
                    uint32_t vis[4];
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const int rel = lim - (kbase + 32 * q);
                        const uint32_t below = rel >= 32 ? 0xffffffffu : (rel <= 0 ? 0u : ((1u << rel) - 1u));
                        const int rlo = lo - (kbase + 32 * q);
                        const uint32_t above = rlo <= 0 ? 0xffffffffu : (rlo >= 32 ? 0u : ~((1u << rlo) - 1u));
                        vis[q] = mw[q] & below & above;
                    }
                    if (capped) {
#pragma unroll
                        for (int c = 0; c < BN; ++c) {
                            const float x = ((vis[c / 32] >> (c % 32)) & 1u)
                                                ? softcap_log2(s[c], cap_i, cap_out) : -INFINITY;
                            s[c] = x;
                            mx8[c & 7] = fmaxf(mx8[c & 7], x);
                        }
                    } else {
#pragma unroll
                        for (int c = 0; c < BN; ++c) {
                            const float x = ((vis[c / 32] >> (c % 32)) & 1u) ? s[c] * sl : -INFINITY;
                            s[c] = x;
                            mx8[c & 7] = fmaxf(mx8[c & 7], x);
                        }
                    }
                }
#pragma unroll
                for (int e = 0; e < 4; ++e) mx8[e] = fmaxf(mx8[e], mx8[e + 4]);
                const float mx_raw = fmaxf(fmaxf(mx8[0], mx8[1]), fmaxf(mx8[2], mx8[3]));
                const float mx = !fast ? mx_raw : (late_cap ? tanh_mufu(mx_raw * to_y) * mul : mx_raw * mul);
                float alpha = 1.f;
                // (the difference of two near values is exact: no large score rounds past the threshold)
                if (KV8 ? mx - m_ref > most_lead : mx > m_ref + kRescaleThreshold) {
                    const float ref = KV8 ? mx - kLead8 : mx;
                    alpha = fast_exp2(m_ref - ref);
                    m_ref = ref;
                }
                const float m_use = m_ref == -INFINITY ? 0.f : m_ref;
                const float fa = fast ? mul : 1.f;
                float rs;
                if (late_cap) {
                    rs = capped_exp(tmem + lane_addr + col_s, to_y, cap_out, m_use);
                } else {
                    uint32_t pk[BN / 2];
                    rs = exp_row<MF16>(s, fa, m_use, pk);
                    tmem_st64(tmem + lane_addr + col_s, pk);      // P over the first 64 columns of S
                }
                l_run = l_run * alpha + rs;
                if constexpr (KV8) has_ref = __all_sync(0xffffffffu, m_ref != -INFINITY);

                if (it > 0 && __any_sync(0xffffffffu, alpha != 1.f)) {
                    // PV of the previous tile must have completed before O is rescaled
                    ok = __all_sync(0xffffffffu, mbar_wait(o_ready, (gt - 1) & 1, abort_flag));
                    if (!ok) break;
                    tc_fence_after();
#pragma unroll 1
                    for (int c = 0; c < D / 32; ++c) {
                        float o[32];
                        tmem_ld32(tmem + lane_addr + COL_O + 32 * c, o);
#pragma unroll
                        for (int e = 0; e < 32; ++e) o[e] *= alpha;
                        tmem_st32(tmem + lane_addr + COL_O + 32 * c, reinterpret_cast<uint32_t*>(o));
                    }
                }
                tc_fence_before();
                mbar_arrive(p_full(gt & 1));
                ++it;
                ++gt;
                j = jn;
#pragma unroll
                for (int q = 0; q < 4; ++q) mb[q] = mbn[q];
            }
            if (!ok) break;
            // hand the row statistics to the epilogue once it has read the previous ones
            if (n > 0) {
                ok = __all_sync(0xffffffffu, mbar_wait(stats_empty, (n - 1) & 1, abort_flag));
                if (!ok) break;
            }
            st_m[r] = m_ref;
            st_l[r] = l_run;
            if (r == 0) *st_cnt = it;
            mbar_arrive(stats_full);
            ++n;
        }
        named_bar_arrive(2, C::TMEM_USERS);
    } else {
        regs_dec<KV8 ? kRegsEpi8 : kRegsEpi>();
        // ------------------------------------------------------------ epilogue warps 4-7
        const int r = (warp - WARP_EPI0) * 32 + lane;
        const uint32_t lane_addr = (uint32_t)((warp % 4) * 32) << 16;
        const int rq = r / g, rh = r % g;           // query and head of this row within the block
        int n = 0;                   // items finished
        int nb = 0;                  // output boxes stored (staging buffer alternation)
        bool ok = true;
        // kPaged8: the Q block of item w (fill_q8), an item ahead
        int nq = 0, w = -1, w_after = -1;
        auto fill_q = [&]() -> bool {
            if (w_after < 0) return true;
            const Item it = describe(w_after);
            if (it.t.n_tiles == it.first) return true;
            return fill_q8<D, F16, C>(a, smem, q_full, q_empty, abort_flag, it.qs + it.t.q0, it.t.rows_valid * g, it.hkv,
                                      g, warp % 4, lane, tmem, nq);
        };
        if constexpr (KV8) {
            w_after = next_item(0);
            ok = fill_q();
        }
        for (int rr = 0;; ++rr) {
            w = KV8 ? w_after : next_item(rr);
            if (w < 0) break;
            bool q_ok = ok;
            if constexpr (KV8) {
                w_after = next_item(rr + 1);
                q_ok = q_ok && fill_q();
            }
            const Item itm = describe(w);
            const TileInfo ti = itm.t;
            // warp-collective waits: the warp must be converged at the
            // .aligned barrier below and at every tcgen05.ld
            ok = q_ok && __all_sync(0xffffffffu, mbar_wait(stats_full, n & 1, abort_flag));
            if (ok) ok = __all_sync(0xffffffffu, mbar_wait(o_final, n & 1, abort_flag));
            if (!named_bar_and(3, BM, ok)) break;     // the whole warpgroup stops together
            tc_fence_after();
            const int cnt = *st_cnt;
            const float m_ref = st_m[r];
            const float l_run = st_l[r];
            const int head = itm.hq + (PACKED ? rh : 0);
            const bool row_ok = (PACKED ? r < g * qpb : true) && rq < ti.rows_valid;
            // output row: [B, Sq, Hq] (kBSHD) or [total_q, Hq] (packed)
            const size_t orow = PACKED ? ((size_t)itm.qs + ti.q0 + rq) * a.Hq + head
                                       : ((size_t)itm.b * a.Sq + ti.q0 + rq) * a.Hq + head;
            // kPaged8: only a sum of exactly 0 means a row without a key; a NaN sum (a
            // query that is no number) goes on as it is, to the joining kernel too
            const bool some = KV8 ? l_run != 0.f : l_run > 0.f;
            float inv = some ? 1.f / l_run : 0.f;
            float lse2 = some ? m_ref + log2f(l_run) : -INFINITY;
            if (sinks && some && parts == 1) {
                const float s2 = sinks[head] * 1.4426950408889634f;
                if (s2 == INFINITY && !(KV8 && isnan(l_run))) {
                    inv = 0.f;
                    lse2 = INFINITY;
                } else {
                    const float M = fmaxf(m_ref, s2);
                    const float keep = fast_exp2(m_ref - M);
                    const float l_tot = l_run * keep + fast_exp2(s2 - M);
                    inv = keep / l_tot;
                    lse2 = M + log2f(l_tot);
                }
            }
            if constexpr (KV8)
                if (a.v_scale) inv *= a.v_scale[itm.b * a.Hkv + itm.hkv];
            if (KV8 && parts > 1) {
                // a part of the keys: FP32 rows for the joining kernel
                const size_t prow = (size_t)w * BM + r;
                if (cnt > 0) {
#pragma unroll 1
                    for (int c = 0; c < D / 32; ++c) {
                        float f[32];
                        __syncwarp();
                        tmem_ld32(tmem + lane_addr + COL_O + 32 * c, f);
                        if (c == D / 32 - 1) {
                            tc_fence_before();
                            mbar_arrive(stats_empty);
                            mbar_arrive(o_empty);
                        }
                        if (row_ok) {
                            float4* dst = reinterpret_cast<float4*>(a.part_o + prow * D + 32 * c);
#pragma unroll
                            for (int e = 0; e < 8; ++e)
                                dst[e] = make_float4(f[4 * e] * inv, f[4 * e + 1] * inv, f[4 * e + 2] * inv,
                                                     f[4 * e + 3] * inv);
                        }
                    }
                } else {
                    mbar_arrive(stats_empty);
                    mbar_arrive(o_empty);
                }
                if (row_ok) a.part_lse[prow] = lse2;
                ++n;
                continue;
            }
            // Whole blocks go out with TMA; a packed block cut by its request's
            // end is written row by row (its box would reach the next request).
            // The choice is the same for every thread of the item.
            const bool boxed = !PACKED || ti.rows_valid == qpb;
            constexpr int HALF = KV8 || D < 128 ? 64 : 128;     // O columns read per pass
            // O / l packed to 16 bits, HALF columns at a time; O is free once the
            // last columns are read
            auto read_o = [&](int half, uint32_t* ow) {
                // tcgen05.ld is warp-collective (.sync.aligned): reconverge first
                __syncwarp();
#pragma unroll
                for (int c = 0; c < HALF / 32; ++c) {
                    float f[32];
                    tmem_ld32(tmem + lane_addr + COL_O + HALF * half + 32 * c, f);
#pragma unroll
                    for (int e = 0; e < 16; ++e) ow[16 * c + e] = pack2<F16>(f[2 * e] * inv, f[2 * e + 1] * inv);
                }
                if (half == D / HALF - 1) {
                    tc_fence_before();
                    mbar_arrive(stats_empty);
                    mbar_arrive(o_empty);
                }
            };
            constexpr int UNROLL = KV8 ? 1 : D / HALF;  // small code (see prepare_scores)
            if (cnt > 0 && boxed) {
#pragma unroll UNROLL
                for (int half = 0; half < D / HALF; ++half) {
                    uint32_t ow[HALF / 2];
                    read_o(half, ow);
                    // 64-column boxes through the alternating staging buffers
#pragma unroll
                    for (int sub = 0; sub < HALF / 64; ++sub, ++nb) {
                        const uint32_t stage = sb + C::OFF_STAGE + (nb & 1) * BOX;
                        if (r == 0) bulk_wait_read_1();       // the store two boxes back has read this buffer
                        __syncwarp();
                        named_bar_sync(3, BM);
#pragma unroll
                        for (int q = 0; q < 8; ++q) {
                            const uint32_t* u = ow + 32 * sub + 4 * q;
                            st_shared_v4(stage + r * 128 + ((q ^ (r & 7)) << 4), u[0], u[1], u[2], u[3]);
                        }
                        fence_proxy_async_smem();
                        named_bar_sync(3, BM);
                        if (r == 0) {
                            const int col = HALF * half + 64 * sub;
                            if constexpr (PACKED)
                                tma_store_3d(&tm_o, stage, col, itm.hq, itm.qs + ti.q0);
                            else
                                tma_store_4d(&tm_o, stage, col, ti.q0, itm.hq, itm.b);
                            bulk_commit_group();
                        }
                    }
                }
            } else if (cnt > 0) {
#pragma unroll UNROLL
                for (int half = 0; half < D / HALF; ++half) {
                    uint32_t ow[HALF / 2];
                    read_o(half, ow);
                    if (row_ok) {
                        uint4* dst = reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.o) + orow * D + HALF * half);
#pragma unroll
                        for (int e = 0; e < HALF / 8; ++e)
                            dst[e] = make_uint4(ow[4 * e], ow[4 * e + 1], ow[4 * e + 2], ow[4 * e + 3]);
                    }
                }
            } else {
                mbar_arrive(stats_empty);
                mbar_arrive(o_empty);
                if (row_ok) {
                    uint4* dst = reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.o) + orow * D);
#pragma unroll
                    for (int e = 0; e < D / 8; ++e) dst[e] = make_uint4(0u, 0u, 0u, 0u);
                }
            }
            if (row_ok && a.lse) a.lse[orow] = lse2 * kLn2;
            ++n;
        }
        if (r == 0) bulk_wait_read_all();
        tc_fence_before();
        named_bar_arrive(2, C::TMEM_USERS);
    }
    if (threadIdx.x == 0 && *abort_flag) atomicExch(&g_onetile_error, (int)kErrPrefillWait);
}

template <int D, int MODE, bool OPTS, bool F16>
cudaError_t launch_onetile(const CUtensorMap& tm_q, const CUtensorMap& tm_k, const CUtensorMap& tm_v,
                           const CUtensorMap& tm_o, const PrefillArgs& a, long max_items, int n_qtiles,
                           cudaStream_t stream) {
    using C = Cfg<D, MODE>;
    cudaError_t e = cudaFuncSetAttribute(onetile_kernel<D, MODE, OPTS, F16>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM_BYTES);
    if (e != cudaSuccess) return e;
    const long sms = a.num_sms > 0 ? a.num_sms : 148;
    const long grid = max_items < sms ? max_items : sms;    // persistent: one CTA per SM
    if (grid <= 0) return cudaSuccess;
    onetile_kernel<D, MODE, OPTS, F16><<<(unsigned)grid, num_threads(MODE), C::SMEM_BYTES, stream>>>(tm_q, tm_k, tm_v,
                                                                                              tm_o, a, n_qtiles);
    return cudaGetLastError();
}

int take_error() {
    int v = 0;
    if (cudaMemcpyFromSymbol(&v, g_onetile_error, sizeof(int)) != cudaSuccess) return -1;
    if (v != 0) {
        const int zero = 0;
        cudaMemcpyToSymbol(g_onetile_error, &zero, sizeof(int));
    }
    return v;
}

}  // namespace ot
}  // namespace
}  // namespace gqa
