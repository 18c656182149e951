// Latent attention in its expanded form, for prompts and chunks: packed queries
// over the keys and values that a projection of the latents gives each head.
//
//   s_ij = scale * (q_i[0:128] . k_j + q_i[128:192] . k_pe_j),  j <= i + Skv - Sq
//   o_i = sum_j softmax(s_i)_j v_j                              (FP32, base 2)
//
// per head; k and v are strided slices of the projection's output and the 64
// rotated dims k_pe are one row for all heads, so no [total_kv, H, 192] key tensor
// is ever written.  640 FLOP a (query, key, head): tensor bound.
//
// As prefill.cu, one CTA holds two 128-row query tiles of consecutive row blocks of
// one request and head, S and O of both in TMEM (S0 | S1 | O0 | O1), and the tensor
// core works on one while the other is softmaxed (TileOPs "Attention Operators",
// GQAVarlenFwdOp, mask and statistics).  What differs is the memory: a query
// tile is 48 KB, a key tile 48 KB and a value tile 32 KB, which no ring of whole
// tiles holds twice.  Keys and values go through one ring of eight 16 KB slots
// instead, in the order K0 V0 K1 V1 ...: a key tile is three slots of 64 dims, a
// value tile two of 64 keys, each of which the MMAs use and release by itself.
//   warp 8      producer: claims items (entry of the plan, head), loads
//   warp 9      MMA issuer
//   warps 0-7   softmax of the two tiles, one row per thread, and the output
//   warps 10-11 zero the value rows past a request's end in its last tile
// Items go in the plan's order (requests by their whole cost, the heaviest first, each
// one's blocks from the last, with the most keys, to the first) within groups of heads
// whose keys and values fit L2 together.  What does not fill a last round of CTAs is cut
// along the keys (Split) into FP32 parts that latent_varlen_join_kernel adds up.
//
// Measured (bf16): a chunk of 2048 tokens at the end of 16384 keys, 64 heads, 807 to 811
// us (1.59 PFLOP/s of unmasked products), eight prompts of 300 to 4000 tokens, 32 heads,
// 449, one of 4096, 20 heads, 87 replayed from a graph; a 4096-token prompt beside one query over
// 8192 keys, 12 heads, 87 in five parts of its tail (122 uncut).  The tensor core is the bound, under the power cap (1.55 to 1.7
// GHz in a loop of the long ones); short prompts lose to masked halves of diagonal tiles and
// to row blocks that a request does not fill.
#include <cmath>

#include "internal.h"
#include "prefill_tiles.cuh"
#include "ptx.cuh"

namespace gqa {
namespace {

__device__ int g_latent_varlen_error;

using namespace pf;
constexpr int NQ = 2;
constexpr int DQ = kLatentNope + kLatentRope;   // 192
constexpr int DV = kLatentV;                    // 128
constexpr int NUM_THREADS = 384;
constexpr int WARP_LOAD = 8;
constexpr int WARP_MMA = 9;
// registers as in prefill.cu: 192 * 256 + 120 * 128 = 168 * 384, the launch total
constexpr int kRegsSoftmax = 192;
constexpr int kRegsOther = 120;

constexpr int SLOT = BN * 128;                  // bytes: 128 keys x 64 dims, or 64 keys x 128 dims
constexpr int NS = 8;                           // ring slots
constexpr int KU = DQ / 64, VU = 2;             // slots of a key and a value tile
constexpr int UNITS = KU + VU;
constexpr int Q_TILE = KU * SLOT;
constexpr int OFF_Q = 0;
constexpr int OFF_RING = OFF_Q + NQ * Q_TILE;
constexpr int OFF_BAR = OFF_RING + NS * SLOT;
// q_full[2], q_empty[2], full[NS], empty[NS], s_full[2], p_full[2], o_final[2],
// drain, info_full[2], info_empty[2], v_landed, v_fixed
constexpr int NBAR = 4 + 2 * NS + 6 + 1 + 4 + 2;
constexpr int OFF_MISC = OFF_BAR + NBAR * 8;
constexpr int OFF_INFO = OFF_MISC + 16;         // two item records: claimed item, tiles of Q0 and of Q1
constexpr int REC = 4;
constexpr int OFF_SPLIT = OFF_INFO + 2 * REC * 4;
constexpr int SMEM_BYTES = OFF_SPLIT + 32 + 1024;
constexpr uint32_t COL_S0 = 0, COL_S1 = 128, COL_O0 = 256, COL_O1 = 256 + DV, TMEM_COLS = 512;
static_assert(SMEM_BYTES <= 227 * 1024, "shared memory budget");

// Items [n0, n_items), a last round of CTAs that is not full, are cut into up to P parts of
// `len` key tiles at most (the plan kernel's choice, in the header of its list).
struct Split {
    int n_entries, n_items, n0;
    int P, len;                          // P = 1: none is cut
    __device__ __forceinline__ int claims() const { return n0 + (n_items - n0) * P; }
};

struct Item {
    int h, q0, qs, sq, ks, skv;     // head; first query of the item; first query / key row of the request and its counts
    TileInfo t0, t1;
    int lo, c0, c1;                 // this part's first key tile, and its tiles for either query tile
    int parts;                      // > 1: results go to part slot `slot`; 0: nothing to do
    int slot;
};

// Part `part` of item w, cut into equal parts of `len` key tiles at most (0: the whole of it).
__device__ __forceinline__ Item describe_item(const PrefillArgs& a, int n_entries, int w, int part, int len, int slot) {
    Item it;
    // the plan's entries within a group of heads: the heads of an entry, then the next entry
    const int hg = a.head_group, grp = w / (n_entries * hg), x = w - grp * n_entries * hg;
    const int heads = min(hg, a.Hq - grp * hg);
    const int4* e = reinterpret_cast<const int4*>(a.entries + (size_t)(x / heads) * 8);
    const int4 e0 = e[0], e1 = e[1];
    it.h = grp * hg + x % heads;
    it.q0 = e0.y;
    it.qs = e0.z;
    it.sq = e0.w;
    it.ks = e1.x;
    it.skv = e1.y;
    it.t0 = tile_info_n(it.q0, BM, it.sq, it.skv, a.causal, -1, -1);
    it.t1 = tile_info_n(it.q0 + BM, BM, it.sq, it.skv, a.causal, -1, -1);
    const int n = max(it.t0.n_tiles, it.t1.n_tiles);
    int parts = 1, each = max(1, n);
    if (len > 0) {
        parts = max(1, (n + len - 1) / len);
        each = max(1, (n + parts - 1) / parts);       // (parts of `each` are as many again)
    }
    it.lo = part * each;
    it.c0 = max(0, min(it.t0.n_tiles - it.lo, each));
    it.c1 = max(0, min(it.t1.n_tiles - it.lo, each));
    it.parts = part < parts ? parts : 0;
    it.slot = slot;
    return it;
}
__device__ __forceinline__ Item describe_claim(const PrefillArgs& a, const Split& s, int w) {
    // (one copy of describe_item a role: two made short calls 1 us and a long one 6 us of 740 slower)
    const int x = w - s.n0, P = s.P;
    int item = w, part = 0, len = 0;
    if (x >= 0) {
        item = s.n0 + x / P;
        part = x - (item - s.n0) * P;
        len = s.len;
    }
    return describe_item(a, s.n_entries, item, part, len, x);
}
__device__ __forceinline__ Split find_split(const PrefillArgs& a) {
    Split s;
    s.n_entries = *a.n_entries;
    s.n_items = s.n_entries * a.Hq;
    s.len = a.part_o ? a.n_entries[2] : 0;
    s.P = a.part_o ? a.n_entries[3] : 1;
    s.n0 = s.P > 1 ? s.n_items - s.n_items % a.grid : s.n_items;
    return s;
}

template <bool F16>
__global__ void __launch_bounds__(NUM_THREADS, 1)
latent_varlen_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                     const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_pe,
                     const PrefillArgs a) {
    constexpr uint32_t IDESC_QK = make_idesc_16<F16>(BM, BN, false, false);
    constexpr uint32_t IDESC_PV = make_idesc_16<F16>(BM, DV, false, true);
    griddep_launch_dependents();                 // the joining kernel may be scheduled (it waits for this grid)
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw_base = smem_u32(smem_raw);
    uint8_t* smem = smem_raw + ((1024 - (raw_base & 1023)) & 1023);
    const uint32_t sb = smem_u32(smem);
    // through a shuffle, so that the compiler knows the roles' branches to be uniform
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x / 32, 0), lane = threadIdx.x % 32;

    const uint32_t bar0 = sb + OFF_BAR;
    auto q_full = [&](int k) { return bar0 + 8u * k; };
    auto q_empty = [&](int k) { return bar0 + 8u * (2 + k); };
    auto full = [&](int i) { return bar0 + 8u * (4 + i); };
    auto empty = [&](int i) { return bar0 + 8u * (4 + NS + i); };
    auto s_full = [&](int k) { return bar0 + 8u * (4 + 2 * NS + k); };
    auto p_full = [&](int k) { return bar0 + 8u * (6 + 2 * NS + k); };
    auto o_final = [&](int k) { return bar0 + 8u * (8 + 2 * NS + k); };
    const uint32_t drain = bar0 + 8u * (10 + 2 * NS);
    auto info_full = [&](int i) { return bar0 + 8u * (11 + 2 * NS + i); };
    auto info_empty = [&](int i) { return bar0 + 8u * (13 + 2 * NS + i); };
    const uint32_t v_landed = bar0 + 8u * (15 + 2 * NS), v_fixed = bar0 + 8u * (16 + 2 * NS);
    int* info = reinterpret_cast<int*>(smem + OFF_INFO);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + OFF_MISC);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + OFF_MISC + 4);
    // Unit u of the loads (KU key slots, then VU value slots, per tile) is use u / NS of slot u % NS.
    auto slot_addr = [&](uint32_t u) { return sb + OFF_RING + u % NS * SLOT; };
    auto parity_of = [&](uint32_t u) { return u / NS & 1; };

    if (threadIdx.x == 0) {
        for (int k = 0; k < NQ; ++k) {
            mbar_init(q_full(k), 1);
            mbar_init(q_empty(k), 1);
            mbar_init(s_full(k), 1);
            mbar_init(p_full(k), BM);
            mbar_init(o_final(k), 1);
            mbar_init(info_full(k), 1);
            mbar_init(info_empty(k), 1 + 8 + 2);   // the MMA thread, the softmax warps, warps 10-11
        }
        for (int i = 0; i < NS; ++i) { mbar_init(full(i), 1); mbar_init(empty(i), 1); }
        mbar_init(drain, 1);
        mbar_init(v_landed, 1);
        mbar_init(v_fixed, 2);
        *abort_flag = 0;
        fence_mbar_init();
    }
    Split& sp = *reinterpret_cast<Split*>(smem + OFF_SPLIT);     // (in shared memory: a softmax thread has no registers to spare)
    if (threadIdx.x == 32 * WARP_LOAD) sp = find_split(a);
    if (warp == WARP_MMA) {
        tmem_alloc(smem_u32(tmem_slot), TMEM_COLS);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;

    // As in prefill.cu each role ends by itself; the MMA warp frees TMEM once the
    // softmax warps have arrived on barrier 2.
    if (warp >= 8) {
        regs_dec<kRegsOther>();
        if (warp == WARP_LOAD) {
            // ------------------------------------------------------------ producer (one elected lane)
            uint32_t nu = 0;                       // units loaded (modulo 2^32, a multiple of NS)
            int nq[2] = {0, 0};
            if (elect_one()) {
                tma_prefetch_desc(&tm_q);
                tma_prefetch_desc(&tm_k);
                tma_prefetch_desc(&tm_v);
                tma_prefetch_desc(&tm_pe);
                bool ok = true;
                for (int r = 0; ok; ++r) {
                    const int w = atomicAdd(a.work, 1);
                    const bool none = w >= sp.claims();
                    int c[2] = {0, 0};
                    Item it;
                    if (!none) {
                        it = describe_claim(a, sp, w);
                        c[0] = it.c0;
                        c[1] = it.c1;
                    }
                    ok = mbar_wait(info_empty(r & 1), ((r >> 1) & 1) ^ 1, abort_flag);
                    if (!ok) break;
                    int* rec = info + REC * (r & 1);
                    rec[0] = none ? -1 : w;
                    rec[1] = c[0];
                    rec[2] = c[1];
                    mbar_arrive(info_full(r & 1));
                    if (none) break;
                    auto load_q = [&](int k) {
                        if (!mbar_wait(q_empty(k), (nq[k] & 1) ^ 1, abort_flag)) return false;
                        mbar_arrive_expect_tx(q_full(k), Q_TILE);
#pragma unroll
                        for (int s = 0; s < KU; ++s)
                            tma_load_3d(sb + OFF_Q + k * Q_TILE + s * SLOT, &tm_q, q_full(k), s * 64, it.h,
                                        it.qs + it.q0 + k * BM);
                        ++nq[k];
                        return true;
                    };
                    if (c[0] > 0) ok = load_q(0);
                    const int n = max(c[0], c[1]);
                    for (int j = 0; j < n && ok; ++j) {
                        const int key = it.ks + (it.lo + j) * BN;
                        for (int x = 0; x < UNITS && ok; ++x, ++nu) {
                            const uint32_t f = full(nu % NS);
                            ok = mbar_wait(empty(nu % NS), parity_of(nu) ^ 1u, abort_flag);
                            if (!ok) break;
                            const uint32_t dst = slot_addr(nu);
                            mbar_arrive_expect_tx(f, SLOT);
                            if (x < KU - 1) {
                                tma_load_3d(dst, &tm_k, f, x * 64, it.h, key);
                            } else if (x == KU - 1) {
                                tma_load_3d(dst, &tm_pe, f, 0, 0, key);
                            } else {
                                const int k0 = key + (x - KU) * 64;
                                tma_load_3d(dst, &tm_v, f, 0, it.h, k0);
                                tma_load_3d(dst + SLOT / 2, &tm_v, f, 64, it.h, k0);
                            }
                            // Q1 behind the first key tile, so that S0 starts early
                            if (j == 0 && x == KU - 1 && c[1] > 0) ok = load_q(1);
                        }
                    }
                }
                if (*abort_flag) {
                    // let the copies in flight land: the last load of each slot
                    for (uint32_t u = nu < NS ? 0 : nu - NS; u != nu; ++u) mbar_drain(full(u % NS), parity_of(u));
                    for (int k = 0; k < 2; ++k)
                        if (nq[k] > 0) mbar_drain(q_full(k), (nq[k] - 1) & 1);
                }
            }
            __syncwarp();
        } else if (warp == WARP_MMA) {
            // ------------------------------------------------------------ MMA issuer (one elected lane)
            if (elect_one()) {
                uint32_t u0 = 0;                   // first unit of the item
                int nq[2] = {0, 0}, np[2] = {0, 0}, nfix = 0;
                bool ok = true;
                for (int r = 0; ok; ++r) {
                    ok = mbar_wait(info_full(r & 1), (r >> 1) & 1, abort_flag);
                    if (!ok) break;
                    const int* rec = info + REC * (r & 1);
                    const int w = rec[0], c0 = rec[1], c1 = rec[2];
                    mbar_arrive(info_empty(r & 1));
                    if (w < 0) break;
                    const int n = max(c0, c1);
                    // (no tcgen05 fence: the slots come by TMA, and the fence would wait for
                    // the MMAs under way)
                    auto unit_ready = [&](uint32_t u) { return mbar_wait(full(u % NS), parity_of(u), abort_flag); };
                    // S_k of tile i; `last`: no other query tile needs these keys
                    auto issue_s = [&](int k, int i, bool last) {
                        const uint32_t d = tmem + (k == 0 ? COL_S0 : COL_S1);
                        const uint32_t qb = sb + OFF_Q + k * Q_TILE;
#pragma unroll
                        for (int x = 0; x < KU; ++x) {
                            const uint32_t u = u0 + i * UNITS + x;
                            if (!unit_ready(u)) return false;
                            const uint64_t qd = make_sdesc_sw128(qb + x * SLOT, 16, 1024);
                            const uint64_t kd = make_sdesc_sw128(slot_addr(u), 16, 1024);
#pragma unroll
                            for (int kk = 0; kk < 4; ++kk)
                                mma_bf16_ss(d, desc_at(qd, 32 * kk), desc_at(kd, 32 * kk), IDESC_QK,
                                            (x > 0 || kk > 0) ? 1u : 0u);
                            if (last) mma_commit(empty(u % NS));
                        }
                        mma_commit(s_full(k));
                        return true;
                    };
                    auto issue_pv = [&](int k, int i, bool last) {
                        if (!mbar_wait(p_full(k), np[k]++ & 1, abort_flag)) return false;
                        tc_fence_after();
                        const uint32_t d = tmem + (k == 0 ? COL_O0 : COL_O1), p = tmem + (k == 0 ? COL_S0 : COL_S1);
#pragma unroll
                        for (int x = 0; x < VU; ++x) {
                            const uint32_t u = u0 + i * UNITS + KU + x;
                            // dims-major B: 64-dim halves 8 KB apart, 8-key groups 1 KB apart
                            const uint64_t vd = make_sdesc_sw128(slot_addr(u), SLOT / 2, 1024);
#pragma unroll
                            for (int kk = 0; kk < 4; ++kk)
                                mma_bf16_ts(d, p + (4 * x + kk) * 8, desc_at(vd, kk * 2048), IDESC_PV,
                                            (i > 0 || x > 0 || kk > 0) ? 1u : 0u);
                            if (last) mma_commit(empty(u % NS));
                        }
                        return true;
                    };
                    auto values_ready = [&](int i) {
                        for (int x = 0; x < VU; ++x)
                            if (!unit_ready(u0 + i * UNITS + KU + x)) return false;
                        if (i == n - 1) {
                            // the item's last tile: rows past the request's end are zeroed first
                            mbar_arrive(v_landed);
                            if (!mbar_wait(v_fixed, nfix++ & 1, abort_flag)) return false;
                            tc_fence_after();
                        }
                        return true;
                    };
                    if (c0 > 0) {
                        ok = mbar_wait(q_full(0), nq[0]++ & 1, abort_flag) && issue_s(0, 0, c1 == 0);
                        if (ok && c0 == 1) mma_commit(q_empty(0));
                    }
                    if (ok && c1 > 0) {
                        ok = mbar_wait(q_full(1), nq[1]++ & 1, abort_flag) && issue_s(1, 0, true);
                        if (ok && c1 == 1) mma_commit(q_empty(1));
                    }
                    for (int i = 0; i < n && ok; ++i) {
                        ok = values_ready(i);
                        if (ok && i < c0) {
                            ok = issue_pv(0, i, i >= c1);
                            if (ok && i + 1 == c0) mma_commit(o_final(0));
                            if (ok && i + 1 < c0) {
                                ok = issue_s(0, i + 1, i + 1 >= c1);
                                if (ok && i + 2 == c0) mma_commit(q_empty(0));
                            }
                        }
                        if (ok && i < c1) {
                            ok = issue_pv(1, i, true);
                            if (ok && i + 1 == c1) mma_commit(o_final(1));
                            if (ok && i + 1 < c1) {
                                ok = issue_s(1, i + 1, true);
                                if (ok && i + 2 == c1) mma_commit(q_empty(1));
                            }
                        }
                    }
                    u0 += n * UNITS;
                }
                mma_commit(drain);                // every MMA issued above has completed once this arrives
                mbar_drain(drain, 0);
            }
            __syncwarp();
            named_bar_sync(2, 8 * 32 + 32);       // softmax warps are done with TMEM
            tc_fence_after();
            tmem_dealloc(tmem, TMEM_COLS);
        } else {
            // ------------------------------------------------------------ warps 10-11
            // Value rows past the request's end hold the next request's rows, where
            // 0 * NaN would not vanish: zero them before the last tile's P V.
            const int t = (warp - 10) * 32 + lane;
            uint32_t u0 = 0;
            int nl = 0;
            for (int r = 0;; ++r) {
                const bool got = __all_sync(0xffffffffu, mbar_wait(info_full(r & 1), (r >> 1) & 1, abort_flag));
                const int* rec = info + REC * (r & 1);
                const int w = got ? rec[0] : -1, n = got ? max(rec[1], rec[2]) : 0;
                __syncwarp();
                if (lane == 0) mbar_arrive(info_empty(r & 1));
                if (w < 0) break;
                if (n == 0) continue;
                const Item it = describe_claim(a, sp, w);
                const uint32_t uv = u0 + (n - 1) * UNITS + KU;
                u0 += n * UNITS;
                if (!__all_sync(0xffffffffu, mbar_wait(v_landed, nl & 1, abort_flag))) break;
                ++nl;
                for (int x = 0; x < VU; ++x) {
                    // the MMA thread has seen the slot full; so does the writer here
                    if (!__all_sync(0xffffffffu, mbar_wait(full((uv + x) % NS), parity_of(uv + x), abort_flag)))
                        break;
                    const int r0 = it.skv - (it.lo + n - 1) * BN - x * 64;   // first row of the half past the end
                    uint8_t* base = smem + (slot_addr(uv + x) - sb);
                    for (int y = max(r0, 0) * 16 + t; y < 64 * 16; y += 64) {
                        const int row = y / 16, sl = (y / 8) % 2, q = y % 8;
                        *reinterpret_cast<uint4*>(base + sl * (SLOT / 2) + row * 128 + q * 16) = make_uint4(0u, 0u, 0u, 0u);
                    }
                }
                fence_proxy_async_smem();           // generic writes, read by the tensor core
                __syncwarp();
                if (lane == 0) mbar_arrive(v_fixed);
            }
        }
    } else {
        regs_inc<kRegsSoftmax>();
        // ------------------------------------------------------------ softmax warps 0-7
        const int k = warp / 4;
        const int r = (warp % 4) * 32 + lane;                  // row of the tile == TMEM lane
        const uint32_t lane_addr = (uint32_t)((warp % 4) * 32) << 16;
        const uint32_t col_s = k == 0 ? COL_S0 : COL_S1, col_o = k == 0 ? COL_O0 : COL_O1;
        const float sl = a.scale_log2;
        // As in latent_paged.cu: a float16 P keeps 2^-31 of the strongest weight.
        constexpr float kLead = F16 ? 6.f : 0.f;
        int sf = 0;                  // S tiles taken so far (s_full parity)
        int n_done = 0;              // items with a tile finished (o_final parity)
        bool ok = true;
        // Item rr into `itm`; the claim, -1 for none.
        auto take = [&](int rr, Item& itm) {
            ok = __all_sync(0xffffffffu, mbar_wait(info_full(rr & 1), (rr >> 1) & 1, abort_flag));
            const int w = ok ? info[REC * (rr & 1)] : -1;
            __syncwarp();
            if (lane == 0) mbar_arrive(info_empty(rr & 1));
            __syncwarp();
            if (w >= 0) itm = describe_claim(a, sp, w);
            return w;
        };
        Item itm, next{};
        int w = take(0, itm);
        for (int rr = 0; named_bar_and(3 + k, BM, ok) && w >= 0; ++rr, itm = next) {   // (the warpgroup stops together)
            const TileInfo ti = k == 0 ? itm.t0 : itm.t1;
            const int n_tiles = k == 0 ? itm.c0 : itm.c1;
            const int lim = (int)key_hi((long)ti.q0 + r + itm.skv - itm.sq, itm.skv, a.causal, -1);   // keys this row sees
            float m_ref = -INFINITY;     // reference max (log2 units, scaled)
            float l_run = 0.f;
            for (int j = 0; j < n_tiles; ++j) {
                const int kbase = (itm.lo + j) * BN;
                ok = __all_sync(0xffffffffu, mbar_wait(s_full(k), sf & 1, abort_flag));
                ++sf;
                if (!ok) break;
                tc_fence_after();
                uint32_t sr[BN];
                tmem_ld128(tmem + lane_addr + col_s, sr);
                float* s = reinterpret_cast<float*>(sr);
                // raw scores where the whole tile is visible and the scale positive
                // (the scale goes into the exponent's FMA), logits with -inf for
                // hidden keys otherwise
                const bool fast = kbase + BN <= ti.lim_first && sl > 0.f;
                auto to_logits = [&]() {
                    if (fast) return;
#pragma unroll
                    for (int c = 0; c < BN; ++c) s[c] = kbase + c < lim ? s[c] * sl : -INFINITY;
                };
                to_logits();
                const float fa = fast ? sl : 1.f;
                float alpha = 1.f, rs = 0.f;
                // as in prefill.cu: against the standing reference while the row
                // sums stay below the limit, else with the tile's row maximum
                bool done = false;
                if (__all_sync(0xffffffffu, m_ref != -INFINITY)) {
                    uint32_t pk[BN / 2];
                    rs = exp_row<F16>(s, fa, m_ref, pk);
                    if (!__any_sync(0xffffffffu, !(rs <= sum_limit<F16>()))) {
                        tmem_st64(tmem + lane_addr + col_s, pk);
                        done = true;
                    }
                }
                if (!done) {
                    tmem_ld128(tmem + lane_addr + col_s, sr);
                    to_logits();
                    float mx8[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) mx8[e] = -INFINITY;
#pragma unroll
                    for (int c = 0; c < BN; c += 2) mx8[(c >> 1) & 7] = fmax3(mx8[(c >> 1) & 7], s[c], s[c + 1]);
#pragma unroll
                    for (int e = 0; e < 4; ++e) mx8[e] = fmaxf(mx8[e], mx8[e + 4]);
                    const float mx_raw = fmaxf(fmaxf(mx8[0], mx8[1]), fmaxf(mx8[2], mx8[3]));
                    const float mx = fast ? mx_raw * sl : mx_raw;
                    if (mx > m_ref + kRescaleThreshold) {
                        alpha = fast_exp2(m_ref - (mx - kLead));
                        m_ref = mx - kLead;
                    }
                    const float m_use = m_ref == -INFINITY ? 0.f : m_ref;
                    uint32_t pk[BN / 2];
                    rs = exp_row<F16>(s, fa, m_use, pk);
                    tmem_st64(tmem + lane_addr + col_s, pk);
                }
                l_run = l_run * alpha + rs;
                // P V of the tile before is complete (this S landed after it)
                if (j > 0 && __any_sync(0xffffffffu, alpha != 1.f)) {
#pragma unroll 1
                    for (int c = 0; c < DV; c += 32) {
                        float o[32];
                        tmem_ld32(tmem + lane_addr + col_o + c, o);
#pragma unroll
                        for (int e = 0; e < 32; ++e) o[e] *= alpha;
                        tmem_st32(tmem + lane_addr + col_o + c, reinterpret_cast<uint32_t*>(o));
                    }
                }
                tc_fence_before();
                mbar_arrive(p_full(k));
            }
            // ---- the tile's end (also after a wait gave up: all four warps pass the barrier above)
            // the next item first, whose record comes while the last P V runs
            if (ok) w = take(rr + 1, next);
            // An item without a tile for this warpgroup has no phase of o_final: the
            // MMA thread could end it before the phase of the item before has been seen.
            if (ok && n_tiles > 0) {
                ok = __all_sync(0xffffffffu, mbar_wait(o_final(k), n_done & 1, abort_flag));
                ++n_done;
                if (ok) tc_fence_after();
            }
            const bool row_ok = r < ti.rows_valid;
            const size_t orow = (size_t)(itm.qs + ti.q0 + r) * a.Hq + itm.h;
            const bool some = l_run != 0.f && n_tiles > 0;       // 0: no key; NaN goes on
            const float inv = some ? 1.f / l_run : 0.f;
            if (row_ok && a.lse && ok && itm.parts == 1) a.lse[orow] = some ? (m_ref + log2f(l_run)) * kLn2 : -INFINITY;
            uint16_t* dst = static_cast<uint16_t*>(a.o) + orow * DV;
            if (ti.rows_valid > 0 && ok && itm.parts > 1) {
                // a part: O as it is, four dims a step, with the row's maximum and sum
                const size_t at = (size_t)itm.slot * 2 + k;
                reinterpret_cast<float2*>(a.part_lse)[at * BM + r] = some ? make_float2(m_ref, l_run) : make_float2(-INFINITY, 0.f);
                if (n_tiles > 0) {
                    float4* part = reinterpret_cast<float4*>(a.part_o) + at * (DV / 4) * BM + r;
#pragma unroll 1
                    for (int c = 0; c < DV; c += 32) {
                        float o[32];
                        __syncwarp();
                        tmem_ld32(tmem + lane_addr + col_o + c, o);
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            part[(c / 4 + e) * BM] = make_float4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
                    }
                }
            } else if (ti.rows_valid > 0 && ok && itm.parts == 1) {
#pragma unroll 1
                for (int c = 0; c < DV; c += 32) {
                    float o[32];
                    __syncwarp();
                    if (n_tiles > 0) {
                        tmem_ld32(tmem + lane_addr + col_o + c, o);
                    } else {
#pragma unroll
                        for (int e = 0; e < 32; ++e) o[e] = 0.f;
                    }
                    if (row_ok) {
                        uint32_t wd[16];
#pragma unroll
                        for (int e = 0; e < 16; ++e)
                            wd[e] = pack2<F16>(some ? o[2 * e] * inv : 0.f, some ? o[2 * e + 1] * inv : 0.f);
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            *reinterpret_cast<uint4*>(dst + c + 8 * e) =
                                make_uint4(wd[4 * e], wd[4 * e + 1], wd[4 * e + 2], wd[4 * e + 3]);
                    }
                }
            }
            tc_fence_before();
        }
        __syncwarp();
        named_bar_arrive(2, 8 * 32 + 32);
        if (threadIdx.x == 0 && *abort_flag) atomicExch(&g_latent_varlen_error, (int)kErrPrefillWait);
    }
}

// Adds up the parts of cut items: o = sum_p w_p O_p / sum_p w_p l_p with w_p = 2^(m_p -
// M).  Block (cut item, query tile; 32 of the dims), thread = row: each load covers four
// dims of 32 rows, 512 bytes in a row.
template <bool F16>
__global__ void __launch_bounds__(BM) latent_varlen_join_kernel(const PrefillArgs a) {
    griddep_wait();
    const Split sp = find_split(a);
    const int x = blockIdx.x / 2, k = blockIdx.x % 2, r = threadIdx.x;
    if (x >= sp.n_items - sp.n0) return;
    const Item it = describe_item(a, sp.n_entries, sp.n0 + x, 0, sp.len, x * sp.P);
    const TileInfo ti = k == 0 ? it.t0 : it.t1;
    if (it.parts <= 1 || r >= ti.rows_valid) return;
    const float2* ml = reinterpret_cast<const float2*>(a.part_lse) + ((size_t)it.slot * 2 + k) * BM + r;
    const float4* src = reinterpret_cast<const float4*>(a.part_o) + (((size_t)it.slot * 2 + k) * (DV / 4) + blockIdx.y * 8) * BM + r;
    float M = -INFINITY, L = 0.f;
    for (int p = 0; p < it.parts; ++p) M = fmaxf(M, ml[(size_t)p * 2 * BM].x);
    float4 acc[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) acc[e] = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int p = 0; p < it.parts; ++p) {
        const float2 s = ml[(size_t)p * 2 * BM];
        const float w = s.y == 0.f ? 0.f : fast_exp2(s.x - M);
        L += w * s.y;
        if (w == 0.f) continue;                    // a part without a key has not written its O
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float4 o = src[((size_t)p * 2 * (DV / 4) + e) * BM];
            acc[e].x = fmaf(w, o.x, acc[e].x);
            acc[e].y = fmaf(w, o.y, acc[e].y);
            acc[e].z = fmaf(w, o.z, acc[e].z);
            acc[e].w = fmaf(w, o.w, acc[e].w);
        }
    }
    const float inv = L != 0.f ? 1.f / L : 0.f;
    const size_t orow = (size_t)(it.qs + ti.q0 + r) * a.Hq + it.h;
    uint4* dst = reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.o) + orow * DV + blockIdx.y * 32);
#pragma unroll
    for (int e = 0; e < 4; ++e)
        dst[e] = make_uint4(pack2<F16>(acc[2 * e].x * inv, acc[2 * e].y * inv), pack2<F16>(acc[2 * e].z * inv, acc[2 * e].w * inv),
                            pack2<F16>(acc[2 * e + 1].x * inv, acc[2 * e + 1].y * inv),
                            pack2<F16>(acc[2 * e + 1].z * inv, acc[2 * e + 1].w * inv));
    if (blockIdx.y == 0 && a.lse) a.lse[orow] = L != 0.f ? (M + log2f(L)) * kLn2 : -INFINITY;
}

template <bool F16>
cudaError_t launch_t(const CUtensorMap& tm_q, const CUtensorMap& tm_k, const CUtensorMap& tm_v, const CUtensorMap& tm_pe,
                     const PrefillArgs& a, cudaStream_t stream) {
    static SmemLimit limit;
    cudaError_t e = limit.set(reinterpret_cast<const void*>(latent_varlen_kernel<F16>), SMEM_BYTES);
    if (e != cudaSuccess) return e;
    latent_varlen_kernel<F16><<<(unsigned)a.grid, NUM_THREADS, SMEM_BYTES, stream>>>(tm_q, tm_k, tm_v, tm_pe, a);
    e = cudaGetLastError();
    if (e != cudaSuccess || a.part_o == nullptr) return e;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(2 * a.grid, DV / 32);
    cfg.blockDim = dim3(BM);
    cfg.stream = stream;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, latent_varlen_join_kernel<F16>, a);
}

}  // namespace

cudaError_t launch_latent_varlen(const CUtensorMap& tm_q, const CUtensorMap& tm_k, const CUtensorMap& tm_v,
                                 const CUtensorMap& tm_pe, const PrefillArgs& a, cudaStream_t stream) {
    return a.f16 ? launch_t<true>(tm_q, tm_k, tm_v, tm_pe, a, stream) : launch_t<false>(tm_q, tm_k, tm_v, tm_pe, a, stream);
}

int latent_varlen_take_device_error() {
    int v = 0;
    if (cudaMemcpyFromSymbol(&v, g_latent_varlen_error, sizeof(int)) != cudaSuccess) return -1;
    if (v != 0) {
        const int zero = 0;
        cudaMemcpyToSymbol(g_latent_varlen_error, &zero, sizeof(int));
    }
    return v;
}

}  // namespace gqa
