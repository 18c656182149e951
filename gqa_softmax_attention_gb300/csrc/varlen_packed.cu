// Packed variable-length calls (TileOPs "Attention Operators",
// GQAVarlenFwdOp): q [total_q, Hq, D], k / v [total_kv, Hkv, D], request b
// owning query rows [cu_seqlens_q[b], cu_seqlens_q[b + 1]) and key rows
// [cu_seqlens_kv[b], cu_seqlens_kv[b + 1]).  Also the plan kernel shared with
// the paged calls: it lists the (request, row block) entries on the device,
// so the host never reads the offsets back.
#include "onetile.cuh"

namespace gqa {
namespace {

// One CTA of 1024 threads.  Request b gets ceil(Sq_b / qpb) entries
// {b, q0, qs, Sq_b, ks, L_b}.  Offsets are clamped into [0, total] and
// lengths into [0, kv_cap], so malformed metadata can give wrong results but
// no access out of range; entries past max_entries are dropped.  The
// requests are then ordered by estimated cost, heaviest first (a counting
// sort over NBUCKET cost buckets, requests of one bucket in their own order),
// each request's blocks together and its heaviest (last) block first.
constexpr int NBUCKET = 2048;
// SM time of one cached key of a decode step against one plan cost unit (see
// the end of varlen_plan_kernel), as the two kernels run side by side: the
// split decode kernel streams about 70 GB/s per SM on a share of the SMs, the
// one-tile kernel about 7.2 TFLOP/s per SM, so (4 bytes / 70 GB/s) / (2^15
// FLOP / 7.2 TFLOP/s) = 0.0126.  Set a little below: the chunks' persistent
// grid cannot grow into SMs the decode steps leave, while the decode CTAs do
// fill the SMs the chunks leave (measured on the mixed serving batch: 0.622,
// 0.606 and 0.683 ms at 0.009, 0.0126 and 0.016).
constexpr double kDecPerKey = 0.011;
// Over e4m3 caches a cached key is half the bytes and the split kernel is bound by
// its instructions.  60 steps and 4 chunks (1 chunk), mean of three draws of lengths:
//   0.002  0.0035  0.005  0.007  0.009  0.012
//    574     573    576    574    608    660   us at 32/8 heads, D = 128
//   (292)   (285)  (288)  (304)  (345)  (386)
//    747     746    752    749    749    762   at 24/2, D = 256, pages of 64
//   (332)   (333)  (333)  (332)  (330)  (359)
// so one constant does for both.
constexpr double kDecPerKey8 = 0.005;

__device__ __forceinline__ int entry_cost(const int4 e0, const int4 e1, int qpb, int g, int causal) {
    const int q0 = e0.y, sq = e0.w, L = e1.y;
    const int nq = min(qpb, sq - q0);
    const int last = q0 + nq - 1;                         // last query of the block
    const int keys = causal ? max(0, min(L, last + L - sq + 1)) : L;
    const int tiles = (keys + 127) / 128;
    // a block with few rows streams its keys at memory speed: weigh its tiles more
    return min(NBUCKET - 1, tiles * (nq * g >= 64 ? 2 : 3));
}

// Which items of an expanded latent call are cut along the keys.  With n_items = q grid
// + tail, the last `tail` items would keep all but that many CTAs waiting for a whole
// item's time; they are cut into up to P parts each instead, of at least kPartTiles key
// tiles, shorter ones into fewer or none.  They are no alike, and the longest may be the
// last of all: a few queries over a long context weigh less than a prompt as a whole and
// come after its lightest blocks.  So the length goes by the longest of the tail.  Parts
// taken one after the other by all CTAs end by (W - l) / grid + l, W the tile times
// of all of them (2 more a part for its start and end) and l those of the longest
// part; P takes the least of that, if it saves more than the joining costs
// (kJoinTiles).  From kMaxRounds rounds on the tail is short against the rest (a CTA's
// share of it is under an eighth).  (By the tail's first item alone, before: a 4096-token
// prompt beside one query over 8192 keys, 12 heads, 122 us uncut, 87 in five parts; 20 heads
// 169 and 132; three prompts of 3000 beside 16 queries over 12000 keys, 8 heads, 177 and 125.
// A call of which nothing is cut pays 1 us for the choice.)
constexpr int kJoinTiles = 4, kMaxRounds = 8;

__global__ void __launch_bounds__(1024) varlen_plan_kernel(const int32_t* cu_q, const int32_t* kv, int paged,
                                                          int B, int qpb, int g, int causal, int total_q,
                                                          long kv_cap, int32_t* tmp, int32_t* entries,
                                                          int32_t* n_entries, int max_entries, int grid,
                                                          double dec_per_key, int split_grid, int Hkv, int wl, int wr,
                                                          const TailSplit ts) {
    __shared__ int warp_sum[32];
    __shared__ unsigned long long pre_cost, dec_keys;   // listed blocks' cost; decode steps' cached keys
    __shared__ unsigned base;                           // blocks of earlier requests (step 1)
    __shared__ int most_tiles;                          // most key tiles that a block visits
    __shared__ int bucket[NBUCKET];
    __shared__ int chain[NBUCKET], group_next[1024], group_sum[1024];   // step 3
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    // pairs (flag bit 2): an entry covers two consecutive row blocks
    const bool pairs = (paged & 4) != 0;
    const int span = pairs ? 2 * qpb : qpb;            // queries per entry
    auto cost_of = [&](int b, int q0, int qs, int sq, int ks, int L) {
        int c = entry_cost(make_int4(b, q0, qs, sq), make_int4(ks, L, 0, 0), qpb, g, causal);
        if (pairs && q0 + qpb < sq) c += entry_cost(make_int4(b, q0 + qpb, qs, sq), make_int4(ks, L, 0, 0), qpb, g, causal);
        return c;
    };
    if (threadIdx.x == 0) {
        base = 0;
        most_tiles = 0;
        pre_cost = 0;
        dec_keys = 0;
    }
    for (int i = threadIdx.x; i < NBUCKET; i += 1024) {
        bucket[i] = 0;
        chain[i] = -1;
    }
    __syncthreads();
    // 1. entries in request order
    for (int b0 = 0; b0 < B; b0 += 1024) {
        const int b = b0 + threadIdx.x;
        int qs = 0, sq = 0, ks = 0, L = 0, nrb = 0;
        if (b < B) {
            qs = min(max(cu_q[b], 0), total_q);
            sq = min(max(cu_q[b + 1], qs), total_q) - qs;
            if (paged & 1) {
                L = (int)min((long)max(kv[b], 0), kv_cap);
            } else {
                ks = (int)min((long)max(kv[b], 0), kv_cap);
                L = (int)min((long)max(kv[b + 1], ks), kv_cap) - ks;
            }
            nrb = (sq + span - 1) / span;
            if ((paged & 2) && sq == 1) nrb = 0;      // a decode step, run by the split decode kernel
        }
        // inclusive scan within the warp; sums stop at max_entries, where the list ends
        // (malformed offsets can list the same rows again and again)
        auto sum = [&](unsigned p, unsigned q) { return min(p + q, (unsigned)max_entries); };
        unsigned x = min(nrb, max_entries);
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const unsigned y = __shfl_up_sync(0xffffffffu, x, o);
            if (lane >= o) x = sum(x, y);
        }
        if (lane == 31) warp_sum[warp] = (int)x;
        __syncthreads();
        if (warp == 0) {
            unsigned s = (unsigned)warp_sum[lane];
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const unsigned y = __shfl_up_sync(0xffffffffu, s, o);
                if (lane >= o) s = sum(s, y);
            }
            warp_sum[lane] = (int)s;
        }
        __syncthreads();
        const unsigned before = __shfl_up_sync(0xffffffffu, x, 1);
        const unsigned first = sum(base, sum(warp > 0 ? (unsigned)warp_sum[warp - 1] : 0u, lane > 0 ? before : 0u));
        // the request's estimated cost: the sum of its blocks' costs
        // (2047 units for every 128 queries pass 31 bits at 134 million: it stops far past the last bucket)
        int total = 0;
        for (int k = 0; k < nrb; ++k) total = min(total + cost_of(b, k * span, qs, sq, ks, L), 1 << 30);
        if (total > 0) atomicAdd(&pre_cost, (unsigned long long)total);
        if (split_grid > 0) {
            int most = 0;
            for (int k = 0; k < nrb; ++k) {
                const pf::TileInfo t = pf::tile_info_n(k * span, span, sq, L, causal, wl, wr);
                most = max(most, t.n_tiles - t.kv_begin / pf::BN);
            }
            if (most > 0) atomicMax(&most_tiles, most);
        }
        if ((paged & 2) && sq == 1 && b < B && L > 0) atomicAdd(&dec_keys, (unsigned long long)L);
        const int key = min(NBUCKET - 1, total / 16);
        for (int k = 0; k < nrb; ++k) {
            const unsigned e = first + k;
            if (e >= (unsigned)max_entries) break;
            int4* dst = reinterpret_cast<int4*>(tmp + (size_t)e * ot::ENTRY_INTS);
            dst[0] = make_int4(b, k * span, qs, sq);
            dst[1] = make_int4(ks, L, key, 0);             // .w: the request's start once placed
        }
        __syncthreads();
        if (threadIdx.x == 1023) base = sum(first, min(nrb, max_entries));
        __syncthreads();
    }
    const int n = (int)base;
    // a thread's first entry stays in registers (fewer loads: most calls have no other)
    int4 f0 = make_int4(0, 1, 0, 0), f1 = f0;
    auto entry = [&](int e, int4& e0, int4& e1) {
        const int4* src = reinterpret_cast<const int4*>(tmp + (size_t)e * ot::ENTRY_INTS);
        e0 = e < 1024 ? f0 : src[0];
        e1 = e < 1024 ? f1 : src[1];
    };
    if (threadIdx.x < n) {
        const int4* src = reinterpret_cast<const int4*>(tmp + (size_t)threadIdx.x * ot::ENTRY_INTS);
        f0 = src[0];
        f1 = src[1];
    }
    // 2. requests ordered by estimated cost, heaviest first (a counting sort of
    // their total costs), each request's blocks kept together and placed from
    // its last block (the most keys under a causal mask) to its first: the
    // grid's snake order then works through one request's keys at a time,
    // which stay in L2 while its blocks need them.  A request's first entry
    // (q0 = 0) stands for the whole request.
    for (int e = threadIdx.x; e < n; e += 1024) {
        int4 e0, e1;
        entry(e, e0, e1);
        // blocks of the request that made the list (all of them unless the
        // cap cut it short), so that the placed entries fill [0, n)
        if (e0.y == 0) atomicAdd(&bucket[e1.z], min((e0.w + span - 1) / span, n - e));
    }
    __syncthreads();
    {
        // bucket starts in descending cost order: thread t owns buckets
        // NBUCKET-1-2t and NBUCKET-2-2t; an exclusive block scan over threads
        static_assert(NBUCKET == 2 * 1024, "two buckets per thread");
        const int c1 = NBUCKET - 1 - 2 * threadIdx.x, c2 = c1 - 1;
        const int n1 = bucket[c1], n2 = bucket[c2];
        int x = n1 + n2;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, x, o);
            if (lane >= o) x += y;
        }
        __syncthreads();                               // warp_sum is free again
        if (lane == 31) warp_sum[warp] = x;
        __syncthreads();
        if (warp == 0) {
            int t = warp_sum[lane];
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, t, o);
                if (lane >= o) t += y;
            }
            warp_sum[lane] = t;
        }
        __syncthreads();
        const int start = (warp > 0 ? warp_sum[warp - 1] : 0) + x - n1 - n2;
        bucket[c1] = start;
        bucket[c2] = start + n1;
    }
    __syncthreads();
    // 3. each request reserves its range, within a bucket in the order of the
    // requests; then every block takes its place.  (Ranges taken by atomics alone stood
    // in whatever order the warps came: which items a call cuts along the keys, and so
    // the last bits of their results, changed from run to run.)  1024 entries at a
    // time: a warp's requests of one bucket form a group, its first lane's; the groups
    // of a bucket are chained in any order, and each adds up those of lower threads.
    for (int e_first = 0; e_first < n; e_first += 1024) {
        const int e = e_first + threadIdx.x;
        int key = -1, cnt = 0;
        if (e < n) {
            int4 e0, e1;
            entry(e, e0, e1);
            if (e0.y == 0) {
                key = e1.z;
                cnt = min((e0.w + span - 1) / span, n - e);
            }
        }
        const unsigned same = __match_any_sync(0xffffffffu, key);
        const int leader = __ffs(same) - 1;
        int before, sum;                               // blocks of the group's lower lanes, of all
        if (__all_sync(0xffffffffu, cnt <= 1)) {
            before = __popc(same & ((1u << lane) - 1));
            sum = __popc(same);
        } else {
            before = sum = 0;
            for (unsigned rest = __ballot_sync(0xffffffffu, cnt > 0); rest != 0; rest &= rest - 1) {
                const int l = __ffs(rest) - 1, c = __shfl_sync(0xffffffffu, cnt, l);
                if ((same >> l) & 1) {
                    sum += c;
                    before += l < lane ? c : 0;
                }
            }
        }
        const bool leads = key >= 0 && lane == leader;
        if (leads) {
            group_sum[threadIdx.x] = sum;
            group_next[threadIdx.x] = atomicExch(&chain[key], (int)threadIdx.x);
        }
        __syncthreads();
        int start = 0;
        if (leads) {
            start = bucket[key];
            for (int t = chain[key]; t >= 0; t = group_next[t]) start += t < (int)threadIdx.x ? group_sum[t] : 0;
        }
        start = __shfl_sync(0xffffffffu, start, leader);
        if (key >= 0) tmp[(size_t)e * ot::ENTRY_INTS + 7] = start + before;
        __syncthreads();
        if (e_first + 1024 >= n) break;
        if (leads) {
            atomicAdd(&bucket[key], sum);
            chain[key] = -1;
        }
        __syncthreads();
    }
    for (int e = threadIdx.x; e < n; e += 1024) {
        int4 e0, e1;
        entry(e, e0, e1);
        const int k = e0.y / span;
        const int cnt = min((e0.w + span - 1) / span, n - (e - k));
        const int start = reinterpret_cast<const int4*>(tmp + (size_t)(e - k) * ot::ENTRY_INTS)[1].w;
        const int pos = start + cnt - 1 - k;
        if (pos < 0 || pos >= n) continue;
        int4* dst = reinterpret_cast<int4*>(entries + (size_t)pos * ot::ENTRY_INTS);
        dst[0] = e0;
        dst[1] = make_int4(e1.x, e1.y, 0, 0);
    }
    if (ts.grid > 0) {
        const int n_items = n * ts.H, tail = n_items % ts.grid;      // tail < grid <= 1024
        unsigned* best = reinterpret_cast<unsigned*>(&warp_sum[0]);  // a cost's bits, its P in the last five
        int* longest = &warp_sum[1];
        int* tiles = group_sum;                                      // of each item of the tail
        const bool may = tail > 0 && n_items / ts.grid < kMaxRounds;
        if (threadIdx.x == 0) {
            *best = ~31u | 1u;
            *longest = 0;
        }
        __syncthreads();                                             // (and every entry is in its place)
        if (may && threadIdx.x < tail) {
            const int w = n_items - tail + threadIdx.x, grp = w / (n * ts.head_group);
            const int heads = min(ts.head_group, ts.H - grp * ts.head_group);
            const int4* e = reinterpret_cast<const int4*>(entries + (size_t)((w - grp * n * ts.head_group) / heads) * ot::ENTRY_INTS);
            const int4 e0 = e[0], e1 = e[1];
            const int t = pf::tile_info_n(e0.y, span, e0.w, e1.y, causal, wl, wr).n_tiles;
            tiles[threadIdx.x] = t;
            atomicMax(longest, t);
        }
        __syncthreads();
        const int t_max = *longest;
        const int most = may ? min(min(kLatentMaxParts, kLatentPartSlots * ts.grid / tail), t_max / kPartTiles) : 0;
        if (most > 1 && warp < most) {
            const int p = warp + 1, len = p > 1 ? max(kPartTiles, (t_max + p - 1) / p) : t_max;
            float w = 0.f;
            for (int x = lane; x < tail; x += 32) w += (float)(tiles[x] + 2 * max(1, (tiles[x] + len - 1) / len));
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) w += __shfl_xor_sync(0xffffffffu, w, o);
            const float l = (float)(len + 2), cost = (w - l) / (float)ts.grid + l + (p > 1 ? (float)kJoinTiles : 0.f);
            if (lane == 0) atomicMin(best, (__float_as_uint(cost) & ~31u) + p);      // (positive floats order as their bits)
        }
        __syncthreads();
        if (threadIdx.x == 0) {
            const int p = (int)(*best & 31u);
            n_entries[2] = p > 1 ? max(kPartTiles, (t_max + p - 1) / p) : 0;
            n_entries[3] = p;
        }
    }
    if (threadIdx.x == 0) {
        n_entries[0] = n;
        n_entries[1] = 0;                              // the attention kernel's item counter
        // The listed blocks' share of `grid` persistent CTAs when decode steps
        // run beside them: their estimated SM time against the decode steps',
        // so that both end together.  A cost unit is half a 128-key tile of a
        // full 128-row block (128 x 128 x D x 2 FLOP per KV head); a cached key
        // of a decode step is 4 D bytes per KV head (16-bit K and V); D and
        // Hkv cancel, and dec_per_key converts the second into the first.
        int ge = grid;
        if (grid > 0 && pre_cost > 0 && dec_keys > 0) {
            const double tp = (double)pre_cost, td = (double)dec_keys * dec_per_key;
            ge = (int)lrint((double)grid * tp / (tp + td));
            ge = min(grid, max(ge, min(grid, 8)));
        }
        if (ts.grid == 0) n_entries[2] = ge;
        if (split_grid > 0) {
            // as many parts as leave every one a CTA, but no more than give the block
            // with the most visited tiles kPartTiles each (shorter blocks fill fewer
            // parts: onetile_kernel); none where cutting does not pay
            const int ctas = grid > 0 ? ge : split_grid;
            const long blocks = (long)n * Hkv;
            n_entries[3] = blocks > 0 && cut_pays(most_tiles, blocks)
                               ? (int)max(1L, min(ctas / blocks, (long)(most_tiles / kPartTiles)))
                               : 1;
        }
    }
}

}  // namespace

cudaError_t launch_varlen_plan(const int32_t* cu_q, const int32_t* kv, bool paged, int B, int qpb, int g, int causal,
                               int total_q, long kv_cap, int32_t* tmp, int32_t* entries, int32_t* n_entries,
                               int max_entries, cudaStream_t stream, bool skip_single, bool pairs, int grid,
                               bool fp8, int split_grid, int Hkv, int wl, int wr, const TailSplit& tail) {
    // flags: bit 0 paged (kv holds cache lengths), bit 1 skip single-query
    // requests, bit 2 pairs of row blocks
    const int flags = (paged ? 1 : 0) | (skip_single ? 2 : 0) | (pairs ? 4 : 0);
    varlen_plan_kernel<<<1, 1024, 0, stream>>>(cu_q, kv, flags, B, qpb, g, causal, total_q, kv_cap, tmp,
                                               entries, n_entries, max_entries, grid,
                                               fp8 ? kDecPerKey8 : kDecPerKey, split_grid, Hkv, wl, wr, tail);
    return cudaGetLastError();
}

cudaError_t launch_varlen_packed(const CUtensorMap& tm_q, const CUtensorMap& tm_k, const CUtensorMap& tm_v,
                                 const CUtensorMap& tm_o, const PrefillArgs& a, long max_items, cudaStream_t stream) {
    switch (a.D * 2 + (a.f16 ? 1 : 0)) {
        case 64 * 2: return ot::launch_onetile<64, ot::kPacked, true, false>(tm_q, tm_k, tm_v, tm_o, a, max_items, 0, stream);
        case 64 * 2 + 1: return ot::launch_onetile<64, ot::kPacked, true, true>(tm_q, tm_k, tm_v, tm_o, a, max_items, 0, stream);
        case 128 * 2: return ot::launch_onetile<128, ot::kPacked, true, false>(tm_q, tm_k, tm_v, tm_o, a, max_items, 0, stream);
        case 128 * 2 + 1: return ot::launch_onetile<128, ot::kPacked, true, true>(tm_q, tm_k, tm_v, tm_o, a, max_items, 0, stream);
        case 256 * 2: return ot::launch_onetile<256, ot::kPacked, true, false>(tm_q, tm_k, tm_v, tm_o, a, max_items, 0, stream);
        case 256 * 2 + 1: return ot::launch_onetile<256, ot::kPacked, true, true>(tm_q, tm_k, tm_v, tm_o, a, max_items, 0, stream);
        default: return cudaErrorInvalidValue;
    }
}

int varlen_packed_take_device_error() { return ot::take_error(); }

}  // namespace gqa
