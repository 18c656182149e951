// Block tables, packed offsets and slot map of one serving step, built on the
// device from the requests' lengths.
//
// Request b holds past_b tokens in its pages and brings new_b more: its new
// tokens take the positions past_b .. past_b + new_b - 1 and, beyond the pages
// it has, ceil((past_b + new_b) / page_size) - ceil(past_b / page_size) pages
// of the free list, handed out in request order.  Token t of the packed batch
// belongs to the request whose range [cu_b, cu_b + new_b) holds it; its slot is
// page * page_size + position % page_size.
//
// The whole call is one launch: the prefix sums over the requests (new tokens,
// new pages) are short, so every block computes them for itself, 512 requests
// a round, and fills its own range of tokens from the round that holds them;
// nothing is handed between blocks.  A token finds its request by binary
// search among the round's 512 first tokens in shared memory.  A fresh page is
// entered in the table by the token at its first position, which is always a
// new token.  Bound by latency: a round is two dependent loads, a block scan
// and the search.  Measured: 3.1 us on the GPU for 64 requests of one token (10 us
// a call from Python, 11 for 768 requests of up to 331 tokens, which write 3 MB).
#include <climits>

#include "internal.h"

namespace gqa {
namespace {

constexpr int NT = 512;            // threads of a block = requests of a round
constexpr int NW = NT / 32;

struct Pair {                      // new tokens, new pages (sums of 32-bit lengths need 64 bits)
    long long tok, pag;
};

__device__ __forceinline__ Pair warp_scan(Pair x, int lane) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long t = __shfl_up_sync(0xffffffffu, x.tok, o);
        const long long p = __shfl_up_sync(0xffffffffu, x.pag, o);
        if (lane >= o) {
            x.tok += t;
            x.pag += p;
        }
    }
    return x;
}

__device__ __forceinline__ int sat_int(long long x) { return (int)min(x, (long long)INT_MAX); }

__global__ void __launch_bounds__(NT) paged_slots_kernel(const SlotArgs a, int tokens_per_block) {
    __shared__ Pair wsum[NW];
    __shared__ long long s_first[NT];   // first token of each request of the round
    __shared__ long long s_page[NT];    // index in the free list of its first fresh page
    __shared__ int s_past[NT], s_n0[NT];
    const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
    const long long t0 = (long long)blockIdx.x * tokens_per_block;
    const long long t1 = min(t0 + tokens_per_block, (long long)a.max_tokens);
    const bool lead = blockIdx.x == 0;  // also writes the per-request results
    const long long cap = (long long)a.max_pages * a.page_size;
    const int free0 = a.free_start ? max(*a.free_start, 0) : 0;
    long long tok = 0, pag = 0;         // totals of the rounds so far
    for (int b0 = 0; b0 < a.B; b0 += NT) {
        const int b = b0 + tid;
        int past = 0, nw = 0, n0 = 0;
        Pair x{0, 0};
        if (b < a.B) {
            past = (int)min((long long)max(a.past_lens[b], 0), cap);
            nw = max(a.new_lens[b], 0);
            const long long end = (long long)past + nw;
            n0 = (past + a.page_size - 1) / a.page_size;
            const long long n1 = min((end + a.page_size - 1) / a.page_size, (long long)a.max_pages);
            x.tok = nw;
            x.pag = max(0LL, n1 - n0);
            if (lead) a.cache_seqlens[b] = (int)min(end, cap);
        }
        Pair inc = warp_scan(x, lane);
        if (lane == 31) wsum[warp] = inc;
        __syncthreads();
        if (warp == 0) {
            Pair s = lane < NW ? wsum[lane] : Pair{0, 0};
            s = warp_scan(s, lane);
            if (lane < NW) wsum[lane] = s;
        }
        __syncthreads();
        if (warp > 0) {
            inc.tok += wsum[warp - 1].tok;
            inc.pag += wsum[warp - 1].pag;
        }
        const Pair all = wsum[NW - 1];
        s_first[tid] = tok + inc.tok - x.tok;      // past the last request: the total
        s_page[tid] = free0 + pag + inc.pag - x.pag;
        s_past[tid] = past;
        s_n0[tid] = n0;
        if (lead && b < a.B) {
            if (b == 0) a.cu_seqlens_q[0] = 0;
            a.cu_seqlens_q[b + 1] = (int)min(tok + inc.tok, (long long)a.max_tokens);
        }
        __syncthreads();
        // this block's tokens among the round's
        const long long lo = max(t0, tok), hi = min(t1, tok + all.tok);
        for (long long t = lo + tid; t < hi; t += NT) {
            int l = 0, r = NT;                      // last request of the round with first <= t
            while (r - l > 1) {
                const int m = (l + r) >> 1;
                if (s_first[m] <= t) l = m; else r = m;
            }
            // Requests without a token share their successor's first token:
            // the last of them is the one that has it.
            const int bb = b0 + l;
            const long long pos = s_past[l] + (t - s_first[l]);
            int slot = -1;
            if (pos < cap) {
                const int page = (int)pos / a.page_size, off = (int)pos % a.page_size;
                int32_t* entry = a.block_table + (size_t)bb * a.max_pages + page;
                int id;
                if (page >= s_n0[l]) {
                    const long long f = s_page[l] + (page - s_n0[l]);
                    id = f < a.num_free ? a.free_pages[f] : -1;
                    if (off == 0) *entry = id;
                } else {
                    id = *entry;
                }
                if (id >= 0 && id < a.num_pages) slot = id * a.page_size + off;
            }
            a.slots[t] = slot;
            a.positions[t] = sat_int(pos);
            a.requests[t] = bb;
        }
        tok += all.tok;
        pag += all.pag;
        if (!lead && tok >= t1) break;              // uniform; block 0 goes through every request
        __syncthreads();                            // the next round overwrites the shared arrays
    }
    for (long long t = max(t0, tok) + tid; t < t1; t += NT) {
        a.slots[t] = -1;
        a.positions[t] = 0;
        a.requests[t] = -1;
    }
    if (lead && tid == 0) {
        a.counts[0] = sat_int(tok);
        a.counts[1] = sat_int(pag);
        a.counts[2] = sat_int(free0 + pag);
    }
}

}  // namespace

cudaError_t launch_paged_slots(const SlotArgs& a, int num_sms, cudaStream_t stream) {
    // At least 512 tokens a block (one per thread), at most two blocks per SM:
    // more blocks would only repeat the prefix sums.
    const long most = 2L * (num_sms > 0 ? num_sms : 148);
    long per = ((long)a.max_tokens + most - 1) / most;
    per = per < NT ? NT : (per + 31) / 32 * 32;
    const long blocks = a.max_tokens > 0 ? (a.max_tokens + per - 1) / per : 1;
    paged_slots_kernel<<<(unsigned)blocks, NT, 0, stream>>>(a, (int)per);
    return cudaGetLastError();
}

}  // namespace gqa
