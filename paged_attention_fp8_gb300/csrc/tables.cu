// tables.cu -- block tables and slot maps of one step, built on the GPU from
// request lengths.  sm_103a.
//
// Request b holds c_b tokens and takes n_b new ones; with P tokens a page it
// has h_b = ceil(c_b / P) pages and needs t_b = ceil((c_b + n_b) / P).  Its
// pages j in [h_b, t_b) come from the free list in request order: page j is
// free_pages[used + sum_{a<b} (t_a - h_a) + j - h_b].  From these follow the
// CSR page table (kv_indptr, kv_indices, last_page_len), and for token u of
// request b its position c_b + u and its cache slot page * P + position % P.
// For a drafted tree the parents give token u's depth (the number of its
// ancestors), its rotary position c_b + depth, and its mask: bit w is set when
// token w is u or an ancestor of u.
//
// One launch.  The three prefix sums (pages, free pages, tokens) are not
// scanned by a kernel of their own: every block adds up the lengths of the
// requests before its own (8 bytes each, read through L2) and scans its own
// eight, one a warp.  A second launch costs about 2 us; the redundant sums
// cost less than that up to some ten thousand requests.  Long page lists are
// split over blockIdx.y, so one request of a million tokens spreads over the
// device too.  Bounded by latency (the length loads, the block's reductions,
// one dependent page load): 7-8 us with everything cold for one request, 9
// for 64, 15-16 for 1021 of up to 32768 tokens, whose page ids take 1.3 us at
// the copy rate.
#include "../../include/pafp8.h"
#include "internal.h"

namespace pafp8 {
namespace {

constexpr int kTblThreads = 256;
constexpr int kTblWarps = kTblThreads / 32;  // requests per block, one a warp

struct Lens {
    int cached, fresh;  // tokens held, new tokens
    bool bad;
};
// A negative length, or a sum past int32, counts as zero (and is reported).
__device__ __forceinline__ Lens load_lens(const TablesParams& p, int b) {
    int c = __ldg(p.cached_lens + b), n = __ldg(p.new_lens + b);
    const bool bad = c < 0 || n < 0 || (long long)c + n > 0x7FFFFFFFll - p.page_size;
    return Lens{bad ? 0 : c, bad ? 0 : n, bad};
}
__device__ __forceinline__ int pages_of(int tokens, int page_size) { return (tokens + page_size - 1) / page_size; }

__device__ __forceinline__ long long warp_sum(long long v) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, d);
    return v;
}

__global__ void __launch_bounds__(kTblThreads) tables_kernel(const TablesParams p) {
    __shared__ long long s_sum[3][kTblWarps];
    __shared__ int s_own[3][kTblWarps];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int b0 = blockIdx.x * kTblWarps;
    const int P = p.page_size;
    bool bad = false;

    // Sums over the requests before this block's.
    long long pages = 0, need = 0, toks = 0;
    for (int b = threadIdx.x; b < b0; b += kTblThreads) {
        const Lens l = load_lens(p, b);
        const int h = pages_of(l.cached, P), t = pages_of(l.cached + l.fresh, P);
        pages += t;
        need += t - h;
        toks += l.fresh;
    }
    pages = warp_sum(pages);
    need = warp_sum(need);
    toks = warp_sum(toks);
    // This warp's own request.
    const int b = b0 + warp;
    const bool live = b < p.batch;
    Lens own{0, 0, false};
    if (live) own = load_lens(p, b);
    bad |= own.bad;
    const int have = pages_of(own.cached, P), total = pages_of(own.cached + own.fresh, P);
    if (lane == 0) {
        s_sum[0][warp] = pages;
        s_sum[1][warp] = need;
        s_sum[2][warp] = toks;
        s_own[0][warp] = total;
        s_own[1][warp] = total - have;
        s_own[2][warp] = own.fresh;
    }
    const int used = __ldg(p.free_used);
    __syncthreads();
    long long base_page = 0, base_need = 0, base_tok = 0;
#pragma unroll
    for (int w = 0; w < kTblWarps; ++w) {
        base_page += s_sum[0][w];
        base_need += s_sum[1][w];
        base_tok += s_sum[2][w];
        if (w < warp) {
            base_page += s_own[0][w];
            base_need += s_own[1][w];
            base_tok += s_own[2][w];
        }
    }

    if (live) {
        const int step = 32 * gridDim.y, first = 32 * blockIdx.y + lane;
        int* row = p.block_table + (long long)b * p.block_stride;
        const long long take = (long long)used + base_need - have;  // page j is free_pages[take + j]
        auto fresh_page = [&](int j) -> int {
            const long long f = take + j;
            return used >= 0 && f < p.num_free ? __ldg(p.free_pages + f) : -1;
        };
        // Page list.  Entries from the free list go into the block table as
        // well; nothing here reads an entry that this launch writes.
#pragma unroll 4
        for (int j = first; j < total; j += step) {
            int page = -1;
            if (j < p.block_width) {
                page = j < have ? row[j] : fresh_page(j);
                if (j >= have) row[j] = page;
            }
            bad |= page < 0 || page >= p.num_pages;
            if (base_page + j < p.max_pages) p.kv_indices[base_page + j] = page;
        }
        // Tokens.  (Unsigned: the last step of nearly 2^31 tokens passes int's range.)
        for (unsigned i = first; i < (unsigned)own.fresh; i += step) {
            const int u = (int)i;
            const long long t = base_tok + u;
            if (t >= p.max_tokens) {
                bad = true;
                break;
            }
            const int pos = own.cached + u;
            const int j = pos / P;
            int page = -1;
            if (j < p.block_width) page = j < have ? row[j] : fresh_page(j);
            p.batch_indices[t] = b;
            p.positions[t] = pos;
            p.slots[t] = page >= 0 && page < p.num_pages ? (long long)page * P + (pos - j * P) : -1ll;
            // Ancestors come in falling order, so the mask's words are
            // finished one after the other from the top.
            int depth = 0;
            const int words = p.tree_mask != nullptr ? p.mask_words : 0;
            uint32_t* mrow = p.tree_mask + t * p.mask_words;
            if (p.parents != nullptr) {
                int w = words - 1;
                uint32_t bits = 0;
                if (words > 0 && u >= 32 * words) bad = true;
                for (int a = u;;) {
                    if (words > 0 && (a >> 5) < words) {
                        for (; w > (a >> 5); --w) {
                            mrow[w] = bits;
                            bits = 0;
                        }
                        bits |= 1u << (a & 31);
                    }
                    const int up = __ldg(p.parents + base_tok + a);
                    if (up < 0 || up >= a) {
                        bad |= up != -1;
                        break;
                    }
                    a = up;
                    ++depth;
                }
                for (; w >= 0; --w) {
                    mrow[w] = bits;
                    bits = 0;
                }
            } else {  // a chain: token u follows u - 1
                depth = u;
                if (words > 0 && u >= 32 * words) bad = true;
                for (int w = 0; w < words; ++w) {
                    const int k = u + 1 - 32 * w;  // bits of this word
                    mrow[w] = k >= 32 ? 0xFFFFFFFFu : k > 0 ? (1u << k) - 1u : 0u;
                }
            }
            if (p.rope_positions != nullptr) p.rope_positions[t] = own.cached + depth;
        }
        if (blockIdx.y == 0 && lane == 0) {
            p.kv_indptr[b] = (int)base_page;
            p.qo_indptr[b] = (int)base_tok;
            p.last_page_len[b] = total > 0 ? own.cached + own.fresh - (total - 1) * P : 0;
            bad |= total > p.block_width || base_page + total > p.max_pages || base_page + total > 0x7FFFFFFFll ||
                   base_tok + own.fresh > 0x7FFFFFFFll || (total > have && (used < 0 || take + total > p.num_free));
        }
    }
    // The last request's block closes the CSR arrays and blanks the tokens
    // behind it: no request, no slot, position 0, an empty mask.
    if (blockIdx.x == gridDim.x - 1) {
        long long tok_end = 0, page_end = 0, need_end = 0;
#pragma unroll
        for (int w = 0; w < kTblWarps; ++w) {
            page_end += s_sum[0][w] + s_own[0][w];
            need_end += s_sum[1][w] + s_own[1][w];
            tok_end += s_sum[2][w] + s_own[2][w];
        }
        if (blockIdx.y == 0 && threadIdx.x == 0) {
            p.kv_indptr[p.batch] = (int)page_end;
            p.qo_indptr[p.batch] = (int)tok_end;
            const long long end = used + need_end;
            *p.free_used_out = (int)(end < p.num_free ? end : p.num_free > used ? p.num_free : used);
        }
        for (long long t = tok_end + (long long)blockIdx.y * kTblThreads + threadIdx.x; t < p.max_tokens;
             t += (long long)gridDim.y * kTblThreads) {
            p.batch_indices[t] = -1;
            p.positions[t] = 0;
            p.slots[t] = -1;
            if (p.rope_positions != nullptr) p.rope_positions[t] = 0;
            if (p.tree_mask != nullptr)
                for (int w = 0; w < p.mask_words; ++w) p.tree_mask[t * p.mask_words + w] = 0;
        }
    }
    if (p.status != nullptr && __any_sync(0xFFFFFFFFu, bad) && lane == 0) atomicOr(p.status, kStatusBounds);
}

}  // namespace

cudaError_t launch_tables(const TablesParams& p, cudaStream_t stream) {
    const int gx = p.batch > 0 ? (p.batch + kTblWarps - 1) / kTblWarps : 1;
    // Rows of the grid so that a warp walks about 128 entries of an average
    // request, up to two waves of 152 SMs x 8 blocks.
    const long long per = (p.max_pages > p.max_tokens ? p.max_pages : p.max_tokens) / (p.batch > 0 ? p.batch : 1);
    long long gy = (per + 127) / 128;
    const long long most = 2432 / gx > 1 ? 2432 / gx : 1;
    if (gy > most) gy = most;
    if (gy < 1) gy = 1;
    tables_kernel<<<dim3((unsigned)gx, (unsigned)gy), kTblThreads, 0, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace pafp8
