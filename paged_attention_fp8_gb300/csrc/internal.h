// internal.h -- declarations shared by the host code and the kernels of
// libpafp8 (not part of the public ABI).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/pafp8.h"

namespace pafp8 {

constexpr int kHeadDim = 128;   // head_dim served by this library
constexpr int kPageSize = 16;   // page_size served by this library
constexpr int kMaxGroupDecode = 8;
constexpr int kMaxGroupPrefill = 16;
constexpr int kMaxGroupTree = 128;
constexpr int kTileRows = 128;   // prefill query rows (token x head) per tile
constexpr int kTileKeys = 128;   // prefill keys per KV tile (8 pages)
// Default bound of a kernel's pipeline waits, in SM clock cycles (~1 s).
constexpr long long kWaitCyclesDefault = 2000000000LL;

// Layout of the int32 partition metadata that the plan builds on the host and
// uploads to the head of the workspace.  Word offsets of the variable-length
// arrays are stored in the header.
enum MetaHeader : int {
    kMetaMagic = 0,      // 0x38464150 ("PAF8" little-endian)
    kMetaMode,           // 0 decode, 1 prefill
    kMetaBatch,
    kMetaHeadBlocks,     // number of KV-head blocks (nhb)
    kMetaHeadsPerCta,    // KV heads per block (hpc)
    kMetaGroup,          // query heads per KV head
    kMetaNumCtas,        // persistent CTAs of the main kernel (0: no launch)
    kMetaNumSegs,
    kMetaNumPartials,
    kMetaNumMerge,
    kMetaOffReqPage,     // int32[batch]   first entry of the request in kv_indices
    kMetaOffReqKvLen,    // int32[batch]   kv_len of the request
    kMetaOffCtaSeg,      // int32[num_ctas+1] CSR of segments per CTA
    kMetaOffSeg,         // int32[4*num_segs] (row, page_begin, page_end, out_slot); tree: [kTreeSegWords*num_segs]
                         // hk, first row, tile_begin, tile_end, slot, qo_begin, qo_len, kv_len, page_begin, 0, 0, 0
    kMetaOffMergePtr,    // int32[num_merge+1]
    kMetaOffMergeRow,    // int32[num_merge]
    kMetaOffMergeSlot,   // int32[num_partials]
    kMetaOffReqQo,       // int32[batch+1] qo_indptr (prefill)
    kMetaNumTiles,       // prefill tiles
    kMetaOffTile,        // int32[8*num_tiles] prefill items: b, hk, t0, nkv, qo_begin, qo_len, kv_len, page_begin
                         // (under a window: its gap of 16-token pages for b, and kv_len without them);
                         // tree: int32[8*num_merge] split lines: slot0, slot1, qo_begin, hk, rows, first row, 0, 0
    kMetaTileRows,       // packed query rows per prefill tile
    kMetaOffRowMerge,    // int32[rows] merge entry of each decode row, or -1
    kMetaNumChunks,      // decode pages handed out at run time, in chunks
    kMetaOffChunk,       // int32[4*num_chunks] (row, page_begin, page_end, out_slot)
    kMetaHeaderWords = 32
};

constexpr int kTreeSegWords = 12;

// Decode work handed out at run time: the last 1/kDynDiv of every row's
// pages, cut into chunks of about 1/kDynChunksPerCta of a CTA's share of
// them, when the batch has at least kDynMinPagesPerCta pages per CTA and at
// least one row per kDynMinRowsDiv CTAs (with fewer, longer rows the chunks
// would add many partial states to each row and slow its merge).  Each CTA
// takes chunks from a counter in the workspace after its own pages; a row's
// chunks add one or two partial states to it.
constexpr int kDynDiv = 16;
constexpr int kDynChunksPerCta = 1;
constexpr int kDynMinChunk = 4;
constexpr int kDynMinPagesPerCta = 16;
constexpr int kDynMinRowsDiv = 4;
// Word offsets in the workspace's 256-byte status block: the status word,
// the chunk counter and the count of CTAs done with chunks (both reset by the
// last CTA of each launch).
constexpr int kStatusWord = 0, kChunkCounterWord = 32, kChunkDoneWord = 48;
constexpr int32_t kMetaMagicValue = 0x38464150;

// What masked logits (-inf) are multiplied by stays above zero, or they would
// turn into NaN: a product of small scales that underflows becomes fp32's
// smallest number, under which every logit is zero all the same.  (One maximum
// that passes NaN on; a comparison and a selection took the bf16-query prefill
// over block scales 1 us longer.)
__host__ __device__ __forceinline__ float above_zero(float factor) {
#ifdef __CUDA_ARCH__
    asm("max.NaN.f32 %0, %1, 0f00000001;" : "=f"(factor) : "f"(factor));
    return factor;
#else
    return factor == 0.0f ? 1.4012984643e-45f : factor;
#endif
}

// log2-domain softmax scale, folded in double by the host (per-tensor scales)
// and the kernels (per-head ones) in the same order, so equal scales give the
// same float.
__host__ __device__ __forceinline__ float fold_scale_log2(float sm_scale, float q_scale, float k_scale) {
    return above_zero((float)((double)sm_scale * (double)q_scale * (double)k_scale * 1.4426950408889634));
}

// A load from an array that earlier work of the stream may have written (page
// ids, lengths, queries, scales).  A grid launched programmatically (EARLY) is
// resident while that work still runs, and __ldg wants memory that nothing
// writes as long as the grid lives: such a grid loads plainly, after its
// griddepcontrol.wait.  The plans' metadata comes by copies, which no launch
// overlaps, and keeps __ldg.
template <bool EARLY, typename T>
__device__ __forceinline__ T load_input(const T* p) {
    if constexpr (EARLY) return *p;
    else return __ldg(p);
}

// A request's 16-token sub-page vp (a page of 16 m tokens is m of them) as
// TMA coordinates: the pool page holding it and its first token slot there
// (the cache maps span whole pages, page_size slots; sub-page j of a page
// starts at slot 16 j).  A page id outside [0, num_pages) reads page 0 and
// sets `bad`.
struct SubPageAt {
    int slot, page;
};
template <bool EARLY>
__device__ __forceinline__ SubPageAt sub_page(const int32_t* idx, int vp, int m, int num_pages, bool& bad) {
    const int e = m == 1 ? vp : vp / m;
    const int pg = load_input<EARLY>(idx + e);
    bad = pg < 0 || pg >= num_pages;
    return SubPageAt{(vp - e * m) * kPageSize, bad ? 0 : pg};
}

// The keys that a row at position p sees under a window of w keys and s first
// tokens that stay visible: j <= p with j < s or j > p - w.  A work item reads
// the 16-token pages 0 .. head - 1 (the sinks') and, gap pages further, those
// from its first window key on; they are numbered without the gap, page u
// standing for u + gap from head on.  first_key: the first key in the window of
// the item's first row (negative: the window reaches past the start).  Without
// a window gap is 0.
struct WindowUnits {
    int head, gap;
    __host__ __device__ int at(int u) const { return u < head ? u : u + gap; }
};
__host__ __device__ inline WindowUnits window_units(int first_key, int sinks) {
    const int head = sinks > 0 ? (sinks - 1) / kPageSize + 1 : 0;
    const int from = first_key > 0 ? first_key / kPageSize : 0;
    return WindowUnits{head, from > head ? from - head : 0};
}

// Variants of the decode and prefill kernels, beside the plain one: a sliding
// window, and block scales (with or without a window).
constexpr int kVarPlain = 0, kVarWindow = 1, kVarBlocks = 2;

// Status word bits written by the kernels into the workspace.
enum : uint32_t {
    kStatusBounds = 1u,   // a page index outside [0, num_pages)
    kStatusTimeout = 2u,  // a bounded mbarrier wait expired
};

struct DecodeParams {
    const void* q;           // [batch, Hq, D]
    const int32_t* kv_indices;
    void* o;                 // [batch, Hq, D]
    float* lse;              // [batch, Hq] or nullptr
    const int32_t* meta;     // device copy of the metadata words
    float* part_o;           // [num_partials, hpc*group, D]
    float* part_lse;         // [num_partials, hpc*group] (log2 domain)
    uint32_t* status;        // status block: status word, chunk counter, CTAs done
    int head_dim;            // 128 or 64
    int q_dtype, kv_dtype, o_dtype;
    int num_qo_heads, num_kv_heads, num_pages;
    int page_mult;           // page_size / 16: a page is read as page_mult 16-token sub-pages
    float sm_scale_log2;     // sm_scale * q_scale * k_scale * log2(e)
    float v_scale;
    // Per-head scale tensors (device arrays) instead of the per-tensor scales
    // folded above, when k_scales is not null: q_scales [Hq] (or null: 1),
    // k_scales and v_scales [Hkv]; the kernels fold sm_scale with them.
    const float* q_scales;
    const float* k_scales;
    const float* v_scales;
    float sm_scale;
    // Scales of 16-token blocks, [num_pages, page_mult, Hkv], when not null
    // (sm_scale_log2 then holds no k_scale, and v_scale is 1).
    const float* k_blocks;
    const float* v_blocks;
    int window, sinks;       // keys a row sees besides the first `sinks`; window 0: all
    long long wait_cycles;   // bound of a pipeline wait (SM clock cycles)
};

struct AppendParams {
    const void* k_new;       // [nnz, Hkv, D] of src_dtype
    const void* v_new;
    const int32_t* batch_indices;  // [nnz]
    const int32_t* positions;      // [nnz]
    const int32_t* kv_indptr;      // [batch + 1]
    const int32_t* kv_indices;
    void* k_cache;           // [num_pages, page_size, Hkv, D] of kv_dtype (fp8)
    void* v_cache;
    uint32_t* status;        // or nullptr
    long long nnz;
    int num_kv_heads, batch, num_pages;
    int src_dtype, kv_dtype;
    int hnd;                 // cache layout: 0 [page][slot][head][d], 1 [page][head][slot][d]
    int page_size;
    int head_dim;            // 128 or 64
    float k_inv, v_inv;      // fp32(1 / scale)
};

using TablesParams = pafp8_tables_desc;  // the kernel takes the call's description as it is

struct RopeParams {
    const void* q;               // [nnz, Hq, D], tokens q_stride elements apart
    const void* k;               // [nnz, Hkv, D]
    const void* v;
    long long q_stride, k_stride, v_stride;
    const void* q_weight;        // [D] of src_dtype, or nullptr: no norm
    const void* k_weight;
    const float* cos_sin;        // [max_position, rot_dim]: cosines, then sines
    const int32_t* positions;    // [num_axes] rows pos_stride apart, of nnz
    const uint8_t* pair_axis;    // [rot_dim / 2] or nullptr (axis 0)
    const long long* slots;      // [nnz]
    void* q_out;                 // [nnz, Hq, D] of q_out_dtype
    void* k_cache;
    void* v_cache;
    uint32_t* status;            // or nullptr
    long long nnz, pos_stride, num_slots;
    int num_qo_heads, num_kv_heads, head_dim, rot_dim, max_position, num_axes;
    int src_dtype, kv_dtype, q_out_dtype;
    int interleaved;             // pairs: 0 dims (i, i + rot_dim / 2), 1 dims (2i, 2i + 1)
    int hnd, page_size;
    float eps, q_inv, k_inv, v_inv;  // inv: fp32(1 / scale)
};

struct BlockAppendParams {
    const void* k;               // [nnz, Hkv, D] of src_dtype, tokens k_stride elements apart
    const void* v;
    const int32_t* qo_indptr;    // [batch + 1]: rows of each request's new tokens
    const int32_t* cached_lens;  // [batch]: position of its first new token
    const int32_t* kv_indptr;    // [batch + 1]
    const int32_t* kv_indices;
    void* k_cache;
    void* v_cache;
    float* k_scales;             // [num_pages, page_size / 16, Hkv]
    float* v_scales;
    uint32_t* status;            // or nullptr
    long long nnz, k_stride, v_stride;
    int batch, num_kv_heads, head_dim, num_pages, page_size;
    int src_dtype, kv_dtype, hnd;
    int span;                    // set by the launcher: new tokens a warp looks through for its blocks
};

struct ReadParams {
    const void* k_cache;
    const void* v_cache;
    const int32_t* out_indptr;   // [batch + 1]: output rows of each request
    const int32_t* starts;       // [batch]: position of its first row
    const int32_t* kv_indptr;
    const int32_t* kv_indices;
    void* k_out;                 // [nnz, Hkv, D] of out_dtype
    void* v_out;
    const float* k_scales;       // [num_pages, page_size / 16, Hkv], or nullptr: k_scale
    const float* v_scales;
    uint32_t* status;            // or nullptr
    long long nnz;
    int batch, num_kv_heads, head_dim, num_pages, page_size;
    int kv_dtype, out_dtype, hnd;
    int tile;                    // set by the launcher: output rows a thread block
    float k_scale, v_scale;
};

struct PrefillParams {
    const void* q;           // [nnz_qo, Hq, D]
    int head_dim;            // D: 128 or 64
    const int32_t* kv_indices;
    void* o;                 // [nnz_qo, Hq, D]
    float* lse;              // [nnz_qo, Hq] or nullptr
    const int32_t* meta;     // device copy of the metadata words
    uint32_t* status;
    int q_dtype, kv_dtype, o_dtype;
    int num_qo_heads, num_kv_heads, num_pages;
    int page_mult;           // page_size / 16: a page is read as page_mult 16-token sub-pages
    int group;               // query heads per KV head
    int tile_tokens;         // query tokens per 128-row tile (128 / group)
    float sm_scale_log2;     // sm_scale * q_scale * k_scale * log2(e)
    float v_scale;
    // Per-head scale tensors (device arrays) instead of the per-tensor scales
    // folded above, when k_scales is not null: q_scales [Hq] (or null: 1),
    // k_scales and v_scales [Hkv]; the kernels fold sm_scale with them.
    const float* q_scales;
    const float* k_scales;
    const float* v_scales;
    float sm_scale;
    // Scales of 16-token blocks, [num_pages, page_mult, Hkv], when not null
    // (sm_scale_log2 then holds no k_scale, and v_scale is 1).
    const float* k_blocks;
    const float* v_blocks;
    int window, sinks;       // keys a row sees besides the first `sinks`; window 0: all
    long long wait_cycles;   // bound of a pipeline wait (SM clock cycles)
};

struct TreeParams {
    const void* q;           // [nnz_qo, Hq, D]
    const int32_t* kv_indices;
    void* o;                 // [nnz_qo, Hq, D]
    float* lse;              // [nnz_qo, Hq] or nullptr
    const int32_t* meta;     // device copy of the metadata words
    float* part_o;           // [num_partials, rows_pad, D]
    float* part_lse;         // [num_partials, rows_pad] (log2 domain)
    uint32_t* status;
    const uint32_t* tree_mask;  // [nnz_qo, mask_words]
    int mask_words;
    int rows_pad;            // rows of the largest row tile
    int q_dtype, kv_dtype, o_dtype;
    int q_pieces;            // e4m3 pieces of a query row (1 for an fp8 query or a 2-byte cache)
    int q_buffers, stages;   // set by the launcher from the shared memory there is
    int num_qo_heads, num_pages, page_mult, group;
    uint32_t group_magic;    // ceil(2^32 / group) (0 for group 1): n / group is the high word of n times it, n < 2^25
    float sm_scale_log2;     // sm_scale * q_scale * k_scale * log2(e)
    float v_scale;
    const float* q_scales;   // per-head scales, as in DecodeParams
    const float* k_scales;
    const float* v_scales;
    float sm_scale;
    long long wait_cycles;   // bound of a pipeline wait (SM clock cycles)
};

// Launchers (decode*.cu, prefill_d128.cu / prefill_d64.cu).  Return the launch's cudaError_t.
// heads_per_box: KV heads covered by one TMA box of the cache maps (the
// whole head block when the page-wide map could be encoded, else 1).
using DecodeLaunch = cudaError_t(const DecodeParams& p, const CUtensorMap& tmap_k, const CUtensorMap& tmap_v, int num_ctas,
                                 int heads_per_cta, int group, int heads_per_box, cudaStream_t stream);
DecodeLaunch launch_decode, launch_decode_window, launch_decode_blocks;  // the first picks among the variants
cudaError_t launch_append(const AppendParams& p, cudaStream_t stream);
cudaError_t launch_tables(const TablesParams& p, cudaStream_t stream);
cudaError_t launch_rope(const RopeParams& p, cudaStream_t stream);
cudaError_t launch_append_blocks(const BlockAppendParams& p, cudaStream_t stream);
cudaError_t launch_read_kv(const ReadParams& p, cudaStream_t stream);
// Size of the built-in scratch of the no-allocation decode entry point, and
// the device ordinals it serves.
constexpr size_t kNoAllocScratchBytes = PAFP8_NOALLOC_SCRATCH_BYTES;
constexpr int kMaxDevices = 64;
// Device address of the built-in scratch on the current device (looked up
// once per device; decode.cu).
cudaError_t noalloc_scratch(void** ptr);

cudaError_t launch_merge(const DecodeParams& p, int num_merge, int heads_per_cta, int group,
                         cudaStream_t stream);
// Whether a prefill plan's items are those of CTA pairs: a 2-byte cache at
// head_dim 128, with a window of 896 keys or more if it has one.  Short windows
// mean many items of a few tiles, and a pair's item covers twice the tokens, so
// more of its tiles lie outside each row's window.  (us on pairs / on single
// CTAs, one prompt of 16384 tokens, 32 / 8 heads: window 500 219 / 184, 700 248 /
// 233, 896 286 / 266, 1000 289 / 295, 1500 386 / 411; 9 prompts of 1000-4000, 16 /
// 4 heads: 500 178 / 148, 700 195 / 184, 896 226 / 210, 1000 238 / 231, 1500 284 /
// 303.  The two meet at 1000: just above the bound pairs still cost up to 8 %.)
constexpr int kPairWindow = 896;
inline bool prefill_pairs(int head_dim, int kv_dtype, int window) {
    return head_dim == kHeadDim && (kv_dtype == PAFP8_F16 || kv_dtype == PAFP8_BF16) &&
           (window == 0 || window >= kPairWindow);
}

// tmap_o: map over o with the 2-byte query tile's box (the fp8-query kernel
// writes full output tiles with bulk tensor stores through it).  One
// translation unit per head size (prefill_d128.cu, prefill_d64.cu).
using PrefillLaunch = cudaError_t(const PrefillParams& p, const CUtensorMap& tmap_q, const CUtensorMap& tmap_k,
                                  const CUtensorMap& tmap_v, const CUtensorMap& tmap_o, int num_ctas, cudaStream_t stream);
PrefillLaunch launch_prefill_d128, launch_prefill_d64, launch_prefill_window_d128, launch_prefill_window_d64,
    launch_prefill_blocks_d128, launch_prefill_blocks_d64;
inline PrefillLaunch* prefill_launcher(const PrefillParams& p) {
    if (p.k_blocks != nullptr) return p.head_dim == 64 ? launch_prefill_blocks_d64 : launch_prefill_blocks_d128;
    if (p.window > 0) return p.head_dim == 64 ? launch_prefill_window_d64 : launch_prefill_window_d128;
    return p.head_dim == 64 ? launch_prefill_d64 : launch_prefill_d128;
}

// The tree kernel over its plan's segments and, with split lines, the merge of
// their partial states.  One translation unit per head size and row count.
using TreeLaunch = cudaError_t(const TreeParams& p, const CUtensorMap& tmap_k, const CUtensorMap& tmap_v, int num_ctas,
                               int num_merge, cudaStream_t stream);
TreeLaunch launch_tree_d128_r32, launch_tree_d128_r64, launch_tree_d64_r32, launch_tree_d64_r64;
// Rows of a row tile: 32 when every draft fits, else 64 (of which a draft may
// take several).  8 requests of 32768 keys with 32 rows take 98.2 us in tiles of
// 32 and 119 in tiles of 64; 64 requests of 512-4096 keys with 64 rows 109 us
// in tiles of 32 (the cache read and converted for twice as many tiles) and 83.5
// in one of 64; drafts of 68 to 244 rows 92.5 and 78.4; up to 48 rows over a bf16
// cache 72.8 and 59.8.  Batches of short and long drafts were not measured.
inline int tree_tile_rows(int most_rows) { return most_rows <= 32 ? 32 : 64; }
inline TreeLaunch* tree_launcher(int head_dim, int tile_rows) {
    if (head_dim == 64) return tile_rows == 32 ? launch_tree_d64_r32 : launch_tree_d64_r64;
    return tile_rows == 32 ? launch_tree_d128_r32 : launch_tree_d128_r64;
}

}  // namespace pafp8
