// prefill.cuh -- ragged causal prefill attention over a paged fp8 KV cache on
// the tcgen05 tensor cores (sm_103a).  Included by one translation unit per
// head size (prefill_d128.cu, prefill_d64.cu), which compile in parallel.
//
// What it computes: for request b with qo_len new query rows and kv_len keys,
// query row i (0-based among the new rows) of head h attends to keys
// j <= i + kv_len - qo_len (bottom-right aligned causal mask) of KV head
// h / group: o = v_scale * softmax(sm_scale * q_scale * k_scale * q.k) V,
// lse = ln sum exp(logits).  KV stays fp8 in HBM and is dequantized on load
// ("fp8 KV cache in the in-tree prefill kernel", Kernel note: KV is widened
// into a 2-byte shared-memory tile in the global -> shared path); with an fp8
// query the QK product runs natively in fp8 ("Enable Hopper FA3 FP8 attention
// in decode.py", review note on q_scale folding into sm_scale for FP8 BMM1).
//
// Work item: one KV head of one request and two query tiles A and B of 128
// rows each, packed as (token, head-of-group) pairs -- 128/group consecutive
// new tokens times the group's query heads per tile, B right after A -- so a
// dequantized K/V tile serves 256 query rows.  KV tiles are 128 keys (8
// pages).  Persistent CTAs take items from a longest-first list built by the
// plan, dealt in snake order (item_at).
//
// Roles (512 threads, four warpgroups; registers are moved by setmaxnreg from
// the dequant warpgroup (64) and the producer/MMA warpgroup (64) to the two
// softmax warpgroups (192), which hold a whole S row without spilling):
//   warps 0-3   dequant: raw fp8 K -> f16 K tile (2-byte query path); raw fp8
//               V -> f16 V tile (both paths; a 2-byte V tile is copied), in
//               the layout a 2-byte tile lands in ([64-dim half][key][128 B]),
//               zero beyond the request's keys;
//   warps 4-7   softmax of tile A, warps 8-11 softmax of tile B: thread r owns
//               TMEM lane r = query row r of its tile.  Reads S, masks, keeps
//               the running max and sum, writes P (f16) over the first half of
//               S in TMEM, rescales O in TMEM only when the max rises by more
//               than 2^8, and in the epilogue normalizes O and stores o, lse.
//               With a bf16 query on an fp8 cache each thread brings its Q
//               row into f16 range by an exact power of two and converts it in
//               place, for the next item as soon as its last pass of the
//               current one is done (before that item's epilogue);
//   warp 12     TMA producer: both Q tiles, K and V pages (one box per page);
//   warp 13     MMA issuer and TMEM owner (warps 14-15 idle).  Per KV tile j:
//                 S_A = Q_A K_j^T, S_B = Q_B K_j^T    (kind::f16 or kind::f8f6f4)
//                 O_A += P_A V_j,  O_B += P_B V_j      (kind::f16, A = P from TMEM)
//               issued as ... PV_A(j), QK_A(j+1), PV_B(j), QK_B(j+1) ... so
//               each tile's softmax overlaps the other tile's tensor work.
// TMEM columns: S_A/P_A 0-127, S_B/P_B 128-255, O_A 256-383, O_B 384-511.
// O_X is released by its softmax warps after each epilogue they run; the
// MMA warp waits for that release only before the first O_X write of the
// next item in which tile X has rows (so an empty tile B never advances the
// barrier ahead of the wait).
// The tensor pipe runs one CTA's MMAs in order, so an MMA writing S_X after
// O_X += P_X V has been issued cannot overtake it, and s_full(X, j) implies
// that the previous O update of X is complete.  Q and K in shared memory are
// K-major operands with the 128-byte swizzle (64-byte for the 64-byte fp8 rows
// of head_dim 64); V is the MN-major B operand of P V (dims along 128-byte
// rows, one row per key), so no role transposes it.  All waits are bounded; on
// expiry the kernel records a status bit and winds down.
//
// Pages of 16 m tokens (m > 1) are read as m sub-pages of 16: the TMA box of
// sub-page j is at token slot 16 j of its page, which covers both layouts.
// That path (kSlots) is its own instantiation so that the 16-token path keeps
// a producer loop without the division by m.
//
// Variants (VAR, each its own instantiations).
// Window: an item reads the 16-token pages of the sinks and, `gap` pages
// further, those from the first key that its first row sees on.  Positions and
// tiles count without the gap -- masks, limits and lengths are those of the
// shortened request -- and only the page lookups add it, so that the sinks cost
// a page rather than a tile.  Softmax rows mask keys between the sinks and
// their own first one, and a row whose tiles so far showed it nothing keeps its
// maximum at -inf, so that its first visible key sets it.  A prompt of 16384
// tokens under a window of 1024 with 4 sinks (276 GFLOP in visible pairs) takes
// 299 us: 923 TFLOP/s, 47 % of the measured rate, where the plain kernel reaches
// 53 % (and this one 64 % under a window of 4000).  A CTA has 13 or 14 items of 9
// tiles (1152 keys for each row's 1028), about 3700 cycles a tile; between an item's
// last P and the next item's first S passed 10,000 with Q's arrival and fit, the
// output and the first QK.  Leaving out the softmax of the columns that no row of a
// warp sees gained nothing (314 us against the 312 of that time) and cost block
// scales a fifth.
// Block scales: with s = ks_c q.k (ks_c the K scale of 16-key block c, folded
// with the softmax scale) and vs_c the block's V scale, P' = 2^(s + log2 vs_c -
// m) and m the running maximum of s + log2 vs_c: the V scale rides in the
// exponent, so that O = sum P' code needs no product of its own and P' keeps
// f16's range whatever the scales are, and l = sum_c (sum of P' over block c) /
// vs_c is the softmax's sum.  Warp 14, idle otherwise, looks the scales up four
// tiles at a time and hands them over through a ring of kScaleSlots tiles; the
// softmax warps read them before they wait for S.  The ragged prefill of 16
// prompts (32 / 8 heads of 128, bf16 query, 218 GFLOP) takes 237 us where one
// scale for the tensor takes 209; with an fp8 query 204 and 177.  What it costs
// most are registers: with 48 for the dequant and producer warps each, 192 a
// softmax thread took 285 us, 200 262 and 208 242; 208, 32 and 64 take 237.
#pragma once
#include <type_traits>

#include "../../include/pafp8.h"
#include "internal.h"
#include "ptx.cuh"

namespace pafp8 {
namespace {

using namespace ptx;

constexpr int kThreads = 512;  // four warpgroups; warps 14-15 only lend registers
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kHalfTile = kTileKeys * 128;  // 16 KB: 128 rows x 128 B
__device__ __forceinline__ uint32_t col_s(int x) { return 128u * (uint32_t)x; }  // S_X / P_X

// Sizes that depend on the head size DH (128 or 64).  A 2-byte row of DH
// elements is DH / 64 rows of 128 B ("halves", each under the 128-byte
// swizzle); an fp8 row is DH bytes (128-byte swizzle for 128, 64-byte for 64).
template <int DH>
struct Dims {
    static constexpr int NH = DH / 64;                       // 128-B halves of a 2-byte row
    static constexpr uint32_t kRawTile = kTileKeys * DH;      // fp8 K or V tile (128 keys)
    static constexpr uint32_t kRawPage = kPageSize * DH;      // fp8 page box (16 tokens)
    static constexpr uint32_t kF16Tile = NH * kHalfTile;      // 2-byte K or V tile (128 keys) or Q tile
};
template <int DH>
__device__ __forceinline__ uint32_t col_o(int x) { return 256u + (uint32_t)DH * (uint32_t)x; }  // O_X

constexpr int kScaleSlots = 8;                                    // tiles in the ring of block scales
// A tile's scales: the K scales of its 8 blocks, each twice (a packed pair),
// log2 of the V scales, 1 / V scale twice each.
constexpr uint32_t kScaleTile = kTileKeys / kPageSize * 20;

template <bool kF8, bool k2, int DH, int VAR = kVarPlain>
struct Layout {
    using Dm = Dims<DH>;
    // The 2-byte-query path spends its shared memory on two f16 K tiles (the
    // dequant of K_{j+1} may start while QK_B(j) still reads K_j) and keeps a
    // single raw fp8 stage per tensor; the fp8 path multiplies raw K directly.
    // A 2-byte cache (k2) brings K and V straight into the 16-bit tiles and has
    // no raw stages, but a third V tile: the dequant warps only zero, in place,
    // the V rows that no query row sees.  (Copying V from a raw stage took 130.7
    // us where this takes 126.3: 9 prompts, 16 / 4 heads of 64.)
    static constexpr int NKR = kF8 ? 4 : (k2 ? 0 : 1);  // raw K stages
    static constexpr int NVR = kF8 ? 2 : (k2 ? 0 : 1);  // raw V stages
    static constexpr int NK16 = kF8 ? 0 : 2;   // f16 K stages
    static constexpr int NV16 = k2 ? 3 : 2;    // f16 V stages
    static constexpr int nVr = k2 ? NV16 : NVR;  // V tiles that copies land in
    static constexpr uint32_t kQTile = kF8 ? kTileRows * DH : Dm::kF16Tile;
    static constexpr uint32_t q = 0;                     // Q_A, then Q_B
    static constexpr uint32_t kr = 2 * kQTile;
    static constexpr uint32_t vr = kr + NKR * Dm::kRawTile;
    static constexpr uint32_t k16 = vr + NVR * Dm::kRawTile;
    static constexpr uint32_t v16 = k16 + NK16 * Dm::kF16Tile;
    // fp8 query: a 16 KB staging half per query tile for the output's bulk
    // tensor stores (64 dims of 128 rows, 128-byte rows swizzled).
    static constexpr uint32_t ostage = v16 + NV16 * Dm::kF16Tile;
    static constexpr int NSC = VAR == kVarBlocks ? kScaleSlots : 0;
    static constexpr uint32_t scales = ostage + (kF8 ? 2 * kHalfTile : 0);
    static constexpr uint32_t bars = scales + NSC * kScaleTile;
    // barrier indices (8 bytes each)
    static constexpr int bQFull = 0, bQReady = 1, bQEmpty = 2;
    static constexpr int bKrFull = 3, bKrEmpty = bKrFull + NKR;
    static constexpr int bVrFull = bKrEmpty + NKR, bVrEmpty = bVrFull + nVr;
    static constexpr int bK16Full = bVrEmpty + NVR, bK16Empty = bK16Full + NK16;
    static constexpr int bV16Full = bK16Empty + NK16, bV16Empty = bV16Full + NV16;
    static constexpr int bSFull = bV16Empty + NV16;  // [2]
    static constexpr int bPFull = bSFull + 2;        // [2]
    static constexpr int bOFull = bPFull + 2;        // [2]
    static constexpr int bOEmpty = bOFull + 2;       // [2]
    static constexpr int bStageFree = bOEmpty + 2;    // [2]
    static constexpr int bStageReady = bStageFree + 2;  // [2]
    static constexpr int bDrain = bStageReady + 2;
    static constexpr int bScFull = bDrain + 1, bScEmpty = bScFull + NSC;
    static constexpr int nBars = bScEmpty + NSC;
    static constexpr uint32_t tmem_slot = bars + 8 * nBars;
    static constexpr uint32_t abort_flag = tmem_slot + 4;
    static constexpr uint32_t bytes = abort_flag + 4;
};
static_assert(1024 + Layout<false, false, 128>::bytes <= 232448, "shared memory budget (2-byte query)");
static_assert(1024 + Layout<true, false, 128>::bytes <= 232448, "shared memory budget (fp8 query)");
static_assert(1024 + Layout<false, true, 128>::bytes <= 232448, "shared memory budget (2-byte cache)");
static_assert(1024 + Layout<false, false, 64>::bytes <= 232448, "shared memory budget (2-byte query, D 64)");
static_assert(1024 + Layout<true, false, 64>::bytes <= 232448, "shared memory budget (fp8 query, D 64)");
static_assert(1024 + Layout<false, true, 64>::bytes <= 232448, "shared memory budget (2-byte cache, D 64)");
static_assert(1024 + Layout<false, false, 128, kVarBlocks>::bytes <= 232448 &&
                  1024 + Layout<true, false, 128, kVarBlocks>::bytes <= 232448,
              "shared memory budget (block scales)");
// Swizzled tiles start on 1024-byte boundaries (the 128-byte swizzle's atom).
static_assert(Layout<true, false, 64>::kr % 1024 == 0 && Layout<true, false, 64>::v16 % 1024 == 0 &&
                  Layout<false, false, 64>::v16 % 1024 == 0 && Layout<false, true, 64>::v16 % 1024 == 0,
              "1024-byte alignment of the D 64 tiles");

// The larger magnitude of two bf16 pairs, each half by itself.
__device__ __forceinline__ uint32_t max_abs_bf162(uint32_t a, uint32_t b) {
    const __nv_bfloat162 r = __hmax2(*reinterpret_cast<const __nv_bfloat162*>(&a),
                                     __habs2(*reinterpret_cast<const __nv_bfloat162*>(&b)));
    return *reinterpret_cast<const uint32_t*>(&r);
}

// f16x2 of fp8 values as bf16x2: exact, since an fp8 value has 4 significant bits
// and an exponent that both types hold.
__device__ __forceinline__ uint32_t half2_to_bf162(uint32_t h) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
    return pack_bf162(f.x, f.y);
}

struct Ring {
    int idx = 0;
    uint32_t phase = 0;
    __device__ __forceinline__ void next(int n) {
        if (++idx == n) {
            idx = 0;
            phase ^= 1u;
        }
    }
};

struct Item {
    int gap, hk, t0, nkv;        // nkv: KV tiles of the item (tile B's, or A's if B is empty)
    int qo0, qo_len, kv_len, page0;  // the request's first query row, rows, keys, first page entry
};

// One plan record per item, with the request fields the kernel needs, so an
// item start costs one round of independent loads.
__device__ __forceinline__ Item load_item(const int* items, int t) {
    const int* r = items + 8 * t;
    return Item{__ldg(r), __ldg(r + 1), __ldg(r + 2), __ldg(r + 3), __ldg(r + 4), __ldg(r + 5), __ldg(r + 6), __ldg(r + 7)};
}

// KV tiles that query tile `x` (0 = A, 1 = B) of an item needs: its last
// token's causal limit, capped by the request's own key tiles; 0 if the tile
// has no rows.
__device__ __forceinline__ int tile_nkv(int t0, int x, int TQ, int qo_len, int kv_len) {
    const int first = t0 + x * TQ;
    if (first >= qo_len) return 0;
    const int last = min(first + TQ, qo_len) - 1;
    const int lim = last + kv_len - qo_len;
    return min((kv_len + kTileKeys - 1) / kTileKeys, lim / kTileKeys + 1);
}

// The item's 16-token pages as it numbers them: under a window the plan takes
// the pages between the sinks' and the first that its first row sees (gap of
// them) out of the item, whose kv_len and positions count without them.
template <int VAR>
__device__ __forceinline__ int page_at(const PrefillParams& p, const Item& it, int vp) {
    if (VAR == kVarPlain || p.window == 0) return vp;
    return WindowUnits{p.sinks > 0 ? (p.sinks - 1) / kPageSize + 1 : 0, it.gap}.at(vp);
}

// The item that persistent worker i of G takes in round r.  Items are sorted
// longest first; even rounds deal them to workers 0 .. G-1, odd rounds back
// from G-1 to 0 (a snake), so each worker's total evens out while the items
// in flight at any time are the same neighbours as in plain round robin.  A
// worker stops at its first round whose item is past the list (no later
// round has one for it).
__device__ __forceinline__ int item_at(int r, int i, int G) { return r * G + ((r & 1) ? G - 1 - i : i); }

__device__ __forceinline__ void set_abort(uint32_t flag_addr, uint32_t* status) {
    asm volatile("st.shared.u32 [%0], 1;" ::"r"(flag_addr) : "memory");
    atomicOr(status, kStatusTimeout);
}

__device__ __forceinline__ bool aborted(uint32_t flag_addr) {
    uint32_t v;
    asm volatile("ld.volatile.shared.u32 %0, [%1];" : "=r"(v) : "r"(flag_addr) : "memory");
    return v != 0;
}

// Bounded wait that also gives up once another role has aborted.  A
// diagnostic instantiation (kDiag) polls with the host's shortened bound.
template <bool kDiag>
__device__ __forceinline__ bool wait_or_abort(uint32_t bar, uint32_t parity, uint32_t flag_addr,
                                              uint32_t* status, long long limit) {
    if constexpr (kDiag) {
        if (mbar_poll(bar, parity, limit)) return true;
        set_abort(flag_addr, status);
        return false;
    }
    if (mbar_try_wait(bar, parity)) return true;
    const long long t0 = clock64();
    while (!mbar_try_wait(bar, parity)) {
        if (aborted(flag_addr)) return false;
        if (clock64() - t0 > kWaitCycles) {
            set_abort(flag_addr, status);
            return false;
        }
    }
    return true;
}

template <bool kF8, int KT, bool kDiag, int DH, bool kSlots, int VAR>
__global__ void __launch_bounds__(kThreads, 1)
    prefill_kernel(const __grid_constant__ PrefillParams p, const __grid_constant__ CUtensorMap tmq,
                   const __grid_constant__ CUtensorMap tmk, const __grid_constant__ CUtensorMap tmv,
                   const __grid_constant__ CUtensorMap tmo) {
    // Nothing is read or written before the stream's earlier work is complete.
    constexpr bool kEarly = VAR != kVarPlain;  // launched programmatically
    if constexpr (kEarly) asm volatile("griddepcontrol.wait;" ::: "memory");
    constexpr bool k2 = KT == PAFP8_F16 || KT == PAFP8_BF16;  // 2-byte cache, same dtype as q
    constexpr bool kBF = KT == PAFP8_BF16;                    // bf16 MMA operands
    // A bf16 query on an fp8 cache is brought into f16 range (per row, by the
    // softmax warps) before the QK MMAs; every other path multiplies Q as loaded.
    // Under a window K is widened to bf16 for it instead, exactly too: a hundred
    // cycles a tile in the dequant warps, but no fit between two items, of which a
    // window makes many short ones.  (A prompt of 16384 tokens: window 300 150 us
    // against 160, 1024 299 and 305, 1536 399 and 400, 2048 498 and 494, 4000 835
    // and 816: the longest lose 2 % by it.  Block scales, whose
    // dequant warps have fewer registers, take 254 us so and 242 with the fit.)
    const bool wide_k = VAR == kVarWindow && !kF8 && !k2 && p.q_dtype == PAFP8_BF16;
    const bool fit_q = VAR != kVarWindow && !kF8 && !k2 && p.q_dtype == PAFP8_BF16;
    const bool bf_qk = kBF || wide_k;  // QK of bf16 operands
    using L = Layout<kF8, k2, DH, VAR>;
    using Dm = Dims<DH>;
    constexpr int NH = Dm::NH;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t base = (smem_addr(smem_raw) + 1023u) & ~1023u;
    auto bar = [&](int i) -> uint32_t { return base + L::bars + 8u * (uint32_t)i; };
    const uint32_t flag_addr = base + L::abort_flag;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int* meta = p.meta;
    const int n_items = meta[kMetaNumTiles];
    const int* items = meta + meta[kMetaOffTile];
    const int g = p.group, TQ = p.tile_tokens;

    if (threadIdx.x == 0) {
        mbar_init(bar(L::bQFull), 1);
        mbar_init(bar(L::bQReady), 256);
        mbar_init(bar(L::bQEmpty), 1);
        for (int i = 0; i < L::NKR; ++i) {
            mbar_init(bar(L::bKrFull + i), 1);
            mbar_init(bar(L::bKrEmpty + i), kF8 ? 1 : 128);
        }
        for (int i = 0; i < L::nVr; ++i) mbar_init(bar(L::bVrFull + i), 1);
        for (int i = 0; i < L::NVR; ++i) mbar_init(bar(L::bVrEmpty + i), 128);
        for (int i = 0; i < L::NK16; ++i) {
            mbar_init(bar(L::bK16Full + i), k2 ? 1 : 128);  // TMA, or the dequant warps
            mbar_init(bar(L::bK16Empty + i), 1);
        }
        for (int i = 0; i < L::NV16; ++i) {
            mbar_init(bar(L::bV16Full + i), 128);
            mbar_init(bar(L::bV16Empty + i), 1);
        }
        for (int x = 0; x < 2; ++x) {
            mbar_init(bar(L::bSFull + x), 1);
            mbar_init(bar(L::bPFull + x), 128);
            mbar_init(bar(L::bOFull + x), 1);
            mbar_init(bar(L::bOEmpty + x), 128);
            mbar_init(bar(L::bStageFree + x), 1);
            mbar_init(bar(L::bStageReady + x), 128);
        }
        mbar_init(bar(L::bDrain), 1);
        for (int i = 0; i < L::NSC; ++i) {
            mbar_init(bar(L::bScFull + i), kTileKeys / kPageSize);  // the lanes that hold the tile's scales
            mbar_init(bar(L::bScEmpty + i), 8);                     // the softmax warps
        }
        asm volatile("st.shared.u32 [%0], 0;" ::"r"(flag_addr) : "memory");
        mbar_init_fence();
    }
    if (warp == 13) tc_alloc(base + L::tmem_slot, kTmemCols);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    uint32_t tmem;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(tmem) : "r"(base + L::tmem_slot) : "memory");
    // Registers per thread: launched at 128; each warpgroup's branch below
    // starts by resizing: softmax 192, dequant 64, producer/MMA 64
    // (4 x 32 x (64 + 2 x 192 + 64) = 65,536, what the block launched with);
    // with block scales softmax 208, dequant 32, producer/MMA 64, the same sum.

    if (warp >= 12) {
      asm volatile("setmaxnreg.dec.sync.aligned.u32 64;" ::: "memory");
      if (warp == 12) {
        // ------------------------------------------------------------ producer
        if (lane == 0) {
            prefetch_tmap(&tmq);
            prefetch_tmap(&tmk);
            prefetch_tmap(&tmv);
        }
        Ring kr, vr;  // kr: raw K ring, or the 16-bit K ring for a 2-byte cache
        uint32_t qphase = 0;
        long long issued_k = 0, issued_v = 0, issued_q = 0;
        constexpr int nkr = k2 ? L::NK16 : L::NKR;
        constexpr int bkf = k2 ? L::bK16Full : L::bKrFull, bke = k2 ? L::bK16Empty : L::bKrEmpty;
        bool ok = true;
        for (int rnd = 0, t = blockIdx.x; t < n_items && ok; t = item_at(++rnd, blockIdx.x, gridDim.x)) {
            const Item it = load_item(items, t);
            const int q0 = it.qo0 + it.t0;
            const int kv_len = it.kv_len;
            // 16-token sub-pages of the request (a page of 16 * m tokens is m
            // of them).  The page entries of the next KV tile are loaded one
            // tile ahead and checked only when used, so the load's latency
            // stays hidden; the first tile's pass under the wait for the Q buffer
            // (window 300: 149.7 us without, 148.1 with).
            const int m = p.page_mult;
            const int npages = (kv_len + kPageSize - 1) / kPageSize;
            const int* idx = p.kv_indices + it.page0;
            int page_next = 0;
            {
                const int np0 = min(kTileKeys / kPageSize, npages), e = page_at<VAR>(p, it, lane);
                if (lane < np0) page_next = load_input<kEarly>(idx + (m == 1 ? e : e / m));
            }
            if (lane == 0) {
                ok = wait_or_abort<kDiag>(bar(L::bQEmpty), qphase ^ 1u, flag_addr, p.status, p.wait_cycles);
                if (ok) {
                    const uint32_t qb = bar(L::bQFull);
                    if (kF8) {
                        mbar_arrive_expect_tx(qb, (uint32_t)(2 * DH * g * TQ));
                        tma_load_3d(base + L::q, &tmq, qb, 0, it.hk * g, q0);
                        tma_load_3d(base + L::q + L::kQTile, &tmq, qb, 0, it.hk * g, q0 + TQ);
                    } else {
                        mbar_arrive_expect_tx(qb, (uint32_t)(4 * DH * g * TQ));
                        for (int x = 0; x < 2; ++x) {
                            const uint32_t dst = base + L::q + x * L::kQTile;
                            for (int h = 0; h < NH; ++h)
                                tma_load_3d(dst + h * kHalfTile, &tmq, qb, 64 * h, it.hk * g, q0 + x * TQ);
                        }
                    }
                    ++issued_q;
                }
            }
            ok = __shfl_sync(0xFFFFFFFFu, ok, 0);
            qphase ^= 1u;
            for (int j = 0; j < it.nkv && ok; ++j) {
                const int pg0 = j * (kTileKeys / kPageSize);
                const int np = min(kTileKeys / kPageSize, npages - pg0);
                int page = page_next;
                if (j + 1 < it.nkv) {
                    const int pg1 = pg0 + kTileKeys / kPageSize;
                    const int np1 = min(kTileKeys / kPageSize, npages - pg1);
                    const int e = page_at<VAR>(p, it, pg1 + lane);
                    page_next = lane < np1 ? load_input<kEarly>(idx + (m == 1 ? e : e / m)) : 0;
                }
                const bool bad = lane < np && (page < 0 || page >= p.num_pages);
                if (bad) page = 0;
                else if (kSlots) page = page * m + page_at<VAR>(p, it, pg0 + lane) % m;
                if (__any_sync(0xFFFFFFFFu, bad) && lane == 0) atomicOr(p.status, kStatusBounds);
                // Lane i < np holds the id of the tile's sub-page i (page * m + j
                // with kSlots; sub-page j of a page is the box at token slot 16 j
                // of that page) and issues its copies through load(slot, page).
                auto for_page = [&](auto&& load) {
                    if constexpr (kSlots) {
                        const int pg = page / m;
                        load((page - pg * m) * kPageSize, pg);
                    } else {
                        load(0, page);
                    }
                };
                // A 2-byte cache has two boxes per page (the 64-dim halves): lane
                // 8 h + i issues half h of page i, so 16 lanes share them.
                const int hpage = __shfl_sync(0xFFFFFFFFu, page, lane & 7);
                auto for_half_page = [&](auto&& load) {
                    if constexpr (kSlots) {
                        const int pg = hpage / m;
                        load((hpage - pg * m) * kPageSize, pg);
                    } else {
                        load(0, hpage);
                    }
                };
                const bool half_lane = (lane & 7) < np && (lane >> 3) < NH;
                // Lane 0 waits for the stage and posts the byte count; then lane
                // i issues page i's box, or lane 8 h + i half h of it for a
                // 2-byte cache (a thread needs about 100 cycles per TMA box, so
                // the pages go out from several lanes at once).
                if (lane == 0) {
                    ok = wait_or_abort<kDiag>(bar(bke + kr.idx), kr.phase ^ 1u, flag_addr, p.status, p.wait_cycles);
                    if (ok) mbar_arrive_expect_tx(bar(bkf + kr.idx), (uint32_t)np * kPageSize * DH * (k2 ? 2 : 1));
                }
                ok = __shfl_sync(0xFFFFFFFFu, ok, 0);
                if (!ok) break;
                if (k2) {
                    if (half_lane) {
                        // Each page as one box per 64-dim half into the halves of
                        // the 16-bit K tile: [half][key][128 B].
                        const uint32_t dst = base + L::k16 + kr.idx * Dm::kF16Tile;
                        const int h = lane >> 3, i = lane & 7;
                        for_half_page([&](int slot, int pg) {
                            tma_load_5d(dst + h * kHalfTile + i * 2048u, &tmk, bar(bkf + kr.idx), 0, h, slot, it.hk, pg);
                        });
                    }
                } else if (lane < np) {
                    const uint32_t dst = base + L::kr + kr.idx * Dm::kRawTile;
                    for_page([&](int slot, int pg) {
                        tma_load_4d(dst + lane * Dm::kRawPage, &tmk, bar(bkf + kr.idx), 0, it.hk, slot, pg);
                    });
                }
                ++issued_k;
                kr.next(nkr);
                if (lane == 0) {
                    ok = wait_or_abort<kDiag>(bar((k2 ? L::bV16Empty : L::bVrEmpty) + vr.idx), vr.phase ^ 1u, flag_addr,
                                              p.status, p.wait_cycles);
                    if (ok) mbar_arrive_expect_tx(bar(L::bVrFull + vr.idx), (uint32_t)np * kPageSize * DH * (k2 ? 2 : 1));
                }
                ok = __shfl_sync(0xFFFFFFFFu, ok, 0);
                if (!ok) break;
                if (k2) {
                    if (half_lane) {
                        const uint32_t dst = base + L::v16 + vr.idx * Dm::kF16Tile;
                        const int h = lane >> 3, i = lane & 7;
                        for_half_page([&](int slot, int pg) {
                            tma_load_5d(dst + h * kHalfTile + i * 2048u, &tmv, bar(L::bVrFull + vr.idx), 0, h, slot, it.hk,
                                        pg);
                        });
                    }
                } else if (lane < np) {
                    const uint32_t dst = base + L::vr + vr.idx * Dm::kRawTile;
                    for_page([&](int slot, int pg) {
                        tma_load_4d(dst + lane * Dm::kRawPage, &tmv, bar(L::bVrFull + vr.idx), 0, it.hk, slot, pg);
                    });
                }
                ++issued_v;
                vr.next(L::nVr);
            }
        }
        if (lane == 0) {
            // Let every copy issued by this CTA land before it may exit.
            if (issued_q > 0) mbar_wait(bar(L::bQFull), (uint32_t)((issued_q - 1) & 1));
            for (int s = 0; s < nkr && s < issued_k; ++s)
                mbar_wait(bar(bkf + s), (uint32_t)(((issued_k - 1 - s) / nkr) & 1));
            for (int s = 0; s < L::nVr && s < issued_v; ++s)
                mbar_wait(bar(L::bVrFull + s), (uint32_t)(((issued_v - 1 - s) / L::nVr) & 1));
        }
      } else if (warp == 13) {
        // ------------------------------------------------------------- MMA
        if (lane == 0) {
            const uint32_t idesc_qk =
                kF8 ? make_idesc(p.q_dtype == PAFP8_E5M2 ? 1 : 0, KT == PAFP8_E5M2 ? 1 : 0, 128, 128)
                    : make_idesc(bf_qk ? 1 : 0, bf_qk ? 1 : 0, 128, 128);
            const uint32_t idesc_pv = make_idesc_bmn(kBF ? 1 : 0, kBF ? 1 : 0, 128, DH);
            const int nk = kF8 ? L::NKR : L::NK16;
            const int kfull = kF8 ? L::bKrFull : L::bK16Full;
            const int kempty = kF8 ? L::bKrEmpty : L::bK16Empty;
            Ring kring, v16;
            uint32_t qphase = 0;
            uint32_t pphase[2] = {0, 0};
            int nonempty[2] = {0, 0};  // earlier items in which tile A / B had rows
            long long issued_any = 0;
            bool ok = true;
            // S_X = Q_X K^T for the K tile at the head of kring.
            auto qk = [&](int x) {
                const uint32_t dS = tmem + col_s(x);
                const uint32_t qa = base + L::q + x * L::kQTile;
                // The K steps' descriptor offsets are immediates inside one asm
                // statement (tc_mma_*_k*): start addresses are 16-byte units.
                if (kF8) {
                    // fp8 rows of DH bytes: 128- or 64-byte swizzle, 32 B per K step
                    const uint64_t dq = DH == 128 ? sw128_kmajor_desc(qa) : sw64_kmajor_desc(qa);
                    const uint32_t ka = base + L::kr + kring.idx * Dm::kRawTile;
                    const uint64_t dk = DH == 128 ? sw128_kmajor_desc(ka) : sw64_kmajor_desc(ka);
                    if constexpr (DH == 128) tc_mma_f8_ss_k4(dS, dq, dk, idesc_qk, 0u);
                    else tc_mma_f8_ss_k2(dS, dq, dk, idesc_qk, 0u);
                } else {
                    // 2-byte rows of DH elements: DH / 64 halves of 128 B, 32 B per K step
                    const uint64_t dq = sw128_kmajor_desc(qa);
                    const uint64_t dk = sw128_kmajor_desc(base + L::k16 + kring.idx * Dm::kF16Tile);
                    if constexpr (DH == 128) tc_mma_f16_ss_k8<kHalfTile, kHalfTile>(dS, dq, dk, idesc_qk, 0u);
                    else tc_mma_f16_ss_k4(dS, dq, dk, idesc_qk, 0u);
                }
                tc_commit(bar(L::bSFull + x));
                ++issued_any;
            };
            // O_X (+)= P_X V for the V tile at the head of the v16 ring.
            auto pv = [&](int x, bool accumulate) -> bool {
                // The first O_X write of an item waits for the epilogue of the
                // previous item that used O_X.
                if (!accumulate && nonempty[x] > 0 &&
                    !wait_or_abort<kDiag>(bar(L::bOEmpty + x), (uint32_t)((nonempty[x] - 1) & 1), flag_addr,
                                   p.status, p.wait_cycles))
                    return false;
                if (!wait_or_abort<kDiag>(bar(L::bPFull + x), pphase[x], flag_addr, p.status, p.wait_cycles)) return false;
                pphase[x] ^= 1u;
                tc_fence_after();
                // V [64-dim half][key][128 B] as the MN-major B operand: K = 128
                // keys in 8 steps of 16 rows, the dim halves kHalfTile apart.
                const uint64_t dv = sw128_mnmajor_desc(base + L::v16 + v16.idx * Dm::kF16Tile, kHalfTile);
                tc_mma_f16_ts_mn_k8(tmem + col_o<DH>(x), tmem + col_s(x), dv, idesc_pv, accumulate ? 1u : 0u);
                ++issued_any;
                return true;
            };
            for (int rnd = 0, t = blockIdx.x; t < n_items && ok; t = item_at(++rnd, blockIdx.x, gridDim.x)) {
                const Item it = load_item(items, t);
                const int qo_len = it.qo_len;
                const int kv_len = it.kv_len;
                const int nA = tile_nkv(it.t0, 0, TQ, qo_len, kv_len);
                const int nB = tile_nkv(it.t0, 1, TQ, qo_len, kv_len);
                const int n = it.nkv;
                ok = wait_or_abort<kDiag>(bar(fit_q ? L::bQReady : L::bQFull), qphase, flag_addr, p.status, p.wait_cycles);
                qphase ^= 1u;
                if (!ok) break;
                tc_fence_after();
                // K tile 0 for both query tiles.
                ok = wait_or_abort<kDiag>(bar(kfull + kring.idx), kring.phase, flag_addr, p.status, p.wait_cycles);
                if (!ok) break;
                tc_fence_after();
                if (nA > 0) qk(0);
                if (nB > 0) qk(1);
                tc_commit(bar(kempty + kring.idx));
                kring.next(nk);
                if (n == 1) tc_commit(bar(L::bQEmpty));
                for (int j = 0; j < n && ok; ++j) {
                    ok = wait_or_abort<kDiag>(bar(L::bV16Full + v16.idx), v16.phase, flag_addr, p.status, p.wait_cycles);
                    if (!ok) break;
                    tc_fence_after();
                    if (j < nA) {
                        if (!(ok = pv(0, j > 0))) break;
                        if (j == nA - 1) tc_commit(bar(L::bOFull + 0));
                    }
                    const bool more = j + 1 < n;
                    if (more) {
                        ok = wait_or_abort<kDiag>(bar(kfull + kring.idx), kring.phase, flag_addr, p.status, p.wait_cycles);
                        if (!ok) break;
                        tc_fence_after();
                        if (j + 1 < nA) qk(0);
                    }
                    if (j < nB) {
                        if (!(ok = pv(1, j > 0))) break;
                        if (j == nB - 1) tc_commit(bar(L::bOFull + 1));
                    }
                    tc_commit(bar(L::bV16Empty + v16.idx));
                    v16.next(L::NV16);
                    if (more) {
                        if (j + 1 < nB) qk(1);
                        tc_commit(bar(kempty + kring.idx));
                        kring.next(nk);
                        if (j + 1 == n - 1) tc_commit(bar(L::bQEmpty));
                    }
                }
                nonempty[0] += nA > 0;
                nonempty[1] += nB > 0;
            }
            // Drain: every MMA issued above completes before TMEM is freed.
            if (issued_any > 0) {
                tc_commit(bar(L::bDrain));
                mbar_wait(bar(L::bDrain), 0);
            }
        }
        __syncwarp();
      } else if (VAR == kVarBlocks && warp == 14) {
        // -------------------------------------------------- block scales
        // Lane 8 k + i looks up block i of tile j0 + k.
        const int k = lane >> 3, i = lane & 7, m = p.page_mult;
        uint32_t count = 0;  // tiles handed over so far
        bool ok = true;
        for (int rnd = 0, t = blockIdx.x; t < n_items && ok; t = item_at(++rnd, blockIdx.x, gridDim.x)) {
            const Item it = load_item(items, t);
            const int npages = (it.kv_len + kPageSize - 1) / kPageSize;
            const int* idx = p.kv_indices + it.page0;
            for (int j0 = 0; j0 < it.nkv && ok; j0 += 4) {
                const int j = j0 + k;
                float ks = 1.f, lv = 0.f, rv = 1.f;  // blocks past the request's end: all their keys are masked
                const int vp = j * (kTileKeys / kPageSize) + i;
                if (j < it.nkv && vp < npages) {
                    bool bad;  // (the producer reports it)
                    const SubPageAt at = sub_page<kEarly>(idx, page_at<VAR>(p, it, vp), m, p.num_pages, bad);
                    const size_t e = ((size_t)at.page * m + at.slot / kPageSize) * p.num_kv_heads + it.hk;
                    const float v = load_input<kEarly>(p.v_blocks + e);
                    ks = above_zero(p.sm_scale_log2 * load_input<kEarly>(p.k_blocks + e));
                    lv = __log2f(v);
                    rv = __frcp_rn(v);
                }
                const uint32_t tile = count + k, slot = tile % kScaleSlots;
                if (j < it.nkv) {
                    ok = wait_or_abort<kDiag>(bar(L::bScEmpty + slot), ((tile / kScaleSlots) & 1u) ^ 1u, flag_addr,
                                              p.status, p.wait_cycles);
                    if (ok) {
                        const uint32_t dst = base + L::scales + slot * kScaleTile;
                        sts64(dst + i * 8, __float_as_uint(ks), __float_as_uint(ks));
                        sts32(dst + 64 + i * 4, __float_as_uint(lv));
                        sts64(dst + 96 + i * 8, __float_as_uint(rv), __float_as_uint(rv));
                        mbar_arrive(bar(L::bScFull + slot));
                    }
                }
                ok = __all_sync(0xFFFFFFFFu, ok);
                count += min(4, it.nkv - j0);
            }
        }
      }
    } else if (warp < 4) {
        if constexpr (VAR == kVarBlocks) asm volatile("setmaxnreg.dec.sync.aligned.u32 32;" ::: "memory");
        else asm volatile("setmaxnreg.dec.sync.aligned.u32 64;" ::: "memory");
        // ---------------------------------------------------------- dequant
        const int wd = warp, q8 = lane >> 3, e = lane & 7;
        Ring kr, vr, k16, v16;
        bool ok = true;
        // A raw fp8 K or V tile [key][DH bytes] -> f16 [64-dim half][key][128 B]
        // under the 128-byte swizzle (the layout a 2-byte tile lands in), keys
        // `valid` and beyond zeroed.  K serves as the K-major B operand of Q K^T,
        // V as the MN-major B operand of P V.
        // (Under a window so are keys hide .. show - 1 of a V tile.)
        auto widen_as = [&](auto bf, uint32_t src, uint32_t dst, int valid, int hide, int show) {
            constexpr bool kToBf = decltype(bf)::value;
            // (Block scales leave 32 registers: K and V two rows at a time take 250
            // us in place of 237.)
            constexpr int kTurns = VAR == kVarBlocks && !kF8 ? 1 : 2;
            auto lo = [](uint32_t w) { return kToBf ? half2_to_bf162(fp8x2_lo<KT>(w)) : fp8x2_lo<KT>(w); };
            auto hi = [](uint32_t w) { return kToBf ? half2_to_bf162(fp8x2_hi<KT>(w)) : fp8x2_hi<KT>(w); };
            auto gone = [&](int row) { return row >= valid || (VAR != kVarPlain && row >= hide && row < show); };
            if constexpr (k2) {
                return;  // a 2-byte cache has no fp8 tile
            } else if constexpr (DH == 128) {
#pragma unroll kTurns
                for (int i = 0; i < 8; ++i) {
                    const int combo = wd * 8 + i;
                    const int row = (combo >> 1) * 8 + e;
                    const int c = (combo & 1) * 4 + q8;
                    uint4 w = lds128(src + row * 128 + ((c ^ e) << 4));
                    if (gone(row)) w = make_uint4(0u, 0u, 0u, 0u);
                    const uint32_t hb = dst + (c >> 2) * kHalfTile + row * 128;
                    sts128(hb + (((2 * q8) ^ e) << 4), lo(w.x), hi(w.x), lo(w.y), hi(w.y));
                    sts128(hb + (((2 * q8 + 1) ^ e) << 4), lo(w.z), hi(w.z), lo(w.w), hi(w.w));
                }
            } else {
                // 64-B fp8 rows under the 64-byte swizzle (16-byte chunk c of
                // row r at c ^ ((r >> 1) & 3)) -> one 128-B f16 half.
#pragma unroll kTurns
                for (int i = 0; i < 4; ++i) {
                    const int row = (wd * 4 + i) * 8 + e, c = q8;
                    uint4 w = lds128(src + row * 64 + ((c ^ ((row >> 1) & 3)) << 4));
                    if (gone(row)) w = make_uint4(0u, 0u, 0u, 0u);
                    const uint32_t hb = dst + row * 128;
                    sts128(hb + (((2 * c) ^ e) << 4), lo(w.x), hi(w.x), lo(w.y), hi(w.y));
                    sts128(hb + (((2 * c + 1) ^ e) << 4), lo(w.z), hi(w.z), lo(w.w), hi(w.w));
                }
            }
        };
        auto widen = [&](uint32_t src, uint32_t dst, int valid, int hide, int show) {
            widen_as(std::false_type{}, src, dst, valid, hide, show);
        };
        for (int rnd = 0, t = blockIdx.x; t < n_items && ok; t = item_at(++rnd, blockIdx.x, gridDim.x)) {
            const Item it = load_item(items, t);
            const int kv_len = it.kv_len;
            // No row of the item sees keys p.sinks .. first - 1.
            const int first = VAR != kVarPlain && p.window > 0 ? it.t0 + kv_len - it.qo_len - p.window + 1 : 0;
            for (int j = 0; j < it.nkv && ok; ++j) {
                const int key0 = j * kTileKeys;
                const int valid = min(kTileKeys, kv_len - key0);
                const int hide = VAR != kVarPlain ? p.sinks - key0 : 0, show = VAR != kVarPlain ? first - key0 : 0;
                if constexpr (!kF8 && !k2) {
                    ok = wait_or_abort<kDiag>(bar(L::bKrFull + kr.idx), kr.phase, flag_addr, p.status, p.wait_cycles) &&
                         wait_or_abort<kDiag>(bar(L::bK16Empty + k16.idx), k16.phase ^ 1u, flag_addr, p.status, p.wait_cycles);
                    if (!ok) break;
                    const uint32_t from = base + L::kr + kr.idx * Dm::kRawTile, to = base + L::k16 + k16.idx * Dm::kF16Tile;
                    if (wide_k) widen_as(std::true_type{}, from, to, kTileKeys, 0, 0);
                    else widen(from, to, kTileKeys, 0, 0);
                    fence_async_smem();
                    mbar_arrive(bar(L::bK16Full + k16.idx));
                    mbar_arrive(bar(L::bKrEmpty + kr.idx));
                    kr.next(L::NKR);
                    k16.next(L::NK16);
                }
                ok = wait_or_abort<kDiag>(bar(L::bVrFull + vr.idx), vr.phase, flag_addr, p.status, p.wait_cycles) &&
                     (k2 || wait_or_abort<kDiag>(bar(L::bV16Empty + v16.idx), v16.phase ^ 1u, flag_addr, p.status,
                                                 p.wait_cycles));
                if (!ok) break;
                const uint32_t dst = base + L::v16 + v16.idx * Dm::kF16Tile;
                if constexpr (k2) {
                    // A 2-byte V tile is where the MMA reads it: thread t zeroes key
                    // row t if no query row sees it.
                    const int row = (int)threadIdx.x;
                    if (row >= valid || (VAR != kVarPlain && row >= hide && row < show)) {
#pragma unroll
                        for (int c = 0; c < 8 * NH; ++c)
                            sts128(dst + (c >> 3) * kHalfTile + row * 128 + (c & 7) * 16, 0u, 0u, 0u, 0u);
                    }
                } else {
                    widen(base + L::vr + vr.idx * Dm::kRawTile, dst, valid, hide, show);
                }
                fence_async_smem();
                mbar_arrive(bar(L::bV16Full + v16.idx));
                if constexpr (!k2) mbar_arrive(bar(L::bVrEmpty + vr.idx));
                vr.next(L::nVr);
                v16.next(L::NV16);
            }
        }
    } else {
        if constexpr (VAR == kVarBlocks) asm volatile("setmaxnreg.inc.sync.aligned.u32 208;" ::: "memory");
        else asm volatile("setmaxnreg.inc.sync.aligned.u32 192;" ::: "memory");
        // ---------------------------------------------------------- softmax
        const int x = warp < 8 ? 0 : 1;        // query tile A or B
        const int r = threadIdx.x - 128 * (1 + x);  // row of the tile = TMEM lane
        const uint32_t lane_base = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
        const uint32_t tS = lane_base + col_s(x), tO = lane_base + col_o<DH>(x);
        uint32_t qphase = 0, sphase = 0, ophase = 0;
        [[maybe_unused]] uint32_t sc_count = 0;  // tiles of block scales read so far
        uint32_t stage_round = 0;  // staging rounds of this tile so far (fp8 query)
        const bool issuer = (threadIdx.x & 127) == 0;
        const bool o_32b = (reinterpret_cast<uintptr_t>(p.o) & 31u) == 0;  // rows are 256 B apart
        bool ok = true;
        // Range fit of this thread's Q row (bf16 query on an fp8 cache): wait
        // for the item's Q tiles, scale the row into f16 range by an exact power
        // of two, convert it in place and return the power (it multiplies the
        // logit scale).  Both warpgroups arrive on q_ready for every item.
        auto fit_row = [&]() -> float {
            float up = 1.f;
            ok = __all_sync(0xFFFFFFFFu, wait_or_abort<kDiag>(bar(L::bQFull), qphase, flag_addr, p.status, p.wait_cycles));
            qphase ^= 1u;
            if (!ok) return up;
            if (r < TQ * g) {
                // The row stays in registers between its maximum and its conversion
                // (209 us for the ragged prefill in place of 213); block scales read it
                // twice and compare word by word (held 252 us in place of 237, with
                // packed maxima 241: a faster fit is in the other query tile's way).
                constexpr bool kHold = VAR != kVarBlocks;
                constexpr int kTurns = kHold ? 8 * NH : 4;
                const uint32_t qrow = base + L::q + x * L::kQTile + r * 128;
                auto at = [&](int c) { return qrow + (c >> 3) * kHalfTile + (((c & 7) ^ (r & 7)) << 4); };
                uint4 held[kHold ? 8 * NH : 1];
                [[maybe_unused]] uint32_t top[4] = {};  // pairs of bf16 magnitudes (a NaN beside a number does not count)
                uint32_t mx = 0;
#pragma unroll
                for (int c = 0; c < 8 * NH; ++c) {
                    const uint4 w = lds128(at(c));
                    if constexpr (kHold) held[c] = w;
                    const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        if constexpr (kHold) {
                            top[k] = max_abs_bf162(top[k], ws[k]);
                        } else {
                            mx = max(mx, (ws[k] & 0x7FFFu) << 16);
                            mx = max(mx, ws[k] & 0x7FFF0000u);
                        }
                    }
                }
                if constexpr (kHold) {
                    top[0] = max_abs_bf162(max_abs_bf162(top[0], top[1]), max_abs_bf162(top[2], top[3]));
                    mx = max(top[0] << 16, top[0] & 0xFFFF0000u);
                }
                const int ex = (int)((mx >> 23) & 0xFF) - 127;
                const int shift = ex > 14 ? ex - 14 : 0;
                const float down = __int_as_float((127 - shift) << 23);
                up = __int_as_float((127 + shift) << 23);
#pragma unroll kTurns
                for (int c = 0; c < 8 * NH; ++c) {
                    uint4 w;
                    if constexpr (kHold) w = held[c];
                    else w = lds128(at(c));
                    const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
                    uint32_t o4[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        o4[k] = pack_half2(__uint_as_float(ws[k] << 16) * down,
                                           __uint_as_float(ws[k] & 0xFFFF0000u) * down);
                    sts128(at(c), o4[0], o4[1], o4[2], o4[3]);
                }
                fence_async_smem();
            }
            mbar_arrive(bar(L::bQReady));
            return up;
        };
        // The next item's Q is fitted right after this item's last softmax pass
        // and before its epilogue, so the next item's first QK does not wait
        // for the epilogues.
        float up_next = 1.f;
        if (fit_q && (int)blockIdx.x < n_items) up_next = fit_row();
        Item it_next = (int)blockIdx.x < n_items ? load_item(items, blockIdx.x) : Item{};
        for (int rnd = 0, t = blockIdx.x; t < n_items && ok; t = item_at(++rnd, blockIdx.x, gridDim.x)) {
            const Item it = it_next;
            const int qo0 = it.qo0;
            const int qo_len = it.qo_len;
            const int kv_len = it.kv_len;
            const int t0 = it.t0 + x * TQ;
            const int nX = tile_nkv(it.t0, x, TQ, qo_len, kv_len);
            const int tok = r / g, hh = r - tok * g;
            const bool valid_row = (tok < TQ) && (t0 + tok < qo_len);
            const int limit = valid_row ? t0 + tok + kv_len - qo_len : -1;
            // Keys p.sinks .. low - 1 lie before the row's window.
            const int low = VAR != kVarPlain && p.window > 0 ? limit - p.window + 1 : 0;
            float scale = (VAR == kVarBlocks ? 1.f : p.sm_scale_log2) * up_next;
            float vsc = p.v_scale;
            if (VAR != kVarBlocks && p.k_scales != nullptr) {  // per-head scale tensors
                const int qh = it.hk * g + min(hh, g - 1);
                scale = fold_scale_log2(p.sm_scale, p.q_scales != nullptr ? load_input<kEarly>(p.q_scales + qh) : 1.0f,
                                        load_input<kEarly>(p.k_scales + it.hk)) *
                        up_next;
                vsc = load_input<kEarly>(p.v_scales + it.hk);
            }
            float m = -INFINITY, l = 0.f;  // m in scaled (log2) units
            for (int j = 0; j < nX && ok; ++j) {
                // Block scales: here already, so read before the wait for S.
                const uint32_t sc_tile = base + L::scales + (sc_count % kScaleSlots) * kScaleTile;
                f32x2 kf2[8];  // per block: K scale with the softmax scale
                float lv[8];   // log2 of the V scale
                if constexpr (VAR == kVarBlocks) {
                    ok = __all_sync(0xFFFFFFFFu, wait_or_abort<kDiag>(bar(L::bScFull + sc_count % kScaleSlots),
                                                                      (sc_count / kScaleSlots) & 1u, flag_addr, p.status,
                                                                      p.wait_cycles));
                    if (!ok) break;
                    const f32x2 row2 = make_f32x2(scale, scale);
#pragma unroll
                    for (int c = 0; c < 8; c += 2) {
                        const uint4 w = lds128(sc_tile + 8 * c);
                        kf2[c] = mul2(make_f32x2(__uint_as_float(w.x), __uint_as_float(w.y)), row2);
                        kf2[c + 1] = mul2(make_f32x2(__uint_as_float(w.z), __uint_as_float(w.w)), row2);
                    }
#pragma unroll
                    for (int c = 0; c < 8; c += 4) {
                        const uint4 w = lds128(sc_tile + 64 + 4 * c);
                        lv[c] = __uint_as_float(w.x), lv[c + 1] = __uint_as_float(w.y);
                        lv[c + 2] = __uint_as_float(w.z), lv[c + 3] = __uint_as_float(w.w);
                    }
                }
                ok = __all_sync(0xFFFFFFFFu, wait_or_abort<kDiag>(bar(L::bSFull + x), sphase, flag_addr, p.status, p.wait_cycles));
                sphase ^= 1u;
                if (!ok) break;
                tc_fence_after();
                const int key0 = j * kTileKeys;
                const bool below = VAR != kVarPlain && key0 < low && key0 + kTileKeys > p.sinks;
                const bool need_mask = key0 + kTileKeys - 1 > limit || below;
                // The whole S row (128 columns) in registers, one wait.
                uint32_t v[128];
#pragma unroll
                for (int c = 0; c < 4; ++c) tc_ld32(tS + 32 * c, *reinterpret_cast<uint32_t(*)[32]>(v + 32 * c));
                tc_wait_ld();
                // row max of the raw logits (scale > 0); masked logits -> -inf.
                // Eight independent partial maxima keep the chain short.
                if (need_mask) {
                    const int lim = limit - key0;
#pragma unroll
                    for (int i = 0; i < 128; ++i)
                        if (i > lim) v[i] = __float_as_uint(-INFINITY);
                    if (below) {
                        const int hide = p.sinks - key0, show = low - key0;
#pragma unroll
                        for (int i = 0; i < 128; ++i)
                            if (i >= hide && i < show) v[i] = __float_as_uint(-INFINITY);
                    }
                }
                float m_new;
                if constexpr (VAR == kVarBlocks) {
                    // Each block's maximum, then that of s + log2 of its V scale.
                    m_new = m;
#pragma unroll
                    for (int c = 0; c < 8; ++c) {
                        float a = __uint_as_float(v[16 * c]), b = __uint_as_float(v[16 * c + 1]);
#pragma unroll
                        for (int i = 2; i < 16; i += 4) {
                            a = max3(a, __uint_as_float(v[16 * c + i]), __uint_as_float(v[16 * c + i + 1]));
                            if (i + 2 < 16) b = max3(b, __uint_as_float(v[16 * c + i + 2]), __uint_as_float(v[16 * c + i + 3]));
                        }
                        float kf, again;
                        split_f32x2(kf2[c], kf, again);
                        m_new = fmaxf(m_new, fmaf(fmaxf(a, b), kf, lv[c]));
                    }
                } else {
                    // Four independent three-input maxima keep the chain short.
                    float pm[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) pm[k] = __uint_as_float(v[k]);
#pragma unroll
                    for (int i = 4; i < 128; i += 2)
                        pm[(i >> 1) & 3] = max3(pm[(i >> 1) & 3], __uint_as_float(v[i]), __uint_as_float(v[i + 1]));
                    const float mx = fmaxf(max3(pm[0], pm[1], pm[2]), pm[3]);
                    m_new = fmaxf(m, mx * scale);
                }
                float m_use = m;
                bool rescale = false;
                if (j == 0) {
                    m_use = m_new;
                } else if (m_new > m + 8.0f) {
                    m_use = m_new;
                    rescale = true;
                }
                // A row with no admissible key so far: without a window it never
                // gets one, under a window its maximum stays at -inf.
                const float m_keep = m_use;
                if (m_use == -INFINITY) m_use = 0.f;
                // tcgen05.ld/st are warp-collective: the whole warp rescales
                // when any of its rows must (alpha = 1 for the others).
                if (__any_sync(0xFFFFFFFFu, rescale)) {
                    // O_X += P V of the previous KV tile has completed (in-order
                    // tensor pipe, S of this tile was written after it).
                    const float alpha = rescale ? ex2(m - m_use) : 1.f;
                    const f32x2 alpha2 = make_f32x2(alpha, alpha);
                    l *= alpha;
#pragma unroll 1
                    for (int c = 0; c < DH / 32; ++c) {
                        uint32_t v[32];
                        tc_ld32(tO + 32 * c, v);
                        tc_wait_ld();
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            float a, b;
                            split_f32x2(mul2(make_f32x2(__uint_as_float(v[2 * i]), __uint_as_float(v[2 * i + 1])),
                                             alpha2),
                                        a, b);
                            v[2 * i] = __float_as_uint(a);
                            v[2 * i + 1] = __float_as_uint(b);
                        }
                        tc_st32(tO + 32 * c, v);
                    }
                    tc_wait_st();
                }
                // P = exp2(s * scale - m) (masked logits are -inf: P = 0), row
                // sum, P -> TMEM as f16 over the first half of S.  Pairs of
                // columns go through the packed fp32 pipe.
                [[maybe_unused]] const f32x2 scale2 = make_f32x2(scale, scale), negm2 = make_f32x2(-m_use, -m_use);
                // P overwrites the S values it consumed: P of columns 2i, 2i+1
                // goes to v[i], which held column i (already used).  Two
                // independent packed partial sums keep the chain short.
                if constexpr (VAR == kVarBlocks) {
                    f32x2 l2 = make_f32x2(l, 0.f);
                    uint4 rv;  // 1 / V scale of two blocks, twice each
#pragma unroll
                    for (int c = 0; c < 8; ++c) {
                        if (c % 2 == 0) rv = lds128(sc_tile + 96 + 8 * c);
                        const float off = lv[c] - m_use;
                        const f32x2 off2 = make_f32x2(off, off);
                        f32x2 ps = make_f32x2(0.f, 0.f);
#pragma unroll
                        for (int i = 8 * c; i < 8 * c + 8; ++i) {
                            float a, b;
                            split_f32x2(fma2(make_f32x2(__uint_as_float(v[2 * i]), __uint_as_float(v[2 * i + 1])), kf2[c],
                                             off2),
                                        a, b);
                            const float e0 = ex2(a), e1 = ex2(b);
                            ps = i == 8 * c ? make_f32x2(e0, e1) : add2(ps, make_f32x2(e0, e1));
                            v[i] = pack_half2(e0, e1);
                        }
                        l2 = fma2(ps, c % 2 ? make_f32x2(__uint_as_float(rv.z), __uint_as_float(rv.w))
                                            : make_f32x2(__uint_as_float(rv.x), __uint_as_float(rv.y)),
                                  l2);
                    }
                    {
                        float a, b;
                        split_f32x2(l2, a, b);
                        l = a + b;
                    }
                    // The tile's scales are read: one arrival a warp.
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar(L::bScEmpty + sc_count % kScaleSlots));
                    ++sc_count;
                } else {
                    // (P takes V's type, since a product's operands have one: over a bf16
                    // cache 8 bits, half a step 2^-8 in place of f16's 2^-11, and an output
                    // error of 0.0023 where f16 gives 0.0017; the sum is of the fp32 values.)
                    f32x2 ps[2] = {make_f32x2(0.f, 0.f), make_f32x2(0.f, 0.f)};
#pragma unroll
                    for (int i = 0; i < 64; ++i) {
                        float a, b;
                        split_f32x2(fma2(make_f32x2(__uint_as_float(v[2 * i]), __uint_as_float(v[2 * i + 1])), scale2,
                                         negm2),
                                    a, b);
                        const float e0 = ex2(a), e1 = ex2(b);
                        const f32x2 e = make_f32x2(e0, e1);
                        ps[i & 1] = add2(ps[i & 1], e);
                        v[i] = kBF ? pack_bf162(e0, e1) : pack_half2(e0, e1);
                    }
                    {
                        float a, b, c, d;
                        split_f32x2(ps[0], a, b);
                        split_f32x2(ps[1], c, d);
                        l += (a + b) + (c + d);
                    }
                }
                tc_st32(tS, *reinterpret_cast<uint32_t(*)[32]>(v));
                tc_st32(tS + 32, *reinterpret_cast<uint32_t(*)[32]>(v + 32));
                tc_wait_st();
                tc_fence_before();
                mbar_arrive(bar(L::bPFull + x));
                m = VAR != kVarPlain ? m_keep : m_use;
            }
            if (!ok) break;
            if constexpr (VAR == kVarBlocks) {
                // Tiles that only the other query tile reads: their scales are
                // waited for all the same, so that no warp's arrivals run ahead.
                for (int j = nX; j < it.nkv && ok; ++j, ++sc_count) {
                    ok = __all_sync(0xFFFFFFFFu, wait_or_abort<kDiag>(bar(L::bScFull + sc_count % kScaleSlots),
                                                                      (sc_count / kScaleSlots) & 1u, flag_addr, p.status,
                                                                      p.wait_cycles));
                    if (ok && lane == 0) mbar_arrive(bar(L::bScEmpty + sc_count % kScaleSlots));
                }
                if (!ok) break;
            }
            // The next item's record, loaded here so that its latency passes
            // during the epilogue rather than before the next item's first pass.
            {
                const int tn = item_at(rnd + 1, blockIdx.x, gridDim.x);
                if (tn < n_items) it_next = load_item(items, tn);
            }
            if (fit_q && item_at(rnd + 1, blockIdx.x, gridDim.x) < n_items) {
                up_next = fit_row();
                if (!ok) break;
            }
            if (nX == 0) continue;  // tile B past the request's last row
            // epilogue: the tile's last O update must have completed.
            ok = __all_sync(0xFFFFFFFFu, wait_or_abort<kDiag>(bar(L::bOFull + x), ophase, flag_addr, p.status, p.wait_cycles));
            ophase ^= 1u;
            if (!ok) break;
            tc_fence_after();
            const float inv = valid_row && l > 0.f ? vsc / l : 0.f;
            const size_t orow = (size_t)(qo0 + t0 + tok) * p.num_qo_heads + (size_t)it.hk * g + hh;
            if (kF8 && t0 + TQ <= qo_len) {
                // A full tile: two rounds of 64 dims through this tile's staging
                // half, each written out by one bulk tensor store (asynchronous;
                // the next round waits until the store has read the staging).
                const uint32_t stg = base + L::ostage + (uint32_t)x * kHalfTile;
                bool sok = true;
#pragma unroll 1
                for (int h = 0; h < NH && sok; ++h, ++stage_round) {
                    uint32_t v[64];
                    tc_ld32(tO + 64 * h, *reinterpret_cast<uint32_t(*)[32]>(v));
                    tc_ld32(tO + 64 * h + 32, *reinterpret_cast<uint32_t(*)[32]>(v + 32));
                    tc_wait_ld();
                    if (h == NH - 1) {
                        // O_X is read: release it to the next item's first PV.
                        tc_fence_before();
                        mbar_arrive(bar(L::bOEmpty + x));
                    }
                    uint32_t w[32];
                    const f32x2 inv2 = make_f32x2(inv, inv);
#pragma unroll
                    for (int i = 0; i < 32; ++i) {
                        float a0, a1;
                        split_f32x2(mul2(make_f32x2(__uint_as_float(v[2 * i]), __uint_as_float(v[2 * i + 1])), inv2),
                                    a0, a1);
                        w[i] = pack_out2(a0, a1, p.o_dtype);
                    }
                    if (issuer) {
                        bulk_wait_read_all();
                        mbar_arrive(bar(L::bStageFree + x));
                    }
                    sok = __all_sync(0xFFFFFFFFu, wait_or_abort<kDiag>(bar(L::bStageFree + x), stage_round & 1u, flag_addr,
                                                                p.status, p.wait_cycles));
                    if (!sok) break;
#pragma unroll
                    for (int c = 0; c < 8; ++c)
                        sts128(stg + r * 128 + ((c ^ (r & 7)) << 4), w[4 * c], w[4 * c + 1], w[4 * c + 2], w[4 * c + 3]);
                    fence_async_smem();
                    mbar_arrive(bar(L::bStageReady + x));
                    if (issuer) {
                        sok = wait_or_abort<kDiag>(bar(L::bStageReady + x), stage_round & 1u, flag_addr, p.status, p.wait_cycles);
                        if (sok) {
                            tma_store_3d(&tmo, stg, 64 * h, it.hk * g, qo0 + t0);
                            bulk_commit();
                        }
                    }
                    sok = __all_sync(0xFFFFFFFFu, sok);
                }
                ok = sok;
                if (!ok) break;
                if (valid_row && p.lse != nullptr) p.lse[orow] = (m + __log2f(l)) * 0.69314718055994531f;
                continue;
            }
#pragma unroll 1
            for (int c = 0; c < DH / 32; ++c) {
                uint32_t v[32];
                tc_ld32(tO + 32 * c, v);
                tc_wait_ld();
                if (valid_row) {
                    uint32_t w[16];
                    const f32x2 inv2 = make_f32x2(inv, inv);
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        float a, b;
                        split_f32x2(mul2(make_f32x2(__uint_as_float(v[2 * i]), __uint_as_float(v[2 * i + 1])), inv2),
                                    a, b);
                        w[i] = pack_out2(a, b, p.o_dtype);
                    }
                    uint16_t* dst = static_cast<uint16_t*>(p.o) + orow * DH + 32 * c;
                    if (o_32b) {
                        // 32-byte stores: every access fills whole sectors.
                        stg256(dst, w);
                        stg256(dst + 16, w + 8);
                    } else {
                        uint4* d4 = reinterpret_cast<uint4*>(dst);
#pragma unroll
                        for (int i = 0; i < 4; ++i) d4[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
                    }
                }
            }
            if (valid_row && p.lse != nullptr) p.lse[orow] = (m + __log2f(l)) * 0.69314718055994531f;
            tc_fence_before();
            mbar_arrive(bar(L::bOEmpty + x));
        }
    }

    if (kF8 && (warp == 4 || warp == 8) && lane == 0) bulk_wait_all();  // this thread's output stores
    tc_fence_before();
    __syncthreads();
    if (warp == 13) {
        tc_fence_after();
        tc_dealloc(tmem, kTmemCols);
    }
}

template <bool kF8, int KT, bool kDiag, int DH, bool kSlots, int VAR>
cudaError_t launch_t(const PrefillParams& p, const CUtensorMap& tq, const CUtensorMap& tk,
                     const CUtensorMap& tv, const CUtensorMap& to, int num_ctas, cudaStream_t stream) {
    const size_t smem = 1024 + Layout<kF8, KT == PAFP8_F16 || KT == PAFP8_BF16, DH, VAR>::bytes;
    auto kern = prefill_kernel<kF8, KT, kDiag, DH, kSlots, VAR>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    if constexpr (VAR == kVarPlain) {
        kern<<<num_ctas, kThreads, smem, stream>>>(p, tq, tk, tv, to);
        return cudaGetLastError();
    } else {
        // The variants wait for the stream's work before them in the kernel
        // rather than before the launch, which then passes under that work.
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(num_ctas);
        cfg.blockDim = dim3(kThreads);
        cfg.dynamicSmemBytes = smem;
        cfg.stream = stream;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        return cudaLaunchKernelEx(&cfg, kern, p, tq, tk, tv, to);
    }
}

// The diagnostic instantiation runs only under a shortened wait bound (and
// takes any page size); pages of 16 tokens and of 16 m tokens have one each,
// but for the variants, which take any page size too.
template <bool kF8, int KT, int DH, int VAR>
cudaError_t launch_one(const PrefillParams& p, const CUtensorMap& tq, const CUtensorMap& tk,
                       const CUtensorMap& tv, const CUtensorMap& to, int num_ctas, cudaStream_t stream) {
    if (p.wait_cycles < kWaitCyclesDefault)
        return launch_t<kF8, KT, true, DH, true, VAR>(p, tq, tk, tv, to, num_ctas, stream);
    if constexpr (VAR == kVarPlain)
        if (p.page_mult == 1) return launch_t<kF8, KT, false, DH, false, VAR>(p, tq, tk, tv, to, num_ctas, stream);
    return launch_t<kF8, KT, false, DH, true, VAR>(p, tq, tk, tv, to, num_ctas, stream);
}

// Dispatch on the query and cache dtypes for head size DH (block scales go
// with an fp8 cache only; a 2-byte one of head size 128 runs on pairs, but for
// short windows).
template <int DH, int VAR = kVarPlain>
cudaError_t launch_prefill_head(const PrefillParams& p, const CUtensorMap& tmap_q, const CUtensorMap& tmap_k,
                                const CUtensorMap& tmap_v, const CUtensorMap& tmap_o, int num_ctas,
                                cudaStream_t stream) {
    const bool f8 = p.q_dtype == PAFP8_E4M3FN || p.q_dtype == PAFP8_E5M2;
    if (f8)
        return p.kv_dtype == PAFP8_E4M3FN
                   ? launch_one<true, PAFP8_E4M3FN, DH, VAR>(p, tmap_q, tmap_k, tmap_v, tmap_o, num_ctas, stream)
                   : launch_one<true, PAFP8_E5M2, DH, VAR>(p, tmap_q, tmap_k, tmap_v, tmap_o, num_ctas, stream);
    if (p.kv_dtype == PAFP8_E4M3FN)
        return launch_one<false, PAFP8_E4M3FN, DH, VAR>(p, tmap_q, tmap_k, tmap_v, tmap_o, num_ctas, stream);
    if (p.kv_dtype == PAFP8_E5M2)
        return launch_one<false, PAFP8_E5M2, DH, VAR>(p, tmap_q, tmap_k, tmap_v, tmap_o, num_ctas, stream);
    if constexpr (VAR == kVarWindow || (VAR == kVarPlain && DH == 64)) {
        if (p.kv_dtype == PAFP8_F16)
            return launch_one<false, PAFP8_F16, DH, VAR>(p, tmap_q, tmap_k, tmap_v, tmap_o, num_ctas, stream);
        if (p.kv_dtype == PAFP8_BF16)
            return launch_one<false, PAFP8_BF16, DH, VAR>(p, tmap_q, tmap_k, tmap_v, tmap_o, num_ctas, stream);
    }
    return cudaErrorInvalidValue;
}

}  // namespace
}  // namespace pafp8
