// tree.cuh -- attention of a tree of drafted tokens over the paged KV cache on
// the tcgen05 tensor cores (sm_103a).  Included by one translation unit per
// head size (tree_d128.cu, tree_d64.cu).
//
// What it computes: request b has T new (drafted) tokens, whose keys are the
// last T of its L cached ones.  Drafted token u sees every key j < L - T and
// key L - T + w where bit w of its mask row is set.  For query head h of KV
// head h / group: o = v_scale * softmax(sm_scale * q_scale * k_scale * q.k) V
// over the keys it sees, lse = ln sum exp(logits); a row that sees no key
// gives o = 0, lse = -inf.
//
// What bounds it: with R = T * group rows per KV head a key costs 2 D bytes
// (fp8) from HBM and 4 D R flops, so up to R of about 128 the cache's bytes
// bound it, and the tensor and softmax work per byte has to stay below that.
// Widening an fp8 tile to 16 bits in shared memory would cost more shared
// memory traffic than reading it once from HBM does, so nothing is widened:
//   * S = Q K^T takes K as it landed (kind::f8f6f4).  A 2-byte query row is
//     scaled by a power of two to a maximum in [128, 256) and split into
//     e4m3 pieces (4 significant bits each: two for bf16's 8, three for f16's
//     11) whose products accumulate in one accumulator: x = a + b (+ c), each
//     piece the e4m3 rounding of what the earlier ones left, exact but for
//     elements below 2^-10 of the row's largest, which lose 2^-18 of it at
//     most.
//   * O += P V takes V as it landed, the MN-major B operand, and P as e4m3
//     pieces from TMEM: P' = 2^7 p in [0, 256), hi = e4m3(P'),
//     lo = e4m3(32 (P' - hi)), in two accumulators O_hi and O_lo (O = O_hi +
//     O_lo / 32), so that P carries 8 significant bits (a bf16's worth, 2^-9
//     off) down to p = 2^-16 and never less than 2^-23 of the row's largest
//     off.  An f16 output adds a third piece, e4m3 of what lo left,
//     accumulated with lo: 12 bits.
//   * A 2-byte cache of the query's dtype runs kind::f16 on Q, K and V as
//     they are, P rounded to that type.
//
// Work: the plan lays the 128-key tiles of all (request, row tile of 128 /
// group tokens) lines end to end, cuts them into equal ranges, and gives each
// range to a group of CTAs, one a KV head, so that the CTAs that read the
// heads of one token-major page run side by side.  A range's part of a line
// is a segment; a segment that is not its whole line writes a partial state,
// and a merge kernel (a programmatic dependent) joins them.
//
// An MMA has 128 rows whatever R is.  When a row tile has at most 64 or 32
// rows, the 128 lanes hold 2 or 4 copies of them, copy c taking the softmax of
// its share of each tile's keys (its P is zero elsewhere, its maximum, sum and
// accumulators its own), and the epilogue joins the copies like split-KV
// states: the softmax work per tile, which would otherwise fall on R lanes,
// stays spread over all threads.
//
// Roles (512 threads):
//   warps 0-7   softmax: lane r of TMEM is owned by threads r (first half of
//               the row's columns) and r + 128 (second half); the halves agree
//               on the maximum through shared memory;
//   warps 8-11  helpers: build the next segment's Q pieces, then the finished
//               segment's epilogue;
//   warps 12, 14, 15  TMA producers;  warp 13  MMA issuer and TMEM owner.
// TMEM columns: S / P buffers 0-127 and 128-255 (tile parity), O_hi from 256,
// O_lo from 256 + D.  MMA order: QK(j + 1) before PV(j), across segments, so
// the softmax of a tile overlaps the tensor work of its neighbours.
// All waits are bounded; on expiry a status bit is set and the CTA winds down.
#pragma once
#include "../../include/pafp8.h"
#include "internal.h"
#include "ptx.cuh"

namespace pafp8 {
namespace {

using namespace ptx;

constexpr int kTreeThreads = 512;
constexpr uint32_t kColO = 256;
constexpr int kMaxStages = 8;
// O is rescaled when a row's maximum rises by more than 2^kHead; P' is at most
// 2^(kShift + kHead).
template <int KT>
struct PShift {  // fp8 pieces: P' < 2^8, e4m3 reaches 448
    static constexpr float kShift = 7.f, kHead = 1.f;
};
template <>
struct PShift<PAFP8_BF16> {
    static constexpr float kShift = 0.f, kHead = 8.f;
};
template <>
struct PShift<PAFP8_F16> {
    static constexpr float kShift = 0.f, kHead = 8.f;
};

// Shared memory: [Q buffers][K stages][V stages][staging][state rings][barriers].
struct TreeSmem {
    uint32_t q, k, v, stage, ml, fac, xmax, bars, tmem_slot, abort_flag, bytes;
};
constexpr int kStageRow = 36;  // floats: 32 dims of a row, 16-byte aligned, 8 rows on distinct banks
enum TreeBar : int {
    tQFull = 0,                  // [2]
    tQEmpty = 2,                 // [2]
    tInfo = 4,                   // [2] row factors of a segment written
    tState = 6,                  // [2] m and l of a segment written
    tSFull = 8,                  // [2]
    tPFull = 10,                 // [2]
    tOFull = 12, tOEmpty = 13,
    tXmax = 14,                  // [4] quadrants
    tStage = 18,                 // helpers' staging
    tDrain = 19,
    tKFull = 20,
    tKEmpty = tKFull + kMaxStages,
    tVFull = tKEmpty + kMaxStages,
    tVEmpty = tVFull + kMaxStages,
    tNumBars = tVEmpty + kMaxStages
};
__host__ __device__ inline TreeSmem tree_smem(uint32_t q_bytes, uint32_t tile_bytes, int stages) {
    TreeSmem s{};
    s.q = 0;
    s.k = q_bytes;
    s.v = s.k + (uint32_t)stages * tile_bytes;
    s.stage = s.v + (uint32_t)stages * tile_bytes;
    s.ml = s.stage + 128 * kStageRow * 4;          // [2][3][128] floats: m, l of either half
    s.fac = s.ml + 2 * 3 * 128 * 4;                // [2][128] floats
    s.xmax = s.fac + 2 * 128 * 4;                  // [2][2][128] floats
    s.bars = s.xmax + 2 * 2 * 128 * 4;
    s.tmem_slot = s.bars + 8 * tNumBars;
    s.abort_flag = s.tmem_slot + 4;
    s.bytes = s.abort_flag + 4;
    return s;
}

__device__ __forceinline__ float lds_f(uint32_t a) {
    float v;
    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ float4 lds_f4(uint32_t a) {
    float4 v;
    asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ void sts_f(uint32_t a, float v) { asm volatile("st.shared.f32 [%0], %1;" ::"r"(a), "f"(v) : "memory"); }

__device__ __forceinline__ void tree_abort(uint32_t flag, uint32_t* status) {
    asm volatile("st.shared.u32 [%0], 1;" ::"r"(flag) : "memory");
    atomicOr(status, kStatusTimeout);
}
// Bounded wait that gives up once another role has; a bound below the default
// polls without suspending (try_wait could outlast it).
__device__ __forceinline__ bool tree_wait(uint32_t bar, uint32_t parity, uint32_t flag, uint32_t* status, long long limit) {
    const bool shortened = limit < kWaitCyclesDefault;
    if (shortened ? mbar_test_wait(bar, parity) : mbar_try_wait(bar, parity)) return true;
    const long long t0 = clock64();
    while (!(shortened ? mbar_test_wait(bar, parity) : mbar_try_wait(bar, parity))) {
        uint32_t v;
        asm volatile("ld.volatile.shared.u32 %0, [%1];" : "=r"(v) : "r"(flag) : "memory");
        if (v != 0) return false;
        if (clock64() - t0 > limit) {
            tree_abort(flag, status);
            return false;
        }
    }
    return true;
}

// One segment: key tiles [tile0, tile1) of a line (request, KV head, row tile).
struct Seg {
    int hk, t0, tile0, tile1, slot;  // slot: partial state, or -1 for a whole line
    int qo0, qo_len, kv_len, page0;
};
__device__ __forceinline__ Seg load_seg(const int* segs, int i) {
    const int4* r = reinterpret_cast<const int4*>(segs + kTreeSegWords * (long long)i);
    const int4 a = __ldg(r), b = __ldg(r + 1), c = __ldg(r + 2);
    return Seg{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w, c.x};
}
// log2 of the copies a row tile of `rows` rows is held in.
__device__ __forceinline__ int copies_log2(int rows) { return rows <= 32 ? 2 : rows <= 64 ? 1 : 0; }

// 32 bits of mask row `row` from bit u0 on (bits below 0: keys of the context,
// seen; bits from T on: none).
__device__ __forceinline__ uint32_t mask_word(const uint32_t* row, int w, int words, int T) {
    if (w < 0) return 0xFFFFFFFFu;
    if (w >= words || 32 * w >= T) return 0;
    const uint32_t x = __ldg(row + w);
    const int n = T - 32 * w;
    return n >= 32 ? x : x & ((1u << n) - 1u);
}
__device__ __forceinline__ uint32_t mask_bits(const uint32_t* row, int u0, int words, int T) {
    const int w = u0 >> 5, s = u0 & 31;  // floor division: w may be negative
    const uint32_t lo = mask_word(row, w, words, T);
    return s == 0 ? lo : __funnelshift_r(lo, mask_word(row, w + 1, words, T), s);
}

__device__ __forceinline__ uint32_t e4m3_pair(float lo, float hi) {
    unsigned short d;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(d) : "f"(hi), "f"(lo));
    return d;
}
__device__ __forceinline__ float2 e4m3_back(uint32_t pair) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((unsigned short)pair));
    return __half22float2(*reinterpret_cast<__half2*>(&h));
}

template <int NC>
__device__ __forceinline__ void ld_cols(uint32_t t, uint32_t (&v)[NC]) {
    if constexpr (NC == 16) {
        tc_ld16(t, v);
    } else {
#pragma unroll
        for (int c = 0; c < NC / 32; ++c) tc_ld32(t + 32 * c, *reinterpret_cast<uint32_t(*)[32]>(v + 32 * c));
    }
}
template <int N>
__device__ __forceinline__ void st_cols(uint32_t t, const uint32_t (&v)[N]) {
    if constexpr (N == 4) tc_st4(t, v);
    if constexpr (N == 8) tc_st8(t, v);
    if constexpr (N == 16) tc_st16(t, v);
    if constexpr (N == 32) tc_st32(t, v);
}

// What a softmax thread keeps of its row over a segment.
struct RowState {
    float m, l;  // running maximum (log2 units), sum of P' over this thread's columns
};

struct TileArgs {
    uint32_t tS, tO;          // this warp's S / P buffer and O_hi, lane base added
    uint32_t xmax, xbar;      // exchange slots [half][128] and barrier of this tile
    uint32_t xphase;
    uint32_t prev_bar, prev_phase;  // completes when the previous tile's PV has
    uint32_t pbar;
    uint32_t flag;
    uint32_t* status;
    long long limit;
    const uint32_t* mrow;     // mask row
    int words, T, u0;         // u0: mask bit of this thread's first column (negative: context)
    int r, half, copy;
    bool first;               // first tile of the segment
    float scale;
};

// One tile's softmax on NC columns of this thread's row: maximum, rescale of O
// when it rose, P pieces into TMEM.  Warp-collective; false when a wait gave up.
template <int KT, int NP, int DH, int NC>
__device__ __forceinline__ bool softmax_tile(RowState& st, const TileArgs& a) {
    constexpr bool k2 = KT == PAFP8_BF16 || KT == PAFP8_F16;
    constexpr int C = 64 / NC;  // copies
    constexpr float kShift = PShift<KT>::kShift, kHead = PShift<KT>::kHead;
    const int col0 = a.copy * (128 / C) + a.half * NC;
    uint32_t v[NC];
    ld_cols<NC>(a.tS + col0, v);
    tc_wait_ld();
    if (a.u0 + NC > 0) {  // some of these keys are drafted tokens (or lie behind the last)
#pragma unroll
        for (int c = 0; c < NC; c += 32) {
            const uint32_t bits = mask_bits(a.mrow, a.u0 + c, a.words, a.T);
#pragma unroll
            for (int i = 0; i < 32 && c + i < NC; ++i)
                if (!((bits >> i) & 1u)) v[c + i] = 0xFF800000u;  // -inf
        }
    }
    float pm[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) pm[k] = __uint_as_float(v[k]);
#pragma unroll
    for (int i = 4; i < NC; i += 2)
        pm[(i >> 1) & 3] = max3(pm[(i >> 1) & 3], __uint_as_float(v[i]), __uint_as_float(v[i + 1]));
    float mx = fmaxf(max3(pm[0], pm[1], pm[2]), pm[3]);
    sts_f(a.xmax + 4u * (128 * a.half + a.r), mx);
    warp_arrive(a.xbar);
    if (!__all_sync(0xFFFFFFFFu, tree_wait(a.xbar, a.xphase, a.flag, a.status, a.limit))) return false;
    mx = fmaxf(mx, lds_f(a.xmax + 4u * (128 * (a.half ^ 1) + a.r)));
    const float m_new = fmaxf(st.m, mx * a.scale);
    float m_use = st.m;
    bool rescale = false;
    if (a.first) {
        m_use = m_new;
    } else if (m_new > st.m + kHead) {
        m_use = m_new;
        rescale = true;
    }
    if (__any_sync(0xFFFFFFFFu, rescale)) {
        // Every O update of the earlier tiles has to be complete.
        if (!__all_sync(0xFFFFFFFFu, tree_wait(a.prev_bar, a.prev_phase, a.flag, a.status, a.limit))) return false;
        tc_fence_after();
        const float alpha = rescale ? ex2(st.m - m_use) : 1.f;
        const f32x2 alpha2 = make_f32x2(alpha, alpha);
        st.l *= alpha;
        // The two threads of a row take half of its O columns each.
        constexpr int kCols = k2 ? DH / 2 : DH;
#pragma unroll 1
        for (int c = 0; c < kCols / 32; ++c) {
            uint32_t o[32];
            const uint32_t at = a.tO + a.half * kCols + 32 * c;
            tc_ld32(at, o);
            tc_wait_ld();
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                float x, y;
                split_f32x2(mul2(make_f32x2(__uint_as_float(o[2 * i]), __uint_as_float(o[2 * i + 1])), alpha2), x, y);
                o[2 * i] = __float_as_uint(x);
                o[2 * i + 1] = __float_as_uint(y);
            }
            tc_st32(at, o);
        }
        tc_wait_st();
    }
    st.m = m_use;
    // A row that has seen no key yet keeps m = -inf; its P is exp2(-inf) = 0.
    const float neg = m_use == -INFINITY ? 0.f : kShift - m_use;
    const f32x2 scale2 = make_f32x2(a.scale, a.scale), neg2 = make_f32x2(neg, neg);
    f32x2 ps[2] = {make_f32x2(0.f, 0.f), make_f32x2(0.f, 0.f)};
    constexpr int W = NC / (k2 ? 2 : 4);  // words of one P piece
    uint32_t p0[W], p1[k2 ? 1 : W], p2[NP == 3 ? W : 1];
#pragma unroll
    for (int i = 0; i < NC / 2; ++i) {
        float x, y;
        split_f32x2(fma2(make_f32x2(__uint_as_float(v[2 * i]), __uint_as_float(v[2 * i + 1])), scale2, neg2), x, y);
        const f32x2 e = make_f32x2(ex2(x), ex2(y));
        ps[i & 1] = add2(ps[i & 1], e);
        split_f32x2(e, x, y);
        if constexpr (KT == PAFP8_BF16) {
            p0[i] = pack_bf162(x, y);
        } else if constexpr (KT == PAFP8_F16) {
            p0[i] = pack_half2(x, y);
        } else {
            const uint32_t hi = e4m3_pair(x, y);
            const float2 hb = e4m3_back(hi);
            const f32x2 rest = mul2(fma2(make_f32x2(hb.x, hb.y), make_f32x2(-1.f, -1.f), e), make_f32x2(32.f, 32.f));
            split_f32x2(rest, x, y);
            const uint32_t lo = e4m3_pair(x, y);
            uint32_t lo2 = 0;
            if constexpr (NP == 3) {
                const float2 lb = e4m3_back(lo);
                split_f32x2(fma2(make_f32x2(lb.x, lb.y), make_f32x2(-1.f, -1.f), rest), x, y);
                lo2 = e4m3_pair(x, y);
            }
            if (i & 1) {
                p0[i >> 1] = prmt(p0[i >> 1], hi, 0x5410u);
                p1[i >> 1] = prmt(p1[i >> 1], lo, 0x5410u);
                if constexpr (NP == 3) p2[i >> 1] = prmt(p2[i >> 1], lo2, 0x5410u);
            } else {
                p0[i >> 1] = hi;
                p1[i >> 1] = lo;
                if constexpr (NP == 3) p2[i >> 1] = lo2;
            }
        }
    }
    {
        float x, y, z, w;
        split_f32x2(ps[0], x, y);
        split_f32x2(ps[1], z, w);
        st.l += (x + y) + (z + w);
    }
    // P over S (both halves have read it): piece i in 32 (fp8) or 64 columns
    // from 32 i on; the other copies' keys have P = 0.
    constexpr int kPer = (k2 ? 64 : 32) / C;  // columns of one copy
    uint32_t zero[W];
#pragma unroll
    for (int i = 0; i < W; ++i) zero[i] = 0;
#pragma unroll
    for (int c = 0; c < C; ++c) {
        const uint32_t at = a.tS + c * kPer + a.half * W;
        const bool mine = c == a.copy;
        if (C == 1 || mine) {
            st_cols<W>(at, p0);
            if constexpr (!k2) st_cols<W>(at + 32, p1);
            if constexpr (NP == 3) st_cols<W>(at + 64, p2);
        } else {
            st_cols<W>(at, zero);
            if constexpr (!k2) st_cols<W>(at + 32, zero);
            if constexpr (NP == 3) st_cols<W>(at + 64, zero);
        }
    }
    tc_wait_st();
    tc_fence_before();
    return true;
}

template <int KT, int NP, int DH>
__global__ void __launch_bounds__(kTreeThreads, 1)
    tree_kernel(const __grid_constant__ TreeParams p, const __grid_constant__ CUtensorMap tmk,
                const __grid_constant__ CUtensorMap tmv) {
    constexpr bool k2 = KT == PAFP8_BF16 || KT == PAFP8_F16;
    constexpr int ES = k2 ? 2 : 1;
    constexpr uint32_t kTile = kTileKeys * DH * ES;   // one K, V or Q-piece tile
    constexpr uint32_t kHalf = kTileKeys * 128;       // a 64-dim half of a 2-byte tile
    constexpr int NH = DH / 64;                       // halves of a 2-byte row
    extern __shared__ uint8_t smem_raw[];
    const uint32_t base = (smem_addr(smem_raw) + 1023u) & ~1023u;
    const TreeSmem L = tree_smem((uint32_t)(p.q_buffers * p.q_pieces) * kTile, kTile, p.stages);
    auto bar = [&](int i) -> uint32_t { return base + L.bars + 8u * (uint32_t)i; };
    const uint32_t flag = base + L.abort_flag;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int NS = p.stages, NQB = p.q_buffers;
    const int* meta = p.meta;
    const int s_begin = __ldg(meta + meta[kMetaOffCtaSeg] + blockIdx.x);
    const int s_end = __ldg(meta + meta[kMetaOffCtaSeg] + blockIdx.x + 1);
    const int* segs = meta + meta[kMetaOffSeg];
    const int g = p.group, TQ = kTileRows / g;
    auto wait = [&](int b, uint32_t parity) { return tree_wait(bar(b), parity, flag, p.status, p.wait_cycles); };
    auto wait_all = [&](int b, uint32_t parity) { return (bool)__all_sync(0xFFFFFFFFu, wait(b, parity)); };

    if (threadIdx.x == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(bar(tQFull + i), 4);   // helper warps
            mbar_init(bar(tQEmpty + i), 1);  // commit
            mbar_init(bar(tInfo + i), 4);
            mbar_init(bar(tState + i), 8);   // softmax warps
            mbar_init(bar(tSFull + i), 1);
            mbar_init(bar(tPFull + i), 8);
        }
        mbar_init(bar(tOFull), 1);
        mbar_init(bar(tOEmpty), 4);
        for (int i = 0; i < 4; ++i) mbar_init(bar(tXmax + i), 2);
        mbar_init(bar(tStage), 4);
        mbar_init(bar(tDrain), 1);
        for (int i = 0; i < NS; ++i) {
            mbar_init(bar(tKFull + i), 3);  // producer warps
            mbar_init(bar(tKEmpty + i), 1);
            mbar_init(bar(tVFull + i), 3);
            mbar_init(bar(tVEmpty + i), 1);
        }
        asm volatile("st.shared.u32 [%0], 0;" ::"r"(flag) : "memory");
        mbar_init_fence();
    }
    if (warp == 13) tc_alloc(base + L.tmem_slot, 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    uint32_t tmem;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(tmem) : "r"(base + L.tmem_slot) : "memory");

    if (warp == 12 || warp >= 14) {
        // ----------------------------------------------------------- producers
        // A box holds the 16 tokens of one (sub-)page, and a warp's box takes it
        // about 130 cycles to issue, 16 boxes a tile 2100: more than the tile's
        // time at full bandwidth (1400).  So three warps share the boxes, every
        // third one each, and each warp expects its own bytes.
        const int pw = warp == 12 ? 0 : warp - 13;
        if (lane == 0) {
            prefetch_tmap(&tmk);
            prefetch_tmap(&tmv);
        }
        constexpr int kBoxes = 8 * (k2 ? NH : 1);      // boxes of a K or V tile: (half, sub-page)
        const int box = 3 * lane + pw, i8 = box & 7;   // this lane's box
        constexpr uint32_t kBoxBytes = k2 ? 2048u : (uint32_t)(kPageSize * DH);
        long long n = 0;  // tiles issued
        int stage = 0;
        uint32_t phase = 0;
        bool ok = true, k_only = false;
        for (int si = s_begin; si < s_end && ok; ++si) {
            const Seg sg = load_seg(segs, si);
            const int m = p.page_mult;
            const int nsub = (sg.kv_len + kPageSize - 1) / kPageSize;  // 16-token sub-pages of the request
            const int* idx = p.kv_indices + sg.page0;
            auto fetch = [&](int tile) -> int {  // the page entry of this lane's sub-page
                const int v = tile * (kTileKeys / kPageSize) + i8;
                return v < nsub ? __ldg(idx + (m == 1 ? v : v / m)) : 0;
            };
            int next = fetch(sg.tile0);
            for (int t = sg.tile0; t < sg.tile1 && ok; ++t) {
                int page = next;
                if (t + 1 < sg.tile1) next = fetch(t + 1);
                const int sub = t * (kTileKeys / kPageSize) + i8;
                const bool mine = box < kBoxes && sub < nsub;
                const bool bad = mine && (page < 0 || page >= p.num_pages);
                if (bad) {
                    page = 0;
                    atomicOr(p.status, kStatusBounds);
                }
                const int slot = m == 1 ? 0 : (sub % m) * kPageSize;
                const uint32_t bytes = (uint32_t)__popc(__ballot_sync(0xFFFFFFFFu, mine)) * kBoxBytes;
                for (int kv = 0; kv < 2; ++kv) {
                    const int full = (kv ? tVFull : tKFull) + stage, empty = (kv ? tVEmpty : tKEmpty) + stage;
                    if (lane == 0) {
                        ok = wait(empty, phase ^ 1u);
                        if (ok) mbar_arrive_expect_tx(bar(full), bytes);
                    }
                    ok = __shfl_sync(0xFFFFFFFFu, ok, 0);
                    if (!ok) {
                        k_only = kv == 1;
                        break;
                    }
                    const CUtensorMap* map = kv ? &tmv : &tmk;
                    const uint32_t dst = base + (kv ? L.v : L.k) + (uint32_t)stage * kTile + (uint32_t)box * kBoxBytes;
                    if (mine) {
                        if constexpr (k2)
                            tma_load_5d(dst, map, bar(full), 0, box >> 3, slot, sg.hk, page);
                        else
                            tma_load_4d(dst, map, bar(full), 0, sg.hk, slot, page);
                    }
                    __syncwarp();
                }
                if (!ok) break;
                ++n;
                if (++stage == NS) {
                    stage = 0;
                    phase ^= 1u;
                }
            }
        }
        if (lane == 0) {
            // Every copy lands before the CTA may exit.
            const long long nk = n + (k_only ? 1 : 0);
            for (int s = 0; s < NS; ++s) {
                if (s < nk) mbar_wait(bar(tKFull + s), (uint32_t)(((nk - 1 - s) / NS) & 1));
                if (s < n) mbar_wait(bar(tVFull + s), (uint32_t)(((n - 1 - s) / NS) & 1));
            }
        }
        __syncwarp();
    } else if (warp == 13) {
        // ----------------------------------------------------------------- MMA
        if (lane == 0 && s_begin < s_end) {
            const int kvf = k2 ? (KT == PAFP8_BF16 ? 1 : 0) : (p.kv_dtype == PAFP8_E5M2 ? 1 : 0);
            const int qf = k2 ? kvf : (p.q_dtype == PAFP8_E5M2 ? 1 : 0);
            const uint32_t idesc_qk = make_idesc(qf, kvf, 128, 128);
            const uint32_t idesc_pv = make_idesc_bmn(k2 ? kvf : 0, kvf, 128, DH);
            bool ok = true, issued = false;
            // QK cursor: segment qs, tile qt, tile count qn so far; PV cursor alike.
            int qs = s_begin, qn = 0;
            int kstage = 0, vstage = 0;
            uint32_t kphase = 0, vphase = 0;
            Seg qg = load_seg(segs, qs);
            int qt = qg.tile0;
            auto qk = [&]() -> bool {
                const int nth = qs - s_begin, buf = NQB == 2 ? nth & 1 : 0;
                if (qt == qg.tile0) {
                    if (!wait(tQFull + buf, (uint32_t)((NQB == 2 ? nth >> 1 : nth) & 1))) return false;
                }
                if (!wait(tKFull + kstage, kphase)) return false;
                tc_fence_after();
                const uint32_t d = tmem + 128u * (qn & 1);
                const uint32_t qa = base + L.q + (uint32_t)(buf * p.q_pieces) * kTile;
                const uint32_t ka = base + L.k + (uint32_t)kstage * kTile;
                if constexpr (k2) {
                    const uint64_t dq = sw128_kmajor_desc(qa), dk = sw128_kmajor_desc(ka);
                    if constexpr (DH == 128)
                        tc_mma_f16_ss_k8<kHalf, kHalf>(d, dq, dk, idesc_qk, 0u);
                    else
                        tc_mma_f16_ss_k4(d, dq, dk, idesc_qk, 0u);
                } else {
                    for (int i = 0; i < p.q_pieces; ++i) {
                        if constexpr (DH == 128)
                            tc_mma_f8_ss_k4(d, sw128_kmajor_desc(qa + i * kTile), sw128_kmajor_desc(ka), idesc_qk, i > 0);
                        else
                            tc_mma_f8_ss_k2(d, sw64_kmajor_desc(qa + i * kTile), sw64_kmajor_desc(ka), idesc_qk, i > 0);
                    }
                }
                issued = true;
                tc_commit(bar(tSFull + (qn & 1)));
                tc_commit(bar(tKEmpty + kstage));
                if (++kstage == NS) {
                    kstage = 0;
                    kphase ^= 1u;
                }
                ++qn;
                if (++qt == qg.tile1) {
                    tc_commit(bar(tQEmpty + buf));
                    if (++qs < s_end) {
                        qg = load_seg(segs, qs);
                        qt = qg.tile0;
                    }
                }
                return true;
            };
            ok = qk();
            int pn = 0;
            for (int ps = s_begin; ps < s_end && ok; ++ps) {
                const Seg pg = load_seg(segs, ps);
                for (int t = pg.tile0; t < pg.tile1; ++t, ++pn) {
                    if (qs < s_end && !(ok = qk())) break;
                    // O of the segment before has been read by its epilogue.
                    if (t == pg.tile0 && ps > s_begin && !(ok = wait(tOEmpty, (uint32_t)((ps - s_begin - 1) & 1)))) break;
                    if (!(ok = wait(tVFull + vstage, vphase))) break;
                    if (!(ok = wait(tPFull + (pn & 1), (uint32_t)((pn >> 1) & 1)))) break;
                    tc_fence_after();
                    const uint32_t acc = t > pg.tile0 ? 1u : 0u;
                    const uint32_t pa = tmem + 128u * (pn & 1);
                    const uint32_t va = base + L.v + (uint32_t)vstage * kTile;
                    if constexpr (k2) {
                        tc_mma_f16_ts_mn_k8(tmem + kColO, pa, sw128_mnmajor_desc(va, DH == 128 ? kHalf : 16u), idesc_pv, acc);
                    } else {
                        const uint64_t dv = DH == 128 ? sw128_mnmajor_desc(va, 16u) : sw64_mnmajor_desc(va);
                        tc_mma_f8_ts_mn_k4<DH>(tmem + kColO, pa, dv, idesc_pv, acc);
                        tc_mma_f8_ts_mn_k4<DH>(tmem + kColO + DH, pa + 32, dv, idesc_pv, acc);
                        if constexpr (NP == 3) tc_mma_f8_ts_mn_k4<DH>(tmem + kColO + DH, pa + 64, dv, idesc_pv, 1u);
                    }
                    tc_commit(bar(tVEmpty + vstage));
                    if (t + 1 == pg.tile1) tc_commit(bar(tOFull));
                    if (++vstage == NS) {
                        vstage = 0;
                        vphase ^= 1u;
                    }
                }
            }
            if (issued) {  // every MMA completes before TMEM is freed
                tc_commit(bar(tDrain));
                mbar_wait(bar(tDrain), 0);
            }
        }
        __syncwarp();
    } else if (warp < 8) {
        // ------------------------------------------------------------- softmax
        const int quad = warp & 3, half = warp >> 2;
        const int r = 32 * quad + lane;
        const uint32_t lane_base = tmem + ((uint32_t)(32 * quad) << 16);
        const uint32_t tO = lane_base + kColO;
        int j = 0;  // tiles so far
        int stage = 0;
        uint32_t sphase = 0;  // phase of V stage `stage`
        bool ok = true;
        for (int si = s_begin; si < s_end && ok; ++si) {
            const Seg sg = load_seg(segs, si);
            const int nth = si - s_begin;
            const int ntok = min(TQ, sg.qo_len - sg.t0), rows = ntok * g;
            const int cl = copies_log2(rows);
            const int rp = 128 >> cl, row = r & (rp - 1), copy = r >> (7 - cl);
            const int tok = min(row / g, ntok - 1);
            const int ctx = sg.kv_len - sg.qo_len;
            const uint32_t* mrow = p.tree_mask + (long long)(sg.qo0 + sg.t0 + tok) * p.mask_words;
            if (!(ok = wait_all(tInfo + (nth & 1), (uint32_t)((nth >> 1) & 1)))) break;
            float scale = p.sm_scale_log2;
            if (p.k_scales != nullptr) {
                const int qh = sg.hk * g + row % g;
                scale = fold_scale_log2(p.sm_scale, p.q_scales != nullptr ? __ldg(p.q_scales + qh) : 1.0f,
                                        __ldg(p.k_scales + sg.hk));
            }
            scale *= lds_f(base + L.fac + 4u * (128 * (nth & 1) + r));
            RowState st{-INFINITY, 0.f};
            for (int t = sg.tile0; t < sg.tile1; ++t, ++j) {
                if (!(ok = wait_all(tSFull + (j & 1), (uint32_t)((j >> 1) & 1)))) break;
                tc_fence_after();
                TileArgs a;
                a.tS = lane_base + 128u * (j & 1);
                a.tO = tO;
                a.xmax = base + L.xmax + 1024u * (j & 1);
                a.xbar = bar(tXmax + quad);
                a.xphase = (uint32_t)(j & 1);
                a.prev_bar = bar(tVEmpty + (stage == 0 ? NS - 1 : stage - 1));
                a.prev_phase = stage == 0 ? sphase ^ 1u : sphase;
                a.flag = flag;
                a.status = p.status;
                a.limit = p.wait_cycles;
                a.mrow = mrow;
                a.words = p.mask_words;
                a.T = sg.qo_len;
                a.u0 = t * kTileKeys + copy * rp + half * (rp >> 1) - ctx;
                a.r = r;
                a.half = half;
                a.copy = copy;
                a.first = t == sg.tile0;
                a.scale = scale;
                if (cl == 0)
                    ok = softmax_tile<KT, NP, DH, 64>(st, a);
                else if (cl == 1)
                    ok = softmax_tile<KT, NP, DH, 32>(st, a);
                else
                    ok = softmax_tile<KT, NP, DH, 16>(st, a);
                if (!ok) break;
                // Key rows behind the request's end (the tail of its last page and
                // rows no page filled) hold anything: zero them, P = 0 there must
                // not meet a NaN.
                const int valid = sg.kv_len - t * kTileKeys;
                if (valid < kTileKeys) {
                    if (!(ok = wait_all(tVFull + stage, sphase))) break;
                    if (half == 0 && r >= valid) {
                        const uint32_t vrow = base + L.v + (uint32_t)stage * kTile + (uint32_t)r * (k2 ? 128u : (uint32_t)DH);
#pragma unroll
                        for (int c = 0; c < (k2 ? 8 : DH / 16); ++c) {
                            sts128(vrow + 16u * c, 0u, 0u, 0u, 0u);
                            if (k2 && NH == 2) sts128(vrow + kHalf + 16u * c, 0u, 0u, 0u, 0u);
                        }
                    }
                    fence_async_smem();
                }
                warp_arrive(bar(tPFull + (j & 1)));
                if (++stage == NS) {
                    stage = 0;
                    sphase ^= 1u;
                }
            }
            if (!ok) break;
            const uint32_t ml = base + L.ml + 1536u * (nth & 1);
            if (half == 0) sts_f(ml + 4u * r, st.m);
            sts_f(ml + 512u * (1 + half) + 4u * r, st.l);
            warp_arrive(bar(tState + (nth & 1)));
        }
    } else if (warp < 12) {
        // ------------------------------------------------- Q pieces, epilogues
        const int r = threadIdx.x - 256;
        const uint32_t tO = tmem + ((uint32_t)(32 * (warp & 3)) << 16) + kColO;
        uint32_t stage_phase = 0;
        bool ok = true;
        // Segment si's Q rows into its buffer: DH / 8 lanes a row, eight elements
        // a lane, each row stored to all its copies.  A compact loop: unrolled
        // over whole rows the code ran once a segment and spent 10 us on
        // instruction fetches.
        auto build_q = [&](int si) -> bool {
            const Seg sg = load_seg(segs, si);
            const int nth = si - s_begin, buf = NQB == 2 ? nth & 1 : 0;
            const int use = NQB == 2 ? nth >> 1 : nth;  // earlier uses of this buffer
            const int rows = min(TQ, sg.qo_len - sg.t0) * g;
            const int cl = copies_log2(rows), rp = 128 >> cl;
            constexpr int LPR = DH / 8, RPI = 32 / LPR;  // lanes a row, rows a warp's round
            const int e = lane % LPR, row0 = (warp - 8) * RPI + lane / LPR;
            const bool q1 = !k2 && p.q_pieces == 1;      // an fp8 query as it is
            const size_t head0 = (size_t)(sg.qo0 + sg.t0) * p.num_qo_heads + (size_t)sg.hk * g;
            const uint32_t dst = base + L.q + (uint32_t)(buf * p.q_pieces) * kTile;
            const uint32_t fdst = base + L.fac + 512u * (nth & 1);
            constexpr int kBatch = 4;  // rows in flight per lane group
            bool ready = false;
#pragma unroll 1
            for (int first = row0; first - row0 < rp; first += 4 * RPI * kBatch) {
                uint4 raw[kBatch];
#pragma unroll
                for (int k = 0; k < kBatch; ++k) {
                    const int row = first + 4 * RPI * k;
                    raw[k] = make_uint4(0, 0, 0, 0);
                    if (row < rows) {
                        const int tok = row / g;
                        const size_t at = (head0 + (size_t)tok * p.num_qo_heads + (row - tok * g)) * DH + 8 * e;
                        if (q1) {
                            const uint2 x = __ldg(reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(p.q) + at));
                            raw[k] = make_uint4(x.x, x.y, 0, 0);
                        } else {
                            raw[k] = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.q) + at));
                        }
                    }
                }
                if (!ready) {  // the buffer is free once its last segment's QK has run
                    if (!wait_all(tQEmpty + buf, (uint32_t)((use + 1) & 1))) return false;
                    ready = true;
                }
#pragma unroll 1
                for (int k = 0; k < kBatch; ++k) {
                    const int row = first + 4 * RPI * k;
                    if (row - lane / LPR >= rp) break;  // uniform: rp is a multiple of a round's rows
                    const uint4 rw = k == 0 ? raw[0] : k == 1 ? raw[1] : k == 2 ? raw[2] : raw[3];
                    if constexpr (k2) {
                        for (int c = 0; c < 1 << cl; ++c) {
                            const int r2 = row + c * rp;
                            sts128(dst + (e >> 3) * kHalf + r2 * 128u + (uint32_t)(((e & 7) ^ (r2 & 7)) << 4), rw.x, rw.y, rw.z,
                                   rw.w);
                            if (e == 0) sts_f(fdst + 4u * r2, 1.f);
                        }
                        continue;
                    }
                    // An eight-byte element group's place in a piece's tile row.
                    const uint32_t at = DH == 128 ? row * 128u + (uint32_t)(((e >> 1) ^ (row & 7)) << 4) + 8u * (e & 1)
                                                  : row * 64u + (uint32_t)(((e >> 1) ^ ((row >> 1) & 3)) << 4) + 8u * (e & 1);
                    const uint32_t copy_bytes = (uint32_t)rp * DH;
                    float fac = 1.f;
                    if (q1) {
                        for (int c = 0; c < 1 << cl; ++c) sts64(dst + at + c * copy_bytes, rw.x, rw.y);
                    } else {
                        const bool bf = p.q_dtype == PAFP8_BF16;
                        const uint32_t w[4] = {rw.x, rw.y, rw.z, rw.w};
                        uint32_t top = 0;  // the row's largest magnitude as a 16-bit pattern
#pragma unroll
                        for (int i = 0; i < 4; ++i) top = max(top, max(w[i] & 0x7FFFu, (w[i] >> 16) & 0x7FFFu));
#pragma unroll
                        for (int d = LPR / 2; d > 0; d >>= 1) top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, d));
                        const float amax = bf ? __uint_as_float(top << 16) : __half2float(__ushort_as_half((unsigned short)top));
                        // 2^ex brings the largest magnitude into [128, 256).  A row with an
                        // infinity or a NaN gives NaN, as its logits would.
                        const int up = 7 - ((int)((__float_as_uint(amax) >> 23) & 0xFFu) - 127);
                        const int ex = amax == 0.f ? 0 : max(-120, min(100, up));
                        const float mul = __uint_as_float((uint32_t)(127 + ex) << 23);
                        fac = isfinite(amax) ? __uint_as_float((uint32_t)(127 - ex) << 23) : __uint_as_float(0x7FC00000u);
                        float x[8];
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            if (bf) {
                                x[2 * i] = __uint_as_float(w[i] << 16) * mul;
                                x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u) * mul;
                            } else {
                                const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
                                x[2 * i] = f.x * mul;
                                x[2 * i + 1] = f.y * mul;
                            }
                        }
#pragma unroll 1
                        for (int pc = 0; pc < p.q_pieces; ++pc) {
                            uint32_t pr[4];
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                pr[i] = e4m3_pair(x[2 * i], x[2 * i + 1]);
                                const float2 b = e4m3_back(pr[i]);
                                x[2 * i] -= b.x;
                                x[2 * i + 1] -= b.y;
                            }
                            for (int c = 0; c < 1 << cl; ++c)
                                sts64(dst + pc * kTile + at + c * copy_bytes, pr[0] | (pr[1] << 16), pr[2] | (pr[3] << 16));
                        }
                    }
                    if (e == 0)
                        for (int c = 0; c < 1 << cl; ++c) sts_f(fdst + 4u * (row + c * rp), fac);
                }
            }
            fence_async_smem();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(bar(tQFull + buf));
                mbar_arrive(bar(tInfo + (nth & 1)));
            }
            return true;
        };
        if (s_begin < s_end) ok = build_q(s_begin);
        for (int si = s_begin; si < s_end && ok; ++si) {
            if (si + 1 < s_end && !(ok = build_q(si + 1))) break;
            const Seg sg = load_seg(segs, si);
            const int nth = si - s_begin;
            const int rows = min(TQ, sg.qo_len - sg.t0) * g;
            const int cl = copies_log2(rows), rp = 128 >> cl, C = 1 << cl;
            const float vsc = p.v_scales != nullptr ? __ldg(p.v_scales + sg.hk) : p.v_scale;
            if (!(ok = wait_all(tState + (nth & 1), (uint32_t)((nth >> 1) & 1)))) break;
            const uint32_t ml = base + L.ml + 1536u * (nth & 1);
            auto state_m = [&](int x) { return lds_f(ml + 4u * x); };
            auto state_l = [&](int x) { return lds_f(ml + 512u + 4u * x) + lds_f(ml + 1024u + 4u * x); };
            // Row `row` over its copies: the largest maximum M, the sum L at M.
            auto joined = [&](int row, float& M, float& Lsum) {
                M = state_m(row);
                for (int c = 1; c < C; ++c) M = fmaxf(M, state_m(row + c * rp));
                Lsum = 0.f;
                const float m0 = M == -INFINITY ? 0.f : M;
                for (int c = 0; c < C; ++c) Lsum += ex2(state_m(row + c * rp) - m0) * state_l(row + c * rp);
            };
            float M, Ls;
            joined(r & (rp - 1), M, Ls);
            const float m0 = M == -INFINITY ? 0.f : M;
            const bool whole = sg.slot < 0;
            // Weight of this lane's O: its copy's share, 1 / L, v_scale in the end.
            const float wgt = Ls == 0.f ? 0.f : ex2(state_m(r) - m0) / Ls * (whole ? vsc : 1.f);
            if (!(ok = wait_all(tOFull, (uint32_t)(nth & 1)))) break;
            tc_fence_after();
            const int row_o = r >> cl;  // the row this thread writes out, and its dims of each 32
            const int nd = 32 >> cl, d0 = (r & (C - 1)) * nd;
            const bool live = row_o < rows;
            const int tok = live ? row_o / g : 0, hh = live ? row_o - tok * g : 0;
            const size_t orow = (size_t)(sg.qo0 + sg.t0 + tok) * p.num_qo_heads + (size_t)sg.hk * g + hh;
            const size_t prow = (size_t)max(sg.slot, 0) * p.rows_pad + (live ? row_o : 0);
#pragma unroll 1
            for (int c = 0; c < DH / 32; ++c) {
                uint32_t hi[32];
                tc_ld32(tO + 32 * c, hi);
                if constexpr (!k2) {
                    uint32_t lo[32];
                    tc_ld32(tO + DH + 32 * c, lo);
                    tc_wait_ld();
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        hi[i] = __float_as_uint(fmaf(__uint_as_float(lo[i]), 1.f / 32.f, __uint_as_float(hi[i])));
                } else {
                    tc_wait_ld();
                }
                if (c + 1 == DH / 32) {  // O is read: the next segment may write it
                    tc_fence_before();
                    warp_arrive(bar(tOEmpty));
                }
#pragma unroll
                for (int i = 0; i < 32; ++i) hi[i] = Ls == 0.f ? 0u : __float_as_uint(__uint_as_float(hi[i]) * wgt);
                if (C > 1) {
                    // The copies meet in shared memory: every row's 32 dims of each,
                    // then each thread sums its 32 / C dims of one row.
                    const uint32_t stg = base + L.stage;
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        sts128(stg + (uint32_t)(r * kStageRow + 4 * i) * 4u, hi[4 * i], hi[4 * i + 1], hi[4 * i + 2], hi[4 * i + 3]);
                    warp_arrive(bar(tStage));
                    if (!(ok = wait_all(tStage, stage_phase))) break;
                    stage_phase ^= 1u;
#pragma unroll
                    for (int q = 0; q < 4; ++q) {  // up to 16 dims, four at a time
                        if (4 * q < nd) {
                            float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
                            for (int k = 0; k < C; ++k) {
                                const float4 x = lds_f4(stg + (uint32_t)((row_o + k * rp) * kStageRow + d0 + 4 * q) * 4u);
                                s.x += x.x, s.y += x.y, s.z += x.z, s.w += x.w;
                            }
                            hi[4 * q] = __float_as_uint(s.x), hi[4 * q + 1] = __float_as_uint(s.y);
                            hi[4 * q + 2] = __float_as_uint(s.z), hi[4 * q + 3] = __float_as_uint(s.w);
                        }
                    }
                    warp_arrive(bar(tStage));  // staging may be written again
                    if (!(ok = wait_all(tStage, stage_phase))) break;
                    stage_phase ^= 1u;
                }
                if (live) {
                    const int d = 32 * c + d0;
                    if (whole) {
                        uint4* dst = reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.o) + orow * DH + d);
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            if (8 * i < nd) {
                                uint32_t w[4];
#pragma unroll
                                for (int k = 0; k < 4; ++k)
                                    w[k] = pack_out2(__uint_as_float(hi[8 * i + 2 * k]), __uint_as_float(hi[8 * i + 2 * k + 1]),
                                                     p.o_dtype);
                                dst[i] = make_uint4(w[0], w[1], w[2], w[3]);
                            }
                    } else {
                        uint4* dst = reinterpret_cast<uint4*>(p.part_o + prow * DH + d);
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            if (4 * i < nd) dst[i] = make_uint4(hi[4 * i], hi[4 * i + 1], hi[4 * i + 2], hi[4 * i + 3]);
                    }
                }
            }
            if (!ok) break;
            if (live && d0 == 0) {
                float Mo, Lo;
                joined(row_o, Mo, Lo);
                const float lse2 = Lo == 0.f ? -INFINITY : Mo - PShift<KT>::kShift + __log2f(Lo);
                if (!whole)
                    p.part_lse[prow] = lse2;
                else if (p.lse != nullptr)
                    p.lse[orow] = lse2 * 0.69314718055994531f;
            }
        }
    }

    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (warp == 13) {
        tc_fence_after();
        tc_dealloc(tmem, 512);
    }
}

// Join the partial states of every split line's rows: one warp a row, lane l
// holding dims (D / 32) l .. of it; o = v_scale sum(2^lse_s O_s) / sum(2^lse_s).
constexpr int kTreeMergeWarps = 4;
template <int DH>
__global__ void __launch_bounds__(32 * kTreeMergeWarps) tree_merge_kernel(const __grid_constant__ TreeParams p) {
    constexpr int DPL = DH / 32;
    const int* meta = p.meta;
    const int4* rec = reinterpret_cast<const int4*>(meta + meta[kMetaOffTile]) + 2 * (long long)blockIdx.x;
    const int4 a = __ldg(rec), b = __ldg(rec + 1);  // slot0, slot1, first row of q, hk; rows
    const int row = blockIdx.y * kTreeMergeWarps + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (row >= b.x) return;
    const float vsc = p.v_scales != nullptr ? __ldg(p.v_scales + a.w) : p.v_scale;
    float m = -INFINITY, sum = 0.f, acc[DPL];
#pragma unroll
    for (int i = 0; i < DPL; ++i) acc[i] = 0.f;
    constexpr int kBatch = 4;  // states in flight
    for (int s = a.x; s < a.y; s += kBatch) {
        float l[kBatch], o[kBatch][DPL];
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            const size_t at = (size_t)min(s + k, a.y - 1) * p.rows_pad + row;
            l[k] = __ldcg(p.part_lse + at);
            const float* src = p.part_o + at * DH + DPL * lane;
            if constexpr (DPL == 4) {
                const float4 x = __ldcg(reinterpret_cast<const float4*>(src));
                o[k][0] = x.x, o[k][1] = x.y, o[k][2] = x.z, o[k][3] = x.w;
            } else {
                const float2 x = __ldcg(reinterpret_cast<const float2*>(src));
                o[k][0] = x.x, o[k][1] = x.y;
            }
        }
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            const float lk = s + k < a.y ? l[k] : -INFINITY;
            const float mn = fmaxf(m, lk);
            if (lk == -INFINITY) continue;  // a state that saw no key (or none at all)
            const float f = ex2(m - mn), w = ex2(lk - mn);
            sum = sum * f + w;
#pragma unroll
            for (int i = 0; i < DPL; ++i) acc[i] = acc[i] * f + w * o[k][i];
            m = mn;
        }
    }
    const float inv = sum == 0.f ? 0.f : vsc / sum;
    const int tok = row / p.group, hh = row - tok * p.group;
    const size_t orow = (size_t)(a.z + tok) * p.num_qo_heads + (size_t)a.w * p.group + hh;
    uint32_t w[DPL / 2];
#pragma unroll
    for (int i = 0; i < DPL / 2; ++i) w[i] = pack_out2(acc[2 * i] * inv, acc[2 * i + 1] * inv, p.o_dtype);
    uint16_t* dst = static_cast<uint16_t*>(p.o) + orow * DH + DPL * lane;
    if constexpr (DPL == 4)
        *reinterpret_cast<uint2*>(dst) = make_uint2(w[0], w[DPL > 2 ? 1 : 0]);
    else
        *reinterpret_cast<uint32_t*>(dst) = w[0];
    if (lane == 0 && p.lse != nullptr) p.lse[orow] = (m + __log2f(sum)) * 0.69314718055994531f;
}

template <int KT, int NP, int DH>
cudaError_t launch_tree_t(TreeParams p, const CUtensorMap& tk, const CUtensorMap& tv, int num_ctas, int num_merge,
                          cudaStream_t stream) {
    constexpr bool k2 = KT == PAFP8_BF16 || KT == PAFP8_F16;
    constexpr uint32_t tile = kTileKeys * DH * (k2 ? 2 : 1);
    // Two Q buffers (the next segment's Q is built during the current one)
    // unless three pieces of 16 KB leave too little for the K and V ring.
    p.q_buffers = p.q_pieces * tile > 40960 ? 1 : 2;
    const uint32_t q_bytes = (uint32_t)(p.q_buffers * p.q_pieces) * tile;
    constexpr uint32_t budget = 232448 - 1024;
    int stages = 2;
    while (stages < kMaxStages && tree_smem(q_bytes, tile, stages + 1).bytes <= budget) ++stages;
    p.stages = stages;
    const size_t smem = 1024 + tree_smem(q_bytes, tile, stages).bytes;
    auto kern = tree_kernel<KT, NP, DH>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    kern<<<num_ctas, kTreeThreads, smem, stream>>>(p, tk, tv);
    if ((e = cudaGetLastError()) != cudaSuccess || num_merge == 0) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(num_merge, (p.rows_pad + kTreeMergeWarps - 1) / kTreeMergeWarps);
    cfg.blockDim = dim3(32 * kTreeMergeWarps);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, tree_merge_kernel<DH>, p);
}

template <int DH>
cudaError_t launch_tree_head(const TreeParams& p, const CUtensorMap& tk, const CUtensorMap& tv, int num_ctas,
                             int num_merge, cudaStream_t stream) {
    switch (p.kv_dtype) {
        case PAFP8_F16: return launch_tree_t<PAFP8_F16, 1, DH>(p, tk, tv, num_ctas, num_merge, stream);
        case PAFP8_BF16: return launch_tree_t<PAFP8_BF16, 1, DH>(p, tk, tv, num_ctas, num_merge, stream);
        default: break;
    }
    // An f16 output keeps 11 bits: three pieces of P.
    return p.o_dtype == PAFP8_F16 ? launch_tree_t<PAFP8_E4M3FN, 3, DH>(p, tk, tv, num_ctas, num_merge, stream)
                                  : launch_tree_t<PAFP8_E4M3FN, 2, DH>(p, tk, tv, num_ctas, num_merge, stream);
}

}  // namespace
}  // namespace pafp8
