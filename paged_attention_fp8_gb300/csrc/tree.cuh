// tree.cuh -- attention of a tree of drafted tokens over the paged KV cache on
// the tcgen05 tensor cores (sm_103a).  Included by one translation unit per
// head size and row count (tree_d*_r*.cu), which compile in parallel.
//
// What it computes: request b has T new (drafted) tokens, whose keys are the
// last T of its L cached ones.  Drafted token u sees every key j < L - T and
// key L - T + w where bit w of its mask row is set.  For query head h of KV
// head h / group: o = v_scale * softmax(sm_scale * q_scale * k_scale * q.k) V
// over the keys it sees, lse = ln sum exp(logits); a row that sees no key
// gives o = 0, lse = -inf.
//
// What bounds it: with T * group rows per KV head a key costs 2 D bytes (fp8)
// from HBM and 4 D T group flops, so up to about 128 rows the cache's bytes
// bound it, and the tensor and softmax work per byte has to stay below that.
// Widening an fp8 tile to 16 bits in shared memory would cost more shared
// memory traffic than reading it once from HBM does, so nothing is widened:
//   * S^T = K Q^T takes K as it landed (kind::f8f6f4).  A 2-byte query row is
//     scaled by a power of two to a maximum in [128, 256) and split into
//     e4m3 pieces (4 significant bits each: two for bf16's 8, three for f16's
//     11) whose products add up in one accumulator: x = a + b (+ c), each
//     piece the e4m3 rounding of what the earlier ones left.  e4m3's smallest
//     step is 2^-9, so at most 2^-10 is lost (2^-17 of a largest magnitude of
//     128), and that only of elements with bits below the step: under 2^-2
//     (bf16; 2^-9 of the largest) or 2 (f16; 2^-6).
//   * O^T += V^T P^T takes V as it landed and P' = 2^5 p in [0, 256] as two fp8
//     pieces from shared memory: hi = e4m3(P') and lo = e5m2(P' - hi), whose
//     products add up in one accumulator.  P is then 2^-8
//     off at most, as a bf16 is, down to p = 2^-11, and below that never more
//     than 2^-19 of the row's largest.  e5m2 reaches low enough that lo needs
//     no scale of its own and so no second accumulator: an e4m3 lo is off by
//     half as much, but its accumulator's reads and TMEM columns cost 64
//     requests of 512-4096 keys 4.4 us (89.4 against 85.0, when the choice was
//     made; they take 83-84 now).
//   * An f16 output takes three: hi, lo = e4m3(32 (P' - hi)) and e4m3 of what lo
//     left, which is P' rounded to f16 (2^-11 off) down to p = 2^-9 and never
//     more than 2^-20 of the row's largest off below.  hi and lo lie side by side along N, so that one MMA reads V
//     once for both and leaves O_hi and O_lo (O = O_hi + O_lo / 32) in
//     neighbouring columns; the third piece is accumulated onto O_lo.
//   * A 2-byte cache of the query's dtype runs kind::f16 on Q, K and V as
//     they are, P rounded to that type.
//
// Both products are transposed: keys (of K) and dims (of V) are the 128 rows of
// the MMAs, query rows their N, so the tensor time follows the row count R (32
// or 64) instead of always paying for 128 rows.  With query rows as M, a
// 16-row draft spent 1400 cycles of the tensor pipe per 128-key tile, as much
// as the tile's HBM time; transposed it is about 500 at R = 32 and 700 at
// R = 64.  A softmax thread then owns a key, every lane is busy whatever R is,
// and P is written to shared memory, which frees S right away.  Drafts of more
// than 64 rows are cut into row tiles of 64, each of which reads the keys
// again: in this form 128 rows at once would take as long as two such tiles.
// (Query rows as M, a thread a row, would suit those drafts better, as in the
// prefill kernel; that form is not built.)
//
// One tile's softmax is a chain of some 2000 cycles (wait, load, scale, exp,
// convert, store, vote, hand on), longer than a tile's HBM time (1400).  So two
// groups of four warps take turns, one the even tiles, one the odd ones, each
// with its own accumulator in TMEM, maxima and sums: nothing passes between
// them, and the epilogue joins the two states.
//
// The running maximum: a row's maximum over a tile lies across 128 lanes, so it
// is not taken per tile.  P' is formed with the row's reference maximum, and
// only when some P' would pass 2^8, eight times that maximum's (a vote per tile,
// its latency hidden behind the exponentials and the stores of P), are the
// column maxima taken (redux), O and l rescaled and the tile's P redone; the
// first tile of a segment always takes them.
//
// Work: the plan lays the 128-key tiles of all (request, row tile) lines end to
// end, cuts them into equal ranges, and gives each range to a group of CTAs,
// one a KV head, so that the CTAs that read the heads of one token-major page
// run side by side.  A range's part of a line is a segment; a segment that is
// not its whole line writes a partial state, and a merge kernel (a
// programmatic dependent) joins them.
//
// Roles (512 threads; setmaxnreg moves registers to the softmax warps):
//   warps 0-3, 4-7  softmax of the even and of the odd tiles: thread = key
//               32 (w % 4) + lane of the tile;
//   warps 8-11  helpers: build the next segment's Q pieces, then the finished
//               segment's epilogue (lane = dim);
//   warps 12, 14, 15  TMA producers;  warp 13  MMA issuer and TMEM owner.
// TMEM columns: a ring of three S^T buffers (R columns each), then the O^T
// accumulators of the two groups (R columns each, 2 R for an f16 output over an
// fp8 cache), twice where there is room, so that the next segment may start while the
// epilogue reads the last one.  QK runs two tiles ahead of PV, into the next
// segment too.
// Measured (152 CTAs, caches larger than L2): 8 requests of 32768 keys, 4 drafted
// tokens of 8 heads a KV head, f16 over e5m2: 98 us, 81 % of the copy rate.  64
// requests of 512-4096 keys, 64 rows: 83-84 us, where the cache's bytes take 46: the
// softmax warps' chain bounds it (a scheduler issues in 49 % of its cycles, the
// tensor pipe is active in 23 %), two tiles at a time, and each of a CTA's four or
// so segments costs about five tiles to start and end.  32 requests over a bf16
// cache: 59.7 us (the bytes take 40), with two stages of K and V that leave HBM idle
// between bursts.
//
// All waits are bounded; on expiry a status bit is set and the CTA winds down.
#pragma once
#include "../../include/pafp8.h"
#include "internal.h"
#include "ptx.cuh"
#include "ring.h"

namespace pafp8 {
namespace {

using namespace ptx;

constexpr int kTreeThreads = 512;
constexpr int kMaxStages = 8;
constexpr int kSegCache = 32;  // segment records kept in shared memory
// Reference maxima rise when some P' would pass 2^(kShift + kHead).
template <int KT>
struct PShift {  // fp8 pieces: P' <= 2^8, e4m3 reaches 448
    static constexpr float kShift = 5.f, kHead = 3.f;
};
template <>
struct PShift<PAFP8_BF16> {
    static constexpr float kShift = 0.f, kHead = 8.f;
};
template <>
struct PShift<PAFP8_F16> {
    static constexpr float kShift = 0.f, kHead = 8.f;
};
// kShift - m of a row that has seen no key: any logit passes the bound.
constexpr float kUnseen = 1e30f;

// Sizes of one instantiation.  R: rows of a row tile, 32 or 64.
template <int KT, int NP, int DH, int R>
struct TreeDims {
    static constexpr bool k2 = KT == PAFP8_BF16 || KT == PAFP8_F16;
    static constexpr int ES = k2 ? 2 : 1;
    static constexpr uint32_t kTile = kTileKeys * DH * ES;  // a K or V tile
    static constexpr uint32_t kHalf = kTileKeys * 128;      // a 64-dim half of a 2-byte tile
    static constexpr int NH = DH / 64;                      // halves of a 2-byte row
    static constexpr uint32_t kQPiece = R * DH * ES;        // 2-byte: [half][R rows][128 B]
    static constexpr int W = R * ES;                        // bytes of a key's row of a P piece
    static constexpr uint32_t kPPiece = 128 * W;            // [128 keys][R]
    static constexpr bool kTwo = NP == 3;                   // O_hi and O_lo
    static constexpr int OC = kTwo ? 2 * R : R;             // columns of an accumulator
    static constexpr int NOB = 3 * R + 4 * OC <= 512 ? 2 : 1;  // accumulators of a group
    static constexpr uint32_t kColO = 3 * R;                // [NOB][group]
    static constexpr uint32_t kCols = kColO + NOB * 2 * OC <= 256 ? 256 : 512;
    static_assert(R == 32 || R == 64, "row tiles");
    static_assert(kColO + NOB * 2 * OC <= kCols, "TMEM columns");
};

struct TreeSmem {
    uint32_t q, k, v, p, sc, neg, alpha, wmax, lsum, mst, wt, rowp, seg, bars, next, tmem_slot, abort_flag, bytes;
};
enum TreeBar : int {
    tQFull = 0,              // [2]
    tQEmpty = 2,             // [2]
    tInfo = 4,               // [2] row scales of a segment written
    tState = 6,              // [2] m and l of a segment written
    tSFull = 8,              // [3]
    tPFull = 11,             // [3]
    tOFull = 14,             // [2]
    tOEmpty = 16,            // [2 buffers][2 groups]
    tHelp = 20,              // the helper warps
    tDrain = 21,
    tKFull = 22,
    tKEmpty = tKFull + kMaxStages,
    tVFull = tKEmpty + kMaxStages,
    tVEmpty = tVFull + kMaxStages,
    tNumBars = tVEmpty + kMaxStages
};
template <typename D, int R, int NP>
__host__ __device__ constexpr TreeSmem tree_smem(int q_tiles, int stages) {
    TreeSmem s{};
    s.q = 0;
    s.k = (uint32_t)q_tiles * D::kQPiece;
    s.v = s.k + (uint32_t)stages * D::kTile;
    s.p = s.v + (uint32_t)stages * D::kTile;
    s.sc = s.p + 3 * NP * D::kPPiece;       // [2][R] floats: log2 scale of each row
    s.neg = s.sc + 2 * R * 4;               // [8 warps][R]: kShift - reference maximum
    s.alpha = s.neg + 8 * R * 4;            // [8 warps][R]
    s.wmax = s.alpha + 8 * R * 4;           // [2][group][4 quadrants][32]
    s.lsum = s.wmax + 2 * 2 * 4 * 32 * 4;   // [2][8 warps][R]
    s.mst = s.lsum + 2 * 8 * R * 4;         // [2][group][R]
    s.wt = s.mst + 2 * 2 * R * 4;           // [2][group][R]
    s.rowp = s.wt + 2 * 2 * R * 4;          // [2][R] byte offsets of the rows in o (64 bits)
    s.seg = s.rowp + 2 * R * 8;             // the CTA's first kSegCache segment records
    s.bars = s.seg + kSegCache * kTreeSegWords * 4;
    s.next = s.bars + 8 * tNumBars;         // [K, V][3 producers]: one past the last tile loaded
    s.tmem_slot = s.next + 2 * 3 * 4;
    s.abort_flag = s.tmem_slot + 4;
    s.bytes = s.abort_flag + 4;
    return s;
}
// Q buffers and K / V stages of a launch.  Two Q buffers (the next segment's Q
// is built during the current one) if the ring keeps three stages of K and V,
// or two of a 2-byte cache.
constexpr uint32_t kSmemBudget = 232448 - 1024;
struct TreeRing {
    int q_buffers, stages;
};
template <typename D, int R, int NP>
__host__ __device__ constexpr TreeRing tree_ring(int q_pieces) {
    TreeRing r{tree_smem<D, R, NP>(2 * q_pieces, D::k2 ? 2 : 3).bytes <= kSmemBudget ? 2 : 1, 2};
    while (r.stages < kMaxStages && tree_smem<D, R, NP>(r.q_buffers * q_pieces, r.stages + 1).bytes <= kSmemBudget) ++r.stages;
    return r;
}
// Whether some query type leaves an instantiation two stages (a 2-byte cache at
// head_dim 128).
template <typename D, int R, int NP>
__host__ __device__ constexpr bool two_stages() {
    for (int q_pieces = 1; q_pieces <= (D::k2 ? 1 : 3); ++q_pieces)
        if (tree_ring<D, R, NP>(q_pieces).stages < 3) return true;
    return false;
}

__device__ __forceinline__ float lds_f(uint32_t a) {
    float v;
    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ uint32_t lds_u(uint32_t a) {
    uint32_t v;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ float4 lds_f4(uint32_t a) {
    float4 v;
    asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ void sts_f(uint32_t a, float v) { asm volatile("st.shared.f32 [%0], %1;" ::"r"(a), "f"(v) : "memory"); }

// A value that every lane holds, in a form that the compiler knows to be the
// same in all of them.  Control flow on anything else (a loaded loop bound, a
// warp index from threadIdx) counts as divergent, and every shuffle, vote or
// reduction under it is then compiled with a fallback that costs hundreds of
// cycles: a segment's column sums took 9000 cycles that way.
__device__ __forceinline__ int uniform(int x) { return __shfl_sync(0xFFFFFFFFu, x, 0); }

// Bounded wait that gives up once another role has (`flag`), and past `limit`
// cycles sets the flag and the status bit itself.  The loop is one compact asm
// block: some thirty waits are inlined, and the instruction cache holds little
// more than the tile loops.  `hint` is how long (ns) one try may suspend the
// thread; NAP, how long it sleeps between tries: a warp that polls takes issue
// slots from the working ones (eight polling warps took a fifth of them), so the
// roles that run ahead or wait long sleep.  With hint 0 (a shortened limit, which a suspended try could outlast) it only
// tests.
template <int NAP>
__device__ __forceinline__ bool tree_wait(uint32_t bar, uint32_t parity, uint32_t flag, uint32_t* status, long long limit,
                                          uint32_t hint) {
    if (mbar_test_wait(bar, parity)) return true;
    uint32_t ok;
    asm volatile(
        "{\n .reg .pred p, q;\n .reg .b64 t, u;\n .reg .b32 f;\n"
        " setp.eq.u32 q, %6, 0;\n mov.u64 t, %%clock64;\n"
        "LOOP:\n"
        " @q mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n"
        " @!q mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %6;\n @p bra DONE;\n"
        " ld.volatile.shared.u32 f, [%3];\n setp.ne.u32 p, f, 0;\n @p bra FAIL;\n"
        " nanosleep.u32 %8;\n"
        " mov.u64 u, %%clock64;\n sub.s64 u, u, t;\n setp.le.s64 p, u, %5;\n @p bra LOOP;\n"
        " st.shared.u32 [%3], 1;\n red.global.or.b32 [%4], %7;\n"
        "FAIL:\n mov.u32 %0, 0;\n bra END;\n"
        "DONE:\n mov.u32 %0, 1;\n"
        "END:\n}\n"
        : "=r"(ok)
        : "r"(bar), "r"(parity), "r"(flag), "l"(status), "l"(limit), "r"(hint), "n"((int)kStatusTimeout), "n"(NAP)
        : "memory");
    return ok != 0;
}

// One segment: key tiles [tile0, tile1) of a line (request, KV head, row tile).
// Row i of the tile is query head (r0 + i) % group of drafted token (r0 + i) /
// group.
struct Seg {
    int hk, r0, tile0, tile1, slot;  // slot: partial state, or -1 for a whole line
    int qo0, qo_len, kv_len, page0;
};
// The CTA's segment i (of its own list): from shared memory, or from global
// memory behind the first kSegCache.  A record is at the head of every role's
// work on a segment; from L2 each cost about a microsecond there.
__device__ __forceinline__ Seg load_seg(const int* segs, uint32_t cache, int i) {
    int4 a, b, c;
    if (i < kSegCache) {
        const uint32_t r = cache + (uint32_t)(kTreeSegWords * 4 * i);
        const uint4 x = lds128(r), y = lds128(r + 16), z = lds128(r + 32);
        a = make_int4((int)x.x, (int)x.y, (int)x.z, (int)x.w);
        b = make_int4((int)y.x, (int)y.y, (int)y.z, (int)y.w);
        c = make_int4((int)z.x, 0, 0, 0);
    } else {
        const int4* r = reinterpret_cast<const int4*>(segs + kTreeSegWords * (long long)i);
        a = __ldg(r), b = __ldg(r + 1), c = __ldg(r + 2);
    }
    return Seg{uniform(a.x), uniform(a.y), uniform(a.z), uniform(a.w), uniform(b.x), uniform(b.y), uniform(b.z), uniform(b.w),
               uniform(c.x)};
}

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

__device__ __forceinline__ __half2 half2_of_e4m3(uint32_t pair) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((unsigned short)pair));
    return *reinterpret_cast<__half2*>(&h);
}
__device__ __forceinline__ uint32_t e4m3_of_half2(__half2 x) {
    unsigned short d;
    asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(d) : "r"(*reinterpret_cast<uint32_t*>(&x)));
    return d;
}
// Four f16 values to e4m3 codes (returned), and what the codes leave of them, in
// place (exact).  In one asm block the 16-bit codes need no widening (64 requests
// of 512-4096 keys: 85.3 -> 83.6 us).
__device__ __forceinline__ uint32_t e4m3_quad(uint32_t& h0, uint32_t& h1) {
    uint32_t w;
    asm("{\n .reg .b16 a, b;\n .reg .b32 x, y;\n"
        " cvt.rn.satfinite.e4m3x2.f16x2 a, %1;\n cvt.rn.satfinite.e4m3x2.f16x2 b, %2;\n"
        " cvt.rn.f16x2.e4m3x2 x, a;\n cvt.rn.f16x2.e4m3x2 y, b;\n mov.b32 %0, {a, b};\n"
        " sub.rn.f16x2 %1, %1, x;\n sub.rn.f16x2 %2, %2, y;\n}\n"
        : "=&r"(w), "+r"(h0), "+r"(h1));
    return w;
}
__device__ __forceinline__ uint32_t times32(uint32_t h) {
    const __half2 x = __hmul2(*reinterpret_cast<__half2*>(&h), __float2half2_rn(32.f));
    return *reinterpret_cast<const uint32_t*>(&x);
}

// Four P' (at most 2^8) as fp8 pieces, four codes a word: hi = e4m3(P'), and
// lo = e5m2(P' - hi), an e5m2 code being the high byte of the f16 of equal
// value (rounded half up: adding half a step to the bits); with NP = 3
// lo = e4m3(32 (P' - hi)) and lo2 = e4m3 of what lo left.  P' is first rounded
// to f16 (2^-11 off), in which the differences are exact.
template <int NP>
__device__ __forceinline__ void p_pieces(const float* x, uint32_t& hi, uint32_t& lo, uint32_t& lo2) {
    uint32_t h0 = pack_half2(x[0], x[1]), h1 = pack_half2(x[2], x[3]);
    hi = e4m3_quad(h0, h1);
    if constexpr (NP == 3) {
        h0 = times32(h0), h1 = times32(h1);
        lo = e4m3_quad(h0, h1);
        lo2 = e4m3_quad(h0, h1);
    } else {
        lo = prmt(h0 + 0x00800080u, h1 + 0x00800080u, 0x7531u);
    }
}

// 32 columns of this thread's TMEM lane; loaded values are there after tc_wait_ld.
__device__ __forceinline__ void ld_cols(uint32_t t, float (&v)[32]) { tc_ld32(t, reinterpret_cast<uint32_t(&)[32]>(v)); }
__device__ __forceinline__ void st_cols(uint32_t t, const float (&v)[32]) {
    tc_st32(t, reinterpret_cast<const uint32_t(&)[32]>(v));
}

// The 128 threads of a softmax group meet; true if any of them says so.  A
// hardware barrier and not an mbarrier: the votes of an mbarrier's waiters came
// 400 cycles late.  It has no bound, so every warp of a group goes through the
// same barriers whatever its own waits did, and the group leaves together.
__device__ __forceinline__ bool group_any(int id, bool mine) {
    uint32_t r;
    asm volatile(
        "{\n .reg .pred p, q;\n setp.ne.u32 p, %2, 0;\n barrier.cta.red.or.pred q, %1, 128, p;\n selp.u32 %0, 1, 0, q;\n}\n"
        : "=r"(r)
        : "r"(id), "r"((uint32_t)mine)
        : "memory");
    return __any_sync(0xFFFFFFFFu, r != 0);
}

// Sums of v[0 .. 31] over the warp's lanes: lane l returns column l's.
__device__ __forceinline__ float column_sum(float (&a)[32], int lane) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) {
        const bool up = (lane & d) != 0;
#pragma unroll
        for (int i = 0; i < d; ++i) {
            const float keep = up ? a[i + d] : a[i], send = up ? a[i] : a[i + d];
            a[i] = keep + __shfl_xor_sync(0xFFFFFFFFu, send, d);
        }
    }
    return a[0];
}

template <int KT, int NP, int DH, int R>
__global__ void __launch_bounds__(kTreeThreads, 1)
    tree_kernel(const __grid_constant__ TreeParams p, const __grid_constant__ CUtensorMap tmk,
                const __grid_constant__ CUtensorMap tmv) {
    using D = TreeDims<KT, NP, DH, R>;
    constexpr bool k2 = D::k2;
    constexpr uint32_t kTile = D::kTile, kHalf = D::kHalf;
    constexpr int NH = D::NH, NOB = D::NOB;
    constexpr float kShift = PShift<KT>::kShift, kHead = PShift<KT>::kHead;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t base = (smem_addr(smem_raw) + 1023u) & ~1023u;
    const TreeSmem L = tree_smem<D, R, NP>(p.q_buffers * p.q_pieces, p.stages);
    auto bar = [&](int i) -> uint32_t { return base + L.bars + 8u * (uint32_t)i; };
    const uint32_t flag = base + L.abort_flag;
    const int warp = uniform((int)(threadIdx.x >> 5)), lane = threadIdx.x & 31;
    const int NS = p.stages, NQB = p.q_buffers;
    const int* meta = p.meta;
    const int s_first = __ldg(meta + meta[kMetaOffCtaSeg] + blockIdx.x);
    const int n_seg = uniform(__ldg(meta + meta[kMetaOffCtaSeg] + blockIdx.x + 1) - s_first);
    const int* segs = meta + meta[kMetaOffSeg] + kTreeSegWords * (long long)s_first;
    const uint32_t seg_cache = base + L.seg;
    const int g = p.group;
    // n / group for n < 2^25 (a plan has no more rows in a request).
    auto token_of = [&](int n) -> int { return g == 1 ? n : (int)__umulhi((uint32_t)n, p.group_magic); };
    const uint32_t hint = p.wait_cycles < kWaitCyclesDefault ? 0u : 20000u;
    auto wait_all = [&](int b, uint32_t parity) {
        return (bool)__all_sync(0xFFFFFFFFu, tree_wait<0>(bar(b), parity, flag, p.status, p.wait_cycles, hint));
    };
    auto wait_idle = [&](int b, uint32_t parity) {  // for the roles that may come a little late
        return (bool)__all_sync(0xFFFFFFFFu, tree_wait<100>(bar(b), parity, flag, p.status, p.wait_cycles, hint));
    };

    if (threadIdx.x == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(bar(tQFull + i), 4);   // helper warps
            mbar_init(bar(tQEmpty + i), 1);  // commit
            mbar_init(bar(tInfo + i), 4);
            mbar_init(bar(tState + i), 8);   // softmax warps
            mbar_init(bar(tOFull + i), 1);
        }
        for (int i = 0; i < 3; ++i) {
            mbar_init(bar(tSFull + i), 1);
            mbar_init(bar(tPFull + i), 4);   // a group's warps
        }
        for (int i = 0; i < 4; ++i) mbar_init(bar(tOEmpty + i), 4);
        mbar_init(bar(tHelp), 4);
        mbar_init(bar(tDrain), 1);
        for (int i = 0; i < NS; ++i) {
            mbar_init(bar(tKFull + i), 1);  // the tile's producer warp
            mbar_init(bar(tKEmpty + i), 1);
            mbar_init(bar(tVFull + i), 1);
            mbar_init(bar(tVEmpty + i), 1);
        }
        asm volatile("st.shared.u32 [%0], 0;" ::"r"(flag) : "memory");
        mbar_init_fence();
    }
    for (int i = threadIdx.x; i < min(n_seg, kSegCache) * kTreeSegWords; i += kTreeThreads)
        sts32(seg_cache + 4u * i, (uint32_t)__ldg(segs + i));
    if (warp == 13) tc_alloc(base + L.tmem_slot, D::kCols);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const uint32_t tmem = lds_u(base + L.tmem_slot);  // (the records and barriers above are visible from here on)

    if (warp >= 12) {
      asm volatile("setmaxnreg.dec.sync.aligned.u32 72;" ::: "memory");
      if (warp != 13) {
        // ----------------------------------------------------------- producers
        // A box holds the 16 tokens of one (sub-)page; a warp takes about 130 cycles
        // to issue one, 16 a tile 2100, more than the tile's time at full bandwidth
        // (1400).  So three warps take every third tile each.  A warp that waits
        // for a V slot (freed by the tile's softmax and PV) holds up none of the
        // next two tiles' K.  With two stages only two warps take part: a wait
        // names its phase by parity, so it has to follow the completion of the
        // phase two before, that is, of tile n - 2 stages; the warp's tile before,
        // n - step, vouches for tile n - step - stages, which is enough when step
        // <= stages.
        const int pw = warp == 12 ? 0 : warp - 13;
        const int step = min(3, NS);
        if (lane == 0) {
            prefetch_tmap(&tmk);
            prefetch_tmap(&tmv);
        }
        constexpr int kBoxes = 8 * (k2 ? NH : 1);  // boxes of a K or V tile, one a lane: (half, sub-page)
        constexpr uint32_t kBoxBytes = k2 ? 2048u : (uint32_t)(kPageSize * DH);
        const int m = p.page_mult;
        int n = pw < step ? pw : 1 << 30, total = 0;  // this warp's next tile; tiles of the segments so far
        int stage = pw % NS;
        uint32_t phase = (uint32_t)(pw / NS) & 1u;
        bool ok = true, k_only = false;
        for (int si = 0; si < n_seg && ok; ++si) {
            const Seg sg = load_seg(segs, seg_cache, si);
            const int nsub = (sg.kv_len + kPageSize - 1) / kPageSize;  // 16-token sub-pages of the request
            const int* idx = p.kv_indices + sg.page0;
            auto fetch = [&](int tile) -> int {  // the page entry of this lane's sub-page
                const int v = tile * (kTileKeys / kPageSize) + (lane & 7);
                return v < nsub ? __ldg(idx + (m == 1 ? v : v / m)) : 0;
            };
            int t = min(sg.tile0 + (n - total), sg.tile1 + 8);
            total += sg.tile1 - sg.tile0;
            int next = t < sg.tile1 ? fetch(t) : 0;
            for (; t < sg.tile1; t += step, n += step) {
                int page = next;
                if (t + step < sg.tile1) next = fetch(t + step);
                const int sub = t * (kTileKeys / kPageSize) + (lane & 7);
                const bool mine = lane < kBoxes && sub < nsub;
                if (mine && (page < 0 || page >= p.num_pages)) {
                    page = 0;
                    atomicOr(p.status, kStatusBounds);
                }
                const int slot = m == 1 ? 0 : (sub % m) * kPageSize;
                const uint32_t bytes = (uint32_t)__popc(__ballot_sync(0xFFFFFFFFu, mine)) * kBoxBytes;
                for (int kv = 0; kv < 2; ++kv) {
                    const int full = (kv ? tVFull : tKFull) + stage;
                    if (!(ok = wait_idle((kv ? tVEmpty : tKEmpty) + stage, phase ^ 1u))) {
                        k_only = kv == 1;
                        break;
                    }
                    if (lane == 0) mbar_arrive_expect_tx(bar(full), bytes);
                    __syncwarp();
                    const CUtensorMap* map = kv ? &tmv : &tmk;
                    const uint32_t dst = base + (kv ? L.v : L.k) + (uint32_t)stage * kTile + (uint32_t)lane * kBoxBytes;
                    if (mine) {
                        if constexpr (k2)
                            tma_load_5d(dst, map, bar(full), 0, lane >> 3, slot, sg.hk, page);
                        else
                            tma_load_4d(dst, map, bar(full), 0, sg.hk, slot, page);
                    }
                    __syncwarp();
                }
                if (!ok) break;
                for (stage += step; stage >= NS; stage -= NS) phase ^= 1u;
            }
        }
        // Every copy lands before the CTA may exit: the last one of each slot.  After
        // an expired wait another warp may have filled a slot once more, so the warps
        // meet first (each comes here, its waits being bounded) and say how far they got.
        if (lane == 0) {
            sts32(base + L.next + 4u * pw, (uint32_t)(pw < step ? n + (!ok && k_only) : 0));
            sts32(base + L.next + 12u + 4u * pw, (uint32_t)(pw < step ? n : 0));
        }
        asm volatile("barrier.cta.sync 3, 96;" ::: "memory");
        if (pw == 0 && lane < 2 * NS) {
            const int kv = lane >= NS, slot = lane - (kv ? NS : 0);
            const uint32_t at = base + L.next + 12u * kv;
            const int next[3] = {(int)lds_u(at), (int)lds_u(at + 4u), (int)lds_u(at + 8u)};
            const int x = ring_last_load(next, step, NS, slot);
            if (x >= 0) mbar_wait(bar((kv ? tVFull : tKFull) + slot), (uint32_t)((x / NS) & 1));
        }
        __syncwarp();
      } else {
        // ----------------------------------------------------------------- MMA
        // The whole warp walks the loop in step and one lane issues: with the
        // loop under `if (lane == 0)` every operand went through vector
        // registers, some 800 instructions a tile, and the issuing thread, not
        // the tensor pipe, set the tile's time.
        const uint32_t elect = elect_one();
        const int kvf = k2 ? (KT == PAFP8_BF16 ? 1 : 0) : (p.kv_dtype == PAFP8_E5M2 ? 1 : 0);
        const int qf = k2 ? kvf : (p.q_dtype == PAFP8_E5M2 ? 1 : 0);
        const uint32_t idesc_qk = make_idesc(kvf, qf, 128, R);
        const uint32_t idesc_pv = make_idesc_mn(kvf, k2 ? kvf : 0, 128, D::OC);
        const uint32_t idesc_p2 = make_idesc_mn(kvf, D::kTwo ? 0 : 1, 128, R);  // the last piece
        const uint32_t tm = (uint32_t)uniform((int)tmem);
        auto tiles_of = [&](int si) -> int {
            const Seg sg = load_seg(segs, seg_cache, si);
            return sg.tile1 - sg.tile0;
        };
        // Descriptors: the constant halves, and the words of the tiles at offset 0.
        constexpr uint64_t kQKd = (k2 || DH == 128) ? 1 : 0;  // 128-byte rows, else 64
        const uint64_t qk_proto = kQKd ? sw128_kmajor_desc(0) : sw64_kmajor_desc(0);
        const uint64_t v_proto = k2 ? mnmajor_desc<128>(0, DH == 128 ? kHalf : kTile) : mnmajor_desc<(k2 ? 128 : DH)>(0, kTile);
        const uint64_t p_proto = mnmajor_desc<D::W>(0, D::kPPiece);
        const uint32_t qk_hi = (uint32_t)(qk_proto >> 32), v_hi = (uint32_t)(v_proto >> 32), p_hi = (uint32_t)(p_proto >> 32);
        const uint32_t k_lo = (uint32_t)qk_proto + ((base + L.k) >> 4), q_lo = (uint32_t)qk_proto + ((base + L.q) >> 4);
        const uint32_t v_lo = (uint32_t)v_proto + ((base + L.v) >> 4), p_lo = (uint32_t)p_proto + ((base + L.p) >> 4);
        bool ok = true;
        int qs = 0, qn = 0, qbuf = 0;  // QK's segment, tile count and Q buffer
        uint32_t qphase = 0;
        int kstage = 0, vstage = 0;
        uint32_t kphase = 0, vphase = 0;
        int sbuf = 0, pbuf = 0;        // ring of three: S of QK's tile, P of PV's
        uint32_t pphase = 0;
        int qleft = n_seg > 0 ? tiles_of(0) : 0;
        bool qfirst = true;
        int pn = 0;
        for (int ps = 0; ps < n_seg && ok; ++ps) {
            const int ob = ps % NOB;
            const int nt = tiles_of(ps);
            for (int t = 0; t < nt; ++t, ++pn) {
                // QK(j + 2) goes before PV(j), into the next segment at most (the Q of
                // the one after is built only when this one's epilogue is done).  So
                // QK(j) follows PV(j - 3), which waited for P(j - 3): S(j - 3) has been
                // read, and once S(j) is complete so is PV(j - 3) and P's buffer free.
                while (qs < n_seg && qn <= pn + 2 && qs <= ps + 1) {
                    if (qfirst) {
                        if (!(ok = wait_all(tQFull + qbuf, qphase))) break;
                        qfirst = false;
                    }
                    if (!(ok = wait_all(tKFull + kstage, kphase))) break;
                    tc_fence_after();
                    // S^T = K Q^T: A = K (keys), B = Q (rows), both K-major.
                    const uint32_t d = tm + (uint32_t)(R * sbuf);
                    const uint32_t ka = k_lo + (uint32_t)kstage * (kTile >> 4);
                    uint32_t qa = q_lo + (uint32_t)(qbuf * p.q_pieces) * (D::kQPiece >> 4);
                    if constexpr (k2) {
#pragma unroll
                        for (int i = 0; i < DH / 16; ++i)  // K = 16: 32 bytes on, then the other 64-dim half
                            tc_mma_elect<false>(d, ka + (i >> 2) * (kHalf >> 4) + 2 * (i & 3), qk_hi,
                                                qa + (i >> 2) * (R * 128 >> 4) + 2 * (i & 3), qk_hi, idesc_qk, i > 0, elect);
                    } else {
                        for (int pc = 0; pc < p.q_pieces; ++pc, qa += D::kQPiece >> 4) {
#pragma unroll
                            for (int i = 0; i < DH / 32; ++i)
                                tc_mma_elect<true>(d, ka + 2 * i, qk_hi, qa + 2 * i, qk_hi, idesc_qk, pc > 0 || i > 0, elect);
                        }
                    }
                    tc_commit_elect(bar(tSFull + sbuf), elect);
                    tc_commit_elect(bar(tKEmpty + kstage), elect);
                    if (++kstage == NS) {
                        kstage = 0;
                        kphase ^= 1u;
                    }
                    if (++sbuf == 3) sbuf = 0;
                    ++qn;
                    if (--qleft == 0) {
                        tc_commit_elect(bar(tQEmpty + qbuf), elect);
                        if (++qbuf == NQB) {
                            qbuf = 0;
                            qphase ^= 1u;
                        }
                        qfirst = true;
                        if (++qs < n_seg) qleft = tiles_of(qs);
                    }
                }
                if (!ok) break;
                // O of the segment that last used this accumulator has been read.
                const int gr = pn & 1;
                if (t < 2 && ps >= NOB && !(ok = wait_all(tOEmpty + 2 * ob + gr, (uint32_t)((ps / NOB + 1) & 1)))) break;
                if (!(ok = wait_all(tVFull + vstage, vphase))) break;
                if (!(ok = wait_all(tPFull + pbuf, pphase))) break;
                tc_fence_after();
                // O^T += V^T P^T: A = V (dims), B = P (rows), both MN-major.  64 dims
                // fill half of M = 128: the other half reads the shared memory one
                // tile on and its lanes of O are never used.
                const uint32_t d = tm + D::kColO + (uint32_t)(D::OC * (2 * ob + gr));
                const uint32_t va = v_lo + (uint32_t)vstage * (kTile >> 4);
                const uint32_t pa = p_lo + (uint32_t)pbuf * (NP * D::kPPiece >> 4);
                constexpr int W = D::W;
                if constexpr (k2) {
#pragma unroll
                    for (int i = 0; i < 8; ++i)  // K = 16 keys
                        tc_mma_elect<false>(d, va + 128 * i, v_hi, pa + W * i, p_hi, idesc_pv, t >= 2 || i > 0, elect);
                } else {
#pragma unroll
                    for (int i = 0; i < 4; ++i)  // K = 32 keys
                        tc_mma_elect<true>(d, va + 2 * DH * i, v_hi, pa + 2 * W * i, p_hi, idesc_pv, t >= 2 || i > 0, elect);
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        tc_mma_elect<true>(D::kTwo ? d + R : d, va + 2 * DH * i, v_hi,
                                           pa + ((NP - 1) * D::kPPiece >> 4) + 2 * W * i, p_hi, idesc_p2, 1u, elect);
                }
                tc_commit_elect(bar(tVEmpty + vstage), elect);
                if (t + 1 == nt) tc_commit_elect(bar(tOFull + ob), elect);
                if (++vstage == NS) {
                    vstage = 0;
                    vphase ^= 1u;
                }
                if (++pbuf == 3) {
                    pbuf = 0;
                    pphase ^= 1u;
                }
            }
        }
        if (qn > 0) {  // every MMA completes before TMEM is freed
            tc_commit_elect(bar(tDrain), elect);
            mbar_wait(bar(tDrain), 0);
        }
        __syncwarp();
      }
    } else if (warp < 8) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 176;" ::: "memory");
        // ------------------------------------------------------------- softmax
        const int quad = warp & 3, gr = warp >> 2;  // this group's tiles have parity gr
        const int krow = 32 * quad + lane;          // this thread's key in a tile
        const uint32_t lane_base = tmem + ((uint32_t)(32 * quad) << 16);
        const uint32_t negt = base + L.neg + (uint32_t)(warp * R) * 4u;
        const uint32_t alt = base + L.alpha + (uint32_t)(warp * R) * 4u;
        const int vbar = 1 + gr;                    // the group's hardware barrier
        // Ring positions of this group's current tile: V stage (and the one of its
        // tile before), S and P buffer.
        int stage = 0, prev_stage = 0, buf = 0;
        uint32_t vphase = 0, prev_phase = 0, bphase = 0;
        auto advance = [&]() {
            if (++stage == NS) {
                stage = 0;
                vphase ^= 1u;
            }
            if (++buf == 3) {
                buf = 0;
                bphase ^= 1u;
            }
        };
        int j = 0;  // tiles of the CTA before the next one
        uint32_t wbuf = 0;
        // Whether one of this warp's waits gave up: it goes on (its results no
        // longer matter) until the group's next vote, where all four leave.
        bool dead = false, out = false;
        for (int si = 0; si < n_seg && !out; ++si) {
            const Seg sg = load_seg(segs, seg_cache, si);
            const int rows = min(R, sg.qo_len * g - sg.r0);
            const int ctx = sg.kv_len - sg.qo_len;
            const uint32_t tO = lane_base + D::kColO + (uint32_t)(D::OC * (2 * (si % NOB) + gr));
            const uint32_t sct = base + L.sc + (uint32_t)((si & 1) * R) * 4u;
            // Sums of P' over this thread's keys, rows 0-31 and 32-63.
            f32x2 l[R / 32][16];
#pragma unroll
            for (int i = 0; i < 16; ++i) l[0][i] = l[R / 32 - 1][i] = make_f32x2(0.f, 0.f);
            // Mask bits of this warp's 32 keys of a tile, lane i holding those of rows
            // i and i + 32, fetched a tile ahead.
            constexpr int NL = R / 32;
            const uint32_t* mrow[NL];
#pragma unroll
            for (int i = 0; i < NL; ++i)
                mrow[i] = p.tree_mask + (long long)(sg.qo0 + token_of(sg.r0 + min(32 * i + lane, rows - 1))) * p.mask_words;
            uint32_t bits[NL];
            auto fetch_bits = [&](int t) {
#pragma unroll
                for (int i = 0; i < NL; ++i)
                    bits[i] = (t + 1) * kTileKeys > ctx
                                  ? mask_bits(mrow[i], t * kTileKeys + 32 * quad - ctx, p.mask_words, sg.qo_len)
                                  : 0xFFFFFFFFu;
            };
            const int t_first = sg.tile0 + ((j ^ gr) & 1);  // this group's first tile of the segment
            fetch_bits(t_first);
            dead |= !wait_all(tInfo + (si & 1), (uint32_t)((si >> 1) & 1));
            for (int t = sg.tile0; t < sg.tile1 && !out; ++t, ++j) {
                if ((j & 1) != gr) {
                    advance();
                    continue;
                }
                const bool first = t == t_first;
                const uint32_t tS = lane_base + (uint32_t)(R * buf);
                dead |= !wait_all(tSFull + buf, bphase);
                tc_fence_after();
                const uint32_t pb = base + L.p + (uint32_t)buf * (NP * D::kPPiece);
                // 32 rows at a time: P' in place of the logits.  After P is stored the group
                // votes on the reference maxima; a raised one redoes the rows.  Rolled:
                // with two copies of this code the rare path was never in the
                // instruction cache and cost 6000 cycles each time.
#pragma unroll 1
                for (int sub = 0; sub < NL; ++sub) {
                    const uint32_t tSs = tS + 32u * sub, scs = sct + 128u * sub, ngs = negt + 128u * sub, als = alt + 128u * sub;
                    float v[32];
                    int rise = first;
#pragma unroll 1
                    while (true) {
                        ld_cols(tSs, v);
                        tc_wait_ld();
                        if ((t + 1) * kTileKeys > ctx) {  // keys that a row does not see become -inf
#pragma unroll
                            for (int c = 0; c < 32; ++c)
                                if (!((__shfl_sync(0xFFFFFFFFu, sub == 0 ? bits[0] : bits[NL - 1], c) >> lane) & 1u)) v[c] = -INFINITY;
                        }
                        if (rise) {
                            // Column maxima of the tile: over this warp's lanes, then over the
                            // group's four warps.  Lane i settles row i.
                            float cm = 0.f;
#pragma unroll
                            for (int c = 0; c < 32; ++c) {
                                const float m = warp_max(v[c]);
                                if (lane == c) cm = m;
                            }
                            const uint32_t wm = base + L.wmax + (uint32_t)((wbuf * 2 + gr) * 128 + lane) * 4u;
                            wbuf ^= 1u;
                            sts_f(wm + 128u * quad, cm);
                            group_any(vbar, false);
                            const float top = fmaxf(max3(lds_f(wm), lds_f(wm + 128u), lds_f(wm + 256u)), lds_f(wm + 384u)) * lds_f(scs + 4u * lane);
                            const float was = first ? kUnseen : lds_f(ngs + 4u * lane);
                            const float m_old = was >= kUnseen ? -INFINITY : kShift - was;
                            const float m_new = fmaxf(m_old, top);
                            sts_f(als + 4u * lane, m_old == -INFINITY ? 0.f : ex2(m_old - m_new));
                            sts_f(ngs + 4u * lane, m_new == -INFINITY ? kUnseen : kShift - m_new);
                            __syncwarp();
                            if (!first) {
                                // This accumulator's last update has to be complete.
                                dead |= !wait_all(tVEmpty + prev_stage, prev_phase);
                                tc_fence_after();
#pragma unroll 1
                                for (int c0 = 32 * sub; c0 < D::OC; c0 += R) {  // O_hi, O_lo
                                    float o[32];
                                    ld_cols(tO + c0, o);
                                    tc_wait_ld();
#pragma unroll
                                    for (int i = 0; i < 32; i += 4) {
                                        const float4 a = lds_f4(als + 4u * i);
                                        o[i] *= a.x, o[i + 1] *= a.y, o[i + 2] *= a.z, o[i + 3] *= a.w;
                                    }
                                    st_cols(tO + c0, o);
                                }
#pragma unroll
                                for (int i = 0; i < 16; i += 2) {
                                    const float4 a = lds_f4(als + 8u * i);
                                    const f32x2 a0 = make_f32x2(a.x, a.y), a1 = make_f32x2(a.z, a.w);
                                    if (sub == 0) {
                                        l[0][i] = mul2(l[0][i], a0);
                                        l[0][i + 1] = mul2(l[0][i + 1], a1);
                                    } else {
                                        l[NL - 1][i] = mul2(l[NL - 1][i], a0);
                                        l[NL - 1][i + 1] = mul2(l[NL - 1][i + 1], a1);
                                    }
                                }
                                tc_wait_st();
                            }
                        }
                        // x = s * scale + (kShift - m)
#pragma unroll
                        for (int c = 0; c < 32; c += 4) {
                            const float4 sc = lds_f4(scs + 4u * c), ng = lds_f4(ngs + 4u * c);
                            split_f32x2(fma2(make_f32x2(v[c], v[c + 1]), make_f32x2(sc.x, sc.y), make_f32x2(ng.x, ng.y)), v[c],
                                        v[c + 1]);
                            split_f32x2(fma2(make_f32x2(v[c + 2], v[c + 3]), make_f32x2(sc.z, sc.w), make_f32x2(ng.z, ng.w)),
                                        v[c + 2], v[c + 3]);
                        }
                        float pm[2] = {v[0], v[1]};
#pragma unroll
                        for (int c = 2; c < 32; c += 2) pm[(c >> 1) & 1] = max3(pm[(c >> 1) & 1], v[c], v[c + 1]);
#pragma unroll
                        for (int c = 0; c < 32; ++c) v[c] = ex2(v[c]);
                        // P into shared memory: the buffer's last product was complete before S.
                        constexpr int W = D::W;
                        constexpr int kElems = 16 / D::ES;  // rows a 16-byte chunk
                        const uint32_t swz = W == 128 ? krow & 7 : W == 64 ? (krow >> 1) & 3 : (krow >> 2) & 1;
#pragma unroll
                        for (int c = 0; c < 32; c += kElems) {
                            const uint32_t at = pb + (uint32_t)krow * W + (((uint32_t)(32 / kElems * sub + c / kElems) ^ swz) << 4);
                            uint32_t w0[4], w1[4], w2[4];
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                if constexpr (KT == PAFP8_BF16) {
                                    w0[i] = pack_bf162(v[c + 2 * i], v[c + 2 * i + 1]);
                                } else if constexpr (KT == PAFP8_F16) {
                                    w0[i] = pack_half2(v[c + 2 * i], v[c + 2 * i + 1]);
                                } else {
                                    p_pieces<NP>(v + c + 4 * i, w0[i], w1[i], w2[i]);
                                }
                            }
                            sts128(at, w0[0], w0[1], w0[2], w0[3]);
                            if constexpr (!k2) sts128(at + D::kPPiece, w1[0], w1[1], w1[2], w1[3]);
                            if constexpr (NP == 3) sts128(at + 2 * D::kPPiece, w2[0], w2[1], w2[2], w2[3]);
                        }
                        if (!group_any(vbar, dead || (!rise && fmaxf(pm[0], pm[1]) > kShift + kHead))) break;
                        if (group_any(vbar, dead)) {
                            out = true;
                            break;
                        }
                        rise = 1;
                    }
                    if (out) break;
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const f32x2 e = make_f32x2(v[2 * i], v[2 * i + 1]);
                        if (sub == 0)
                            l[0][i] = add2(l[0][i], e);
                        else
                            l[NL - 1][i] = add2(l[NL - 1][i], e);
                    }
                }
                if (out) break;
                // Value rows behind the request's end (the tail of its last page and
                // rows no page filled) hold anything: zero them, P = 0 there must
                // not meet a NaN.  The wait for V names its phase by parity, so the
                // phase before it, V of tile j - NS, has to be known complete: S(j)
                // vouches for PV(j - 3), which with two stages says nothing of
                // V(j - 2): the wait could pass before that had landed, and the zeros
                // go into that tile's rows.  So with two stages PV(j - 2) is waited for
                // first (a phase that follows PV(j - 4), for which S(j) does vouch; it
                // always ends, this group's P(j - 2) being given).
                const int valid = sg.kv_len - t * kTileKeys;
                if (valid < kTileKeys) {
                    if constexpr (two_stages<D, R, NP>()) dead |= !wait_all(tVEmpty + stage, vphase ^ 1u);
                    dead |= !wait_all(tVFull + stage, vphase);
                    if (krow >= valid) {
                        const uint32_t vrow = base + L.v + (uint32_t)stage * kTile + (uint32_t)krow * (k2 ? 128u : (uint32_t)DH);
#pragma unroll
                        for (int c = 0; c < (k2 ? 8 : DH / 16); ++c) {
                            sts128(vrow + 16u * c, 0u, 0u, 0u, 0u);
                            if (k2 && NH == 2) sts128(vrow + kHalf + 16u * c, 0u, 0u, 0u, 0u);
                        }
                    }
                }
                fence_async_smem();
                tc_fence_before();
                warp_arrive(bar(tPFull + buf));
                if (t + 2 < sg.tile1) fetch_bits(t + 2);
                prev_stage = stage;
                prev_phase = vphase;
                advance();
            }
            if (out) break;
            // The segment's sums (over this warp's keys) and this group's maxima for
            // the epilogue; a group without a tile in it leaves an empty state.
            const bool none = t_first >= sg.tile1;
#pragma unroll 1
            for (int i = 0; i < NL; ++i) {
                float ls[32];
#pragma unroll
                for (int c = 0; c < 16; ++c) split_f32x2(i == 0 ? l[0][c] : l[NL - 1][c], ls[2 * c], ls[2 * c + 1]);
                const float sum = column_sum(ls, lane);
                const int row = 32 * i + lane;
                sts_f(base + L.lsum + 4u * (((si & 1) * 8 + warp) * R + row), sum);
                const float ng = lds_f(negt + 4u * row);
                if (quad == 0)
                    sts_f(base + L.mst + 4u * (((si & 1) * 2 + gr) * R + row), none || ng >= kUnseen ? -INFINITY : kShift - ng);
            }
            warp_arrive(bar(tState + (si & 1)));
        }
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 88;" ::: "memory");
        // ------------------------------------------------- Q pieces, epilogues
        const int d = threadIdx.x - 256;  // the dim (TMEM lane) this thread writes out
        uint32_t help_phase = 0;
        int j_base = 0;  // tiles of the segments before
        bool ok = true;
        // Segment si's Q rows into its buffer: DH / 8 lanes a row, eight elements
        // a lane; rows of no token are zero.  A compact loop, and few instructions
        // a row: a helper warp shares its scheduler with two softmax warps and
        // gets one instruction in about eight cycles.
        auto build_q = [&](int si) -> bool {
            const Seg sg = load_seg(segs, seg_cache, si);
            const int buf = NQB == 2 ? si & 1 : 0;
            const int use = NQB == 2 ? si >> 1 : si;  // earlier uses of this buffer
            const int rows = min(R, sg.qo_len * g - sg.r0);
            constexpr int LPR = DH / 8, RPI = 32 / LPR;  // lanes a row, rows a warp's round
            const int e = lane % LPR, row0 = (warp - 8) * RPI + lane / LPR;
            const bool q1 = !k2 && p.q_pieces == 1;      // an fp8 query as it is
            const bool bf = p.q_dtype == PAFP8_BF16;
            const size_t head0 = (size_t)sg.qo0 * p.num_qo_heads + (size_t)sg.hk * g;
            const uint32_t dst = base + L.q + (uint32_t)(buf * p.q_pieces) * D::kQPiece;
            const uint32_t fdst = base + L.sc + (uint32_t)((si & 1) * R) * 4u;
            const float ks = p.k_scales != nullptr ? __ldg(p.k_scales + sg.hk) : 0.f;
            constexpr int kBatch = 4;  // rows in flight per lane group
            bool ready = false;
#pragma unroll 1
            for (int first = row0; first - row0 < R; first += 4 * RPI * kBatch) {
                uint4 raw[kBatch];
#pragma unroll
                for (int k = 0; k < kBatch; ++k) {
                    const int row = first + 4 * RPI * k;
                    raw[k] = make_uint4(0, 0, 0, 0);
                    if (row < rows) {
                        const int tok = token_of(sg.r0 + row);
                        const size_t at = (head0 + (size_t)tok * p.num_qo_heads + (sg.r0 + row - tok * g)) * DH + 8 * e;
                        if (q1) {
                            const uint2 x = __ldg(reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(p.q) + at));
                            raw[k] = make_uint4(x.x, x.y, 0, 0);
                        } else {
                            raw[k] = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.q) + at));
                        }
                    }
                }
                if (!ready) {  // the buffer is free once its last segment's QK has run
                    if (!wait_idle(tQEmpty + buf, (uint32_t)((use + 1) & 1))) return false;
                    ready = true;
                }
#pragma unroll 1
                for (int k = 0; k < kBatch; ++k) {
                    const int row = first + 4 * RPI * k;
                    if (row - lane / LPR >= R) break;  // uniform: R is a multiple of a round's rows
                    const uint4 rw = k == 0 ? raw[0] : k == 1 ? raw[1] : k == 2 ? raw[2] : raw[3];
                    // log2 scale of this row's logits, but for the pieces' power of two.
                    float scale = p.sm_scale_log2;
                    if (p.k_scales != nullptr) {
                        const int n = sg.r0 + row, qh = sg.hk * g + (n - token_of(n) * g);
                        scale = fold_scale_log2(p.sm_scale, p.q_scales != nullptr ? __ldg(p.q_scales + qh) : 1.0f, ks);
                    }
                    if constexpr (k2) {
                        sts128(dst + (e >> 3) * (R * 128u) + row * 128u + (uint32_t)(((e & 7) ^ (row & 7)) << 4), rw.x, rw.y, rw.z,
                               rw.w);
                    } else {
                        // An eight-byte element group's place in a piece's tile row.
                        const uint32_t at = dst + (DH == 128 ? row * 128u + (uint32_t)(((e >> 1) ^ (row & 7)) << 4) + 8u * (e & 1)
                                                             : row * 64u + (uint32_t)(((e >> 1) ^ ((row >> 1) & 3)) << 4) + 8u * (e & 1));
                        if (q1) {
                            sts64(at, rw.x, rw.y);
                        } else {
                            const uint32_t w[4] = {rw.x, rw.y, rw.z, rw.w};
                            // The row's largest magnitude as a 16-bit pattern.
                            uint32_t top = __vmaxu2(__vmaxu2(w[0] & 0x7FFF7FFFu, w[1] & 0x7FFF7FFFu),
                                                    __vmaxu2(w[2] & 0x7FFF7FFFu, w[3] & 0x7FFF7FFFu));
                            top = max(top & 0xFFFFu, top >> 16);
#pragma unroll
                            for (int x = LPR / 2; x > 0; x >>= 1) top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, x));
                            const float amax = bf ? __uint_as_float(top << 16) : __half2float(__ushort_as_half((unsigned short)top));
                            // 2^ex brings the largest magnitude into [128, 256).  A row with an
                            // infinity or a NaN gives NaN, as its logits would.
                            const int up = 7 - ((int)((__float_as_uint(amax) >> 23) & 0xFFu) - 127);
                            const int ex = amax == 0.f ? 0 : max(-120, min(100, up));
                            const float mul = __uint_as_float((uint32_t)(127 + ex) << 23);
                            scale *= isfinite(amax) ? __uint_as_float((uint32_t)(127 - ex) << 23) : __uint_as_float(0x7FC00000u);
                            // In f16 from here on: below 2^8 it holds bf16's 8 bits and its own
                            // 11 down to 2^-14, and the differences are exact.
                            __half2 h[4];
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                float2 f;
                                if (bf)
                                    f = make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u));
                                else
                                    f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
                                h[i] = __floats2half2_rn(f.x * mul, f.y * mul);
                            }
#pragma unroll 1
                            for (int pc = 0; pc < p.q_pieces; ++pc) {
                                uint32_t pr[4];
#pragma unroll
                                for (int i = 0; i < 4; ++i) {
                                    pr[i] = e4m3_of_half2(h[i]);
                                    h[i] = __hsub2(h[i], half2_of_e4m3(pr[i]));
                                }
                                sts64(at + pc * D::kQPiece, prmt(pr[0], pr[1], 0x5410u), prmt(pr[2], pr[3], 0x5410u));
                            }
                        }
                    }
                    // A scale that underflows to zero would turn -inf (unseen) into NaN.
                    if (e == 0) sts_f(fdst + 4u * row, scale < 1.2e-38f ? 1.2e-38f : scale);
                }
            }
            fence_async_smem();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(bar(tQFull + buf));
                mbar_arrive(bar(tInfo + (si & 1)));
            }
            return true;
        };
        for (int sq = 0; sq <= n_seg && n_seg > 0; ++sq) {  // Q of segment sq, epilogue of the one before
            if (sq < n_seg && !(ok = build_q(sq))) break;
            if (sq == 0) continue;
            const int si = sq - 1;
            const Seg sg = load_seg(segs, seg_cache, si);
            const int ob = si % NOB;
            const int rows = min(R, sg.qo_len * g - sg.r0);
            const bool whole = sg.slot < 0;
            const float vsc = p.v_scales != nullptr ? __ldg(p.v_scales + sg.hk) : p.v_scale;
            const size_t head0 = (size_t)sg.qo0 * p.num_qo_heads + (size_t)sg.hk * g;
            const size_t prow0 = (size_t)max(sg.slot, 0) * p.rows_pad;
            const uint32_t wt = base + L.wt + (uint32_t)((si & 1) * 2 * R) * 4u, rowp = base + L.rowp + (uint32_t)((si & 1) * R) * 8u;
            if (!(ok = wait_idle(tState + (si & 1), (uint32_t)((si >> 1) & 1)))) break;
            if (d < R) {
                // Row d: the groups' states joined, M and L at it, and each group's weight.
                float m[2], sum[2] = {0.f, 0.f};
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    m[i] = lds_f(base + L.mst + 4u * (((si & 1) * 2 + i) * R + d));
#pragma unroll
                    for (int w = 0; w < 4; ++w) sum[i] += lds_f(base + L.lsum + 4u * (((si & 1) * 8 + 4 * i + w) * R + d));
                }
                const float M = fmaxf(m[0], m[1]), m0 = M == -INFINITY ? 0.f : M;
                const float f0 = ex2(m[0] - m0), f1 = ex2(m[1] - m0);
                // (an empty state counts for nothing; a NaN sum stays one)
                const float L2 = (sum[0] == 0.f ? 0.f : f0 * sum[0]) + (sum[1] == 0.f ? 0.f : f1 * sum[1]);
                const float w = L2 == 0.f ? 0.f : (whole ? vsc : 1.f) / L2;
                sts_f(wt + 4u * d, sum[0] == 0.f ? 0.f : f0 * w);
                sts_f(wt + 4u * (R + d), sum[1] == 0.f ? 0.f : f1 * w);
                const int tok = token_of(sg.r0 + d);
                const size_t orow = head0 + (size_t)tok * p.num_qo_heads + (sg.r0 + d - tok * g);
                const uint64_t at = (uint64_t)orow * (DH * 2);  // the row's place in o, in bytes
                asm volatile("st.shared.b64 [%0], %1;" ::"r"(rowp + 8u * d), "l"(at) : "memory");
                if (d < rows) {
                    const float lse2 = L2 == 0.f ? -INFINITY : M - kShift + __log2f(L2);
                    if (!whole)
                        p.part_lse[prow0 + d] = lse2;
                    else if (p.lse != nullptr)
                        p.lse[orow] = lse2 * 0.69314718055994531f;
                }
            }
            warp_arrive(bar(tHelp));
            if (!(ok = wait_all(tHelp, help_phase))) break;
            help_phase ^= 1u;
            if (!(ok = wait_all(tOFull + ob, (uint32_t)((si / NOB) & 1)))) break;
            tc_fence_after();
            const uint32_t tO = tmem + ((uint32_t)(32 * (warp & 3)) << 16) + D::kColO + (uint32_t)(2 * D::OC * ob);
            // Rows eight at a time, a warp writing 32 dims of each: 64 bytes of o, or
            // 128 of a partial state.  Rows in pairs (packed fp32).
            const bool both = sg.tile1 - sg.tile0 > 1;  // else one group's accumulator holds anything
            const int g0 = j_base & 1;                  // the group of the segment's first tile
            j_base += sg.tile1 - sg.tile0;
            uint8_t* const o_base = static_cast<uint8_t*>(p.o) + 2 * d;
            float* part = p.part_o + prow0 * DH + d;
            const f32x2 fold = make_f32x2(1.f / 32.f, 1.f / 32.f);
#pragma unroll 1
            for (int r0 = 0; r0 < rows; r0 += 8) {
                float o[8], o1[8];
                {
                    float lo[8], lo1[8];
                    tc_ld8(tO + D::OC * g0 + r0, reinterpret_cast<uint32_t(&)[8]>(o));
                    if constexpr (D::kTwo) tc_ld8(tO + D::OC * g0 + R + r0, reinterpret_cast<uint32_t(&)[8]>(lo));
                    if (both) {
                        tc_ld8(tO + D::OC * (g0 ^ 1) + r0, reinterpret_cast<uint32_t(&)[8]>(o1));
                        if constexpr (D::kTwo) tc_ld8(tO + D::OC * (g0 ^ 1) + R + r0, reinterpret_cast<uint32_t(&)[8]>(lo1));
                    }
                    tc_wait_ld();
                    if (r0 + 8 >= rows) {  // O is read: another segment may write the accumulators
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) {
                            mbar_arrive(bar(tOEmpty + 2 * ob));
                            mbar_arrive(bar(tOEmpty + 2 * ob + 1));
                        }
                    }
                    if (DH == 64 && d >= 64) continue;
                    const uint32_t wa = wt + 4u * (g0 * R + r0), wb = wt + 4u * ((g0 ^ 1) * R + r0);
#pragma unroll
                    for (int k = 0; k < 8; k += 4) {
                        const float4 w = lds_f4(wa + 4u * k);
                        f32x2 x = make_f32x2(o[k], o[k + 1]), y = make_f32x2(o[k + 2], o[k + 3]);
                        if constexpr (D::kTwo) {
                            x = fma2(make_f32x2(lo[k], lo[k + 1]), fold, x);
                            y = fma2(make_f32x2(lo[k + 2], lo[k + 3]), fold, y);
                        }
                        x = mul2(x, make_f32x2(w.x, w.y));
                        y = mul2(y, make_f32x2(w.z, w.w));
                        if (both) {
                            const float4 u = lds_f4(wb + 4u * k);
                            f32x2 x1 = make_f32x2(o1[k], o1[k + 1]), y1 = make_f32x2(o1[k + 2], o1[k + 3]);
                            if constexpr (D::kTwo) {
                                x1 = fma2(make_f32x2(lo1[k], lo1[k + 1]), fold, x1);
                                y1 = fma2(make_f32x2(lo1[k + 2], lo1[k + 3]), fold, y1);
                            }
                            x = fma2(x1, make_f32x2(u.x, u.y), x);
                            y = fma2(y1, make_f32x2(u.z, u.w), y);
                        }
                        split_f32x2(x, o[k], o[k + 1]);
                        split_f32x2(y, o[k + 2], o[k + 3]);
                    }
                }
                const int n = rows - r0;
                if (whole) {
#pragma unroll
                    for (int k = 0; k < 8; k += 2) {
                        const uint32_t v2 = pack_out2(o[k], o[k + 1], p.o_dtype);
                        const uint4 at = lds128(rowp + 8u * (r0 + k));  // two rows' places
                        if (k < n) *reinterpret_cast<uint16_t*>(o_base + (((uint64_t)at.y << 32) | at.x)) = (uint16_t)v2;
                        if (k + 1 < n) *reinterpret_cast<uint16_t*>(o_base + (((uint64_t)at.w << 32) | at.z)) = (uint16_t)(v2 >> 16);
                    }
                } else {
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        if (k < n) part[k * DH] = o[k];
                    part += 8 * DH;
                }
            }
        }
    }

    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (warp == 13) {
        tc_fence_after();
        tc_dealloc(tmem, D::kCols);
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
    const int4 a = __ldg(rec), b = __ldg(rec + 1);  // slot0, slot1, the request's first token, hk; rows, first row
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
    const int tok = (b.y + row) / p.group, hh = b.y + row - tok * p.group;
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

template <int KT, int NP, int DH, int R>
cudaError_t launch_tree_t(TreeParams p, const CUtensorMap& tk, const CUtensorMap& tv, int num_ctas, int num_merge,
                          cudaStream_t stream) {
    using D = TreeDims<KT, NP, DH, R>;
    const TreeRing ring = tree_ring<D, R, NP>(p.q_pieces);
    p.q_buffers = ring.q_buffers;
    p.stages = ring.stages;
    const size_t smem = 1024 + tree_smem<D, R, NP>(p.q_buffers * p.q_pieces, p.stages).bytes;
    if (smem > 232448) return cudaErrorInvalidValue;
    auto kern = tree_kernel<KT, NP, DH, R>;
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

template <int DH, int R>
cudaError_t launch_tree_rows(const TreeParams& p, const CUtensorMap& tk, const CUtensorMap& tv, int num_ctas,
                             int num_merge, cudaStream_t stream) {
    switch (p.kv_dtype) {
        case PAFP8_F16: return launch_tree_t<PAFP8_F16, 1, DH, R>(p, tk, tv, num_ctas, num_merge, stream);
        case PAFP8_BF16: return launch_tree_t<PAFP8_BF16, 1, DH, R>(p, tk, tv, num_ctas, num_merge, stream);
        default: break;
    }
    // An f16 output keeps 11 bits: three pieces of P.
    return p.o_dtype == PAFP8_F16 ? launch_tree_t<PAFP8_E4M3FN, 3, DH, R>(p, tk, tv, num_ctas, num_merge, stream)
                                  : launch_tree_t<PAFP8_E4M3FN, 2, DH, R>(p, tk, tv, num_ctas, num_merge, stream);
}

}  // namespace
}  // namespace pafp8
