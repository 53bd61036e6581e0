// blocks.cu -- the cache with a scale for each block of 16 tokens and KV head:
// quantizing tokens as they are written, and reading token ranges back.  sm_103a.
//
// Writing.  A block of 16 token slots of one KV head holds fp8 codes of
// x / s under one scale s.  s is a power of two: a floating-point code keeps
// its relative precision under any scale that avoids overflow and the type's
// subnormals, so a finer scale would gain nothing, and a block that grows by
// 2^k turns its earlier codes into themselves divided by 2^k, exactly but for
// subnormals.  With M the type's largest finite value and amax the largest
// finite magnitude among the new values of the block,
//   s_new  = the smallest power of two >= 2^-64 with amax <= M s_new
//   s      = s_new in a block that the step begins, max(s_old, s_new) in one
//            that holds tokens of earlier steps
//   code   = fp8(RNE, saturating)(x * fp32(1 / s))
//   code'  = fp8(RNE)(code * fp32(s_old / s)) for those tokens, if s > s_old.
// A request's new tokens are contiguous, so one warp owns a block of K or V of
// one head (of two heads of 64): no atomics, and the result is a function of the
// inputs.  The warp keeps the block's 16 rows in shared memory (fp32 rows in
// registers) between the maximum and the conversion, so the source is read once.
//
// Reading.  Rows out_indptr[b] .. out_indptr[b + 1] - 1 are tokens starts[b]
// on of request b, as fp32(code) * scale rounded once to the output's type.
//
// Both are streams, bounded by HBM, and by launch and table lookups for a few
// tokens.  Measured in a graph, inputs of three steps in turn: the append of 16
// ragged prompts (8 heads of 128, bf16 to e4m3fn, 45.7 MB) 11.8 us, 57 % of the
// measured copy rate, of 64 such prompts (206 MB) 35.7 us, 85 %: a warp waits for
// its request (32 probes of qo_indptr a step), lengths and page before its rows,
// which few calls are long enough to hide.  One warp for K and V both takes a
// fourth longer; positions in 64 bits, whose divisions were a third of the
// instructions, 43.2 us with 64 prompts where 32 bits took 41.9.  64 single
// tokens take 3.8 us.  The read-back of 64 requests of 512-4096 tokens (891 MB)
// takes 138 us, 95 % of the copy rate.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <type_traits>

#include "../../include/pafp8.h"
#include "internal.h"
#include "ptx.cuh"

namespace pafp8 {
namespace {

constexpr int kThreads = 256;
constexpr int kAppendThreads = 128;
constexpr int kAppendBlocks = 8;  // thread blocks an SM, for 64 registers a thread (fp32 rows: 3, for 168)
constexpr uint32_t kAll = 0xFFFFFFFFu;

// Both kernels are launched early (launch_dependent below).
template <typename T>
__device__ __forceinline__ T now(const T* p) {
    return load_input<true>(p);
}

// The request that owns row t, by one warp together: the last r with
// indptr[r] <= t (32 probes a step; any r for a t outside the rows), and the
// rows it starts and ends at.  Every index probed lies in (0, n), n >= 1.
struct Owner {
    int r, begin, end;
};
__device__ __forceinline__ Owner owner(const int32_t* indptr, int n, int t) {
    const int lane = threadIdx.x & 31;
    int lo = 0, hi = n, at_lo = now(indptr), at_hi = now(indptr + n);
    while (hi - lo > 1) {
        const int step = (hi - lo + 31) / 32;
        const uint32_t at = (uint32_t)lo + (uint32_t)(lane + 1) * (uint32_t)step;
        const int v = at < (uint32_t)hi ? now(indptr + at) : 0;
        const uint32_t b = __ballot_sync(kAll, at < (uint32_t)hi && v <= t);
        const int steps = b == kAll ? 32 : __ffs(~b) - 1;
        const int below = __shfl_sync(kAll, v, max(steps - 1, 0)), above = __shfl_sync(kAll, v, min(steps, 31));
        if (steps > 0) at_lo = below;
        if (steps < 32 && (uint32_t)lo + (uint32_t)(steps + 1) * (uint32_t)step < (uint32_t)hi) at_hi = above;
        lo += steps * step;
        hi = min(hi, lo + step);
    }
    return Owner{lo, at_lo, at_hi};
}

// Where token `pos` of the request with page entries e0 .. e1 - 1 lies: its
// page and the slot in it, or page -1 when the position or the page id is out
// of range.
__device__ __forceinline__ int page_of(const int32_t* kv_indices, int e0, int e1, uint32_t pos, int page_size, int num_pages,
                                       int& slot) {
    const uint32_t at = pos / (uint32_t)page_size;  // (at most 2^28, so that e0 + at does not wrap)
    slot = (int)(pos - at * (uint32_t)page_size);
    const uint32_t e = (uint32_t)e0 + at;
    if (e0 < 0 || e1 < 0 || e >= (uint32_t)e1) return -1;
    const int pg = now(kv_indices + e);
    return pg >= 0 && pg < num_pages ? pg : -1;
}

// Both kernels wait for the stream's work before them themselves, so that the
// launch passes under that work (16 prompts' appends one after the other, without
// a graph, 14.3 us each where this takes 11.9; the read-back of 64 requests 139.4
// and 137.2).
template <typename P>
cudaError_t launch_dependent(void (*kern)(P), unsigned blocks, int threads, const P& p, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(blocks);
    cfg.blockDim = dim3((unsigned)threads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, p);
}

// ------------------------------------------------------------------ writing

// Eight elements of a row.
template <int SRC>
struct Raw8 {
    static constexpr int kVecs = SRC == PAFP8_F32 ? 2 : 1;
    uint4 v[kVecs];
};

template <int SRC>
__device__ __forceinline__ void to_float8(const Raw8<SRC>& r, float (&x)[8]) {
    const uint32_t w[8] = {r.v[0].x, r.v[0].y, r.v[0].z, r.v[0].w, r.v[Raw8<SRC>::kVecs - 1].x, r.v[Raw8<SRC>::kVecs - 1].y,
                           r.v[Raw8<SRC>::kVecs - 1].z, r.v[Raw8<SRC>::kVecs - 1].w};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        if constexpr (SRC == PAFP8_F32)
            x[i] = __uint_as_float(w[i]);
        else if constexpr (SRC == PAFP8_BF16)
            x[i] = __uint_as_float((i & 1) ? (w[i >> 1] & 0xFFFF0000u) : (w[i >> 1] << 16));
        else
            x[i] = __half2float(__ushort_as_half((unsigned short)(w[i >> 1] >> (16 * (i & 1)))));
    }
}

// Codes of (lo, hi): lo in the low byte.
template <int KV>
__device__ __forceinline__ uint32_t cvt_pair(float lo, float hi) {
    unsigned short d;
    if constexpr (KV == PAFP8_E4M3FN)
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(d) : "f"(hi), "f"(lo));
    else
        asm("cvt.rn.satfinite.e5m2x2.f32 %0, %1, %2;" : "=h"(d) : "f"(hi), "f"(lo));
    return d;
}

template <int KV>
__device__ __forceinline__ uint2 codes8(const float (&x)[8], float by) {
    const ptx::f32x2 by2 = ptx::make_f32x2(by, by);
    uint32_t h[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float lo, hi;
        ptx::split_f32x2(ptx::mul2(ptx::make_f32x2(x[2 * i], x[2 * i + 1]), by2), lo, hi);
        h[i] = cvt_pair<KV>(lo, hi);
    }
    return make_uint2(h[0] | (h[1] << 16), h[2] | (h[3] << 16));
}

// Eight codes as floats (exact).
template <int KV>
__device__ __forceinline__ void values8(uint2 c, float (&x)[8]) {
    const uint32_t w[2] = {c.x, c.y};
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint32_t lo = ptx::fp8x2_lo<KV>(w[i]), hi = ptx::fp8x2_hi<KV>(w[i]);
        const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&lo));
        const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&hi));
        x[4 * i] = a.x, x[4 * i + 1] = a.y, x[4 * i + 2] = b.x, x[4 * i + 3] = b.y;
    }
}

// The block's own scale from the bits of its largest magnitude: 448 = 1.75 * 2^8
// and 57344 = 1.75 * 2^15 are the types' largest values.
template <int KV>
__device__ __forceinline__ float power_scale(uint32_t amax) {
    const int e = (int)(amax >> 23) - 127 - (KV == PAFP8_E4M3FN ? 8 : 15) + ((amax & 0x7FFFFFu) > 0x600000u ? 1 : 0);
    return __uint_as_float((uint32_t)(max(e, -64) + 127) << 23);
}

// A block's rows of K or V in one warp: lane l holds dims 8 (l % 16) .. + 7 (of
// 128: one head of 128, or two of 64) of rows 2 i + l / 16.  Rows of earlier
// tokens hold their 8 codes, new rows their elements.
//
// Rows of a 2-byte type go through shared memory by asynchronous copies, 16
// bytes of which each lane writes and reads alone: 64 registers a thread, so 32
// warps an SM with their rows in flight.  64 ragged prompts (8 heads of 128)
// take 36.3 us where rows in registers (80 a thread, 24 warps) take 41.9, 512
// single tokens 8.9 and 9.9, 16 prompts 12.4 and 11.8.  fp32 rows, twice the
// bytes a lane, stay in registers: 15.9 us for 16 prompts against 23.5.
constexpr int kRowsPerPass = 2, kPasses = kPageSize / kRowsPerPass;

template <int SRC>
struct InShared {
    static constexpr int kBytes = kPasses * 512;  // of a warp
    uint32_t buf;                                 // this lane's first 16 bytes
    __device__ __forceinline__ void fetch(int i, const uint4* g) {
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(buf + i * 512), "l"(g) : "memory");
    }
    __device__ __forceinline__ void fetch_codes(int i, const uint2* g) {
        asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(buf + i * 512), "l"(g) : "memory");
    }
    __device__ __forceinline__ void clear(int i) { ptx::sts128(buf + i * 512, 0u, 0u, 0u, 0u); }
    __device__ __forceinline__ void wait() { asm volatile("cp.async.wait_all;" ::: "memory"); }
    __device__ __forceinline__ Raw8<SRC> row(int i) const { return Raw8<SRC>{{ptx::lds128(buf + i * 512)}}; }
    __device__ __forceinline__ uint2 codes(int i) const { return ptx::lds64(buf + i * 512); }
};

template <int SRC>
struct InRegisters {
    static constexpr int kBytes = 0;
    Raw8<SRC> raw[kPasses];
    __device__ __forceinline__ void fetch(int i, const uint4* g) {
#pragma unroll
        for (int k = 0; k < Raw8<SRC>::kVecs; ++k) raw[i].v[k] = __ldcs(g + k);
    }
    __device__ __forceinline__ void fetch_codes(int i, const uint2* g) {
        const uint2 c = *g;
        raw[i].v[0].x = c.x;
        raw[i].v[0].y = c.y;
    }
    __device__ __forceinline__ void clear(int i) { raw[i] = Raw8<SRC>{}; }
    __device__ __forceinline__ void wait() {}
    __device__ __forceinline__ Raw8<SRC> row(int i) const { return raw[i]; }
    __device__ __forceinline__ uint2 codes(int i) const { return make_uint2(raw[i].v[0].x, raw[i].v[0].y); }
};

template <int SRC>
using Rows = std::conditional_t<SRC == PAFP8_F32, InRegisters<SRC>, InShared<SRC>>;

// FULL: all 16 rows are new (nearly every block of a prompt), so that no row
// needs a condition of its own.
template <int SRC, bool FULL>
__device__ __forceinline__ void load_rows(Rows<SRC>& rows, const uint8_t* src, size_t stride, int s0, int m) {
    const int sub = (threadIdx.x & 31) / 16;
    const uint8_t* row = src + (ptrdiff_t)(sub - s0) * (ptrdiff_t)stride;
#pragma unroll
    for (int i = 0; i < kPasses; ++i, row += kRowsPerPass * stride) {
        const int s = i * kRowsPerPass + sub - s0;
        // (Rows of earlier tokens are read as codes alone, which load_codes brings.)
        if (FULL || (s >= 0 && s < m)) rows.fetch(i, reinterpret_cast<const uint4*>(row));
        else if (s >= m || Rows<SRC>::kBytes == 0) rows.clear(i);
    }
}

template <int SRC>
__device__ __forceinline__ void load_codes(Rows<SRC>& rows, const uint8_t* dst, size_t row_bytes, int s0) {
    const int sub = (threadIdx.x & 31) / 16;
#pragma unroll
    for (int i = 0; i < kPasses; ++i) {
        const int at = i * kRowsPerPass + sub;
        if (at < s0) rows.fetch_codes(i, reinterpret_cast<const uint2*>(dst + at * row_bytes));
    }
}

// The bits (as fp32) of this lane's largest finite magnitude among the new rows.
template <int SRC, bool FULL>
__device__ __forceinline__ uint32_t largest(const Rows<SRC>& rows, int s0) {
    const int sub = (threadIdx.x & 31) / 16;
    constexpr uint32_t kInf = SRC == PAFP8_F32 ? 0x7F800000u : SRC == PAFP8_BF16 ? 0x7F80u : 0x7C00u;
    uint32_t top = 0;  // (the maximum of a number and a NaN is the number)
#pragma unroll
    for (int i = 0; i < kPasses; ++i) {
        const Raw8<SRC> raw = rows.row(i);
#pragma unroll
        for (int k = 0; k < Raw8<SRC>::kVecs; ++k) {
            const uint32_t w[4] = {raw.v[k].x, raw.v[k].y, raw.v[k].z, raw.v[k].w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const uint32_t x = FULL || i * kRowsPerPass + sub >= s0 ? w[j] : 0u;
                if constexpr (SRC == PAFP8_F32) {
                    top = __float_as_uint(fmaxf(__uint_as_float(top), fabsf(__uint_as_float(x))));
                } else if constexpr (SRC == PAFP8_BF16) {
                    const __nv_bfloat162 r = __hmax2(*reinterpret_cast<const __nv_bfloat162*>(&top),
                                                     __habs2(*reinterpret_cast<const __nv_bfloat162*>(&x)));
                    top = *reinterpret_cast<const uint32_t*>(&r);
                } else {
                    const __half2 r = __hmax2(*reinterpret_cast<const __half2*>(&top), __habs2(*reinterpret_cast<const __half2*>(&x)));
                    top = *reinterpret_cast<const uint32_t*>(&r);
                }
            }
        }
    }
    uint32_t best = SRC == PAFP8_F32 ? top : max(top & 0xFFFFu, top >> 16);
    if (best >= kInf) {  // infinities do not count: once more without them
        best = 0;
        constexpr int kUnroll = SRC == PAFP8_F32 ? kPasses : 1;  // (rows in registers need constant indices)
#pragma unroll kUnroll
        for (int i = 0; i < kPasses; ++i) {
            float x[8];
            to_float8<SRC>(rows.row(i), x);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const uint32_t a = __float_as_uint(x[k]) & 0x7FFFFFFFu;
                if ((FULL || i * kRowsPerPass + sub >= s0) && a < 0x7F800000u) best = max(best, a);
            }
        }
        return best;
    }
    if constexpr (SRC == PAFP8_F32) return best;
    else if constexpr (SRC == PAFP8_BF16) return best << 16;
    else return __float_as_uint(__half2float(__ushort_as_half((unsigned short)best)));
}

// Scale, earlier codes and new codes of the block whose rows are loaded (new
// ones: slots s0 .. s0 + m - 1).  dst: this lane's dims of the block's first row.
template <int SRC, int KV, int DH, bool FULL>
__device__ __forceinline__ void write_rows(Rows<SRC>& rows, uint8_t* dst, size_t row_bytes, float* scale,
                                           float old, int s0, int m, bool active) {
    const int lane = threadIdx.x & 31, sub = lane / 16;
    rows.wait();
    uint32_t amax = largest<SRC, FULL>(rows, s0);
    if constexpr (DH == 128) {
        amax = __reduce_max_sync(kAll, amax);
    } else {  // lanes l and l ^ 8 hold different heads
#pragma unroll
        for (int off = 1; off < 32; off <<= 1)
            if (off != 8) amax = max(amax, __shfl_xor_sync(kAll, amax, off));
    }
    if (!active) return;
    const float own = power_scale<KV>(amax);
    const float s = !FULL && s0 != 0 && old >= own ? old : own;
    if (!FULL && s0 != 0 && s > old) {
        const float ratio = __fdiv_rn(old, s);
#pragma unroll
        for (int i = 0; i < kPasses; ++i) {
            const int at = i * kRowsPerPass + sub;
            if (at < s0) {
                float x[8];
                values8<KV>(rows.codes(i), x);
                *reinterpret_cast<uint2*>(dst + at * row_bytes) = codes8<KV>(x, ratio);
            }
        }
    }
    const float inv = __fdiv_rn(1.0f, s);
    uint8_t* row = dst + sub * row_bytes;
#pragma unroll
    for (int i = 0; i < kPasses; ++i, row += kRowsPerPass * row_bytes) {
        const int at = i * kRowsPerPass + sub;
        if (FULL || (at >= s0 && at < s0 + m)) {
            float x[8];
            to_float8<SRC>(rows.row(i), x);
            *reinterpret_cast<uint2*>(row) = codes8<KV>(x, inv);
        }
    }
    if (lane % (DH / 8) == 0 && lane < 16) *scale = s;
}

// One warp per (group of p.span new tokens, K or V, 128 / DH KV heads): it
// takes the blocks whose first new token lies in its group, one after the other.
// A block of a 2-byte source is 4 KB in flight a warp, of fp32 8 KB.
template <int SRC, int KV, int DH>
__global__ void __launch_bounds__(kAppendThreads, SRC == PAFP8_F32 ? 3 : kAppendBlocks)
    append_blocks_kernel(const BlockAppendParams p) {
    constexpr int HPW = 128 / DH;
    constexpr int ESZ = SRC == PAFP8_F32 ? 4 : 2;
    // Nothing is read or written before the stream's earlier work is complete.
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int lane = threadIdx.x & 31;
    const int col = 8 * (lane & 15);
    Rows<SRC> rows_of;
    if constexpr (SRC != PAFP8_F32) {
        __shared__ __align__(16) uint8_t held[kAppendThreads / 32][Rows<SRC>::kBytes];
        rows_of.buf = ptx::smem_addr(held[threadIdx.x >> 5]) + lane * 16;
    }
    const int head_groups = (p.num_kv_heads + HPW - 1) / HPW;
    const uint32_t u = blockIdx.x * (kAppendThreads / 32) + (threadIdx.x >> 5);
    const uint32_t group = u / (uint32_t)(2 * head_groups);
    const int part = (int)(u - group * (uint32_t)(2 * head_groups));
    const bool is_v = part >= head_groups;
    const int h = (is_v ? part - head_groups : part) * HPW + col / DH;  // this lane's head
    const bool active = h < p.num_kv_heads;
    // Rows are below 2^31, so that sums of two of them fit 32 unsigned bits.
    const uint32_t nnz = (uint32_t)p.nnz;
    uint32_t t = group * (uint32_t)p.span;
    if (t >= nnz || p.batch == 0) return;
    const uint32_t all = (uint32_t)max(0, now(p.qo_indptr + p.batch)), first_row = (uint32_t)max(0, now(p.qo_indptr));
    const Owner who = owner(p.qo_indptr, p.batch, (int)max(t, first_row));
    const uint32_t rows = min(nnz, all);
    if (all > nnz && u == 0 && lane == 0 && p.status != nullptr) atomicOr(p.status, kStatusBounds);
    const uint32_t t_end = min(t + (uint32_t)p.span, rows);
    t = max(t, first_row);
    int r = who.r;
    uint32_t r0 = (uint32_t)max(0, who.begin), r1 = min((uint32_t)max(0, who.end), rows);
    const uint8_t* const src = static_cast<const uint8_t*>(is_v ? p.v : p.k) + ((size_t)h * DH + col % DH) * ESZ;
    const size_t stride = (size_t)(is_v ? p.v_stride : p.k_stride) * ESZ;
    uint8_t* const cache = static_cast<uint8_t*>(is_v ? p.v_cache : p.k_cache);
    float* const scales = is_v ? p.v_scales : p.k_scales;
    while (t < t_end) {
        if (t >= r1) {  // (requests without new tokens lie in between)
            if (++r >= p.batch) break;
            r0 = (uint32_t)max(0, now(p.qo_indptr + r));
            r1 = min((uint32_t)max(0, now(p.qo_indptr + r + 1)), rows);
            continue;
        }
        const int cached = now(p.cached_lens + r), e0 = now(p.kv_indptr + r), e1 = now(p.kv_indptr + r + 1);
        const uint32_t pos = (uint32_t)cached + (t - r0);
        const int s0 = (int)(pos & (kPageSize - 1));
        const int m = (int)min((uint32_t)(kPageSize - s0), r1 - t);
        if (s0 != 0 && t != r0) {  // the block belongs to an earlier token's warp
            t += m;
            continue;
        }
        const uint8_t* const from = src + (size_t)t * stride;
        // (two heads of 64 a warp: the last warp of an odd count has one)
        const bool full = m == kPageSize && (DH == 128 || __all_sync(kAll, active));
        if (full)
            load_rows<SRC, true>(rows_of, from, stride, 0, kPageSize);
        else
            load_rows<SRC, false>(rows_of, from, stride, s0, active ? m : 0);
        int slot = 0;
        const int page = cached < 0 ? -1 : page_of(p.kv_indices, e0, e1, pos, p.page_size, p.num_pages, slot);
        t += m;
        if (page < 0) {
            rows_of.wait();
            if (lane == 0 && p.status != nullptr) atomicOr(p.status, kStatusBounds);
            continue;
        }
        slot -= s0;  // the block's first slot in the page
        float* const scale = scales + ((size_t)page * (p.page_size / kPageSize) + slot / kPageSize) * p.num_kv_heads + (active ? h : 0);
        const size_t row_bytes = p.hnd ? DH : (size_t)p.num_kv_heads * DH;
        uint8_t* const dst = cache + (p.hnd ? (((size_t)page * p.num_kv_heads + h) * p.page_size + slot) * DH
                                            : (((size_t)page * p.page_size + slot) * p.num_kv_heads + h) * DH) + col % DH;
        float old = 0.f;
        if (s0 != 0) {
            old = *scale;
            if (active) load_codes<SRC>(rows_of, dst, row_bytes, s0);
        }
        if (full)
            write_rows<SRC, KV, DH, true>(rows_of, dst, row_bytes, scale, 0.f, 0, kPageSize, true);
        else
            write_rows<SRC, KV, DH, false>(rows_of, dst, row_bytes, scale, old, s0, m, active);
    }
}

// A warp looks through `span` new tokens for its blocks: 16, which in a prompt
// hold one or two, or fewer where requests have fewer tokens each or where the
// call is so short that twice the warps are still at most 24 an SM, so that a
// decode step's requests go to a warp each rather than 16 to one in turn.  (64
// requests of 1-8 tokens 5.4 us, 16 tokens a warp 11.5; 256 of 4 tokens 6.7 and
// 11.4; one of 100 3.4 and 4.4.)  24 is a measure for either row size, not what
// is resident, 32 warps for 2-byte rows and 12 for fp32 ones: with these in its
// place 2-byte rows take the same (one request of 1000 tokens 3.8 us and 3.95
// with 32), fp32 rows mostly longer (64 requests of 1-8 5.0 and 5.65 with 12,
// one of 1000 4.1 and 4.35, two prompts 3.97 and 3.71, 16 the same 15.8).
constexpr long long kSpanWarps = 152 * 24;

template <int SRC, int KV, int DH>
cudaError_t launch_append_t(BlockAppendParams p, cudaStream_t stream) {
    constexpr int HPW = 128 / DH, W = kAppendThreads / 32;
    const long long parts = 2LL * ((p.num_kv_heads + HPW - 1) / HPW);
    p.span = kPageSize;
    while (p.span > 1 && (p.nnz < (long long)p.span * p.batch || p.nnz * parts * 2 <= kSpanWarps * p.span)) p.span /= 2;
    const long long units = (p.nnz + p.span - 1) / p.span * parts;
    const long long blocks = (units + W - 1) / W;
    if (blocks > INT32_MAX / W) return cudaErrorInvalidConfiguration;
    return launch_dependent(append_blocks_kernel<SRC, KV, DH>, (unsigned)blocks, kAppendThreads, p, stream);
}

template <int SRC, int KV>
cudaError_t launch_append_kv(const BlockAppendParams& p, cudaStream_t stream) {
    return p.head_dim == 64 ? launch_append_t<SRC, KV, 64>(p, stream) : launch_append_t<SRC, KV, 128>(p, stream);
}

template <int SRC>
cudaError_t launch_append_src(const BlockAppendParams& p, cudaStream_t stream) {
    return p.kv_dtype == PAFP8_E4M3FN ? launch_append_kv<SRC, PAFP8_E4M3FN>(p, stream)
                                      : launch_append_kv<SRC, PAFP8_E5M2>(p, stream);
}

// ------------------------------------------------------------------ reading

constexpr int kReadRows = 16;  // rows of a thread block's tile, at most

// One thread block per p.tile output rows, all heads, K and V: the first
// warp looks the rows up, then every thread takes 16 codes at a time.
template <int OUT, int KV, int DH>
__global__ void __launch_bounds__(kThreads) read_kv_kernel(const ReadParams p) {
    constexpr int CPR = DH / 16;  // 16-code chunks of a row
    constexpr int ESZ = OUT == PAFP8_F32 ? 4 : 2;
    __shared__ long long s_row[kReadRows];    // byte offset of head 0's row in the cache, or -1
    __shared__ long long s_scale[kReadRows];  // index of head 0's scale
    // Nothing is read or written before the stream's earlier work is complete.
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const long long all = now(p.out_indptr + p.batch);
    const long long rows = min(p.nnz, all);
    const long long t0 = (long long)blockIdx.x * p.tile;
    if (all > p.nnz && blockIdx.x == 0 && threadIdx.x == 0 && p.status != nullptr) atomicOr(p.status, kStatusBounds);
    if (t0 >= rows) return;
    const long long head_step = p.hnd ? (long long)p.page_size * DH : DH;
    if (threadIdx.x < 32) {
        const int lane = threadIdx.x;
        const long long low = now(p.out_indptr);
        const long long base = max(t0, low);
        const int r0 = base < rows ? owner(p.out_indptr, p.batch, (int)base).r : 0;
        const long long t = t0 + lane;
        if (lane < p.tile) {
            long long row = -1, scale = 0;
            if (t >= low && t < rows) {
                int r = r0;
                while (r + 1 < p.batch && t >= now(p.out_indptr + r + 1)) ++r;
                int slot = 0;
                const int start = now(p.starts + r);
                const long long pos = (long long)start + (t - now(p.out_indptr + r));
                const int page = start < 0 || pos > 0xFFFFFFFFLL
                                     ? -1
                                     : page_of(p.kv_indices, now(p.kv_indptr + r), now(p.kv_indptr + r + 1), (uint32_t)pos,
                                               p.page_size, p.num_pages, slot);
                if (page >= 0) {
                    row = p.hnd ? ((long long)page * p.num_kv_heads * p.page_size + slot) * DH
                                : ((long long)page * p.page_size + slot) * p.num_kv_heads * DH;
                    scale = ((long long)page * (p.page_size / kPageSize) + slot / kPageSize) * p.num_kv_heads;
                } else if (p.status != nullptr) {
                    atomicOr(p.status, kStatusBounds);
                }
            }
            s_row[lane] = row;
            s_scale[lane] = scale;
        }
    }
    __syncthreads();
    const int per_row = p.num_kv_heads * CPR;
    const int half = p.tile * per_row, work = 2 * half;
    for (int i = threadIdx.x; i < work; i += kThreads) {
        const int kv = i >= half, j = i - kv * half;
        const int row = j / per_row, c = j - row * per_row;
        const int h = c / CPR, d = (c - h * CPR) * 16;
        if (s_row[row] < 0) continue;
        const uint8_t* src = static_cast<const uint8_t*>(kv ? p.v_cache : p.k_cache) + s_row[row] + h * head_step + d;
        const float* scales = kv ? p.v_scales : p.k_scales;
        const float s = scales != nullptr ? now(scales + s_scale[row] + h) : (kv ? p.v_scale : p.k_scale);
        const uint4 w = __ldcs(reinterpret_cast<const uint4*>(src));
        float x[16];
        values8<KV>(make_uint2(w.x, w.y), reinterpret_cast<float(&)[8]>(x[0]));
        values8<KV>(make_uint2(w.z, w.w), reinterpret_cast<float(&)[8]>(x[8]));
#pragma unroll
        for (int k = 0; k < 16; ++k) x[k] = __fmul_rn(x[k], s);
        uint4* dst = reinterpret_cast<uint4*>(static_cast<uint8_t*>(kv ? p.v_out : p.k_out) +
                                              (((t0 + row) * p.num_kv_heads + h) * DH + d) * ESZ);
        if constexpr (OUT == PAFP8_F32) {
#pragma unroll
            for (int k = 0; k < 4; ++k)
                __stcs(dst + k, make_uint4(__float_as_uint(x[4 * k]), __float_as_uint(x[4 * k + 1]),
                                           __float_as_uint(x[4 * k + 2]), __float_as_uint(x[4 * k + 3])));
        } else {
            uint32_t o[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) o[k] = ptx::pack_out2(x[2 * k], x[2 * k + 1], OUT);
            __stcs(dst, make_uint4(o[0], o[1], o[2], o[3]));
            __stcs(dst + 1, make_uint4(o[4], o[5], o[6], o[7]));
        }
    }
}

template <int OUT, int KV, int DH>
cudaError_t launch_read_t(ReadParams p, cudaStream_t stream) {
    // A tile's lookups are waited for once, its rows streamed after them: few
    // rows go in small tiles over more thread blocks (about eight an SM), many
    // in tiles of 16.
    p.tile = 2;
    while (p.tile < kReadRows && p.nnz > 1216LL * p.tile) p.tile *= 2;
    return launch_dependent(read_kv_kernel<OUT, KV, DH>, (unsigned)((p.nnz + p.tile - 1) / p.tile), kThreads, p, stream);
}

template <int OUT>
cudaError_t launch_read_out(const ReadParams& p, cudaStream_t stream) {
    if (p.kv_dtype == PAFP8_E4M3FN)
        return p.head_dim == 64 ? launch_read_t<OUT, PAFP8_E4M3FN, 64>(p, stream)
                                : launch_read_t<OUT, PAFP8_E4M3FN, 128>(p, stream);
    return p.head_dim == 64 ? launch_read_t<OUT, PAFP8_E5M2, 64>(p, stream) : launch_read_t<OUT, PAFP8_E5M2, 128>(p, stream);
}

}  // namespace

cudaError_t launch_append_blocks(const BlockAppendParams& p, cudaStream_t stream) {
    switch (p.src_dtype) {
        case PAFP8_F16: return launch_append_src<PAFP8_F16>(p, stream);
        case PAFP8_BF16: return launch_append_src<PAFP8_BF16>(p, stream);
        case PAFP8_F32: return launch_append_src<PAFP8_F32>(p, stream);
        default: return cudaErrorInvalidValue;
    }
}

cudaError_t launch_read_kv(const ReadParams& p, cudaStream_t stream) {
    switch (p.out_dtype) {
        case PAFP8_F16: return launch_read_out<PAFP8_F16>(p, stream);
        case PAFP8_BF16: return launch_read_out<PAFP8_BF16>(p, stream);
        case PAFP8_F32: return launch_read_out<PAFP8_F32>(p, stream);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace pafp8
