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
// A request's new tokens are contiguous, so one warp owns a (block, head, K or
// V): no atomics, and the result is a function of the inputs.  The warp keeps
// the block's 16 rows in registers between the maximum and the conversion, so
// the source is read once.
//
// Reading.  Rows out_indptr[b] .. out_indptr[b + 1] - 1 are tokens starts[b]
// on of request b, as fp32(code) * scale rounded once to the output's type.
//
// Both are streams, bounded by HBM, and by launch and table lookups for a few
// tokens.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "../../include/pafp8.h"
#include "internal.h"
#include "ptx.cuh"

namespace pafp8 {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr uint32_t kAll = 0xFFFFFFFFu;

// The request that owns row t, by one warp together: the last r with
// indptr[r] <= t (32 probes a step; indptr[0] <= t < indptr[n] by the caller's
// check).  Every index probed lies in (0, n).
__device__ __forceinline__ int owner(const int32_t* indptr, int n, long long t) {
    const int lane = threadIdx.x & 31;
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int step = (hi - lo + 31) / 32;
        const long long at = (long long)lo + (long long)(lane + 1) * step;
        const bool below = at < hi && __ldg(indptr + at) <= t;
        const uint32_t b = __ballot_sync(kAll, below);
        const int steps = b == kAll ? 32 : __ffs(~b) - 1;
        lo += steps * step;
        hi = min(hi, lo + step);
    }
    return lo;
}

// Where token `pos` of request r lies: its page and the slot in it, or page -1
// when the position or the page id is out of range.
__device__ __forceinline__ int page_of(const int32_t* kv_indptr, const int32_t* kv_indices, int r, long long pos,
                                       int page_size, int num_pages, int& slot) {
    if (pos < 0) return -1;
    const int e0 = __ldg(kv_indptr + r), e1 = __ldg(kv_indptr + r + 1);
    const long long e = e0 + pos / page_size;
    slot = (int)(pos % page_size);
    if (e0 < 0 || e >= e1) return -1;
    const int pg = __ldg(kv_indices + e);
    return pg >= 0 && pg < num_pages ? pg : -1;
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
    uint32_t h[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) h[i] = cvt_pair<KV>(__fmul_rn(x[2 * i], by), __fmul_rn(x[2 * i + 1], by));
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

// One warp per (group of p.span new tokens, KV head, K or V): it takes the
// blocks whose first new token lies in its group, one after the other.
template <int SRC, int KV, int DH>
__global__ void __launch_bounds__(kThreads) append_blocks_kernel(const BlockAppendParams p) {
    constexpr int LPR = DH / 8;       // lanes per row
    constexpr int RPP = 32 / LPR;     // rows per pass
    constexpr int NP = kPageSize / RPP;
    constexpr int ESZ = SRC == PAFP8_F32 ? 4 : 2;
    const int lane = threadIdx.x & 31;
    const int sub = lane / LPR, col = (lane % LPR) * 8;
    const long long all = __ldg(p.qo_indptr + p.batch);
    const long long rows = min(p.nnz, all);
    if (all > p.nnz && blockIdx.x == 0 && threadIdx.x == 0 && p.status != nullptr) atomicOr(p.status, kStatusBounds);
    const long long first_row = __ldg(p.qo_indptr);
    const long long units = (rows + p.span - 1) / p.span * (2 * p.num_kv_heads);
    for (long long u = (long long)blockIdx.x * kWarps + (threadIdx.x >> 5); u < units; u += (long long)gridDim.x * kWarps) {
        const long long group = u / (2 * p.num_kv_heads);
        const int hv = (int)(u - group * (2 * p.num_kv_heads));
        const bool is_v = hv >= p.num_kv_heads;
        const int h = is_v ? hv - p.num_kv_heads : hv;
        const uint8_t* const src = static_cast<const uint8_t*>(is_v ? p.v : p.k) + ((size_t)h * DH + col) * ESZ;
        const size_t stride = (size_t)(is_v ? p.v_stride : p.k_stride) * ESZ;
        uint8_t* const cache = static_cast<uint8_t*>(is_v ? p.v_cache : p.k_cache);
        float* const scales = is_v ? p.v_scales : p.k_scales;
        long long t = max(group * p.span, first_row);
        const long long t_end = min((group + 1) * p.span, rows);
        if (t >= t_end) continue;
        int r = owner(p.qo_indptr, p.batch, t);
        while (t < t_end) {
            const long long r0 = __ldg(p.qo_indptr + r), r1 = min((long long)__ldg(p.qo_indptr + r + 1), rows);
            if (t >= r1) {  // (requests without new tokens lie in between)
                if (++r >= p.batch) break;
                continue;
            }
            const int cached = __ldg(p.cached_lens + r);
            const long long pos = (long long)cached + (t - r0);
            const int s0 = (int)(pos & (kPageSize - 1));
            const int m = (int)min((long long)(kPageSize - s0), r1 - t);
            if (s0 != 0 && t != r0) {  // the block belongs to an earlier token's warp
                t += m;
                continue;
            }
            // The new rows: slots s0 .. s0 + m - 1 of the block.
            Raw8<SRC> raw[NP];
#pragma unroll
            for (int i = 0; i < NP; ++i) {
                const int s = i * RPP + sub - s0;
#pragma unroll
                for (int k = 0; k < Raw8<SRC>::kVecs; ++k) raw[i].v[k] = make_uint4(0u, 0u, 0u, 0u);
                if (s >= 0 && s < m) {
                    const uint4* g = reinterpret_cast<const uint4*>(src + (size_t)(t + s) * stride);
#pragma unroll
                    for (int k = 0; k < Raw8<SRC>::kVecs; ++k) raw[i].v[k] = __ldcs(g + k);
                }
            }
            int slot = 0;
            const int page = cached < 0 ? -1 : page_of(p.kv_indptr, p.kv_indices, r, pos, p.page_size, p.num_pages, slot);
            t += m;
            if (page < 0) {
                if (lane == 0 && p.status != nullptr) atomicOr(p.status, kStatusBounds);
                continue;
            }
            slot -= s0;  // the block's first slot in the page
            float* const scale = scales + ((size_t)page * (p.page_size / kPageSize) + slot / kPageSize) * p.num_kv_heads + h;
            const float old = s0 != 0 ? *scale : 0.f;
            uint32_t amax = 0;
#pragma unroll
            for (int i = 0; i < NP; ++i) {
                float x[8];
                to_float8<SRC>(raw[i], x);
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const uint32_t a = __float_as_uint(x[k]) & 0x7FFFFFFFu;
                    amax = max(amax, a < 0x7F800000u ? a : 0u);
                }
            }
            amax = __reduce_max_sync(kAll, amax);
            const float own = power_scale<KV>(amax);
            const float s = s0 != 0 && old >= own ? old : own;
            const size_t row_bytes = p.hnd ? DH : (size_t)p.num_kv_heads * DH;
            uint8_t* const dst = cache + (p.hnd ? (((size_t)page * p.num_kv_heads + h) * p.page_size + slot) * DH
                                                : (((size_t)page * p.page_size + slot) * p.num_kv_heads + h) * DH) + col;
            if (s0 != 0 && s > old) {
                const float ratio = __fdiv_rn(old, s);
#pragma unroll
                for (int i = 0; i < NP; ++i) {
                    const int at = i * RPP + sub;
                    if (at < s0) {
                        uint2* const c = reinterpret_cast<uint2*>(dst + at * row_bytes);
                        float x[8];
                        values8<KV>(*c, x);
                        *c = codes8<KV>(x, ratio);
                    }
                }
            }
            const float inv = __fdiv_rn(1.0f, s);
#pragma unroll
            for (int i = 0; i < NP; ++i) {
                const int at = i * RPP + sub;
                if (at >= s0 && at < s0 + m) {
                    float x[8];
                    to_float8<SRC>(raw[i], x);
                    *reinterpret_cast<uint2*>(dst + at * row_bytes) = codes8<KV>(x, inv);
                }
            }
            if (lane == 0) *scale = s;
        }
    }
}

template <int SRC, int KV, int DH>
cudaError_t launch_append_t(BlockAppendParams p, cudaStream_t stream) {
    p.span = p.nnz <= 4LL * p.batch ? 1 : kPageSize;
    const long long units = (p.nnz + p.span - 1) / p.span * (2LL * p.num_kv_heads);
    const long long blocks = (units + kWarps - 1) / kWarps;
    append_blocks_kernel<SRC, KV, DH><<<(int)min(blocks, (long long)INT32_MAX), kThreads, 0, stream>>>(p);
    return cudaGetLastError();
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

constexpr int kReadRows = 16;  // rows of a thread block's tile

// One thread block per kReadRows output rows, all heads, K and V: the first
// warp looks the rows up, then every thread takes 16 codes at a time.
template <int OUT, int KV, int DH>
__global__ void __launch_bounds__(kThreads) read_kv_kernel(const ReadParams p) {
    constexpr int CPR = DH / 16;  // 16-code chunks of a row
    constexpr int ESZ = OUT == PAFP8_F32 ? 4 : 2;
    __shared__ long long s_row[kReadRows];    // byte offset of head 0's row in the cache, or -1
    __shared__ long long s_scale[kReadRows];  // index of head 0's scale
    const long long all = __ldg(p.out_indptr + p.batch);
    const long long rows = min(p.nnz, all);
    const long long t0 = (long long)blockIdx.x * kReadRows;
    if (all > p.nnz && blockIdx.x == 0 && threadIdx.x == 0 && p.status != nullptr) atomicOr(p.status, kStatusBounds);
    if (t0 >= rows) return;
    const long long head_step = p.hnd ? (long long)p.page_size * DH : DH;
    if (threadIdx.x < 32) {
        const int lane = threadIdx.x;
        const long long low = __ldg(p.out_indptr);
        const long long base = max(t0, low);
        const int r0 = base < rows ? owner(p.out_indptr, p.batch, base) : 0;
        const long long t = t0 + lane;
        if (lane < kReadRows) {
            long long row = -1, scale = 0;
            if (t >= low && t < rows) {
                int r = r0;
                while (r + 1 < p.batch && t >= __ldg(p.out_indptr + r + 1)) ++r;
                int slot = 0;
                const int start = __ldg(p.starts + r);
                const long long pos = (long long)start + (t - __ldg(p.out_indptr + r));
                const int page = start < 0 ? -1 : page_of(p.kv_indptr, p.kv_indices, r, pos, p.page_size, p.num_pages, slot);
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
    const int work = 2 * kReadRows * per_row;
    for (int i = threadIdx.x; i < work; i += kThreads) {
        const int kv = i / (kReadRows * per_row), j = i - kv * (kReadRows * per_row);
        const int row = j / per_row, c = j - row * per_row;
        const int h = c / CPR, d = (c - h * CPR) * 16;
        if (s_row[row] < 0) continue;
        const uint8_t* src = static_cast<const uint8_t*>(kv ? p.v_cache : p.k_cache) + s_row[row] + h * head_step + d;
        const float* scales = kv ? p.v_scales : p.k_scales;
        const float s = scales != nullptr ? __ldg(scales + s_scale[row] + h) : (kv ? p.v_scale : p.k_scale);
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
cudaError_t launch_read_t(const ReadParams& p, cudaStream_t stream) {
    read_kv_kernel<OUT, KV, DH><<<(unsigned)((p.nnz + kReadRows - 1) / kReadRows), kThreads, 0, stream>>>(p);
    return cudaGetLastError();
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
