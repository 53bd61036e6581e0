// rope.cu -- per-head RMS norm of queries and keys, rotary rotation and the
// append of keys and values to the paged cache, in one pass.  sm_103a.
//
// For every token and every q or k head, with x the head's D elements in fp32:
//   x'  = x * rsqrt(mean(x^2) + eps) * w                      (w NULL: x' = x)
//   pair i < R/2 of the first R dims (halves: dims i, i + R/2; neighbours:
//   dims 2i, 2i + 1) with c, s = cos_sin[pos][i], cos_sin[pos][R/2 + i]:
//   (y_a, y_b) = (a c - b s, b c + a s)
// where pos is the token's position on the pair's axis (pair_axis: time,
// height, width; one axis otherwise).  Queries are written out (fp8 ones as
// fp8(y * fp32(1 / q_scale))); keys, and values as they come, go to the
// cache slot of the token, an fp8 cache storing
// fp8(y * fp32(1 / scale)), rounded to nearest even and saturating, a 2-byte
// cache the value rounded once.  Nothing is rounded between the steps: the
// sum of squares, the norm and the rotation stay in fp32.
//
// The work is a stream of reads and writes ((Hq + 2 Hkv) D elements in,
// Hq D + 2 Hkv D out a token), but at 16 bytes a thread its instructions weigh
// as much as the bytes: HBM bandwidth leaves a warp time for about 160 while it
// moves eight elements a lane.  This takes about 100:
//   * a thread owns eight dims of a head, two quads R / 2 apart, so that a pair
//     lies in one thread and rotating needs no shuffle (as one octet a thread,
//     with eight shuffles a head, 8838 tokens of 32 + 2 x 8 heads of 128 dims
//     took 76 us);
//   * it keeps the same kHeads heads of one kind for all its tokens, so head
//     type, weights, output type and addresses are worked out once, and the
//     angles, slot and address of a token serve four heads;
//   * nothing branches on a loaded value around a shuffle, which the compiler
//     would have to guard lane by lane;
//   * with four heads a thread its eight 8-byte loads are in flight while
//     the token before is worked on: 16 warps an SM with 128 registers each
//     carry more of them than more warps with fewer heads.  8838 tokens took
//     39 us (30 at the copy rate), 32768 tokens 113 us (90); with two heads and
//     18 warps 45 and 135, with one and 32 warps 70 and 225; with four heads
//     and 18 warps, whose registers spill, 74 and 216.
// Decode steps are bound by latency (64 tokens: 6 us).
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>

#include "../../include/pafp8.h"
#include "internal.h"
#include "ptx.cuh"

namespace pafp8 {
namespace {

using namespace ptx;

constexpr int kWarps = 16;  // resident warps an SM
constexpr int kHeads = 4;   // of a thread

// Four 16-bit elements in fp32.
template <bool kBF>
__device__ __forceinline__ void widen4(const uint2& r, f32x2 (&x)[2]) {
    const uint32_t w[2] = {r.x, r.y};
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        if constexpr (kBF) {
            x[i] = make_f32x2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u));
        } else {
            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
            x[i] = make_f32x2(f.x, f.y);
        }
    }
}

// Four elements, rounded once to the 16-bit type.
template <bool kBF>
__device__ __forceinline__ void store_half(uint8_t* dst, const f32x2 (&x)[2]) {
    uint32_t w[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        float lo, hi;
        split_f32x2(x[i], lo, hi);
        if constexpr (kBF) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
            w[i] = *reinterpret_cast<const uint32_t*>(&h);
        } else {
            const __half2 h = __floats2half2_rn(lo, hi);
            w[i] = *reinterpret_cast<const uint32_t*>(&h);
        }
    }
    *reinterpret_cast<uint2*>(dst) = make_uint2(w[0], w[1]);
}

// Four fp8 codes of x * inv (the product rounded once in fp32).
template <bool kE4M3>
__device__ __forceinline__ void store_fp8(uint8_t* dst, const f32x2 (&x)[2], float inv) {
    const f32x2 inv2 = make_f32x2(inv, inv);
    uint16_t w[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        float lo, hi;
        split_f32x2(mul2(x[i], inv2), lo, hi);
        if constexpr (kE4M3)
            asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(w[i]) : "f"(hi), "f"(lo));
        else
            asm("cvt.rn.satfinite.e5m2x2.f32 %0, %1, %2;" : "=h"(w[i]) : "f"(hi), "f"(lo));
    }
    *reinterpret_cast<uint32_t*>(dst) = w[0] | ((uint32_t)w[1] << 16);
}

template <bool kBF, int DH, bool kPairs>  // kPairs: neighbouring dims rotate together
__global__ void __launch_bounds__(64, kWarps / 2) rope_kernel(const __grid_constant__ RopeParams p) {
    constexpr int TPR = DH / 8;  // threads per head
    const int g = blockIdx.y * blockDim.x + threadIdx.x, c = g % TPR, u = g / TPR;
    const int half = p.rot_dim >> 1;
    const bool turns = 8 * c < p.rot_dim;
    // This thread's two quads of dims; its pairs are 4 c .. 4 c + 3.
    const int da = !kPairs && turns ? 4 * c : 8 * c;
    const int db = !kPairs && turns ? half + 4 * c : 8 * c + 4;

    // Its heads: head .. head + n - 1 of the queries, the keys or the values.
    const int uq = (p.num_qo_heads + kHeads - 1) / kHeads, uk = (p.num_kv_heads + kHeads - 1) / kHeads;
    const bool is_q = u < uq, is_k = !is_q && u < uq + uk;
    const int head = kHeads * (is_q ? u : is_k ? u - uq : min(u - uq - uk, uk - 1));
    const int n = u < uq + 2 * uk ? (is_q ? p.num_qo_heads : p.num_kv_heads) - head : 0;  // its outputs
    const long long stride = is_q ? p.q_stride : is_k ? p.k_stride : p.v_stride;
    const int dtype = is_q ? p.q_out_dtype : p.kv_dtype;
    const bool e4m3 = dtype == PAFP8_E4M3FN, fp8 = e4m3 || dtype == PAFP8_E5M2;
    const float scale_inv = is_q ? p.q_inv : is_k ? p.k_inv : p.v_inv;

    const void* weight = is_q ? p.q_weight : is_k ? p.k_weight : nullptr;
    const bool norm = weight != nullptr;
    f32x2 wa[2], wb[2];
    wa[0] = wa[1] = wb[0] = wb[1] = make_f32x2(1.f, 1.f);
    if (norm) {
        widen4<kBF>(__ldg(reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(weight) + da)), wa);
        widen4<kBF>(__ldg(reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(weight) + db)), wb);
    }
    // Warps without a head to normalise skip that part; the shuffles in it need
    // the decision to be one of the whole warp.
    const bool norms = __shfl_sync(0xFFFFFFFFu, (int)__any_sync(0xFFFFFFFFu, norm && n > 0), 0) != 0;
    const bool rotates = turns && (is_q || is_k);
    // The axes of this thread's pairs, a byte each; one past the last axis
    // counts as the last.
    uint32_t axes = 0;
    if (rotates && p.pair_axis != nullptr) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            axes |= (uint32_t)min((int)__ldg(p.pair_axis + 4 * c + i), p.num_axes - 1) << (8 * i);
    }
    const int axis = axes & 0xFF;
    const bool one_axis = axes == (uint32_t)axis * 0x01010101u;
    const uint32_t rot = (uint32_t)p.rot_dim, limit = (uint32_t)p.max_position;
    const float* const cos_at = p.cos_sin + 4 * c;
    const float* const sin_at = cos_at + half;

    // What moves on from token to token is a pointer with its step, so that the
    // loop has no 64-bit products but the slot's.
    const long long tok0 = blockIdx.x, hop = gridDim.x;
    const uint16_t* src_a = static_cast<const uint16_t*>(is_q ? p.q : is_k ? p.k : p.v) + (long long)head * DH + tok0 * stride + da;
    const uint16_t* src_b = src_a + (db - da);
    const long long src_step = hop * stride;
    const long long* slot_at = p.slots + tok0;
    const int32_t* pos_at = p.positions + tok0;
    // Outputs: a query's row follows its token, a cached one its slot.  Offsets
    // in bytes; head_bytes from one head to the next.
    const uint32_t size = fp8 ? 1 : 2, row_bytes = (uint32_t)(is_q ? p.num_qo_heads : p.num_kv_heads) * DH * size;
    const uint32_t page_size = (uint32_t)p.page_size;
    const bool paged = !is_q && p.hnd;
    const size_t head_bytes = (paged ? (size_t)page_size : 1) * DH * size;
    uint8_t* dst = static_cast<uint8_t*>(is_q ? p.q_out : is_k ? p.k_cache : p.v_cache) + (size_t)head * head_bytes + da * size;
    if (is_q) dst += (size_t)tok0 * row_bytes;
    const uint32_t dst_b = (db - da) * size;
    const size_t dst_step = is_q ? (size_t)hop * row_bytes : 0;

    // The elements, the slot and the angles of a token are read while the one
    // before it is worked on, its position, on which the angles depend, one
    // token earlier still.
    uint32_t pos[3] = {0, 0, 0};
    auto load_pos = [&]() {
        pos[0] = (uint32_t)__ldg(pos_at);
        if (p.num_axes > 1) {
            pos[1] = (uint32_t)__ldg(pos_at + p.pos_stride);
            if (p.num_axes > 2) pos[2] = (uint32_t)__ldg(pos_at + 2 * p.pos_stride);
        }
        pos_at += hop;
    };
    long long slot = 0;
    bool bad = false;
    float4 next_co = make_float4(1.f, 1.f, 1.f, 1.f), next_si = make_float4(0.f, 0.f, 0.f, 0.f);
    uint2 ra[kHeads], rb[kHeads];
    // Past the last head the last one is read again, and not written.
    const int last = min(kHeads, (is_q ? p.num_qo_heads : p.num_kv_heads) - head) - 1;
    auto load = [&]() {
        slot = __ldg(slot_at);
#pragma unroll
        for (int i = 0; i < kHeads; ++i) {
            ra[i] = __ldcs(reinterpret_cast<const uint2*>(src_a + min(i, last) * DH));
            rb[i] = __ldcs(reinterpret_cast<const uint2*>(src_b + min(i, last) * DH));
        }
        slot_at += hop, src_a += src_step, src_b += src_step;
        bad = max(pos[0], max(pos[1], pos[2])) >= limit;
        if (rotates && !bad) {
            if (one_axis) {
                const size_t at = (size_t)rot * (axis == 0 ? pos[0] : axis == 1 ? pos[1] : pos[2]);
                next_co = __ldg(reinterpret_cast<const float4*>(cos_at + at));
                next_si = __ldg(reinterpret_cast<const float4*>(sin_at + at));
            } else {
                float* const cp[4] = {&next_co.x, &next_co.y, &next_co.z, &next_co.w};
                float* const sp[4] = {&next_si.x, &next_si.y, &next_si.z, &next_si.w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int x = (axes >> (8 * i)) & 0xFF;
                    const size_t at = (size_t)rot * (x == 0 ? pos[0] : x == 1 ? pos[1] : pos[2]) + i;
                    *cp[i] = __ldg(cos_at + at);
                    *sp[i] = __ldg(sin_at + at);
                }
            }
        }
    };
    load_pos();
    load();
    int left = (int)((p.nnz - tok0 + hop - 1) / hop);  // tokens of this block
    if (left > 1) load_pos();
    for (; left > 0; --left) {
        f32x2 a[kHeads][2], b[kHeads][2];
#pragma unroll
        for (int i = 0; i < kHeads; ++i) {
            widen4<kBF>(ra[i], a[i]);
            widen4<kBF>(rb[i], b[i]);
        }
        const float4 co = next_co, si = next_si;
        // A padding token (slot -1) is not written, nor is one with a position
        // outside the table; one with a slot outside the pool only as a query.
        // All of them run through the same code: a branch on loaded values
        // around the shuffles below would cost more than these tokens do.
        const bool pad = slot == -1, bad_slot = (unsigned long long)slot >= (unsigned long long)p.num_slots;
        if (g == 0 && !pad && (bad || bad_slot) && p.status != nullptr) atomicOr(p.status, kStatusBounds);
        const bool put = !pad && !bad && (is_q || !bad_slot);
        uint8_t* out = dst;
        if (paged) {
            if (put) {
                const long long page = slot >> 32 ? slot / page_size : (long long)((uint32_t)slot / page_size);
                out += (size_t)page * p.num_kv_heads * head_bytes + (size_t)(slot - page * page_size) * (DH * size);
            }
        } else if (!is_q) {
            out += (size_t)slot * row_bytes;
        }
        dst += dst_step;
        if (left > 1) load();
        if (left > 2) load_pos();

        if (norms) {
#pragma unroll
            for (int i = 0; i < kHeads; ++i) {
                f32x2 s2 = mul2(a[i][0], a[i][0]);
                s2 = fma2(a[i][1], a[i][1], s2);
                s2 = fma2(b[i][0], b[i][0], s2);
                s2 = fma2(b[i][1], b[i][1], s2);
                float ss, s1;
                split_f32x2(s2, ss, s1);
                ss += s1;
#pragma unroll
                for (int d = TPR / 2; d > 0; d >>= 1) ss += __shfl_xor_sync(0xFFFFFFFFu, ss, d);
                const float inv = norm ? rsqrtf(ss * (1.0f / DH) + p.eps) : 1.f;
                const f32x2 inv2 = make_f32x2(inv, inv);
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    a[i][e] = mul2(mul2(a[i][e], inv2), wa[e]);
                    b[i][e] = mul2(mul2(b[i][e], inv2), wb[e]);
                }
            }
        }
        if (rotates) {
#pragma unroll
            for (int i = 0; i < kHeads; ++i) {
                if constexpr (kPairs) {
                    auto turn = [](f32x2 x, float c1, float s1) {
                        float x0, x1;
                        split_f32x2(x, x0, x1);
                        return fma2(make_f32x2(x1, x0), make_f32x2(-s1, s1), mul2(x, make_f32x2(c1, c1)));
                    };
                    a[i][0] = turn(a[i][0], co.x, si.x);
                    a[i][1] = turn(a[i][1], co.y, si.y);
                    b[i][0] = turn(b[i][0], co.z, si.z);
                    b[i][1] = turn(b[i][1], co.w, si.w);
                } else {
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const f32x2 c2 = e == 0 ? make_f32x2(co.x, co.y) : make_f32x2(co.z, co.w), x = a[i][e];
                        a[i][e] = fma2(b[i][e], e == 0 ? make_f32x2(-si.x, -si.y) : make_f32x2(-si.z, -si.w), mul2(x, c2));
                        b[i][e] = fma2(x, e == 0 ? make_f32x2(si.x, si.y) : make_f32x2(si.z, si.w), mul2(b[i][e], c2));
                    }
                }
            }
        }
        if (put) {
            if (!fp8) {
#pragma unroll
                for (int i = 0; i < kHeads; ++i, out += head_bytes) {
                    if (i < n) {
                        store_half<kBF>(out, a[i]);
                        store_half<kBF>(out + dst_b, b[i]);
                    }
                }
            } else if (e4m3) {
#pragma unroll
                for (int i = 0; i < kHeads; ++i, out += head_bytes) {
                    if (i < n) {
                        store_fp8<true>(out, a[i], scale_inv);
                        store_fp8<true>(out + dst_b, b[i], scale_inv);
                    }
                }
            } else {
#pragma unroll
                for (int i = 0; i < kHeads; ++i, out += head_bytes) {
                    if (i < n) {
                        store_fp8<false>(out, a[i], scale_inv);
                        store_fp8<false>(out + dst_b, b[i], scale_inv);
                    }
                }
            }
        }
    }
}

template <bool kBF, int DH>
cudaError_t launch_d(const RopeParams& p, cudaStream_t stream) {
    const auto kernel = p.interleaved ? rope_kernel<kBF, DH, true> : rope_kernel<kBF, DH, false>;
    // A token's warps go two to a block if they are even (8838 tokens of 6 warps:
    // 37.2 us, 38.1 with one), else one (5003 tokens of 3 warps: 16.4 us, 18.4
    // with two, one of which would idle); a block takes the tokens blockIdx.x,
    // blockIdx.x + gridDim.x, ...
    const long long units = (p.num_qo_heads + kHeads - 1) / kHeads + 2 * ((p.num_kv_heads + kHeads - 1) / kHeads);
    const long long warps = (units * (DH / 8) + 31) / 32, per_block = warps % 2 == 0 ? 2 : 1;
    const long long blocks = std::min<long long>(p.nnz, std::max<long long>(1, 152 * kWarps / warps));
    kernel<<<dim3((unsigned)blocks, (unsigned)(warps / per_block)), (unsigned)(32 * per_block), 0, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_rope(const RopeParams& p, cudaStream_t stream) {
    if (p.nnz == 0) return cudaSuccess;
    if (p.src_dtype == PAFP8_BF16)
        return p.head_dim == 64 ? launch_d<true, 64>(p, stream) : launch_d<true, 128>(p, stream);
    return p.head_dim == 64 ? launch_d<false, 64>(p, stream) : launch_d<false, 128>(p, stream);
}

}  // namespace pafp8
