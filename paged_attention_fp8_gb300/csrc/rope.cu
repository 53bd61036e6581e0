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
// The work is a stream of reads and writes, bounded by HBM bandwidth (per
// token (Hq + 2 Hkv) D elements in, Hq D + 2 Hkv D out) or, for the tokens of
// a decode step, by latency.  A thread owns eight consecutive dims of a head,
// D / 8 threads a head, so every load and store is 16 bytes (8 for fp8) and
// a neighbouring pair lies in one thread; the other half of a pair at
// distance R / 2 comes from a lane R / 16 away, which is why R is a multiple
// of 16.  A block takes whole tokens: its threads keep one dim octet, so the
// norm weights are loaded once a block and the angles once a token, and the
// heads of a token are loaded kBatch at a time before any is used.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "../../include/pafp8.h"
#include "internal.h"

namespace pafp8 {
namespace {

constexpr int kThreads = 256;
constexpr int kBatch = 3;  // heads in flight per thread: 32 / 8 heads of 128 dims are three rounds of a block

template <bool kBF>
__device__ __forceinline__ void widen8(const uint4& r, float (&x)[8]) {
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (kBF) {
            x[2 * i] = __uint_as_float(w[i] << 16);
            x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        } else {
            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
            x[2 * i] = f.x;
            x[2 * i + 1] = f.y;
        }
    }
}

template <bool kBF>
__device__ __forceinline__ uint4 narrow8(const float (&x)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (kBF) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t*>(&h);
        } else {
            const __half2 h = __floats2half2_rn(x[2 * i], x[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t*>(&h);
        }
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// Eight fp8 codes of x * inv (the product rounded once in fp32).
__device__ __forceinline__ uint2 codes8(const float (&x)[8], float inv, bool e4m3) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float lo = __fmul_rn(x[2 * i], inv), hi = __fmul_rn(x[2 * i + 1], inv);
        unsigned short d;
        if (e4m3)
            asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(d) : "f"(hi), "f"(lo));
        else
            asm("cvt.rn.satfinite.e5m2x2.f32 %0, %1, %2;" : "=h"(d) : "f"(hi), "f"(lo));
        w[i] = d;
    }
    return make_uint2(w[0] | (w[1] << 16), w[2] | (w[3] << 16));
}

template <bool kBF>
__device__ __forceinline__ void store8(void* base, size_t elem, const float (&x)[8], int dtype, float inv) {
    if (dtype == PAFP8_E4M3FN || dtype == PAFP8_E5M2)
        *reinterpret_cast<uint2*>(static_cast<uint8_t*>(base) + elem) = codes8(x, inv, dtype == PAFP8_E4M3FN);
    else
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(base) + elem) = narrow8<kBF>(x);
}

template <bool kBF, int DH, bool kPairs>  // kPairs: neighbouring dims rotate together
__global__ void __launch_bounds__(kThreads) rope_kernel(const __grid_constant__ RopeParams p) {
    constexpr int TPR = DH / 8;            // threads per head
    constexpr int RPB = kThreads / TPR;    // heads per round of a block
    const int c = threadIdx.x % TPR, r0 = threadIdx.x / TPR;
    const int half = p.rot_dim >> 1;
    const int heads = p.num_qo_heads + 2 * p.num_kv_heads;
    const int hk = p.num_qo_heads, hv = hk + p.num_kv_heads;
    const bool turns = 8 * c < p.rot_dim;
    // Halves: this octet's pairs are pair0 .. pair0 + 7, the octet is the pair's
    // second half from `half` on, and its partner sits half / 8 lanes away.
    const bool second = !kPairs && 8 * c >= half;
    const int pair0 = kPairs ? 4 * c : (second ? 8 * c - half : 8 * c);
    const int lane = threadIdx.x & 31;
    const int partner = kPairs || !turns ? lane : (second ? lane - half / 8 : lane + half / 8);
    constexpr int NP = kPairs ? 4 : 8;  // pairs of an octet

    const bool norm_q = p.q_weight != nullptr, norm_k = p.k_weight != nullptr;
    uint4 wq{}, wk{};
    if (norm_q) wq = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.q_weight) + 8 * c));
    if (norm_k) wk = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.k_weight) + 8 * c));

    for (long long tok = blockIdx.x; tok < p.nnz; tok += gridDim.x) {
        // The heads do not depend on slot or position: their loads go first.
        uint4 raw[kBatch];
        auto load = [&](int first) {
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                const int r = first + i * RPB;
                const uint16_t* src =
                    r < hk   ? static_cast<const uint16_t*>(p.q) + tok * p.q_stride + (long long)r * DH
                    : r < hv ? static_cast<const uint16_t*>(p.k) + tok * p.k_stride + (long long)(r - hk) * DH
                             : static_cast<const uint16_t*>(p.v) + tok * p.v_stride + (long long)(r - hv) * DH;
                raw[i] = r < heads ? __ldcs(reinterpret_cast<const uint4*>(src + 8 * c)) : make_uint4(0, 0, 0, 0);
            }
        };
        load(r0);
        const long long slot = __ldg(p.slots + tok);
        if (slot == -1) continue;  // padding: nothing is written
        int pos[3] = {0, 0, 0};
        bool bad = false;
#pragma unroll
        for (int a = 0; a < 3; ++a) {
            if (a < p.num_axes) {
                pos[a] = __ldg(p.positions + a * p.pos_stride + tok);
                if (pos[a] < 0 || pos[a] >= p.max_position) {
                    bad = true;
                    pos[a] = 0;
                }
            }
        }
        // A token with a position outside the table is not written at all,
        // one with a slot outside the pool only as a query.
        const bool bad_slot = slot < 0 || slot >= p.num_slots;
        if ((bad || bad_slot) && threadIdx.x == 0 && p.status != nullptr) atomicOr(p.status, kStatusBounds);
        if (bad) continue;

        float cs[NP], sn[NP];
#pragma unroll
        for (int i = 0; i < NP; ++i) {
            cs[i] = 1.f;
            sn[i] = 0.f;
        }
        if (turns) {
            if (p.pair_axis == nullptr) {
                const float4* tc = reinterpret_cast<const float4*>(p.cos_sin + (size_t)pos[0] * p.rot_dim + pair0);
                const float4* ts = reinterpret_cast<const float4*>(p.cos_sin + (size_t)pos[0] * p.rot_dim + half + pair0);
#pragma unroll
                for (int i = 0; i < NP / 4; ++i) {
                    const float4 a = __ldg(tc + i), b = __ldg(ts + i);
                    cs[4 * i] = a.x, cs[4 * i + 1] = a.y, cs[4 * i + 2] = a.z, cs[4 * i + 3] = a.w;
                    sn[4 * i] = b.x, sn[4 * i + 1] = b.y, sn[4 * i + 2] = b.z, sn[4 * i + 3] = b.w;
                }
            } else {
#pragma unroll
                for (int i = 0; i < NP; ++i) {
                    const int a = __ldg(p.pair_axis + pair0 + i);  // an axis past the last one counts as the last
                    const int at = a == 0 || p.num_axes == 1 ? pos[0] : a == 1 || p.num_axes == 2 ? pos[1] : pos[2];
                    const float* row = p.cos_sin + (size_t)at * p.rot_dim + pair0 + i;
                    cs[i] = __ldg(row);
                    sn[i] = __ldg(row + half);
                }
            }
            if (second) {
#pragma unroll
                for (int i = 0; i < NP; ++i) sn[i] = -sn[i];
            }
        }
        size_t kv_row = 0;  // element offset of KV head 0, and the stride of a head
        size_t kv_head = DH;
        if (!bad_slot) {
            if (p.hnd) {
                const long long page = slot / p.page_size;
                kv_row = ((size_t)page * p.num_kv_heads * p.page_size + (size_t)(slot - page * p.page_size)) * DH;
                kv_head = (size_t)p.page_size * DH;
            } else {
                kv_row = (size_t)slot * p.num_kv_heads * DH;
            }
        }
        for (int first = r0;;) {
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                const int r = first + i * RPB;
                const bool is_q = r < hk, is_v = r >= hv;
                float x[8];
                widen8<kBF>(raw[i], x);
                float ss = 0.f;
#pragma unroll
                for (int e = 0; e < 8; ++e) ss = fmaf(x[e], x[e], ss);
#pragma unroll
                for (int d = TPR / 2; d > 0; d >>= 1) ss += __shfl_xor_sync(0xFFFFFFFFu, ss, d);
                if (is_q ? norm_q : norm_k && !is_v) {
                    const float inv = rsqrtf(ss * (1.0f / DH) + p.eps);
                    float w[8];
                    widen8<kBF>(is_q ? wq : wk, w);
#pragma unroll
                    for (int e = 0; e < 8; ++e) x[e] = x[e] * inv * w[e];
                }
                float y[8];
                if constexpr (kPairs) {
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        y[2 * k] = x[2 * k] * cs[k] - x[2 * k + 1] * sn[k];
                        y[2 * k + 1] = x[2 * k + 1] * cs[k] + x[2 * k] * sn[k];
                    }
                } else {
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const float o = __shfl_sync(0xFFFFFFFFu, x[e], partner);
                        y[e] = x[e] * cs[e] - o * sn[e];
                    }
                }
                if (is_v || !turns) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) y[e] = x[e];
                }
                if (is_q) {
                    store8<kBF>(p.q_out, ((size_t)tok * p.num_qo_heads + r) * DH + 8 * c, y, p.q_out_dtype, p.q_inv);
                } else if (r < heads && !bad_slot) {
                    store8<kBF>(is_v ? p.v_cache : p.k_cache, kv_row + (size_t)(r - (is_v ? hv : hk)) * kv_head + 8 * c, y,
                                p.kv_dtype, is_v ? p.v_inv : p.k_inv);
                }
            }
            // The whole block makes the same number of rounds: the shuffles
            // above need every lane of a warp.
            first += kBatch * RPB;
            if (first - r0 >= heads) break;
            load(first);
        }
    }
}

template <bool kBF, int DH>
cudaError_t launch_d(const RopeParams& p, cudaStream_t stream) {
    // One token a block up to eight blocks an SM; more tokens are taken in turn.
    const int grid = (int)(p.nnz < 1216 ? p.nnz : 1216);
    if (p.interleaved)
        rope_kernel<kBF, DH, true><<<grid, kThreads, 0, stream>>>(p);
    else
        rope_kernel<kBF, DH, false><<<grid, kThreads, 0, stream>>>(p);
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
