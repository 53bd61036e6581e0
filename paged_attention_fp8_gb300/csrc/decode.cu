// decode.cu -- the split-KV merge, the built-in scratch, and the dispatch of the
// decode kernel (decode.cuh).  sm_103a.
#include <mutex>

#include "decode.cuh"

namespace pafp8 {
namespace {

// Combine the partial states of each split (request, KV-head block) row.
// The plan numbers a row's partial states consecutively (slots mptr[e] ..
// mptr[e+1] - 1, in page order), so no slot list is read.
// One warp per (merge entry, query head of the block), kMergeWarps per block;
// lane l holds dims (D/32) l .. (D/32) l + D/32 - 1.  The warp loads the
// row's slots in batches of kMergeBatch (every lane the batch's lse values
// and its own dims of the O vectors, all loads of a batch in flight
// together), keeps a running max m of the log2-domain lse_c and the rescaled
// sums of 2^lse_c and 2^lse_c O_c, and writes
// o = v_scale * sum(2^lse_c O_c) / sum(2^lse_c), lse = ln(sum) + m.
// Launched as a programmatic dependent of the decode kernel: the row's
// metadata (written by the host) is read before griddepcontrol.wait, which
// returns once the decode grid has completed and its writes are visible.
constexpr int kMergeBatch = 8;
constexpr int kMergeWarps = 4;  // query heads per merge block

// kMergeBatch lse values and O vectors (DPL floats) of partial states, all
// loads issued in one instruction block (L2, bypassing L1), so the batch's
// latencies overlap.
template <int DPL>
__device__ __forceinline__ void load_batch(const float* const (&lp)[kMergeBatch], const float* const (&op)[kMergeBatch],
                                           float (&l)[kMergeBatch], float (&o)[kMergeBatch][DPL]);
template <>
__device__ __forceinline__ void load_batch<4>(const float* const (&lp)[kMergeBatch], const float* const (&op)[kMergeBatch],
                                              float (&l)[kMergeBatch], float (&o)[kMergeBatch][4]) {
    asm volatile(
        "ld.global.cg.f32 %0, [%40];\n ld.global.cg.f32 %1, [%41];\n ld.global.cg.f32 %2, [%42];\n"
        " ld.global.cg.f32 %3, [%43];\n ld.global.cg.f32 %4, [%44];\n ld.global.cg.f32 %5, [%45];\n"
        " ld.global.cg.f32 %6, [%46];\n ld.global.cg.f32 %7, [%47];\n"
        " ld.global.cg.v4.f32 {%8, %9, %10, %11}, [%48];\n ld.global.cg.v4.f32 {%12, %13, %14, %15}, [%49];\n"
        " ld.global.cg.v4.f32 {%16, %17, %18, %19}, [%50];\n ld.global.cg.v4.f32 {%20, %21, %22, %23}, [%51];\n"
        " ld.global.cg.v4.f32 {%24, %25, %26, %27}, [%52];\n ld.global.cg.v4.f32 {%28, %29, %30, %31}, [%53];\n"
        " ld.global.cg.v4.f32 {%32, %33, %34, %35}, [%54];\n ld.global.cg.v4.f32 {%36, %37, %38, %39}, [%55];\n"
        : "=f"(l[0]), "=f"(l[1]), "=f"(l[2]), "=f"(l[3]), "=f"(l[4]), "=f"(l[5]), "=f"(l[6]), "=f"(l[7]),
          "=f"(o[0][0]), "=f"(o[0][1]), "=f"(o[0][2]), "=f"(o[0][3]), "=f"(o[1][0]), "=f"(o[1][1]), "=f"(o[1][2]),
          "=f"(o[1][3]), "=f"(o[2][0]), "=f"(o[2][1]), "=f"(o[2][2]), "=f"(o[2][3]), "=f"(o[3][0]), "=f"(o[3][1]),
          "=f"(o[3][2]), "=f"(o[3][3]), "=f"(o[4][0]), "=f"(o[4][1]), "=f"(o[4][2]), "=f"(o[4][3]), "=f"(o[5][0]),
          "=f"(o[5][1]), "=f"(o[5][2]), "=f"(o[5][3]), "=f"(o[6][0]), "=f"(o[6][1]), "=f"(o[6][2]), "=f"(o[6][3]),
          "=f"(o[7][0]), "=f"(o[7][1]), "=f"(o[7][2]), "=f"(o[7][3])
        : "l"(lp[0]), "l"(lp[1]), "l"(lp[2]), "l"(lp[3]), "l"(lp[4]), "l"(lp[5]), "l"(lp[6]), "l"(lp[7]),
          "l"(op[0]), "l"(op[1]), "l"(op[2]), "l"(op[3]), "l"(op[4]), "l"(op[5]), "l"(op[6]), "l"(op[7])
        : "memory");
    // Every result is live here, so no use of one can be scheduled before
    // the last load of the batch has been issued.
    asm volatile("" ::"f"(l[0]), "f"(l[1]), "f"(l[2]), "f"(l[3]), "f"(l[4]), "f"(l[5]), "f"(l[6]), "f"(l[7]),
                 "f"(o[0][0]), "f"(o[0][1]), "f"(o[0][2]), "f"(o[0][3]), "f"(o[1][0]), "f"(o[1][1]), "f"(o[1][2]),
                 "f"(o[1][3]), "f"(o[2][0]), "f"(o[2][1]), "f"(o[2][2]), "f"(o[2][3]), "f"(o[3][0]), "f"(o[3][1]),
                 "f"(o[3][2]), "f"(o[3][3]), "f"(o[4][0]), "f"(o[4][1]), "f"(o[4][2]), "f"(o[4][3]), "f"(o[5][0]),
                 "f"(o[5][1]), "f"(o[5][2]), "f"(o[5][3]), "f"(o[6][0]), "f"(o[6][1]), "f"(o[6][2]), "f"(o[6][3]),
                 "f"(o[7][0]), "f"(o[7][1]), "f"(o[7][2]), "f"(o[7][3]));
}
template <>
__device__ __forceinline__ void load_batch<2>(const float* const (&lp)[kMergeBatch], const float* const (&op)[kMergeBatch],
                                              float (&l)[kMergeBatch], float (&o)[kMergeBatch][2]) {
    asm volatile(
        "ld.global.cg.f32 %0, [%24];\n ld.global.cg.f32 %1, [%25];\n ld.global.cg.f32 %2, [%26];\n"
        " ld.global.cg.f32 %3, [%27];\n ld.global.cg.f32 %4, [%28];\n ld.global.cg.f32 %5, [%29];\n"
        " ld.global.cg.f32 %6, [%30];\n ld.global.cg.f32 %7, [%31];\n"
        " ld.global.cg.v2.f32 {%8, %9}, [%32];\n ld.global.cg.v2.f32 {%10, %11}, [%33];\n"
        " ld.global.cg.v2.f32 {%12, %13}, [%34];\n ld.global.cg.v2.f32 {%14, %15}, [%35];\n"
        " ld.global.cg.v2.f32 {%16, %17}, [%36];\n ld.global.cg.v2.f32 {%18, %19}, [%37];\n"
        " ld.global.cg.v2.f32 {%20, %21}, [%38];\n ld.global.cg.v2.f32 {%22, %23}, [%39];\n"
        : "=f"(l[0]), "=f"(l[1]), "=f"(l[2]), "=f"(l[3]), "=f"(l[4]), "=f"(l[5]), "=f"(l[6]), "=f"(l[7]),
          "=f"(o[0][0]), "=f"(o[0][1]), "=f"(o[1][0]), "=f"(o[1][1]), "=f"(o[2][0]), "=f"(o[2][1]), "=f"(o[3][0]),
          "=f"(o[3][1]), "=f"(o[4][0]), "=f"(o[4][1]), "=f"(o[5][0]), "=f"(o[5][1]), "=f"(o[6][0]), "=f"(o[6][1]),
          "=f"(o[7][0]), "=f"(o[7][1])
        : "l"(lp[0]), "l"(lp[1]), "l"(lp[2]), "l"(lp[3]), "l"(lp[4]), "l"(lp[5]), "l"(lp[6]), "l"(lp[7]),
          "l"(op[0]), "l"(op[1]), "l"(op[2]), "l"(op[3]), "l"(op[4]), "l"(op[5]), "l"(op[6]), "l"(op[7])
        : "memory");
    asm volatile("" ::"f"(l[0]), "f"(l[1]), "f"(l[2]), "f"(l[3]), "f"(l[4]), "f"(l[5]), "f"(l[6]), "f"(l[7]),
                 "f"(o[0][0]), "f"(o[0][1]), "f"(o[1][0]), "f"(o[1][1]), "f"(o[2][0]), "f"(o[2][1]), "f"(o[3][0]),
                 "f"(o[3][1]), "f"(o[4][0]), "f"(o[4][1]), "f"(o[5][0]), "f"(o[5][1]), "f"(o[6][0]), "f"(o[6][1]),
                 "f"(o[7][0]), "f"(o[7][1]));
}

template <int DPL>
__device__ __forceinline__ void merge_head(const DecodeParams& p, int hpb, int hh, int s0, int s1, size_t oh,
                                           float vscale) {
    const int lane = threadIdx.x & 31;
    float m = -INFINITY, sum = 0.f, acc[DPL];
#pragma unroll
    for (int i = 0; i < DPL; ++i) acc[i] = 0.f;
    for (int s = s0; s < s1; s += kMergeBatch) {
        float l[kMergeBatch], o[kMergeBatch][DPL];
        const float* lp[kMergeBatch];
        const float* op[kMergeBatch];
#pragma unroll
        for (int k = 0; k < kMergeBatch; ++k) {
            const size_t idx = (size_t)(s + k < s1 ? s + k : s) * hpb + hh;  // a row's slots are consecutive
            lp[k] = p.part_lse + idx;
            op[k] = p.part_o + idx * p.head_dim + DPL * lane;
        }
        load_batch<DPL>(lp, op, l, o);  // every load of the batch in flight together
        // Slot s (k = 0) exists, so m is finite from here on; padding slots
        // (lse -inf) get weight 0.
#pragma unroll
        for (int k = 0; k < kMergeBatch; ++k) {
            const float lk = s + k < s1 ? l[k] : -INFINITY;
            const float mn = fmaxf(m, lk);
            const float a = ex2(m - mn), wt = ex2(lk - mn);
            sum = sum * a + wt;
#pragma unroll
            for (int i = 0; i < DPL; ++i) acc[i] = acc[i] * a + wt * o[k][i];
            m = mn;
        }
    }
    const float inv = vscale / sum;
    uint32_t wd[DPL / 2];
#pragma unroll
    for (int i = 0; i < DPL / 2; ++i) wd[i] = pack_out2(acc[2 * i] * inv, acc[2 * i + 1] * inv, p.o_dtype);
    uint16_t* dst = static_cast<uint16_t*>(p.o) + oh * p.head_dim + DPL * lane;
    if constexpr (DPL == 4)
        *reinterpret_cast<uint2*>(dst) = make_uint2(wd[0], wd[DPL > 2 ? 1 : 0]);
    else
        *reinterpret_cast<uint32_t*>(dst) = wd[0];
    if (lane == 0 && p.lse != nullptr) p.lse[oh] = (m + __log2f(sum)) * 0.69314718055994531f;
}

// One (merge entry, query head) pair's metadata: its slots, output row and
// v_scale.  The metadata is the host's, so it may be read before the
// partial states are complete.
struct MergePair {
    int hh, s0, s1;
    size_t oh;
    float vscale;
};

__device__ __forceinline__ MergePair merge_pair_args(const DecodeParams& p, int hpc, int group, int e, int hh) {
    const int* meta = p.meta;
    const int nhb = meta[kMetaHeadBlocks];
    const int* mptr = meta + meta[kMetaOffMergePtr];
    const int* mrow = meta + meta[kMetaOffMergeRow];
    const int hpb = hpc * group;
    const int row = mrow[e];
    const int b = row / nhb, hb = row - b * nhb;
    const int head = hb * hpb + hh;  // query head: (hb * hpc + hh / group) * group + hh % group
    MergePair a;
    a.hh = hh;
    a.s0 = mptr[e];
    a.s1 = mptr[e + 1];
    a.oh = (size_t)b * p.num_qo_heads + head;
    a.vscale = p.v_scales != nullptr ? __ldg(p.v_scales + head / group) : p.v_scale;
    return a;
}

__device__ __forceinline__ void merge_pair(const DecodeParams& p, int hpb, const MergePair& a) {
    if (p.head_dim == 64)
        merge_head<2>(p, hpb, a.hh, a.s0, a.s1, a.oh, a.vscale);
    else
        merge_head<4>(p, hpb, a.hh, a.s0, a.s1, a.oh, a.vscale);
}

__global__ void __launch_bounds__(32 * kMergeWarps)
    merge_kernel(const __grid_constant__ DecodeParams p, int hpc, int group) {
    // The metadata (written by the host) is read before the wait.
    const int hpb = hpc * group;
    const int bpr = (hpb + kMergeWarps - 1) / kMergeWarps;  // blocks per merge row
    const int e = blockIdx.x / bpr;
    const int hh = (blockIdx.x - e * bpr) * kMergeWarps + (threadIdx.x >> 5);
    MergePair a{};
    if (hh < hpb) a = merge_pair_args(p, hpc, group, e, hh);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (hh >= hpb) return;
    merge_pair(p, hpb, a);
}

}  // namespace

// Built-in scratch for callers that cannot allocate device memory (see
// pafp8_run_decode_noalloc).  It stands in for the caller's workspace: the
// plan's metadata, the split-KV partial states and the status word.  Every
// GPU that loads the library holds these bytes until the process exits, and
// every call shares them.
static __device__ __align__(256) uint8_t g_noalloc_scratch[kNoAllocScratchBytes];

// Device address of g_noalloc_scratch on the current device.  The symbol's
// host-side name is only a stand-in, so the address is looked up once per
// device (with that device current) and cached.
cudaError_t noalloc_scratch(void** ptr) {
    static std::mutex mu;
    static void* addr[kMaxDevices] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
    std::lock_guard<std::mutex> lock(mu);
    if (addr[dev] == nullptr) {
        void* a = nullptr;
        e = cudaGetSymbolAddress(&a, g_noalloc_scratch);
        if (e != cudaSuccess) return e;
        addr[dev] = a;
    }
    *ptr = addr[dev];
    return cudaSuccess;
}

cudaError_t launch_decode(const DecodeParams& p, const CUtensorMap& tmap_k, const CUtensorMap& tmap_v,
                          int num_ctas, int hpc, int group, int heads_per_box, cudaStream_t stream) {
    if (p.k_blocks != nullptr) return launch_decode_blocks(p, tmap_k, tmap_v, num_ctas, hpc, group, heads_per_box, stream);
    if (p.window > 0) return launch_decode_window(p, tmap_k, tmap_v, num_ctas, hpc, group, heads_per_box, stream);
    return launch_decode_var<kVarPlain>(p, tmap_k, tmap_v, num_ctas, hpc, group, heads_per_box, stream);
}

cudaError_t launch_merge(const DecodeParams& p, int num_merge, int hpc, int group, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(num_merge * ((hpc * group + kMergeWarps - 1) / kMergeWarps));
    cfg.blockDim = dim3(32 * kMergeWarps);
    cfg.dynamicSmemBytes = 0;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, merge_kernel, p, hpc, group);
}

}  // namespace pafp8
