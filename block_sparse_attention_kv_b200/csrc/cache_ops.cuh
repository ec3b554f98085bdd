// Declarations shared by the whole-cache operators: exact decode attention
// over every token of the paged cache (full_decode.cu), its part over a
// prefix that the batch shares (shared_prefix.cu), eviction (evict.cu) and
// their entry points (cache_abi.cu).
#pragma once

#include <atomic>

#include "absp_internal.cuh"

namespace absp {

constexpr float kLog2E = 1.4426950408889634f;

// What the whole-cache kernels need of a layer (KvDesc without the block
// tables of the sparse path).
struct CacheDesc {
    int32_t S, Hq, Hkv, G;
    int32_t max_pages;
    int32_t shared;               // tokens of the shared prefix (a multiple of 16), 0: none
    int64_t num_phys_pages;
    const int32_t* seq_lens;
    const int32_t* page_table;
};

// Length of sequence s, 0 where the table cannot hold it (reported).
__device__ __forceinline__ int checked_len(const CacheDesc& c, int s, int32_t* err) {
    const int len = c.seq_lens[s];
    if (len < 0 || len > c.max_pages * kPage) {
        set_error(err, ABSP_ERR_DEVICE_FAULT, s);
        return 0;
    }
    return len;
}

// First token that sequence s attends to by itself: behind the shared
// prefix, or token 0 where the sequence does not hold the whole prefix.
__device__ __forceinline__ int own_start(const CacheDesc& c, int len) {
    return len >= c.shared ? c.shared : 0;
}

__device__ __forceinline__ float exp2_approx(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// 3-D tensor tile load into this CTA's own shared memory.
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* map, int x, int y,
                                            int z, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar)
        : "memory");
}

// The same with an L2 cache policy.
__device__ __forceinline__ void tma_load_3d_hint(uint32_t dst, const CUtensorMap* map, int x, int y,
                                                 int z, uint32_t bar, uint64_t policy) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        ".L2::cache_hint [%0], [%1, {%2, %3, %4}], [%5], %6;" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar), "l"(policy)
        : "memory");
}

// Data that is read once: first to leave L2.
__device__ __forceinline__ uint64_t evict_first_policy() {
    uint64_t p;
    asm("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(p));
    return p;
}

// 16-byte asynchronous copy global -> shared; bytes behind `bytes` (0 or 16)
// are zero.
__device__ __forceinline__ void cp_async_16_zfill(uint32_t dst, const void* src, uint32_t bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes)
                 : "memory");
}

// Workspace of the decode calls (cache_abi.cu lays it out).
struct FullWs {
    int32_t* err;
    int32_t* cum;                 // [S + 1] own pages per KV head before sequence s
    float2* ml;                   // [slots][G] running maximum (log2 units) and sum of a partial
    float* o;                     // [slots][G][128] unnormalised partial outputs
    float* scratch;               // [workers][G][128] parts that neighbouring warps join
    float* scores;                // [S][Hq][16 * max_pages] scores in log2 units (weights only)
    float2* pml;                  // [prefix slots][128] the same of the shared prefix's partials
    float* po;                    // [prefix slots][128][128]
};

// Work over the shared prefix: units of up to two 128-row query tiles of one
// KV head, each meeting every 128-token tile of the prefix.
struct PrefixPlan {
    int32_t tiles;                // token tiles
    int32_t row_tiles;            // query-row tiles per KV head (rows: sequence-major, then head)
    int32_t units;                // ceil(row_tiles / 2) * Hkv, the head running fastest
};
__host__ __device__ inline PrefixPlan prefix_plan(int shared, int S, int G, int Hkv) {
    PrefixPlan p;
    p.tiles = (shared + 127) / 128;
    p.row_tiles = static_cast<int32_t>((static_cast<int64_t>(S) * G + 127) / 128);
    p.units = (p.row_tiles + 1) / 2 * Hkv;
    return p;
}

struct FullArgs {
    CacheDesc c;
    FullWs ws;
    const __nv_bfloat16* q;
    __nv_bfloat16* out;
    const float* weights_in;      // may be null: zeros
    float* weights_out;           // null: no weights
    int32_t weights_from;         // first token with weights, in sequences that hold as many
    int32_t workers;              // warps of the split grid
    int32_t prefix_ctas;          // CTAs of the prefix grid, 0 without a shared prefix
    PrefixPlan prefix;
};

constexpr int kFullWarps = 8;     // workers (warps) per CTA of the split kernel
constexpr int kMaxSms = 160;      // the workspace is sized for at most that many
int unit_cluster(int S, int Hkv, int max_pages);   // CTAs per (sequence, head), 0: split and merge
int device_sms();                 // SMs used on the current device (<= kMaxSms)

// tmk, tmv: a box is a (page, head) slice, its two 64-channel halves one
// behind the other; tmk_half: a box is one half of a slice.
cudaError_t launch_full(const FullArgs& a, const CUtensorMap& tmk, const CUtensorMap& tmv,
                        const CUtensorMap& tmk_half, bool pdl, cudaStream_t st);
cudaError_t launch_prefix(const FullArgs& a, const CUtensorMap& tmk_half, const CUtensorMap& tmv,
                          bool pdl, cudaStream_t st);

// A kernel's one-time set-up on the current device: loads it (a first launch
// inside a stream capture would, and end the capture), raises its
// shared-memory limit to `bytes` (0: the default), allows clusters of more
// than 8.  In relaxed capture mode, as no call here touches a stream.
template <typename K>
cudaError_t prepare_kernel(K kern, int bytes, bool big_cluster, std::atomic<uint64_t>* done) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 64 && (done->load(std::memory_order_relaxed) >> dev) & 1) return cudaSuccess;
    cudaStreamCaptureMode mode = cudaStreamCaptureModeRelaxed;
    cudaThreadExchangeStreamCaptureMode(&mode);
    cudaFuncAttributes attr;
    e = cudaFuncGetAttributes(&attr, kern);
    if (e == cudaSuccess && bytes > 0)
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess && big_cluster)
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    cudaThreadExchangeStreamCaptureMode(&mode);
    if (e == cudaSuccess && dev < 64) done->fetch_or(1ull << dev, std::memory_order_relaxed);
    return e;
}

struct EvictArgs {
    CacheDesc c;
    int32_t* err;
    __nv_bfloat16* k_pages;
    __nv_bfloat16* v_pages;
    const float* weights_in;
    float* weights_out;
    const int32_t* dst_table;
    int32_t dst_max_pages;
    int32_t keep, protect, recent;
    int32_t* kept;
    int32_t* new_lens;
    int32_t* flags;               // [S][Hkv] units whose rows have to move in order
    int32_t compact;              // the destination table is the page table
    int32_t early;                // the move kernel may start while the select runs
};
cudaError_t launch_evict(const EvictArgs& a, bool pdl, cudaStream_t st);

}  // namespace absp
