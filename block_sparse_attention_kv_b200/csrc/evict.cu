// Eviction from the paged cache by accumulated attention weight.
//
// Per (sequence, KV head) with L > keep tokens: the first `protect` and the
// last `recent` tokens stay, and of those between them the keep - protect -
// recent with the largest weights (equal weights: the lower positions; NaN
// ranks below everything).  Kept tokens move, in their order, to the front
// of the destination pages; kept[r] is the position that rank r came from.
//
// Two launches.  A select kernel finds each unit's threshold by a radix
// select on order-preserving keys, lists the kept positions and compacts the
// weights.  The rows then move: by evict_copy_kernel, every token on its own,
// where source and destination pages differ; by evict_compact_kernel, in an
// order that allows source and destination to be the same pages, where the
// destination table is the page table itself.
//
// What bounds it is moving the kept rows, 1 KiB read and written per token
// and head in 256-byte pieces from anywhere in the pools.  Measured on a
// B200: 32 x 32K tokens, 8 heads, cut to 4096 with the first 1024 where they
// are (805 MB of rows) 193 us: 58 of selection, 137 of rows at 5.9 TB/s (91 %
// of the measured copy bandwidth), 201 us with the page table itself as the
// destination; a ragged batch of 24 cut to 16383 472 us; one 32K sequence cut
// to 8192 30 us (16 and 14).
#include <algorithm>
#include <atomic>

#include "cache_ops.cuh"

namespace absp {

namespace {

constexpr int kThreads = 512;
constexpr int kWarpsE = kThreads / 32;
constexpr int kPer = 8;                        // consecutive positions per thread
constexpr int kChunk = kThreads * kPer;        // positions per pass over a slice's piece
constexpr int kMaxCluster = 16;

// Order-preserving key of a weight: larger weight, larger key; NaN lowest;
// -0 counts as 0.
__device__ __forceinline__ uint32_t key_of(float w) {
    if (w != w) return 0u;
    const uint32_t u = __float_as_uint(w + 0.0f);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}

__device__ __forceinline__ uint32_t dsmem_ld_u32(uint32_t addr) {
    uint32_t v;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr));
    return v;
}

__device__ __forceinline__ void cluster_sync() {
    cluster_arrive();
    cluster_wait();
}

struct SelectShared {
    uint32_t hist[2][256];         // this CTA's counts of a digit (read by the cluster)
    uint32_t digit, above;         // the threshold's digit, keys above it (cluster-wide)
    uint32_t mine[2];              // this slice's tokens that stay for sure, and equal keys
    uint32_t in_place;             // a destination page is its own source page
    uint32_t warp_n[2][kWarpsE];
};

// Sum over the cluster of the word at `at` in every CTA's shared memory; `n`
// CTAs, all loads in flight together.
__device__ __forceinline__ uint32_t cluster_total(const uint32_t* at, int n) {
    uint32_t v[kMaxCluster];
#pragma unroll
    for (int r = 0; r < kMaxCluster; ++r) v[r] = r < n ? dsmem_ld_u32(dsmem_addr(smem_u32(at), r)) : 0u;
    uint32_t t = 0;
#pragma unroll
    for (int r = 0; r < kMaxCluster; ++r) t += v[r];
    return t;
}

// Few units of many tokens: one cluster per unit, its positions cut into one
// slice per CTA.  Four 8-bit digits from the top: each CTA counts its slice's
// keys that agree with the threshold's digits so far, the cluster's counts
// are added through distributed shared memory.  A slice of at most kChunk
// positions stays in registers through all passes; longer ones are read
// again (from L2).
__global__ void __launch_bounds__(kThreads, 2) evict_select_cluster_kernel(const EvictArgs p) {
    __shared__ SelectShared sh;
    const CacheDesc& c = p.c;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int C = static_cast<int>(cluster_nctarank()), rank = static_cast<int>(cluster_ctarank());
    const int unit = blockIdx.x / C;
    const int s = unit / c.Hkv;
    const int cap = c.max_pages * kPage;
    if (tid == 0) sh.in_place = 0;
    if (tid < 256) sh.hist[0][tid] = 0;
    pdl_wait();
    if (p.early) pdl_trigger();
    int len = c.seq_lens[s];
    if (len < 0 || len > cap) {
        if (tid == 0) set_error(p.err, ABSP_ERR_DEVICE_FAULT, s);
        len = 0;
    }
    const int keep = p.keep, n_new = min(len, keep);
    const bool cut = len > keep;
    const float* w_in = p.weights_in + static_cast<int64_t>(unit) * cap;
    float* w_out = p.weights_out + static_cast<int64_t>(unit) * cap;
    const bool alias = w_in == w_out;
    int32_t* kept = p.kept + static_cast<int64_t>(unit) * keep;
    const int t0 = rank * kThreads + tid, tn = C * kThreads;   // this thread among the cluster's
    __syncthreads();

    // protected tokens never move, so only the pages behind them matter; an
    // uncut sequence keeps every position
    if (!p.compact && cut) {
        const int32_t* src_row = c.page_table + static_cast<int64_t>(s) * c.max_pages;
        const int32_t* dst_row = p.dst_table + static_cast<int64_t>(s) * p.dst_max_pages;
        for (int i = p.protect / kPage + t0; i < (n_new + kPage - 1) / kPage; i += tn)
            if (dst_row[i] == src_row[i]) sh.in_place = 1;
    }

    // this CTA's slice of the positions, whole groups of kPer
    const int groups = (len + kPer - 1) / kPer, per = (groups + C - 1) / C * kPer;
    const int i0 = min(len, rank * per), i1 = min(len, i0 + per);
    const int chunks = (i1 - i0 + kChunk - 1) / kChunk;
    float w[kPer];
    auto load = [&](int ch, float (&v)[kPer]) {
        const int i = i0 + ch * kChunk + tid * kPer;
        if (i < i1) {   // rows are 64-byte aligned and end on whole pages
            *reinterpret_cast<float4*>(v) = *reinterpret_cast<const float4*>(w_in + i);
            *reinterpret_cast<float4*>(v + 4) = *reinterpret_cast<const float4*>(w_in + i + 4);
        }
    };
    uint32_t prefix = 0, left = 0;      // the threshold's key; keys equal to it that stay
    uint32_t gt0 = 0, eq0 = 0;          // before this slice: tokens that stay for sure, equal keys
    if (cut) {
        const int a = p.protect, b = len - p.recent;     // the middle
        left = static_cast<uint32_t>(keep - p.protect - p.recent);
        uint32_t gt = 0, eq = 0;
        if (left == 0) {
            prefix = 0xffffffffu;                        // no key is above or equal: NaNs have others
        } else {
            uint32_t mask = 0;
            int buf = 0;
            for (int shift = 24; shift >= 0; shift -= 8) {
                float nxt[kPer];
                if (chunks > 1 || shift == 24) load(0, w);
                for (int ch = 0; ch < chunks; ++ch) {
                    if (ch + 1 < chunks) load(ch + 1, nxt);
                    const int i = i0 + ch * kChunk + tid * kPer;
#pragma unroll
                    for (int e = 0; e < kPer; ++e) {
                        const uint32_t k = key_of(w[e]);
                        if (i + e >= a && i + e < min(b, i1) && (k & mask) == prefix)
                            atomicAdd(&sh.hist[buf][(k >> shift) & 255u], 1u);
                    }
                    if (ch + 1 < chunks) {
#pragma unroll
                        for (int e = 0; e < kPer; ++e) w[e] = nxt[e];
                    }
                }
                cluster_sync();
                // thread t holds the t-th bin from the top
                const uint32_t n = tid < 256 ? cluster_total(&sh.hist[buf][255 - tid], C) : 0u;
                uint32_t incl = n;
                for (int d = 1; d < 32; d *= 2) {
                    const uint32_t y = __shfl_up_sync(0xffffffffu, incl, d);
                    if (lane >= d) incl += y;
                }
                if (lane == 31) sh.warp_n[0][warp] = incl;
                __syncthreads();
                uint32_t above = incl - n;
#pragma unroll
                for (int k = 0; k < kWarpsE; ++k)
                    if (k < warp) above += sh.warp_n[0][k];
                if (above < left && above + n >= left) {
                    sh.digit = 255 - tid;
                    sh.above = above;
                }
                __syncthreads();
                const uint32_t digit = sh.digit;
                // this slice's keys above the digit
                uint32_t x = tid < 256 && tid > static_cast<int>(digit) ? sh.hist[buf][tid] : 0u;
                x = __reduce_add_sync(0xffffffffu, x);
                if (lane == 0) sh.warp_n[1][warp] = x;
                prefix |= digit << shift;
                mask |= 255u << shift;
                left -= sh.above;      // still needed among the keys of this prefix
                // the other buffer: the cluster may still read this one
                if (shift > 0 && tid < 256) sh.hist[buf ^ 1][tid] = 0;
                __syncthreads();
#pragma unroll
                for (int k = 0; k < kWarpsE; ++k) gt += sh.warp_n[1][k];
                eq = sh.hist[buf][digit];
                buf ^= 1;
                __syncthreads();
            }
        }
        // tokens that stay outside the middle are counted where they lie
        gt += max(0, min(i1, a) - i0) + max(0, i1 - max(i0, b));
        if (tid == 0) {
            sh.mine[0] = gt;
            sh.mine[1] = eq;
        }
        cluster_sync();
        {
            uint32_t g = 0, q = 0;
            if (lane < rank) {
                g = dsmem_ld_u32(dsmem_addr(smem_u32(&sh.mine[0]), lane));
                q = dsmem_ld_u32(dsmem_addr(smem_u32(&sh.mine[1]), lane));
            }
            gt0 = __reduce_add_sync(0xffffffffu, g);
            eq0 = __reduce_add_sync(0xffffffffu, q);
        }
        // ---- the list, chunk by chunk; the weights move along where they
        // have another buffer to go to
        uint32_t at = gt0 + min(eq0, left);
        uint32_t ties = left - min(eq0, left);           // equal keys still to take
        float nxt[kPer];
        if (chunks > 1 || prefix == 0xffffffffu) load(0, w);   // else still in registers
        for (int ch = 0; ch < chunks; ++ch) {
            if (ch + 1 < chunks) load(ch + 1, nxt);
            const int i = i0 + ch * kChunk + tid * kPer;
            uint32_t is_gt = 0, is_eq = 0;
#pragma unroll
            for (int e = 0; e < kPer; ++e) {
                if (i + e < i1) {
                    const bool forced = i + e < a || i + e >= b;
                    const uint32_t k = key_of(w[e]);
                    is_gt |= (forced || k > prefix ? 1u : 0u) << e;
                    is_eq |= (!forced && k == prefix ? 1u : 0u) << e;
                }
            }
            uint32_t n = __popc(is_gt) << 16 | __popc(is_eq);
            uint32_t incl = n;
            for (int d = 1; d < 32; d *= 2) {
                const uint32_t y = __shfl_up_sync(0xffffffffu, incl, d);
                if (lane >= d) incl += y;
            }
            if (lane == 31) sh.warp_n[ch & 1][warp] = incl;
            __syncthreads();
            uint32_t before = incl - n, all = 0;
#pragma unroll
            for (int k = 0; k < kWarpsE; ++k) {
                const uint32_t v = sh.warp_n[ch & 1][k];
                if (k < warp) before += v;
                all += v;
            }
            uint32_t g = before >> 16, q = before & 0xffffu;
#pragma unroll
            for (int e = 0; e < kPer; ++e) {
                const bool take_eq = (is_eq >> e & 1) && q < ties;
                if ((is_gt >> e & 1) || take_eq) {
                    const uint32_t r = at + g + min(q, ties);
                    kept[r] = i + e;
                    if (!alias) w_out[r] = w[e];
                }
                g += is_gt >> e & 1;
                q += is_eq >> e & 1;
            }
            at += (all >> 16) + min(all & 0xffffu, ties);
            ties -= min(all & 0xffffu, ties);
            if (ch + 1 < chunks) {
#pragma unroll
                for (int e = 0; e < kPer; ++e) w[e] = nxt[e];
            }
        }
    } else {
        // (64 bits: the last step behind the largest keep passes 2^31)
        for (int64_t i = t0; i < keep; i += tn) kept[i] = i < len ? static_cast<int32_t>(i) : -1;
        if (!alias)
            for (int i = t0; i < len; i += tn) w_out[i] = w_in[i];
    }
    cluster_sync();
    if (cut && alias) {
        // in place: the loads of a round of ranks, then its
        // stores; rank r comes from a position >= r and ranks ascend, so no
        // store touches what a later round reads
        for (int r0 = 0; r0 < n_new; r0 += tn) {
            const int r = r0 + t0;
            float x = 0.0f;
            if (r < n_new) x = w_in[kept[r]];
            cluster_sync();
            if (r < n_new) w_out[r] = x;
        }
        cluster_sync();
    }
    // positions that tokens left have no weight
    for (int i = n_new + t0; i < len; i += tn) w_out[i] = 0.0f;
    if (warp == 0) {
        const uint32_t x = lane < C ? dsmem_ld_u32(dsmem_addr(smem_u32(&sh.in_place), lane)) : 0u;
        const bool in_place = __any_sync(0xffffffffu, x != 0);
        if (rank == 0 && lane == 0) p.flags[unit] = in_place ? 1 : 0;
    }
    // no CTA leaves while another may still read its shared memory
    cluster_sync();
}

// One CTA per unit, two CTAs per SM: the keys stay in shared memory as far as
// they fit (kCache of them), the rest is read again.  Every warp owns a
// contiguous run of the positions, so that no pass needs a barrier inside and
// every lane has 16-byte loads to overlap.  Protected and recent tokens get
// the key kSure, above every threshold, and need no further test.
//
// A histogram of every key would be bound by its shared-memory atomics (about
// one key per clock and SM).  So the first pass counts a sixteenth of the keys
// by their top 11 bits; the bins that hold the wanted rank of this sample
// give or take four standard deviations bound a range of keys, and the next
// pass counts what lies above the range in registers and only the keys in it
// in 2048 finer bins.  Where the range turns out not to hold the threshold,
// and for few keys, the range is the whole of the keys.  One or two more
// passes over the bin found end at a single key.
constexpr int kOneThreads = 512;
constexpr int kOneWarps = kOneThreads / 32;
constexpr int kCache = 24 * 1024;              // keys in shared memory: 96 KiB
constexpr uint32_t kSure = 0xffffffffu;        // no weight has it (NaN: 0, infinity: 0xff800000)

struct OneShared {
    uint32_t hist[2048 * 2];       // two interleaved copies, by lane parity
    uint32_t digit, low_digit, above, total, in_place;
    uint32_t warp_n[kOneWarps], warp_q[kOneWarps];
};

__global__ void __launch_bounds__(kOneThreads, 2) evict_select_one_kernel(const EvictArgs p, const int per_warp) {
    extern __shared__ __align__(16) uint32_t key_s[];
    __shared__ OneShared sh;
    const CacheDesc& c = p.c;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int unit = blockIdx.x, s = unit / c.Hkv;
    const int cap = c.max_pages * kPage;
    if (tid == 0) sh.in_place = 0;
    for (int i = tid; i < 4096; i += kOneThreads) sh.hist[i] = 0;
    pdl_wait();
    if (p.early) pdl_trigger();
    int len = c.seq_lens[s];
    if (len < 0 || len > cap) {
        if (tid == 0) set_error(p.err, ABSP_ERR_DEVICE_FAULT, s);
        len = 0;
    }
    const int keep = p.keep, n_new = min(len, keep);
    const bool cut = len > keep;
    const float* w_in = p.weights_in + static_cast<int64_t>(unit) * cap;
    float* w_out = p.weights_out + static_cast<int64_t>(unit) * cap;
    const bool alias = w_in == w_out;
    int32_t* kept = p.kept + static_cast<int64_t>(unit) * keep;
    __syncthreads();
    if (!p.compact && cut) {
        // protected tokens never move, so only the pages behind them matter
        const int32_t* src_row = c.page_table + static_cast<int64_t>(s) * c.max_pages;
        const int32_t* dst_row = p.dst_table + static_cast<int64_t>(s) * p.dst_max_pages;
        for (int i = p.protect / kPage + tid; i < (n_new + kPage - 1) / kPage; i += kOneThreads)
            if (dst_row[i] == src_row[i]) sh.in_place = 1;
    }
    if (cut) {
        const int a = p.protect, b = len - p.recent;     // the middle
        uint32_t left = static_cast<uint32_t>(keep - p.protect - p.recent);
        const int run = (len + 128 * kOneWarps - 1) / (128 * kOneWarps) * 128;
        const int i0 = min(len, warp * run), i1 = min(len, i0 + run);
        // each run's first per_warp keys are cached: every warp reads again
        // the same share, and none keeps the others waiting
        const int cached = i0 + per_warp;
        uint32_t* const cache = key_s + warp * per_warp - i0;
        // the keys of the lane's four positions from i on, from their weights
        auto keys_of = [&](int i, const float4& v) {
            uint4 k = make_uint4(key_of(v.x), key_of(v.y), key_of(v.z), key_of(v.w));
            if (i < a || i + 3 >= b) {
                if (i < a || i >= b) k.x = kSure;
                if (i + 1 < a || i + 1 >= b) k.y = kSure;
                if (i + 2 < a || i + 2 >= b) k.z = kSure;
                if (i + 3 < a || i + 3 >= b) k.w = kSure;
                // behind the end: below every threshold and never equal to it,
                // as equal keys are taken from the front
                if (i + 1 >= len) k.y = 0u;
                if (i + 2 >= len) k.z = 0u;
                if (i + 3 >= len) k.w = 0u;
            }
            return k;
        };
        // Keys of four steps of the run (positions i + 128 u), all loads
        // before their first use: neither the cache's stores nor atomics
        // stand between them.  `fill` writes the cache.
        auto fetch = [&](int i, bool fill, uint4 (&k)[4]) {
            float4 v[4];
#pragma unroll
            for (int u = 0; u < 4; ++u)
                if (i + 128 * u < i1 && (fill || i + 128 * u >= cached))
                    v[u] = *reinterpret_cast<const float4*>(w_in + i + 128 * u);   // rows end on whole pages
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const int at = i + 128 * u;
                if (at < i1) {
                    if (!fill && at < cached) {
                        k[u] = *reinterpret_cast<const uint4*>(cache + at);
                    } else {
                        k[u] = keys_of(at, v[u]);
                        if (at < cached) *reinterpret_cast<uint4*>(cache + at) = k[u];
                    }
                }
            }
        };
        auto pass = [&](bool first, auto f) {
#pragma unroll 1
            for (int i = i0 + 4 * lane; i < i1; i += 512) {
                uint4 k[4];
                fetch(i, first, k);
#pragma unroll
                for (int u = 0; u < 4; ++u)
                    if (i + 128 * u < i1) f(k[u], u);
            }
        };
        uint32_t* const hist = sh.hist + (lane & 1);
        // Adds the bins: n of this thread's four (2047 - 4t down to 2044 - 4t),
        // v each, `before` those above them; clears them for the next pass.
        uint32_t v[4], n, before;
        auto gather = [&] {
            uint4* const own = reinterpret_cast<uint4*>(&sh.hist[8 * (511 - tid)]);
            const uint4 x = own[0], y = own[1];
            own[0] = own[1] = make_uint4(0u, 0u, 0u, 0u);
            v[0] = y.z + y.w;
            v[1] = y.x + y.y;
            v[2] = x.z + x.w;
            v[3] = x.x + x.y;
            n = (v[0] + v[1]) + (v[2] + v[3]);
            uint32_t incl = n;
            for (int d = 1; d < 32; d *= 2) {
                const uint32_t z = __shfl_up_sync(0xffffffffu, incl, d);
                if (lane >= d) incl += z;
            }
            if (lane == 31) sh.warp_n[warp] = incl;
            __syncthreads();
            before = __reduce_add_sync(0xffffffffu, lane < warp ? sh.warp_n[lane] : 0u) + incl - n;
            if (tid == kOneThreads - 1) sh.total = before + n;
        };
        // the bin of this thread that holds the rank-th count from the top
        auto bin_of = [&](uint32_t rank, uint32_t* above) {
            uint32_t at = before;
            int j = 0;
#pragma unroll
            for (int k = 0; k < 3; ++k)
                if (j == k && at + v[k] < rank) {
                    at += v[k];
                    ++j;
                }
            *above = at;
            return static_cast<uint32_t>(2047 - 4 * tid - j);
        };
        uint32_t prefix = kSure - 1;    // the threshold; nothing but kSure is above this one
        if (left == 0) {
            pass(true, [](uint4, int) {});
        } else {
            uint32_t lo = 0, end = kSure - 1;   // the threshold lies in lo .. end
            int w = 32;                         // end - lo < 2^w
            bool first = true, bounded = false;
            if (b - a >= 4096) {
                pass(true, [&](uint4 k, int u) {
                    if (u == 0 && k.x != kSure) atomicAdd(hist + (k.x >> 21) * 2, 1u);
                });
                first = false;
                if (tid == 0) {
                    sh.digit = 2047;
                    sh.low_digit = 0;
                }
                __syncthreads();
                gather();
                __syncthreads();
                const float m = static_cast<float>(sh.total);
                const float at = m * (static_cast<float>(left) / static_cast<float>(b - a));
                const float d = 2.0f * sqrtf(m) + 8.0f;
                const uint32_t r_hi = at > d + 1.0f ? static_cast<uint32_t>(at - d) : 0u;
                const uint32_t r_lo = static_cast<uint32_t>(at + d);
                uint32_t u;
                if (r_hi > 0 && before < r_hi && before + n >= r_hi) sh.digit = bin_of(r_hi, &u);
                if (before < r_lo && before + n >= r_lo) sh.low_digit = bin_of(r_lo, &u);
                __syncthreads();
                lo = sh.low_digit << 21;
                end = min(kSure - 1, (sh.digit << 21) + 0x1fffffu);
                w = 32 - __clz(end - lo);       // 21 bits or more
                bounded = true;
            }
            for (;;) {
                const int shift = max(0, w - 11);
                const uint32_t range = end - lo;
                uint32_t over = 0;
                pass(first, [&](uint4 k, int) {
                    over += (k.x > end) + (k.y > end) + (k.z > end) + (k.w > end);
                    if (k.x - lo <= range) atomicAdd(hist + ((k.x - lo) >> shift) * 2, 1u);
                    if (k.y - lo <= range) atomicAdd(hist + ((k.y - lo) >> shift) * 2, 1u);
                    if (k.z - lo <= range) atomicAdd(hist + ((k.z - lo) >> shift) * 2, 1u);
                    if (k.w - lo <= range) atomicAdd(hist + ((k.w - lo) >> shift) * 2, 1u);
                });
                first = false;
                over = __reduce_add_sync(0xffffffffu, over);
                if (lane == 0) sh.warp_q[warp] = over;
                __syncthreads();
                gather();
                // keys above the range that are not there for sure
                over = __reduce_add_sync(0xffffffffu, lane < kOneWarps ? sh.warp_q[lane] : 0u) -
                       static_cast<uint32_t>(a + len - b);
                const uint32_t rank = left - over;
                uint32_t above;
                if (left > over && before < rank && before + n >= rank) {
                    sh.digit = bin_of(rank, &above);
                    sh.above = above;
                }
                __syncthreads();
                const uint32_t total = sh.total, digit = sh.digit, up = sh.above;
                __syncthreads();
                if (bounded && (left <= over || rank > total)) {   // outside the sample's range
                    bounded = false;
                    lo = 0;
                    end = kSure - 1;
                    w = 32;
                    continue;
                }
                bounded = false;
                lo += digit << shift;
                end = min(end, lo + ((1u << shift) - 1u));
                w = shift;
                if (shift == 0) {
                    prefix = lo;
                    left = rank - up;      // keys equal to the threshold that stay
                    break;
                }
            }
        }
        // ---- kept for sure and equal to the threshold, per run
        uint32_t n_sure = 0, n_equal = 0;
        pass(false, [&](uint4 k, int) {
            n_sure += (k.x > prefix) + (k.y > prefix) + (k.z > prefix) + (k.w > prefix);
            n_equal += (k.x == prefix) + (k.y == prefix) + (k.z == prefix) + (k.w == prefix);
        });
        n_sure = __reduce_add_sync(0xffffffffu, n_sure);
        n_equal = __reduce_add_sync(0xffffffffu, n_equal);
        if (lane == 0) {
            sh.warp_n[warp] = n_sure;
            sh.warp_q[warp] = n_equal;
        }
        __syncthreads();
        const uint32_t sure0 = __reduce_add_sync(0xffffffffu, lane < warp ? sh.warp_n[lane] : 0u);
        const uint32_t equal0 = __reduce_add_sync(0xffffffffu, lane < warp ? sh.warp_q[lane] : 0u);
        uint32_t at = sure0 + min(equal0, left);         // rank of the run's first kept token
        uint32_t ties = left - min(equal0, left);        // equal keys still to take
        // ---- the list
        const uint32_t below = (1u << lane) - 1u;
#pragma unroll 1
        for (int j0 = i0; j0 < i1; j0 += 512) {
            uint4 k4[4];
            fetch(j0 + 4 * lane, false, k4);
#pragma unroll
            for (int step = 0; step < 4; ++step) {       // every lane takes part
                const int i = j0 + 128 * step + 4 * lane;
                if (j0 + 128 * step >= i1) break;
                uint32_t u = 0, q = 0;
                if (i < i1) {
                    const uint4 k = k4[step];
                    u = (k.x > prefix ? 1u : 0u) | (k.y > prefix ? 2u : 0u) | (k.z > prefix ? 4u : 0u) |
                        (k.w > prefix ? 8u : 0u);
                    q = (k.x == prefix ? 1u : 0u) | (k.y == prefix ? 2u : 0u) | (k.z == prefix ? 4u : 0u) |
                        (k.w == prefix ? 8u : 0u);
                }
                if (__any_sync(0xffffffffu, q != 0)) {       // ties join in order while some are wanted
                    uint32_t before = 0, all = 0;
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const uint32_t m = __ballot_sync(0xffffffffu, q >> e & 1);
                        before += __popc(m & below);
                        all += __popc(m);
                    }
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (q >> e & 1) {
                            if (before < ties) u |= 1u << e;
                            ++before;
                        }
                    ties -= min(ties, all);
                }
                uint32_t before = 0, all = 0;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const uint32_t m = __ballot_sync(0xffffffffu, u >> e & 1);
                    before += __popc(m & below);
                    all += __popc(m);
                }
                uint32_t r = at + before;
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (u >> e & 1) kept[r++] = i + e;
                at += all;
            }
        }
    } else {
        // (64 bits: the last step behind the largest keep passes 2^31)
        for (int64_t i = tid; i < keep; i += kOneThreads) kept[i] = i < len ? static_cast<int32_t>(i) : -1;
        if (!alias)
            for (int i = tid; i < len; i += kOneThreads) w_out[i] = w_in[i];
    }
    __syncthreads();
    if (cut) {
        // the kept weights, also in place: the loads of a round of ranks, then
        // its stores; rank r comes from a position >= r and ranks ascend, so
        // no store touches what a later round reads
        for (int r0 = 0; r0 < n_new; r0 += 4 * kOneThreads) {
            float x[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int r = r0 + k * kOneThreads + tid;
                if (r < n_new) x[k] = w_in[kept[r]];
            }
            if (alias) __syncthreads();
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int r = r0 + k * kOneThreads + tid;
                if (r < n_new) w_out[r] = x[k];
            }
        }
        if (alias) __syncthreads();
        // positions that tokens left have no weight (whole 16 bytes where four go)
        const int z = (n_new + 3) & ~3, e = len & ~3;
        if (tid < z - n_new && n_new + tid < len) w_out[n_new + tid] = 0.0f;
        for (int i = z + 4 * tid; i < e; i += 4 * kOneThreads)
            *reinterpret_cast<float4*>(w_out + i) = make_float4(0.f, 0.f, 0.f, 0.f);
        if (e >= z && tid < len - e) w_out[e + tid] = 0.0f;
    }
    if (tid == 0) p.flags[unit] = sh.in_place != 0 ? 1 : 0;
}

// A warp moves 32 ranks: lane j finds the place of row j, then the rows go in
// batches of kRows, all loads of a batch in flight together.  Lanes 0..15
// hold a K row, 16..31 the V row.  What counts is bytes in flight: four
// blocks of 256 threads per SM keep 128 KiB of loads outstanding.
constexpr int kRows = 8;
constexpr int kCopyThreads = 256;

// Where the row of rank r comes from and goes to, as row indices of the page
// pools (below 2^31 by the layer checks); `to` is -1 for a row that stays
// where it is or has a bad page.
__device__ __forceinline__ void row_of(const EvictArgs& p, int s, int h, int r, int from, int* src,
                                       int* to) {
    const CacheDesc& c = p.c;
    const int sp = c.page_table[static_cast<int64_t>(s) * c.max_pages + from / kPage];
    const int dp = p.dst_table[static_cast<int64_t>(s) * p.dst_max_pages + r / kPage];
    if (sp < 0 || sp >= c.num_phys_pages || dp < 0 || dp >= c.num_phys_pages) {
        set_error(p.err, ABSP_ERR_DEVICE_FAULT, s);
    } else if (from != r || sp != dp) {
        *src = (sp * c.Hkv + h) * kPage + from % kPage;
        *to = (dp * c.Hkv + h) * kPage + r % kPage;
    }
}

__device__ __forceinline__ int new_len(const EvictArgs& p, int s) {
    // the lengths may be replaced by this launch: both values give the same
    const int len = *(volatile const int32_t*)(p.c.seq_lens + s);
    return len < 0 || len > p.c.max_pages * kPage ? 0 : min(len, p.keep);
}

// Rows j0 .. j0 + kRows - 1 of the warp's places; `between` runs after the
// loads.
template <typename F>
__device__ __forceinline__ void move_batch(__nv_bfloat16* pages, int src, int to, int j0, F between) {
    uint4 v[kRows];
#pragma unroll
    for (int j = 0; j < kRows; ++j) {
        const int from = __shfl_sync(0xffffffffu, src, j0 + j);
        if (from >= 0) v[j] = *reinterpret_cast<const uint4*>(pages + static_cast<int64_t>(from) * kD);
    }
    between();
#pragma unroll
    for (int j = 0; j < kRows; ++j) {
        const int at = __shfl_sync(0xffffffffu, to, j0 + j);
        if (at >= 0) *reinterpret_cast<uint4*>(pages + static_cast<int64_t>(at) * kD) = v[j];
    }
}

// Ranks r0 .. r0 + kRows - 1.
template <typename F>
__device__ __forceinline__ void move_rows(const EvictArgs& p, int s, int h, const int32_t* kept, int r0,
                                          int n, F between) {
    const int lane = threadIdx.x & 31;
    int src = -1, to = -1;
    if (lane < kRows && r0 + lane < n) row_of(p, s, h, r0 + lane, kept[r0 + lane], &src, &to);
    move_batch((lane < 16 ? p.k_pages : p.v_pages) + (lane & 15) * 8, src, to, 0, between);
}

// Every row on its own, a warp per `ranks` (8, 16 or 32) ranks of one unit.
// The warps of a block take the heads of a sequence side by side: the same
// ranks of its heads go to the same pages and come from nearby ones, so a
// block's address translations are shared by its warps (pages lie anywhere in
// pools of gigabytes).  The bound of 64 registers spills eight words of set-up
// per thread.  A unit with a destination page, behind the protected ones, that
// is its own source page is compacted by its first warp alone, in order, eight
// rows per round trip: 1.4 ms for 32 x 32K tokens cut to 4096, where
// evict_compact_kernel takes 0.2 ms, 3.1 ms for one sequence cut to 8192.
__global__ void __launch_bounds__(kCopyThreads, 4)
    evict_copy_kernel(const EvictArgs p, const int groups, const int ranks) {
    const CacheDesc& c = p.c;
    const int lane = threadIdx.x & 31;
    const int64_t wid = static_cast<int64_t>(blockIdx.x) * (kCopyThreads / 32) + (threadIdx.x >> 5);
    const int h = static_cast<int>(wid % c.Hkv);
    const int sg = static_cast<int>(wid / c.Hkv);
    const int s = sg / groups, b = sg - s * groups;
    pdl_wait();
    if (s >= c.S) return;
    const int unit = s * c.Hkv + h;
    const int n = new_len(p, s);
    const int32_t* kept = p.kept + static_cast<int64_t>(unit) * p.keep;
    if (p.flags[unit] == 0) {
        const int r0 = b * ranks;
        if (r0 < n) {
            int src = -1, to = -1;
            if (lane < ranks && r0 + lane < n) row_of(p, s, h, r0 + lane, kept[r0 + lane], &src, &to);
            __nv_bfloat16* const pages = (lane < 16 ? p.k_pages : p.v_pages) + (lane & 15) * 8;
#pragma unroll 1
            for (int j = 0; j < ranks; j += kRows) move_batch(pages, src, to, j, [] {});
        }
    } else if (b == 0) {
        // a batch's stores lie below what later batches read
        for (int r0 = 0; r0 < n; r0 += kRows) move_rows(p, s, h, kept, r0, n, [] { __syncwarp(); });
    }
    if (h == 0 && b == 0 && lane == 0) p.new_lens[s] = n;
}

// The destination table is the page table: a cluster per unit moves the rows
// in rounds of ranks, all loads of a round, a cluster barrier, its stores.
// Rank r comes from a position >= r and ranks ascend, so a round's stores
// never touch what a later round reads.
__global__ void __launch_bounds__(kThreads) evict_compact_kernel(const EvictArgs p) {
    constexpr int kRound = kWarpsE * kRows;
    const CacheDesc& c = p.c;
    const int warp = threadIdx.x >> 5;
    const int C = static_cast<int>(cluster_nctarank()), rank = static_cast<int>(cluster_ctarank());
    const int unit = blockIdx.x / C;
    const int s = unit / c.Hkv, h = unit - s * c.Hkv;
    pdl_wait();
    const int n = new_len(p, s);
    const int32_t* kept = p.kept + static_cast<int64_t>(unit) * p.keep;
    for (int r0 = 0; r0 < n; r0 += C * kRound)
        move_rows(p, s, h, kept, r0 + rank * kRound + warp * kRows, n, [] { cluster_sync(); });
    if (h == 0 && rank == 0 && threadIdx.x == 0) p.new_lens[s] = n;
}

template <typename K, typename... A>
cudaError_t launch(K kern, int most_smem, int grid, int threads, int cluster, int smem, bool pdl, cudaStream_t st,
                   std::atomic<uint64_t>* done, A... args) {
    const cudaError_t e = prepare_kernel(kern, most_smem, cluster > 0, done);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    int n = 0;
    if (cluster > 0) {
        attr[n].id = cudaLaunchAttributeClusterDimension;
        attr[n].val.clusterDim.x = cluster;
        attr[n].val.clusterDim.y = 1;
        attr[n++].val.clusterDim.z = 1;
    }
    if (pdl) {
        attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[n++].val.programmaticStreamSerializationAllowed = 1;
    }
    cfg.attrs = attr;
    cfg.numAttrs = n;
    return cudaLaunchKernelEx(&cfg, kern, args...);
}

}  // namespace

cudaError_t launch_evict(const EvictArgs& args, bool pdl, cudaStream_t st) {
    EvictArgs a = args;
    static std::atomic<uint64_t> done_cluster{0}, done_one{0}, done_compact{0}, done_copy{0};
    const int units = a.c.S * a.c.Hkv;
    const int cap = a.c.max_pages * kPage;
    const int most = std::min(a.keep, cap);
    // Few rows to move: the move kernel's blocks all fit beside the select's
    // and start early, hiding their launch.  (Many that start early run on
    // SMs still set up for the select's shared memory: 166 us against 138 for
    // 800 MB of rows.)
    const bool few = static_cast<int64_t>(units) * ((most + 31) / 32) <= 32ll * device_sms();
    a.early = few ? 1 : 0;
    // CTAs per unit: as many as give every SM two, at most `most`
    const auto cluster_of = [&](int most) {
        int C = 1;
        while (C < kMaxCluster && C < most && static_cast<int64_t>(units) * C <= device_sms()) C *= 2;
        return C;
    };
    const int cs = units <= device_sms() / 2 ? cluster_of((cap + kChunk - 1) / kChunk) : 1;
    cudaError_t e;
    if (cs >= 4) {
        e = launch(evict_select_cluster_kernel, 0, units * cs, kThreads, cs, 0, pdl, st, &done_cluster, a);
    } else {
        const int run = (cap + 128 * kOneWarps - 1) / (128 * kOneWarps) * 128;
        const int per_warp = std::min(run, kCache / kOneWarps);
        e = launch(evict_select_one_kernel, kCache * 4, units, kOneThreads, 0, per_warp * kOneWarps * 4, pdl, st,
                   &done_one, a, per_warp);
    }
    if (e != cudaSuccess) return e;
    if (a.compact) {
        const int cc = cluster_of((most + kWarpsE * kRows - 1) / (kWarpsE * kRows));
        return launch(evict_compact_kernel, 0, units * cc, kThreads, cc, 0, pdl, st, &done_compact, a);
    }
    // up to 32 ranks per warp share one look-up of their places; fewer as long
    // as the SMs hold all warps at once
    int ranks = 32;
    while (ranks > kRows && units * ((2ll * most + ranks - 1) / ranks) <= 32ll * device_sms())
        ranks /= 2;
    const int groups = (most + ranks - 1) / ranks;
    const int64_t warps = static_cast<int64_t>(units) * groups;
    return launch(evict_copy_kernel, 0, static_cast<int>((warps + 7) / 8), kCopyThreads, 0, 0, pdl, st,
                  &done_copy, a, groups, ranks);
}

}  // namespace absp
