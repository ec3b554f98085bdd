// Exact decode attention over the whole paged cache, one new token per
// sequence, with optional accumulation of the attention weights.
//
// For (sequence s, KV head h) and the G query heads g of its group, in log2
// units x[g][t] = (q_g . K_t) * log2(e) / sqrt(128):
//   out_g = sum_t 2^(x[g][t] - m_g) V_t / l_g,   m_g = max_t x, l_g = sum_t 2^(x - m_g)
//   weights_out[t] = weights_in[t] + sum_g 2^(x[g][t] - m_g) / l_g.
// Partial results over disjoint token sets join exactly:
//   m = max m_i, l = sum l_i 2^(m_i - m), out = sum O_i 2^(m_i - m) / l.
//
// Two launches.  The split kernel lays all pages of all (s, h) units end to
// end and gives each warp of a one-CTA-per-SM grid an equal contiguous run,
// so any mix of lengths balances without a host-known plan; the warps of a
// CTA join the parts of the units they cut, a unit that one CTA holds whole
// is written by it, others leave partials.  The merge kernel joins the
// partials and turns the stored scores into weights.  Small calls take one
// launch: a cluster of CTAs per unit does all of it.
//
// What bounds the split kernel is reading K and V once (512 bytes per token
// and KV head, 4 G flops per byte): eight warps with three 8 KiB page buffers
// each keep 192 KiB of copies in flight per SM.  At the rows a token meets (G
// <= 16) the legacy 16-row matrix instruction has time to spare, where a
// 128-row tcgen05 tile would be mostly padding.  Measured on a B200, whole
// call: 96 x 16K tokens, 2 KV heads of 16 query heads (1.61 GB) 267 us, 6.0
// TB/s, 93 % of the measured copy bandwidth; a ragged batch of 32 with
// weights (1.68 GB and 0.1 GB of scores) 308 us, 84 %; one 32K sequence with
// weights (136 MB) 32.0 us, 66 %: about 19 us of streaming, the rest the
// dependent steps before it (lengths, page ids) and behind it (merge).
#include <algorithm>
#include <atomic>

#include "cache_ops.cuh"

namespace absp {

namespace {

constexpr int kThreads = kFullWarps * 32;
constexpr int kStages = 3;                  // page buffers per warp
constexpr int kSlice = kPage * kD * 2;      // 4 KiB: one page of one head
constexpr int kStageBytes = 2 * kSlice;     // K and V
constexpr int kCumCap = 2048;               // sampled entries of the cumulative page counts
constexpr int kSplitSmem = 1024 + kFullWarps * kStages * kStageBytes;

// What a warp's run leaves to be joined with its neighbours': the parts of
// the units that it does not hold whole.
struct RunEnds {
    int32_t first_unit;       // unit that the run starts in the middle of, or -1
    int32_t last_unit;        // unit that the run ends in the middle of, or -1
    const float* first;       // [G][128] unnormalised outputs; a run inside one
    const float* last;        // unit has a single part, its first
};

struct SplitShared {
    uint64_t bar[kFullWarps][kStages];
    int32_t cum[kCumCap];
    int32_t warp_sum[kFullWarps];
    RunEnds ends[kFullWarps];
    float2 ml[kFullWarps][2][ABSP_MAX_GROUP];   // of the first and the last part
    float2 cta_ml[ABSP_MAX_GROUP];              // of the CTA's part (read by the cluster)
    float lse[ABSP_MAX_GROUP];
};

__device__ __forceinline__ float4 dsmem_ld_f32x4(uint32_t addr) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(addr));
    return v;
}

__device__ __forceinline__ float2 dsmem_ld_f32x2(uint32_t addr) {
    float2 v;
    asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(addr));
    return v;
}

__device__ __forceinline__ uint32_t ld_u32g(const __nv_bfloat16* p) {
    return __ldg(reinterpret_cast<const uint32_t*>(p));
}

// Pages that sequence s attends to by itself, and their first token.
__device__ __forceinline__ int own_pages(const CacheDesc& c, int s, int32_t* err, int* start,
                                         int* len) {
    *len = checked_len(c, s, err);
    *start = own_start(c, *len);
    return (*len - *start + kPage - 1) / kPage;
}

// Adds up to four tokens' weights from their stored scores (rows of weights
// and scores end on whole pages, so four tokens can always be read).
__device__ __forceinline__ void add_weights(const FullArgs& p, int64_t score_at, int64_t at, int n, int cap,
                                            const float* lse) {
    float4 w = make_float4(0.f, 0.f, 0.f, 0.f), v = w;
    if (p.weights_in != nullptr) v = *reinterpret_cast<const float4*>(p.weights_in + at);
    for (int g = 0; g < p.c.G; ++g) {
        const float4 x = *reinterpret_cast<const float4*>(p.ws.scores + score_at + static_cast<int64_t>(g) * cap);
        w.x += exp2_approx(x.x - lse[g]);
        w.y += exp2_approx(x.y - lse[g]);
        w.z += exp2_approx(x.z - lse[g]);
        w.w += exp2_approx(x.w - lse[g]);
    }
    w = make_float4(v.x + w.x, v.y + w.y, v.z + w.z, v.w + w.w);
    if (n == 4) {
        *reinterpret_cast<float4*>(p.weights_out + at) = w;
    } else {
        const float y[4] = {w.x, w.y, w.z, w.w};
        for (int i = 0; i < n; ++i) p.weights_out[at + i] = y[i];
    }
}

// Slots of the partial results: two per CTA (the unit that its run starts in
// the middle of; the one that it ends in the middle of), then one per unit.
__device__ __forceinline__ int64_t unit_slot(const FullArgs& p, int unit) {
    return 2ll * (p.workers / kFullWarps) + unit;
}

// BIG: a GQA group of 9..16 heads fills the 16 rows of the matrix tile.
// Otherwise rows 0..7 hold the group and rows 8..15 carry, in the product
// with V, the remainder of the probabilities' rounding to bf16 (p = hi + lo,
// two bf16 numbers: 16 bits of mantissa), at no further matrix instruction;
// with BIG the remainder takes a second product, hidden behind the copies.
// Alone, hi would put an error of the output's own rounding on top of it.
//
// UNIT: a cluster of CTAs takes one unit, its pages cut evenly over the
// cluster's warps, and joins the parts through distributed shared memory:
// outputs and weights are complete, no merge kernel follows (unit_cluster
// says where).
template <bool BIG, bool WEIGHTS, bool UNIT>
__global__ void __launch_bounds__(kThreads, 1)
    full_split_kernel(const FullArgs p, const __grid_constant__ CUtensorMap tmk,
                      const __grid_constant__ CUtensorMap tmv) {
    extern __shared__ uint8_t dyn[];
    __shared__ SplitShared sh;
    uint8_t* ring = dyn + ((1024 - (smem_u32(dyn) & 1023)) & 1023);
    const CacheDesc& c = p.c;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid < kFullWarps * kStages) mbar_init(smem_u32(&sh.bar[0][0] + tid), 1);
    fence_mbar_init();
    if (tid == 0) {
        prefetch_tensormap(&tmk);
        prefetch_tensormap(&tmv);
    }
    // behind the prefix kernel, which waited for everything earlier, this
    // kernel starts while that one still runs and waits for it at its end
    // (the merge, which waits for this kernel, reads the results of both)
    if (p.prefix_ctas == 0) pdl_wait();
    pdl_trigger();

    int f0, f1, step = 1;
    const int worker = blockIdx.x * kFullWarps + warp;
    const int cluster = UNIT ? static_cast<int>(cluster_nctarank()) : 1;
    const int rank = UNIT ? static_cast<int>(cluster_ctarank()) : 0;
    int us, uh, up, un, ustart, ulen;
    if constexpr (UNIT) {
        // f counts the unit's pages; the warps of one CTA far apart, so that
        // a few pages spread over all CTAs
        const int unit = blockIdx.x / cluster;
        us = unit / c.Hkv;
        uh = unit - us * c.Hkv;
        un = own_pages(c, us, p.ws.err, &ustart, &ulen);
        const int chunk = (un + cluster * kFullWarps - 1) / (cluster * kFullWarps);
        f0 = min(un, (warp * cluster + rank) * chunk);
        f1 = min(un, f0 + chunk);
        up = f0;
        __syncthreads();   // the barriers are set up
    } else {
        // cumulative own pages (per KV head) of the sequences; every step-th
        // value stays in shared memory, block 0 writes all for the merge
        step = (c.S + kCumCap - 1) / kCumCap;
        int base = 0;
        for (int s0 = 0; s0 < c.S; s0 += kThreads) {
            const int s = s0 + tid;
            int start, len;
            const int n = s < c.S ? own_pages(c, s, p.ws.err, &start, &len) : 0;
            int x = n;
#pragma unroll
            for (int d = 1; d < 32; d *= 2) {
                const int y = __shfl_up_sync(0xffffffffu, x, d);
                if (lane >= d) x += y;
            }
            if (lane == 31) sh.warp_sum[warp] = x;
            __syncthreads();
            int before = base, all = 0;
            for (int w = 0; w < kFullWarps; ++w) {
                if (w < warp) before += sh.warp_sum[w];
                all += sh.warp_sum[w];
            }
            if (s < c.S) {
                if (s % step == 0) sh.cum[s / step] = before + x - n;
                if (blockIdx.x == 0) p.ws.cum[s] = before + x - n;
            }
            base += all;
            __syncthreads();
        }
        if (blockIdx.x == 0 && tid == 0) p.ws.cum[c.S] = base;
        const int total = base * c.Hkv;
        const int chunk = (total + p.workers - 1) / p.workers;
        f0 = static_cast<int>(min(static_cast<int64_t>(worker) * chunk, static_cast<int64_t>(total)));
        f1 = min(f0 + chunk, total);
        if (lane == 0) sh.ends[warp] = RunEnds{-1, -1, nullptr, nullptr};
    }
    bool gave_up = false;      // the same in every lane
    if (f0 < f1) {
        // the unit and page that run position f0 falls on
        if constexpr (!UNIT) {
            int lo = 0, hi = (c.S - 1) / step;
            while (lo < hi) {
                const int mid = (lo + hi + 1) >> 1;
                if (static_cast<int64_t>(sh.cum[mid]) * c.Hkv <= f0) lo = mid; else hi = mid - 1;
            }
            us = lo * step;
            int before = sh.cum[lo];
            un = own_pages(c, us, p.ws.err, &ustart, &ulen);
            while (static_cast<int64_t>(before + un) * c.Hkv <= f0 && us + 1 < c.S) {
                before += un;
                un = own_pages(c, ++us, p.ws.err, &ustart, &ulen);
            }
            const int r = f0 - before * c.Hkv;
            // (lengths that change during the call end the walk, not the bounds)
            uh = min(r / max(un, 1), c.Hkv - 1);
            up = r - uh * un;
        }

        const uint32_t ring_s = smem_u32(ring) + warp * kStages * kStageBytes;
        uint8_t* ring_g = ring + warp * kStages * kStageBytes;
        const uint32_t bars = smem_u32(&sh.bar[warp][0]);

        // ---- producer: the same walk, kStages pages ahead
        int ps = us, ph = uh, pp = up, pn = un, pstart = ustart, pf = f0;
        int cbase = -64, my_phys = -1;   // page ids cbase .. cbase + 31 of the producer's unit
        uint32_t okmask = 0;
        // keys and values are read once: what stays in L2 is the scores
        const uint64_t policy = evict_first_policy();
        auto issue = [&](int st) {
            if (pp >= cbase + 32 || pp < cbase) {
                cbase = pp;
                my_phys = pp + lane < pn
                              ? c.page_table[static_cast<int64_t>(ps) * c.max_pages + pstart / kPage + pp + lane]
                              : -1;
            }
            const int phys = __shfl_sync(0xffffffffu, my_phys, pp - cbase);
            const bool ok = phys >= 0 && phys < c.num_phys_pages;
            okmask = ok ? okmask | (1u << st) : okmask & ~(1u << st);
            if (lane == 0) {
                if (!ok) set_error(p.ws.err, ABSP_ERR_DEVICE_FAULT, ps);
                const uint32_t bar = bars + 8 * st;
                mbar_arrive_expect_tx(bar, ok ? kStageBytes : 0);
                if (ok) {
                    const int y = (phys * c.Hkv + ph) * kPage;
                    tma_load_3d_hint(ring_s + st * kStageBytes, &tmk, 0, y, 0, bar, policy);
                    tma_load_3d_hint(ring_s + st * kStageBytes + kSlice, &tmv, 0, y, 0, bar, policy);
                }
            }
            ++pf;
            if (++pp == pn && pf < f1) {
                pp = 0;
                cbase = -64;
                if (++ph == c.Hkv) {
                    ph = 0;
                    int len;
                    do pn = own_pages(c, ++ps, p.ws.err, &pstart, &len); while (pn == 0 && ps + 1 < c.S);
                }
            }
        };
        for (int st = 0; st < kStages; ++st)
            if (pf < f1) issue(st);

        const int g = lane >> 2, t4 = lane & 3, mi = lane >> 3, ri = lane & 7;
        const float qks = kLog2E / sqrtf(static_cast<float>(kD));
        int stage = 0, phase = 0;
        int f = f0;
        while (f < f1 && up < un) {
            // ---- one unit, or the part of it in this run
            const int seg_end = min(f1, f - up + un);
            const bool cut_left = up != 0, cut_right = f - up + un > f1;
            const __nv_bfloat16* qg = p.q + (static_cast<int64_t>(us) * c.Hq + uh * c.G) * kD;
            uint32_t qx[8], qy[8], qz[8], qw[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                qx[j] = g < c.G ? ld_u32g(qg + g * kD + 16 * j + 2 * t4) : 0u;
                qy[j] = g < c.G ? ld_u32g(qg + g * kD + 16 * j + 8 + 2 * t4) : 0u;
                if constexpr (BIG) {
                    qz[j] = g + 8 < c.G ? ld_u32g(qg + (g + 8) * kD + 16 * j + 2 * t4) : 0u;
                    qw[j] = g + 8 < c.G ? ld_u32g(qg + (g + 8) * kD + 16 * j + 8 + 2 * t4) : 0u;
                }
            }
            float o[16][4];
#pragma unroll
            for (int i = 0; i < 16; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.0f;
            float m0 = -INFINITY, m8 = -INFINITY, l0 = 0.0f, l8 = 0.0f;
            float* sc = nullptr;
            if constexpr (WEIGHTS)
                sc = p.ws.scores + (static_cast<int64_t>(us) * c.Hq + uh * c.G) * c.max_pages * kPage;

            for (; f < seg_end; ++f, ++up) {
                if (!gave_up && __any_sync(0xffffffffu, !mbar_try_wait(bars + 8 * stage, phase))) {
                    mbar_wait_bounded(bars + 8 * stage, phase, p.ws.err, 16);
                    // a wait that gave up (the error is recorded) is the run's
                    // last: no further copies, what is left of the pages counts as
                    // bad, and copies under way are waited for before the end
                    if (__any_sync(0xffffffffu, !mbar_try_wait(bars + 8 * stage, phase))) {
                        gave_up = true;
                        pf = f1;
                        okmask = 0;
                    }
                }
                const int tok0 = ustart + up * kPage;
                const int valid = (okmask >> stage) & 1u ? min(kPage, ulen - tok0) : 0;
                const uint32_t kb = ring_s + stage * kStageBytes, vb = kb + kSlice;
                if (valid > 0 && valid < kPage) {
                    // V rows past the end may hold anything: 0 * NaN is NaN
                    uint8_t* vg = ring_g + stage * kStageBytes + kSlice;
                    const int nz = (kPage - valid) * 16;
                    for (int i = lane; i < nz; i += 32) {
                        const int row = valid + (i >> 4), half = (i >> 3) & 1;
                        *reinterpret_cast<uint4*>(vg + half * 2048 + row * 128 + (i & 7) * 16) =
                            make_uint4(0u, 0u, 0u, 0u);
                    }
                    __syncwarp();
                }
                const int ta = 2 * t4, tb = 8 + 2 * t4;
                float s0[4] = {0.f, 0.f, 0.f, 0.f}, s1[4] = {0.f, 0.f, 0.f, 0.f};
                if (valid > 0) {
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const int tok = (mi >> 1) * 8 + ri, ch = (j & 3) * 2 + (mi & 1);
                        uint32_t b0, b1, b2, b3;
                        ldsm_x4(kb + (j >> 2) * 2048 + tok * 128 + ((ch ^ ri) << 4), b0, b1, b2, b3);
                        if constexpr (BIG) {
                            mma_bf16(s0[0], s0[1], s0[2], s0[3], qx[j], qz[j], qy[j], qw[j], b0, b1);
                            mma_bf16(s1[0], s1[1], s1[2], s1[3], qx[j], qz[j], qy[j], qw[j], b2, b3);
                        } else {
                            mma_bf16_top(s0[0], s0[1], qx[j], qy[j], b0, b1);
                            mma_bf16_top(s1[0], s1[1], qx[j], qy[j], b2, b3);
                        }
                    }
                }
                // rows g (and g + 8): log2 units, nothing past the end
                auto row = [&](float a, float b, float cc, float d, int r, float& m, float& l, uint32_t& h0,
                               uint32_t& h1, uint32_t& r0, uint32_t& r1) -> float {
                    const float x0 = ta < valid ? a * qks : -INFINITY;
                    const float x1 = ta + 1 < valid ? b * qks : -INFINITY;
                    const float x2 = tb < valid ? cc * qks : -INFINITY;
                    const float x3 = tb + 1 < valid ? d * qks : -INFINITY;
                    if constexpr (WEIGHTS) {
                        if (r < c.G) {
                            float* at = sc + static_cast<int64_t>(r) * c.max_pages * kPage + tok0;
                            *reinterpret_cast<float2*>(at + ta) = make_float2(x0, x1);
                            *reinterpret_cast<float2*>(at + tb) = make_float2(x2, x3);
                        }
                    }
                    float mx = fmaxf(fmaxf(x0, x1), fmaxf(x2, x3));
                    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
                    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
                    const float mn = fmaxf(m, mx);
                    const float ms = mn == -INFINITY ? 0.0f : mn;
                    const float corr = exp2_approx(m - ms);
                    const float p0 = exp2_approx(x0 - ms), p1 = exp2_approx(x1 - ms);
                    const float p2 = exp2_approx(x2 - ms), p3 = exp2_approx(x3 - ms);
                    l = l * corr + ((p0 + p1) + (p2 + p3));
                    m = mn;
                    h0 = pack_bf16x2(p0, p1);
                    h1 = pack_bf16x2(p2, p3);
                    r0 = pack_bf16x2(p0 - bf16lo(h0), p1 - bf16hi(h0));
                    r1 = pack_bf16x2(p2 - bf16lo(h1), p3 - bf16hi(h1));
                    return corr;
                };
                uint32_t pa0, pa2, pr0, pr2, pa1 = 0u, pa3 = 0u, pr1 = 0u, pr3 = 0u;
                const float corr0 = row(s0[0], s0[1], s1[0], s1[1], g, m0, l0, pa0, pa2, pr0, pr2);
                float corr8 = corr0;
                if constexpr (BIG)
                    corr8 = row(s0[2], s0[3], s1[2], s1[3], g + 8, m8, l8, pa1, pa3, pr1, pr3);
                if (__any_sync(0xffffffffu, corr0 != 1.0f || corr8 != 1.0f)) {
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        o[i][0] *= corr0;
                        o[i][1] *= corr0;
                        o[i][2] *= corr8;
                        o[i][3] *= corr8;
                    }
                }
                if (valid > 0) {
#pragma unroll
                    for (int cc = 0; cc < 8; ++cc) {
                        const int tok = (mi & 1) * 8 + ri, ch = (cc & 3) * 2 + (mi >> 1);
                        uint32_t b0, b1, b2, b3;
                        ldsm_x4_trans(vb + (cc >> 2) * 2048 + tok * 128 + ((ch ^ ri) << 4), b0, b1, b2, b3);
                        float* oa = o[2 * cc];
                        float* ob = o[2 * cc + 1];
                        if constexpr (BIG) {
                            mma_bf16(oa[0], oa[1], oa[2], oa[3], pa0, pa1, pa2, pa3, b0, b1);
                            mma_bf16(ob[0], ob[1], ob[2], ob[3], pa0, pa1, pa2, pa3, b2, b3);
                            mma_bf16(oa[0], oa[1], oa[2], oa[3], pr0, pr1, pr2, pr3, b0, b1);
                            mma_bf16(ob[0], ob[1], ob[2], ob[3], pr0, pr1, pr2, pr3, b2, b3);
                        } else {
                            mma_bf16(oa[0], oa[1], oa[2], oa[3], pa0, pr0, pa2, pr2, b0, b1);
                            mma_bf16(ob[0], ob[1], ob[2], ob[3], pa0, pr0, pa2, pr2, b2, b3);
                        }
                    }
                }
                // the buffer's reads (and zeroing) before its next copy
                if (pf < f1) {
                    fence_proxy_async_smem();
                    __syncwarp();
                    issue(stage);
                }
                if (++stage == kStages) {
                    stage = 0;
                    phase ^= 1;
                }
            }

            // ---- the unit's result, or this run's part of it
            l0 += __shfl_xor_sync(0xffffffffu, l0, 1);
            l0 += __shfl_xor_sync(0xffffffffu, l0, 2);
            l8 += __shfl_xor_sync(0xffffffffu, l8, 1);
            l8 += __shfl_xor_sync(0xffffffffu, l8, 2);
            if constexpr (!BIG) {
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    o[i][0] += o[i][2];
                    o[i][1] += o[i][3];
                }
            }
            const int unit = us * c.Hkv + uh;
            const bool whole = !cut_left && !cut_right;
            // a part that later copies of this run cannot overwrite stays in the
            // warp's page buffers; an earlier one goes through the workspace
            const bool at_end = UNIT || f == f1;
            float* part = at_end ? reinterpret_cast<float*>(ring_g)
                                 : p.ws.scratch + static_cast<int64_t>(worker) * c.G * kD;
            __syncwarp();   // every lane is done reading the pages
            auto put = [&](int r, int e, float m, float l) {
                if (r >= c.G) return;
                if (!UNIT && whole && p.prefix_ctas == 0) {
                    const float rl = l > 0.0f ? 1.0f / l : (l == 0.0f ? 0.0f : l);
                    __nv_bfloat16* to = p.out + (static_cast<int64_t>(us) * c.Hq + uh * c.G + r) * kD;
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        *reinterpret_cast<uint32_t*>(to + 8 * i + 2 * t4) =
                            pack_bf16x2(o[i][e] * rl, o[i][e + 1] * rl);
                } else {
                    float* to = !UNIT && whole ? p.ws.o + (unit_slot(p, unit) * c.G + r) * kD : part + r * kD;
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        *reinterpret_cast<float2*>(to + 8 * i + 2 * t4) = make_float2(o[i][e], o[i][e + 1]);
                }
                if (t4 == 0) {
                    if (!UNIT && whole)
                        p.ws.ml[unit_slot(p, unit) * c.G + r] = make_float2(m, l);
                    else
                        sh.ml[warp][UNIT || cut_left ? 0 : 1][r] = make_float2(m, l);
                }
            };
            put(g, 0, m0, l0);
            if constexpr (BIG) put(g + 8, 2, m8, l8);
            if (lane == 0) {
                if (cut_left) {
                    sh.ends[warp].first_unit = unit;
                    sh.ends[warp].first = part;
                } else if (cut_right) {
                    sh.ends[warp].last = part;
                }
                if (cut_right) sh.ends[warp].last_unit = unit;
            }
            // next unit with pages
            up = 0;
            if (!UNIT && f < f1 && ++uh == c.Hkv) {
                uh = 0;
                do un = own_pages(c, ++us, p.ws.err, &ustart, &ulen); while (un == 0 && us + 1 < c.S);
            }
        }
    }
    if (gave_up) {
        // copies in flight end well within this time
        const uint64_t t0 = globaltimer_ns();
        while (globaltimer_ns() - t0 < 10000000ull) {
        }
    }
    __syncthreads();

    if constexpr (UNIT) {
        // ---- the CTA's part: a warp per head, eight warps' parts at most
        float* cta_o = reinterpret_cast<float*>(ring + kStageBytes);   // behind warp 0's own part
        for (int r = warp; r < c.G; r += kFullWarps) {
            float m = -INFINITY, l = 0.0f;
            float2 ml[kFullWarps];
            float4 v[kFullWarps];
#pragma unroll
            for (int k = 0; k < kFullWarps; ++k) {
                // (runs ascend with the warp: an empty one ends the list)
                const int chunk = (un + cluster * kFullWarps - 1) / (cluster * kFullWarps);
                const bool has = (k * cluster + rank) * chunk < un;
                ml[k] = has ? sh.ml[k][0][r] : make_float2(-INFINITY, 0.0f);
                v[k] = has ? reinterpret_cast<const float4*>(ring + k * kStages * kStageBytes + r * kD * 4)[lane]
                           : make_float4(0.f, 0.f, 0.f, 0.f);
                m = fmaxf(m, ml[k].x);
            }
            const float ms = m == -INFINITY ? 0.0f : m;
            float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int k = 0; k < kFullWarps; ++k) {
                const float e = exp2_approx(ml[k].x - ms);
                l = fmaf(ml[k].y, e, l);
                a.x = fmaf(v[k].x, e, a.x);
                a.y = fmaf(v[k].y, e, a.y);
                a.z = fmaf(v[k].z, e, a.z);
                a.w = fmaf(v[k].w, e, a.w);
            }
            reinterpret_cast<float4*>(cta_o + r * kD)[lane] = a;
            if (lane == 0) sh.cta_ml[r] = make_float2(m, l);
        }
        cluster_arrive();
        cluster_wait();
        // ---- the unit's output: head r by CTA r mod the cluster; with weights
        // every CTA needs every head's statistics
        for (int r = warp; r < c.G; r += kFullWarps) {
            const bool mine = r % cluster == rank;
            if (!WEIGHTS && !mine) continue;
            float2 x = make_float2(-INFINITY, 0.0f);
            if (lane < cluster) x = dsmem_ld_f32x2(dsmem_addr(smem_u32(&sh.cta_ml[r]), lane));
            float m = x.x;
            for (int d = 16; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
            const float ms = m == -INFINITY ? 0.0f : m;
            const float e = exp2_approx(x.x - ms);
            float l = x.y * e;
            for (int d = 16; d > 0; d >>= 1) l += __shfl_xor_sync(0xffffffffu, l, d);
            if (lane == 0) sh.lse[r] = l == 0.0f ? INFINITY : m + log2f(l);
            if (!mine) continue;
            float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
            const uint32_t from = smem_u32(cta_o + r * kD) + lane * 16;
#pragma unroll 8
            for (int k = 0; k < cluster; ++k) {
                const float ek = __shfl_sync(0xffffffffu, e, k);
                const float4 v = dsmem_ld_f32x4(dsmem_addr(from, k));
                a.x = fmaf(v.x, ek, a.x);
                a.y = fmaf(v.y, ek, a.y);
                a.z = fmaf(v.z, ek, a.z);
                a.w = fmaf(v.w, ek, a.w);
            }
            const float rl = l > 0.0f ? 1.0f / l : (l == 0.0f ? 0.0f : l);
            reinterpret_cast<uint2*>(p.out + (static_cast<int64_t>(us) * c.Hq + uh * c.G + r) * kD)[lane] =
                make_uint2(pack_bf16x2(a.x * rl, a.y * rl), pack_bf16x2(a.z * rl, a.w * rl));
        }
        cluster_arrive();      // (after it no shared memory of another CTA is read)
        if constexpr (WEIGHTS) {
            __syncthreads();
            // the tokens of this warp's own run
            const int cap = c.max_pages * kPage;
            const int64_t row0 = (static_cast<int64_t>(us) * c.Hq + uh * c.G) * cap;
            const int64_t at0 = (static_cast<int64_t>(us) * c.Hkv + uh) * cap;
            const int from_t = ulen >= p.weights_from ? p.weights_from : 0;
            for (int t = max(f0 * kPage, from_t) + 4 * lane; t < f1 * kPage && t < ulen; t += 128)
                add_weights(p, row0 + t, at0 + t, min(4, ulen - t), cap, sh.lse);
        }
        cluster_wait();
        return;
    }
    // ---- join the warps' parts of the units that this CTA's runs cut.  A
    // chain of parts begins with a run's last part, or with the first warp's
    // first part (of a unit that began in an earlier CTA), and goes on with
    // the first parts of the warps behind it.  A warp per chain and four
    // heads, whose loads are in flight together.
    const uint32_t lasts = __ballot_sync(
        0xffffffffu, lane < kFullWarps && sh.ends[lane & 7].last_unit >= 0 &&
                         sh.ends[lane & 7].last_unit != sh.ends[lane & 7].first_unit);
    const int left0 = sh.ends[0].first_unit >= 0 ? 1 : 0;
    const int quads = (c.G + 3) / 4;
    const int items = (__popc(lasts) + left0) * quads;
    for (int it = warp; it < items; it += kFullWarps) {
        const int chain = it / quads, r0 = (it - chain * quads) * 4;
        const bool left_open = left0 != 0 && chain == 0;
        const int w0 = left_open ? 0 : __fns(lasts, 0, chain - left0 + 1);
        const int unit = left_open ? sh.ends[0].first_unit : sh.ends[w0].last_unit;
        int n = 1;
        while (w0 + n < kFullWarps && sh.ends[w0 + n].first_unit == unit) ++n;
        const bool right_open = sh.ends[w0 + n - 1].last_unit == unit;
        const int rows = min(4, c.G - r0);
        float m[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY}, l[4] = {0.f, 0.f, 0.f, 0.f};
        float4 a[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) a[u] = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int k = 0; k < n; ++k) {
            const float2* ml = sh.ml[w0 + k][k == 0 && !left_open ? 1 : 0] + r0;
#pragma unroll
            for (int u = 0; u < 4; ++u)
                if (u < rows) m[u] = fmaxf(m[u], ml[u].x);
        }
#pragma unroll 2
        for (int k = 0; k < n; ++k) {
            const bool last = k == 0 && !left_open;
            const float2* ml = sh.ml[w0 + k][last ? 1 : 0] + r0;
            const float* from = (last ? sh.ends[w0 + k].last : sh.ends[w0 + k].first) + r0 * kD;
            float4 v[4];
#pragma unroll
            for (int u = 0; u < 4; ++u)
                if (u < rows) v[u] = reinterpret_cast<const float4*>(from + u * kD)[lane];
#pragma unroll
            for (int u = 0; u < 4; ++u)
                if (u < rows) {
                    const float2 x = ml[u];
                    const float e = exp2_approx(x.x - (m[u] == -INFINITY ? 0.0f : m[u]));
                    l[u] = fmaf(x.y, e, l[u]);
                    a[u].x = fmaf(v[u].x, e, a[u].x);
                    a[u].y = fmaf(v[u].y, e, a[u].y);
                    a[u].z = fmaf(v[u].z, e, a[u].z);
                    a[u].w = fmaf(v[u].w, e, a[u].w);
                }
        }
        const bool whole = !left_open && !right_open;
        const int64_t slot = whole ? unit_slot(p, unit) : 2ll * blockIdx.x + (left_open ? 0 : 1);
        const int s = unit / c.Hkv, h = unit - s * c.Hkv;
#pragma unroll
        for (int u = 0; u < 4; ++u)
            if (u < rows) {
                const int r = r0 + u;
                if (whole && p.prefix_ctas == 0) {
                    const float rl = l[u] > 0.0f ? 1.0f / l[u] : (l[u] == 0.0f ? 0.0f : l[u]);
                    reinterpret_cast<uint2*>(p.out + (static_cast<int64_t>(s) * c.Hq + h * c.G + r) * kD)[lane] =
                        make_uint2(pack_bf16x2(a[u].x * rl, a[u].y * rl), pack_bf16x2(a[u].z * rl, a[u].w * rl));
                } else {
                    reinterpret_cast<float4*>(p.ws.o + (slot * c.G + r) * kD)[lane] = a[u];
                }
                if (lane == 0) p.ws.ml[slot * c.G + r] = make_float2(m[u], l[u]);
            }
    }
    // one block holds this grid open until the prefix kernel is complete
    if (p.prefix_ctas != 0 && blockIdx.x == gridDim.x - 1) pdl_wait();
}

// The partials that make up one output row: n of the sequence's own tokens,
// then pn of the shared prefix.
struct Parts {
    int n, w0;       // own: count and the first one's CTA
    bool whole;      // a single own part that one CTA holds whole
    int64_t own_slot, g, G;
    int pn, pw0, pgroup, prow;
    bool pwhole;
    int64_t punit_slot;

    // statistics' and output's index of part i
    __device__ __forceinline__ void at(const FullArgs& p, int i, const float2** ml, const float** o) const {
        if (i < n) {
            const int64_t k = (whole ? own_slot : 2ll * (w0 + i) + (i == 0 ? 1 : 0)) * G + g;
            *ml = p.ws.ml + k;
            *o = p.ws.o + k * kD;
        } else {
            const int j = i - n;
            const int64_t slot = 2 * (pwhole ? punit_slot : 2ll * (pw0 + j) + (j == 0 ? 1 : 0)) + pgroup;
            *ml = p.ws.pml + slot * 128 + prow;
            *o = p.ws.po + (slot * 128 + prow) * kD;
        }
    }
    __device__ __forceinline__ int count() const { return n + pn; }
};

// What is known without the split kernel's results: the prefix's parts.
__device__ __forceinline__ Parts prefix_parts(const FullArgs& p, int s, int h, int g) {
    const CacheDesc& c = p.c;
    Parts r;
    r.own_slot = unit_slot(p, s * c.Hkv + h);
    r.g = g;
    r.G = c.G;
    r.n = r.pn = 0;
    r.w0 = 0;
    r.whole = true;
    const int len = c.seq_lens[s];
    if (p.prefix_ctas != 0 && len >= c.shared && len <= c.max_pages * kPage) {
        const PrefixPlan& pl = p.prefix;
        const int row = s * c.G + g, tile = row >> 7, pair = tile >> 1;
        const int chunk = (pl.tiles * pl.units + p.prefix_ctas - 1) / p.prefix_ctas;
        const int unit = pair * c.Hkv + h, f0 = unit * pl.tiles, f1 = f0 + pl.tiles;
        const int w1 = (f1 - 1) / chunk;
        r.pw0 = f0 / chunk;
        r.pgroup = tile & 1;
        r.prow = row & 127;
        r.pwhole = w1 == r.pw0;
        r.punit_slot = 2ll * p.prefix_ctas + unit;
        r.pn = w1 - r.pw0 + 1;
    }
    return r;
}

__device__ __forceinline__ void add_own_parts(const FullArgs& p, int s, int h, Parts* r) {
    const CacheDesc& c = p.c;
    const int a = p.ws.cum[s], n = p.ws.cum[s + 1] - a, total = p.ws.cum[c.S] * c.Hkv;
    if (n > 0) {
        const int chunk = (total + p.workers - 1) / p.workers * kFullWarps;   // a CTA's
        const int f0 = a * c.Hkv + h * n, f1 = f0 + n;
        const int w1 = (f1 - 1) / chunk;
        r->w0 = f0 / chunk;
        r->n = w1 - r->w0 + 1;
        r->whole = r->n == 1;
    }
}

constexpr int kMergeThreads = 256;
constexpr int kWeightTokens = 1024;   // tokens per weights block

// A row's parts by `per` warps (1, 2, 4 or 8) of the block; lane l holds
// channels 4l .. 4l + 3 and, for the statistics, every 32nd part.
//
// Blocks 0 .. row_blocks - 1 join output rows; the others, `chunks` per unit,
// add the weights of kWeightTokens tokens of their unit at a time.
__global__ void __launch_bounds__(kMergeThreads)
    full_merge_kernel(const FullArgs p, const int row_blocks, const int per, const int chunks) {
    __shared__ float4 acc_s[8][32];
    __shared__ float lse_s[ABSP_MAX_GROUP];
    const CacheDesc& c = p.c;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int rows = c.S * c.Hq;
    if (static_cast<int>(blockIdx.x) < row_blocks) {
        const int sub = warp & (per - 1);
        const int row_at = (blockIdx.x * 8 + warp) / per;
        const int row = min(row_at, rows - 1);     // a block past the end works in vain
        const int s = row / c.Hq, j = row - s * c.Hq;
        const int h = j / c.G, g = j - h * c.G;
        // what came before this call is complete: the kernels ahead of this
        // one waited for it before they let this one start
        Parts pt = prefix_parts(p, s, h, g);
        pdl_wait();
        pdl_trigger();
        add_own_parts(p, s, h, &pt);
        const int n = pt.count();
        __nv_bfloat16* to = p.out + static_cast<int64_t>(row) * kD;
        // written by the split kernel, or no row
        const bool skip = row_at >= rows || (pt.n != 0 && pt.whole && p.prefix_ctas == 0);
        if (per == 1 && skip) return;
        const float2* ml_at;
        const float* o_at;
        float M = -INFINITY;
        for (int i = lane; i < n; i += 32) {
            pt.at(p, i, &ml_at, &o_at);
            M = fmaxf(M, ml_at->x);
        }
        for (int d = 16; d > 0; d >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, d));
        const float ms = M == -INFINITY ? 0.0f : M;
        float L = 0.0f;
        float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int i0 = 0; i0 < n; i0 += 32) {
            float e = 0.0f;
            const float* mine = nullptr;
            if (i0 + lane < n) {
                pt.at(p, i0 + lane, &ml_at, &mine);
                const float2 ml = *ml_at;
                e = ml.y == 0.0f ? 0.0f : exp2_approx(ml.x - ms);
                L = fmaf(ml.y, e, L);
            }
            // eight parts' loads in flight.  Every part counts, one whose factor
            // is 0 as well: a non-finite value in it reaches the output here
            // as it does inside a part
            const int m = min(32, n - i0);
            for (int k0 = sub; k0 < m; k0 += 8 * per) {
                float ek[8];
                float4 v[8];
#pragma unroll
                for (int u = 0; u < 8; ++u) {
                    const int k = k0 + u * per;
                    ek[u] = __shfl_sync(0xffffffffu, e, k & 31);
                    const float* from = reinterpret_cast<const float*>(
                        __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(mine), k & 31));
                    if (k >= m) ek[u] = -1.0f;   // no part
                    v[u] = !(ek[u] < 0.0f) ? reinterpret_cast<const float4*>(from)[lane]
                                           : make_float4(0.f, 0.f, 0.f, 0.f);
                }
#pragma unroll
                for (int u = 0; u < 8; ++u) {
                    a.x = fmaf(v[u].x, ek[u], a.x);
                    a.y = fmaf(v[u].y, ek[u], a.y);
                    a.z = fmaf(v[u].z, ek[u], a.z);
                    a.w = fmaf(v[u].w, ek[u], a.w);
                }
            }
        }
        for (int d = 16; d > 0; d >>= 1) L += __shfl_xor_sync(0xffffffffu, L, d);
        if (per > 1) {
            acc_s[warp][lane] = a;
            __syncthreads();
            if (sub != 0 || skip) return;
            a = make_float4(0.f, 0.f, 0.f, 0.f);
            for (int w = 0; w < per; ++w) {
                const float4 v = acc_s[warp + w][lane];
                a.x += v.x;
                a.y += v.y;
                a.z += v.z;
                a.w += v.w;
            }
        }
        const float rl = L > 0.0f ? 1.0f / L : (L == 0.0f ? 0.0f : L);
        reinterpret_cast<uint2*>(to)[lane] =
            make_uint2(pack_bf16x2(a.x * rl, a.y * rl), pack_bf16x2(a.z * rl, a.w * rl));
        return;
    }
    // ---- weights
    pdl_wait();
    pdl_trigger();
    const int cap = c.max_pages * kPage;
    const int wb = blockIdx.x - row_blocks;
    const int unit = wb / chunks;
    const int s = unit / c.Hkv, h = unit - s * c.Hkv;
    int len = c.seq_lens[s];
    if (len < 0 || len > cap) len = 0;
    const int start = own_start(c, len);
    const int t0 = start + (wb - unit * chunks) * kWeightTokens;
    if (t0 >= len) return;
    for (int g = warp; g < c.G; g += 8) {
        Parts pt = prefix_parts(p, s, h, g);
        add_own_parts(p, s, h, &pt);
        const int n = pt.count();
        float M = -INFINITY, L = 0.0f;
        for (int i = lane; i < n; i += 32) {
            const float2* ml_at;
            const float* o_at;
            pt.at(p, i, &ml_at, &o_at);
            const float2 ml = *ml_at;
            const float mn = fmaxf(M, ml.x);
            const float ms = mn == -INFINITY ? 0.0f : mn;
            L = L * exp2_approx(M - ms) + ml.y * exp2_approx(ml.x - ms);
            M = mn;
        }
        float T = M;
        for (int d = 16; d > 0; d >>= 1) T = fmaxf(T, __shfl_xor_sync(0xffffffffu, T, d));
        L *= exp2_approx(M - (T == -INFINITY ? 0.0f : T));
        for (int d = 16; d > 0; d >>= 1) L += __shfl_xor_sync(0xffffffffu, L, d);
        // no weight to give where nothing was attended to
        if (lane == 0) lse_s[g] = L == 0.0f ? INFINITY : T + log2f(L);
    }
    __syncthreads();
    // the unit's blocks take turns; a row of weights ends on a whole page, so
    // the four tokens of a thread are inside it
    for (int t = t0 + 4 * tid; t < len; t += chunks * kWeightTokens) {
        add_weights(p, (static_cast<int64_t>(s) * c.Hq + h * c.G) * cap + t,
                    static_cast<int64_t>(unit) * cap + t, min(4, len - t), cap, lse_s);
    }
}

template <bool BIG, bool WEIGHTS, bool UNIT>
cudaError_t launch_split(const FullArgs& a, int cluster, const CUtensorMap& tmk, const CUtensorMap& tmv,
                         bool pdl, cudaStream_t st) {
    static std::atomic<uint64_t> done{0};
    auto kern = full_split_kernel<BIG, WEIGHTS, UNIT>;
    cudaError_t e = prepare_kernel(kern, kSplitSmem, UNIT, &done);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(UNIT ? a.c.S * a.c.Hkv * cluster : a.workers / kFullWarps);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kSplitSmem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    int n = 0;
    if (UNIT) {
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
    return cudaLaunchKernelEx(&cfg, kern, a, tmk, tmv);
}

template <bool UNIT>
cudaError_t launch_split_as(const FullArgs& a, int cluster, const CUtensorMap& tmk, const CUtensorMap& tmv,
                            bool pdl, cudaStream_t st) {
    const bool big = a.c.G > 8, weights = a.weights_out != nullptr;
    return big ? (weights ? launch_split<true, true, UNIT>(a, cluster, tmk, tmv, pdl, st)
                          : launch_split<true, false, UNIT>(a, cluster, tmk, tmv, pdl, st))
               : (weights ? launch_split<false, true, UNIT>(a, cluster, tmk, tmv, pdl, st)
                          : launch_split<false, false, UNIT>(a, cluster, tmk, tmv, pdl, st));
}

}  // namespace

// CTAs per unit where a cluster takes a unit, 0 for the split and merge
// kernels.  One launch instead of two, no scan of the lengths and no partials
// in memory: 8.0 us against 10.7 a call at one sequence of 1024 or 2048
// tokens and 32 query over 8 KV heads, 8.0 against 11.8 at 8 of 512, 8.8
// against 11.8 at 4096, 12.6 against 14.0 at 8192 (8 pages per warp).  Beyond
// that the split kernel's use of every SM counts for more (32K tokens: 31.8
// against 44.5 with clusters of 16, not all of which fit at once), and with
// several sequences the fixed cut can leave one cluster the long one, so the
// tables then hold half as much per warp.  Clusters of at most 8 CTAs, which
// every device places.
int unit_cluster(int S, int Hkv, int max_pages) {
    const int64_t units = static_cast<int64_t>(S) * Hkv;
    if (units > device_sms()) return 0;
    int C = 1;
    while (C < 8 && units * C * 2 <= device_sms() && C * kFullWarps < max_pages) C *= 2;
    return max_pages <= (S == 1 ? 8 : 4) * C * kFullWarps ? C : 0;
}

int device_sms() {
    static std::atomic<int> sms_of[64];
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) {
        cudaGetLastError();
        return kMaxSms;
    }
    if (dev < 64) n = sms_of[dev].load(std::memory_order_relaxed);
    if (n <= 0) {
        if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0) {
            cudaGetLastError();
            return kMaxSms;
        }
        n = n < kMaxSms ? n : kMaxSms;
        if (dev < 64) sms_of[dev].store(n, std::memory_order_relaxed);
    }
    return n;
}

cudaError_t launch_full(const FullArgs& a, const CUtensorMap& tmk, const CUtensorMap& tmv,
                        const CUtensorMap& tmk_half, bool pdl, cudaStream_t st) {
    const bool weights = a.weights_out != nullptr;
    cudaError_t e = a.prefix_ctas != 0 ? launch_prefix(a, tmk_half, tmv, pdl, st) : cudaSuccess;
    if (e != cudaSuccess) return e;
    const int cluster = a.prefix_ctas == 0 ? unit_cluster(a.c.S, a.c.Hkv, a.c.max_pages) : 0;
    if (cluster > 0) return launch_split_as<true>(a, cluster, tmk, tmv, pdl, st);
    e = launch_split_as<false>(a, 0, tmk, tmv, pdl, st);
    if (e != cudaSuccess) return e;
    static std::atomic<uint64_t> done{0};
    e = prepare_kernel(full_merge_kernel, 0, false, &done);
    if (e != cudaSuccess) return e;
    // warps per row: as many as the SMs hold at once, 24 each; a batch of
    // eight parts takes a warp 1.3 us, however few rows there are
    const int64_t rows = static_cast<int64_t>(a.c.S) * a.c.Hq;
    int per = 8;
    while (per > 1 && rows * per > 24 * device_sms()) per /= 2;
    const int64_t row_blocks = (rows * per + 7) / 8;
    int64_t blocks = row_blocks;
    // weights: a unit's own tokens in turns of its blocks, about 16 blocks per
    // SM in all (a block for every 1024 tokens of the tables' capacity left
    // thousands that found nothing to do: 8 us over a 32K prefix)
    int chunks = 0;
    if (weights) {
        const int units = a.c.S * a.c.Hkv;
        chunks = std::max(1, (a.c.max_pages * kPage - a.c.shared + kWeightTokens - 1) / kWeightTokens);
        chunks = std::min(chunks, std::max(1, 16 * device_sms() / units));
        blocks += static_cast<int64_t>(units) * chunks;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(blocks));
    cfg.blockDim = dim3(kMergeThreads);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pdl ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, full_merge_kernel, a, static_cast<int>(row_blocks), per, chunks);
}

}  // namespace absp
