// Attention of a whole batch over the prefix that its sequences share.
//
// The S * G query rows of a KV head meet the same keys, so the prefix is a
// pair of dense products per head, S = Q K^T and O = P V with M = S * G
// rows, and its keys and values are read once for the batch instead of once
// per sequence.  Both products run on tcgen05: 128 query rows x 128 tokens,
// Q and K tiles in shared memory (128-byte swizzle, K-major), S in tensor
// memory, P written over S as bf16 and read from there as the A operand, V
// as the MN-major B operand straight from its page slices, O accumulated in
// tensor memory.
//
// One CTA per SM: a copy warp, an instruction warp and two softmax
// warpgroups, each with its own S/P and O columns, so one group's
// exponentials run while the tensor core works for the other.  A unit is
// (pair of 128-row tiles, KV head): with two row tiles both groups take every
// token tile (keys and values are used twice per copy); with one the groups
// take alternate token tiles.  The token tiles of all units laid end to end
// are cut into equal contiguous runs, one per CTA, whose partial outputs the
// merge kernel joins with those of the sequences' own tokens.
//
// The running maximum moves only when it grows by more than 8 (log2 units):
// P stays below 2^8, where a bf16 number and the fp32 sums are as exact as
// below 1, and the rescaling of O in tensor memory becomes rare.  P enters
// the product with V as one bf16 number: a second one for its rounding would
// be half as much tensor work again.
//
// What bounds it: with up to 128 rows (one row tile) the copies of K and V,
// 64 KiB per token tile: 32 sequences x 4 heads over 32K tokens and 8 KV
// heads (134 MB) take 33 us, of which 21 are the bytes' floor and the rest
// set-up, first copies and the partials' way out.  With two row tiles the
// chain of a group bounds it: 1750 clocks of exponentials (the hardware's
// floor is 1024), P V and Q K^T of that group, hand-overs: 3300 clocks per
// token tile; the tensor pipe is 37 % busy over the whole kernel at 512 rows
// over 16K tokens (41 us).  Q K^T takes 100 clocks per instruction instead of
// 64, both operands coming from shared memory.  Jobs of 64 tokens with two S
// buffers per group, which break that chain, made the products (as slow at N
// = 64 as at 128) the bound: 75.9 us a call against 69.0.
#include <atomic>

#include "cache_ops.cuh"

namespace absp {

namespace {

constexpr int kTile = 128;                    // tokens of a tile
constexpr int kPagesPerTile = kTile / kPage;
constexpr int kM = 128;                       // query rows of a tile
constexpr int kTileBytes = 128 * kD * 2;      // 32 KiB: Q, K or V tile
constexpr int kHalf = kTileBytes / 2;         // 64 channels of a K-major tile
constexpr int kBufs = 5;                      // ring of K and V tiles, in the order of their use
constexpr int kMasks = 8;                     // page masks of the tiles in flight
constexpr int kSliceBytes = kPage * kD * 2;
constexpr int kThreads = 384;                 // copy, instruction, 2 idle warps, 2 x 4 softmax warps
// registers per thread: 168 at launch; the first warpgroup gives 96 of them
// up and the softmax groups take 48 each (72 + 2 x 216 = 3 x 168)
constexpr int kRegsCopy = 72, kRegsSoftmax = 216;
constexpr float kLazy = 8.0f;                 // growth of the maximum left unscaled, log2 units

// tensor memory columns
constexpr uint32_t kColS = 0, kColO = 256, kTmemCols = 512;

struct PrefixShared {
    uint64_t full[kBufs], empty[kBufs];
    uint64_t q_full[2], s_full[2], p_full[2][2], o_done[2];   // P: tokens 0..63, 64..127
    uint32_t okmask[kMasks];  // pages of a token tile that hold valid ids
    uint32_t tmem;
    int32_t abort;            // a bounded wait gave up
    float2 stats[2][kM];      // maximum and sum of each group's rows
};

// query tiles, ring and the small state: the whole 227 KiB of an SM
constexpr int kPrefixSmem = (2 + kBufs) * kTileBytes + sizeof(PrefixShared);
static_assert(kPrefixSmem <= 227 * 1024, "shared memory of one SM");

// ------------------------------------------------------------- tcgen05 --

__device__ __forceinline__ void tc_fence_before() {
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tc_fence_after() {
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tc_commit(uint32_t bar) {
    asm volatile(
        "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar)
        : "memory");
}

// True in one lane of a convergent warp.
__device__ __forceinline__ bool elect_one() {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\tselp.u32 %0, 1, 0, e;\n\t}"
        : "=r"(r)::"memory");
    return r != 0;
}

// Shared-memory matrix descriptor, 128-byte swizzle (layout 2, version 1):
// lead: byte stride between 64-element blocks of an MN-major operand (unused
// K-major); stride: between 8-row groups.
__device__ __forceinline__ uint64_t smem_desc(uint32_t addr, uint32_t lead, uint32_t stride) {
    return static_cast<uint64_t>((addr & 0x3FFFF) >> 4) |
           static_cast<uint64_t>(lead >> 4) << 16 | static_cast<uint64_t>(stride >> 4) << 32 |
           1ull << 46 | 2ull << 61;
}

// kind::f16 instruction descriptor: fp32 accumulator, bf16 A and B, M = 128.
__device__ __forceinline__ uint32_t instr_desc(uint32_t n, bool b_mn_major) {
    return 1u << 4 | 1u << 7 | 1u << 10 | (b_mn_major ? 1u << 16 : 0u) | (n >> 3) << 17 |
           (kM >> 4) << 24;
}

__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(acc)
        : "memory");
}

__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(acc)
        : "memory");
}

// 32 columns of this warp's 32 lanes.
__device__ __forceinline__ void tmem_ld32(uint32_t addr, uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]),
          "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]),
          "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]),
          "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(addr)
        : "memory");
}
__device__ __forceinline__ void tmem_ld16(uint32_t addr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]),
          "=r"(r[15])
        : "r"(addr)
        : "memory");
}
__device__ __forceinline__ void tmem_wait_ld() {
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t addr, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
        "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(addr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
        "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}
__device__ __forceinline__ void tmem_st32(uint32_t addr, const uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
        "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
        "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(addr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
        "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]),
        "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]),
        "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
        : "memory");
}
__device__ __forceinline__ void tmem_wait_st() {
    asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}

// Wait for a phase; false once any wait of the CTA gave up (the error word
// is set), so that every role leaves its loop.
__device__ __forceinline__ bool wait_or_abort(uint32_t bar, uint32_t parity, volatile int32_t* abort,
                                              int32_t* err, int where) {
    if (mbar_try_wait(bar, parity)) return true;
    const uint64_t t0 = globaltimer_ns();
    while (!mbar_try_wait(bar, parity)) {
        if (*abort) return false;
        if (globaltimer_ns() - t0 > kWaitLimitNs) {
            set_error(err, ABSP_ERR_TIMEOUT, where);
            *abort = 1;
            return false;
        }
    }
    return true;
}

// A run of token tiles of one unit.
struct Segment {
    int unit, t0, n;      // tiles t0 .. t0 + n - 1
    int h, tile0;         // KV head, first row tile
    bool two;             // two row tiles
    bool cut_left, whole;
    int jobs;             // products of the segment: (token tile, group)
};

__device__ __forceinline__ Segment segment_at(const PrefixPlan& pl, int Hkv, int f, int f1) {
    Segment g;
    g.unit = f / pl.tiles;
    g.t0 = f - g.unit * pl.tiles;
    g.n = min(pl.tiles - g.t0, f1 - f);
    const int pair = g.unit / Hkv;      // pairs outermost: CTAs that read the
    g.h = g.unit - pair * Hkv;          // same tiles at a time share them in L2
    g.tile0 = 2 * pair;
    g.two = g.tile0 + 1 < pl.row_tiles;
    g.cut_left = g.t0 != 0;
    g.whole = g.t0 == 0 && g.n == pl.tiles;
    g.jobs = g.two ? 2 * g.n : g.n;
    return g;
}

__global__ void __launch_bounds__(kThreads, 1)
    prefix_kernel(const FullArgs p, const __grid_constant__ CUtensorMap tmk_half,
                  const __grid_constant__ CUtensorMap tmv) {
    extern __shared__ __align__(1024) uint8_t base[];
    PrefixShared& sh = *reinterpret_cast<PrefixShared*>(base + (2 + kBufs) * kTileBytes);
    const uint32_t q_s = smem_u32(base), ring = q_s + 2 * kTileBytes;
    const CacheDesc& c = p.c;
    const PrefixPlan& pl = p.prefix;
    const int tid = threadIdx.x, lane = tid & 31;
    const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);   // known to be uniform
    if (tid == 0) {
        for (int i = 0; i < kBufs; ++i) {
            mbar_init(smem_u32(&sh.full[i]), 1);
            mbar_init(smem_u32(&sh.empty[i]), 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_u32(&sh.q_full[i]), 4);
            mbar_init(smem_u32(&sh.s_full[i]), 1);
            mbar_init(smem_u32(&sh.p_full[i][0]), 4);
            mbar_init(smem_u32(&sh.p_full[i][1]), 4);
            mbar_init(smem_u32(&sh.o_done[i]), 1);
        }
        fence_mbar_init();
        sh.abort = 0;
        prefetch_tensormap(&tmk_half);
        prefetch_tensormap(&tmv);
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                         smem_u32(&sh.tmem)),
                     "r"(kTmemCols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    const int total = pl.tiles * pl.units;
    const int chunk = (total + p.prefix_ctas - 1) / p.prefix_ctas;
    const int f0 = min(static_cast<int>(blockIdx.x) * chunk, total), f_end = min(f0 + chunk, total);
    const int pages = c.shared / kPage;
    const int rows = c.S * c.G;
    // A softmax warp's 32 query rows of a segment's tile, as 128-byte-swizzled
    // K-major halves; half a warp copies a row, rows behind the last are zero.
    const int sw = (warp - 4) >> 2, quad = warp & 3;
    struct QRow {
        int s, j;                        // of the lane's first row
        const __nv_bfloat16* from;
    };
    auto q_row = [&](const Segment& g) {
        const int r0 = (g.tile0 + (g.two ? sw : 0)) * kM + quad * 32 + (lane >> 4);
        QRow q;
        q.s = r0 / c.G;
        q.j = r0 - q.s * c.G;
        q.from = p.q + static_cast<int64_t>(g.h) * c.G * kD + (lane & 15) * 8;
        return q;
    };
    auto load_q = [&](QRow q) {
        const int hi = lane >> 4, ch = lane & 15;
        const uint32_t to_q = q_s + sw * kTileBytes + (ch >> 3) * kHalf + (quad * 32 + hi) * 128;
#pragma unroll 1
        for (int k = 0; k < 16; ++k) {
            const int live = q.s < c.S ? 1 : 0;
            cp_async_16_zfill(to_q + k * 256 + (((ch & 7) ^ ((2 * k + hi) & 7)) << 4),
                              q.from + (live ? static_cast<int64_t>(q.s) * c.Hq + q.j : 0) * kD, live ? 16 : 0);
            q.j += 2;                    // two rows on: at most two sequences
            if (q.j >= c.G) {
                q.j -= c.G;
                ++q.s;
            }
            if (q.j >= c.G) {
                q.j -= c.G;
                ++q.s;
            }
        }
        cp_async_commit();
    };
    const bool any = f0 < f_end;
    const Segment g0 = any ? segment_at(pl, c.Hkv, f0, f_end) : Segment{};
    const bool early_q = warp >= 4 && any && sw < g0.jobs;
    const QRow q0 = early_q ? q_row(g0) : QRow{};
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = __shfl_sync(0xffffffffu, sh.tmem, 0);
    // nothing of this call's data is read before this point
    pdl_wait();
    pdl_trigger();
    // the first tiles' page ids, guessed to be in the first sequence's row
    int ids_first = -1;
    if (warp == 0 && any && g0.t0 * kPagesPerTile + lane < pages)
        ids_first = c.page_table[g0.t0 * kPagesPerTile + lane];
    if (early_q) load_q(q0);
    // the prefix's pages are listed by the first sequence that holds all of it
    int first = c.S;
    for (int s0 = 0; s0 < c.S && first == c.S; s0 += 32) {
        const int len = s0 + lane < c.S ? c.seq_lens[s0 + lane] : -1;
        const uint32_t m = __ballot_sync(0xffffffffu, len >= c.shared && len <= c.max_pages * kPage);
        if (m != 0) first = s0 + __ffs(m) - 1;
    }
    const int f1 = first < c.S ? f_end : f0;
    volatile int32_t* abort = &sh.abort;

    // Order of the tiles in the ring: that of their first use, which is also
    // that of their release.  One row tile (groups alternate): K0 K1 V0 K2 V1
    // K3 V2 ..; two: K0 V0 K1 V1 ..
    if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsCopy));
    if (warp == 0) {
        // ---------------------------------------------------------- copies
        const int32_t* row = c.page_table + static_cast<int64_t>(first) * c.max_pages;
        const int oob = static_cast<int>(c.num_phys_pages * c.Hkv * kPage);  // reads zeros
        int it = 0;                      // tiles of earlier segments
        int buf = 0, par = 1;
        for (int f = f0; f < f1;) {
            const Segment g = segment_at(pl, c.Hkv, f, f1);
            int ids[2] = {-1, -1};       // page ids of four tiles at a time, K's and V's copy
            bool ok = true;
            auto put = [&](int i, int v) {
                const int pg0 = (g.t0 + i) * kPagesPerTile;
                if ((i & 3) == 0) {
                    if (v == 0) {
                        ids[0] = pg0 + lane < pages ? (it + i == 0 && first == 0 ? ids_first : row[pg0 + lane]) : -1;
                        if (pg0 + lane < pages && (ids[0] < 0 || ids[0] >= c.num_phys_pages)) {
                            set_error(p.ws.err, ABSP_ERR_DEVICE_FAULT, first);
                            ids[0] = -1;
                        }
                    } else {
                        ids[1] = ids[0];
                    }
                }
                const int np = min(kPagesPerTile, pages - pg0);
                const uint32_t good = __ballot_sync(0xffffffffu, ids[v] >= 0) >> ((i & 3) * 8) & 0xffu;
                const int id = __shfl_sync(0xffffffffu, ids[v], (i & 3) * 8 + (lane & 7));
                const int y = id >= 0 ? (id * c.Hkv + g.h) * kPage : oob;
                const uint32_t bar = smem_u32(&sh.full[buf]);
                ok = wait_or_abort(smem_u32(&sh.empty[buf]), par, abort, p.ws.err, 20);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) return;
                if (lane == 0) {
                    if (v == 0) sh.okmask[(it + i) % kMasks] = good;
                    mbar_arrive_expect_tx(bar, np * kSliceBytes);
                }
                __syncwarp();
                const uint32_t dst = ring + buf * kTileBytes;
                if (lane < np) {         // lane l copies page l
                    if (v == 0) {
                        tma_load_3d(dst + lane * (kPage * 128), &tmk_half, 0, y, 0, bar);
                        tma_load_3d(dst + kHalf + lane * (kPage * 128), &tmk_half, 0, y, 1, bar);
                    } else {
                        tma_load_3d(dst + lane * kSliceBytes, &tmv, 0, y, 0, bar);
                    }
                }
                if (++buf == kBufs) {
                    buf = 0;
                    par ^= 1;
                }
            };
            const int lead = g.two ? 0 : 1;   // K tiles ahead of V
            put(0, 0);
            if (lead && g.n > 1 && ok) put(1, 0);
            for (int i = 0; i < g.n && ok; ++i) {
                // V takes the ids of its own four tiles before K moves on
                put(i, 1);
                if (i + 1 + lead < g.n && ok) put(i + 1 + lead, 0);
            }
            if (!ok) break;
            it += g.n;
            f += g.n;
        }
    } else if (warp == 1) {
        // ----------------------------------------------------- instructions
        uint32_t qph0 = 0, qph1 = 0, pph0 = 0, pph1 = 0;
        uint32_t buf = 0, par = 0;             // next tile of the ring
        // descriptors of the tiles' first 16 columns (or tokens); the others
        // differ in the start address, counted in 16 bytes
        const uint64_t dq = smem_desc(q_s, 16, 1024), dk = smem_desc(ring, 16, 1024),
                       dv = smem_desc(ring, 2048, 1024);
        bool ok = true;
        auto wait = [&](uint64_t& bar, uint32_t parity, int where) {
            ok = ok && wait_or_abort(smem_u32(&bar), parity, abort, p.ws.err, where);
            ok = __all_sync(0xffffffffu, ok);
        };
        for (int f = f0; f < f1 && ok;) {
            const Segment g = segment_at(pl, c.Hkv, f, f1);
            uint32_t kbuf = 0, vbuf = 0;       // a tile's buffer: taken at its first use
            auto take = [&](uint32_t& b, int where) {
                b = buf;
                wait(sh.full[buf], par, where);
                if (++buf == kBufs) {
                    buf = 0;
                    par ^= 1;
                }
            };
            // products of job j: group j & 1 and, with two row tiles, token
            // tile j / 2, else j
#pragma unroll 1
            for (int j = -2; j < g.jobs && ok; ++j) {
                const uint32_t w = j & 1;
                const uint32_t ts = tmem + kColS + w * 128;
                if (j >= 0) {                  // O += P V
                    const int i = g.two ? j >> 1 : j;
                    if (!g.two || w == 0) take(vbuf, 25);
                    const uint32_t ph = w ? pph1 : pph0;
                    if (w) pph1 ^= 1; else pph0 ^= 1;
                    const uint32_t idesc = instr_desc(kD, true);
                    const uint64_t db = dv + vbuf * (kTileBytes >> 4);
                    const int np = min(kPagesPerTile, pages - (g.t0 + i) * kPagesPerTile);
                    const uint32_t acc = j >= 2;
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        wait(sh.p_full[w][half], ph, 24);
                        if (!ok) break;
                        tc_fence_after();
                        if (elect_one()) {
#pragma unroll
                            for (int k = 4 * half; k < 4 * half + 4; ++k)   // 16 tokens: one page slice
                                if (k < np)
                                    mma_ts(tmem + kColO + w * 128, ts + 8 * k, db + k * (kSliceBytes >> 4),
                                           idesc, k == 0 ? acc : 1u);
                            if (half == 1) {
                                if (!g.two || w == 1) tc_commit(smem_u32(&sh.empty[vbuf]));
                                if (j + 2 >= g.jobs) tc_commit(smem_u32(&sh.o_done[w]));
                            }
                        }
                        __syncwarp();
                    }
                    if (!ok) break;
                }
                const int jn = j + 2;
                if (jn < g.jobs) {             // S = Q K^T of the group's next job
                    const int i = g.two ? jn >> 1 : jn;
                    if (j < 0) {
                        if (w == 0) {
                            wait(sh.q_full[0], qph0, 22);
                            qph0 ^= 1;
                        } else {
                            wait(sh.q_full[1], qph1, 22);
                            qph1 ^= 1;
                        }
                    }
                    if (!g.two || w == 0) take(kbuf, 23);
                    if (!ok) break;
                    tc_fence_after();
                    const int np = min(kPagesPerTile, pages - (g.t0 + i) * kPagesPerTile);
                    const uint32_t idesc = instr_desc(np * kPage, false);
                    const uint64_t da = dq + w * (kTileBytes >> 4), db = dk + kbuf * (kTileBytes >> 4);
                    if (elect_one()) {
#pragma unroll
                        for (int k = 0; k < 8; ++k) {
                            const uint32_t off = ((k >> 2) * kHalf + (k & 3) * 32) >> 4;
                            mma_ss(ts, da + off, db + off, idesc, k != 0);
                        }
                        tc_commit(smem_u32(&sh.s_full[w]));
                        if (!g.two || w == 1) tc_commit(smem_u32(&sh.empty[kbuf]));
                    }
                    __syncwarp();
                }
            }
            f += g.n;
        }
        __syncwarp();
    }
    } else {
        // ---------------------------------------------------------- softmax
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoftmax));
        const int w = sw;
        const int r = quad * 32 + lane;                       // row of the tile
        const uint32_t lanes = static_cast<uint32_t>(quad * 32) << 16;
        const uint32_t ts = tmem + kColS + w * 128 + lanes, to = tmem + kColO + w * 128 + lanes;
        const float scale = kLog2E / sqrtf(static_cast<float>(kD));
        uint32_t sph = 0, oph = 0;
        bool ok = true;
        // once a wait gave up, the remaining segments only meet the barriers
        for (int f = f0; f < f1;) {
            const Segment g = segment_at(pl, c.Hkv, f, f1);
            const int it0 = f - f0;
            f += g.n;
            const int mt = g.tile0 + (g.two ? w : 0);
            const bool warp_live = mt * kM + quad * 32 < rows;
            const bool busy = w < g.jobs;    // a single token tile goes to group 0
            if (busy) {
                if (it0 != 0) load_q(q_row(g));   // the first segment's are under way
                cp_async_wait_all();
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&sh.q_full[w]));
            }
            float m = -INFINITY, l = 0.0f;
            const int step = g.two ? 1 : 2;
            bool started = false;
            for (int i = g.two ? 0 : w; i < g.n && ok; i += step) {
                ok = wait_or_abort(smem_u32(&sh.s_full[w]), sph & 1, abort, p.ws.err, 26);
                ++sph;
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                tc_fence_after();
                if (warp_live) {
                    // pages behind the prefix's end or with a bad id are left
                    // out.  An entry is written again kMasks tiles later,
                    // after this tile's V was released
                    const uint32_t good = *(volatile uint32_t*)&sh.okmask[(it0 + i) % kMasks];
                    uint32_t v[4][32];
#pragma unroll
                    for (int cc = 0; cc < 4; ++cc) tmem_ld32(ts + cc * 32, v[cc]);
                    tmem_wait_ld();
                    if (good != 0xffu) {
#pragma unroll
                        for (int e = 0; e < 128; ++e)
                            if (!(good >> (e >> 4) & 1)) v[e >> 5][e & 31] = 0xff800000u;  // -inf
                    }
                    float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                    for (int e = 0; e < 32; e += 2)
#pragma unroll
                        for (int cc = 0; cc < 4; ++cc)
                            mx[cc] = fmaxf(fmaxf(mx[cc], __uint_as_float(v[cc][e])),
                                           __uint_as_float(v[cc][e + 1]));
                    const float mn = fmaxf(m, fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * scale);
                    const bool move = mn > m + kLazy;       // also the first finite maximum
                    float corr = 1.0f;
                    if (move) {
                        corr = exp2_approx(m - mn);
                        m = mn;
                        l *= corr;
                    }
                    if (started && __any_sync(0xffffffffu, move)) {
                        // the product before this one is complete: its
                        // successor in the same columns gave this S
#pragma unroll 1
                        for (int cc = 0; cc < 8; ++cc) {
                            uint32_t o[16];
                            tmem_ld16(to + cc * 16, o);
                            tmem_wait_ld();
#pragma unroll
                            for (int e = 0; e < 16; ++e)
                                o[e] = __float_as_uint(__uint_as_float(o[e]) * corr);
                            tmem_st16(to + cc * 16, o);
                        }
                    }
                    const float ms = m == -INFINITY ? 0.0f : m;
                    float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        uint32_t pk[32];
#pragma unroll
                        for (int e = 0; e < 64; e += 2) {
                            const uint32_t* x = &v[2 * half + (e >> 5)][e & 31];
                            const float a = exp2_approx(fmaf(__uint_as_float(x[0]), scale, -ms));
                            const float b = exp2_approx(fmaf(__uint_as_float(x[1]), scale, -ms));
                            sum[(e >> 1) & 3] += a + b;
                            pk[e / 2] = pack_bf16x2(a, b);
                        }
                        tmem_st32(ts + half * 32, pk);
                        tmem_wait_st();
                        // the first half's product runs during the second's exponentials
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(smem_u32(&sh.p_full[w][half]));
                    }
                    l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
                } else {
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) {
                        mbar_arrive(smem_u32(&sh.p_full[w][0]));
                        mbar_arrive(smem_u32(&sh.p_full[w][1]));
                    }
                }
                started = true;
            }
            // ---- the segment's partial output, through the group's query
            // tile in shared memory (32 KiB: 64 channels of every row) so
            // that rows leave in whole 256-byte pieces
            if (busy && ok) {
                ok = wait_or_abort(smem_u32(&sh.o_done[w]), oph & 1, abort, p.ws.err, 27);
                ++oph;
                ok = __all_sync(0xffffffffu, ok);
            }
            tc_fence_after();
            const int64_t slot =
                2ll * (g.whole ? 2 * p.prefix_ctas + g.unit
                               : 2 * static_cast<int>(blockIdx.x) + (g.cut_left ? 0 : 1)) +
                (g.two ? w : 0);
            float* po = p.ws.po + slot * (kM * kD);
            auto chunk_at = [&](uint8_t* t, int rr, int ch) {
                return reinterpret_cast<float4*>(t + rr * 256 + ((ch ^ (rr & 15)) << 4));
            };
            auto leave = [&](uint8_t* t, int half) {   // this warp's 32 rows
                float* to_o = po + (quad * 32 + (lane >> 4)) * kD + half * 64 + (lane & 15) * 4;
                const int n = min(32, rows - mt * kM - quad * 32) - (lane >> 4);
#pragma unroll 8
                for (int k = 0; k < 16; ++k)
                    if (2 * k < n)
                        *reinterpret_cast<float4*>(to_o + 2 * k * kD) =
                            *chunk_at(t, quad * 32 + 2 * k + (lane >> 4), lane & 15);
            };
            // 64 channels of this thread's row: scaled, plus what `t` holds
            // of it when `add`, into `t`
            auto stage = [&](uint8_t* t, int half, float e, bool add) {
                uint32_t v[2][32];
                tmem_ld32(to + half * 64, v[0]);
                tmem_ld32(to + half * 64 + 32, v[1]);
                tmem_wait_ld();
#pragma unroll
                for (int k = 0; k < 16; ++k) {
                    const uint32_t* x = &v[k >> 3][4 * (k & 7)];
                    float4* at = chunk_at(t, r, k);
                    float4 y = add ? *at : make_float4(0.f, 0.f, 0.f, 0.f);
                    y.x = fmaf(__uint_as_float(x[0]), e, y.x);
                    y.y = fmaf(__uint_as_float(x[1]), e, y.y);
                    y.z = fmaf(__uint_as_float(x[2]), e, y.z);
                    y.w = fmaf(__uint_as_float(x[3]), e, y.w);
                    *at = y;
                }
            };
            uint8_t* mine = base + w * kTileBytes;
            if (g.two) {
                if (warp_live) {
#pragma unroll 1
                    for (int half = 0; half < 2; ++half) {
                        stage(mine, half, 1.0f, false);
                        __syncwarp();
                        leave(mine, half);
                        __syncwarp();
                    }
                    if (mt * kM + r < rows) p.ws.pml[slot * kM + r] = make_float2(m, l);
                }
                // the next segment's query rows land where other warps of the
                // group have staged theirs (256 bytes a row here, two halves of
                // 128 there): every warp, live or not, waits for the group's
                // four.  Once per change of unit inside a run.
                if (f < f1) asm volatile("bar.sync %0, 128;" ::"r"(1 + w) : "memory");
            } else {
                // the two groups' parts of the same rows joined: each hands
                // the other 64 channels and finishes the other 64.  A group
                // without a tile has nothing to add.
                sh.stats[w][r] = make_float2(m, l);
                asm volatile("bar.sync 3, 256;" ::: "memory");
                const float2 x = sh.stats[1 - w][r];
                const float M = fmaxf(m, x.x);
                const float e_own = m == -INFINITY ? 0.0f : exp2_approx(m - M);
                const float e_other = x.x == -INFINITY ? 0.0f : exp2_approx(x.x - M);
                const bool both = g.jobs > 1;
                uint8_t* other = base + (1 - w) * kTileBytes;
                if (warp_live && busy && both) stage(mine, 1 - w, e_own, false);
                asm volatile("bar.sync 3, 256;" ::: "memory");
                if (warp_live && busy) {
                    stage(other, w, e_own, both);
                    __syncwarp();
                    leave(other, w);
                    if (!both) {
                        __syncwarp();
                        stage(other, 1, e_own, false);
                        __syncwarp();
                        leave(other, 1);
                    }
                    if (w == 0 && mt * kM + r < rows)
                        p.ws.pml[slot * kM + r] = make_float2(M, l * e_own + x.y * e_other);
                }
                // both query tiles are free again
                asm volatile("bar.sync 3, 256;" ::: "memory");
            }
            tc_fence_before();
        }
    }
    __syncwarp();
    cp_async_wait_all();   // query rows that no segment took
    if (*abort) {
        // copies and products in flight end well within this time
        const uint64_t t0 = globaltimer_ns();
        while (globaltimer_ns() - t0 < 10000000ull) {
        }
    }
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols)
                     : "memory");
    }
}

}  // namespace

cudaError_t launch_prefix(const FullArgs& a, const CUtensorMap& tmk_half, const CUtensorMap& tmv, bool pdl,
                          cudaStream_t st) {
    static std::atomic<uint64_t> done{0};
    cudaError_t e = prepare_kernel(prefix_kernel, kPrefixSmem, false, &done);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(a.prefix_ctas);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kPrefixSmem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pdl ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, prefix_kernel, a, tmk_half, tmv);
}

}  // namespace absp
