// Products of block-scaled FP8 matrices on the tensor cores:
//
//   out[m][n] = sum over blocks b of 2^(ea[b][m] + eb[b][n]) (A[m, b] . B[n, b])
//
// A and B hold E4M3 codes in rows along the contraction, with one E8M0 byte
// per block of 128 (per row, or for B per 128 x 128 tile).  tcgen05.mma
// kind::mxf8f6f4 applies the scales itself while it accumulates in fp32, so
// no partial sum leaves tensor memory on the way; a bf16 result is rounded
// once.  The instruction takes a scale per 32 values: each of the four
// 32-wide steps of a block reads the block's byte, one of the four in its
// row's scale word (the words hold four blocks, fp8_block.cuh), so a 512-byte
// piece of the stored scales serves 128 rows for four blocks and goes through
// a bulk copy and one tcgen05.cp as it is.  Scales of 128 x 128 tiles are
// spread over such pieces by a warp of their own.
//
// fp8_gemm_kernel (many tiles): persistent, one CTA per SM, tiles of 128 x
//   256.  Warp 0 streams 128-byte-wide pieces of A and B by TMA through an
//   mbarrier ring; warp 2 fetches the scales through a ring of their own, two
//   groups ahead, and spreads tile scales; warp 1 copies scales to tensor
//   memory and issues the MMAs; warps 3-10 store finished tiles.  Tensor
//   memory holds the scales (two sets of 12 columns) and two accumulators,
//   which overlap by 32 columns: the epilogue drains these first, and the
//   next tile's MMAs start while it works on the rest.  Where the last round
//   of tiles would leave more than half of the SMs idle, its tiles are cut in
//   two (128 x 128).
//   Measured: 8192 x 4096 x 4096 to bf16 82 us (3350 TFLOP/s), 4096 x 10240 x
//   2560 70 (3050), 8192 x 4096 x 16384 346 (3180); 16384 x 4096 x 8192 to fp32
//   360 to 380 (2900 to 3050, with the power limit).
//   What bounds it: the MMAs alone run at 512 clocks for a block of 128 (the
//   peak), the loads at 192 KB in flight per SM and the latency of L2 under
//   load (8192 x 4096 x 16384 of zeros at 2070 MHz: four stages 299 us, three
//   352, two 559; the MMAs alone would take 222), and with real operands the
//   power limit (1.75 GHz).  Sharing B between two CTAs, by multicast or as a
//   cta_group::2 pair with six stages of 32 KB, took the same time or a
//   little longer (88 against 86 us at 8192 x 4096 x 4096).
//
// fp8_gemm_split_kernel (few tiles: single tokens to small batches): the
//   roles of the operands are exchanged - B's rows (weights) take the 128
//   lanes and A's rows (tokens) the columns, 16 to 128 of them - so that a
//   token costs little beyond the weights' bytes.  A cluster of S CTAs
//   splits the contraction; the partial sums meet in distributed shared
//   memory, added in the order of the split, each CTA finishing a share of
//   the columns.  No workspace, no atomics, and a fixed summation order.
//
// Either kernel sums an fp32 result over more than 1536 values of a CTA in
// pieces: the tensor core's accumulator truncates, which biases long coherent
// sums (measured on a weight gradient over 4096 tokens: 1.9e-6 of its norm in
// one piece, where an fp32 matrix product has 3.7e-7; 6.2e-7 in pieces), so each
// piece is added in the epilogue's registers, rounded.  A bf16 result is one
// sum, whose bias is far below its rounding (16384 positive values: 6e-6 of the
// sum, where bf16's half step is 2^-9 to 2^-8).
//
// Every mbarrier wait is time-limited; one that runs out sets a flag that
// taco_device_error() reads, and the CTA winds down.  Tensor memory is never
// waited for: no SM holds more CTAs of a kernel than have columns (fp8_plan.h,
// and kGemmSmem leaves room for one), the next grid may start only after a CTA
// has its columns, and a cluster's CTAs give them back before they meet.

#include "device_utils.cuh"
#include "fp8_block.cuh"
#include "fp8_plan.h"
#include "internal.h"
#include "tcgen05.cuh"

namespace taco {

// Watchdog flag of this file's kernels (bit 6), read by taco_device_error().
__device__ unsigned int g_fp8_error;

namespace {

constexpr uint32_t kErrFp8 = 64u;

__device__ __forceinline__ uint32_t lds32(uint32_t addr)
{
    uint32_t v;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(addr));
    return v;
}

__device__ __forceinline__ void mbar_arrive(uint32_t bar)
{
    asm volatile("mbarrier.arrive.release.cta.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}

__device__ __forceinline__ void report_timeout() { atomicOr(&g_fp8_error, kErrFp8); }

// The scales of one operand: 512-byte pieces [row tile][group of four
// blocks], or (tiles) bytes [block][row tile].
struct Scales {
    const uint8_t *p;
    int64_t row_tiles;
    bool tiles;
};

// Shared-memory layout: a ring of `stages` slots for operand pieces of 128
// and `bn` rows, `extra` bytes, a ring of scale slots of `sf_bytes` (128 A or
// lane-side rows, then the others), barriers.
struct Ring {
    uint32_t base, stage_bytes, scales, sf_bytes, extra, bars;
    int stages;
    __device__ __forceinline__ uint32_t a(int s) const { return base + s * stage_bytes; }
    __device__ __forceinline__ uint32_t b(int s) const { return base + s * stage_bytes + kTileA; }
    __device__ __forceinline__ uint32_t sf(int s) const { return scales + s * sf_bytes; }
    __device__ __forceinline__ uint32_t bar(int i) const { return bars + 8 * i; }
    __device__ __forceinline__ uint32_t full(int s) const { return bar(s); }
    __device__ __forceinline__ uint32_t empty(int s) const { return bar(kMaxStages + s); }
    // scales: landed / ready / copied
    __device__ __forceinline__ uint32_t sf_load(int s) const { return bar(2 * kMaxStages + s); }
    __device__ __forceinline__ uint32_t sf_full(int s) const { return bar(2 * kMaxStages + kScaleSlots + s); }
    __device__ __forceinline__ uint32_t sf_empty(int s) const { return bar(2 * kMaxStages + 2 * kScaleSlots + s); }
    __device__ __forceinline__ uint32_t acc_full(int a) const { return bar(2 * kMaxStages + 3 * kScaleSlots + a); }
    __device__ __forceinline__ uint32_t acc_free(int a) const { return bar(2 * kMaxStages + 3 * kScaleSlots + 2 + a); }
    __device__ __forceinline__ uint32_t drain() const { return bar(2 * kMaxStages + 3 * kScaleSlots + 4); }
    __device__ __forceinline__ uint32_t tmem_slot() const { return bar(2 * kMaxStages + 3 * kScaleSlots + 5); }
};

// bn: the operand rows beside A's 128 that a stage of this CTA holds.
__device__ __forceinline__ Ring make_ring(const uint8_t *smem, int bn, int stages, uint32_t sf_bytes, uint32_t extra)
{
    Ring r;
    r.base = (smem_u32(smem) + 1023u) & ~1023u;
    r.stages = stages;
    r.stage_bytes = stage_bytes_of(bn);
    r.extra = r.base + stages * r.stage_bytes;
    r.scales = r.extra + extra;
    r.sf_bytes = sf_bytes;
    r.bars = r.scales + kScaleSlots * sf_bytes;
    return r;
}

// (one thread)  sf_arrivals: the arrivals that make a scale slot ready.
__device__ __forceinline__ void init_barriers(const Ring &r, int sf_arrivals, int epilogue_warps)
{
    for (int s = 0; s < r.stages; ++s) {
        mbar_init(r.full(s), 1);
        mbar_init(r.empty(s), 1);
    }
    for (int s = 0; s < kScaleSlots; ++s) {
        mbar_init(r.sf_load(s), 1);
        mbar_init(r.sf_full(s), sf_arrivals);
        mbar_init(r.sf_empty(s), 1);
    }
    for (int a = 0; a < 2; ++a) {
        mbar_init(r.acc_full(a), 1);
        mbar_init(r.acc_free(a), epilogue_warps);
    }
    mbar_init(r.drain(), 1);
    fence_barrier_init();
}

// A position in a ring: slot and the parity of its use.
struct Slot {
    int s = 0;
    uint32_t phase = 0;
    __device__ __forceinline__ void next(int n)
    {
        if (++s == n) {
            s = 0;
            phase ^= 1;
        }
    }
};

// A new group of four blocks starts at kb (or the contraction's range does).
__device__ __forceinline__ bool starts_group(int kb, int kb0) { return (kb & 3) == 0 || kb == kb0; }

// (the elected thread)  Four MMAs of 32 values each: one block of the
// contraction, whose scales are byte kb % 4 of their words.
__device__ __forceinline__ void mma_block(const Ring &r, int s, uint32_t d, uint32_t sfa, uint32_t sfb, uint32_t idesc,
                                          int kb, uint32_t accumulate)
{
    const uint32_t a = smem_desc_lo(r.a(s)), b = smem_desc_lo(r.b(s)), id = idesc_scale_byte(idesc, kb & 3);
#pragma unroll
    for (int k = 0; k < 4; ++k)  // 32 codes = 32 bytes = 2 descriptor units
        mma_mxf8(d, a + 2 * k, b + 2 * k, id, sfa, sfb, k == 0 ? accumulate : 1u);
    mma_commit(r.empty(s));  // the slot is free once these have read it
}

// (one warp)  Tile scales of blocks 4 g .. 4 g + 3 for row tiles t and t + 1:
// lanes 0-3 hold tile t's bytes, lanes 4-7 tile t + 1's.
__device__ __forceinline__ uint32_t load_tile_scales(const Scales &s, int g, int64_t t, int KB, int lane)
{
    const int kb = 4 * g + (lane & 3);
    const int64_t tile = t + ((lane >> 2) & 1);
    return lane < 8 && kb < KB && tile < s.row_tiles ? __ldg(s.p + kb * s.row_tiles + tile) : 127u;
}

// Spreads them over the 512-byte pieces at dst (`pieces` of them).
__device__ __forceinline__ void spread_tile_scales(uint32_t v, uint32_t dst, int pieces, int lane)
{
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        uint32_t w = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j)
            w |= __shfl_sync(0xFFFFFFFFu, v, 4 * i + j) << (8 * j);
        if (i < pieces)
            sts128(dst + 512 * i + 16 * lane, w, w, w, w);
    }
}

// ------------------------------------------------------------ many tiles --

constexpr int kGThreads = 352;             // warps: 0 TMA, 1 MMA, 2 scales, 3-10 epilogue
constexpr uint32_t kStaging = 8 * 2048;   // 2 KB per epilogue warp
constexpr int kStages = 4;
constexpr uint32_t kAcc1 = 224;            // second accumulator: columns 224 .. 479
constexpr uint32_t kSfColumn = 480;        // tensor-memory columns 480 .. 503: scales
constexpr int kGroupM = 16;                // row tiles walked together (operands shared through L2)
constexpr uint32_t kGemmSmem = 1024 + kStages * stage_bytes_of(kBN) + kStaging + kScaleSlots * 1536 + kBarBytes;
static_assert(kGemmSmem <= kSmemLimit, "shared memory per CTA");

// The work of the grid: `full` whole tiles, then the others as two halves
// each; every item in `segs` pieces of `seg_kb` blocks.
struct Work {
    int tiles_m, tiles_n, full, items, segs, seg_kb, KB;
    int64_t N;
    // Item idx: its row tile, its first column, and its width (256 or 128).
    // False for the second half of a tile that has none.
    __device__ __forceinline__ bool at(int idx, int &tm, int64_t &n0, int &bn) const
    {
        const int t = idx < full ? idx : full + (idx - full) / 2;
        const int per = kGroupM * tiles_n, g = t / per, r = t - g * per;
        const int left = tiles_m - g * kGroupM, gm = left < kGroupM ? left : kGroupM;
        const int tn = r / gm;
        tm = g * kGroupM + (r - tn * gm);
        n0 = static_cast<int64_t>(tn) * kBN;
        bn = kBN;
        if (idx >= full) {
            n0 += 128 * ((idx - full) & 1);
            bn = 128;
        }
        if (N - n0 <= 128)
            bn = 128;
        return n0 < N;
    }
    __device__ __forceinline__ int first(int seg) const { return seg * seg_kb; }
    __device__ __forceinline__ int last(int seg) const
    {
        const int e = (seg + 1) * seg_kb;
        return e < KB ? e : KB;
    }
};

// The groups of four blocks of a CTA's items, in order.
struct ScaleWalk {
    const Work &w;
    int idx, step, g, tm, bn;
    int64_t n0;
    bool more;
    __device__ __forceinline__ ScaleWalk(const Work &work, int idx0, int by) : w(work), idx(idx0 - by), step(by)
    {
        item();
    }
    __device__ __forceinline__ void item()
    {
        do {
            idx += step;
            more = idx < w.items;
        } while (more && !w.at(idx, tm, n0, bn));
        g = 0;
    }
    __device__ __forceinline__ void next()  // pieces start at whole groups: every group once
    {
        if (4 * ++g >= w.KB)
            item();
    }
};

constexpr int kRowLoads = 16;  // rows' loads in flight where they are stored element by element

// 64 bytes of each of a warp's 32 rows (32 bf16 or 16 fp32 columns) from the
// rows' packed words through the staging area to the output, by TMA where
// the output's rows allow it (`tma`), else element by element with the lanes
// along the row (777 x 5119 x 1300: 10 us, 5120 columns by TMA 9; with a branch
// after every row 14).
template <bool BF16>
__device__ __forceinline__ void store_chunk(const uint32_t (&w)[16], uint32_t stage, int lane, bool tma,
                                            const CUtensorMap *map, void *out, int64_t M, int64_t N, int64_t row0,
                                            int64_t col0)
{
    if (lane == 0)
        bulk_wait_read_all();  // the store that used this staging area before has read it
    __syncwarp();
    const uint32_t row = stage + 64 * lane, swz = (lane >> 1) & 3;
#pragma unroll
    for (int j = 0; j < 4; ++j)
        sts128(row + ((j ^ swz) << 4), w[4 * j], w[4 * j + 1], w[4 * j + 2], w[4 * j + 3]);
    if (tma) {
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
            if (row0 < M && col0 < N)
                tma_store_2d(map, static_cast<int32_t>(col0), static_cast<int32_t>(row0), stage);
            bulk_commit();
        }
    } else {
        __syncwarp();
        // a round of loads, then their stores: no branch between them
        const int rows = static_cast<int>(M - row0 < 32 ? M - row0 : 32);
        if constexpr (BF16) {
            const bool inside = col0 + lane < N;
            uint16_t *p = static_cast<uint16_t *>(out) + row0 * N + col0 + lane;
#pragma unroll
            for (int r0 = 0; r0 < 32; r0 += kRowLoads) {
                uint16_t h[kRowLoads];
#pragma unroll
                for (int k = 0; k < kRowLoads; ++k) {
                    const int r = r0 + k;
                    asm volatile("ld.shared.u16 %0, [%1];"
                                 : "=h"(h[k])
                                 : "r"(stage + 64 * r + (((lane >> 3) ^ ((r >> 1) & 3)) << 4) + 2 * (lane & 7)));
                }
#pragma unroll
                for (int k = 0; k < kRowLoads; ++k, p += N)
                    if (inside && r0 + k < rows)
                        *p = h[k];
            }
        } else {  // two rows at a time
            const int l = lane & 15, up = lane >> 4;
            const bool inside = col0 + l < N;
            uint32_t *p = static_cast<uint32_t *>(out) + (row0 + up) * N + col0 + l;
#pragma unroll
            for (int r0 = 0; r0 < 32; r0 += 2 * kRowLoads) {
                uint32_t v[kRowLoads];
#pragma unroll
                for (int k = 0; k < kRowLoads; ++k) {
                    const int r = r0 + 2 * k + up;
                    v[k] = lds32(stage + 64 * r + (((l >> 2) ^ ((r >> 1) & 3)) << 4) + 4 * (l & 3));
                }
#pragma unroll
                for (int k = 0; k < kRowLoads; ++k, p += 2 * N)
                    if (inside && r0 + 2 * k + up < rows)
                        *p = v[k];
            }
        }
        __syncwarp();
    }
}

template <bool BF16>
__global__ void __launch_bounds__(kGThreads, 1)
    fp8_gemm_kernel(const __grid_constant__ CUtensorMap a_map, const __grid_constant__ CUtensorMap b_map,
                    const __grid_constant__ CUtensorMap o_map, Scales sa, Scales sb, void *__restrict__ out, int64_t M,
                    int64_t N, Work work, int tma_out)
{
    extern __shared__ uint8_t smem_raw[];
    const Ring r = make_ring(smem_raw, kBN, kStages, 1536, kStaging);
    const int warp = __shfl_sync(0xFFFFFFFFu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const int groups = (work.KB + 3) / 4;  // scale pieces per row tile
    const int step = gridDim.x;

    if (threadIdx.x == 0)
        init_barriers(r, 1, 8);
    if (warp == 1) {
        tmem_alloc(r.tmem_slot(), 512);
        tmem_relinquish_alloc_permit();
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    // (this CTA holds its tensor memory: the next grid's cannot take it first)
    if (work.items <= 2 * step)
        pdl_trigger();
    pdl_wait();
    const uint32_t tmem = lds32(r.tmem_slot());

    if (warp == 0) {  // the whole warp, so that operands stay uniform; one thread issues
        if (elect_one()) {
            tma_prefetch_map(&a_map);
            tma_prefetch_map(&b_map);
        }
        __syncwarp();
        Slot p;
        int64_t issued = 0;
        bool ok = true;
        for (int idx = blockIdx.x; ok && idx < work.items; idx += step) {
            int tm, bn;
            int64_t n0;
            if (!work.at(idx, tm, n0, bn))
                continue;
            const int32_t mc = tm * 128, nc = static_cast<int32_t>(n0);
            for (int kb = 0; kb < work.KB; ++kb) {
                if (!__all_sync(0xFFFFFFFFu, mbar_wait(r.empty(p.s), p.phase ^ 1))) {
                    ok = false;
                    break;
                }
                if (elect_one()) {
                    const int32_t kc = kb * 128;
                    mbar_arrive_expect_tx(r.full(p.s), stage_bytes_of(bn));
                    tma_load_2d(r.a(p.s), &a_map, kc, mc, r.full(p.s));
                    tma_load_2d(r.b(p.s), &b_map, kc, nc, r.full(p.s));
                    if (bn > 128)
                        tma_load_2d(r.b(p.s) + kTileA, &b_map, kc, nc + 128, r.full(p.s));
                }
                __syncwarp();
                p.next(kStages);
                ++issued;
            }
        }
        if (!ok && lane == 0)
            report_timeout();
        // leave no load in flight into this CTA's shared memory
        for (int64_t i = issued > kStages ? issued - kStages : 0; i < issued; ++i)
            mbar_wait(r.full(static_cast<int>(i % kStages)), static_cast<uint32_t>(i / kStages) & 1);
    } else if (warp == 1) {  // likewise
        Slot p, f;
        int i = 0;  // accumulations done: items times segments
        uint32_t set = 0, sfa = 0;
        bool ok = true;
        auto wait = [&](uint32_t bar, uint32_t parity) { return __all_sync(0xFFFFFFFFu, mbar_wait(bar, parity)); };
        for (int idx = blockIdx.x; ok && idx < work.items; idx += step) {
            int tm, bn;
            int64_t n0;
            if (!work.at(idx, tm, n0, bn))
                continue;
            const uint32_t idesc = idesc_mxf8(bn);
            for (int seg = 0; ok && seg < work.segs; ++seg, ++i) {
                // every epilogue warp has drained the columns this
                // accumulator shares with accumulation i - 1 and, before
                // that, all of i - 2, this accumulator's last
                if (i > 0 && !wait(r.acc_free((i - 1) & 1), ((i - 1) >> 1) & 1)) {
                    ok = false;
                    break;
                }
                tc_fence_after_sync();
                const uint32_t d = tmem + (i & 1 ? kAcc1 : 0u);
                const int kb0 = work.first(seg), kb1 = work.last(seg);
                for (int kb = kb0; kb < kb1; ++kb) {
                    if (starts_group(kb, kb0)) {
                        if (!wait(r.sf_full(f.s), f.phase)) {
                            ok = false;
                            break;
                        }
                        tc_fence_after_sync();
                        sfa = tmem + kSfColumn + 12 * set;
                        set ^= 1;
                        if (elect_one()) {
                            tmem_copy_scales(sfa, r.sf(f.s));
                            tmem_copy_scales(sfa + 4, r.sf(f.s) + 512);
                            if (bn > 128)
                                tmem_copy_scales(sfa + 8, r.sf(f.s) + 1024);
                            mma_commit(r.sf_empty(f.s));
                        }
                        __syncwarp();
                        f.next(kScaleSlots);
                    }
                    if (!wait(r.full(p.s), p.phase)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after_sync();
                    if (elect_one())
                        mma_block(r, p.s, d, sfa, sfa + 4, idesc, kb, kb != kb0);
                    __syncwarp();
                    p.next(kStages);
                }
                if (ok && elect_one())
                    mma_commit(r.acc_full(i & 1));
                __syncwarp();
            }
        }
        if (!ok) {  // tensor memory is freed below: wait for what was issued
            if (elect_one()) {
                report_timeout();
                mma_commit(r.drain());
            }
            __syncwarp();
            mbar_wait(r.drain(), 0);
        }
    } else if (warp == 2) {
        // Scales, two groups ahead of the one being handed on: their loads
        // run on their own, not behind the stages'.
        ScaleWalk ahead(work, blockIdx.x, step), now(work, blockIdx.x, step);
        Slot fa, f;
        bool ok = true;
        auto issue = [&]() {
            if (!ahead.more)
                return true;
            if (!__all_sync(0xFFFFFFFFu, mbar_wait(r.sf_empty(fa.s), fa.phase ^ 1)))
                return false;
            if (elect_one()) {
                const int pieces = sb.tiles ? 0 : ahead.bn / 128;
                mbar_arrive_expect_tx(r.sf_load(fa.s), 512 + 512 * pieces);
                bulk_load(r.sf(fa.s), sa.p + (static_cast<int64_t>(ahead.tm) * groups + ahead.g) * 512, 512,
                          r.sf_load(fa.s));
                for (int i = 0; i < pieces; ++i)
                    bulk_load(r.sf(fa.s) + 512 + 512 * i, sb.p + ((ahead.n0 / 128 + i) * groups + ahead.g) * 512, 512,
                              r.sf_load(fa.s));
            }
            __syncwarp();
            fa.next(kScaleSlots);
            ahead.next();
            return true;
        };
        ok = issue() && issue();
        uint32_t v = now.more && sb.tiles ? load_tile_scales(sb, now.g, now.n0 / 128, work.KB, lane) : 0u;
        while (ok && now.more) {
            const int pieces = now.bn / 128;
            now.next();
            const uint32_t nv = now.more && sb.tiles ? load_tile_scales(sb, now.g, now.n0 / 128, work.KB, lane) : 0u;
            if (!(ok = issue() && __all_sync(0xFFFFFFFFu, mbar_wait(r.sf_load(f.s), f.phase))))
                break;
            if (sb.tiles)
                spread_tile_scales(v, r.sf(f.s) + 512, pieces, lane);
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0)
                mbar_arrive(r.sf_full(f.s));
            f.next(kScaleSlots);
            v = nv;
        }
        if (!ok) {
            if (lane == 0)
                report_timeout();
            // leave none of them in flight
            for (; f.s != fa.s || f.phase != fa.phase; f.next(kScaleSlots))
                mbar_wait(r.sf_load(f.s), f.phase);
        }
    } else {
        // warps 3-6 take columns 0 .. 127 of a tile, upwards, 7-10 columns 255
        // .. 128: the columns that the accumulators share, the second's first
        // 32 and the first's last 32, come first
        const int q = warp & 3, half = (warp - 3) >> 2;
        const uint32_t staging = r.extra + 2048 * (warp - 3);
        int i = 0;
        bool ok = true;
        for (int idx = blockIdx.x; ok && idx < work.items; idx += step) {
            int tm, bn;
            int64_t n0;
            if (!work.at(idx, tm, n0, bn))
                continue;
            const bool mine = 128 * half < bn;
            const int64_t row0 = static_cast<int64_t>(tm) * 128 + 32 * q;
            const int64_t col0 = n0 + 128 * half;
            auto wait_full = [&]() {
                if (!__all_sync(0xFFFFFFFFu, mbar_wait(r.acc_full(i & 1), (i >> 1) & 1))) {
                    if (lane == 0)
                        report_timeout();
                    return false;
                }
                tc_fence_after_sync();
                return true;
            };
            // this warp has read the shared columns (if they are its own),
            // and all of its earlier tiles
            auto free_shared = [&]() {
                tc_fence_before_sync();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(r.acc_free(i & 1));
            };
            auto columns = [&]() {
                return tmem + (i & 1 ? kAcc1 : 0u) + 128 * half + (static_cast<uint32_t>(32 * q) << 16);
            };
            if constexpr (BF16) {
                if (!(ok = wait_full()))
                    break;
                if (!mine) {
                    free_shared();
                } else {
                    const uint32_t tq = columns();
#pragma unroll 1
                    for (int c = 0; c < 4; ++c) {
                        const int j = half ? 3 - c : c;
                        float x[32];
                        tmem_load_32(tq + 32 * j, x);
                        if (c == 0)
                            free_shared();
                        uint32_t w[16];
#pragma unroll
                        for (int k = 0; k < 16; ++k)
                            w[k] = f32x2_to_bf16x2(x[2 * k], x[2 * k + 1]);
                        store_chunk<true>(w, staging, lane, tma_out != 0, &o_map, out, M, N, row0, col0 + 32 * j);
                    }
                }
                ++i;
            } else {
                float sum[8][16] = {};  // 16 columns each, in the order they are read
                for (int seg = 0; seg < work.segs; ++seg, ++i) {
                    if (!(ok = wait_full()))
                        break;
                    if (!mine) {
                        free_shared();
                        continue;
                    }
                    const uint32_t tq = columns();
#pragma unroll
                    for (int j = 0; j < 16; ++j) {
                        float x[8];
                        tmem_load_8(tq + 16 * (half ? 7 - j / 2 : j / 2) + 8 * (j & 1), x);
                        if (j == 3)
                            free_shared();
#pragma unroll
                        for (int k = 0; k < 8; ++k)
                            sum[j / 2][8 * (j & 1) + k] += x[k];
                    }
                }
                if (!ok)
                    break;
                if (mine)
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        uint32_t w[16];
#pragma unroll
                        for (int k = 0; k < 16; ++k)
                            w[k] = __float_as_uint(sum[j][k]);
                        store_chunk<false>(w, staging, lane, tma_out != 0, &o_map, out, M, N, row0,
                                           col0 + 16 * (half ? 7 - j : j));
                    }
            }
        }
        if (lane == 0)
            bulk_wait_all();
    }
    tc_fence_before_sync();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after_sync();
        tmem_dealloc(tmem, 512);
    }
}

// ------------------------------------------------------------- few tiles --

// All threads of the cluster's CTAs meet.
__device__ __forceinline__ void cluster_sync()
{
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// The address of CTA `rank`'s shared memory at this CTA's address `addr`.
__device__ __forceinline__ uint32_t map_cluster(uint32_t addr, uint32_t rank)
{
    uint32_t a;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(addr), "r"(rank));
    return a;
}

__device__ __forceinline__ float4 ld_cluster_f32x4(uint32_t addr)
{
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(addr));
    return v;
}

template <bool BF16> __device__ __forceinline__ void store_one(void *out, int64_t at, float v)
{
    if constexpr (BF16) {
        uint16_t h;
        asm("cvt.rn.bf16.f32 %0, %1;" : "=h"(h) : "f"(v));
        static_cast<uint16_t *>(out)[at] = h;
    } else {
        static_cast<float *>(out)[at] = v;
    }
}

// CTA `rank` of the cluster of tile t takes blocks KB rank / S .. KB (rank +
// 1) / S of the contraction.  Lanes: rows of B (n); columns: rows of A (m),
// BN of them from a multiple of 128.  SUMS: SplitPlan::sums.  If not 0, the
// share is summed in pieces, each of them added in the epilogue's registers: up
// to 64 columns in two accumulators in turn, the MMAs filling one while the
// other is read; up to 128 in one, which is all that the columns allow, by
// twice as many warps.  Two CTAs share an SM either way.
// Measured, in pieces against one: 256 x 256 x 65536 22.4 and 22.3 us, 512 x 512
// x 65536 31.5 and 33.5, 64 x 128 x 100000 26.9 and 25.4, 16 x 16384 x 16384
// 44.0 and 44.3.
__host__ __device__ constexpr int epilogue_warps(int sums) { return sums == 128 ? 8 : 4; }
// warps: 0 TMA, 1 MMA, 2 scales, then the epilogue
__host__ __device__ constexpr int split_threads(int sums) { return 32 * (3 + epilogue_warps(sums)); }

template <bool BF16, int SUMS>
__global__ void __launch_bounds__(split_threads(SUMS), 2)
    fp8_gemm_split_kernel(const __grid_constant__ CUtensorMap a_map, const __grid_constant__ CUtensorMap b_map,
                          Scales sa, Scales sb, void *__restrict__ out, int64_t M, int64_t N, int KB, int BN,
                          int stages, int tiles_m, int split)
{
    extern __shared__ uint8_t smem_raw[];
    const Ring r = make_ring(smem_raw, BN, stages, 1024, 0);
    const int warp = __shfl_sync(0xFFFFFFFFu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const int rank = blockIdx.x % split, tile = blockIdx.x / split;
    const int tn = tile / tiles_m, tm = tile - tn * tiles_m;
    const int64_t n0 = static_cast<int64_t>(tn) * 128, m0 = static_cast<int64_t>(tm) * 128;
    const int kb0 = static_cast<int>(static_cast<int64_t>(KB) * rank / split);
    const int kb1 = static_cast<int>(static_cast<int64_t>(KB) * (rank + 1) / split);
    const int groups = (KB + 3) / 4;
    constexpr int kAccs = SUMS == 64 ? 2 : 1;
    const int share = kb1 - kb0, pieces = SUMS ? (share + kPieceBlocks - 1) / kPieceBlocks : 1;
    const int piece = (share + pieces - 1) / pieces;  // blocks of one

    if (threadIdx.x == 0)
        init_barriers(r, sb.tiles ? 2 : 1, epilogue_warps(SUMS));
    if (warp == 1) {
        tmem_alloc(r.tmem_slot(), kSplitTmem);
        tmem_relinquish_alloc_permit();
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    // (this CTA holds its tensor memory: the next grid's cannot take it first)
    pdl_trigger();
    pdl_wait();
    const uint32_t tmem = lds32(r.tmem_slot());

    if (warp == 0) {
        Slot p, f;
        int issued = 0, scales = 0;
        bool ok = true;
        for (int kb = kb0; kb < kb1; ++kb) {
            if (starts_group(kb, kb0)) {
                if (!__all_sync(0xFFFFFFFFu, mbar_wait(r.sf_empty(f.s), f.phase ^ 1))) {
                    ok = false;
                    break;
                }
                if (elect_one()) {
                    mbar_arrive_expect_tx(r.sf_full(f.s), sb.tiles ? 512 : 1024);
                    bulk_load(r.sf(f.s) + 512, sa.p + (static_cast<int64_t>(tm) * groups + (kb >> 2)) * 512, 512,
                              r.sf_full(f.s));
                    if (!sb.tiles)
                        bulk_load(r.sf(f.s), sb.p + (static_cast<int64_t>(tn) * groups + (kb >> 2)) * 512, 512,
                                  r.sf_full(f.s));
                }
                __syncwarp();
                f.next(kScaleSlots);
                ++scales;
            }
            if (!__all_sync(0xFFFFFFFFu, mbar_wait(r.empty(p.s), p.phase ^ 1))) {
                ok = false;
                break;
            }
            if (elect_one()) {
                mbar_arrive_expect_tx(r.full(p.s), r.stage_bytes);
                tma_load_2d(r.a(p.s), &b_map, kb * 128, static_cast<int32_t>(n0), r.full(p.s));
                tma_load_2d(r.b(p.s), &a_map, kb * 128, static_cast<int32_t>(m0), r.full(p.s));
            }
            __syncwarp();
            p.next(stages);
            ++issued;
        }
        if (!ok && lane == 0)
            report_timeout();
        for (int i = issued > stages ? issued - stages : 0; i < issued; ++i)
            mbar_wait(r.full(i % stages), static_cast<uint32_t>(i / stages) & 1);
        for (int i = scales > kScaleSlots ? scales - kScaleSlots : 0; i < scales; ++i)
            mbar_wait(r.sf_full(i % kScaleSlots), static_cast<uint32_t>(i / kScaleSlots) & 1);
    } else if (warp == 1) {
        const uint32_t idesc = idesc_mxf8(BN);
        Slot p, f;
        uint32_t set = 0, sf = 0;
        int i = 0, first = kb0;  // this piece and its first block
        bool ok = true;
        for (int kb = kb0; kb < kb1; ++kb) {
            if (SUMS != 0 && kb == first + piece) {
                if (elect_one())
                    mma_commit(r.acc_full(i % kAccs));
                __syncwarp();
                first = kb;
                // the last piece in these columns has been read
                if (++i >= kAccs && !__all_sync(0xFFFFFFFFu, mbar_wait(r.acc_free(i % kAccs), (i / kAccs - 1) & 1))) {
                    ok = false;
                    break;
                }
                tc_fence_after_sync();
            }
            if (starts_group(kb, kb0)) {
                if (!__all_sync(0xFFFFFFFFu, mbar_wait(r.sf_full(f.s), f.phase))) {
                    ok = false;
                    break;
                }
                tc_fence_after_sync();
                sf = tmem + 128 + 8 * set;
                set ^= 1;
                if (elect_one()) {
                    tmem_copy_scales(sf, r.sf(f.s));
                    tmem_copy_scales(sf + 4, r.sf(f.s) + 512);
                    mma_commit(r.sf_empty(f.s));
                }
                __syncwarp();
                f.next(kScaleSlots);
            }
            if (!__all_sync(0xFFFFFFFFu, mbar_wait(r.full(p.s), p.phase))) {
                ok = false;
                break;
            }
            tc_fence_after_sync();
            if (elect_one())
                mma_block(r, p.s, tmem + i % kAccs * SUMS, sf, sf + 4, idesc, kb, kb != first);
            __syncwarp();
            p.next(stages);
        }
        if (elect_one()) {
            if (!ok)
                report_timeout();
            mma_commit(ok ? r.acc_full(i % kAccs) : r.drain());
        }
        __syncwarp();
        if (!ok)
            mbar_wait(r.drain(), 0);
    } else if (warp == 2) {
        if (sb.tiles) {
            Slot f;
            const int g1 = (kb1 + 3) / 4;
            int g = kb0 / 4;
            uint32_t v = load_tile_scales(sb, g, tn, KB, lane);
            for (; g < g1; ++g) {
                const uint32_t nv = load_tile_scales(sb, g + 1, tn, KB, lane);
                if (!__all_sync(0xFFFFFFFFu, mbar_wait(r.sf_empty(f.s), f.phase ^ 1))) {
                    if (lane == 0)
                        report_timeout();
                    break;
                }
                spread_tile_scales(v, r.sf(f.s), 1, lane);
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(r.sf_full(f.s));
                f.next(kScaleSlots);
                v = nv;
            }
        }
    } else {
        const int q = warp & 3, row = 32 * q + lane;
        const int64_t n = n0 + row;
        const uint32_t tq = tmem + (static_cast<uint32_t>(32 * q) << 16);
        auto wait_full = [&](int i) {
            const bool ok = __all_sync(0xFFFFFFFFu, mbar_wait(r.acc_full(i % kAccs), (i / kAccs) & 1));
            if (!ok && lane == 0)
                report_timeout();
            tc_fence_after_sync();
            return ok;
        };
        // once every load of this CTA has landed and been read (acc_full of
        // the last piece), the ring's memory holds the partial sums, [column]
        // [128 rows]
        auto put = [&](int c, float v) {
            asm volatile("st.shared.f32 [%0], %1;" ::"r"(r.base + 4 * (128 * c + row)), "f"(v) : "memory");
        };
        if constexpr (SUMS == 0) {
            if (wait_full(0)) {
#pragma unroll 1
                for (int j = 0; j < BN; j += 32) {
                    float x[32];
                    tmem_load_32(tq + j, x);
#pragma unroll
                    for (int c = 0; c < 32; ++c) {
                        if (split > 1) {
                            if (j + c < BN)
                                put(j + c, x[c]);
                        } else if (j + c < BN && m0 + j + c < M && n < N) {
                            store_one<BF16>(out, (m0 + j + c) * N + n, x[c]);
                        }
                    }
                }
            }
        } else {
            constexpr int kColumns = 4 * SUMS / epilogue_warps(SUMS);
            const int c0 = kColumns * ((warp - 3) >> 2);  // this warp's columns
            float sum[kColumns] = {};
            bool ok = true;
            for (int i = 0, kb = kb0; ok && kb < kb1; ++i, kb += piece) {
                if (!(ok = wait_full(i)))
                    break;
#pragma unroll
                for (int j = 0; j < kColumns; j += 8)
                    if (c0 + j < BN) {
                        float x[8];
                        tmem_load_8(tq + i % kAccs * SUMS + c0 + j, x);
#pragma unroll
                        for (int c = 0; c < 8; ++c)
                            sum[j + c] += x[c];
                    }
                tc_fence_before_sync();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(r.acc_free(i % kAccs));
            }
            if (ok)
#pragma unroll
                for (int j = 0; j < kColumns; j += 8)
                    if (c0 + j < BN)
#pragma unroll
                        for (int c = 0; c < 8; ++c)
                            put(c0 + j + c, sum[j + c]);
        }
    }
    // tensor memory goes back before the CTAs wait for one another, so that
    // none that waits for it waits for a cluster
    tc_fence_before_sync();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after_sync();
        tmem_dealloc(tmem, kSplitTmem);
    }
    if (SUMS != 0 || split > 1) {
        __syncwarp();
        cluster_sync();
        // this CTA's share of the columns, a column a warp (four rows a
        // lane): the S partials' loads in flight together, then added in the
        // order of the split
        const int64_t n = n0 + 4 * lane;
        uint32_t parts[kMaxSplit];
#pragma unroll
        for (int p = 0; p < kMaxSplit; ++p)
            parts[p] = map_cluster(r.base, p < split ? p : 0) + 16 * lane;
        for (int c = rank + split * warp; c < BN && m0 + c < M; c += split * (split_threads(SUMS) / 32)) {
            float4 v[kMaxSplit];
#pragma unroll
            for (int p = 0; p < kMaxSplit; ++p)
                if (p < split)
                    v[p] = ld_cluster_f32x4(parts[p] + 512 * c);
            float4 acc = v[0];
#pragma unroll
            for (int p = 1; p < kMaxSplit; ++p)
                if (p < split) {
                    acc.x += v[p].x;
                    acc.y += v[p].y;
                    acc.z += v[p].z;
                    acc.w += v[p].w;
                }
            const int64_t at = (m0 + c) * N + n;
            if (n + 3 < N && (N & 3) == 0) {
                if constexpr (BF16)
                    *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(out) + at) =
                        make_uint2(f32x2_to_bf16x2(acc.x, acc.y), f32x2_to_bf16x2(acc.z, acc.w));
                else
                    *reinterpret_cast<float4 *>(static_cast<float *>(out) + at) = acc;
            } else {
                if (n < N)
                    store_one<BF16>(out, at, acc.x);
                if (n + 1 < N)
                    store_one<BF16>(out, at + 1, acc.y);
                if (n + 2 < N)
                    store_one<BF16>(out, at + 2, acc.z);
                if (n + 3 < N)
                    store_one<BF16>(out, at + 3, acc.w);
            }
        }
        __syncwarp();
        cluster_sync();  // no CTA leaves while another reads its shared memory
    }
}

Scales scales_of(const Fp8Operand &x, int64_t rows) { return {x.scale, ceil_div(rows, 128), x.tiles}; }

// Boxes of 128 codes of `box_rows` rows.
int operand_map(CUtensorMap *map, const Fp8Operand &x, int64_t rows, int64_t K, int box_rows)
{
    return encode_tensor_map_2d(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, const_cast<uint8_t *>(x.codes), K, rows, x.stride,
                                128, box_rows);
}

template <bool BF16, int SUMS>
cudaError_t launch_split(const SplitPlan &p, const Fp8Operand &a, const Fp8Operand &b, int64_t M, int64_t N, int64_t K,
                         void *out, const DeviceInfo &di, cudaStream_t stream)
{
    CUtensorMap am, bm;
    if (operand_map(&am, a, M, K, p.bn) != 0 || operand_map(&bm, b, N, K, 128) != 0)
        return cudaErrorInvalidValue;
    static std::atomic<bool> set[kMaxDevices];
    cudaError_t e = ensure_smem(fp8_gemm_split_kernel<BF16, SUMS>, kSmemLimit / 2, di.device, set);
    if (e != cudaSuccess)
        return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = static_cast<unsigned>(p.tiles * p.split);
    cfg.blockDim = split_threads(SUMS);
    cfg.dynamicSmemBytes = p.smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = p.split;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, fp8_gemm_split_kernel<BF16, SUMS>, am, bm, scales_of(a, M), scales_of(b, N), out, M,
                              N, static_cast<int>(ceil_div(K, 128)), p.bn, p.stages, p.tiles_m, p.split);
}

template <bool BF16>
cudaError_t run_split(const Fp8Operand &a, const Fp8Operand &b, int64_t M, int64_t N, int64_t K,
                      void *out, const DeviceInfo &di, cudaStream_t stream)
{
    const SplitPlan p = split_plan(M, N, K, di.num_sms, BF16);
    if constexpr (!BF16) {
        if (p.sums == 64)
            return launch_split<BF16, 64>(p, a, b, M, N, K, out, di, stream);
        if (p.sums == 128)
            return launch_split<BF16, 128>(p, a, b, M, N, K, out, di, stream);
    }
    return launch_split<BF16, 0>(p, a, b, M, N, K, out, di, stream);
}

template <bool BF16>
cudaError_t run_tiles(const Fp8Operand &a, const Fp8Operand &b, int64_t M, int64_t N, int64_t K,
                      void *out, const DeviceInfo &di, cudaStream_t stream)
{
    CUtensorMap am, bm, om;
    if (operand_map(&am, a, M, K, 128) != 0 || operand_map(&bm, b, N, K, 128) != 0)
        return cudaErrorInvalidValue;
    static std::atomic<bool> set[kMaxDevices];
    cudaError_t e = ensure_smem(fp8_gemm_kernel<BF16>, kGemmSmem, di.device, set);
    if (e != cudaSuccess)
        return e;
    const uint64_t row_bytes = static_cast<uint64_t>(N) * (BF16 ? 2 : 4);
    const int tma_out = row_bytes % 16 == 0;
    om = am;
    if (tma_out && encode_tensor_map_2d(&om, BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32,
                                        out, N, M, row_bytes, BF16 ? 32 : 16, 32, CU_TENSOR_MAP_SWIZZLE_64B) != 0)
        return cudaErrorInvalidValue;
    Work w;
    w.KB = static_cast<int>(ceil_div(K, 128));
    w.N = N;
    w.tiles_m = static_cast<int>(ceil_div(M, 128));
    w.tiles_n = static_cast<int>(ceil_div(N, kBN));
    // fp32: pieces of whole scale groups
    w.segs = BF16 ? 1 : static_cast<int>(ceil_div(w.KB, kPieceBlocks));
    w.seg_kb = static_cast<int>(ceil_div(ceil_div(w.KB, w.segs), 4) * 4);
    w.segs = static_cast<int>(ceil_div(w.KB, w.seg_kb));
    // a last round that fills at most half of the SMs goes in halves
    const int tiles = w.tiles_m * w.tiles_n, rem = tiles % di.num_sms;
    w.full = rem <= di.num_sms / 2 ? tiles - rem : tiles;
    w.items = w.full + 2 * (tiles - w.full);
    const int grid = w.items < di.num_sms ? w.items : di.num_sms;
    return launch_pdl(fp8_gemm_kernel<BF16>, dim3(grid), dim3(kGThreads), kGemmSmem, stream, am, bm, om,
                      scales_of(a, M), scales_of(b, N), out, M, N, w, tma_out);
}

template <bool BF16>
cudaError_t run_gemm(const Fp8Operand &a, const Fp8Operand &b, int64_t M, int64_t N, int64_t K,
                     void *out, const DeviceInfo &di, cudaStream_t stream)
{
    return use_split(M, N, K, di.num_sms) ? run_split<BF16>(a, b, M, N, K, out, di, stream)
                                          : run_tiles<BF16>(a, b, M, N, K, out, di, stream);
}

}  // namespace

cudaError_t read_fp8_error(uint32_t *flags, bool clear)
{
    unsigned int v = 0;
    cudaError_t e = cudaMemcpyFromSymbol(&v, g_fp8_error, sizeof v);
    if (e != cudaSuccess)
        return e;
    *flags = v;
    if (clear) {
        v = 0;
        e = cudaMemcpyToSymbol(g_fp8_error, &v, sizeof v);
    }
    return e;
}

cudaError_t launch_fp8_gemm(const Fp8Operand &a, const Fp8Operand &b, int64_t M, int64_t N, int64_t K, void *out,
                            bool out_bf16, cudaStream_t stream)
{
    if (K == 0)  // an empty contraction: zeros
        return cudaMemsetAsync(out, 0, static_cast<size_t>(M) * N * (out_bf16 ? 2 : 4), stream);
    DeviceInfo di;
    cudaError_t e = current_device_info(&di);
    if (e != cudaSuccess)
        return e;
    return out_bf16 ? run_gemm<true>(a, b, M, N, K, out, di, stream) : run_gemm<false>(a, b, M, N, K, out, di, stream);
}

}  // namespace taco
