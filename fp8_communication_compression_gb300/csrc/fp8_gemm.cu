// Products of block-scaled FP8 matrices on the tensor cores:
//
//   out[m][n] = sum over blocks b of 2^(ea[b][m] + eb[b][n]) (A[m, b] . B[n, b])
//
// A and B hold E4M3 codes in rows along the contraction, with one E8M0 byte
// per block of 128 (per row, or for B per 128 x 128 tile).  tcgen05.mma
// kind::mxf8f6f4 applies the scales itself while it accumulates in fp32, so
// no partial sum leaves tensor memory before the end of the contraction;
// the result is rounded once, to bf16 or not at all.  The instruction takes
// a scale per 32 values: each of the four 32-wide steps of a block reads the
// block's byte.
//
// Two kernels share the stage pipeline below.
//
// fp8_gemm_kernel (many tiles): persistent, one CTA per SM, tiles of 128 x
//   BN.  Warp 0 streams 128-byte-wide tiles of A and B by TMA through an
//   mbarrier ring; warp 6 reads the block's scale bytes and lays them out
//   for tcgen05.cp in the same ring slot; one thread of warp 1 copies them to
//   tensor memory and issues the MMAs; warps 2-5 store finished tiles.
//   Tensor memory holds the scales (2 x 12 columns, alternating between
//   blocks) and two accumulators.  At BN = 256 the two overlap by 32
//   columns: the epilogue drains these first and the next tile's MMAs start
//   while it works on the rest.
//
// fp8_gemm_split_kernel (few tiles: single tokens to small batches): the
//   roles of the operands are exchanged - B's rows (weights) take the 128
//   lanes and A's rows (tokens) the columns, 16 to 128 of them - so that a
//   token costs little beyond the weights' bytes.  A cluster of S CTAs
//   splits the contraction; the partial sums meet in distributed shared
//   memory, added in the order of the split, each CTA finishing a share of
//   the columns.  No workspace, no atomics, and a fixed summation order.
//
// Every mbarrier wait is time-limited; one that runs out sets a flag that
// taco_device_error() reads, and the CTA winds down.

#include <atomic>

#include "device_utils.cuh"
#include "fp8_block.cuh"
#include "internal.h"
#include "tcgen05.cuh"

namespace taco {

// Watchdog flag of this file's kernels (bit 6), read by taco_device_error().
__device__ unsigned int g_fp8_error;

namespace {

constexpr uint32_t kErrFp8 = 64u;
constexpr int kThreads = 224;  // warps: 0 TMA, 1 MMA, 2-5 epilogue, 6 scales
constexpr int kMaxStages = 10;
constexpr uint32_t kTileA = 128 * 128;
constexpr uint32_t kSmemLimit = 232448;

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

// Scale bytes of one operand: [blocks][rows], or [blocks][ceil(rows / 128)]
// with one byte per 128 rows.
struct Scales {
    const uint8_t *p;
    int64_t rows;
    bool tiles;
};

// Four blocks' scale bytes of GROUPS x 128 operand rows, as loaded: lane l
// holds rows 128 g + 32 c + l.
template <int GROUPS> struct ScaleBatch {
    uint32_t v[4][GROUPS][4];

    __device__ __forceinline__ void load(const Scales &s, int64_t row0, int kb, int kb_end, int lane)
    {
        const int64_t stride = s.tiles ? (s.rows + 127) / 128 : s.rows;
#pragma unroll
        for (int k = 0; k < 4; ++k)
#pragma unroll
            for (int g = 0; g < GROUPS; ++g)
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    const int64_t row = row0 + 128 * g + 32 * c + lane;
                    v[k][g][c] = 127u;
                    if (kb + k < kb_end && row < s.rows)
                        v[k][g][c] = __ldg(s.p + (kb + k) * stride + (s.tiles ? row >> 7 : row));
                }
    }
    // block k's bytes into the 512-byte areas at `dst`, each byte repeated
    // over its word
    __device__ __forceinline__ void store(int k, uint32_t dst, int lane) const
    {
#pragma unroll
        for (int g = 0; g < GROUPS; ++g) {
            const uint32_t *w = v[k][g];
            sts128(dst + 512 * g + 16 * lane, w[0] * 0x01010101u, w[1] * 0x01010101u, w[2] * 0x01010101u,
                   w[3] * 0x01010101u);
        }
    }
};

// Shared-memory layout of a ring of `stages` slots for operand tiles of 128
// and `bn` rows, scale areas beside them, and `extra` bytes.
struct Ring {
    uint32_t base, stage_bytes, scales, scale_bytes, extra, bars;
    int stages;
    __device__ __forceinline__ uint32_t a(int s) const { return base + s * stage_bytes; }
    __device__ __forceinline__ uint32_t b(int s) const { return base + s * stage_bytes + kTileA; }
    __device__ __forceinline__ uint32_t sf(int s) const { return scales + s * scale_bytes; }
    __device__ __forceinline__ uint32_t full(int s) const { return bars + 8 * s; }
    __device__ __forceinline__ uint32_t empty(int s) const { return bars + 8 * (kMaxStages + s); }
    __device__ __forceinline__ uint32_t acc_full(int a) const { return bars + 8 * (2 * kMaxStages + a); }
    __device__ __forceinline__ uint32_t acc_free(int a) const { return bars + 8 * (2 * kMaxStages + 2 + a); }
    __device__ __forceinline__ uint32_t drain() const { return bars + 8 * (2 * kMaxStages + 4); }
    __device__ __forceinline__ uint32_t tmem_slot() const { return bars + 8 * (2 * kMaxStages + 5); }
};
constexpr uint32_t kBarBytes = 8 * (2 * kMaxStages + 5) + 16;

__host__ __device__ constexpr uint32_t stage_bytes_of(int bn) { return kTileA + 128u * bn; }

__device__ __forceinline__ Ring make_ring(const uint8_t *smem, int bn, int stages, uint32_t scale_bytes,
                                          uint32_t extra)
{
    Ring r;
    r.base = (smem_u32(smem) + 1023u) & ~1023u;
    r.stages = stages;
    r.stage_bytes = stage_bytes_of(bn);
    r.extra = r.base + stages * r.stage_bytes;
    r.scales = r.extra + extra;
    r.scale_bytes = scale_bytes;
    r.bars = r.scales + stages * scale_bytes;
    return r;
}

// A position in the ring: slot and the parity of its use.
struct Slot {
    int s = 0;
    uint32_t phase = 0;
    __device__ __forceinline__ void next(int stages)
    {
        if (++s == stages) {
            s = 0;
            phase ^= 1;
        }
    }
};

// One block of the contraction: its scales to tensor memory, then four MMAs
// of 32 values each.
__device__ __forceinline__ void mma_block(const Ring &r, int s, uint32_t d, uint32_t sfa, uint32_t sfb,
                                          int b_groups, uint32_t idesc, bool accumulate)
{
    tmem_copy_scales(sfa, r.sf(s));
    tmem_copy_scales(sfb, r.sf(s) + 512);
    if (b_groups > 1)
        tmem_copy_scales(sfb + 4, r.sf(s) + 1024);
    const uint64_t ad = smem_desc_k_sw128(r.a(s)), bd = smem_desc_k_sw128(r.b(s));
#pragma unroll
    for (int k = 0; k < 4; ++k)  // 32 codes = 32 bytes = 2 descriptor units
        mma_mxf8(d, ad + 2 * k, bd + 2 * k, idesc, sfa, sfb, accumulate || k != 0);
    mma_commit(r.empty(s));  // the slot is free once these have read it
}

// ------------------------------------------------------------ many tiles --

constexpr uint32_t kStaging = 4 * 4096;   // 4 KB per epilogue warp
constexpr uint32_t kSfColumn = 480;        // tensor-memory columns 480 .. 503: scales
constexpr int kGroupM = 16;                // row tiles walked together (operands shared through L2)

struct TileWalk {
    int tiles_m, tiles_n;
    __device__ __forceinline__ void at(int idx, int &tm, int &tn) const
    {
        const int per = kGroupM * tiles_n, g = idx / per, r = idx - g * per;
        const int left = tiles_m - g * kGroupM, gm = left < kGroupM ? left : kGroupM;
        tn = r / gm;
        tm = g * kGroupM + (r - tn * gm);
    }
};

// 32 columns of a warp's 32 rows: rounded into the staging area and stored,
// by TMA where the output's rows allow it (`tma`), else element by element
// with the lanes along the row.
template <bool BF16>
__device__ __forceinline__ void store_chunk(const float (&x)[32], uint32_t stage, int lane, bool tma,
                                            const CUtensorMap *map, void *out, int64_t M, int64_t N, int64_t row0,
                                            int64_t col0)
{
    if (lane == 0) {
        // the store that used this staging area before has read it (bf16
        // has two areas in turn, fp32 one)
        if (BF16)
            asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");
        else
            bulk_wait_read_all();
    }
    __syncwarp();
    if constexpr (BF16) {
        const uint32_t row = stage + 64 * lane, swz = (lane >> 1) & 3;
#pragma unroll
        for (int j = 0; j < 4; ++j)
            sts128(row + ((j ^ swz) << 4), f32x2_to_bf16x2(x[8 * j], x[8 * j + 1]),
                   f32x2_to_bf16x2(x[8 * j + 2], x[8 * j + 3]), f32x2_to_bf16x2(x[8 * j + 4], x[8 * j + 5]),
                   f32x2_to_bf16x2(x[8 * j + 6], x[8 * j + 7]));
    } else {
        const uint32_t row = stage + 128 * lane, swz = lane & 7;
#pragma unroll
        for (int j = 0; j < 8; ++j)
            sts128(row + ((j ^ swz) << 4), __float_as_uint(x[4 * j]), __float_as_uint(x[4 * j + 1]),
                   __float_as_uint(x[4 * j + 2]), __float_as_uint(x[4 * j + 3]));
    }
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
        const int64_t col = col0 + lane;
#pragma unroll 4
        for (int r = 0; r < 32; ++r) {
            if (row0 + r >= M)
                break;
            if constexpr (BF16) {
                uint16_t h;
                asm volatile("ld.shared.u16 %0, [%1];"
                             : "=h"(h)
                             : "r"(stage + 64 * r + (((lane >> 3) ^ ((r >> 1) & 3)) << 4) + 2 * (lane & 7)));
                if (col < N)
                    static_cast<uint16_t *>(out)[(row0 + r) * N + col] = h;
            } else {
                const uint32_t w = lds32(stage + 128 * r + (((lane >> 2) ^ (r & 7)) << 4) + 4 * (lane & 3));
                if (col < N)
                    static_cast<uint32_t *>(out)[(row0 + r) * N + col] = w;
            }
        }
        __syncwarp();
    }
}

template <bool BF16>
__global__ void __launch_bounds__(kThreads, 1)
    fp8_gemm_kernel(const __grid_constant__ CUtensorMap a_map, const __grid_constant__ CUtensorMap b_map,
                    const __grid_constant__ CUtensorMap o_map, Scales sa, Scales sb, void *__restrict__ out,
                    int64_t M, int64_t N, int KB, int BN, int stages, TileWalk walk, int tma_out)
{
    extern __shared__ uint8_t smem_raw[];
    const Ring r = make_ring(smem_raw, BN, stages, 1536, kStaging);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int ntiles = walk.tiles_m * walk.tiles_n;
    // the second accumulator's first column; above 240 columns the two share
    // some
    const bool overlap = 2 * BN > static_cast<int>(kSfColumn);
    const uint32_t acc1 = overlap ? kSfColumn - BN : BN;

    if (threadIdx.x == 0) {
        for (int s = 0; s < stages; ++s) {
            mbar_init(r.full(s), 2);   // the TMA warp's expect-tx arrival and the scale warp's
            mbar_init(r.empty(s), 1);
        }
        for (int a = 0; a < 2; ++a) {
            mbar_init(r.acc_full(a), 1);
            mbar_init(r.acc_free(a), 4);   // one arrival per epilogue warp
        }
        mbar_init(r.drain(), 1);
        fence_barrier_init();
    }
    if (warp == 1) {
        tmem_alloc(r.tmem_slot(), 512);
        tmem_relinquish_alloc_permit();
    }
    pdl_wait();
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem = lds32(r.tmem_slot());

    if (warp == 0) {
        if (lane == 0) {
            tma_prefetch_map(&a_map);
            tma_prefetch_map(&b_map);
            Slot p;
            int64_t issued = 0;
            bool ok = true;
            for (int idx = blockIdx.x; ok && idx < ntiles; idx += gridDim.x) {
                int tm, tn;
                walk.at(idx, tm, tn);
                for (int kb = 0; kb < KB; ++kb) {
                    if (!mbar_wait(r.empty(p.s), p.phase ^ 1)) {
                        report_timeout();
                        ok = false;
                        break;
                    }
                    mbar_arrive_expect_tx(r.full(p.s), r.stage_bytes);
                    tma_load_2d(r.a(p.s), &a_map, kb * 128, tm * 128, r.full(p.s));
                    tma_load_2d(r.b(p.s), &b_map, kb * 128, tn * BN, r.full(p.s));
                    p.next(stages);
                    ++issued;
                }
            }
            // leave no load in flight into this CTA's shared memory
            for (int64_t i = issued > stages ? issued - stages : 0; i < issued; ++i)
                mbar_wait(r.full(static_cast<int>(i % stages)), static_cast<uint32_t>(i / stages) & 1);
        }
    } else if (warp == 1) {
        if (lane == 0) {
            const uint32_t idesc = idesc_mxf8(BN);
            const int groups = BN > 128 ? 2 : 1;
            Slot p;
            int i = 0;
            uint32_t blk = 0;
            bool ok = true;
            for (int idx = blockIdx.x; ok && idx < ntiles; idx += gridDim.x, ++i) {
                // the epilogue has drained this accumulator's last tile (i -
                // 2); or, where the two overlap, the columns shared with
                // tile i - 1 (which it reaches after all of tile i - 2)
                const int j = overlap ? i - 1 : i - 2;
                if (j >= 0 && !mbar_wait(r.acc_free(j & 1), (j >> 1) & 1)) {
                    report_timeout();
                    ok = false;
                    break;
                }
                tc_fence_after_sync();
                const uint32_t d = tmem + (i & 1 ? acc1 : 0u);
                for (int kb = 0; kb < KB; ++kb, ++blk) {
                    if (!mbar_wait(r.full(p.s), p.phase)) {
                        report_timeout();
                        ok = false;
                        break;
                    }
                    tc_fence_after_sync();
                    const uint32_t sfa = tmem + kSfColumn + 12 * (blk & 1);
                    mma_block(r, p.s, d, sfa, sfa + 4, groups, idesc, kb != 0);
                    p.next(stages);
                }
                if (ok)
                    mma_commit(r.acc_full(i & 1));
            }
            if (!ok) {  // tensor memory is freed below: wait for what was issued
                mma_commit(r.drain());
                mbar_wait(r.drain(), 0);
            }
        }
    } else if (warp == 6) {
        Slot p;
        bool ok = true;
        ScaleBatch<1> ba, na;
        ScaleBatch<2> bb, nb;
        int idx = blockIdx.x, tm = 0, tn = 0;
        if (idx < ntiles) {
            walk.at(idx, tm, tn);
            ba.load(sa, static_cast<int64_t>(tm) * 128, 0, KB, lane);
            bb.load(sb, static_cast<int64_t>(tn) * BN, 0, KB, lane);
        }
        int kb = 0;
        while (ok && idx < ntiles) {
            // the next batch's loads in flight while this one is handed on
            int nidx = idx, nkb = kb + 4;
            if (nkb >= KB) {
                nkb = 0;
                nidx += gridDim.x;
                if (nidx < ntiles)
                    walk.at(nidx, tm, tn);
            }
            if (nidx < ntiles) {
                na.load(sa, static_cast<int64_t>(tm) * 128, nkb, KB, lane);
                nb.load(sb, static_cast<int64_t>(tn) * BN, nkb, KB, lane);
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                if (!ok || kb + k >= KB)
                    continue;
                if (!__all_sync(0xFFFFFFFFu, mbar_wait(r.empty(p.s), p.phase ^ 1))) {
                    if (lane == 0)
                        report_timeout();
                    ok = false;
                    continue;
                }
                ba.store(k, r.sf(p.s), lane);
                bb.store(k, r.sf(p.s) + 512, lane);
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(r.full(p.s));
                p.next(stages);
            }
            ba = na;
            bb = nb;
            idx = nidx;
            kb = nkb;
        }
    } else {
        const int q = warp & 3;
        const uint32_t staging = r.extra + 4096 * q;
        const int chunks = BN / 32;
        int i = 0;
        uint32_t area = 0;  // bf16: the staging area of the next chunk, 0 or 2048
        for (int idx = blockIdx.x; idx < ntiles; idx += gridDim.x, ++i) {
            int tm, tn;
            walk.at(idx, tm, tn);
            if (!__all_sync(0xFFFFFFFFu, mbar_wait(r.acc_full(i & 1), (i >> 1) & 1))) {
                if (lane == 0)
                    report_timeout();
                break;
            }
            tc_fence_after_sync();
            const uint32_t tq = tmem + (i & 1 ? acc1 : 0u) + (static_cast<uint32_t>(32 * q) << 16);
            const int64_t row0 = static_cast<int64_t>(tm) * 128 + 32 * q, col0 = static_cast<int64_t>(tn) * BN;
            // the first accumulator shares its last columns with the second,
            // which shares its first: drain those first
#pragma unroll 1
            for (int c = 0; c < chunks; ++c) {
                const int j = i & 1 ? c : chunks - 1 - c;
                float x[32];
                tmem_load_32(tq + 32 * j, x);
                if (c == (overlap ? 0 : chunks - 1)) {
                    tc_fence_before_sync();
                    __syncwarp();
                    if (lane == 0)
                        mbar_arrive(r.acc_free(i & 1));
                }
                store_chunk<BF16>(x, staging + area, lane, tma_out != 0, &o_map, out, M, N, row0, col0 + 32 * j);
                if (BF16)
                    area ^= 2048;
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

__device__ __forceinline__ void cluster_sync()
{
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

__device__ __forceinline__ float ld_cluster_f32(uint32_t addr, uint32_t rank)
{
    float v;
    asm volatile("{\n\t.reg .b32 a;\n\tmapa.shared::cluster.u32 a, %1, %2;\n\tld.shared::cluster.f32 %0, [a];\n\t}"
                 : "=f"(v)
                 : "r"(addr), "r"(rank)
                 : "memory");
    return v;
}

constexpr uint32_t kSplitTmem = 256;       // accumulator: columns 0 .. 127, scales from 128

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
// 1) / S of the contraction.  Lanes: rows of B (n); columns: rows of A (m).
template <bool BF16>
__global__ void __launch_bounds__(kThreads)
    fp8_gemm_split_kernel(const __grid_constant__ CUtensorMap a_map, const __grid_constant__ CUtensorMap b_map,
                          Scales sa, Scales sb, void *__restrict__ out, int64_t M, int64_t N, int KB, int BN,
                          int stages, int tiles_m, int split)
{
    extern __shared__ uint8_t smem_raw[];
    const Ring r = make_ring(smem_raw, BN, stages, 1024, 0);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = blockIdx.x % split, tile = blockIdx.x / split;
    const int64_t n0 = static_cast<int64_t>(tile / tiles_m) * 128, m0 = static_cast<int64_t>(tile % tiles_m) * BN;
    const int kb0 = static_cast<int>(static_cast<int64_t>(KB) * rank / split);
    const int kb1 = static_cast<int>(static_cast<int64_t>(KB) * (rank + 1) / split);

    if (threadIdx.x == 0) {
        for (int s = 0; s < stages; ++s) {
            mbar_init(r.full(s), 2);
            mbar_init(r.empty(s), 1);
        }
        mbar_init(r.acc_full(0), 1);
        mbar_init(r.drain(), 1);
        fence_barrier_init();
    }
    if (warp == 1) {
        tmem_alloc(r.tmem_slot(), kSplitTmem);
        tmem_relinquish_alloc_permit();
    }
    pdl_wait();
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem = lds32(r.tmem_slot());

    if (warp == 0) {
        if (lane == 0) {
            Slot p;
            int issued = 0;
            for (int kb = kb0; kb < kb1; ++kb) {
                if (!mbar_wait(r.empty(p.s), p.phase ^ 1)) {
                    report_timeout();
                    break;
                }
                mbar_arrive_expect_tx(r.full(p.s), r.stage_bytes);
                tma_load_2d(r.a(p.s), &b_map, kb * 128, static_cast<int32_t>(n0), r.full(p.s));
                tma_load_2d(r.b(p.s), &a_map, kb * 128, static_cast<int32_t>(m0), r.full(p.s));
                p.next(stages);
                ++issued;
            }
            for (int i = issued > stages ? issued - stages : 0; i < issued; ++i)
                mbar_wait(r.full(i % stages), static_cast<uint32_t>(i / stages) & 1);
        }
    } else if (warp == 1) {
        if (lane == 0) {
            const uint32_t idesc = idesc_mxf8(BN);
            Slot p;
            bool ok = true;
            for (int kb = kb0; kb < kb1; ++kb) {
                if (!mbar_wait(r.full(p.s), p.phase)) {
                    report_timeout();
                    ok = false;
                    break;
                }
                tc_fence_after_sync();
                const uint32_t sf = tmem + 128 + 8 * (kb & 1);
                mma_block(r, p.s, tmem, sf, sf + 4, 1, idesc, kb != kb0);
                p.next(stages);
            }
            mma_commit(ok ? r.acc_full(0) : r.drain());
            if (!ok)
                mbar_wait(r.drain(), 0);
        }
    } else if (warp == 6) {
        Slot p;
        bool ok = true;
        ScaleBatch<1> ba, bb;
        for (int kb = kb0; ok && kb < kb1; kb += 4) {
            bb.load(sb, n0, kb, kb1, lane);
            ba.load(sa, m0, kb, kb1, lane);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                if (!ok || kb + k >= kb1)
                    continue;
                if (!__all_sync(0xFFFFFFFFu, mbar_wait(r.empty(p.s), p.phase ^ 1))) {
                    if (lane == 0)
                        report_timeout();
                    ok = false;
                    continue;
                }
                bb.store(k, r.sf(p.s), lane);
                ba.store(k, r.sf(p.s) + 512, lane);
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(r.full(p.s));
                p.next(stages);
            }
        }
    } else {
        const int q = warp & 3, row = 32 * q + lane;
        const int64_t n = n0 + row;
        if (!__all_sync(0xFFFFFFFFu, mbar_wait(r.acc_full(0), 0))) {
            if (lane == 0)
                report_timeout();
        } else {
            tc_fence_after_sync();
            const uint32_t tq = tmem + (static_cast<uint32_t>(32 * q) << 16);
#pragma unroll 1
            for (int j = 0; j < BN; j += 32) {
                float x[32];
                tmem_load_32(tq + j, x);
#pragma unroll
                for (int c = 0; c < 32; ++c) {
                    if (split > 1) {
                        // every load of this CTA has landed and been read
                        // (acc_full): the ring's memory holds the partials,
                        // [column][128 rows]
                        if (j + c < BN)
                            asm volatile("st.shared.f32 [%0], %1;" ::"r"(r.base + 4 * (128 * (j + c) + row)), "f"(x[c])
                                         : "memory");
                    } else if (j + c < BN && m0 + j + c < M && n < N) {
                        store_one<BF16>(out, (m0 + j + c) * N + n, x[c]);
                    }
                }
            }
        }
    }
    tc_fence_before_sync();
    if (split > 1) {
        __syncwarp();
        cluster_sync();
        // this CTA's share of the columns: the 128 rows of a column across
        // four warps, the partials added in the order of the split
        const int t = threadIdx.x;
        if (t < 128 && n0 + t < N) {
            for (int c = rank; c < BN && m0 + c < M; c += split) {
                float acc = 0.0f;
                for (int p = 0; p < split; ++p)
                    acc += ld_cluster_f32(r.base + 4 * (128 * c + t), p);
                store_one<BF16>(out, (m0 + c) * N + n0 + t, acc);
            }
        }
        __syncwarp();
        cluster_sync();  // no CTA leaves while another reads its shared memory
    } else {
        __syncthreads();
    }
    if (warp == 1) {
        tc_fence_after_sync();
        tmem_dealloc(tmem, kSplitTmem);
    }
}

constexpr int kMaxDevices = 64;

template <class K> cudaError_t ensure_smem(K kernel, uint32_t bytes, int device, std::atomic<bool> *set)
{
    if (set[device].load(std::memory_order_acquire))
        return cudaSuccess;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(bytes));
    if (e == cudaSuccess)
        set[device].store(true, std::memory_order_release);
    return e;
}

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

struct Plan {
    bool split_kernel;
    int bn, split;
};

// Which kernel, tile width and split a product takes.
Plan plan_gemm(int64_t M, int64_t N, int KB, int sms)
{
    Plan p{};
    const int64_t tm = ceil_div(M, 128);
    if (tm * ceil_div(N, 256) >= sms / 2) {
        // whole rounds of one tile per SM: the width whose rounds cost least
        double best = 0.0;
        for (int bn = 256; bn >= 128; bn -= 32) {
            const double cost = static_cast<double>(ceil_div(tm * ceil_div(N, bn), sms)) * (bn + 8);
            if (p.bn == 0 || cost < best) {
                best = cost;
                p.bn = bn;
            }
        }
        p.split = 1;
        return p;
    }
    p.split_kernel = true;
    p.bn = static_cast<int>(M >= 128 ? 128 : ceil_div(M, 16) * 16);
    const int64_t tiles = ceil_div(N, 128) * ceil_div(M, p.bn);
    p.split = 1;
    while (p.split < 8 && tiles * (p.split + 1) <= 2 * sms && KB / (p.split + 1) >= 2)
        ++p.split;
    return p;
}

template <bool BF16>
cudaError_t run_gemm(const uint8_t *a, Scales sa, const uint8_t *b, Scales sb, int64_t M, int64_t N, int64_t K,
                     void *out, const DeviceInfo &di, cudaStream_t stream)
{
    const int KB = static_cast<int>(ceil_div(K, 128));
    const Plan p = plan_gemm(M, N, KB, di.num_sms);
    CUtensorMap am, bm, om;
    const uint32_t arows = p.split_kernel ? p.bn : 128, brows = p.split_kernel ? 128 : p.bn;
    if (encode_tensor_map_2d(&am, CU_TENSOR_MAP_DATA_TYPE_UINT8, const_cast<uint8_t *>(a), K, M, K, 128, arows) != 0 ||
        encode_tensor_map_2d(&bm, CU_TENSOR_MAP_DATA_TYPE_UINT8, const_cast<uint8_t *>(b), K, N, K, 128, brows) != 0)
        return cudaErrorInvalidValue;
    if (p.split_kernel) {
        static std::atomic<bool> set[kMaxDevices];
        const uint32_t per = stage_bytes_of(p.bn) + 1024;
        // two CTAs share an SM; the ring also holds the partial sums (512
        // bytes a column)
        int stages = static_cast<int>((kSmemLimit / 2 - 2048 - kBarBytes) / per);
        const int need = static_cast<int>(ceil_div(KB, p.split));
        const int min_stages = static_cast<int>(ceil_div(512 * p.bn, stage_bytes_of(p.bn)));
        stages = stages > kMaxStages ? kMaxStages : stages;
        stages = stages > need ? need : stages;
        stages = stages < min_stages ? min_stages : stages;
        const uint32_t smem = 1024 + stages * per + kBarBytes;
        cudaError_t e = ensure_smem(fp8_gemm_split_kernel<BF16>, kSmemLimit / 2, di.device, set);
        if (e != cudaSuccess)
            return e;
        const int tiles_m = static_cast<int>(ceil_div(M, p.bn));
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = static_cast<unsigned>(ceil_div(N, 128) * tiles_m * p.split);
        cfg.blockDim = kThreads;
        cfg.dynamicSmemBytes = smem;
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
        return cudaLaunchKernelEx(&cfg, fp8_gemm_split_kernel<BF16>, am, bm, sa, sb, out, M, N, KB, p.bn, stages,
                                  tiles_m, p.split);
    }
    static std::atomic<bool> set[kMaxDevices];
    cudaError_t e = ensure_smem(fp8_gemm_kernel<BF16>, kSmemLimit, di.device, set);
    if (e != cudaSuccess)
        return e;
    const uint32_t es = BF16 ? 2 : 4;
    const int tma_out = (static_cast<uint64_t>(N) * es) % 16 == 0;
    om = am;
    if (tma_out &&
        encode_tensor_map_2d(&om, BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32, out, N, M,
                             static_cast<uint64_t>(N) * es, 32, 32,
                             BF16 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B) != 0)
        return cudaErrorInvalidValue;
    const uint32_t per = stage_bytes_of(p.bn) + 1536;
    int stages = static_cast<int>((kSmemLimit - 1024 - kStaging - kBarBytes) / per);
    stages = stages > kMaxStages ? kMaxStages : stages;
    const uint32_t smem = 1024 + stages * per + kStaging + kBarBytes;
    TileWalk walk{static_cast<int>(ceil_div(M, 128)), static_cast<int>(ceil_div(N, p.bn))};
    const int64_t tiles = static_cast<int64_t>(walk.tiles_m) * walk.tiles_n;
    const int grid = static_cast<int>(tiles < di.num_sms ? tiles : di.num_sms);
    return launch_pdl(fp8_gemm_kernel<BF16>, grid, kThreads, smem, stream, am, bm, om, sa, sb, out, M, N, KB, p.bn,
                      stages, walk, tma_out);
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

cudaError_t launch_fp8_gemm(const uint8_t *a, const uint8_t *a_scale, const uint8_t *b, const uint8_t *b_scale,
                            bool b_scale_tiles, int64_t M, int64_t N, int64_t K, void *out, bool out_bf16,
                            cudaStream_t stream)
{
    if (K == 0)  // an empty contraction: zeros
        return cudaMemsetAsync(out, 0, static_cast<size_t>(M) * N * (out_bf16 ? 2 : 4), stream);
    DeviceInfo di;
    cudaError_t e = current_device_info(&di);
    if (e != cudaSuccess)
        return e;
    const Scales sa{a_scale, M, false}, sb{b_scale, N, b_scale_tiles};
    return out_bf16 ? run_gemm<true>(a, sa, b, sb, M, N, K, out, di, stream)
                    : run_gemm<false>(a, sa, b, sb, M, N, K, out, di, stream);
}

}  // namespace taco
