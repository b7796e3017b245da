// How a block-scaled FP8 product is laid over the GPU: which kernel takes it,
// its tiles, and what a CTA takes of its SM.  Arithmetic without CUDA calls,
// so that the rules can be checked on any machine.
#pragma once

#include <cstdint>

#ifdef __CUDACC__
#define TACO_HOST_DEVICE __host__ __device__
#else
#define TACO_HOST_DEVICE
#endif

namespace taco {

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

constexpr uint32_t kSmemLimit = 232448;      // shared memory a CTA may have
constexpr uint32_t kSmemOfSm = 228 * 1024;   // shared memory of an SM; a CTA takes kSmemOfCta more than it asks for
constexpr uint32_t kSmemOfCta = 1024;
constexpr uint32_t kTmemColumns = 512;       // tensor memory of an SM

// A ring of stages (128 rows of 128 codes of one operand, `bn` of the other),
// one of scale pieces, and barriers.
constexpr int kMaxStages = 10;
constexpr int kScaleSlots = 4;
constexpr uint32_t kTileA = 128 * 128;
constexpr uint32_t kBarBytes = 8 * (2 * kMaxStages + 3 * kScaleSlots + 5) + 16;
TACO_HOST_DEVICE constexpr uint32_t stage_bytes_of(int bn) { return kTileA + 128u * bn; }

// Many tiles: width of a tile.
constexpr int kBN = 256;

// An fp32 result: most blocks summed in tensor memory, whose sums truncate.
constexpr int kPieceBlocks = 12;

// Few tiles: CTAs that share a contraction (a portable cluster), and the
// tensor memory of one.  tcgen05.alloc waits without a limit for columns that
// are not free, so no SM may hold more of these CTAs than have columns: each
// asks for more than a third of an SM's shared memory.
constexpr int kMaxSplit = 8;
constexpr uint32_t kSplitTmem = 256;         // accumulators: columns 0 .. 127, scales from 128
constexpr uint32_t kSplitLeastSmem = kSmemOfSm / 3;
static_assert(kSmemOfSm / (kSplitLeastSmem + kSmemOfCta) * kSplitTmem <= kTmemColumns,
              "CTAs on an SM whose tensor memory exceeds the SM's");

// Which kernel: the split one where the other would leave more than half of
// the SMs without a tile and either there are at most 64 tokens and the
// contraction is at least 12 blocks long, or it is at least 48 blocks long and
// a quarter of the SMs cover the 128 x 128 tiles.  Measured, split against
// tiles: 37 x 10240 x 2560 8.9 and 12.1 us, 64 x 4096 x 4096 9.3 and 10.9, 64 x
// 1024 x 1024 6.5 and 5.7, 128 x 4096 x 4096 13.2 and 11.3, 512 x 4096 x 4096
// 16.3 and 11.7, 300 x 300 x 8192 10.6 and 20.8.
inline bool use_split(int64_t M, int64_t N, int64_t K, int sms)
{
    const int64_t KB = ceil_div(K, 128);
    if (ceil_div(M, 128) * ceil_div(N, kBN) >= sms / 2)
        return false;
    return (M <= 64 && KB >= 12) || (KB >= 48 && ceil_div(M, 128) * ceil_div(N, 128) * 4 <= sms);
}

struct SplitPlan {
    int bn;         // columns of a tile (rows of A)
    int tiles_m;
    int64_t tiles;
    int split;      // CTAs to a tile
    int stages;
    uint32_t smem;  // dynamic shared memory of a CTA
    int sums;       // 64 or 128: a CTA's share in pieces, whose sums of up to so many columns are added in registers;
                    // 0: in one piece
};

inline SplitPlan split_plan(int64_t M, int64_t N, int64_t K, int sms, bool out_bf16 = true)
{
    SplitPlan p;
    const int64_t KB = ceil_div(K, 128);
    p.bn = static_cast<int>(M >= 128 ? 128 : ceil_div(M, 16) * 16);
    p.tiles_m = static_cast<int>(ceil_div(M, 128));
    p.tiles = ceil_div(N, 128) * p.tiles_m;
    p.split = 1;
    while (p.split < kMaxSplit && p.tiles * (p.split + 1) <= 2 * sms && KB / (p.split + 1) >= 2)
        ++p.split;
    p.sums = out_bf16 || ceil_div(KB, p.split) <= kPieceBlocks ? 0 : p.bn <= 64 ? 64 : 128;
    // two CTAs share an SM; the ring also holds the partial sums (512 bytes
    // a column)
    const uint32_t per = stage_bytes_of(p.bn), fixed = 1024 + kScaleSlots * 1024 + kBarBytes;
    const int64_t room = (kSmemLimit / 2 - kSmemOfCta - fixed) / per;
    const int64_t need = ceil_div(KB, p.split), least = ceil_div(512 * p.bn, per);
    int64_t stages = room < kMaxStages ? room : kMaxStages;
    stages = stages > need ? need : stages;
    p.stages = static_cast<int>(stages < least ? least : stages);
    p.smem = fixed + p.stages * per;
    p.smem = p.smem < kSplitLeastSmem ? kSplitLeastSmem : p.smem;
    return p;
}

}  // namespace taco
