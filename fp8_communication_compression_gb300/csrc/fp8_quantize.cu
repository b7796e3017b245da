// Quantises a bf16 matrix to the block-scaled FP8 format: in blocks of 128
// along its rows (the operand of y = x W^T and dx = dy W), in blocks of 128
// along its columns with the codes transposed (the operand of dW = dy^T x,
// whose contraction runs over the rows), both in one pass over the data, or
// in 128 x 128 tiles with the transposed codes beside (weights).
//
// Bound by HBM: 2 bytes read and 1 byte written per element and direction.
// A CTA of 256 threads takes a 128 x 128 tile; a thread holds 8 rows of 8
// columns as packed bf16 in 32 registers, so all of its eight 16-byte loads
// are in flight at once and the maxima are 16-bit packed integer maxima on
// the bit patterns.  Row maxima meet in 4 shuffles between the 16 lanes of a
// row; column maxima through shared memory.  The transposed codes go
// through a 16 KB tile whose 16-byte chunks are swizzled by the column
// group, so that both its 8-byte writes and its 16-byte reads take the
// fewest possible shared-memory cycles.
// Measured at 8192 x 16384: rows 66 us (6120 GB/s), columns 73, both 102
// (5260 GB/s; then it is instructions, 0.71 of the issue slots, that bound
// it).  Where rows are no whole 16-byte granules a thread joins its
// eight columns from two granules: 8192 x 16380 in 99, 108 and 138 us (118,
// 129 and 158 with loads of single elements).

#include "device_utils.cuh"
#include "fp8_block.cuh"
#include "internal.h"

namespace taco {

namespace {

constexpr int kQThreads = 256;
// The next grid may start early after a small one (its product's prologue
// runs meanwhile: 37 x 2560 -> 10240 in 8.7 instead of 10.5 us); after a large
// one that costs bandwidth (both directions of 8192 x 4096: 35 us against 31).
constexpr int kTriggerCtas = 608;  // four on each of the 152 SMs

__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) { return __vmaxu2(a, b); }

// fp32 bit pattern of the larger 16-bit half of a packed pair of bf16
// magnitudes.
__device__ __forceinline__ uint32_t larger_half_f32(uint32_t w)
{
    const uint32_t lo = w << 16, hi = w & 0xFFFF0000u;
    return lo > hi ? lo : hi;
}

// TILE: one scale per 128 x 128 tile; else row blocks (codes) and / or
// column blocks (codes_t).  The CTAs from `second` on take the other matrix
// (a backward pass quantises two in one launch).
template <bool TILE>
__global__ void __launch_bounds__(kQThreads)
    fp8_quantize_kernel(const __grid_constant__ Fp8Quantize first, const __grid_constant__ Fp8Quantize other,
                        unsigned second)
{
    const bool is_other = !TILE && blockIdx.x >= second;
    const Fp8Quantize &job = is_other ? other : first;
    const uint16_t *__restrict__ x = static_cast<const uint16_t *>(job.x);
    uint8_t *__restrict__ codes = job.codes, *__restrict__ scale = job.scale;
    uint8_t *__restrict__ codes_t = job.codes_t, *__restrict__ scale_t = job.scale_t;
    const int64_t rows = job.rows, cols = job.cols, stride = job.stride, stride_t = job.stride_t;
    const int64_t col_tiles = (cols + 127) / 128, tile = blockIdx.x - (is_other ? second : 0u);
    __shared__ uint4 tile_t[128 * 8];       // transposed codes: [column][8 chunks of 16 rows], swizzled
    __shared__ uint4 col_max[8][16];        // per warp: packed maxima of the 128 columns
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int cc = tid & 15, rg = tid >> 4;  // this thread's columns 8 cc .. + 7 and rows 8 rg .. + 7
    const int64_t tr = tile / col_tiles, tc = tile - tr * col_tiles;
    const int64_t r0 = tr * 128, c0 = tc * 128;
    const int64_t r = r0 + 8 * rg, c = c0 + 8 * cc;
    const int64_t pitch = fp8_pitch(cols), pitch_t = fp8_pitch(rows);  // codes and zeros written of a row
    if (gridDim.x <= kTriggerCtas)
        pdl_trigger();
    pdl_wait();

    uint32_t v[8][4];
    const bool vec = (cols & 7) == 0;  // every row starts on a 16-byte boundary
    const int64_t whole = rows * cols & ~int64_t(7);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        uint4 q = make_uint4(0, 0, 0, 0);
        if (r + i < rows) {
            const int64_t at = (r + i) * cols + c;
            if (vec) {
                if (c < cols)
                    q = ldg128_stream(x + at);
            } else if (c < cols) {
                // the row starts `shift` elements into a granule, the same
                // in all threads as r is a multiple of 8
                const int shift = i * static_cast<int>(cols & 7) & 7;
                if (at + 16 - shift <= whole) {
                    q = __ldg(reinterpret_cast<const uint4 *>(x + at - shift));
                    if (shift != 0)
                        q = join(q, __ldg(reinterpret_cast<const uint4 *>(x + at - shift + 8)), shift);
                    if (c + 8 > cols)
                        q = first_elements(q, static_cast<int>(cols - c));
                } else {  // next to the matrix's end
                    uint32_t e[8];
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        e[j] = c + j < cols ? __ldg(x + at + j) : 0u;
                    q = make_uint4(e[0] | e[1] << 16, e[2] | e[3] << 16, e[4] | e[5] << 16, e[6] | e[7] << 16);
                }
            }
        }
        v[i][0] = q.x;
        v[i][1] = q.y;
        v[i][2] = q.z;
        v[i][3] = q.w;
    }

    constexpr uint32_t kAbs = 0x7FFF7FFFu;
    uint32_t tile_byte = 0;
    uint32_t cm[4] = {0, 0, 0, 0};
    if (TILE || codes_t) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j)
                cm[j] = max_u16x2(cm[j], v[i][j] & kAbs);
#pragma unroll
        for (int j = 0; j < 4; ++j)
            cm[j] = max_u16x2(cm[j], __shfl_xor_sync(0xFFFFFFFFu, cm[j], 16));
        if (TILE) {
            const uint32_t m = max_u16x2(max_u16x2(cm[0], cm[1]), max_u16x2(cm[2], cm[3]));
            const uint32_t w = __reduce_max_sync(0xFFFFFFFFu, larger_half_f32(m));
            if (lane == 0)
                col_max[warp][0].x = w;
        } else if (lane < 16) {
            col_max[warp][cc] = make_uint4(cm[0], cm[1], cm[2], cm[3]);
        }
        __syncthreads();
        if (TILE) {
            uint32_t m = 0;
#pragma unroll
            for (int w = 0; w < 8; ++w)
                m = max(m, col_max[w][0].x);
            tile_byte = fp8_scale_byte(m);
        } else {
#pragma unroll
            for (int w = 0; w < 8; ++w) {
                const uint4 o = col_max[w][cc];
                cm[0] = max_u16x2(cm[0], o.x);
                cm[1] = max_u16x2(cm[1], o.y);
                cm[2] = max_u16x2(cm[2], o.z);
                cm[3] = max_u16x2(cm[3], o.w);
            }
        }
    }

    if (codes) {
        uint32_t byte[8];
        if (TILE) {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                byte[i] = tile_byte;
        } else {
            uint32_t rm[4];  // maxima of rows 2 i (low half) and 2 i + 1 (high half)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                uint32_t m[2];
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const uint32_t *w = v[2 * i + k];
                    m[k] = max_u16x2(max_u16x2(w[0] & kAbs, w[1] & kAbs), max_u16x2(w[2] & kAbs, w[3] & kAbs));
                }
                // the larger half of each row's pair
                rm[i] = max_u16x2(__byte_perm(m[0], m[1], 0x5410), __byte_perm(m[0], m[1], 0x7632));
            }
#pragma unroll
            for (int s = 1; s < 16; s <<= 1)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    rm[i] = max_u16x2(rm[i], __shfl_xor_sync(0xFFFFFFFFu, rm[i], s));
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                byte[2 * i] = fp8_scale_byte(rm[i] << 16);
                byte[2 * i + 1] = fp8_scale_byte(rm[i] & 0xFFFF0000u);
            }
            if (cc < 8 && r + cc < rows) {
                uint32_t b = byte[0];
#pragma unroll
                for (int i = 1; i < 8; ++i)
                    b = cc == i ? byte[i] : b;
                scale[fp8_scale_at(r + cc, tc, (col_tiles + 3) / 4)] = static_cast<uint8_t>(b);
            }
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float f = fp8_inv_scale(byte[i]);
            uint32_t o[2];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const uint32_t a = v[i][2 * k], b = v[i][2 * k + 1];
                o[k] = f32x4_to_e4m3x4(bf16lo_to_f32(a) * f, bf16hi_to_f32(a) * f, bf16lo_to_f32(b) * f,
                                       bf16hi_to_f32(b) * f);
            }
            if (r + i < rows && c < pitch)
                *reinterpret_cast<uint2 *>(codes + (r + i) * stride + c) = make_uint2(o[0], o[1]);
        }
    }

    if (codes_t) {
        uint32_t byte[8];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            byte[2 * j] = TILE ? tile_byte : fp8_scale_byte(cm[j] << 16);
            byte[2 * j + 1] = TILE ? tile_byte : fp8_scale_byte(cm[j] & 0xFFFF0000u);
        }
        if (!TILE && rg == 0) {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (c + j < cols)
                    scale_t[fp8_scale_at(c + j, tr, ((rows + 127) / 128 + 3) / 4)] = static_cast<uint8_t>(byte[j]);
        }
        uint8_t *t = reinterpret_cast<uint8_t *>(tile_t) + (((rg >> 1) ^ (cc & 7)) << 4) + ((rg & 1) << 3);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float f = fp8_inv_scale(byte[j]);
            float e[8];
#pragma unroll
            for (int i = 0; i < 8; ++i)
                e[i] = (j & 1 ? bf16hi_to_f32(v[i][j >> 1]) : bf16lo_to_f32(v[i][j >> 1])) * f;
            *reinterpret_cast<uint2 *>(t + (8 * cc + j) * 128) =
                make_uint2(f32x4_to_e4m3x4(e[0], e[1], e[2], e[3]), f32x4_to_e4m3x4(e[4], e[5], e[6], e[7]));
        }
        __syncthreads();
#pragma unroll
        for (int it = 0; it < 4; ++it) {
            const int col = 32 * it + (tid >> 3), ch = tid & 7;
            if (c0 + col < cols && r0 + 16 * ch < pitch_t)
                *reinterpret_cast<uint4 *>(codes_t + (c0 + col) * stride_t + r0 + 16 * ch) =
                    tile_t[col * 8 + (ch ^ ((col >> 3) & 7))];
        }
    }
    if (TILE && tid == 0) {
        const int64_t row_tiles = (rows + 127) / 128;
        if (scale)
            scale[tc * row_tiles + tr] = static_cast<uint8_t>(tile_byte);
        if (scale_t)
            scale_t[tr * col_tiles + tc] = static_cast<uint8_t>(tile_byte);
    }
}

}  // namespace

static unsigned tiles_of(const Fp8Quantize &q)
{
    return static_cast<unsigned>((q.rows + 127) / 128 * ((q.cols + 127) / 128));
}

cudaError_t launch_fp8_quantize(const Fp8Quantize &q, bool tiles, cudaStream_t stream)
{
    const unsigned n = tiles_of(q);
    return tiles ? launch_pdl(fp8_quantize_kernel<true>, dim3(n), kQThreads, 0, stream, q, q, n)
                 : launch_pdl(fp8_quantize_kernel<false>, dim3(n), kQThreads, 0, stream, q, q, n);
}

cudaError_t launch_fp8_quantize_two(const Fp8Quantize &a, const Fp8Quantize &b, cudaStream_t stream)
{
    const unsigned n = tiles_of(a);
    return launch_pdl(fp8_quantize_kernel<false>, dim3(n + tiles_of(b)), kQThreads, 0, stream, a, b, n);
}

}  // namespace taco
