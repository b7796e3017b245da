// The FP8 operand format of the block-scaled products: E4M3 codes with one
// power-of-two scale (an E8M0 byte, 2^(byte - 127)) per block of 128.
//
//   E = the smallest integer with amax <= 448 2^E, at least -127
//   code = E4M3(x 2^-E), byte = E + 127; byte 127 for a block of zeros
//
// 448 is 1.75 2^8, so E is amax's exponent - 8, and one more where its
// fraction is above 1.75: an integer addition to amax's bit pattern that
// carries into the exponent.  x 2^-E is exact (the scale is a power of two
// and the product cannot overflow), so the only rounding is the one to
// E4M3 (nearest even), and the codes do not depend on the precision or the
// order of the arithmetic.  A block that holds an Inf or a NaN gets the
// format's NaN scale (byte 255) and NaN codes, so that it stays visible in
// every product that reads it.
#pragma once

#include <cstdint>

#include "device_utils.cuh"

namespace taco {

// Codes are stored in rows padded with zero codes to a multiple of 16 bytes
// (the stride a TMA tensor map needs).
__host__ __device__ inline int64_t fp8_pitch(int64_t n) { return (n + 15) & ~int64_t(15); }

// Row length of codes that live in a call's workspace: whole 128-byte lines,
// so that a TMA box of 128 codes touches one line a row.  (A product of 4096 x
// 4096 over 8176 codes takes 160 us with rows of 8176 bytes, 124 with 8160, a
// multiple of 32, 108 with 8128, of 64, and 101 over 8192.)
__host__ __device__ inline int64_t fp8_work_pitch(int64_t n) { return (n + 127) & ~int64_t(127); }

// Scales are stored as the tensor core reads them: a 512-byte piece holds the
// bytes of 128 rows for four consecutive blocks, row r's four bytes in the
// word at 16 (r % 32) + 4 (r / 32); pieces [ceil(rows / 128)][ceil(blocks /
// 4)].  Bytes of rows and blocks past the matrix's end are not read into any
// result.
__host__ __device__ inline int64_t fp8_scale_bytes(int64_t rows, int64_t cols)
{
    return ((rows + 127) / 128) * ((cols + 511) / 512) * 512;
}

// Where block b's byte of a row lies; groups = ceil(blocks / 4).
__host__ __device__ inline int64_t fp8_scale_at(int64_t row, int64_t b, int64_t groups)
{
    return ((row >> 7) * groups + (b >> 2)) * 512 + ((row & 31) << 4) + (((row >> 5) & 3) << 2) + (b & 3);
}

// Scale byte from the bit pattern of max |x| (fp32, the sign bit clear; an
// unsigned maximum of such patterns puts Inf and NaN on top).
__device__ __forceinline__ uint32_t fp8_scale_byte(uint32_t amax_bits)
{
    if (amax_bits >= 0x7F800000u)
        return 255u;
    const int b = static_cast<int>((amax_bits + 0x1FFFFFu) >> 23) - 8;
    return amax_bits == 0u ? 127u : static_cast<uint32_t>(b > 0 ? b : 0);
}

// 2^-E of a scale byte; NaN for the NaN scale.  (Bytes of finite blocks are
// at most 247, so the exponent field 254 - byte is that of a normal number.)
__device__ __forceinline__ float fp8_inv_scale(uint32_t byte)
{
    return __uint_as_float(byte == 255u ? 0x7FFFFFFFu : (254u - byte) << 23);
}

}  // namespace taco
