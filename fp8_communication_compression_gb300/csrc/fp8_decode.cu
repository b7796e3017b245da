// fp8_linear for one to eight tokens (serving) in one launch:
//
//   y[m][n] = sum over blocks b of 2^(ex[m][b] + ew[b][n / 128]) (Qx[m, b] . W[n, b])
//
// Bound by the weight's bytes (one per element; 16.8 MB or 2.5 us of HBM at
// 4096 x 4096) and, below some 10 MB, by latency: so one kernel, no split of
// the contraction over CTAs and no tensor memory.  A CTA of eight warps takes
// 16 rows of the weight at a time, warp w the blocks w, w + 8, ... of them; a
// lane loads 16 bytes of two rows, which are the operands of warp-level
// E4M3 MMAs (16 rows x 8 tokens x 32 values) as they lie in memory, since the
// contraction's order inside a block is free.  One token, 4096 x 4096: 5.5 us
// of device time among others of its kind.  (Decoding the codes in
// registers and multiplying them one by one took 17.8 us at 16384 x 4096 for
// one token and 44 for four, bound by instructions.)  A block's four MMAs
// start from zero; its sum is scaled and added in fp32, and the warps' sums
// meet in shared memory in a fixed order.
//
// Every CTA quantises the tokens for itself, to the same codes as
// fp8_quantize, while its first weight loads are in flight; it then walks
// over its share of the rows, each register of weights reloaded as soon as it
// is used, so that loads are in flight throughout.

#include "device_utils.cuh"
#include "fp8_block.cuh"
#include "internal.h"

namespace taco {

namespace {

constexpr int kDThreads = 256, kDWarps = kDThreads / 32;
constexpr int kTokens = 8;
constexpr int kUnits = 4;  // 8-value units of the tokens a thread loads together
constexpr int kAhead = 4;  // blocks whose loads are issued together

// Scale factor 2^(byte - 127) as two factors of half the exponent (byte 255:
// NaN).  A block's sum is multiplied by the product of the first halves of its
// two scales and then by that of the second ones: 2^(ex + ew) itself may lie
// outside fp32 where the scaled sum does not.  The halves' products lie inside,
// and the first multiplication leaves the range only where the result does.
__device__ __forceinline__ float2 scale_halves(uint32_t byte)
{
    const int e = static_cast<int>(byte) - 127, lo = e >> 1;
    const float nan = __uint_as_float(0x7FFFFFFFu);
    return byte == 255u ? make_float2(nan, nan)
                        : make_float2(__int_as_float((lo + 127) << 23), __int_as_float((e - lo + 127) << 23));
}

// c += A B for 16 rows, 8 tokens and 32 values.
__device__ __forceinline__ void mma_e4m3(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1)
{
    asm volatile("mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                 "{%0, %1, %2, %3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Shared memory: the tokens' codes [M][stride] (stride = blocks * 128 + 64
// bytes, so that a warp's 16-byte reads of eight tokens spread over the
// banks), their scale factors' halves [blocks][8], and the warps' sums.
__global__ void __launch_bounds__(kDThreads)
    fp8_decode_kernel(const uint16_t *__restrict__ x, const uint8_t *__restrict__ codes,
                      const uint8_t *__restrict__ scale, int M, int64_t N, int K, int P, void *__restrict__ y,
                      int y_bf16)
{
    extern __shared__ uint8_t smem[];
    __shared__ float part[2][kDWarps][16 * kTokens];
    const int KB = (K + 127) / 128, stride = KB * 128 + 64;
    float2 *xscale = reinterpret_cast<float2 *>(smem + M * stride);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int g = lane >> 2, t = lane & 3;  // this lane's rows g, g + 8 (and token g), and its 16 bytes of every 64
    const int64_t row_tiles = (N + 127) / 128, groups = (N + 15) / 16;
    pdl_wait();

    // block b of rows g (i = 0, 1: bytes 0-63, 64-127) and g + 8 (i = 2, 3)
    auto load = [&](int64_t grp, int b, int i) {
        const int64_t n = grp * 16 + g + 8 * (i >> 1);
        const int c = 128 * b + 64 * (i & 1) + 16 * t;
        return grp < groups && n < N && c < P ? ldg128_stream(codes + n * P + c) : make_uint4(0, 0, 0, 0);
    };
    uint4 w[kAhead][4];
#pragma unroll
    for (int u = 0; u < kAhead; ++u)
#pragma unroll
        for (int i = 0; i < 4; ++i)
            w[u][i] = load(blockIdx.x, warp + kDWarps * u, i);

    // Q(x): 8 values a thread, 16 neighbouring lanes a block (tokens that are
    // not there stay unwritten: their sums are not stored)
    const bool vec = (K & 7) == 0;
    const int units = KB * 16;
    for (int j0 = tid; j0 < M * units; j0 += kUnits * kDThreads) {
        uint4 q[kUnits];  // a batch's loads in flight together
#pragma unroll
        for (int u = 0; u < kUnits; ++u) {
            const int j = j0 + u * kDThreads, m = j / units, c = 8 * (j - m * units);
            const uint16_t *src = x + static_cast<int64_t>(m) * K + c;
            q[u] = make_uint4(0, 0, 0, 0);
            if (m < M) {
                if (vec) {
                    if (c < K)
                        q[u] = __ldg(reinterpret_cast<const uint4 *>(src));
                } else {
                    uint32_t e[8];
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        e[k] = c + k < K ? __ldg(src + k) : 0u;
                    q[u] = make_uint4(e[0] | e[1] << 16, e[2] | e[3] << 16, e[4] | e[5] << 16, e[6] | e[7] << 16);
                }
            }
        }
#pragma unroll
        for (int u = 0; u < kUnits; ++u) {
            const int j = j0 + u * kDThreads, m = j / units, c = 8 * (j - m * units);
            constexpr uint32_t kAbs = 0x7FFF7FFFu;
            uint32_t mx = __vmaxu2(__vmaxu2(q[u].x & kAbs, q[u].y & kAbs), __vmaxu2(q[u].z & kAbs, q[u].w & kAbs));
            const uint32_t half = 0xFFFFu << (lane & 16);
#pragma unroll
            for (int k = 1; k < 16; k <<= 1)
                mx = __vmaxu2(mx, __shfl_xor_sync(half, mx, k));
            mx = max(mx << 16, mx & 0xFFFF0000u);
            const uint32_t byte = fp8_scale_byte(mx);
            const float f = fp8_inv_scale(byte);
            if (m < M) {
                *reinterpret_cast<uint2 *>(smem + m * stride + c) = make_uint2(
                    f32x4_to_e4m3x4(bf16lo_to_f32(q[u].x) * f, bf16hi_to_f32(q[u].x) * f, bf16lo_to_f32(q[u].y) * f,
                                    bf16hi_to_f32(q[u].y) * f),
                    f32x4_to_e4m3x4(bf16lo_to_f32(q[u].z) * f, bf16hi_to_f32(q[u].z) * f, bf16lo_to_f32(q[u].w) * f,
                                    bf16hi_to_f32(q[u].w) * f));
                if ((c & 127) == 0)
                    xscale[(c >> 7) * kTokens + m] = scale_halves(byte);
            }
        }
    }
    __syncthreads();

    int buf = 0;
    for (int64_t grp = blockIdx.x; grp < groups; grp += gridDim.x, buf ^= 1) {
        float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        const int64_t tile = grp >> 3;  // 16 rows lie in one row tile
        for (int b0 = warp; b0 < KB; b0 += kDWarps * kAhead) {
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                const int b = b0 + kDWarps * u;
                if (b < KB) {
                    const float2 f = scale_halves(__ldg(scale + b * row_tiles + tile));
                    float c[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        uint4 xb = make_uint4(0, 0, 0, 0);
                        if (g < M)
                            xb = *reinterpret_cast<const uint4 *>(smem + g * stride + 128 * b + 64 * i + 16 * t);
                        const uint4 lo = w[u][i], hi = w[u][2 + i];
                        mma_e4m3(c, lo.x, hi.x, lo.y, hi.y, xb.x, xb.y);
                        mma_e4m3(c, lo.z, hi.z, lo.w, hi.w, xb.z, xb.w);
                    }
                    const float4 s = *reinterpret_cast<const float4 *>(xscale + b * kTokens + 2 * t);
                    acc[0] = fmaf(c[0] * (f.x * s.x), f.y * s.y, acc[0]);
                    acc[1] = fmaf(c[1] * (f.x * s.z), f.y * s.w, acc[1]);
                    acc[2] = fmaf(c[2] * (f.x * s.x), f.y * s.y, acc[2]);
                    acc[3] = fmaf(c[3] * (f.x * s.z), f.y * s.w, acc[3]);
                    // the block this register holds next, of these rows or
                    // of the CTA's next ones
                    const bool more = b + kDWarps * kAhead < KB;
                    const int64_t ng = more ? grp : grp + gridDim.x;
                    const int nb = more ? b + kDWarps * kAhead : warp + kDWarps * u;
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        w[u][i] = load(ng, nb, i);
                }
            }
        }
        // sums of tokens 2 t, 2 t + 1 for rows g, g + 8: [token][row]
        float *p = part[buf][warp];
        p[16 * (2 * t) + g] = acc[0];
        p[16 * (2 * t + 1) + g] = acc[1];
        p[16 * (2 * t) + g + 8] = acc[2];
        p[16 * (2 * t + 1) + g + 8] = acc[3];
        __syncthreads();
        const int m = tid >> 4;
        const int64_t n = grp * 16 + (tid & 15);
        if (m < M && n < N) {
            float v = 0.0f;
#pragma unroll
            for (int k = 0; k < kDWarps; ++k)
                v += part[buf][k][tid];
            const int64_t at = static_cast<int64_t>(m) * N + n;
            if (y_bf16)
                static_cast<uint16_t *>(y)[at] = static_cast<uint16_t>(f32x2_to_bf16x2(v, 0.0f));
            else
                static_cast<float *>(y)[at] = v;
        }
    }
}

constexpr int64_t kMaxK = 16384;

uint32_t decode_smem(int64_t M, int64_t K)
{
    const uint32_t KB = static_cast<uint32_t>((K + 127) / 128);
    return static_cast<uint32_t>(M) * (KB * 128 + 64) + 8 * kTokens * KB;
}

}  // namespace

bool fp8_decode_takes(int64_t M, int64_t K) { return M <= kTokens && K <= kMaxK; }

cudaError_t launch_fp8_decode(const void *x_bf16, const uint8_t *codes, const uint8_t *scale, int64_t M, int64_t N,
                              int64_t K, void *y, bool y_bf16, cudaStream_t stream)
{
    DeviceInfo di;
    cudaError_t e = current_device_info(&di);
    if (e != cudaSuccess)
        return e;
    static std::atomic<bool> set[kMaxDevices];
    if ((e = ensure_smem(fp8_decode_kernel, decode_smem(kTokens, kMaxK), di.device, set)) != cudaSuccess)
        return e;
    const uint32_t smem = decode_smem(M, K);
    const int64_t groups = (N + 15) / 16, most = (smem <= 100 * 1024 ? 2 : 1) * static_cast<int64_t>(di.num_sms);
    return launch_pdl(fp8_decode_kernel, dim3(static_cast<unsigned>(groups < most ? groups : most)), dim3(kDThreads),
                      smem, stream, static_cast<const uint16_t *>(x_bf16), codes, scale, static_cast<int>(M), N,
                      static_cast<int>(K), static_cast<int>(fp8_pitch(K)), y, static_cast<int>(y_bf16));
}

}  // namespace taco
