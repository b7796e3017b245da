// fp8_linear for one to four tokens (single-token serving) in one launch:
//
//   y[m][n] = sum over blocks b of 2^(ew[b][n / 128]) (Q(x)[m, b] . W[n, b])
//
// Bound by the weight's bytes (one per element; 16.8 MB or 2.5 us of HBM at
// 4096 x 4096) and, below some 10 MB, by latency: so no tensor cores, no
// second kernel for x and no split.  Every CTA quantises x for itself (the
// same values as fp8_quantize: the maximum over 16 lanes of 8 values each,
// then the E4M3 conversion) into shared memory as bf16, which holds a code
// times its scale exactly, while its first weight loads are in flight.  A
// warp takes R rows of the weight and 512 values of them at a time, 16 a
// lane, so that a lane's 16 bytes lie in one block; products are exact in
// fp32 and summed there.

#include <atomic>

#include "device_utils.cuh"
#include "fp8_block.cuh"
#include "internal.h"

namespace taco {

namespace {

constexpr int kDThreads = 256;
constexpr int kAhead = 4;  // steps of 512 values whose loads are issued together

// Scale factor 2^(byte - 127); byte 0 is a subnormal, 255 the NaN scale.
__device__ __forceinline__ float scale_factor(uint32_t byte)
{
    return __uint_as_float(byte == 255u ? 0x7FFFFFFFu : byte == 0u ? 0x00400000u : byte << 23);
}

// MT tokens (the last ones absent where M < MT), R weight rows a warp.
template <int MT, int R>
__global__ void __launch_bounds__(kDThreads)
    fp8_decode_kernel(const uint16_t *__restrict__ x, const uint8_t *__restrict__ codes,
                      const uint8_t *__restrict__ scale, int M, int64_t N, int K, int P, void *__restrict__ y,
                      int y_bf16)
{
    extern __shared__ uint4 xs[];  // [MT][ceil(K / 512) * 512] bf16 values of Q(x)
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int steps = (K + 511) / 512;
    const int64_t n0 = (static_cast<int64_t>(blockIdx.x) * (kDThreads / 32) + warp) * R;
    const int64_t row_tiles = (N + 127) / 128;
    pdl_wait();

    // 16 codes of row n0 + i at step s
    auto load = [&](int s, int i) {
        const int c = 512 * s + 16 * lane;
        return c < P && n0 + i < N ? ldg128_stream(codes + (n0 + i) * P + c) : make_uint4(0, 0, 0, 0);
    };
    uint4 w[kAhead][R];
#pragma unroll
    for (int u = 0; u < kAhead; ++u)
#pragma unroll
        for (int i = 0; i < R; ++i)
            w[u][i] = load(u, i);

    // Q(x): 8 values a thread, 16 neighbouring lanes a block
    const int units = steps * 64;  // 8-value units of a token, in whole warps
    const bool vec = (K & 7) == 0;
#pragma unroll
    for (int m = 0; m < MT; ++m) {
        for (int j = tid; j < units; j += kDThreads) {
            const int c = 8 * j;
            uint4 q = make_uint4(0, 0, 0, 0);
            if (m < M) {
                const uint16_t *src = x + static_cast<int64_t>(m) * K + c;
                if (vec) {
                    if (c < K)
                        q = __ldg(reinterpret_cast<const uint4 *>(src));
                } else {
                    uint32_t e[8];
#pragma unroll
                    for (int t = 0; t < 8; ++t)
                        e[t] = c + t < K ? __ldg(src + t) : 0u;
                    q = make_uint4(e[0] | e[1] << 16, e[2] | e[3] << 16, e[4] | e[5] << 16, e[6] | e[7] << 16);
                }
            }
            constexpr uint32_t kAbs = 0x7FFF7FFFu;
            uint32_t mx = __vmaxu2(__vmaxu2(q.x & kAbs, q.y & kAbs), __vmaxu2(q.z & kAbs, q.w & kAbs));
#pragma unroll
            for (int k = 1; k < 16; k <<= 1)
                mx = __vmaxu2(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, k));
            mx = max(mx << 16, mx & 0xFFFF0000u);
            const uint32_t byte = fp8_scale_byte(mx);
            const float f = fp8_inv_scale(byte), g = scale_factor(byte);
            uint32_t v[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                float lo, hi;
                e4m3x2_to_f32x2(f32x2_to_e4m3x2(bf16lo_to_f32(v[t]) * f, bf16hi_to_f32(v[t]) * f), lo, hi);
                v[t] = f32x2_to_bf16x2(lo * g, hi * g);
            }
            xs[m * units + j] = make_uint4(v[0], v[1], v[2], v[3]);
        }
    }
    __syncthreads();

    float acc[MT][R] = {};
    const int64_t tile = n0 >> 7;  // R divides 128: one row tile a warp
    for (int s0 = 0; s0 < steps; s0 += kAhead) {
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            const int s = s0 + u;
            if (s < steps) {
                const int b = 4 * s + (lane >> 3);  // this lane's block
                const float f = 128 * b < K && n0 < N ? scale_factor(__ldg(scale + b * row_tiles + tile)) : 0.0f;
                float xv[MT][16];
#pragma unroll
                for (int m = 0; m < MT; ++m) {
                    const uint4 a = xs[m * units + 64 * s + 2 * lane], c = xs[m * units + 64 * s + 2 * lane + 1];
                    const uint32_t t[8] = {a.x, a.y, a.z, a.w, c.x, c.y, c.z, c.w};
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        xv[m][2 * k] = bf16lo_to_f32(t[k]);
                        xv[m][2 * k + 1] = bf16hi_to_f32(t[k]);
                    }
                }
#pragma unroll
                for (int i = 0; i < R; ++i) {
                    const uint32_t t[4] = {w[u][i].x, w[u][i].y, w[u][i].z, w[u][i].w};
                    float dot[MT] = {};
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        float e0, e1, e2, e3;
                        e4m3x2_to_f32x2(t[k], e0, e1);
                        e4m3x2_to_f32x2(t[k] >> 16, e2, e3);
#pragma unroll
                        for (int m = 0; m < MT; ++m) {
                            dot[m] = fmaf(e0, xv[m][4 * k], dot[m]);
                            dot[m] = fmaf(e1, xv[m][4 * k + 1], dot[m]);
                            dot[m] = fmaf(e2, xv[m][4 * k + 2], dot[m]);
                            dot[m] = fmaf(e3, xv[m][4 * k + 3], dot[m]);
                        }
                    }
#pragma unroll
                    for (int m = 0; m < MT; ++m)
                        acc[m][i] = fmaf(f, dot[m], acc[m][i]);
                    w[u][i] = load(s + kAhead, i);
                }
            }
        }
    }
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int i = 0; i < R; ++i) {
#pragma unroll
            for (int k = 16; k >= 1; k >>= 1)
                acc[m][i] += __shfl_xor_sync(0xFFFFFFFFu, acc[m][i], k);
            if (lane == 0 && m < M && n0 + i < N) {
                const int64_t at = static_cast<int64_t>(m) * N + n0 + i;
                if (y_bf16)
                    static_cast<uint16_t *>(y)[at] = static_cast<uint16_t>(f32x2_to_bf16x2(acc[m][i], 0.0f));
                else
                    static_cast<float *>(y)[at] = acc[m][i];
            }
        }
}

constexpr int kMaxDevices = 64;
constexpr uint32_t kDecodeSmem = 128 * 1024;

uint32_t x_bytes(int mt, int64_t K) { return static_cast<uint32_t>(2 * mt * ((K + 511) / 512) * 512); }

template <int MT, int R>
cudaError_t run_decode(const void *x, const uint8_t *codes, const uint8_t *scale, int64_t M, int64_t N, int64_t K,
                       void *y, bool y_bf16, int device, cudaStream_t stream)
{
    static std::atomic<bool> set[kMaxDevices];
    if (!set[device].load(std::memory_order_acquire)) {
        cudaError_t e = cudaFuncSetAttribute(fp8_decode_kernel<MT, R>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             static_cast<int>(kDecodeSmem));
        if (e != cudaSuccess)
            return e;
        set[device].store(true, std::memory_order_release);
    }
    const int64_t per = (kDThreads / 32) * R;
    return launch_pdl(fp8_decode_kernel<MT, R>, dim3(static_cast<unsigned>((N + per - 1) / per)), dim3(kDThreads),
                      x_bytes(MT, K), stream, static_cast<const uint16_t *>(x), codes, scale, static_cast<int>(M), N,
                      static_cast<int>(K), static_cast<int>(fp8_pitch(K)), y, static_cast<int>(y_bf16));
}

template <int MT>
cudaError_t decode_rows(const void *x, const uint8_t *codes, const uint8_t *scale, int64_t M, int64_t N, int64_t K,
                        void *y, bool y_bf16, const DeviceInfo &di, cudaStream_t stream)
{
    // four rows a warp once that gives two CTAs an SM, else two, else one
    const int64_t warps = 2 * di.num_sms * (kDThreads / 32);
    if (N >= 4 * warps)
        return run_decode<MT, 4>(x, codes, scale, M, N, K, y, y_bf16, di.device, stream);
    if (N >= warps)
        return run_decode<MT, 2>(x, codes, scale, M, N, K, y, y_bf16, di.device, stream);
    return run_decode<MT, 1>(x, codes, scale, M, N, K, y, y_bf16, di.device, stream);
}

}  // namespace

bool fp8_decode_takes(int64_t M, int64_t K)
{
    return M <= 4 && K <= 16384 && x_bytes(M > 2 ? 4 : static_cast<int>(M), K) <= kDecodeSmem;
}

cudaError_t launch_fp8_decode(const void *x_bf16, const uint8_t *codes, const uint8_t *scale, int64_t M, int64_t N,
                              int64_t K, void *y, bool y_bf16, cudaStream_t stream)
{
    DeviceInfo di;
    cudaError_t e = current_device_info(&di);
    if (e != cudaSuccess)
        return e;
    if (M == 1)
        return decode_rows<1>(x_bf16, codes, scale, M, N, K, y, y_bf16, di, stream);
    if (M == 2)
        return decode_rows<2>(x_bf16, codes, scale, M, N, K, y, y_bf16, di, stream);
    return decode_rows<4>(x_bf16, codes, scale, M, N, K, y, y_bf16, di, stream);
}

}  // namespace taco
