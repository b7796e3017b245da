// C ABI of the library (include/taco.h): argument validation on the host,
// then one kernel launch on the caller's stream.  No allocation, no
// synchronisation, no exception crosses this boundary.  The host pipeline
// calls are the exception their declarations state: a pipeline owns CUDA
// streams and events, and one run enqueues copies and launches per chunk.

#include <cfloat>
#include <cmath>
#include <cstdint>
#include <mutex>
#include <new>

#include "../../include/taco.h"
#include "fp8_block.cuh"
#include "internal.h"

namespace taco {

cudaError_t current_device_info(DeviceInfo *out)
{
    constexpr int kMax = 64;
    static DeviceInfo cache[kMax];
    static bool ready[kMax];
    static std::mutex mu;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess)
        return e;
    if (dev < 0 || dev >= kMax)
        return cudaErrorInvalidDevice;
    std::lock_guard<std::mutex> lock(mu);
    if (!ready[dev]) {
        DeviceInfo di{dev, 0, 0};
        if ((e = cudaDeviceGetAttribute(&di.num_sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess)
            return e;
        if ((e = cudaDeviceGetAttribute(&di.max_smem_optin, cudaDevAttrMaxSharedMemoryPerBlockOptin, dev)) !=
            cudaSuccess)
            return e;
        cache[dev] = di;
        ready[dev] = true;
    }
    *out = cache[dev];
    return cudaSuccess;
}

}  // namespace taco

namespace {

bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// [a, a + na) and [b, b + nb) overlap
bool overlap(const void *a, uint64_t na, const void *b, uint64_t nb)
{
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return na && nb && x < y + nb && y < x + na;
}

bool positive_finite(float v) { return std::isfinite(v) && v > 0.0f; }

taco_status from_cuda(cudaError_t e) { return e == cudaSuccess ? TACO_OK : TACO_ERR_CUDA; }

// The 128-element row view used by the TMA kernels must fit int32 tile
// coordinates.
constexpr int64_t kMaxRows128 = (int64_t(1) << 31) - 256;

taco_status check_taco_shape(int64_t rows, int64_t d, int32_t block)
{
    if (rows < 0 || d <= 0)
        return TACO_ERR_INVALID_ARG;
    if (!taco_block_supported(block))
        return TACO_ERR_UNSUPPORTED;
    if (d % block != 0)
        return TACO_ERR_INVALID_ARG;
    if (rows > 0 && d > INT64_MAX / rows)
        return TACO_ERR_INVALID_ARG;
    if (rows * d / 128 > kMaxRows128)
        return TACO_ERR_UNSUPPORTED;
    return TACO_OK;
}


// Shared checks of the two reduce entry points; fills `sp`.  `out` (the
// optional reconstruction of the sum) may be null.
taco_status check_reduce_args(int32_t P, const uint8_t *const *codes, const float *const *alpha,
                                     const float *const *scale, int64_t rows, int64_t d, int32_t block,
                                     float e_target, float eps, const uint8_t *out_codes,
                                     const float *out_alpha, const float *out_scale, const void *out,
                                     uint64_t out_bytes_per_elem, taco::ShardPtrs *sp)
{
    taco_status st = check_taco_shape(rows, d, block);
    if (st != TACO_OK)
        return st;
    if (P < 1 || P > TACO_MAX_SHARDS)
        return TACO_ERR_UNSUPPORTED;
    if (!positive_finite(e_target) || !positive_finite(eps))
        return TACO_ERR_INVALID_ARG;
    if (rows == 0)
        return TACO_OK;
    if (!codes || !alpha || !scale || !out_codes || !out_alpha || !out_scale)
        return TACO_ERR_INVALID_ARG;
    const uint64_t n = static_cast<uint64_t>(rows * d), nb = n / block;
    if (!aligned(out_codes, 16) || !aligned(out_alpha, 4) || !aligned(out_scale, 4) ||
        (out && !aligned(out, 16)))
        return TACO_ERR_MISALIGNED;
    const void *outs[4] = {out_codes, out_alpha, out_scale, out};
    const uint64_t olen[4] = {n, 4 * nb, 4 * nb, out ? n * out_bytes_per_elem : 0};
    for (int i = 0; i < 4; ++i)
        for (int j = i + 1; j < 4; ++j)
            if (overlap(outs[i], olen[i], outs[j], olen[j]))
                return TACO_ERR_INVALID_ARG;
    for (int p = 0; p < P; ++p) {
        if (!codes[p] || !alpha[p] || !scale[p])
            return TACO_ERR_INVALID_ARG;
        if (!aligned(codes[p], 16) || !aligned(alpha[p], 4) || !aligned(scale[p], 4))
            return TACO_ERR_MISALIGNED;
        const void *ins[3] = {codes[p], alpha[p], scale[p]};
        const uint64_t lens[3] = {n, 4 * nb, 4 * nb};
        for (int i = 0; i < 3; ++i)
            for (int j = 0; j < 4; ++j)
                if (overlap(ins[i], lens[i], outs[j], olen[j]))
                    return TACO_ERR_INVALID_ARG;
        sp->codes[p] = codes[p];
        sp->alpha[p] = alpha[p];
        sp->scale[p] = scale[p];
    }
    return TACO_OK;
}

}  // namespace

extern "C" {

const char *taco_status_string(taco_status s)
{
    switch (s) {
    case TACO_OK:
        return "ok";
    case TACO_ERR_INVALID_ARG:
        return "invalid argument";
    case TACO_ERR_UNSUPPORTED:
        return "unsupported block size, shard count or size";
    case TACO_ERR_MISALIGNED:
        return "misaligned pointer";
    case TACO_ERR_CUDA:
        return "CUDA error";
    }
    return "unknown status";
}

int taco_abi_version(void) { return TACO_ABI_VERSION; }

int taco_block_supported(int32_t block) { return block == 128 || block == 256; }

static taco_status compress_any(const void *x_bf16, int64_t rows, int64_t d, int32_t block, float e_target,
                                float eps, uint8_t *codes, float *alpha, float *scale, bool int8_codes,
                                taco_stream_t stream)
{
    taco_status st = check_taco_shape(rows, d, block);
    if (st != TACO_OK)
        return st;
    if (!positive_finite(e_target) || !positive_finite(eps))
        return TACO_ERR_INVALID_ARG;
    if (rows == 0)
        return TACO_OK;
    if (!x_bf16 || !codes || !alpha || !scale)
        return TACO_ERR_INVALID_ARG;
    if (!aligned(x_bf16, 16) || !aligned(codes, 16) || !aligned(alpha, 4) || !aligned(scale, 4))
        return TACO_ERR_MISALIGNED;
    const uint64_t n = static_cast<uint64_t>(rows * d), nb = n / block;
    if (overlap(x_bf16, 2 * n, codes, n) || overlap(x_bf16, 2 * n, alpha, 4 * nb) ||
        overlap(x_bf16, 2 * n, scale, 4 * nb) || overlap(codes, n, alpha, 4 * nb) ||
        overlap(codes, n, scale, 4 * nb) || overlap(alpha, 4 * nb, scale, 4 * nb))
        return TACO_ERR_INVALID_ARG;
    return from_cuda(taco::launch_compress(x_bf16, rows * d / 128, block, e_target, eps, codes, alpha,
                                           scale, int8_codes, reinterpret_cast<cudaStream_t>(stream)));
}

taco_status taco_compress(const void *x_bf16, int64_t rows, int64_t d, int32_t block, float e_target,
                          float eps, uint8_t *codes, float *alpha, float *scale, taco_stream_t stream)
{
    return compress_any(x_bf16, rows, d, block, e_target, eps, codes, alpha, scale, false, stream);
}

taco_status taco_compress_int8(const void *x_bf16, int64_t rows, int64_t d, int32_t block, float e_target,
                               float eps, int8_t *codes, float *alpha, float *scale, taco_stream_t stream)
{
    return compress_any(x_bf16, rows, d, block, e_target, eps, reinterpret_cast<uint8_t *>(codes), alpha,
                        scale, true, stream);
}

static taco_status decompress_any(const uint8_t *codes, const float *alpha, const float *scale, int64_t rows,
                                  int64_t d, int32_t block, void *out, int32_t out_is_bf16, bool int8_codes,
                                  taco_stream_t stream)
{
    taco_status st = check_taco_shape(rows, d, block);
    if (st != TACO_OK)
        return st;
    if (rows == 0)
        return TACO_OK;
    if (!codes || !alpha || !scale || !out)
        return TACO_ERR_INVALID_ARG;
    if (!aligned(codes, 16) || !aligned(out, 16) || !aligned(alpha, 4) || !aligned(scale, 4))
        return TACO_ERR_MISALIGNED;
    const uint64_t n = static_cast<uint64_t>(rows * d), nb = n / block;
    const uint64_t out_bytes = n * (out_is_bf16 ? 2 : 4);
    if (overlap(out, out_bytes, codes, n) || overlap(out, out_bytes, alpha, 4 * nb) ||
        overlap(out, out_bytes, scale, 4 * nb))
        return TACO_ERR_INVALID_ARG;
    return from_cuda(taco::launch_decompress(codes, alpha, scale, rows * d / 128, block, out,
                                             out_is_bf16 != 0, int8_codes,
                                             reinterpret_cast<cudaStream_t>(stream)));
}

taco_status taco_decompress(const uint8_t *codes, const float *alpha, const float *scale, int64_t rows,
                            int64_t d, int32_t block, void *out, int32_t out_is_bf16,
                            taco_stream_t stream)
{
    return decompress_any(codes, alpha, scale, rows, d, block, out, out_is_bf16, false, stream);
}

taco_status taco_decompress_int8(const int8_t *codes, const float *alpha, const float *scale, int64_t rows,
                                 int64_t d, int32_t block, void *out, int32_t out_is_bf16,
                                 taco_stream_t stream)
{
    return decompress_any(reinterpret_cast<const uint8_t *>(codes), alpha, scale, rows, d, block, out,
                          out_is_bf16, true, stream);
}

taco_status taco_reduce_shards(int32_t P, const uint8_t *const *codes, const float *const *alpha,
                               const float *const *scale, int64_t rows, int64_t d, int32_t block,
                               float e_target, float eps, uint8_t *out_codes, float *out_alpha,
                               float *out_scale, taco_stream_t stream)
{
    taco::ShardPtrs sp{};
    taco_status st = check_reduce_args(P, codes, alpha, scale, rows, d, block, e_target, eps, out_codes,
                                       out_alpha, out_scale, nullptr, 0, &sp);
    if (st != TACO_OK || rows == 0)
        return st;
    return from_cuda(taco::launch_taco_reduce(P, sp, rows * d / block, block, e_target, eps, out_codes,
                                              out_alpha, out_scale, reinterpret_cast<cudaStream_t>(stream)));
}

taco_status taco_reduce_decompress(int32_t P, const uint8_t *const *codes, const float *const *alpha,
                                   const float *const *scale, int64_t rows, int64_t d, int32_t block,
                                   float e_target, float eps, uint8_t *out_codes, float *out_alpha,
                                   float *out_scale, void *out, int32_t out_is_bf16, taco_stream_t stream)
{
    taco::ShardPtrs sp{};
    if (rows > 0 && !out)
        return TACO_ERR_INVALID_ARG;
    taco_status st = check_reduce_args(P, codes, alpha, scale, rows, d, block, e_target, eps, out_codes,
                                       out_alpha, out_scale, out, out_is_bf16 ? 2 : 4, &sp);
    if (st != TACO_OK || rows == 0)
        return st;
    return from_cuda(taco::launch_reduce_decompress(P, sp, rows * d / 128, block, e_target, eps, out_codes,
                                                    out_alpha, out_scale, out, out_is_bf16 != 0,
                                                    reinterpret_cast<cudaStream_t>(stream)));
}

taco_status agoq_fp8_accumulate(uint8_t *main_codes, float *main_scale, const void *grad_bf16, int64_t n,
                                int32_t block, taco_stream_t stream)
{
    if (n < 0)
        return TACO_ERR_INVALID_ARG;
    if (!taco_block_supported(block))
        return TACO_ERR_UNSUPPORTED;
    if (n % block != 0)
        return TACO_ERR_INVALID_ARG;
    if (n == 0)
        return TACO_OK;
    if (!main_codes || !main_scale || !grad_bf16)
        return TACO_ERR_INVALID_ARG;
    if (!aligned(main_codes, 16) || !aligned(grad_bf16, 16) || !aligned(main_scale, 4))
        return TACO_ERR_MISALIGNED;
    const uint64_t nb = static_cast<uint64_t>(n / block);
    if (overlap(main_codes, n, main_scale, 4 * nb) || overlap(grad_bf16, 2 * n, main_codes, n) ||
        overlap(grad_bf16, 2 * n, main_scale, 4 * nb))
        return TACO_ERR_INVALID_ARG;
    return from_cuda(taco::launch_agoq_accumulate(main_codes, main_scale, grad_bf16, n, block,
                                                  reinterpret_cast<cudaStream_t>(stream)));
}

taco_status agoq_reduce_shards(int32_t P, const uint8_t *const *codes, const float *const *scale, int64_t n,
                               int32_t block, uint8_t *out_codes, float *out_scale, taco_stream_t stream)
{
    if (n < 0)
        return TACO_ERR_INVALID_ARG;
    if (!taco_block_supported(block) || P < 1 || P > TACO_MAX_SHARDS)
        return TACO_ERR_UNSUPPORTED;
    if (n % block != 0)
        return TACO_ERR_INVALID_ARG;
    if (n == 0)
        return TACO_OK;
    if (!codes || !scale || !out_codes || !out_scale)
        return TACO_ERR_INVALID_ARG;
    if (!aligned(out_codes, 16) || !aligned(out_scale, 4))
        return TACO_ERR_MISALIGNED;
    const uint64_t nb = static_cast<uint64_t>(n / block);
    if (overlap(out_codes, n, out_scale, 4 * nb))
        return TACO_ERR_INVALID_ARG;
    taco::ShardPtrs sp{};
    for (int p = 0; p < P; ++p) {
        if (!codes[p] || !scale[p])
            return TACO_ERR_INVALID_ARG;
        if (!aligned(codes[p], 16) || !aligned(scale[p], 4))
            return TACO_ERR_MISALIGNED;
        if (overlap(codes[p], n, out_codes, n) || overlap(codes[p], n, out_scale, 4 * nb) ||
            overlap(scale[p], 4 * nb, out_codes, n) || overlap(scale[p], 4 * nb, out_scale, 4 * nb))
            return TACO_ERR_INVALID_ARG;
        sp.codes[p] = codes[p];
        sp.scale[p] = scale[p];
    }
    return from_cuda(taco::launch_agoq_reduce(P, sp, n, block, out_codes, out_scale,
                                              reinterpret_cast<cudaStream_t>(stream)));
}

static taco_status check_laaq(int64_t n, int32_t block, int32_t bits)
{
    if (n < 0)
        return TACO_ERR_INVALID_ARG;
    if (!(block == 32 || block == 64 || block == 128 || block == 256) ||
        !(bits == 4 || bits == 5 || bits == 6 || bits == 8))
        return TACO_ERR_UNSUPPORTED;
    if (n % block != 0)
        return TACO_ERR_INVALID_ARG;
    return TACO_OK;
}

taco_status agoq_laaq_quantize(const void *x_bf16, int64_t n, int32_t block, int32_t bits, uint8_t *packed,
                               float *scale, taco_stream_t stream)
{
    taco_status st = check_laaq(n, block, bits);
    if (st != TACO_OK || n == 0)
        return st;
    if (!x_bf16 || !packed || !scale)
        return TACO_ERR_INVALID_ARG;
    if (!aligned(x_bf16, 16) || !aligned(packed, 16) || !aligned(scale, 4))
        return TACO_ERR_MISALIGNED;
    const uint64_t nb = static_cast<uint64_t>(n / block), pb = static_cast<uint64_t>(n) * bits / 8;
    if (overlap(x_bf16, 2 * n, packed, pb) || overlap(x_bf16, 2 * n, scale, 4 * nb) ||
        overlap(packed, pb, scale, 4 * nb))
        return TACO_ERR_INVALID_ARG;
    return from_cuda(taco::launch_laaq_quantize(x_bf16, n, block, bits, packed, scale,
                                                reinterpret_cast<cudaStream_t>(stream)));
}

// Shared checks of the dequantizing entry points: the stream, its
// multipliers and an output of n fp32 or bf16 values that overlaps neither.
static taco_status check_laaq_out(const uint8_t *packed, const float *scale, int64_t n, int32_t block,
                                  int32_t bits, const void *out, int32_t out_is_bf16)
{
    if (!packed || !scale || !out)
        return TACO_ERR_INVALID_ARG;
    if (!aligned(packed, 16) || !aligned(scale, 4) || !aligned(out, 16))
        return TACO_ERR_MISALIGNED;
    const uint64_t nb = static_cast<uint64_t>(n / block), pb = static_cast<uint64_t>(n) * bits / 8;
    const uint64_t ob = static_cast<uint64_t>(n) * (out_is_bf16 ? 2 : 4);
    if (overlap(out, ob, packed, pb) || overlap(out, ob, scale, 4 * nb))
        return TACO_ERR_INVALID_ARG;
    return TACO_OK;
}

taco_status agoq_laaq_dequantize(const uint8_t *packed, const float *scale, int64_t n, int32_t block,
                                 int32_t bits, void *out, int32_t out_is_bf16, taco_stream_t stream)
{
    taco_status st = check_laaq(n, block, bits);
    if (st != TACO_OK || n == 0)
        return st;
    if ((st = check_laaq_out(packed, scale, n, block, bits, out, out_is_bf16)) != TACO_OK)
        return st;
    return from_cuda(taco::launch_laaq_dequantize(packed, scale, n, block, bits, out, out_is_bf16 != 0, false,
                                                  reinterpret_cast<cudaStream_t>(stream)));
}

taco_status agoq_laaq_dequantize_silu(const uint8_t *packed, const float *scale, int64_t n, int32_t block,
                                      int32_t bits, void *out, int32_t out_is_bf16, taco_stream_t stream)
{
    taco_status st = check_laaq(n, block, bits);
    if (st != TACO_OK || n == 0)
        return st;
    if ((st = check_laaq_out(packed, scale, n, block, bits, out, out_is_bf16)) != TACO_OK)
        return st;
    return from_cuda(taco::launch_laaq_dequantize(packed, scale, n, block, bits, out, out_is_bf16 != 0, true,
                                                  reinterpret_cast<cudaStream_t>(stream)));
}

taco_status agoq_laaq_dequantize_rmsnorm(const uint8_t *packed, const float *scale, int64_t rows, int64_t d,
                                         int32_t block, int32_t bits, const float *gamma, float eps, void *out,
                                         int32_t out_is_bf16, taco_stream_t stream)
{
    if (rows < 0 || d < 0 || !(eps >= 0.0f) || !(eps <= FLT_MAX))
        return TACO_ERR_INVALID_ARG;
    if (d > (int64_t(1) << 31) || (d > 0 && rows > INT64_MAX / 8 / d))
        return TACO_ERR_UNSUPPORTED;
    const int64_t n = rows * d;
    taco_status st = check_laaq(n, block, bits);
    if (st != TACO_OK)
        return st;
    if (rows == 0 || d == 0)
        return TACO_OK;
    if (d % block != 0)
        return TACO_ERR_INVALID_ARG;
    if ((st = check_laaq_out(packed, scale, n, block, bits, out, out_is_bf16)) != TACO_OK)
        return st;
    if (!gamma)
        return TACO_ERR_INVALID_ARG;
    if (!aligned(gamma, 16))
        return TACO_ERR_MISALIGNED;
    if (overlap(out, static_cast<uint64_t>(n) * (out_is_bf16 ? 2 : 4), gamma, 4 * static_cast<uint64_t>(d)))
        return TACO_ERR_INVALID_ARG;
    return from_cuda(taco::launch_laaq_rmsnorm(packed, scale, rows, d, block, bits, gamma, eps, out, out_is_bf16 != 0,
                                               reinterpret_cast<cudaStream_t>(stream)));
}

// The GEMM shapes the tensor-core kernel takes (M, N > 0).
static bool gemm_shape_supported(int64_t M, int64_t N, int64_t K)
{
    return K > 0 && M % 128 == 0 && N % 128 == 0 && K % 64 == 0 && M / 128 <= 65535 && N <= (int64_t(1) << 30) &&
           K <= (int64_t(1) << 30) && (M / 128) * (N / 128) <= (int64_t(1) << 30);
}

// Shared checks of the GEMM entry points.  codes hold code_bits bits per
// element of Y; alpha may be null (only the compressor has one); y_out may
// be null; a null workspace or one of 0 bytes is none.
static taco_status check_gemm_args(const void *a_bf16, const void *b_bf16, int64_t M, int64_t N, int64_t K,
                                   int32_t block, const uint8_t *codes, int code_bits, const float *alpha,
                                   bool need_alpha, const float *scale, const float *y_out, const void *workspace,
                                   uint64_t workspace_bytes)
{
    if (M < 0 || N < 0 || K < 0)
        return TACO_ERR_INVALID_ARG;
    if (block != 128)
        return TACO_ERR_UNSUPPORTED;
    if (M == 0 || N == 0)
        return TACO_OK;
    if (!gemm_shape_supported(M, N, K))
        return TACO_ERR_UNSUPPORTED;
    if (!a_bf16 || !b_bf16 || !codes || (need_alpha && !alpha) || !scale)
        return TACO_ERR_INVALID_ARG;
    const bool ws = workspace && workspace_bytes > 0;
    if (!aligned(a_bf16, 16) || !aligned(b_bf16, 16) || !aligned(codes, 16) || (alpha && !aligned(alpha, 4)) ||
        !aligned(scale, 4) || (y_out && !aligned(y_out, 16)) || (ws && !aligned(workspace, 256)))
        return TACO_ERR_MISALIGNED;
    const uint64_t mn = static_cast<uint64_t>(M) * N, nb = mn / 128;
    const void *outs[5] = {codes, alpha, scale, y_out, ws ? workspace : nullptr};
    const uint64_t olen[5] = {mn * code_bits / 8, alpha ? 4 * nb : 0, 4 * nb, y_out ? 4 * mn : 0,
                              ws ? workspace_bytes : 0};
    const void *ins[2] = {a_bf16, b_bf16};
    const uint64_t ilen[2] = {2 * static_cast<uint64_t>(M) * K, 2 * static_cast<uint64_t>(N) * K};
    for (int i = 0; i < 5; ++i) {
        for (int j = i + 1; j < 5; ++j)
            if (overlap(outs[i], olen[i], outs[j], olen[j]))
                return TACO_ERR_INVALID_ARG;
        for (int j = 0; j < 2; ++j)
            if (overlap(outs[i], olen[i], ins[j], ilen[j]))
                return TACO_ERR_INVALID_ARG;
    }
    return TACO_OK;
}

taco_status taco_gemm_workspace_bytes(int64_t M, int64_t N, int64_t K, uint64_t *bytes)
{
    if (!bytes || M < 0 || N < 0 || K < 0)
        return TACO_ERR_INVALID_ARG;
    *bytes = 0;
    if (M == 0 || N == 0)
        return TACO_OK;
    if (!gemm_shape_supported(M, N, K))
        return TACO_ERR_UNSUPPORTED;
    return from_cuda(taco::gemm_workspace_bytes(M, N, K, bytes));
}

taco_status taco_gemm_compress(const void *a_bf16, const void *b_bf16, int64_t M, int64_t N, int64_t K,
                               int32_t block, float e_target, float eps, uint8_t *codes, float *alpha,
                               float *scale, float *y_out, void *workspace, uint64_t workspace_bytes,
                               taco_stream_t stream)
{
    if (!positive_finite(e_target) || !positive_finite(eps))
        return TACO_ERR_INVALID_ARG;
    taco_status st = check_gemm_args(a_bf16, b_bf16, M, N, K, block, codes, 8, alpha, true, scale, y_out,
                                     workspace, workspace_bytes);
    if (st != TACO_OK || M == 0 || N == 0)
        return st;
    return from_cuda(taco::launch_gemm_compress(a_bf16, b_bf16, M, N, K, e_target, eps, codes, alpha, scale, y_out,
                                                workspace, workspace_bytes, reinterpret_cast<cudaStream_t>(stream)));
}

taco_status agoq_gemm_accumulate(const void *a_bf16, const void *b_bf16, int64_t M, int64_t N, int64_t K,
                                 int32_t block, uint8_t *main_codes, float *main_scale, float *y_out,
                                 void *workspace, uint64_t workspace_bytes, taco_stream_t stream)
{
    taco_status st = check_gemm_args(a_bf16, b_bf16, M, N, K, block, main_codes, 8, nullptr, false, main_scale,
                                     y_out, workspace, workspace_bytes);
    if (st != TACO_OK || M == 0 || N == 0)
        return st;
    return from_cuda(taco::launch_gemm_agoq_accumulate(a_bf16, b_bf16, M, N, K, main_codes, main_scale, y_out,
                                                       workspace, workspace_bytes,
                                                       reinterpret_cast<cudaStream_t>(stream)));
}

taco_status agoq_gemm_laaq_quantize(const void *a_bf16, const void *b_bf16, int64_t M, int64_t N, int64_t K,
                                    int32_t block, int32_t bits, uint8_t *packed, float *scale, float *y_out,
                                    void *workspace, uint64_t workspace_bytes, taco_stream_t stream)
{
    if (bits != 4 && bits != 5 && bits != 6 && bits != 8)
        return TACO_ERR_UNSUPPORTED;
    taco_status st = check_gemm_args(a_bf16, b_bf16, M, N, K, block, packed, bits, nullptr, false, scale, y_out,
                                     workspace, workspace_bytes);
    if (st != TACO_OK || M == 0 || N == 0)
        return st;
    return from_cuda(taco::launch_gemm_laaq_quantize(a_bf16, b_bf16, M, N, K, bits, packed, scale, y_out, workspace,
                                                     workspace_bytes, reinterpret_cast<cudaStream_t>(stream)));
}

taco_status taco_e4m3_encode(const float *x, int64_t n, uint8_t *codes, taco_stream_t stream)
{
    if (n < 0)
        return TACO_ERR_INVALID_ARG;
    if (n == 0)
        return TACO_OK;
    if (!x || !codes)
        return TACO_ERR_INVALID_ARG;
    if (!aligned(x, 16) || !aligned(codes, 16))
        return TACO_ERR_MISALIGNED;
    if (overlap(x, 4 * static_cast<uint64_t>(n), codes, static_cast<uint64_t>(n)))
        return TACO_ERR_INVALID_ARG;
    return from_cuda(taco::launch_e4m3_encode(x, n, codes, reinterpret_cast<cudaStream_t>(stream)));
}

int64_t fp8_pitch(int64_t cols) { return taco::fp8_pitch(cols); }
int64_t fp8_scale_bytes(int64_t rows, int64_t cols) { return taco::fp8_scale_bytes(rows, cols); }

// Sizes whose tile grids and TMA coordinates fit the kernels' 32-bit indices.
static bool fp8_dims_fit(int64_t rows, int64_t cols)
{
    constexpr int64_t kMax = int64_t(1) << 30;
    return rows <= kMax && cols <= kMax && ((rows + 127) / 128) * ((cols + 127) / 128) <= kMax;
}

static int64_t fp8_blocks(int64_t n) { return (n + 127) / 128; }

// A buffer of a call: no output may overlap an input or another output.
struct Span {
    const void *p;
    uint64_t n;
};

static bool apart(const Span *outs, int n_outs, const Span *ins, int n_ins)
{
    for (int i = 0; i < n_outs; ++i) {
        for (int j = i + 1; j < n_outs; ++j)
            if (overlap(outs[i].p, outs[i].n, outs[j].p, outs[j].n))
                return false;
        for (int j = 0; j < n_ins; ++j)
            if (overlap(outs[i].p, outs[i].n, ins[j].p, ins[j].n))
                return false;
    }
    return true;
}

static taco_status fp8_quantize_any(const void *x, int64_t rows, int64_t cols, bool tiles, uint8_t *codes,
                                    uint8_t *scale, uint8_t *codes_t, uint8_t *scale_t, taco_stream_t stream)
{
    if (rows < 0 || cols < 0)
        return TACO_ERR_INVALID_ARG;
    if (!fp8_dims_fit(rows, cols))
        return TACO_ERR_UNSUPPORTED;
    if (rows == 0 || cols == 0)
        return TACO_OK;
    if ((codes == nullptr) != (scale == nullptr) || (codes_t == nullptr) != (scale_t == nullptr) ||
        (!codes && !codes_t) || !x)
        return TACO_ERR_INVALID_ARG;
    if (!aligned(x, 16) || !aligned(codes, 16) || !aligned(codes_t, 16) ||
        (!tiles && (!aligned(scale, 16) || !aligned(scale_t, 16))))
        return TACO_ERR_MISALIGNED;
    const uint64_t r = rows, c = cols, rb = fp8_blocks(rows), cb = fp8_blocks(cols);
    const Span outs[4] = {{codes, codes ? r * taco::fp8_pitch(cols) : 0},
                          {scale, !scale ? 0 : tiles ? cb * rb : taco::fp8_scale_bytes(rows, cols)},
                          {codes_t, codes_t ? c * taco::fp8_pitch(rows) : 0},
                          {scale_t, !scale_t ? 0 : tiles ? cb * rb : taco::fp8_scale_bytes(cols, rows)}};
    const Span ins[1] = {{x, 2 * r * c}};
    if (!apart(outs, 4, ins, 1))
        return TACO_ERR_INVALID_ARG;
    return from_cuda(taco::launch_fp8_quantize({x, rows, cols, codes, scale, codes_t, scale_t, taco::fp8_pitch(cols),
                                                taco::fp8_pitch(rows)},
                                               tiles, reinterpret_cast<cudaStream_t>(stream)));
}

taco_status fp8_quantize(const void *x_bf16, int64_t rows, int64_t cols, uint8_t *codes, uint8_t *scale,
                         uint8_t *codes_t, uint8_t *scale_t, taco_stream_t stream)
{
    return fp8_quantize_any(x_bf16, rows, cols, false, codes, scale, codes_t, scale_t, stream);
}

taco_status fp8_quantize_weight(const void *x_bf16, int64_t rows, int64_t cols, uint8_t *codes, uint8_t *scale,
                                uint8_t *codes_t, uint8_t *scale_t, taco_stream_t stream)
{
    return fp8_quantize_any(x_bf16, rows, cols, true, codes, scale, codes_t, scale_t, stream);
}

taco_status fp8_gemm(const uint8_t *a, const uint8_t *a_scale, const uint8_t *b, const uint8_t *b_scale,
                     int32_t b_scale_tiles, int64_t M, int64_t N, int64_t K, void *out, int32_t out_is_bf16,
                     taco_stream_t stream)
{
    if (M < 0 || N < 0 || K < 0 || K % 16 != 0)
        return TACO_ERR_INVALID_ARG;
    if (!fp8_dims_fit(M, K) || !fp8_dims_fit(N, K) || !fp8_dims_fit(M, N))
        return TACO_ERR_UNSUPPORTED;
    if (M == 0 || N == 0)
        return TACO_OK;
    if (!out || (K > 0 && (!a || !a_scale || !b || !b_scale)))
        return TACO_ERR_INVALID_ARG;
    if (!aligned(out, 16) || (K > 0 && (!aligned(a, 16) || !aligned(b, 16) || !aligned(a_scale, 16) ||
                                        (!b_scale_tiles && !aligned(b_scale, 16)))))
        return TACO_ERR_MISALIGNED;
    const uint64_t m = M, n = N, k = K;
    const Span outs[1] = {{out, m * n * (out_is_bf16 ? 2 : 4)}};
    const Span ins[4] = {{a, m * k},
                         {b, n * k},
                         {a_scale, static_cast<uint64_t>(taco::fp8_scale_bytes(M, K))},
                         {b_scale, static_cast<uint64_t>(b_scale_tiles ? fp8_blocks(K) * fp8_blocks(N)
                                                                       : taco::fp8_scale_bytes(N, K))}};
    if (!apart(outs, 1, ins, 4))
        return TACO_ERR_INVALID_ARG;
    return from_cuda(taco::launch_fp8_gemm({a, a_scale, K, false}, {b, b_scale, K, b_scale_tiles != 0}, M, N, K, out,
                                           out_is_bf16 != 0, reinterpret_cast<cudaStream_t>(stream)));
}

// The pieces of a linear layer's workspace, each 256-byte aligned: a
// quantised matrix [rows][cols] is its codes, in rows of fp8_work_pitch(cols)
// bytes, and its scales.
static uint64_t fp8_piece(int64_t rows, int64_t cols, uint64_t *scale_at)
{
    const auto up = [](uint64_t v) { return (v + 255) & ~uint64_t(255); };
    const uint64_t codes = up(static_cast<uint64_t>(rows) * taco::fp8_work_pitch(cols));
    if (scale_at)
        *scale_at = codes;
    return codes + up(taco::fp8_scale_bytes(rows, cols));
}

taco_status fp8_linear_workspace_bytes(int64_t M, int64_t N, int64_t K, int32_t backward, uint64_t *bytes)
{
    if (!bytes || M < 0 || N < 0 || K < 0)
        return TACO_ERR_INVALID_ARG;
    *bytes = 0;
    if (!fp8_dims_fit(M, K) || !fp8_dims_fit(N, K) || !fp8_dims_fit(M, N))
        return TACO_ERR_UNSUPPORTED;
    *bytes = backward ? fp8_piece(M, N, nullptr) + fp8_piece(N, M, nullptr) + fp8_piece(K, M, nullptr)
              : taco::fp8_decode_takes(M, K) ? 0 : fp8_piece(M, K, nullptr);
    return TACO_OK;
}

taco_status fp8_linear(const void *x_bf16, const uint8_t *codes, const uint8_t *scale, int64_t M, int64_t N,
                       int64_t K, void *y, int32_t y_is_bf16, void *workspace, uint64_t workspace_bytes,
                       taco_stream_t stream)
{
    uint64_t need = 0, scale_at = 0;
    taco_status st = fp8_linear_workspace_bytes(M, N, K, 0, &need);
    if (st != TACO_OK || M == 0 || N == 0)
        return st;
    if (!y || workspace_bytes < need || (need > 0 && !workspace) || (K > 0 && (!x_bf16 || !codes || !scale)))
        return TACO_ERR_INVALID_ARG;
    if (!aligned(y, 16) || !aligned(x_bf16, 16) || !aligned(codes, 16) || !aligned(workspace, 256))
        return TACO_ERR_MISALIGNED;
    const uint64_t pk = taco::fp8_pitch(K), n = N;
    const Span outs[2] = {{y, static_cast<uint64_t>(M) * n * (y_is_bf16 ? 2 : 4)}, {workspace, need}};
    const Span ins[3] = {{x_bf16, 2 * static_cast<uint64_t>(M) * K},
                         {codes, n * pk},
                         {scale, static_cast<uint64_t>(fp8_blocks(K)) * fp8_blocks(N)}};
    if (!apart(outs, 2, ins, 3))
        return TACO_ERR_INVALID_ARG;
    if (K > 0 && need == 0)  // few tokens: one kernel
        return from_cuda(taco::launch_fp8_decode(x_bf16, codes, scale, M, N, K, y, y_is_bf16 != 0,
                                                 reinterpret_cast<cudaStream_t>(stream)));
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const int64_t kw = taco::fp8_work_pitch(K);
    fp8_piece(M, K, &scale_at);
    cudaError_t e = cudaSuccess;
    if (K > 0)
        e = taco::launch_fp8_quantize({x_bf16, M, K, ws, ws + scale_at, nullptr, nullptr, kw, 0}, false, s);
    if (e == cudaSuccess)
        e = taco::launch_fp8_gemm({ws, ws + scale_at, kw, false}, {codes, scale, static_cast<int64_t>(pk), true}, M, N,
                                  pk, y, y_is_bf16 != 0, s);
    return from_cuda(e);
}

taco_status fp8_linear_backward(const void *dy_bf16, const void *x_bf16, const uint8_t *codes_t,
                                const uint8_t *scale_t, int64_t M, int64_t N, int64_t K, void *dx_bf16, void *dw,
                                int32_t dw_is_bf16, void *workspace, uint64_t workspace_bytes,
                                taco_stream_t stream)
{
    uint64_t need = 0;
    taco_status st = fp8_linear_workspace_bytes(M, N, K, 1, &need);
    if (st != TACO_OK)
        return st;
    const bool want_dx = dx_bf16 && M > 0 && K > 0, want_dw = dw && N > 0 && K > 0;
    if (!dx_bf16 && !dw && M > 0 && N > 0 && K > 0)
        return TACO_ERR_INVALID_ARG;
    if (!want_dx && !want_dw)
        return TACO_OK;
    const bool data = M > 0 && N > 0;  // else both gradients are sums over nothing
    if (data && (!dy_bf16 || !workspace || workspace_bytes < need || (want_dx && (!codes_t || !scale_t)) ||
                 (want_dw && !x_bf16)))
        return TACO_ERR_INVALID_ARG;
    if ((want_dx && !aligned(dx_bf16, 16)) || (want_dw && !aligned(dw, 16)) ||
        (data && (!aligned(dy_bf16, 16) || !aligned(workspace, 256) || (want_dx && !aligned(codes_t, 16)) ||
                  (want_dw && !aligned(x_bf16, 16)))))
        return TACO_ERR_MISALIGNED;
    const uint64_t m = M, n = N, k = K, pn = taco::fp8_pitch(N), pm = taco::fp8_pitch(M);
    const Span outs[3] = {{dx_bf16, want_dx ? 2 * m * k : 0},
                          {dw, want_dw ? n * k * (dw_is_bf16 ? 2 : 4) : 0},
                          {workspace, data ? need : 0}};
    const Span ins[4] = {{dy_bf16, data ? 2 * m * n : 0},
                         {x_bf16, data && want_dw ? 2 * m * k : 0},
                         {codes_t, data && want_dx ? k * pn : 0},
                         {scale_t, data && want_dx ? static_cast<uint64_t>(fp8_blocks(N)) * fp8_blocks(K) : 0}};
    if (!apart(outs, 3, ins, 4))
        return TACO_ERR_INVALID_ARG;
    if (!data) {
        if (want_dx && (st = fp8_gemm(nullptr, nullptr, nullptr, nullptr, 1, M, K, 0, dx_bf16, 1, stream)) != TACO_OK)
            return st;
        return want_dw ? fp8_gemm(nullptr, nullptr, nullptr, nullptr, 0, N, K, 0, dw, dw_is_bf16, stream) : TACO_OK;
    }
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    uint64_t s0 = 0, s1 = 0, s2 = 0;
    uint8_t *q = ws, *qt = q + fp8_piece(M, N, &s0), *xt = qt + fp8_piece(N, M, &s1);
    fp8_piece(K, M, &s2);
    const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const int64_t nw = taco::fp8_work_pitch(N), mw = taco::fp8_work_pitch(M);
    const taco::Fp8Quantize quantize_dy = {dy_bf16, M, N, want_dx ? q : nullptr, want_dx ? q + s0 : nullptr,
                                           want_dw ? qt : nullptr, want_dw ? qt + s1 : nullptr, nw, mw};
    cudaError_t e = want_dw ? taco::launch_fp8_quantize_two(
                                  quantize_dy, {x_bf16, M, K, nullptr, nullptr, xt, xt + s2, 0, mw}, s)
                            : taco::launch_fp8_quantize(quantize_dy, false, s);
    if (e == cudaSuccess && want_dx)
        e = taco::launch_fp8_gemm({q, q + s0, nw, false}, {codes_t, scale_t, static_cast<int64_t>(pn), true}, M, K, pn,
                                  dx_bf16, true, s);
    if (e == cudaSuccess && want_dw)
        e = taco::launch_fp8_gemm({qt, qt + s1, mw, false}, {xt, xt + s2, mw, false}, N, K, pm, dw, dw_is_bf16 != 0, s);
    return from_cuda(e);
}

// Shared checks of the norms around a block.
static taco_status check_norm(int64_t T, int64_t d, int32_t gate_mode, float residual_scale, float eps)
{
    if (T < 0 || d < 1 || !std::isfinite(residual_scale) || !positive_finite(eps))
        return TACO_ERR_INVALID_ARG;
    if (gate_mode < TACO_GATE_NONE || gate_mode > TACO_GATE_FULL)
        return TACO_ERR_INVALID_ARG;
    if (d > TACO_NORM_MAX_D || T > (int64_t(1) << 40))
        return TACO_ERR_UNSUPPORTED;
    return TACO_OK;
}

static bool gate_aligned(const void *gate, int32_t mode)
{
    return mode == TACO_GATE_NONE || aligned(gate, mode == TACO_GATE_TOKEN ? 4 : 16);
}

static uint64_t gate_bytes(int32_t mode, int64_t T, int64_t d)
{
    return mode == TACO_GATE_NONE ? 0 : mode == TACO_GATE_CHANNEL ? 4 * d : mode == TACO_GATE_TOKEN ? 4 * T : 2 * T * d;
}

taco_status rmsnorm_gate_residual(const void *y, const void *h, const float *g_post, const float *g_pre,
                                  const void *gate, int32_t gate_mode, float residual_scale, float eps, int64_t T,
                                  int64_t d, void *h_out, void *n, uint8_t *n_scale, taco_stream_t stream)
{
    taco_status st = check_norm(T, d, gate_mode, residual_scale, eps);
    if (st != TACO_OK || T == 0)
        return st;
    if (!y || !h || !g_post || !g_pre || !h_out || !n || (gate_mode != TACO_GATE_NONE) != (gate != nullptr))
        return TACO_ERR_INVALID_ARG;
    if (!aligned(y, 16) || !aligned(h, 16) || !aligned(g_post, 16) || !aligned(g_pre, 16) || !aligned(h_out, 16) ||
        !aligned(n, 16) || !aligned(n_scale, 16) || !gate_aligned(gate, gate_mode))
        return TACO_ERR_MISALIGNED;
    const uint64_t td = 2 * static_cast<uint64_t>(T) * d, d4 = 4 * static_cast<uint64_t>(d);
    const Span outs[3] = {{h_out, td},
                          {n, n_scale ? static_cast<uint64_t>(T) * taco::fp8_pitch(d) : td},
                          {n_scale, n_scale ? static_cast<uint64_t>(taco::fp8_scale_bytes(T, d)) : 0}};
    const Span ins[5] = {{y, td}, {h, td}, {g_post, d4}, {g_pre, d4}, {gate, gate_bytes(gate_mode, T, d)}};
    if (!apart(outs, 3, ins, 5))
        return TACO_ERR_INVALID_ARG;
    return from_cuda(taco::launch_norm_forward(
        {y, h, g_post, g_pre, gate, gate_mode, residual_scale, eps, T, d, h_out, n, n_scale},
        reinterpret_cast<cudaStream_t>(stream)));
}

taco_status rmsnorm_gate_residual_workspace_bytes(int64_t T, int64_t d, int32_t gate_mode, uint64_t *bytes)
{
    if (!bytes)
        return TACO_ERR_INVALID_ARG;
    *bytes = 0;
    taco_status st = check_norm(T, d, gate_mode, 1.0f, 1.0f);
    if (st != TACO_OK || T == 0)
        return st;
    return from_cuda(taco::norm_backward_workspace(T, d, gate_mode, bytes));
}

taco_status rmsnorm_gate_residual_backward(const void *dn, const void *dh_out, const void *y, const void *h_out,
                                           const float *g_post, const float *g_pre, const void *gate,
                                           int32_t gate_mode, float residual_scale, float eps, int64_t T, int64_t d,
                                           void *dy, void *dh, float *dg_post, float *dg_pre, void *dgate,
                                           void *workspace, uint64_t workspace_bytes, taco_stream_t stream)
{
    taco_status st = check_norm(T, d, gate_mode, residual_scale, eps);
    if (st != TACO_OK)
        return st;
    if (!dg_post || !dg_pre || (gate_mode != TACO_GATE_NONE && !dgate && (T > 0 || gate_mode == TACO_GATE_CHANNEL)) ||
        (gate_mode == TACO_GATE_NONE && dgate))
        return TACO_ERR_INVALID_ARG;
    if (T > 0 && (!dn || !dh_out || !y || !h_out || !g_post || !g_pre || !dy || !dh || !workspace ||
                  (gate_mode != TACO_GATE_NONE) != (gate != nullptr)))
        return TACO_ERR_INVALID_ARG;
    if (!aligned(dg_post, 4) || !aligned(dg_pre, 4) || !gate_aligned(dgate, gate_mode) ||
        (T > 0 && (!aligned(dn, 16) || !aligned(dh_out, 16) || !aligned(y, 16) || !aligned(h_out, 16) ||
                   !aligned(g_post, 16) || !aligned(g_pre, 16) || !gate_aligned(gate, gate_mode) ||
                   !aligned(dy, 16) || !aligned(dh, 16) || !aligned(workspace, 256))))
        return TACO_ERR_MISALIGNED;
    const uint64_t td = 2 * static_cast<uint64_t>(T) * d, d4 = 4 * static_cast<uint64_t>(d);
    const uint64_t gb = gate_bytes(gate_mode, T, d);
    uint64_t need = 0;
    if (T > 0) {
        cudaError_t e = taco::norm_backward_workspace(T, d, gate_mode, &need);
        if (e != cudaSuccess)
            return TACO_ERR_CUDA;
        if (workspace_bytes < need)
            return TACO_ERR_INVALID_ARG;
    }
    const Span outs[6] = {{dy, td}, {dh, td}, {dg_post, d4}, {dg_pre, d4}, {dgate, dgate ? gb : 0}, {workspace, need}};
    const Span ins[7] = {{dn, td}, {dh_out, td}, {y, td}, {h_out, td}, {g_post, d4}, {g_pre, d4}, {gate, gb}};
    if (!apart(outs, 6, ins, T > 0 ? 7 : 0))
        return TACO_ERR_INVALID_ARG;
    return from_cuda(taco::launch_norm_backward({dn, dh_out, y, h_out, g_post, g_pre, gate, gate_mode, residual_scale,
                                                 eps, T, d, dy, dh, dg_post, dg_pre, dgate, workspace},
                                                reinterpret_cast<cudaStream_t>(stream)));
}

struct taco_host_pipeline {
    taco::HostPipeline *impl;
};

taco_status taco_host_pipeline_create(int32_t P, int64_t rows, int64_t d, int32_t block, int32_t chunks,
                                      int32_t out_is_bf16, taco_host_pipeline **pipe_out,
                                      uint64_t *workspace_bytes)
{
    if (!pipe_out || !workspace_bytes)
        return TACO_ERR_INVALID_ARG;
    *pipe_out = nullptr;
    taco_status st = check_taco_shape(rows, d, block);
    if (st != TACO_OK)
        return st;
    if (P < 1 || P > TACO_MAX_SHARDS)
        return TACO_ERR_UNSUPPORTED;
    if (rows < 1 || chunks < 1 || chunks > taco::host_pipeline_max_chunks())
        return TACO_ERR_INVALID_ARG;
    auto *h = new (std::nothrow) taco_host_pipeline{nullptr};
    if (!h)
        return TACO_ERR_CUDA;
    const int c = static_cast<int>(chunks < rows ? chunks : rows);
    cudaError_t e = taco::host_pipeline_create(P, rows, d, block, c, out_is_bf16 != 0, &h->impl, workspace_bytes);
    if (e != cudaSuccess) {
        delete h;
        return TACO_ERR_CUDA;
    }
    *pipe_out = h;
    return TACO_OK;
}

taco_status taco_host_pipeline_run(taco_host_pipeline *pipe, const void *x_host_bf16, void *out_host,
                                   void *workspace, float e_target, float eps, taco_stream_t stream)
{
    if (!pipe || !pipe->impl || !x_host_bf16 || !out_host || !workspace)
        return TACO_ERR_INVALID_ARG;
    if (!positive_finite(e_target) || !positive_finite(eps))
        return TACO_ERR_INVALID_ARG;
    if (!aligned(workspace, 256))
        return TACO_ERR_MISALIGNED;
    int dev = -1;
    if (cudaGetDevice(&dev) != cudaSuccess)
        return TACO_ERR_CUDA;
    if (dev != taco::host_pipeline_device(pipe->impl))
        return TACO_ERR_INVALID_ARG;
    return from_cuda(taco::host_pipeline_run(pipe->impl, x_host_bf16, out_host, workspace, e_target, eps,
                                             reinterpret_cast<cudaStream_t>(stream)));
}

taco_status taco_host_pipeline_destroy(taco_host_pipeline *pipe)
{
    if (!pipe)
        return TACO_ERR_INVALID_ARG;
    taco::host_pipeline_destroy(pipe->impl);
    delete pipe;
    return TACO_OK;
}

taco_status taco_watchdog_selftest(taco_stream_t stream)
{
    return from_cuda(taco::launch_watchdog_selftest(reinterpret_cast<cudaStream_t>(stream)));
}

taco_status taco_device_error(uint32_t *flags_out, int32_t clear)
{
    if (!flags_out)
        return TACO_ERR_INVALID_ARG;
    cudaError_t e = cudaDeviceSynchronize();
    if (e != cudaSuccess)
        return TACO_ERR_CUDA;
    uint32_t codec = 0, gemm = 0, fp8 = 0, norm = 0;
    if ((e = taco::read_codec_error(&codec, clear != 0)) != cudaSuccess ||
        (e = taco::read_gemm_error(&gemm, clear != 0)) != cudaSuccess ||
        (e = taco::read_fp8_error(&fp8, clear != 0)) != cudaSuccess ||
        (e = taco::read_norm_error(&norm, clear != 0)) != cudaSuccess)
        return from_cuda(e);
    *flags_out = codec | gemm | fp8 | norm;
    return TACO_OK;
}

}  // extern "C"
