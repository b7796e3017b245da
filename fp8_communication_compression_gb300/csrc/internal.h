// Host-side declarations shared by the C-ABI layer and the kernel files.
#pragma once

#include <atomic>
#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

#include "../../include/taco.h"

namespace taco {

// Per-device facts the launchers need (cached on first use).
struct DeviceInfo {
    int device;
    int num_sms;
    int max_smem_optin;
};
cudaError_t current_device_info(DeviceInfo *out);

// cuTensorMapEncodeTiled, resolved through the runtime's driver entry point
// (128-byte swizzle unless asked otherwise).  Returns 0 on success.
int encode_tensor_map_2d(CUtensorMap *map, CUtensorMapDataType dtype, void *base, uint64_t inner,
                         uint64_t rows, uint64_t row_stride_bytes, uint32_t box_inner,
                         uint32_t box_rows, CUtensorMapSwizzle swizzle = CU_TENSOR_MAP_SWIZZLE_128B);

// Kernels working on the "128-view" of a TACO tensor: nrows rows of 128
// elements; a block of n elements spans n / 128 consecutive rows.
// int8_codes selects the INT8 code format (Q_max 127) instead of E4M3.
cudaError_t launch_compress(const void *x_bf16, int64_t nrows, int block, float e_target, float eps,
                            uint8_t *codes, float *alpha, float *scale, bool int8_codes,
                            cudaStream_t stream);
cudaError_t launch_decompress(const uint8_t *codes, const float *alpha, const float *scale,
                              int64_t nrows, int block, void *out, bool out_bf16, bool int8_codes,
                              cudaStream_t stream);

// Direct-load kernels (no Hadamard on their path).
struct ShardPtrs {
    const uint8_t *codes[16];
    const float *alpha[16];
    const float *scale[16];
};
cudaError_t launch_taco_reduce(int P, const ShardPtrs &in, int64_t nblocks, int block, float e_target,
                               float eps, uint8_t *out_codes, float *out_alpha, float *out_scale,
                               cudaStream_t stream);
cudaError_t launch_reduce_decompress(int P, const ShardPtrs &in, int64_t nrows, int block, float e_target,
                                     float eps, uint8_t *out_codes, float *out_alpha, float *out_scale,
                                     void *out, bool out_bf16, cudaStream_t stream);
cudaError_t launch_agoq_accumulate(uint8_t *codes, float *scale, const void *grad_bf16, int64_t n,
                                   int block, cudaStream_t stream);
cudaError_t launch_agoq_reduce(int P, const ShardPtrs &in, int64_t n, int block, uint8_t *out_codes,
                               float *out_scale, cudaStream_t stream);

cudaError_t launch_laaq_quantize(const void *x_bf16, int64_t n, int block, int bits, uint8_t *packed,
                                 float *scale, cudaStream_t stream);
cudaError_t launch_laaq_dequantize(const uint8_t *packed, const float *scale, int64_t n, int block, int bits,
                                   void *out, bool out_bf16, bool silu, cudaStream_t stream);
// RMSNorm of each row of d values (d % block == 0) recomputed from the
// stored quantised input: y = x_hat / sqrt(mean(x_hat^2) + eps) * gamma.
cudaError_t launch_laaq_rmsnorm(const uint8_t *packed, const float *scale, int64_t rows, int64_t d, int block,
                                int bits, const float *gamma, float eps, void *out, bool out_bf16,
                                cudaStream_t stream);

cudaError_t launch_e4m3_encode(const float *x, int64_t n, uint8_t *codes, cudaStream_t stream);

// Chunked host-buffer pipeline of the two-shot local path (host_pipeline.cu).
struct HostPipeline;
int host_pipeline_max_chunks();
cudaError_t host_pipeline_create(int P, int64_t rows, int64_t d, int block, int chunks, bool out_bf16,
                                 HostPipeline **out, uint64_t *workspace_bytes);
void host_pipeline_destroy(HostPipeline *p);
int host_pipeline_device(const HostPipeline *p);
uint64_t host_pipeline_workspace(const HostPipeline *p);
cudaError_t host_pipeline_run(HostPipeline *p, const void *x_host, void *out_host, void *workspace, float e_target,
                              float eps, cudaStream_t stream);

// Tensor-core GEMM Y = A B^T (bf16, fp32 accumulate) with the ASH + DS
// compressor in its epilogue (gemm_compress.cu): M % 128 == 0,
// N % 128 == 0, K % 64 == 0, block 128.  y_out (fp32 [M][N]) may be null.
// workspace (workspace_bytes, 256-byte aligned, zeroed before its first
// use) holds the split tail's partial sums; null or too small: no split.
cudaError_t launch_gemm_compress(const void *a_bf16, const void *b_bf16, int64_t M, int64_t N, int64_t K,
                                 float e_target, float eps, uint8_t *codes, float *alpha, float *scale,
                                 float *y_out, void *workspace, uint64_t workspace_bytes, cudaStream_t stream);
// The same GEMM with the AGoQ accumulation into an FP8 main gradient
// ([M][N] codes and [M][N / 128] multipliers, in place) in its epilogue.
cudaError_t launch_gemm_agoq_accumulate(const void *a_bf16, const void *b_bf16, int64_t M, int64_t N, int64_t K,
                                        uint8_t *main_codes, float *main_scale, float *y_out, void *workspace,
                                        uint64_t workspace_bytes, cudaStream_t stream);
// The same GEMM with AGoQ's LAAQ activation quantisation of its output in
// its epilogue: blocks of 128 along each row, `bits` (4, 5, 6 or 8) bits a
// code, packed [M][N * bits / 8] and multipliers [M][N / 128].
cudaError_t launch_gemm_laaq_quantize(const void *a_bf16, const void *b_bf16, int64_t M, int64_t N, int64_t K,
                                      int bits, uint8_t *packed, float *scale, float *y_out, void *workspace,
                                      uint64_t workspace_bytes, cudaStream_t stream);
// Workspace the split tail of an M x N x K GEMM takes on the current device
// (0 when it takes none).
cudaError_t gemm_workspace_bytes(int64_t M, int64_t N, int64_t K, uint64_t *bytes);

// Block-scaled FP8 operands (fp8_quantize.cu; format in fp8_block.cuh) of a
// bf16 matrix x: codes [rows][stride] with their scales, and / or codes_t
// [cols][stride_t] with scale_t; null codes: that direction is left out.
// tiles: one byte per 128 x 128 tile, scale [ceil(cols / 128)][ceil(rows /
// 128)] and scale_t its transpose.
struct Fp8Quantize {
    const void *x;
    int64_t rows, cols;
    uint8_t *codes, *scale, *codes_t, *scale_t;
    int64_t stride, stride_t;
};
cudaError_t launch_fp8_quantize(const Fp8Quantize &q, bool tiles, cudaStream_t stream);
// Two matrices in one launch (together less than 2^31 tiles of 128 x 128).
cudaError_t launch_fp8_quantize_two(const Fp8Quantize &a, const Fp8Quantize &b, cudaStream_t stream);
// An operand of a product: codes in rows of `stride` bytes, and their scales
// (tiles: one byte per 128 x 128 tile).
struct Fp8Operand {
    const uint8_t *codes, *scale;
    int64_t stride;
    bool tiles;
};
// out[M][N] = A B^T (fp8_gemm.cu) over K codes of A's M and B's N rows (K and
// the strides multiples of 16; A without tiles).
cudaError_t launch_fp8_gemm(const Fp8Operand &a, const Fp8Operand &b, int64_t M, int64_t N, int64_t K, void *out,
                            bool out_bf16, cudaStream_t stream);
// fp8_linear for few tokens without a workspace (fp8_decode.cu), where
// fp8_decode_takes(M, K); scale: a weight's (128 x 128 tiles).
bool fp8_decode_takes(int64_t M, int64_t K);
cudaError_t launch_fp8_decode(const void *x_bf16, const uint8_t *codes, const uint8_t *scale, int64_t M, int64_t N,
                              int64_t K, void *y, bool y_bf16, cudaStream_t stream);

// The norms around a block (norm_kernels.cu).  n_scale null: n_out is bf16
// [T][d]; else FP8 codes [T][pitch(d)] and their scales n_scale.
struct NormForward {
    const void *y, *h;
    const float *g_post, *g_pre;
    const void *gate;
    int gate_mode;
    float residual_scale, eps;
    int64_t T, d;
    void *h_out, *n_out;
    uint8_t *n_scale;
};
cudaError_t launch_norm_forward(const NormForward &a, cudaStream_t stream);
struct NormBackward {
    const void *dn, *dh_out, *y, *h_out;
    const float *g_post, *g_pre;
    const void *gate;
    int gate_mode;
    float residual_scale, eps;
    int64_t T, d;
    void *dy, *dh;
    float *dg_post, *dg_pre;
    void *dgate, *workspace;
};
cudaError_t launch_norm_backward(const NormBackward &a, cudaStream_t stream);
cudaError_t norm_backward_workspace(int64_t T, int64_t d, int gate_mode, uint64_t *bytes);

// The losses over the vocabulary (loss_kernels.cu).  Logits [T][N] in bf16 or
// fp32, their first V columns in use.
struct LossRows {
    const void *logits;
    const int64_t *targets;
    int64_t T, V, N;
    float temperature, temperature_low, inv_temperature, inv_temperature_low;  // each in two parts
    float grad_scale;
    float *logp, *lse;                   // forward, or (max, inv_sum, coef) instead of lse:
    float *max, *inv_sum, *coef;         // coef: zeroed in rows that do not count
    const int64_t *offsets;              // rows outside offsets[0] .. offsets[sequences] do not count (may be null)
    int64_t sequences;
    const float *dlogp;                  // backward (with lse, or max and inv_sum)
    const float *old_logp, *advantages, *weights, *ref_logp;  // policy loss
    float clip_lo, clip_hi, kl;
    float *token_loss, *loss;
    void *dlogits;                       // may be null in the policy and the preference loss
};
struct PairArgs {
    const int64_t *targets, *offsets;
    int64_t T, pairs;
    const float *logp, *ref_logp;
    float beta, smoothing;
    bool mean;
    float *loss, *margin, *logratio, *pair_loss, *coef;
};
cudaError_t launch_logprob(const LossRows &a, bool bf16, cudaStream_t stream);
cudaError_t launch_logprob_backward(const LossRows &a, bool bf16, cudaStream_t stream);
cudaError_t launch_policy_loss(const LossRows &a, bool bf16, cudaStream_t stream);
cudaError_t launch_preference_loss(const LossRows &a, const PairArgs &p, bool bf16, cudaStream_t stream);

// The optimizer (adamw_kernels.cu).  `tensors` are host arrays.
constexpr int kAdamWTensors = 320, kNormTensors = 720;  // of one launch
cudaError_t grad_norm_workspace(int64_t count, uint64_t *bytes);
cudaError_t launch_grad_norm(const grad_tensor *tensors, int64_t count, float grad_scale, float *norm,
                             void *workspace, cudaStream_t stream);
struct AdamWStep {
    double beta1, beta2;
    float eps, grad_scale, max_norm;                // max_norm 0: no clipping
    float *norm;                                    // null: not computed
    const float *lr_factor;                         // may be null
    uint64_t seed;
    int64_t *state;
};
// workspace: grad_norm_workspace's, where there is a norm.
cudaError_t launch_adamw(const adamw_tensor *tensors, int64_t count, bool bits8, const AdamWStep &h,
                         void *workspace, cudaStream_t stream);

cudaError_t launch_watchdog_selftest(cudaStream_t stream);
cudaError_t read_codec_error(uint32_t *flags, bool clear);
cudaError_t read_gemm_error(uint32_t *flags, bool clear);
cudaError_t read_fp8_error(uint32_t *flags, bool clear);
cudaError_t read_norm_error(uint32_t *flags, bool clear);
cudaError_t read_loss_error(uint32_t *flags, bool clear);
cudaError_t read_adamw_error(uint32_t *flags, bool clear);

// Raises a kernel's dynamic shared-memory limit once per device.  The flag
// is atomic because host threads may make their first launch concurrently;
// setting the attribute twice is harmless.
constexpr int kMaxDevices = 64;
template <typename K>
cudaError_t ensure_smem(K kernel, uint32_t bytes, int device, std::atomic<bool> *done)
{
    if (done[device].load(std::memory_order_acquire))
        return cudaSuccess;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(bytes));
    if (e == cudaSuccess)
        done[device].store(true, std::memory_order_release);
    return e;
}

// CTAs of `threads` threads and `smem` bytes of dynamic shared memory that fit an
// SM, at least 1.  The last answer for each device is kept in `last` (the query
// takes a microsecond), packed into one word.
template <typename K>
cudaError_t ctas_per_sm(K kernel, int threads, size_t smem, int device, std::atomic<uint64_t> *last, int *ctas)
{
    const uint64_t key = static_cast<uint64_t>(smem) << 32 | static_cast<uint64_t>(threads) << 16;
    const uint64_t known = last[device].load(std::memory_order_relaxed);
    if (known && (known & ~uint64_t(0xFFFF)) == key) {
        *ctas = static_cast<int>(known & 0xFFFF);
        return cudaSuccess;
    }
    int n = 0;
    const cudaError_t e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kernel, threads, smem);
    *ctas = n < 1 ? 1 : n;
    if (e == cudaSuccess)
        last[device].store(key | static_cast<uint64_t>(*ctas), std::memory_order_relaxed);
    return e;
}

// Launches `kernel` with programmatic stream serialization allowed, so that
// it can be scheduled while the previous kernel in the stream drains (every
// kernel of this library waits for its predecessor with griddepcontrol.wait
// before reading inputs).
template <typename... KArgs, typename... Args>
cudaError_t launch_pdl(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t stream,
                       Args &&...args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, static_cast<Args &&>(args)...);
}

} // namespace taco
