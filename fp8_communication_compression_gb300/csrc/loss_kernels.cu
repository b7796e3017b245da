// Losses over the vocabulary: log probabilities of the targets, the clipped
// policy loss, the preference loss, and their gradients at the logits.
//
// Row t of the logits holds V values x_j (its first V of N columns), a = its
// target, tau the temperature:
//
//   logp = x_a / tau - lse,  lse = log sum_j exp(x_j / tau)
//   dlogits_j = dlogp / tau (1[j = a] - exp(x_j / tau - lse))
//
// policy loss, with r = exp(logp - old), d = ref - logp:
//
//   L = w (-min(r A, clip(r, 1 - cl, 1 + ch) A) + kl (exp(d) - 1 - d))
//   dlogp = w (-[r A <= clip(r) A] r A - kl (exp(d) - 1))
//
// preference loss: s_i = sum (or mean) over sequence i of logp - ref,
// z = beta (s_2i - s_2i+1), L = mean_i(-(1 - ls) log sig(z) - ls log sig(-z)).
//
// The sum runs relative to the maximum so far: s <- s exp(m - m') + sum
// exp(x - m'), in fp32, one pass over the row.  The maximum starts at fp32's
// lowest value, not at -inf, so that no difference of infinities arises where
// values are masked with -inf or with the lowest value.  Differences x - m are
// taken before they are scaled: exact where the probability is large.
//
// A row may start anywhere inside a 16-byte granule: threads take whole
// granules of memory, and those at a row's ends leave out what is not its own.

#include "device_utils.cuh"
#include "internal.h"

#include <cfloat>

namespace taco {

namespace {

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

enum Mode { kForward, kPolicy, kBackward };

__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ float neg_inf() { return __int_as_float(0xFF800000); }

// The granules of one row: G elements each, of type E (bf16 as uint16_t, or
// float).
template <typename E> struct Row {
    static constexpr int G = 16 / sizeof(E);
    const E *x;         // the first granule (the row starts `shift` elements in)
    int shift;
    int64_t left;       // elements from x to the end of the tensor

    __device__ Row(const void *logits, int64_t row, int64_t T, int64_t N)
    {
        const int64_t at = row * N;
        shift = static_cast<int>(at & (G - 1));
        x = static_cast<const E *>(logits) + (at - shift);
        left = T * N - (at - shift);
    }

    __device__ uint4 load(int64_t k) const
    {
        if ((k + 1) * G <= left) {
            uint4 v;
            asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                         : "l"(x + k * G));
            return v;
        }
        E e[G];
#pragma unroll
        for (int j = 0; j < G; ++j)
            e[j] = k * G + j < left ? x[k * G + j] : E(0);
        uint4 v;
        memcpy(&v, e, 16);
        return v;
    }
};

__device__ __forceinline__ void values(const uint4 &q, float (&f)[8])
{
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        f[2 * j] = bf16lo_to_f32(w[j]);
        f[2 * j + 1] = bf16hi_to_f32(w[j]);
    }
}
__device__ __forceinline__ void values(const uint4 &q, float (&f)[4])
{
    f[0] = __uint_as_float(q.x), f[1] = __uint_as_float(q.y);
    f[2] = __uint_as_float(q.z), f[3] = __uint_as_float(q.w);
}
__device__ __forceinline__ uint4 packed(const float (&f)[8])
{
    return make_uint4(f32x2_to_bf16x2(f[0], f[1]), f32x2_to_bf16x2(f[2], f[3]), f32x2_to_bf16x2(f[4], f[5]),
                      f32x2_to_bf16x2(f[6], f[7]));
}
__device__ __forceinline__ uint4 packed(const float (&f)[4])
{
    return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
}

// A maximum and a sum relative to it.
struct Sum {
    float m, s;
};
__device__ __forceinline__ Sum join(Sum a, Sum b, float c)
{
    const float m = fmaxf(a.m, b.m);
    return {m, a.s * ex2((a.m - m) * c) + b.s * ex2((b.m - m) * c)};
}

__device__ __forceinline__ float load_element(const uint16_t *p) { return __uint_as_float(uint32_t(*p) << 16); }
__device__ __forceinline__ float load_element(const float *p) { return *p; }

// One CTA a row.
template <typename E, int MODE> __global__ void __launch_bounds__(1024) row_kernel(const LossRows a)
{
    constexpr int G = Row<E>::G;
    __shared__ Sum part[32];
    pdl_wait();
    const int64_t row = blockIdx.x;
    const int tid = threadIdx.x, threads = blockDim.x;
    const Row<E> x(a.logits, row, a.T, a.N);
    const int64_t target = a.targets[row];
    bool active = target >= 0;
    float weight = 1.0f;
    if (MODE == kPolicy) {
        weight = a.weights[row];
        active = active && weight != 0.0f;
    }
    if (MODE == kForward && a.offsets)
        active = active && row >= a.offsets[0] && row < a.offsets[a.sequences];
    if (MODE == kBackward) {
        weight = a.dlogp[row];
        active = active && weight != 0.0f;
    }
    const int64_t granules = (x.shift + a.V + G - 1) / G;
    const float c = a.inv_temperature * kLog2e;
    float coef = 0.0f, ref = 0.0f, inv = 0.0f;  // dlogits = coef / tau (1[j = a] - inv exp2((x - ref) c))
    if (active) {
        const float xa = target < a.V ? load_element(x.x + x.shift + target) : __int_as_float(0x7FFFFFFF);
        if (MODE != kBackward) {
            Sum z = {-FLT_MAX, 0.0f};
            for (int64_t k = tid; k < granules; k += threads) {
                float f[G];
                values(x.load(k), f);
                float m = z.m;
#pragma unroll
                for (int j = 0; j < G; ++j) {
                    const int64_t col = k * G + j - x.shift;
                    if (col < 0 || col >= a.V)
                        f[j] = neg_inf();
                    m = fmaxf(m, f[j]);
                }
                z.s *= ex2((z.m - m) * c);
#pragma unroll
                for (int j = 0; j < G; ++j)
                    z.s += ex2((f[j] - m) * c);
                z.m = m;
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1)
                z = join(z, {__shfl_xor_sync(~0u, z.m, o), __shfl_xor_sync(~0u, z.s, o)}, c);
            if ((tid & 31) == 0)
                part[tid >> 5] = z;
            __syncthreads();
            z = part[0];
            for (int w = 1; w < threads / 32; ++w)
                z = join(z, part[w], c);
            const float ln_s = logf(z.s);
            const float logp = (xa - z.m) * a.inv_temperature - ln_s;
            ref = z.m;
            inv = 1.0f / z.s;
            if (MODE == kForward && tid == 0) {
                a.logp[row] = logp;
                a.lse[row] = z.m * a.inv_temperature + ln_s;
            }
            if (MODE == kPolicy) {
                const float adv = a.advantages[row], r = expf(logp - a.old_logp[row]);
                const float free = adv == 0.0f ? 0.0f : r * adv;
                const float held = fminf(fmaxf(r, a.clip_lo), a.clip_hi) * adv;
                float loss = -fminf(free, held), slope = free <= held ? -free : 0.0f;
                if (isnan(r))
                    loss = slope = r;
                if (a.ref_logp) {
                    const float d = a.ref_logp[row] - logp, em1 = expm1f(d);
                    loss += a.kl * (em1 - d);
                    slope -= a.kl * em1;
                }
                coef = weight * slope * a.grad_scale;
                if (tid == 0) {
                    a.token_loss[row] = weight * loss;
                    a.logp[row] = logp;
                }
            }
        } else {
            // exp(x / tau - lse) = exp2((x - hi) c) exp2(-lo c), hi + lo = lse tau
            const float lse = a.lse[row], hi = lse * a.temperature;
            const float lo = fmaf(lse, a.temperature, -hi);
            ref = hi;
            inv = isfinite(lo) ? ex2(-lo * c) : 1.0f;
            coef = weight * a.grad_scale;
            if (target >= a.V)
                coef = __int_as_float(0x7FFFFFFF);
        }
    } else if (tid == 0) {
        if (MODE != kBackward)
            a.logp[row] = 0.0f;
        if (MODE == kForward)
            a.lse[row] = 0.0f;
        if (MODE == kForward && a.coef)
            a.coef[row] = 0.0f;
        if (MODE == kPolicy)
            a.token_loss[row] = 0.0f;
    }
    if (MODE == kForward || !a.dlogits)
        return;
    coef *= a.inv_temperature;
    const float scaled = coef * inv;
    E *out = static_cast<E *>(a.dlogits) + (x.x - static_cast<const E *>(a.logits));
    const int64_t all = (x.shift + a.N + G - 1) / G;
    for (int64_t k = tid; k < all; k += threads) {
        float f[G], d[G];
        const bool any = active && coef != 0.0f && k < granules;  // a clipped row's gradient is zero
        if (any)
            values(x.load(k), f);
#pragma unroll
        for (int j = 0; j < G; ++j) {
            const int64_t col = k * G + j - x.shift;
            d[j] = any && col < a.V ? -scaled * ex2((f[j] - ref) * c) + (col == target ? coef : 0.0f) : 0.0f;
        }
        const uint4 q = packed(d);
        const int64_t col = k * G - x.shift;
        if (col >= 0 && col + G <= a.N) {
            stg128_stream(out + k * G, q);
        } else {
            E e[G];
            memcpy(e, &q, 16);
#pragma unroll
            for (int j = 0; j < G; ++j)
                if (col + j >= 0 && col + j < a.N)
                    out[k * G + j] = e[j];
        }
    }
}

// Sum over a CTA of 1024 threads in a fixed order, in all threads.
__device__ double block_sum(double v, double *part)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        v += __shfl_xor_sync(~0u, v, o);
    __syncthreads();
    if ((threadIdx.x & 31) == 0)
        part[threadIdx.x >> 5] = v;
    __syncthreads();
    v = 0.0;
    for (int w = 0; w < static_cast<int>(blockDim.x) / 32; ++w)
        v += part[w];
    return v;
}

// out = scale * sum of x: one CTA, in a fixed order.
__global__ void __launch_bounds__(1024) total_kernel(const float *x, int64_t n, float scale, float *out)
{
    __shared__ double part[32];
    pdl_wait();
    double v = 0.0;
    for (int64_t i = threadIdx.x; i < n; i += blockDim.x)
        v += x[i];
    v = block_sum(v, part);
    if (threadIdx.x == 0)
        *out = static_cast<float>(v * scale);
}

// One CTA a pair: the sequences' log ratios, the pair's loss, and the
// gradients at its tokens' log probabilities.  The sums are fp64: the margin is
// a small difference of long sums.
__global__ void __launch_bounds__(256) pair_kernel(const PairArgs a)
{
    __shared__ double part[32];
    pdl_wait();
    const int64_t pair = blockIdx.x;
    int64_t at[3];
    for (int i = 0; i < 3; ++i) {
        const int64_t o = a.offsets[2 * pair + i];
        at[i] = o < 0 ? 0 : o > a.T ? a.T : o;
    }
    double ratio[2], count[2];
    for (int i = 0; i < 2; ++i) {
        double s = 0.0, n = 0.0;
        for (int64_t t = at[i] + threadIdx.x; t < at[i + 1]; t += blockDim.x)
            if (a.targets[t] >= 0) {
                s += static_cast<double>(a.logp[t]) - (a.ref_logp ? a.ref_logp[t] : 0.0f);
                n += 1.0;
            }
        ratio[i] = block_sum(s, part);
        count[i] = a.mean ? fmax(block_sum(n, part), 1.0) : 1.0;
        ratio[i] /= count[i];
    }
    const float z = static_cast<float>(a.beta * (ratio[0] - ratio[1]));
    const float e = expf(-fabsf(z)), soft = log1pf(e);  // -log sig(|z|)
    const float down = z >= 0.0f ? soft : soft - z, up = z >= 0.0f ? soft + z : soft;
    const float sig = z >= 0.0f ? 1.0f / (1.0f + e) : e / (1.0f + e);
    const float far = z >= 0.0f ? e / (1.0f + e) : 1.0f / (1.0f + e);  // sig(-z)
    if (threadIdx.x == 0) {
        a.margin[pair] = z;
        a.logratio[2 * pair] = static_cast<float>(ratio[0]);
        a.logratio[2 * pair + 1] = static_cast<float>(ratio[1]);
        a.pair_loss[pair] = (1.0f - a.smoothing) * down + a.smoothing * up;
    }
    const float slope = (a.smoothing * sig - (1.0f - a.smoothing) * far) * a.beta / static_cast<float>(a.pairs);
    for (int i = 0; i < 2; ++i) {
        const float g = (i ? -slope : slope) / static_cast<float>(count[i]);
        for (int64_t t = at[i] + threadIdx.x; t < at[i + 1]; t += blockDim.x)
            if (a.targets[t] >= 0)
                a.coef[t] = g;
    }
}

template <int MODE> cudaError_t launch_rows(const LossRows &a, bool bf16, cudaStream_t stream)
{
    const int64_t granules = (a.N + (bf16 ? 7 : 3)) / (bf16 ? 8 : 4) + 1;
    int threads = 32;
    while (threads < 512 && threads * 4 < granules)
        threads *= 2;
    const dim3 grid(static_cast<unsigned>(a.T));
    return bf16 ? launch_pdl(row_kernel<uint16_t, MODE>, grid, threads, 0, stream, a)
                : launch_pdl(row_kernel<float, MODE>, grid, threads, 0, stream, a);
}

}  // namespace

cudaError_t launch_logprob(const LossRows &a, bool bf16, cudaStream_t stream)
{
    return launch_rows<kForward>(a, bf16, stream);
}

cudaError_t launch_logprob_backward(const LossRows &a, bool bf16, cudaStream_t stream)
{
    return launch_rows<kBackward>(a, bf16, stream);
}

cudaError_t launch_policy_loss(const LossRows &a, bool bf16, float *loss, cudaStream_t stream)
{
    if (a.T > 0) {
        const cudaError_t e = launch_rows<kPolicy>(a, bf16, stream);
        if (e != cudaSuccess)
            return e;
    }
    return launch_pdl(total_kernel, 1, 1024, 0, stream, static_cast<const float *>(a.token_loss), a.T, 1.0f, loss);
}

cudaError_t launch_preference_loss(const LossRows &a, const PairArgs &p, bool bf16, float *loss, cudaStream_t stream)
{
    cudaError_t e = cudaSuccess;
    if (a.T > 0 && (e = launch_rows<kForward>(a, bf16, stream)) != cudaSuccess)
        return e;
    if ((e = launch_pdl(pair_kernel, dim3(static_cast<unsigned>(p.pairs)), 256, 0, stream, p)) != cudaSuccess)
        return e;
    if (a.T > 0 && a.dlogits && (e = launch_rows<kBackward>(a, bf16, stream)) != cudaSuccess)
        return e;
    return launch_pdl(total_kernel, 1, 1024, 0, stream, static_cast<const float *>(p.pair_loss), p.pairs,
                      1.0f / static_cast<float>(p.pairs), loss);
}

}  // namespace taco
