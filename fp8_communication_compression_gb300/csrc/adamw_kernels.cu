// The optimizer: the norm of all gradients, and AdamW over many tensors.
//
//   g <- grad_scale min(1, max_norm / (norm + 1e-6)) grad
//   m <- b1 m + (1 - b1) g,  v <- b2 v + (1 - b2) g^2
//   p <- p - lr (wd p + (m / (1 - b1^t)) / (sqrt(v / (1 - b2^t)) + eps))
//
// Gradients are fp32, bf16, or FP8 main gradients (E4M3 codes, one fp32
// multiplier per block of 128), each tensor's by itself.  Weights are fp32,
// with an optional bf16 copy.  m and v are fp32, or in 8 bits: E4M3 codes of m
// and of r = sqrt(v) with a multiplier amax / 448 per block of 128 (the main
// gradients' format).  r and not v, as its range is half of v's in powers of
// two.  With steps of a sixteenth to an eighth, the change of one update is
// mostly less than half a step, and rounding to nearest would lose it for
// good; the codes are rounded up with the probability of the rest, by 16 bits
// of a hash of the element, its tensor, the step and a seed, so that they
// follow on average.  r's code is at least 1 where v > 0: a zero would divide
// m by eps alone in the next step.
//
// A launch takes its tensors' descriptions as parameters, so that nothing is
// copied or kept, and finds the tensor of each chunk by bisection.  Bound by
// HBM; a lane takes four consecutive elements, a warp one block of 128, whose
// maximum is one warp reduction.

#include "device_utils.cuh"
#include "internal.h"

#include <cfloat>
#include <cmath>
#include <cstring>

namespace taco {

namespace {

constexpr int kThreads = 256;
constexpr int kUnroll = 4;                                   // blocks of 128 a warp has in flight
constexpr int kChunk = kThreads / 32 * kUnroll * 128;        // elements of a chunk

// Tensors of a launch; first[i]: the first chunk of tensor i.
template <typename D, int MAX> struct Table {
    D tensor[MAX];
    int32_t first[MAX + 1];
    int32_t count;
};

template <typename D, int MAX> __device__ __forceinline__ int tensor_of(const Table<D, MAX> &t, int chunk)
{
    int lo = 0, hi = t.count;  // first[lo] <= chunk < first[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (t.first[mid] <= chunk)
            lo = mid;
        else
            hi = mid;
    }
    return lo;
}

// Elements e .. e + 3 of n, zeros past the end.
__device__ __forceinline__ float4 load4(const float *p, int64_t e, int64_t n)
{
    if (e + 4 <= n)
        return *reinterpret_cast<const float4 *>(p + e);
    return make_float4(e < n ? p[e] : 0.0f, e + 1 < n ? p[e + 1] : 0.0f, e + 2 < n ? p[e + 2] : 0.0f, 0.0f);
}
__device__ __forceinline__ uint32_t load4(const uint8_t *p, int64_t e, int64_t n)
{
    if (e + 4 <= n)
        return *reinterpret_cast<const uint32_t *>(p + e);
    uint32_t w = 0;
    for (int j = 0; j < 3; ++j)
        w |= e + j < n ? uint32_t(p[e + j]) << (8 * j) : 0u;
    return w;
}
__device__ __forceinline__ uint2 load4(const uint16_t *p, int64_t e, int64_t n)
{
    if (e + 4 <= n)
        return *reinterpret_cast<const uint2 *>(p + e);
    return make_uint2((e < n ? p[e] : 0u) | (e + 1 < n ? uint32_t(p[e + 1]) << 16 : 0u), e + 2 < n ? p[e + 2] : 0u);
}
__device__ __forceinline__ void store4(float *p, int64_t e, int64_t n, float4 v)
{
    if (e + 4 <= n) {
        *reinterpret_cast<float4 *>(p + e) = v;
    } else {
        if (e < n)
            p[e] = v.x;
        if (e + 1 < n)
            p[e + 1] = v.y;
        if (e + 2 < n)
            p[e + 2] = v.z;
    }
}
__device__ __forceinline__ void store4(uint8_t *p, int64_t e, int64_t n, uint32_t w)
{
    if (e + 4 <= n)
        *reinterpret_cast<uint32_t *>(p + e) = w;
    else
        for (int j = 0; j < 3; ++j)
            if (e + j < n)
                p[e + j] = static_cast<uint8_t>(w >> (8 * j));
}
__device__ __forceinline__ void store4(uint16_t *p, int64_t e, int64_t n, uint2 w)
{
    if (e + 4 <= n) {
        *reinterpret_cast<uint2 *>(p + e) = w;
    } else {
        if (e < n)
            p[e] = static_cast<uint16_t>(w.x);
        if (e + 1 < n)
            p[e + 1] = static_cast<uint16_t>(w.x >> 16);
        if (e + 2 < n)
            p[e + 2] = static_cast<uint16_t>(w.y);
    }
}

__device__ __forceinline__ float4 from_codes(uint32_t w, float s)
{
    float4 f;
    e4m3x2_to_f32x2(w & 0xFFFFu, f.x, f.y);
    e4m3x2_to_f32x2(w >> 16, f.z, f.w);
    return make_float4(f.x * s, f.y * s, f.z * s, f.w * s);
}

__device__ __forceinline__ float4 load_grad(const void *g, const float *scale, int type, int64_t e, int64_t n)
{
    if (type == TACO_GRAD_F32)
        return load4(static_cast<const float *>(g), e, n);
    if (type == TACO_GRAD_BF16) {
        const uint2 w = load4(static_cast<const uint16_t *>(g), e, n);
        return make_float4(bf16lo_to_f32(w.x), bf16hi_to_f32(w.x), bf16lo_to_f32(w.y), bf16hi_to_f32(w.y));
    }
    return e < n ? from_codes(load4(static_cast<const uint8_t *>(g), e, n), scale[e / 128])
                 : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
}

// ------------------------------------------------------------------- norm --

// Sum of squares of a CTA's chunks, into partial[blockIdx.x].
template <int MAX>
__global__ void __launch_bounds__(kThreads) norm_kernel(const __grid_constant__ Table<grad_tensor, MAX> t,
                                                        double *partial)
{
    __shared__ double part[kThreads / 32];
    pdl_wait();
    double sum = 0.0;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, chunks = t.first[t.count];
    for (int c = blockIdx.x; c < chunks; c += gridDim.x) {
        const int i = tensor_of(t, c);
        const grad_tensor &d = t.tensor[i];
        const int64_t base = static_cast<int64_t>(c - t.first[i]) * kChunk + warp * kUnroll * 128 + lane * 4;
        float s = 0.0f;
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const float4 g = load_grad(d.grad, d.grad_scale, d.grad_type, base + u * 128, d.n);
            s = fmaf(g.x, g.x, fmaf(g.y, g.y, fmaf(g.z, g.z, fmaf(g.w, g.w, s))));
        }
        sum += s;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        sum += __shfl_xor_sync(~0u, sum, o);
    if (lane == 0)
        part[warp] = sum;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int w = 1; w < kThreads / 32; ++w)
            sum += part[w];
        partial[blockIdx.x] = sum;
    }
}

__global__ void __launch_bounds__(kThreads) norm_total_kernel(const double *partial, int n, float scale, float *norm)
{
    __shared__ double part[kThreads / 32];
    pdl_wait();
    double sum = 0.0;
    for (int i = threadIdx.x; i < n; i += kThreads)
        sum += partial[i];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        sum += __shfl_xor_sync(~0u, sum, o);
    if (threadIdx.x % 32 == 0)
        part[threadIdx.x / 32] = sum;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int w = 1; w < kThreads / 32; ++w)
            sum += part[w];
        *norm = static_cast<float>(sqrt(sum) * fabsf(scale));
    }
}

// ------------------------------------------------------------------ AdamW --

// A hash of 32 bits: two rounds of shift, xor and multiplication (golden
// ratio, and digits of pi).  Uniformity and independence of neighbouring
// elements, steps and halves are tested on the host.
__host__ __device__ __forceinline__ uint32_t mix(uint32_t x)
{
    x = (x ^ (x >> 16)) * 0x9E3779B1u;
    x = (x ^ (x >> 15)) * 0x85A308D3u;
    return x ^ (x >> 16);
}

// |x| scaled into 0 .. 448, to an E4M3 code, up with the probability of the
// rest: bits (0 .. 65535) and a half of 65536.  Below 2^-6 E4M3's steps are
// those of [2^-6, 2^-5), so 2^-6 is added there; above, the fraction's 20 low
// bits are what the code leaves out.
__device__ __forceinline__ uint32_t code_up(float y, uint32_t bits)
{
    const bool low = y < 0.015625f;
    const uint32_t f = __float_as_uint(low ? y + 0.015625f : y);
    return ((f + (bits << 4) + 8u) >> 20) - (low ? 968u : 960u);
}

struct Hyper {
    AdamWStep h;
    uint32_t key;             // of the seed
    int32_t first_tensor;     // of this launch
    int32_t last;             // the step's last launch counts it
    float b1, b2, a1, a2;     // b and 1 - b, each rounded from 64 bits
    float ln_beta1, ln_beta2;
};

// Codes and multiplier of a block held by a warp, four values a lane.
template <bool LEAST>
__device__ __forceinline__ uint32_t to_codes(const float (&x)[4], const uint32_t (&bits)[4], float &scale)
{
    float top = fmaxf(fmaxf(fabsf(x[0]), fabsf(x[1])), fmaxf(fabsf(x[2]), fabsf(x[3])));
    bool bad = false;
#pragma unroll
    for (int j = 0; j < 4; ++j)
        bad |= !(fabsf(x[j]) <= FLT_MAX);
    top = __uint_as_float(__reduce_max_sync(~0u, __float_as_uint(top)));
    if (__any_sync(~0u, bad)) {  // an Inf or a NaN: the block is NaN
        scale = 1.0f;
        return 0x7F7F7F7Fu;
    }
    const bool none = top < 0x1p-100f;  // (448 / amax would leave fp32's range)
    scale = none ? 1.0f : top / 448.0f;
    const float inv = none ? 0.0f : 448.0f / top;
    uint32_t w = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        uint32_t c = code_up(fminf(fabsf(x[j]) * inv, 448.0f), bits[j]);
        if (LEAST)
            c = c == 0 && x[j] > 0.0f && !none ? 1u : c;
        else
            c |= (__float_as_uint(x[j]) >> 24) & 0x80u;
        w |= c << (8 * j);
    }
    return w;
}

template <bool BITS8, int MAX>
__global__ void __launch_bounds__(kThreads)
    adamw_kernel(const __grid_constant__ Table<adamw_tensor, MAX> t, const __grid_constant__ Hyper hyper)
{
    pdl_wait();
    const AdamWStep &h = hyper.h;
    const uint64_t steps = static_cast<uint64_t>(h.state[0]);
    float gs = h.grad_scale;
    bool skip = false;
    if (h.norm) {
        const float norm = *h.norm;
        skip = !(norm <= FLT_MAX);  // a gradient that is not finite: the step is left out
        if (h.max_norm > 0.0f)
            gs *= fminf(h.max_norm / (norm + 1e-6f), 1.0f);
    }
    if (skip)
        return;
    const float time = static_cast<float>(steps + 1);
    const float fix1 = -1.0f / expm1f(time * hyper.ln_beta1);
    const float fix2 = rsqrtf(-expm1f(time * hyper.ln_beta2));
    const float factor = h.lr_factor ? *h.lr_factor : 1.0f;
    const float b1 = hyper.b1, b2 = hyper.b2, a1 = hyper.a1, a2 = hyper.a2;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, chunks = t.first[t.count];
    for (int c = blockIdx.x; c < chunks; c += gridDim.x) {
        const int i = tensor_of(t, c);
        const adamw_tensor &d = t.tensor[i];
        const int64_t n = d.n;
        const int64_t base = static_cast<int64_t>(c - t.first[i]) * kChunk + warp * kUnroll * 128;
        const float lr = d.lr * factor, decay = lr * d.weight_decay, rate = lr * fix1;
        uint32_t key = 0;
        if (BITS8) {
            key = mix(mix(hyper.key ^ static_cast<uint32_t>(steps)) ^ static_cast<uint32_t>(hyper.first_tensor + i));
            if (base >> 32)
                key = mix(key ^ static_cast<uint32_t>(base >> 32));
        }
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int64_t block = base + u * 128, e = block + lane * 4;
            if (block >= n)
                break;
            const float4 g4 = load_grad(d.grad, d.grad_scale, d.grad_type, e, n);
            const float4 p4 = load4(d.param, e, n);
            float4 m4, v4;
            if (BITS8) {
                m4 = from_codes(load4(static_cast<const uint8_t *>(d.m), e, n), d.m_scale[block / 128]);
                v4 = from_codes(load4(static_cast<const uint8_t *>(d.v), e, n), d.v_scale[block / 128]);
                v4 = make_float4(v4.x * v4.x, v4.y * v4.y, v4.z * v4.z, v4.w * v4.w);
            } else {
                m4 = load4(static_cast<const float *>(d.m), e, n);
                v4 = load4(static_cast<const float *>(d.v), e, n);
            }
            const float g[4] = {g4.x * gs, g4.y * gs, g4.z * gs, g4.w * gs};
            float p[4] = {p4.x, p4.y, p4.z, p4.w}, m[4] = {m4.x, m4.y, m4.z, m4.w}, v[4] = {v4.x, v4.y, v4.z, v4.w};
            float root[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                m[j] = b1 * m[j] + a1 * g[j];
                v[j] = b2 * v[j] + a2 * g[j] * g[j];
                root[j] = sqrtf(v[j]);
                p[j] -= decay * p[j] + rate * __fdividef(m[j], root[j] * fix2 + h.eps);
            }
            store4(d.param, e, n, make_float4(p[0], p[1], p[2], p[3]));
            if (d.copy_bf16)
                store4(static_cast<uint16_t *>(d.copy_bf16), e, n,
                       make_uint2(f32x2_to_bf16x2(p[0], p[1]), f32x2_to_bf16x2(p[2], p[3])));
            if (BITS8) {
                uint32_t lo[4], hi[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const uint32_t r = mix((static_cast<uint32_t>(e + j) * 0x13198A2Fu) ^ key);
                    lo[j] = r & 0xFFFFu;
                    hi[j] = r >> 16;
                }
                float ms, vs;
                const uint32_t mc = to_codes<false>(m, lo, ms), vc = to_codes<true>(root, hi, vs);
                store4(static_cast<uint8_t *>(d.m), e, n, mc);
                store4(static_cast<uint8_t *>(d.v), e, n, vc);
                if (lane == 0) {
                    d.m_scale[block / 128] = ms;
                    d.v_scale[block / 128] = vs;
                }
            } else {
                store4(static_cast<float *>(d.m), e, n, make_float4(m[0], m[1], m[2], m[3]));
                store4(static_cast<float *>(d.v), e, n, make_float4(v[0], v[1], v[2], v[3]));
            }
        }
    }
    // the last CTA of the step counts it: every CTA has read the count by then
    if (hyper.last) {
        __syncthreads();
        if (threadIdx.x == 0) {
            unsigned int *ticket = reinterpret_cast<unsigned int *>(h.state + 1);
            if (atomicAdd(ticket, 1u) == gridDim.x - 1) {
                *ticket = 0;
                h.state[0] = static_cast<int64_t>(steps + 1);
            }
        }
    }
}

template <typename D, int MAX> int fill(Table<D, MAX> &t, const D *tensors, int64_t count)
{
    t.count = static_cast<int32_t>(count);
    int64_t at = 0;
    for (int64_t i = 0; i < count; ++i) {
        t.tensor[i] = tensors[i];
        t.first[i] = static_cast<int32_t>(at);
        at += (tensors[i].n + kChunk - 1) / kChunk;
    }
    t.first[count] = static_cast<int32_t>(at);
    return static_cast<int>(at);
}

template <typename K> cudaError_t resident(K kernel, int *grid)
{
    DeviceInfo di;
    cudaError_t e = current_device_info(&di);
    int per_sm = 0;
    if (e == cudaSuccess)
        e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kernel, kThreads, 0);
    *grid = di.num_sms * (per_sm < 1 ? 1 : per_sm);
    return e;
}

constexpr int kNormGrid = 2048;  // partial sums of a launch (at most)

template <int MAX>
cudaError_t norm_launch(const grad_tensor *tensors, int64_t count, double *partial, int *used, cudaStream_t stream)
{
    Table<grad_tensor, MAX> t;
    const int chunks = fill(t, tensors, count);
    int grid = 0;
    cudaError_t e = resident(norm_kernel<MAX>, &grid);
    if (e != cudaSuccess)
        return e;
    grid = grid < kNormGrid ? grid : kNormGrid;
    grid = grid < chunks ? grid : chunks < 1 ? 1 : chunks;
    *used = grid;
    return launch_pdl(norm_kernel<MAX>, grid, kThreads, 0, stream, t, partial);
}

template <bool BITS8, int MAX>
cudaError_t adamw_launch(const adamw_tensor *tensors, int64_t count, const Hyper &h, cudaStream_t stream)
{
    Table<adamw_tensor, MAX> t;
    const int chunks = fill(t, tensors, count);
    int grid = 0;
    cudaError_t e = resident(adamw_kernel<BITS8, MAX>, &grid);
    if (e != cudaSuccess)
        return e;
    grid = grid < chunks ? grid : chunks < 1 ? 1 : chunks;
    return launch_pdl(adamw_kernel<BITS8, MAX>, grid, kThreads, 0, stream, t, h);
}

}  // namespace

int grad_norm_launches(int64_t count) { return static_cast<int>((count + kNormTensors - 1) / kNormTensors); }

cudaError_t grad_norm_workspace(int64_t count, uint64_t *bytes)
{
    *bytes = static_cast<uint64_t>(grad_norm_launches(count)) * kNormGrid * sizeof(double);
    return cudaSuccess;
}

cudaError_t launch_grad_norm(const grad_tensor *tensors, int64_t count, float grad_scale, float *norm,
                             void *workspace, cudaStream_t stream)
{
    double *partial = static_cast<double *>(workspace);
    int total = 0;
    for (int64_t i = 0; i < count; i += kNormTensors) {
        const int64_t n = count - i < kNormTensors ? count - i : kNormTensors;
        int used = 0;
        const cudaError_t e = n <= 32 ? norm_launch<32>(tensors + i, n, partial + total, &used, stream)
                                      : norm_launch<kNormTensors>(tensors + i, n, partial + total, &used, stream);
        if (e != cudaSuccess)
            return e;
        total += used;
    }
    return launch_pdl(norm_total_kernel, 1, kThreads, 0, stream, static_cast<const double *>(partial), total,
                      grad_scale, norm);
}

cudaError_t launch_adamw(const adamw_tensor *tensors, int64_t count, bool bits8, const AdamWStep &step,
                         cudaStream_t stream)
{
    Hyper h;
    h.h = step;
    h.key = mix(mix(static_cast<uint32_t>(step.seed)) ^ static_cast<uint32_t>(step.seed >> 32));
    h.b1 = static_cast<float>(step.beta1), h.a1 = static_cast<float>(1.0 - step.beta1);
    h.b2 = static_cast<float>(step.beta2), h.a2 = static_cast<float>(1.0 - step.beta2);
    h.ln_beta1 = static_cast<float>(std::log(step.beta1));
    h.ln_beta2 = static_cast<float>(std::log(step.beta2));
    int64_t i = 0;
    do {
        const int64_t n = count - i < kAdamWTensors ? count - i : kAdamWTensors;
        h.first_tensor = static_cast<int32_t>(i);
        h.last = i + n == count;
        cudaError_t e;
        if (n <= 16)
            e = bits8 ? adamw_launch<true, 16>(tensors + i, n, h, stream)
                      : adamw_launch<false, 16>(tensors + i, n, h, stream);
        else
            e = bits8 ? adamw_launch<true, kAdamWTensors>(tensors + i, n, h, stream)
                      : adamw_launch<false, kAdamWTensors>(tensors + i, n, h, stream);
        if (e != cudaSuccess)
            return e;
        i += n;
    } while (i < count);
    return cudaSuccess;
}

}  // namespace taco
