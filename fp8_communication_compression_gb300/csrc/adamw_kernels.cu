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
constexpr int kBlocks = 4;                                   // blocks of 128 a warp has in flight
constexpr int kChunk = kThreads / 32 * kBlocks * 128;        // values of a chunk of the update
constexpr int kNormChunk = kThreads * 64;                    // and of the norm

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

__device__ __forceinline__ uint4 ldg16(const void *p) { return ldg128_stream(p); }

// Squares of a thread's 64 values of a whole chunk, in 16-byte loads; at most
// 32 terms in a row.
__device__ __forceinline__ float squares(const grad_tensor &d, int64_t base)
{
    const int tid = threadIdx.x;
    float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    if (d.grad_type == TACO_GRAD_FP8) {
        const uint8_t *p = static_cast<const uint8_t *>(d.grad) + base + tid * 16;
        uint4 q[4];
        float m[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            q[i] = ldg16(p + i * kThreads * 16);
            m[i] = __ldg(d.grad_scale + (base + i * kThreads * 16 + tid * 16) / 128);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t w[4] = {q[i].x, q[i].y, q[i].z, q[i].w};
            float2 t = make_float2(0.0f, 0.0f);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                float2 f;
                e4m3x2_to_f32x2(w[j / 2] >> (16 * (j % 2)) & 0xFFFFu, f.x, f.y);
                t = __ffma2_rn(f, f, t);
            }
            s[i] = (t.x + t.y) * m[i] * m[i];
        }
    } else if (d.grad_type == TACO_GRAD_BF16) {
        const uint16_t *p = static_cast<const uint16_t *>(d.grad) + base + tid * 8;
        uint4 q[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
            q[i] = ldg16(p + i * kThreads * 8);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint32_t w[4] = {q[i].x, q[i].y, q[i].z, q[i].w};
            float2 t = make_float2(s[i % 4], 0.0f);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float2 f = make_float2(bf16lo_to_f32(w[j]), bf16hi_to_f32(w[j]));
                t = __ffma2_rn(f, f, t);
            }
            s[i % 4] = t.x + t.y;
        }
    } else {
        const float *p = static_cast<const float *>(d.grad) + base + tid * 4;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            uint4 q[8];
#pragma unroll
            for (int i = 0; i < 8; ++i)
                q[i] = ldg16(p + (h * 8 + i) * kThreads * 4);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float f[4] = {__uint_as_float(q[i].x), __uint_as_float(q[i].y), __uint_as_float(q[i].z),
                                    __uint_as_float(q[i].w)};
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    s[j] = fmaf(f[j], f[j], s[j]);
            }
        }
    }
    return (s[0] + s[1]) + (s[2] + s[3]);
}

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
        const int64_t base = static_cast<int64_t>(c - t.first[i]) * kNormChunk;
        if (base + kNormChunk <= d.n) {
            sum += squares(d, base);
            continue;
        }
        for (int64_t e = base + threadIdx.x * 4; e < d.n; e += kThreads * 4) {
            const float4 g = load_grad(d.grad, d.grad_scale, d.grad_type, e, d.n);
            sum += fmaf(g.x, g.x, fmaf(g.y, g.y, fmaf(g.z, g.z, g.w * g.w)));
        }
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

struct Hyper {
    AdamWStep h;
    uint32_t key;             // of the seed
    int32_t first_tensor;     // of this launch
    int32_t last;             // the step's last launch counts it
    float b1, b2, a1, a2;     // b and 1 - b, each rounded from 64 bits
    float ln_beta1, ln_beta2;
};

__device__ __forceinline__ float2 both(float a) { return make_float2(a, a); }
__device__ __forceinline__ float2 operator*(float2 a, float2 b) { return __fmul2_rn(a, b); }
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) { return __ffma2_rn(a, b, c); }
__device__ __forceinline__ float root_of(float x)
{
    float y;
    asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float inverse(float x)
{
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Four values held by a lane.
struct F4 {
    float2 a, b;
};
__device__ __forceinline__ F4 f4(float4 x) { return {make_float2(x.x, x.y), make_float2(x.z, x.w)}; }
__device__ __forceinline__ F4 decoded(uint32_t w)
{
    F4 f;
    e4m3x2_to_f32x2(w & 0xFFFFu, f.a.x, f.a.y);
    e4m3x2_to_f32x2(w >> 16, f.b.x, f.b.y);
    return f;
}

// |x| inv, within 0 .. 448, to an E4M3 code, up with the probability of the
// rest: rest holds 16 random bits in bits 4 .. 19.  Below 2^-6 E4M3's steps are
// those of [2^-6, 2^-5), so 2^-6 is added there; the 20 low bits of the sum's
// fraction are what the code leaves out.
__device__ __forceinline__ uint32_t code_up(float x, float inv, uint32_t rest)
{
    const float y = fminf(fabsf(x) * inv, 448.0f);
    const bool low = y < 0.015625f;
    const uint32_t f = __float_as_uint(y + (low ? 0.015625f : 0.0f));
    return (f + rest + (8u - ((low ? 968u : 960u) << 20))) >> 20;
}

// Largest magnitude of a block held by a warp, as bits (those of an Inf or a
// NaN are above all others').
__device__ __forceinline__ uint32_t top_of(const F4 &x)
{
    const uint32_t m = 0x7FFFFFFFu;
    const uint32_t a = max(__float_as_uint(x.a.x) & m, __float_as_uint(x.a.y) & m);
    const uint32_t b = max(__float_as_uint(x.b.x) & m, __float_as_uint(x.b.y) & m);
    return __reduce_max_sync(~0u, max(a, b));
}
constexpr uint32_t kInf = 0x7F800000u, kLeast = 0x0D800000u;  // kLeast: 2^-100

// A block's codes; ROOT: no signs, and no code of 0 for a value above 0.
template <bool ROOT>
__device__ __forceinline__ uint32_t to_codes(const F4 &x, float inv, uint32_t top, const uint32_t (&r)[4])
{
    const float v[4] = {x.a.x, x.a.y, x.b.x, x.b.y};
    uint32_t c[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        c[j] = code_up(v[j], inv, (ROOT ? r[j] >> 12 : r[j] << 4) & 0xFFFF0u);
        if (ROOT)
            c[j] = max(c[j], min(__float_as_uint(v[j]), 1u));
    }
    uint32_t w = __byte_perm(__byte_perm(c[0], c[1], 0x0040), __byte_perm(c[2], c[3], 0x0040), 0x5410);
    if (!ROOT) {
        const uint32_t lo = __byte_perm(__float_as_uint(v[0]), __float_as_uint(v[1]), 0x0073);
        const uint32_t hi = __byte_perm(__float_as_uint(v[2]), __float_as_uint(v[3]), 0x0073);
        w |= __byte_perm(lo, hi, 0x5410) & 0x80808080u;
    }
    return top >= kInf ? 0x7F7F7F7Fu : top < kLeast ? 0u : w;
}

struct Update {
    float gs, fix2, eps, b1, b2, a1, a2, decay, rate;
};

__device__ __forceinline__ float2 updated(float2 p, float2 g, float2 &m, float2 &v, float2 &root, const Update &h)
{
    m = fma2(both(h.b1), m, both(h.a1) * g);
    v = fma2(both(h.b2), v, (both(h.a2) * g) * g);
    root = make_float2(root_of(v.x), root_of(v.y));
    const float2 d = fma2(root, both(h.fix2), both(h.eps));
    const float2 u = m * make_float2(inverse(d.x), inverse(d.y));
    const float2 t = fma2(both(h.rate), u, both(h.decay) * p);
    return __fadd2_rn(p, make_float2(-t.x, -t.y));
}

// A warp's four blocks of tensor d, from element `base` on.  All loads are
// issued first; the blocks' multipliers are loaded, inverted and stored by a
// lane each (0 .. 3: m, 4 .. 7: r, 8 .. 11: the gradient's).
template <bool BITS8>
__device__ __forceinline__ void update_blocks(const adamw_tensor &d, int64_t base, const Update &h, uint32_t key)
{
    const int lane = threadIdx.x % 32;
    const int64_t n = d.n;
    F4 g[kBlocks], p[kBlocks], m[kBlocks], v[kBlocks];
    uint32_t mc[kBlocks], vc[kBlocks];
    float scale = 1.0f;
    float *const scales = lane < kBlocks ? d.m_scale : d.v_scale;
    const int64_t mine = base / 128 + lane % kBlocks;
    const bool exists = mine * 128 < n;
    if (BITS8 && lane < 2 * kBlocks && exists)
        scale = scales[mine];
    if (d.grad_type == TACO_GRAD_FP8 && lane / kBlocks == 2 && exists)
        scale = d.grad_scale[mine];
#pragma unroll
    for (int u = 0; u < kBlocks; ++u) {
        const int64_t e = base + u * 128 + lane * 4;
        p[u] = f4(load4(d.param, e, n));
        if (BITS8) {
            mc[u] = load4(static_cast<const uint8_t *>(d.m), e, n);
            vc[u] = load4(static_cast<const uint8_t *>(d.v), e, n);
        } else {
            m[u] = f4(load4(static_cast<const float *>(d.m), e, n));
            v[u] = f4(load4(static_cast<const float *>(d.v), e, n));
        }
    }
    if (d.grad_type == TACO_GRAD_FP8) {
        uint32_t gc[kBlocks];
#pragma unroll
        for (int u = 0; u < kBlocks; ++u)
            gc[u] = load4(static_cast<const uint8_t *>(d.grad), base + u * 128 + lane * 4, n);
#pragma unroll
        for (int u = 0; u < kBlocks; ++u) {
            const float2 s = both(__shfl_sync(~0u, scale, 2 * kBlocks + u));
            const F4 c = decoded(gc[u]);
            g[u] = {c.a * s, c.b * s};
        }
    } else if (d.grad_type == TACO_GRAD_BF16) {
#pragma unroll
        for (int u = 0; u < kBlocks; ++u) {
            const uint2 w = load4(static_cast<const uint16_t *>(d.grad), base + u * 128 + lane * 4, n);
            g[u] = {make_float2(bf16lo_to_f32(w.x), bf16hi_to_f32(w.x)),
                    make_float2(bf16lo_to_f32(w.y), bf16hi_to_f32(w.y))};
        }
    } else {
#pragma unroll
        for (int u = 0; u < kBlocks; ++u)
            g[u] = f4(load4(static_cast<const float *>(d.grad), base + u * 128 + lane * 4, n));
    }
    F4 root[kBlocks];
    uint32_t top = 0, tops[2 * kBlocks];
#pragma unroll
    for (int u = 0; u < kBlocks; ++u) {
        const int64_t e = base + u * 128 + lane * 4;
        if (BITS8) {
            const float2 ms = both(__shfl_sync(~0u, scale, u)), vs = both(__shfl_sync(~0u, scale, kBlocks + u));
            m[u] = decoded(mc[u]), v[u] = decoded(vc[u]);
            m[u] = {m[u].a * ms, m[u].b * ms}, v[u] = {v[u].a * vs, v[u].b * vs};
            v[u] = {v[u].a * v[u].a, v[u].b * v[u].b};
        }
        g[u] = {g[u].a * both(h.gs), g[u].b * both(h.gs)};
        p[u].a = updated(p[u].a, g[u].a, m[u].a, v[u].a, root[u].a, h);
        p[u].b = updated(p[u].b, g[u].b, m[u].b, v[u].b, root[u].b, h);
        store4(d.param, e, n, make_float4(p[u].a.x, p[u].a.y, p[u].b.x, p[u].b.y));
        if (d.copy_bf16)
            store4(static_cast<uint16_t *>(d.copy_bf16), e, n,
                   make_uint2(f32x2_to_bf16x2(p[u].a.x, p[u].a.y), f32x2_to_bf16x2(p[u].b.x, p[u].b.y)));
        if (!BITS8) {
            store4(static_cast<float *>(d.m), e, n, make_float4(m[u].a.x, m[u].a.y, m[u].b.x, m[u].b.y));
            store4(static_cast<float *>(d.v), e, n, make_float4(v[u].a.x, v[u].a.y, v[u].b.x, v[u].b.y));
        } else {
            tops[u] = top_of(m[u]), tops[kBlocks + u] = top_of(root[u]);
            top = lane == u ? tops[u] : lane == kBlocks + u ? tops[kBlocks + u] : top;
        }
    }
    if (!BITS8)
        return;
    const bool none = top < kLeast, bad = top >= kInf;  // (448 / amax would leave fp32's range)
    const float inv = none || bad ? 0.0f : 448.0f / __uint_as_float(top);
    if (lane < 2 * kBlocks && exists)
        scales[mine] = none || bad ? 1.0f : __uint_as_float(top) / 448.0f;
#pragma unroll
    for (int u = 0; u < kBlocks; ++u) {
        const int64_t e = base + u * 128 + lane * 4;
        uint32_t r[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
            r[j] = mix((static_cast<uint32_t>(e + j) * 0x13198A2Fu) ^ key);
        store4(static_cast<uint8_t *>(d.m), e, n,
               to_codes<false>(m[u], __shfl_sync(~0u, inv, u), tops[u], r));
        store4(static_cast<uint8_t *>(d.v), e, n,
               to_codes<true>(root[u], __shfl_sync(~0u, inv, kBlocks + u), tops[kBlocks + u], r));
    }
}

template <bool BITS8, int MAX>
__global__ void __launch_bounds__(kThreads)
    adamw_kernel(const __grid_constant__ Table<adamw_tensor, MAX> t, const __grid_constant__ Hyper hyper)
{
    pdl_wait();
    const AdamWStep &s = hyper.h;
    const uint64_t steps = static_cast<uint64_t>(s.state[0]);
    Update h;
    h.gs = s.grad_scale;
    if (s.norm) {
        const float norm = *s.norm;
        if (!(norm <= FLT_MAX))  // a gradient that is not finite: the step is left out
            return;
        if (s.max_norm > 0.0f)
            h.gs *= fminf(s.max_norm / (norm + 1e-6f), 1.0f);
    }
    const float time = static_cast<float>(steps + 1);
    const float fix1 = -1.0f / expm1f(time * hyper.ln_beta1);
    h.fix2 = rsqrtf(-expm1f(time * hyper.ln_beta2));
    h.eps = s.eps, h.b1 = hyper.b1, h.b2 = hyper.b2, h.a1 = hyper.a1, h.a2 = hyper.a2;
    const float factor = s.lr_factor ? *s.lr_factor : 1.0f;
    const int chunks = t.first[t.count];
    for (int c = blockIdx.x; c < chunks; c += gridDim.x) {
        const int i = tensor_of(t, c);
        const adamw_tensor &d = t.tensor[i];
        const int64_t base = static_cast<int64_t>(c - t.first[i]) * kChunk + threadIdx.x / 32 * (kBlocks * 128);
        if (base >= d.n)
            continue;
        const float lr = d.lr * factor;
        h.decay = lr * d.weight_decay, h.rate = lr * fix1;
        uint32_t key = 0;
        if (BITS8) {
            key = mix(mix(hyper.key ^ static_cast<uint32_t>(steps)) ^ static_cast<uint32_t>(hyper.first_tensor + i));
            if (base >> 32)
                key = mix(key ^ static_cast<uint32_t>(base >> 32));
        }
        update_blocks<BITS8>(d, base, h, key);
    }
    // the last CTA of the step counts it: every CTA has read the count by then
    if (hyper.last) {
        __syncthreads();
        if (threadIdx.x == 0) {
            unsigned int *ticket = reinterpret_cast<unsigned int *>(s.state + 1);
            if (atomicAdd(ticket, 1u) == gridDim.x - 1) {
                *ticket = 0;
                s.state[0] = static_cast<int64_t>(steps + 1);
            }
        }
    }
}

template <typename D, int MAX> int fill(Table<D, MAX> &t, const D *tensors, int64_t count, int chunk)
{
    t.count = static_cast<int32_t>(count);
    int64_t at = 0;
    for (int64_t i = 0; i < count; ++i) {
        t.tensor[i] = tensors[i];
        t.first[i] = static_cast<int32_t>(at);
        at += (tensors[i].n + chunk - 1) / chunk;
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
    const int chunks = fill(t, tensors, count, kNormChunk);
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
    const int chunks = fill(t, tensors, count, kChunk);
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
