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
//
// Bound by HBM.  The forward pass streams a row through registers.  Where the
// gradient is wanted too, a row's granules come by bulk copies into shared
// memory, are summed as they arrive, and are read again from there once the
// sum is known: the logits cross the memory once.  A cluster of CTAs shares a
// row that is long, or whose kind is few, and adds its parts' sums through
// distributed shared memory.

#include "device_utils.cuh"
#include "internal.h"

#include <cfloat>
#include <cstring>

namespace taco {

// Watchdog flag of this file's kernels (bit 8), read by taco_device_error().
__device__ unsigned int g_loss_error;

namespace {

constexpr uint32_t kErrLoss = 256u;
// log2 e = kLog2e + kLog2eLow: with one rounded factor alone all differences
// would be scaled wrongly by the same 2^-26, and so would a sequence's sum.
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLog2eLow = static_cast<float>(1.4426950408889634074 - static_cast<double>(kLog2e));
constexpr float kLn2 = 0.6931471805599453f;
constexpr int kMaxCluster = 8;
constexpr int kChunkSteps = 2;  // granules a thread takes from a chunk in shared memory
constexpr int kMaxChunks = 64;

enum Mode { kForward, kPolicy };

__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float neg_inf() { return __int_as_float(0xFF800000); }
__device__ __forceinline__ float quiet_nan() { return __int_as_float(0x7FFFFFFF); }
__device__ __forceinline__ float2 both(float a) { return make_float2(a, a); }

// The granules of one row: G elements each, of type E (bf16 as uint16_t, or
// float).  Granules first .. last - 1 hold nothing but values of the row's V
// columns; of those before and behind, single elements may be the row's.
template <typename E> struct Row {
    static constexpr int G = 16 / sizeof(E);
    const E *x;      // granule 0; the row starts `shift` elements in
    int shift;
    int first, last; // interior
    int end;         // behind the granule with the last of the N columns
    int64_t left;    // elements from x to the end of the tensor
    int V, N;

    __device__ Row(const LossRows &a, int64_t row)
    {
        const int64_t at = row * a.N;
        V = static_cast<int>(a.V), N = static_cast<int>(a.N);
        shift = static_cast<int>(at & (G - 1));
        x = static_cast<const E *>(a.logits) + (at - shift);
        left = a.T * a.N - (at - shift);
        first = shift ? 1 : 0;
        last = static_cast<int>((static_cast<int64_t>(shift) + V) / G);
        last = last < first ? first : last;
        end = static_cast<int>((static_cast<int64_t>(shift) + N + G - 1) / G);
    }

    __device__ uint4 load(int k) const
    {
        uint4 v;
        asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                     : "l"(x + static_cast<int64_t>(k) * G));
        return v;
    }
    // Element j of granule k is column col(k, j).
    __device__ int64_t col(int k, int j) const { return static_cast<int64_t>(k) * G + j - shift; }
    // A granule at a row's end, element by element: `other` in places of no
    // column of the vocabulary.
    __device__ void load_edge(int k, float other, float (&f)[G]) const
    {
#pragma unroll
        for (int j = 0; j < G; ++j) {
            const int64_t c = col(k, j);
            f[j] = c >= 0 && c < V ? element(x + static_cast<int64_t>(k) * G + j) : other;
        }
    }
    static __device__ __forceinline__ float element(const uint16_t *p) { return __uint_as_float(uint32_t(*p) << 16); }
    static __device__ __forceinline__ float element(const float *p) { return *p; }
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

// exp2 of (x - m) log2(e) / tau for two values.
struct Scale {
    float hi, lo;  // log2(e) / tau
    float inv_temperature;
    __device__ explicit Scale(float inv) : hi(inv * kLog2e), inv_temperature(inv)
    {
        lo = fmaf(inv, kLog2e, -hi) + inv * kLog2eLow;
    }
    __device__ __forceinline__ float2 exponent(float2 x, float2 minus_m) const
    {
        const float2 d = __fadd2_rn(x, minus_m);
        return __ffma2_rn(d, both(lo), __fmul2_rn(d, both(hi)));
    }
    __device__ __forceinline__ float exponent(float x, float m) const
    {
        const float d = x - m;
        return fmaf(d, lo, d * hi);
    }
};

// A maximum and a sum relative to it.
struct Sum {
    float m, s;
};
__device__ __forceinline__ Sum join(Sum a, Sum b, const Scale &c)
{
    const float m = fmaxf(a.m, b.m);
    return {m, a.s * ex2(c.exponent(a.m, m)) + b.s * ex2(c.exponent(b.m, m))};
}

// Adds n values (n even).
template <int n> __device__ __forceinline__ void accumulate(Sum &z, const float (&f)[n], const Scale &c)
{
    float m = fmaxf(f[0], f[1]);
#pragma unroll
    for (int j = 2; j < n; j += 2)
        m = fmaxf(m, fmaxf(f[j], f[j + 1]));
    if (m > z.m) {
        z.s *= ex2(c.exponent(z.m, m));
        z.m = m;
    }
    const float2 minus = both(-z.m);
    float2 s[2] = {make_float2(z.s, 0.0f), make_float2(0.0f, 0.0f)};
#pragma unroll
    for (int j = 0; j < n; j += 2) {
        const float2 y = c.exponent(make_float2(f[j], f[j + 1]), minus);
        s[j / 2 % 2] = __fadd2_rn(s[j / 2 % 2], make_float2(ex2(y.x), ex2(y.y)));
    }
    s[0] = __fadd2_rn(s[0], s[1]);
    z.s = s[0].x + s[0].y;
}

__device__ __forceinline__ uint32_t cluster_rank()
{
    uint32_t r;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

// The sum of CTA `rank` of the cluster at the same place of its shared memory.
__device__ __forceinline__ Sum remote(const Sum *mine, uint32_t rank)
{
    uint32_t at;
    Sum z;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_u32(mine)), "r"(rank));
    asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(z.m), "=f"(z.s) : "r"(at) : "memory");
    return z;
}

// Writes the gradient coef (1[target] - inv exp2(x - ref)) of a row: what all
// of it takes.
template <typename E> struct Gradient {
    static constexpr int G = Row<E>::G;
    const Row<E> &x;
    const Scale &c;
    E *out;             // as Row::x
    float coef, scaled; // coef and -coef inv
    float minus;        // -ref
    int64_t target;
    int at;             // the target's granule

    __device__ Gradient(const Row<E> &row, const LossRows &a, const Scale &scale, float k, float inv, float ref,
                        int64_t token)
        : x(row), c(scale), out(static_cast<E *>(a.dlogits) + (row.x - static_cast<const E *>(a.logits))),
          coef(k * a.inv_temperature), scaled(-coef * inv), minus(-ref), target(token),
          at(static_cast<int>((token + row.shift) / G))
    {
    }
    __device__ __forceinline__ void compute(const float (&f)[G], int k, float (&d)[G]) const
    {
#pragma unroll
        for (int j = 0; j < G; j += 2) {
            const float2 y = c.exponent(make_float2(f[j], f[j + 1]), both(minus));
            const float2 e = __fmul2_rn(make_float2(ex2(y.x), ex2(y.y)), both(scaled));
            d[j] = e.x, d[j + 1] = e.y;
        }
        if (k == at) {
#pragma unroll
            for (int j = 0; j < G; ++j)
                if (x.col(k, j) == target)
                    d[j] += coef;
        }
    }
    __device__ __forceinline__ void interior(int k, const uint4 &q) const
    {
        float f[G], d[G];
        values(q, f);
        compute(f, k, d);
        stg128_stream(out + static_cast<int64_t>(k) * G, packed(d));
    }
    // A granule that is not all the vocabulary's: zeros behind it, nothing
    // outside the row.  zero: the whole row is.
    __device__ void edge(int k, bool zero) const
    {
        float f[G], d[G];
        if (!zero) {
            x.load_edge(k, neg_inf(), f);
            compute(f, k, d);
        }
#pragma unroll
        for (int j = 0; j < G; ++j)
            d[j] = zero || x.col(k, j) >= x.V ? 0.0f : d[j];
        store(k, d);
    }
    __device__ __forceinline__ void store(int k, const float (&d)[G]) const
    {
        const uint4 q = packed(d);
        E *p = out + static_cast<int64_t>(k) * G;
        if (x.col(k, 0) >= 0 && x.col(k, G) <= x.N) {
            stg128_stream(p, q);
            return;
        }
        E e[G];
        memcpy(e, &q, 16);
#pragma unroll
        for (int j = 0; j < G; ++j)
            if (x.col(k, j) >= 0 && x.col(k, j) < x.N)
                p[j] = e[j];
    }
};

// One row a cluster of `parts` CTAs (1: no cluster).  RESIDENT: the part of
// the row is kept in shared memory between the passes.
template <typename E, int MODE, bool CLUSTER, bool RESIDENT>
__global__ void __launch_bounds__(512) row_kernel(const __grid_constant__ LossRows a, int parts, int chunks, int trigger)
{
    constexpr int G = Row<E>::G;
    extern __shared__ __align__(128) uint4 held[];
    __shared__ Sum part[16], mine;
    __shared__ __align__(8) uint64_t bars[kMaxChunks];
    const int tid = threadIdx.x, threads = blockDim.x, lane = tid & 31;
    const int rank = CLUSTER ? static_cast<int>(cluster_rank()) : 0;
    if (trigger)
        pdl_trigger();
    if (RESIDENT && tid == 0) {
        for (int i = 0; i < chunks; ++i)
            mbar_init(smem_u32(&bars[i]), 1);
        fence_barrier_init();
    }
    if (RESIDENT)
        __syncthreads();
    pdl_wait();
    const int64_t row = CLUSTER ? blockIdx.x / parts : blockIdx.x;
    const Row<E> x(a, row);
    const int64_t target = a.targets[row];
    float weight = 1.0f;
    bool active = target >= 0;
    if (MODE == kPolicy) {
        weight = a.weights[row];
        active = active && weight != 0.0f;
    }
    if (MODE == kForward && a.offsets)
        active = active && row >= a.offsets[0] && row < a.offsets[a.sequences];
    // this CTA's interior granules
    const int each = (x.last - x.first + parts - 1) / parts;
    const int lo = min(x.last, x.first + rank * each), hi = min(x.last, lo + each);
    const Scale c(a.inv_temperature);
    Sum z = {-FLT_MAX, 0.0f};
    float coef = 0.0f, inv = 0.0f;
    if (active) {
        float xa = 0.0f, adv = 0.0f, old = 0.0f, ref_logp = 0.0f;
        xa = target < x.V ? Row<E>::element(x.x + x.shift + target) : quiet_nan();
        if (MODE == kPolicy) {
            adv = a.advantages[row], old = a.old_logp[row];
            ref_logp = a.ref_logp ? a.ref_logp[row] : 0.0f;
        }
        if (RESIDENT) {
            const int chunk = threads * kChunkSteps;
            if (tid == 0) {
                for (int i = 0, k = lo; k < hi; ++i, k += chunk) {
                    const uint32_t bytes = static_cast<uint32_t>(min(chunk, hi - k)) * 16, bar = smem_u32(&bars[i]);
                    mbar_arrive_expect_tx(bar, bytes);
                    bulk_load(smem_u32(held + (k - lo)), x.x + static_cast<int64_t>(k) * G, bytes, bar);
                }
            }
            for (int i = 0, k = lo; k < hi; ++i, k += chunk) {
                if (!mbar_wait(smem_u32(&bars[i]), 0) && lane == 0)
                    atomicOr(&g_loss_error, kErrLoss);
#pragma unroll
                for (int j = 0; j < kChunkSteps; ++j) {
                    const int g = k + tid + j * threads;
                    if (g < hi) {
                        float f[G];
                        values(held[g - lo], f);
                        accumulate(z, f, c);
                    }
                }
            }
        } else {
            int k = lo + tid;
            for (; k + 3 * threads < hi; k += 4 * threads) {
                uint4 q[4];
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    q[j] = x.load(k + j * threads);
                float f[4 * G];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    float g[G];
                    values(q[j], g);
#pragma unroll
                    for (int i = 0; i < G; ++i)
                        f[j * G + i] = g[i];
                }
                accumulate(z, f, c);
            }
            for (; k < hi; k += threads) {
                float f[G];
                values(x.load(k), f);
                accumulate(z, f, c);
            }
        }
        // what of the row lies in granules with other elements
        if (rank == 0 && tid == 0 && x.first > 0) {
            float f[G];
            x.load_edge(0, neg_inf(), f);
            accumulate(z, f, c);
        }
        if (rank == parts - 1 && tid == threads - 1 && x.col(x.last, 0) < x.V) {
            float f[G];
            x.load_edge(x.last, neg_inf(), f);
            accumulate(z, f, c);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
            z = join(z, {__shfl_xor_sync(~0u, z.m, o), __shfl_xor_sync(~0u, z.s, o)}, c);
        if (lane == 0)
            part[tid >> 5] = z;
        __syncthreads();
        z = lane < threads / 32 ? part[lane] : Sum{-FLT_MAX, 0.0f};
#pragma unroll
        for (int o = 8; o > 0; o >>= 1)
            z = join(z, {__shfl_xor_sync(~0u, z.m, o), __shfl_xor_sync(~0u, z.s, o)}, c);
        z = {__shfl_sync(~0u, z.m, 0), __shfl_sync(~0u, z.s, 0)};
        if (CLUSTER) {
            if (tid == 0)
                mine = z;
            cluster_arrive();
            cluster_wait();
            z = lane < parts ? remote(&mine, lane) : Sum{-FLT_MAX, 0.0f};
            cluster_arrive();  // no more reads from here; waited for at the end
#pragma unroll
            for (int o = kMaxCluster / 2; o > 0; o >>= 1)
                z = join(z, {__shfl_xor_sync(~0u, z.m, o), __shfl_xor_sync(~0u, z.s, o)}, c);
            z = {__shfl_sync(~0u, z.m, 0), __shfl_sync(~0u, z.s, 0)};
        }
        const float ln_s = logf(z.s);
        const float logp = (xa - z.m) * a.inv_temperature - ln_s;
        if (MODE == kForward && rank == 0 && tid == 0) {
            a.logp[row] = logp;
            a.lse[row] = z.m * a.inv_temperature + ln_s;
        }
        if (MODE == kPolicy) {
            const float r = expf(logp - old);
            const float free = adv == 0.0f ? 0.0f : r * adv;
            const float held_at = fminf(fmaxf(r, a.clip_lo), a.clip_hi) * adv;
            float loss = -fminf(free, held_at), slope = free <= held_at ? -free : 0.0f;
            if (isnan(r))
                loss = slope = r;
            if (a.ref_logp) {
                const float d = ref_logp - logp, em1 = expm1f(d);
                loss += a.kl * (em1 - d);
                slope -= a.kl * em1;
            }
            coef = weight * slope * a.grad_scale;
            inv = 1.0f / z.s;
            if (rank == 0 && tid == 0) {
                a.token_loss[row] = weight * loss;
                a.logp[row] = logp;
            }
        }
    } else if (rank == 0 && tid == 0) {
        a.logp[row] = 0.0f;
        if (MODE == kForward)
            a.lse[row] = 0.0f;
        if (MODE == kForward && a.coef)
            a.coef[row] = 0.0f;
        if (MODE == kPolicy)
            a.token_loss[row] = 0.0f;
    }
    if (MODE == kPolicy && a.dlogits) {
        const Gradient<E> d(x, a, c, coef, inv, z.m, target);
        const bool zero = !(coef != 0.0f);  // also a clipped row's
        if (zero) {
            for (int k = lo + tid; k < hi; k += threads)
                stg128_stream(d.out + static_cast<int64_t>(k) * G, make_uint4(0, 0, 0, 0));
        } else if (RESIDENT) {
            for (int k = lo + tid; k < hi; k += threads)
                d.interior(k, held[k - lo]);
        } else {
            for (int k = lo + tid; k < hi; k += threads)
                d.interior(k, x.load(k));
        }
        if (rank == 0 && tid == 0 && x.first > 0)
            d.edge(0, zero);
        if (rank == parts - 1)
            for (int k = max(x.last, x.first) + tid; k < x.end; k += threads)
                d.edge(k, zero);
    }
    if (CLUSTER && active)
        cluster_wait();
}

// The gradient from a given lse; `parts` CTAs a row, each on its own.
template <typename E>
__global__ void __launch_bounds__(256) backward_kernel(const __grid_constant__ LossRows a, int parts, int trigger)
{
    constexpr int G = Row<E>::G;
    if (trigger)
        pdl_trigger();
    pdl_wait();
    const int tid = threadIdx.x, threads = blockDim.x, rank = blockIdx.x % parts;
    const int64_t row = blockIdx.x / parts;
    const Row<E> x(a, row);
    const int64_t target = a.targets[row];
    const float weight = a.dlogp[row];
    const bool zero = target < 0 || weight == 0.0f;
    const int each = (x.last - x.first + parts - 1) / parts;
    const int lo = min(x.last, x.first + rank * each), hi = min(x.last, lo + each);
    const Scale c(a.inv_temperature);
    // exp(x / tau - lse) = exp2(c (x - hi)) exp2(-c lo), hi + lo = lse tau
    const float lse = a.lse[row], at = lse * a.temperature;
    const float low = fmaf(lse, a.temperature, -at);
    const float inv = fabsf(low) <= FLT_MAX ? ex2(-low * c.hi) : 1.0f;
    const Gradient<E> d(x, a, c, target < x.V ? weight * a.grad_scale : quiet_nan(), inv, at, target);
    int k = lo + tid;
    if (zero) {
        for (; k < hi; k += threads)
            stg128_stream(d.out + static_cast<int64_t>(k) * G, make_uint4(0, 0, 0, 0));
    } else {
        for (; k + 3 * threads < hi; k += 4 * threads) {
            uint4 q[4];
#pragma unroll
            for (int j = 0; j < 4; ++j)
                q[j] = x.load(k + j * threads);
#pragma unroll
            for (int j = 0; j < 4; ++j)
                d.interior(k + j * threads, q[j]);
        }
        for (; k < hi; k += threads)
            d.interior(k, x.load(k));
    }
    if (rank == 0 && tid == 0 && x.first > 0)
        d.edge(0, zero);
    if (rank == parts - 1)
        for (int k = max(x.last, x.first) + tid; k < x.end; k += threads)
            d.edge(k, zero);
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

template <typename K, typename... Args>
cudaError_t launch_cluster(K kernel, int64_t ctas, int threads, size_t smem, int cluster, cudaStream_t stream,
                           Args &&...args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(ctas));
    cfg.blockDim = dim3(static_cast<unsigned>(threads));
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim = {static_cast<unsigned>(cluster), 1, 1};
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, static_cast<Args &&>(args)...);
}

// How a launch splits its rows.
struct Split {
    int parts, threads;
};

template <typename E, int MODE, bool CLUSTER, bool RESIDENT>
cudaError_t launch_row_kernel(const LossRows &a, Split s, size_t smem, int trigger, int device, cudaStream_t stream)
{
    const int chunks = static_cast<int>((smem / 16 + s.threads * kChunkSteps - 1) / (s.threads * kChunkSteps));
    const auto kernel = row_kernel<E, MODE, CLUSTER, RESIDENT>;
    if (RESIDENT) {
        static std::atomic<bool> done[kMaxDevices];
        const cudaError_t e = ensure_smem(kernel, 220 * 1024, device, done);
        if (e != cudaSuccess)
            return e;
    }
    return launch_cluster(kernel, a.T * s.parts, s.threads, smem, CLUSTER ? s.parts : 1, stream, a, s.parts, chunks,
                          trigger);
}

template <typename E, int MODE> cudaError_t launch_rows(const LossRows &a, cudaStream_t stream)
{
    constexpr int G = 16 / sizeof(E);
    DeviceInfo di;
    cudaError_t e = current_device_info(&di);
    if (e != cudaSuccess)
        return e;
    const int64_t granules = a.V / G + 1;
    // the policy loss sums in the same order with and without its gradient
    const bool grad = MODE == kPolicy;
    // a part of at most 55 KB leaves room for four CTAs on an SM
    Split s = {1, 32};
    while (s.parts < kMaxCluster && grad && (granules + s.parts - 1) / s.parts * 16 > 55 * 1024)
        s.parts *= 2;
    while (s.parts < kMaxCluster && a.T * s.parts < 2 * di.num_sms && granules / s.parts >= 512)
        s.parts *= 2;
    const int64_t each = (granules + s.parts - 1) / s.parts;
    while (s.threads < 256 && s.threads * 4 < each)
        s.threads *= 2;
    const size_t smem = static_cast<size_t>(each) * 16;
    const bool resident = grad && smem <= 216 * 1024 && each <= int64_t(kMaxChunks) * s.threads * kChunkSteps;
    const int trigger = a.T * s.parts <= di.num_sms;
    if (s.parts > 1)
        return resident ? launch_row_kernel<E, MODE, true, true>(a, s, smem, trigger, di.device, stream)
                        : launch_row_kernel<E, MODE, true, false>(a, s, 0, trigger, di.device, stream);
    return resident ? launch_row_kernel<E, MODE, false, true>(a, s, smem, trigger, di.device, stream)
                    : launch_row_kernel<E, MODE, false, false>(a, s, 0, trigger, di.device, stream);
}

template <int MODE> cudaError_t launch_rows(const LossRows &a, bool bf16, cudaStream_t stream)
{
    return bf16 ? launch_rows<uint16_t, MODE>(a, stream) : launch_rows<float, MODE>(a, stream);
}

}  // namespace

cudaError_t launch_logprob(const LossRows &a, bool bf16, cudaStream_t stream)
{
    return launch_rows<kForward>(a, bf16, stream);
}

cudaError_t launch_logprob_backward(const LossRows &a, bool bf16, cudaStream_t stream)
{
    DeviceInfo di;
    const cudaError_t e = current_device_info(&di);
    if (e != cudaSuccess)
        return e;
    const int64_t granules = a.N / (bf16 ? 8 : 4) + 1;
    Split s = {1, 32};
    while (s.parts < 64 && a.T * s.parts < 4 * di.num_sms && granules / s.parts >= 512)
        s.parts *= 2;
    while (s.threads < 256 && s.threads * s.parts * 4 < granules)
        s.threads *= 2;
    const int trigger = a.T * s.parts <= di.num_sms;
    return launch_cluster(bf16 ? backward_kernel<uint16_t> : backward_kernel<float>, a.T * s.parts, s.threads, 0, 1,
                          stream, a, s.parts, trigger);
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
    if (a.T > 0 && a.dlogits && (e = launch_logprob_backward(a, bf16, stream)) != cudaSuccess)
        return e;
    return launch_pdl(total_kernel, 1, 1024, 0, stream, static_cast<const float *>(p.pair_loss), p.pairs,
                      1.0f / static_cast<float>(p.pairs), loss);
}

cudaError_t read_loss_error(uint32_t *flags, bool clear)
{
    uint32_t v = 0;
    cudaError_t e = cudaMemcpyFromSymbol(&v, g_loss_error, sizeof v);
    if (e != cudaSuccess)
        return e;
    *flags = v;
    if (clear && v) {
        v = 0;
        e = cudaMemcpyToSymbol(g_loss_error, &v, sizeof v);
    }
    return e;
}

}  // namespace taco
