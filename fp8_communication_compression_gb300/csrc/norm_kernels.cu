// The norms around a block, fused with its gate and residual scale:
//
//   z  = y / sqrt(mean(y^2) + eps) * g_post        (after the block)
//   h' = s h + gate z                              (the residual stream)
//   n  = h' / sqrt(mean(h'^2) + eps) * g_pre       (before the next block)
//
// and their backward pass.  y is the block's output, h the residual stream;
// the gate is absent, one value a channel, one a token, or one an element.
// n leaves in bf16, or already quantised as the FP8 operand of the next
// product (fp8_block.cuh).
//
// With r_y = 1 / sqrt(mean(y^2) + eps), r_h likewise of h', u = dn g_pre:
//
//   G      = dh' + r_h u - h' r_h^3 mean(u h')     (gradient at h')
//   dh     = s G
//   v      = G gate g_post
//   dy     = r_y v - y r_y^3 mean(v y)
//   dg_pre = sum_t dn h' r_h,  dg_post = sum_t gate G y r_y
//   dgate  = G y r_y g_post, summed over what the gate is shared by
//
// The backward pass recomputes both root mean squares from its inputs: they
// cost no extra pass, as the row is held anyway, and nothing has to be saved
// beside y and h'.  All of it is fp32 (sums, statistics, gradients); values
// are rounded once, when they are stored.
//
// Bound by HBM: 8 bytes an element forward, 12 backward.  A CTA takes whole
// rows in turn, 8 V columns a thread.  Rows arrive by bulk copies into a ring
// of row slots in shared memory, several rows ahead of the row being worked
// on, so the loads do not wait for the two block-wide sums that every row
// needs; outputs go straight from registers in 16-byte stores.  Rows that
// are not a multiple of 16 bytes are read element by element.
//
// The gains' gradients are summed over a CTA's rows in registers, written as
// one partial row per CTA, and added over the CTAs in a fixed order by a
// second small kernel: no atomics, the same bits every time.

#include <atomic>

#include "device_utils.cuh"
#include "fp8_block.cuh"
#include "internal.h"

namespace taco {

// Watchdog flag of this file's kernels (bit 7), read by taco_device_error().
__device__ unsigned int g_norm_error;

namespace {

constexpr uint32_t kErrNorm = 128u;
constexpr int kMaxThreads = 512;
constexpr int kMaxSlots = 4;

// Gate modes (include/taco.h).
constexpr int kGateNone = 0, kGateChannel = 1, kGateToken = 2, kGateFull = 3;

__device__ __forceinline__ void bulk_load(uint32_t dst, const void *src, uint32_t bytes, uint32_t bar)
{
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
                 "l"(src), "r"(bytes), "r"(bar)
                 : "memory");
}

// Eight bf16 values of a packed 16-byte unit.
__device__ __forceinline__ void unpack8(const uint4 &q, float (&x)[8])
{
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = bf16lo_to_f32(w[i]);
        x[2 * i + 1] = bf16hi_to_f32(w[i]);
    }
}

__device__ __forceinline__ uint4 pack8(const float (&x)[8])
{
    return make_uint4(f32x2_to_bf16x2(x[0], x[1]), f32x2_to_bf16x2(x[2], x[3]), f32x2_to_bf16x2(x[4], x[5]),
                      f32x2_to_bf16x2(x[6], x[7]));
}

// Columns c .. c + 7 of fp32 vectors of d values (zeros past the end).
template <bool VEC> __device__ __forceinline__ void load_f32x8(const float *p, int c, int d, float (&x)[8])
{
    if (VEC) {
        float4 a = make_float4(0, 0, 0, 0), b = a;
        if (c < d) {
            a = __ldg(reinterpret_cast<const float4 *>(p + c));
            b = __ldg(reinterpret_cast<const float4 *>(p + c) + 1);
        }
        x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            x[j] = c + j < d ? __ldg(p + c + j) : 0.0f;
    }
}

template <bool VEC> __device__ __forceinline__ void store_bf16x8(uint16_t *p, int c, int d, const float (&x)[8])
{
    const uint4 q = pack8(x);
    if (VEC) {
        if (c < d)
            stg128_stream(p + c, q);
    } else {
        const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (c + j < d)
                p[c + j] = static_cast<uint16_t>(w[j >> 1] >> (16 * (j & 1)));
    }
}

// The CTA's rows blockIdx.x, + gridDim.x, ...: NT bf16 tensors' rows, NT
// row-sized pieces to a slot.
template <int NT, bool VEC> struct RowRing {
    const uint16_t *src[NT];
    uint32_t buf, bars, slots, row_bytes;
    int64_t T;
    int d;
    int64_t it = 0;  // rows consumed by this CTA
    bool dead = false;

    __device__ __forceinline__ void issue(int64_t n)  // this CTA's n-th row (one thread)
    {
        const int64_t row = blockIdx.x + n * gridDim.x;
        if (row >= T)
            return;
        const uint32_t s = static_cast<uint32_t>(n % slots), bar = bars + 8 * s;
        mbar_arrive_expect_tx(bar, NT * row_bytes);
#pragma unroll
        for (int k = 0; k < NT; ++k)
            bulk_load(buf + (s * NT + k) * row_bytes, src[k] + row * d, row_bytes, bar);
    }
    __device__ __forceinline__ void start()
    {
        if (VEC && threadIdx.x == 0)
            for (uint32_t n = 0; n < slots; ++n)
                issue(n);
    }
    // The current row has landed (or is read directly).
    __device__ __forceinline__ void wait()
    {
        if (VEC && !dead &&
            !mbar_wait(bars + 8 * static_cast<uint32_t>(it % slots), static_cast<uint32_t>(it / slots) & 1)) {
            atomicOr(&g_norm_error, kErrNorm);
            dead = true;
            // the thread that issues stops issuing: wait for what is in flight
            if (threadIdx.x == 0)
                for (int64_t n = it; n < it + slots && blockIdx.x + n * gridDim.x < T; ++n)
                    mbar_wait(bars + 8 * static_cast<uint32_t>(n % slots), static_cast<uint32_t>(n / slots) & 1);
        }
    }
    // Columns c .. c + 7 of tensor k's current row, zeros past the end.
    __device__ __forceinline__ uint4 get(int k, int c) const
    {
        if (VEC) {
            if (c >= d || dead)
                return make_uint4(0, 0, 0, 0);
            return lds128(buf + (static_cast<uint32_t>(it % slots) * NT + k) * row_bytes + 2 * c);
        }
        const uint16_t *p = src[k] + (blockIdx.x + it * gridDim.x) * d + c;
        uint32_t e[8];
#pragma unroll
        for (int j = 0; j < 8; ++j)
            e[j] = c + j < d ? __ldg(p + j) : 0u;
        return make_uint4(e[0] | e[1] << 16, e[2] | e[3] << 16, e[4] | e[5] << 16, e[6] | e[7] << 16);
    }
    // Every thread has read the current row (a barrier lies behind): refill
    // its slot.
    __device__ __forceinline__ void refill()
    {
        if (VEC && threadIdx.x == 0 && !dead)
            issue(it + slots);
    }
};

// Sums of K values over the CTA; every thread gets them.  `red` holds K * 16
// floats; two calls in turn use two of them, so that one barrier a call is
// enough.
template <int K> __device__ __forceinline__ void block_sum(float (&v)[K], float *red)
{
#pragma unroll
    for (int s = 16; s >= 1; s >>= 1)
#pragma unroll
        for (int k = 0; k < K; ++k)
            v[k] += __shfl_xor_sync(0xFFFFFFFFu, v[k], s);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
    if (lane == 0)
#pragma unroll
        for (int k = 0; k < K; ++k)
            red[16 * k + warp] = v[k];
    __syncthreads();
#pragma unroll
    for (int k = 0; k < K; ++k)
        v[k] = (lane & 15) < warps ? red[16 * k + (lane & 15)] : 0.0f;
#pragma unroll
    for (int s = 8; s >= 1; s >>= 1)
#pragma unroll
        for (int k = 0; k < K; ++k)
            v[k] += __shfl_xor_sync(0xFFFFFFFFu, v[k], s);
}

template <int NT, bool VEC>
__device__ __forceinline__ void ring_init(RowRing<NT, VEC> &ring, uint8_t *smem, uint32_t bars, int64_t T, int d,
                                          int slots)
{
    ring.buf = (smem_u32(smem) + 127u) & ~127u;
    ring.bars = bars;
    ring.slots = slots;
    ring.row_bytes = 2 * d;
    ring.T = T;
    ring.d = d;
    if (VEC && threadIdx.x == 0) {
        for (int s = 0; s < slots; ++s)
            mbar_init(bars + 8 * s, 1);
        fence_barrier_init();
        fence_proxy_async_smem();
    }
    __syncthreads();
}

// ---------------------------------------------------------------- forward --

// V groups of 8 columns a thread (group v: columns 8 (threadIdx.x + v
// blockDim.x)); GATE a gate mode; FP8: n as codes and scales.
template <int V, int GATE, bool FP8, bool VEC>
__global__ void __launch_bounds__(kMaxThreads)
    norm_forward_kernel(const uint16_t *__restrict__ y, const uint16_t *__restrict__ h,
                        const float *__restrict__ g_post, const float *__restrict__ g_pre,
                        const void *__restrict__ gate, float s, float eps, int64_t T, int d, int slots,
                        uint16_t *__restrict__ h_out, void *__restrict__ n_out, uint8_t *__restrict__ n_scale)
{
    constexpr int NT = GATE == kGateFull ? 3 : 2;
    extern __shared__ uint8_t smem_raw[];
    __shared__ uint64_t bars[kMaxSlots];
    __shared__ float red[2][16];
    RowRing<NT, VEC> ring;
    ring.src[0] = y;
    ring.src[1] = h;
    if constexpr (GATE == kGateFull)
        ring.src[2] = static_cast<const uint16_t *>(gate);
    ring_init(ring, smem_raw, smem_u32(bars), T, d, slots);
    const float inv_d = 1.0f / static_cast<float>(d);
    if (T <= 4 * static_cast<int64_t>(gridDim.x))  // short: the next kernel's launch overlaps it
        pdl_trigger();
    pdl_wait();
    ring.start();
    for (int64_t row = blockIdx.x; row < T; row += gridDim.x, ++ring.it) {
        ring.wait();
        uint4 qy[V], qh[V], qg[V];
        float sum[1] = {0.0f};
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int c = 8 * (threadIdx.x + v * blockDim.x);
            qy[v] = ring.get(0, c);
            qh[v] = ring.get(1, c);
            if constexpr (GATE == kGateFull)
                qg[v] = ring.get(2, c);
            float x[8];
            unpack8(qy[v], x);
#pragma unroll
            for (int j = 0; j < 8; ++j)
                sum[0] = fmaf(x[j], x[j], sum[0]);
        }
        float gt = 1.0f;
        if constexpr (GATE == kGateToken)
            gt = __ldg(static_cast<const float *>(gate) + row);
        block_sum(sum, red[0]);
        ring.refill();
        const float ry = rsqrtf(sum[0] * inv_d + eps);
        float h2[V][8];
        sum[0] = 0.0f;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int c = 8 * (threadIdx.x + v * blockDim.x);
            float x[8], g[8];
            unpack8(qy[v], x);
            unpack8(qh[v], h2[v]);
            load_f32x8<VEC>(g_post, c, d, g);
#pragma unroll
            for (int j = 0; j < 8; ++j)
                x[j] = x[j] * ry * g[j];
            if constexpr (GATE == kGateChannel)
                load_f32x8<VEC>(static_cast<const float *>(gate), c, d, g);
            if constexpr (GATE == kGateFull)
                unpack8(qg[v], g);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float z = GATE == kGateNone ? x[j] : GATE == kGateToken ? gt * x[j] : g[j] * x[j];
                h2[v][j] = fmaf(s, h2[v][j], z);
                sum[0] = fmaf(h2[v][j], h2[v][j], sum[0]);
            }
            store_bf16x8<VEC>(h_out + row * d, c, d, h2[v]);
        }
        block_sum(sum, red[1]);
        const float rh = rsqrtf(sum[0] * inv_d + eps);
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int c = 8 * (threadIdx.x + v * blockDim.x);
            float g[8];
            load_f32x8<VEC>(g_pre, c, d, g);
#pragma unroll
            for (int j = 0; j < 8; ++j)
                g[j] = h2[v][j] * rh * g[j];
            if constexpr (FP8) {
                // the block's maximum: 16 lanes of 8 columns
                uint32_t m = 0;
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    m = max(m, __float_as_uint(g[j]) & 0x7FFFFFFFu);
#pragma unroll
                for (int k = 8; k >= 1; k >>= 1)
                    m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, k));
                const uint32_t byte = fp8_scale_byte(m);
                const float f = fp8_inv_scale(byte);
                const int64_t pitch = fp8_pitch(d);
                if (c < pitch)
                    *reinterpret_cast<uint2 *>(static_cast<uint8_t *>(n_out) + row * pitch + c) =
                        make_uint2(f32x4_to_e4m3x4(g[0] * f, g[1] * f, g[2] * f, g[3] * f),
                                   f32x4_to_e4m3x4(g[4] * f, g[5] * f, g[6] * f, g[7] * f));
                if ((threadIdx.x & 15) == 0 && c < d)
                    n_scale[fp8_scale_at(row, c >> 7, (d + 511) / 512)] = static_cast<uint8_t>(byte);
            } else {
                store_bf16x8<VEC>(static_cast<uint16_t *>(n_out) + row * d, c, d, g);
            }
        }
    }
}

// --------------------------------------------------------------- backward --

template <int V, int GATE, bool VEC>
__global__ void __launch_bounds__(kMaxThreads, V == 1 ? 2 : 1)
    norm_backward_kernel(const uint16_t *__restrict__ dn, const uint16_t *__restrict__ dh2,
                         const uint16_t *__restrict__ y, const uint16_t *__restrict__ h2,
                         const float *__restrict__ g_post, const float *__restrict__ g_pre,
                         const void *__restrict__ gate, float s, float eps, int64_t T, int d, int slots,
                         uint16_t *__restrict__ dy, uint16_t *__restrict__ dh, void *__restrict__ dgate,
                         float *__restrict__ partial)
{
    constexpr int NT = GATE == kGateFull ? 5 : 4;
    extern __shared__ uint8_t smem_raw[];
    __shared__ uint64_t bars[kMaxSlots];
    __shared__ float red[2][48];
    RowRing<NT, VEC> ring;
    ring.src[0] = dn;
    ring.src[1] = dh2;
    ring.src[2] = y;
    ring.src[3] = h2;
    if constexpr (GATE == kGateFull)
        ring.src[4] = static_cast<const uint16_t *>(gate);
    ring_init(ring, smem_raw, smem_u32(bars), T, d, slots);
    const float inv_d = 1.0f / static_cast<float>(d);
    float a_pre[V][8] = {}, a_post[V][8] = {};
    if (T <= 4 * static_cast<int64_t>(gridDim.x))  // short: the next kernel's launch overlaps it
        pdl_trigger();
    pdl_wait();
    ring.start();
    for (int64_t row = blockIdx.x; row < T; row += gridDim.x, ++ring.it) {
        ring.wait();
        uint4 qn[V], qd[V], qy[V], qh[V], qg[V];
        float sum[3] = {0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int c = 8 * (threadIdx.x + v * blockDim.x);
            qn[v] = ring.get(0, c);
            qd[v] = ring.get(1, c);
            qy[v] = ring.get(2, c);
            qh[v] = ring.get(3, c);
            if constexpr (GATE == kGateFull)
                qg[v] = ring.get(4, c);
            float a[8], b[8], g[8];
            unpack8(qh[v], a);
            unpack8(qn[v], b);
            load_f32x8<VEC>(g_pre, c, d, g);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                sum[0] = fmaf(a[j], a[j], sum[0]);
                sum[1] = fmaf(b[j] * g[j], a[j], sum[1]);
            }
            unpack8(qy[v], a);
#pragma unroll
            for (int j = 0; j < 8; ++j)
                sum[2] = fmaf(a[j], a[j], sum[2]);
        }
        float gt = 1.0f;
        if constexpr (GATE == kGateToken)
            gt = __ldg(static_cast<const float *>(gate) + row);
        block_sum(sum, red[0]);
        ring.refill();
        const float rh = rsqrtf(sum[0] * inv_d + eps), ry = rsqrtf(sum[2] * inv_d + eps);
        const float ch = rh * rh * rh * (sum[1] * inv_d);
        float G[V][8];
        float dot[1] = {0.0f};
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int c = 8 * (threadIdx.x + v * blockDim.x);
            float a[8], b[8], g[8];
            unpack8(qh[v], a);
            unpack8(qn[v], b);
            unpack8(qd[v], G[v]);
            load_f32x8<VEC>(g_pre, c, d, g);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                a_pre[v][j] = fmaf(b[j], a[j] * rh, a_pre[v][j]);
                G[v][j] = fmaf(-a[j], ch, fmaf(rh * b[j], g[j], G[v][j]));
                b[j] = s * G[v][j];
            }
            store_bf16x8<VEC>(dh + row * d, c, d, b);
            // y r_y G: the sum over tokens behind dg_post and a channel
            // gate's gradient
            unpack8(qy[v], a);
#pragma unroll
            for (int j = 0; j < 8; ++j)
                b[j] = a[j] * ry * G[v][j];
            load_f32x8<VEC>(g_post, c, d, g);
            if constexpr (GATE == kGateFull) {
                float e[8], w[8];
                unpack8(qg[v], w);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    e[j] = b[j] * g[j];
                    b[j] *= w[j];
                    dot[0] = fmaf(b[j], g[j], dot[0]);
                    a_post[v][j] += b[j];
                }
                store_bf16x8<VEC>(static_cast<uint16_t *>(dgate) + row * d, c, d, e);
            } else {
                float w[8];
                if constexpr (GATE == kGateChannel)
                    load_f32x8<VEC>(static_cast<const float *>(gate), c, d, w);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    dot[0] = fmaf(b[j], GATE == kGateChannel ? g[j] * w[j] : g[j], dot[0]);
                    a_post[v][j] = GATE == kGateToken ? fmaf(gt, b[j], a_post[v][j]) : a_post[v][j] + b[j];
                }
            }
        }
        block_sum(dot, red[1]);  // sum of (y r_y) G g_post (and a channel's or element's gate)
        if constexpr (GATE == kGateToken)
            if (threadIdx.x == 0)
                static_cast<float *>(dgate)[row] = dot[0];
        const float cy = ry * ry * (gt * dot[0] * inv_d);
        const float rg = ry * gt;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int c = 8 * (threadIdx.x + v * blockDim.x);
            float a[8], g[8], w[8];
            unpack8(qy[v], a);
            load_f32x8<VEC>(g_post, c, d, g);
            if constexpr (GATE == kGateChannel)
                load_f32x8<VEC>(static_cast<const float *>(gate), c, d, w);
            if constexpr (GATE == kGateFull)
                unpack8(qg[v], w);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                float u = rg * g[j];
                if constexpr (GATE == kGateChannel || GATE == kGateFull)
                    u *= w[j];
                a[j] = fmaf(u, G[v][j], -a[j] * cy);
            }
            store_bf16x8<VEC>(dy + row * d, c, d, a);
        }
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int c = 8 * (threadIdx.x + v * blockDim.x);
        float *p = partial + static_cast<int64_t>(blockIdx.x) * 2 * d;
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (c + j < d) {
                p[c + j] = a_pre[v][j];
                p[d + c + j] = a_post[v][j];
            }
    }
}

// Sums the CTAs' partial rows in a fixed order: 32 columns a CTA, eight
// groups of rows in turn, then the groups.
__global__ void __launch_bounds__(256)
    norm_gains_kernel(const float *__restrict__ partial, int ctas, int d, int gate_mode,
                      const float *__restrict__ g_post, const float *__restrict__ gate, float *__restrict__ dg_pre,
                      float *__restrict__ dg_post, float *__restrict__ dgate)
{
    __shared__ float part[2][8][33];
    const int lane = threadIdx.x & 31, grp = threadIdx.x >> 5, c = blockIdx.x * 32 + lane;
    pdl_wait();
    float a = 0.0f, b = 0.0f;
    if (c < d)
#pragma unroll 4
        for (int i = grp; i < ctas; i += 8) {
            a += partial[static_cast<int64_t>(i) * 2 * d + c];
            b += partial[static_cast<int64_t>(i) * 2 * d + d + c];
        }
    part[0][grp][lane] = a;
    part[1][grp][lane] = b;
    __syncthreads();
    if (grp == 0 && c < d) {
        a = b = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            a += part[0][i][lane];
            b += part[1][i][lane];
        }
        dg_pre[c] = a;
        if (gate_mode == kGateChannel) {
            dg_post[c] = b * gate[c];
            dgate[c] = b * g_post[c];
        } else {
            dg_post[c] = b;
        }
    }
}

// Threads, groups of 8 columns a thread, ring slots and CTAs of a shape.
struct NormPlan {
    int threads, v, slots, grid;
    uint32_t smem;
};

constexpr uint32_t kSmemPerSm = 227 * 1024;

NormPlan plan_norm(int64_t T, int d, int tensors, int per_sm_threads, int sms)
{
    NormPlan p;
    const int units = (d + 7) / 8;
    p.v = units <= kMaxThreads ? 1 : units <= 2 * kMaxThreads ? 2 : 4;
    p.threads = ((units + p.v - 1) / p.v + 31) / 32 * 32;
    int per_sm = per_sm_threads / p.threads;
    per_sm = per_sm < 1 ? 1 : per_sm > 8 ? 8 : per_sm;
    p.slots = 0;
    p.smem = 0;
    if (d % 8 == 0) {
        const uint32_t slot = static_cast<uint32_t>(tensors) * 2 * d;
        while (per_sm > 1 && 2 * slot + 2048 > kSmemPerSm / per_sm)
            --per_sm;
        const uint32_t room = kSmemPerSm / per_sm - 2048;
        p.slots = static_cast<int>(room / slot);
        p.slots = p.slots > kMaxSlots ? kMaxSlots : p.slots < 1 ? 1 : p.slots;
        p.smem = 128 + p.slots * slot;
    }
    const int64_t most = static_cast<int64_t>(per_sm) * sms;
    p.grid = static_cast<int>(T < most ? T : most);
    return p;
}

NormPlan plan_backward(int64_t T, int d, int gate_mode, int sms)
{
    return plan_norm(T, d, gate_mode == kGateFull ? 5 : 4, d <= 8 * kMaxThreads ? 1024 : 512, sms);
}

constexpr int kMaxDevices = 64;

template <class K> cudaError_t allow_smem(K kernel, int device, std::atomic<bool> *set)
{
    if (set[device].load(std::memory_order_acquire))
        return cudaSuccess;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 225 * 1024);
    if (e == cudaSuccess)
        set[device].store(true, std::memory_order_release);
    return e;
}

template <int V, int GATE, bool FP8, bool VEC>
cudaError_t run_forward(const NormPlan &p, const NormForward &a, int device, cudaStream_t stream)
{
    static std::atomic<bool> set[kMaxDevices];
    cudaError_t e = allow_smem(norm_forward_kernel<V, GATE, FP8, VEC>, device, set);
    if (e != cudaSuccess)
        return e;
    return launch_pdl(norm_forward_kernel<V, GATE, FP8, VEC>, dim3(p.grid), dim3(p.threads), p.smem, stream,
                      static_cast<const uint16_t *>(a.y), static_cast<const uint16_t *>(a.h), a.g_post, a.g_pre,
                      a.gate, a.residual_scale, a.eps, a.T, static_cast<int>(a.d), p.slots,
                      static_cast<uint16_t *>(a.h_out), a.n_out, a.n_scale);
}

template <int V, int GATE, bool VEC>
cudaError_t run_backward(const NormPlan &p, const NormBackward &a, int device, cudaStream_t stream)
{
    static std::atomic<bool> set[kMaxDevices];
    cudaError_t e = allow_smem(norm_backward_kernel<V, GATE, VEC>, device, set);
    if (e != cudaSuccess)
        return e;
    e = launch_pdl(norm_backward_kernel<V, GATE, VEC>, dim3(p.grid), dim3(p.threads), p.smem, stream,
                   static_cast<const uint16_t *>(a.dn), static_cast<const uint16_t *>(a.dh_out),
                   static_cast<const uint16_t *>(a.y), static_cast<const uint16_t *>(a.h_out), a.g_post, a.g_pre,
                   a.gate, a.residual_scale, a.eps, a.T, static_cast<int>(a.d), p.slots,
                   static_cast<uint16_t *>(a.dy), static_cast<uint16_t *>(a.dh), a.dgate,
                   static_cast<float *>(a.workspace));
    if (e != cudaSuccess)
        return e;
    return launch_pdl(norm_gains_kernel, dim3(static_cast<unsigned>((a.d + 31) / 32)), dim3(256), 0, stream,
                      static_cast<const float *>(a.workspace), p.grid, static_cast<int>(a.d), GATE, a.g_post,
                      static_cast<const float *>(a.gate), a.dg_pre, a.dg_post, static_cast<float *>(a.dgate));
}

template <int V, int GATE, bool VEC>
cudaError_t forward_out(const NormPlan &p, const NormForward &a, int dev, cudaStream_t s)
{
    return a.n_scale ? run_forward<V, GATE, true, VEC>(p, a, dev, s) : run_forward<V, GATE, false, VEC>(p, a, dev, s);
}

template <int V, bool VEC> cudaError_t forward_gate(const NormPlan &p, const NormForward &a, int dev, cudaStream_t s)
{
    switch (a.gate_mode) {
    case kGateNone:
        return forward_out<V, kGateNone, VEC>(p, a, dev, s);
    case kGateChannel:
        return forward_out<V, kGateChannel, VEC>(p, a, dev, s);
    case kGateToken:
        return forward_out<V, kGateToken, VEC>(p, a, dev, s);
    default:
        return forward_out<V, kGateFull, VEC>(p, a, dev, s);
    }
}

template <int V, bool VEC> cudaError_t backward_gate(const NormPlan &p, const NormBackward &a, int dev, cudaStream_t s)
{
    switch (a.gate_mode) {
    case kGateNone:
        return run_backward<V, kGateNone, VEC>(p, a, dev, s);
    case kGateChannel:
        return run_backward<V, kGateChannel, VEC>(p, a, dev, s);
    case kGateToken:
        return run_backward<V, kGateToken, VEC>(p, a, dev, s);
    default:
        return run_backward<V, kGateFull, VEC>(p, a, dev, s);
    }
}

}  // namespace

cudaError_t read_norm_error(uint32_t *flags, bool clear)
{
    unsigned int v = 0;
    cudaError_t e = cudaMemcpyFromSymbol(&v, g_norm_error, sizeof v);
    if (e != cudaSuccess)
        return e;
    *flags = v;
    if (clear) {
        v = 0;
        e = cudaMemcpyToSymbol(g_norm_error, &v, sizeof v);
    }
    return e;
}

cudaError_t launch_norm_forward(const NormForward &a, cudaStream_t stream)
{
    DeviceInfo di;
    cudaError_t e = current_device_info(&di);
    if (e != cudaSuccess)
        return e;
    const int d = static_cast<int>(a.d);
    const NormPlan p = plan_norm(a.T, d, a.gate_mode == kGateFull ? 3 : 2, 1024, di.num_sms);
    const bool vec = d % 8 == 0;
    switch (p.v) {
    case 1:
        return vec ? forward_gate<1, true>(p, a, di.device, stream) : forward_gate<1, false>(p, a, di.device, stream);
    case 2:
        return vec ? forward_gate<2, true>(p, a, di.device, stream) : forward_gate<2, false>(p, a, di.device, stream);
    default:
        return vec ? forward_gate<4, true>(p, a, di.device, stream) : forward_gate<4, false>(p, a, di.device, stream);
    }
}

cudaError_t norm_backward_workspace(int64_t T, int64_t d, int gate_mode, uint64_t *bytes)
{
    DeviceInfo di;
    cudaError_t e = current_device_info(&di);
    if (e != cudaSuccess)
        return e;
    *bytes = 8 * static_cast<uint64_t>(d) * plan_backward(T, static_cast<int>(d), gate_mode, di.num_sms).grid;
    return cudaSuccess;
}

cudaError_t launch_norm_backward(const NormBackward &a, cudaStream_t stream)
{
    if (a.T == 0) {  // no tokens: the sums over them are zero
        cudaError_t e = cudaMemsetAsync(a.dg_pre, 0, 4 * static_cast<size_t>(a.d), stream);
        if (e == cudaSuccess)
            e = cudaMemsetAsync(a.dg_post, 0, 4 * static_cast<size_t>(a.d), stream);
        if (e == cudaSuccess && a.gate_mode == kGateChannel)
            e = cudaMemsetAsync(a.dgate, 0, 4 * static_cast<size_t>(a.d), stream);
        return e;
    }
    DeviceInfo di;
    cudaError_t e = current_device_info(&di);
    if (e != cudaSuccess)
        return e;
    const NormPlan p = plan_backward(a.T, static_cast<int>(a.d), a.gate_mode, di.num_sms);
    const bool vec = a.d % 8 == 0;
    switch (p.v) {
    case 1:
        return vec ? backward_gate<1, true>(p, a, di.device, stream) : backward_gate<1, false>(p, a, di.device, stream);
    case 2:
        return vec ? backward_gate<2, true>(p, a, di.device, stream) : backward_gate<2, false>(p, a, di.device, stream);
    default:
        return vec ? backward_gate<4, true>(p, a, di.device, stream) : backward_gate<4, false>(p, a, di.device, stream);
    }
}

}  // namespace taco
