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
//   G      = dh' + r_h (u - h' r_h^2 mean(u h'))    (gradient at h')
//   dh     = s G
//   v      = G gate g_post
//   dy     = r_y (v - y r_y^2 mean(v y))
//   dg_pre = sum_t dn h' r_h,  dg_post = sum_t gate G y r_y
//   dgate  = G y r_y g_post, summed over what the gate is shared by
//
// The backward pass recomputes both root mean squares from its inputs: they
// cost no extra pass, as the row is held anyway, and nothing has to be saved
// beside y and h'.  All of it is fp32 (sums, statistics, gradients); values
// are rounded once, when they are stored.
//
// Bound by HBM: 8 bytes an element forward, 12 backward.  A CTA takes whole
// rows in turn, 8 V columns a thread and RPI rows at a time, with the gains
// of its columns in registers.  Rows arrive by bulk copies into a ring of row
// slots in shared memory, several rows ahead of those being worked on, so
// the loads do not wait for the two block-wide sums that every row needs;
// outputs go straight from registers in 16-byte stores.  With one unit a
// thread two rows at a time share a barrier and hide each other's latencies.
// Measured with a channel gate at 8192 rows: forward 4096 columns 44 us (6050
// GB/s), to FP8 48 (4900), 2048 columns 17 (7750, part of it in L2), 5120 57
// (5850), full gate 64 (6550); backward 4096 columns 76 (5300), 2560 59
// (4230), 5120 104 (4850).
//
// Rows that are not a multiple of 16 bytes start anywhere inside a 16-byte
// granule of memory.  A CTA's rows are a multiple of eight apart, so all of
// them start at the same place, `shift` elements into one.  The ring holds a
// row's granules; a thread joins its eight columns from two of them, and
// stores the granule that ends in its columns, with the first elements from
// the lane below.  (Threads that take granules instead of columns would skip
// that, but then a row's sums, and so its last bits, depend on which row of
// the tensor it is.)  8192 x 4095: 82 us forward and 127 backward, against
// 254 and 331 with loads and stores of single elements, and 44 and 76 at 4096
// columns; bound by the integer instructions that join and split.
//
// The gains' gradients are summed over a CTA's rows in registers, written as
// one partial row per CTA, and added over the CTAs in a fixed order by a
// second small kernel: no atomics, the same bits every time.

#include "device_utils.cuh"
#include "fp8_block.cuh"
#include "internal.h"

namespace taco {

// Watchdog flag of this file's kernels (bit 7), read by taco_device_error().
__device__ unsigned int g_norm_error;

namespace {

constexpr uint32_t kErrNorm = 128u;
constexpr int kMaxThreads = 512;
constexpr int kMaxSlots = 8;

// Gate modes (include/taco.h).
constexpr int kGateNone = 0, kGateChannel = 1, kGateToken = 2, kGateFull = 3;

// Eight values in four float2 registers: the arithmetic runs as packed
// fp32x2 instructions (two lanes each).
struct F8 {
    float2 v[4];
};
__device__ __forceinline__ float2 both(float a) { return make_float2(a, a); }
__device__ __forceinline__ float2 operator*(float2 a, float2 b) { return __fmul2_rn(a, b); }
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) { return __ffma2_rn(a, b, c); }

// Eight bf16 values of a packed 16-byte unit.
__device__ __forceinline__ F8 unpack8(const uint4 &q)
{
    F8 x;
    x.v[0] = make_float2(bf16lo_to_f32(q.x), bf16hi_to_f32(q.x));
    x.v[1] = make_float2(bf16lo_to_f32(q.y), bf16hi_to_f32(q.y));
    x.v[2] = make_float2(bf16lo_to_f32(q.z), bf16hi_to_f32(q.z));
    x.v[3] = make_float2(bf16lo_to_f32(q.w), bf16hi_to_f32(q.w));
    return x;
}

__device__ __forceinline__ uint4 pack8(const F8 &x)
{
    return make_uint4(f32x2_to_bf16x2(x.v[0].x, x.v[0].y), f32x2_to_bf16x2(x.v[1].x, x.v[1].y),
                      f32x2_to_bf16x2(x.v[2].x, x.v[2].y), f32x2_to_bf16x2(x.v[3].x, x.v[3].y));
}

// Columns c .. c + 7 of fp32 vectors of d values, zeros past the end (VEC: d is
// a multiple of 8).
template <bool VEC> __device__ __forceinline__ F8 load_f32x8(const float *p, int c, int d)
{
    F8 x;
    if (VEC || c + 8 <= d || c >= d) {
        float4 a = make_float4(0, 0, 0, 0), b = a;
        if (c < d) {
            a = __ldg(reinterpret_cast<const float4 *>(p + c));
            b = __ldg(reinterpret_cast<const float4 *>(p + c) + 1);
        }
        x.v[0] = make_float2(a.x, a.y);
        x.v[1] = make_float2(a.z, a.w);
        x.v[2] = make_float2(b.x, b.y);
        x.v[3] = make_float2(b.z, b.w);
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
            x.v[j] = make_float2(c + 2 * j < d ? __ldg(p + c + 2 * j) : 0.0f,
                                 c + 2 * j + 1 < d ? __ldg(p + c + 2 * j + 1) : 0.0f);
    }
    return x;
}

// Elements first .. last - 1 of q to p + first ..
__device__ __forceinline__ void store_elements(uint16_t *p, const uint4 &q, int first, int last)
{
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int j = 0; j < 8; ++j)
        if (j >= first && j < last)
            p[j] = static_cast<uint16_t>(w[j >> 1] >> (16 * (j & 1)));
}

// Columns c .. c + 7 of the row p, which starts `shift` elements into a
// granule (all lanes of a warp, with 256 columns, call this).
template <bool VEC> __device__ __forceinline__ void store_bf16x8(uint16_t *p, int c, int shift, int d, const F8 &x)
{
    uint4 q = pack8(x);
    if (VEC || shift == 0) {
        if (c + 8 <= d)
            stg128_stream(p + c, q);
        else if (!VEC)
            store_elements(p + c, q, 0, d - c);
        return;
    }
    const int lane = threadIdx.x & 31;
    uint4 below;
    below.x = __shfl_up_sync(0xFFFFFFFFu, q.x, 1);
    below.y = __shfl_up_sync(0xFFFFFFFFu, q.y, 1);
    below.z = __shfl_up_sync(0xFFFFFFFFu, q.z, 1);
    below.w = __shfl_up_sync(0xFFFFFFFFu, q.w, 1);
    // the warp's first granule starts in the warp below, its last one ends in
    // the warp above: lanes 0 and 31 store what is the warp's own in them
    if (lane == 0 || lane == 31)
        store_elements(p + c, q, lane ? 8 - shift : 0, min(lane ? 8 : 8 - shift, d - c));
    if (lane == 0)
        return;
    q = join(below, q, 8 - shift);
    if (c - shift + 8 <= d)
        stg128_stream(p + c - shift, q);
    else
        store_elements(p + c - shift, q, 0, d - c + shift);
}

// The CTA's rows blockIdx.x, + gridDim.x, ...: NT bf16 tensors' rows, NT
// row-sized pieces to a slot, each from the granule that its row starts in.
// `row` and `slot` are those of the first row being worked on, row(i) and
// slot i places on those of the ones after it.
template <int NT, bool VEC> struct RowRing {
    const uint16_t *src[NT];
    uint32_t buf, bars, slots, pitch;  // pitch: bytes of a piece
    int64_t T, row0;
    int d;
    int shift;  // elements between a granule's start and a row's, the same for all rows of the CTA
    uint32_t slot = 0, phase = 0;
    bool dead = false;

    __device__ __forceinline__ int64_t row(int i) const { return row0 + static_cast<int64_t>(i) * gridDim.x; }
    __device__ __forceinline__ uint32_t slot_of(int i) const
    {
        const uint32_t s = slot + i;
        return s >= slots ? s - slots : s;
    }
    // Elements from row r's start to the end of the tensor's whole granules:
    // copies take no more than those, what lies behind is read directly.
    __device__ __forceinline__ int64_t whole(int64_t r) const { return (T * d & ~int64_t(7)) - r * d; }
    __device__ __forceinline__ void issue(int64_t r, uint32_t s)  // row r into slot s (one thread)
    {
        if (r >= T)
            return;
        const uint32_t bar = bars + 8 * s;
        uint32_t bytes = pitch;
        if (!VEC)
            bytes = 2 * static_cast<uint32_t>(min(static_cast<int64_t>((shift + d + 7) & ~7), whole(r) + shift));
        mbar_arrive_expect_tx(bar, NT * bytes);
        if (!VEC && bytes == 0)
            return;
#pragma unroll
        for (int k = 0; k < NT; ++k)
            bulk_load(buf + (s * NT + k) * pitch, src[k] + r * d - shift, bytes, bar);
    }
    __device__ __forceinline__ void start()
    {
        row0 = blockIdx.x;
        shift = VEC ? 0 : static_cast<int>(blockIdx.x & 7) * (d & 7) & 7;
        if (threadIdx.x == 0)
            for (uint32_t s = 0; s < slots; ++s)
                issue(row(s), s);
    }
    // Row i has landed.
    __device__ __forceinline__ void wait(int i)
    {
        if (!dead && row(i) < T && !mbar_wait(bars + 8 * slot_of(i), phase ^ (slot + i >= slots))) {
            atomicOr(&g_norm_error, kErrNorm);
            dead = true;
            // the thread that issues stops issuing: wait for what is in flight
            if (threadIdx.x == 0)
                for (int j = i; j < static_cast<int>(slots) && row(j) < T; ++j)
                    mbar_wait(bars + 8 * slot_of(j), phase ^ (slot + j >= slots));
        }
    }
    // Columns c .. c + 7 of tensor k's row i, zeros past the end.
    __device__ __forceinline__ uint4 get(int i, int k, int c) const
    {
        if (row(i) >= T || c >= d || dead)
            return make_uint4(0, 0, 0, 0);
        const uint32_t at = buf + (slot_of(i) * NT + k) * pitch + 2 * c;
        uint4 q;
        if (VEC) {
            q = lds128(at);
        } else if (c + 8 > whole(row(i))) {
            const uint16_t *p = src[k] + row(i) * d + c;
            uint32_t e[8];
#pragma unroll
            for (int j = 0; j < 8; ++j)
                e[j] = c + j < d ? __ldg(p + j) : 0u;
            q = make_uint4(e[0] | e[1] << 16, e[2] | e[3] << 16, e[4] | e[5] << 16, e[6] | e[7] << 16);
        } else {
            q = lds128(at);
            if (shift != 0)
                q = join(q, lds128(at + 16), shift);
            if (c + 8 > d)
                q = first_elements(q, d - c);
        }
        return q;
    }
    // Every thread has read row i (a barrier lies behind): refill its slot.
    __device__ __forceinline__ void refill(int i)
    {
        if (threadIdx.x == 0 && !dead)
            issue(row(i + static_cast<int>(slots)), slot_of(i));
    }
    __device__ __forceinline__ void next(int rows)
    {
        row0 = row(rows);
        slot += rows;
        if (slot >= slots) {
            slot -= slots;
            phase ^= 1;
        }
    }
};

// Sums of K values over the CTA of at most WARPS warps; every thread gets
// them.  `red` holds WARPS floats for each of K values rounded up to a power
// of two; two calls in turn
// use two of them, so that one barrier a call is enough.  A warp sums all K
// together: in each halving step a lane passes on half of its values and
// keeps the other half, so that the K sums take about K + 5 shuffles and
// land in groups of lanes; the warps' sums are added the same way.
__host__ __device__ constexpr int pow2_at_least(int k) { return k <= 1 ? 1 : k <= 2 ? 2 : k <= 4 ? 4 : 8; }

template <int WARPS, int K> __device__ __forceinline__ void block_sum(float (&v)[K], float *red)
{
    constexpr int P = pow2_at_least(K);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
    float x[P];
#pragma unroll
    for (int k = 0; k < P; ++k)
        x[k] = k < K ? v[k] : 0.0f;
    // after the step with distance s, a lane whose bit s is set holds the
    // upper half of the values
    int dist = 16;
#pragma unroll
    for (int n = P; n > 1; n >>= 1, dist >>= 1) {
        const bool up = lane & dist;
#pragma unroll
        for (int k = 0; k < n / 2; ++k) {
            const float give = up ? x[k] : x[k + n / 2], keep = up ? x[k + n / 2] : x[k];
            x[k] = keep + __shfl_xor_sync(0xFFFFFFFFu, give, dist);
        }
    }
#pragma unroll
    for (int s = 16 / P; s >= 1; s >>= 1)
        x[0] += __shfl_xor_sync(0xFFFFFFFFu, x[0], s);
    // lanes 32 / P i .. hold value i
    if ((lane & (32 / P - 1)) == 0)
        red[WARPS * (lane / (32 / P)) + warp] = x[0];
    __syncthreads();
    constexpr int Q = P * WARPS >= 32 ? P * WARPS / 32 : 1;  // warps a lane adds
    constexpr int L = WARPS / Q;                             // lanes to a value
    const int i = lane / L < P ? lane / L : P - 1, w0 = (lane % L) * Q;
    float sum = 0.0f;
#pragma unroll
    for (int q = 0; q < Q; ++q)
        sum += w0 + q < warps ? red[WARPS * i + w0 + q] : 0.0f;
#pragma unroll
    for (int s = L / 2; s >= 1; s >>= 1)
        sum += __shfl_xor_sync(0xFFFFFFFFu, sum, s);
#pragma unroll
    for (int k = 0; k < K; ++k)
        v[k] = P == 1 ? sum : __shfl_sync(0xFFFFFFFFu, sum, k * L);
}

// Bytes of a row's piece in the ring: whole granules from the one it starts in.
__host__ __device__ inline uint32_t ring_pitch(int d) { return d % 8 == 0 ? 2 * d : 2 * ((d + 7) / 8 * 8 + 8); }

template <int NT, bool VEC>
__device__ __forceinline__ void ring_init(RowRing<NT, VEC> &ring, uint8_t *smem, uint32_t bars, int64_t T, int d,
                                          int slots)
{
    ring.buf = (smem_u32(smem) + 127u) & ~127u;
    ring.bars = bars;
    ring.slots = slots;
    ring.pitch = ring_pitch(d);
    ring.T = T;
    ring.d = d;
    if (threadIdx.x == 0) {
        for (int s = 0; s < slots; ++s)
            mbar_init(bars + 8 * s, 1);
        fence_barrier_init();
        fence_proxy_async_smem();
    }
    __syncthreads();
}

// Tokens' gates of the CTA's next kGateRows rows in shared memory (loaded row
// by row they stood in every round's way: 8192 x 4096 forward 50 us against 46,
// backward 96 against 79, 8192 x 5120 backward 126 against 111).  The arrays in
// static shared memory take at most 2 KB together.
constexpr int kGateRows = 128;
struct TokenGates {
    float *at;
    int used = kGateRows;
    __device__ __forceinline__ explicit TokenGates(float *rows) : at(rows) {}
    // `rows` rows at ring.row(0) are about to be worked on, after `rows` others.
    template <class R> __device__ __forceinline__ void next(int rows, const float *gate, const R &ring)
    {
        used += rows;
        if (used < kGateRows)
            return;
        __syncthreads();  // the last of the previous ones have been read
        for (int i = threadIdx.x; i < kGateRows; i += blockDim.x)
            at[i] = ring.row(i) < ring.T ? __ldg(gate + ring.row(i)) : 0.0f;
        __syncthreads();
        used = 0;
    }
};

// ---------------------------------------------------------------- forward --

// V units of 8 columns a thread (unit threadIdx.x + v blockDim.x), RPI rows
// at a time; GATE a gate mode; FP8: n as codes and scales.
// Two units a thread of rows inside granules: the bound of 640 threads, more
// than any launch has, is there for the 96 registers that it leaves, with
// which two CTAs of up to 5440 columns share an SM (8192 x 5119: 91 us
// against 132 with 118; 8192 x 6001 with a full gate 178 against 163).
template <int V, int RPI, int GATE, bool FP8, bool VEC, bool DENSE>
__global__ void __launch_bounds__(V == 2 && !VEC ? 640 : kMaxThreads, DENSE ? 2 : 1)
    norm_forward_kernel(const uint16_t *__restrict__ y, const uint16_t *__restrict__ h,
                        const float *__restrict__ g_post, const float *__restrict__ g_pre,
                        const void *__restrict__ gate, float s, float eps, int64_t T, int d, int slots,
                        uint16_t *__restrict__ h_out, void *__restrict__ n_out, uint8_t *__restrict__ n_scale)
{
    constexpr int NT = GATE == kGateFull ? 3 : 2;
    extern __shared__ uint8_t smem_raw[];
    __shared__ uint64_t bars[kMaxSlots];
    // tokens' gates ahead in shared memory; with more units a thread the
    // registers that takes cost more (5120 columns: 59 us against 52)
    constexpr bool AHEAD = GATE == kGateToken && V == 1;
    __shared__ float gate_rows[AHEAD ? kGateRows : 1];
    __shared__ float red[2][16 * pow2_at_least(RPI)];
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
    // the columns' gains: a channel gate joins g_post
    F8 gp[V], gq[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int c = 8 * (threadIdx.x + v * blockDim.x);
        gp[v] = load_f32x8<VEC>(g_post, c, d);
        gq[v] = load_f32x8<VEC>(g_pre, c, d);
        if constexpr (GATE == kGateChannel) {
            const F8 w = load_f32x8<VEC>(static_cast<const float *>(gate), c, d);
#pragma unroll
            for (int j = 0; j < 4; ++j)
                gp[v].v[j] = gp[v].v[j] * w.v[j];
        }
    }
    TokenGates gates(gate_rows);
    for (; ring.row(0) < T; ring.next(RPI)) {
        if constexpr (AHEAD)
            gates.next(RPI, static_cast<const float *>(gate), ring);
        uint4 qy[RPI][V], qh[RPI][V], qg[RPI][V];
        float sum[RPI], gt[RPI];
#pragma unroll
        for (int i = 0; i < RPI; ++i) {
            ring.wait(i);
            gt[i] = 1.0f;
            if constexpr (AHEAD)
                gt[i] = gates.at[gates.used + i];
            else if constexpr (GATE == kGateToken)
                if (ring.row(i) < T)
                    gt[i] = __ldg(static_cast<const float *>(gate) + ring.row(i));
            float2 ss = both(0.0f);
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const int c = 8 * (threadIdx.x + v * blockDim.x);
                qy[i][v] = ring.get(i, 0, c);
                qh[i][v] = ring.get(i, 1, c);
                if constexpr (GATE == kGateFull)
                    qg[i][v] = ring.get(i, 2, c);
                const F8 x = unpack8(qy[i][v]);
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    ss = fma2(x.v[j], x.v[j], ss);
            }
            sum[i] = ss.x + ss.y;
        }
        block_sum<16>(sum, red[0]);
#pragma unroll
        for (int i = 0; i < RPI; ++i)
            ring.refill(i);
        F8 h2[RPI][V];
#pragma unroll
        for (int i = 0; i < RPI; ++i) {
            const float2 ry = both(rsqrtf(sum[i] * inv_d + eps) * gt[i]), s2 = both(s);
            float2 ss = both(0.0f);
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const int c = 8 * (threadIdx.x + v * blockDim.x);
                const F8 x = unpack8(qy[i][v]);
                h2[i][v] = unpack8(qh[i][v]);
                F8 w;
                if constexpr (GATE == kGateFull)
                    w = unpack8(qg[i][v]);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    float2 z = x.v[j] * ry * gp[v].v[j];
                    if constexpr (GATE == kGateFull)
                        z = z * w.v[j];
                    h2[i][v].v[j] = fma2(s2, h2[i][v].v[j], z);
                    ss = fma2(h2[i][v].v[j], h2[i][v].v[j], ss);
                }
                if (ring.row(i) < T)
                    store_bf16x8<VEC>(h_out + ring.row(i) * d, c, ring.shift, d, h2[i][v]);
            }
            sum[i] = ss.x + ss.y;
        }
        block_sum<16>(sum, red[1]);
#pragma unroll
        for (int i = 0; i < RPI; ++i) {
            const int64_t row = ring.row(i);
            if (row >= T)
                break;
            const float2 rh = both(rsqrtf(sum[i] * inv_d + eps));
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const int c = 8 * (threadIdx.x + v * blockDim.x);
                F8 n;
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    n.v[j] = h2[i][v].v[j] * rh * gq[v].v[j];
                if constexpr (FP8) {
                    // the block's maximum: 16 lanes of 8 columns
                    uint32_t m = 0;
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        m = max(m, max(__float_as_uint(n.v[j].x) & 0x7FFFFFFFu,
                                       __float_as_uint(n.v[j].y) & 0x7FFFFFFFu));
#pragma unroll
                    for (int k = 8; k >= 1; k >>= 1)
                        m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, k));
                    const uint32_t byte = fp8_scale_byte(m);
                    const float2 f = both(fp8_inv_scale(byte));
                    const int64_t pitch = fp8_pitch(d);
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        n.v[j] = n.v[j] * f;
                    if (c < pitch)
                        *reinterpret_cast<uint2 *>(static_cast<uint8_t *>(n_out) + row * pitch + c) =
                            make_uint2(f32x4_to_e4m3x4(n.v[0].x, n.v[0].y, n.v[1].x, n.v[1].y),
                                       f32x4_to_e4m3x4(n.v[2].x, n.v[2].y, n.v[3].x, n.v[3].y));
                    if ((threadIdx.x & 15) == 0 && c < d)
                        n_scale[fp8_scale_at(row, c >> 7, (d + 511) / 512)] = static_cast<uint8_t>(byte);
                } else {
                    store_bf16x8<VEC>(static_cast<uint16_t *>(n_out) + row * d, c, ring.shift, d, n);
                }
            }
        }
    }
}

// --------------------------------------------------------------- backward --

// MAXT: the most threads of a CTA (512, or 768 with one row at a time in 80
// registers).
template <int V, int RPI, int MAXT, int GATE, bool VEC>
__global__ void __launch_bounds__(MAXT, 1)
    norm_backward_kernel(const uint16_t *__restrict__ dn, const uint16_t *__restrict__ dh2,
                         const uint16_t *__restrict__ y, const uint16_t *__restrict__ h2,
                         const float *__restrict__ g_post, const float *__restrict__ g_pre,
                         const void *__restrict__ gate, float s, float eps, int64_t T, int d, int slots,
                         uint16_t *__restrict__ dy, uint16_t *__restrict__ dh, void *__restrict__ dgate,
                         float *__restrict__ partial)
{
    constexpr int NT = GATE == kGateFull ? 5 : 4;
    // more columns a thread: no registers left for the gains, which are then
    // read (from L1) where they are used
    constexpr bool KEEP = V == 1;
    constexpr int WARPS = MAXT > 512 ? 32 : 16;
    extern __shared__ uint8_t smem_raw[];
    __shared__ uint64_t bars[kMaxSlots];
    __shared__ float gate_rows[GATE == kGateToken ? kGateRows : 1];
    __shared__ float red[2][WARPS * pow2_at_least(3 * RPI)];
    RowRing<NT, VEC> ring;
    ring.src[0] = dn;
    ring.src[1] = dh2;
    ring.src[2] = y;
    ring.src[3] = h2;
    if constexpr (GATE == kGateFull)
        ring.src[4] = static_cast<const uint16_t *>(gate);
    ring_init(ring, smem_raw, smem_u32(bars), T, d, slots);
    const float inv_d = 1.0f / static_cast<float>(d);
    F8 a_pre[V], a_post[V];
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
        for (int j = 0; j < 4; ++j)
            a_pre[v].v[j] = a_post[v].v[j] = both(0.0f);
    if (T <= 4 * static_cast<int64_t>(gridDim.x))  // short: the next kernel's launch overlaps it
        pdl_trigger();
    pdl_wait();
    ring.start();
    // the columns' gains: a channel gate joins g_post (the sum a_post holds
    // neither)
    F8 gp[KEEP ? V : 1], gq[KEEP ? V : 1];
    auto post_gain = [&](int c) {
        F8 g = load_f32x8<VEC>(g_post, c, d);
        if constexpr (GATE == kGateChannel) {
            const F8 w = load_f32x8<VEC>(static_cast<const float *>(gate), c, d);
#pragma unroll
            for (int j = 0; j < 4; ++j)
                g.v[j] = g.v[j] * w.v[j];
        }
        return g;
    };
    if constexpr (KEEP) {
        gp[0] = post_gain(8 * threadIdx.x);
        gq[0] = load_f32x8<VEC>(g_pre, 8 * threadIdx.x, d);
    }
    TokenGates gates(gate_rows);
    for (; ring.row(0) < T; ring.next(RPI)) {
        if constexpr (GATE == kGateToken)
            gates.next(RPI, static_cast<const float *>(gate), ring);
        uint4 qn[RPI][V], qd[RPI][V], qy[RPI][V], qh[RPI][V], qg[RPI][V];
        float sum[3 * RPI], gt[RPI];
#pragma unroll
        for (int i = 0; i < RPI; ++i) {
            ring.wait(i);
            gt[i] = 1.0f;
            if constexpr (GATE == kGateToken)
                gt[i] = gates.at[gates.used + i];
            float2 s0 = both(0.0f), s1 = s0, s2 = s0;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const int c = 8 * (threadIdx.x + v * blockDim.x);
                qn[i][v] = ring.get(i, 0, c);
                qd[i][v] = ring.get(i, 1, c);
                qy[i][v] = ring.get(i, 2, c);
                qh[i][v] = ring.get(i, 3, c);
                if constexpr (GATE == kGateFull)
                    qg[i][v] = ring.get(i, 4, c);
                if constexpr (!KEEP)
                    gq[0] = load_f32x8<VEC>(g_pre, c, d);
                const F8 a = unpack8(qh[i][v]), b = unpack8(qn[i][v]), y8 = unpack8(qy[i][v]);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    s0 = fma2(a.v[j], a.v[j], s0);
                    s1 = fma2(b.v[j] * gq[0].v[j], a.v[j], s1);
                    s2 = fma2(y8.v[j], y8.v[j], s2);
                }
            }
            sum[3 * i] = s0.x + s0.y;
            sum[3 * i + 1] = s1.x + s1.y;
            sum[3 * i + 2] = s2.x + s2.y;
        }
        block_sum<WARPS>(sum, red[0]);
#pragma unroll
        for (int i = 0; i < RPI; ++i)
            ring.refill(i);
        F8 G[RPI][V];
        float dot[RPI], ry[RPI];
#pragma unroll
        for (int i = 0; i < RPI; ++i) {
            // a row past the end is all zeros and adds nothing: no product
            // of two reciprocal roots is formed (they reach 2^75), only of one
            // with a mean or a value that it brings back into range
            const float r1 = rsqrtf(sum[3 * i] * inv_d + eps);
            const float2 rh = both(r1), ch = both(-r1 * (r1 * (sum[3 * i + 1] * inv_d)));
            ry[i] = rsqrtf(sum[3 * i + 2] * inv_d + eps);
            const float2 ry2 = both(ry[i]), gt2 = both(gt[i]), s2 = both(s);
            float2 dd = both(0.0f);
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const int c = 8 * (threadIdx.x + v * blockDim.x);
                if constexpr (!KEEP) {
                    gq[0] = load_f32x8<VEC>(g_pre, c, d);
                    gp[0] = post_gain(c);
                }
                const F8 a = unpack8(qh[i][v]), b = unpack8(qn[i][v]);
                G[i][v] = unpack8(qd[i][v]);
                F8 o;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float2 x = rh * a.v[j];
                    a_pre[v].v[j] = fma2(x, b.v[j], a_pre[v].v[j]);
                    G[i][v].v[j] = fma2(x, ch, fma2(rh * b.v[j], gq[0].v[j], G[i][v].v[j]));
                    o.v[j] = s2 * G[i][v].v[j];
                }
                if (ring.row(i) < T)
                    store_bf16x8<VEC>(dh + ring.row(i) * d, c, ring.shift, d, o);
                // y r_y G: the sum over tokens behind dg_post and a channel
                // gate's gradient
                const F8 y8 = unpack8(qy[i][v]);
                F8 w;
                if constexpr (GATE == kGateFull)
                    w = unpack8(qg[i][v]);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float2 t = y8.v[j] * ry2 * G[i][v].v[j];
                    if constexpr (GATE == kGateFull) {
                        o.v[j] = t * gp[0].v[j];
                        dd = fma2(o.v[j], w.v[j], dd);
                        a_post[v].v[j] = fma2(t, w.v[j], a_post[v].v[j]);
                    } else {
                        dd = fma2(t, gp[0].v[j], dd);
                        a_post[v].v[j] = GATE == kGateToken ? fma2(gt2, t, a_post[v].v[j])
                                                            : __fadd2_rn(a_post[v].v[j], t);
                    }
                }
                if constexpr (GATE == kGateFull)
                    if (ring.row(i) < T)
                        store_bf16x8<VEC>(static_cast<uint16_t *>(dgate) + ring.row(i) * d, c, ring.shift, d, o);
            }
            dot[i] = dd.x + dd.y;
        }
        block_sum<WARPS>(dot, red[1]);  // sum of (y r_y) G g_post (and a channel's or element's gate)
#pragma unroll
        for (int i = 0; i < RPI; ++i) {
            const int64_t row = ring.row(i);
            if (row >= T)
                break;
            if constexpr (GATE == kGateToken)
                if (threadIdx.x == 0)
                    static_cast<float *>(dgate)[row] = dot[i];
            const float2 cy = both(-ry[i] * (dot[i] * inv_d)), rg = both(ry[i] * gt[i]);
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const int c = 8 * (threadIdx.x + v * blockDim.x);
                if constexpr (!KEEP)
                    gp[0] = post_gain(c);
                F8 o = unpack8(qy[i][v]), w;
                if constexpr (GATE == kGateFull)
                    w = unpack8(qg[i][v]);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    float2 u = gp[0].v[j];
                    if constexpr (GATE == kGateFull)
                        u = u * w.v[j];
                    o.v[j] = rg * fma2(u, G[i][v].v[j], o.v[j] * cy);
                }
                store_bf16x8<VEC>(dy + row * d, c, ring.shift, d, o);
            }
        }
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int c = 8 * (threadIdx.x + v * blockDim.x);
        float *p = partial + static_cast<int64_t>(blockIdx.x) * 2 * d;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if (c + 2 * j < d) {
                p[c + 2 * j] = a_pre[v].v[j].x;
                p[d + c + 2 * j] = a_post[v].v[j].x;
            }
            if (c + 2 * j + 1 < d) {
                p[c + 2 * j + 1] = a_pre[v].v[j].y;
                p[d + c + 2 * j + 1] = a_post[v].v[j].y;
            }
        }
    }
}

// Sums the CTAs' partial rows in a fixed order: 32 columns a CTA, sixteen
// groups of rows in turn, then the groups.  One CTA an SM leaves 152 rows, so
// a thread's ten loads of each half are all in flight (in fives: 1.1 us
// longer).
constexpr int kGainLoads = 10;

__global__ void __launch_bounds__(512)
    norm_gains_kernel(const float *__restrict__ partial, int ctas, int d, int gate_mode,
                      const float *__restrict__ g_post, const float *__restrict__ gate, float *__restrict__ dg_pre,
                      float *__restrict__ dg_post, float *__restrict__ dgate)
{
    __shared__ float part[2][16][33];
    const int lane = threadIdx.x & 31, grp = threadIdx.x >> 5, c = blockIdx.x * 32 + lane;
    pdl_wait();
    float a = 0.0f, b = 0.0f;
    if (c < d)
        for (int i0 = grp; i0 < ctas; i0 += 16 * kGainLoads) {
            float va[kGainLoads], vb[kGainLoads];
#pragma unroll
            for (int k = 0; k < kGainLoads; ++k) {
                const int i = i0 + 16 * k;
                const float *p = partial + static_cast<int64_t>(i) * 2 * d + c;
                va[k] = i < ctas ? p[0] : 0.0f;
                vb[k] = i < ctas ? p[d] : 0.0f;
            }
#pragma unroll
            for (int k = 0; k < kGainLoads; ++k) {
                a += va[k];
                b += vb[k];
            }
        }
    part[0][grp][lane] = a;
    part[1][grp][lane] = b;
    __syncthreads();
    if (grp == 0 && c < d) {
        a = b = 0.0f;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
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

// Threads, units a thread, ring slots and CTAs of a shape.
struct NormPlan {
    int threads, v, slots, grid;
    bool dense;    // forward: registers bounded to 64
    bool one_row;  // backward: one row at a time with one unit a thread
    uint32_t smem;
};

constexpr uint32_t kSmemPerSm = 227 * 1024;
constexpr uint32_t kMaxSmem = kSmemPerSm - 2048;  // of a CTA, beside its static arrays

// CTAs whose registers an SM holds (a quarter of them in each of its four
// partitions), eight at most.
int ctas_of(int regs, int threads)
{
    const int n = 4 * (16384 / (32 * regs)) / (threads / 32);
    return n < 1 ? 1 : n > 8 ? 8 : n;
}

// v: units a thread; tensors: rows to a slot; min_rows: the fewest rows in the
// ring of a CTA that shares its SM; regs: the registers a thread of the
// kernel takes, for how many CTAs share an SM.
NormPlan plan_norm(int64_t T, int d, int v, int tensors, int min_rows, int regs, int sms)
{
    NormPlan p = {};
    const int units = (d + 7) / 8;
    p.v = v;
    p.threads = ((units + p.v - 1) / p.v + 31) / 32 * 32;
    int per_sm = ctas_of(regs, p.threads);
    const uint32_t slot = static_cast<uint32_t>(tensors) * ring_pitch(d);
    while (per_sm > 1 && min_rows * slot + 2048 + 128 > kSmemPerSm / per_sm)
        --per_sm;
    const uint32_t room = kSmemPerSm / per_sm - 2048 - 128;  // static arrays; the ring's alignment
    p.slots = static_cast<int>(room / slot);
    p.slots = p.slots > kMaxSlots ? kMaxSlots : p.slots;
    p.smem = 128 + p.slots * slot;
    // a multiple of eight, so that a CTA's rows all start at the same place
    // of a granule (with fewer CTAs each has one row)
    int64_t most = static_cast<int64_t>(per_sm) * sms / 8 * 8;
    most = most < 8 ? 8 : most;
    p.grid = static_cast<int>(T < most ? T : most);
    return p;
}

// An FP8 output works longer on a row once its sums are there, as rows inside
// granules do, and gains more from a second CTA than from a fourth row in the
// ring: 8192 x 5120 with a full gate, three rows against four (one CTA): FP8
// 63 and 81 us, bf16 71 and 66.
//
// One unit a thread and two rows at a time, or two units and one row, with
// more and smaller CTAs.  Measured at 8192 rows, channel gate, one unit
// against two: bf16 1280 columns 13.3 and 13.5 us, 1536 16.5 and 13.2, 2048
// 21.3 and 17.3, 2560 28.0 and 28.8, 3200 37.0 and 34.6, 3584 43.0 and 39.9,
// 4096 44.4 and 48.0; FP8 16.3 and 17.1, 20.7 and 16.9, 25.1 and 21.1, 33.9
// and 27.9, 45.3 and 43.5, 45.7 and 43.5, 48.2 and 44.3 (but both outputs
// have to come from the same sums).  With a full gate two units stop paying
// at 3584 columns (47 and 51 us); rows inside granules at 384 units (2945
// columns 85 and 79 us, 3073 90 and 99).
//
// dense: to FP8 with one unit a thread above 448 units (4096 columns: 54 us
// in 96 registers, one CTA an SM, 48 in 64, two).
NormPlan plan_forward(int64_t T, int d, int gate_mode, bool fp8, int sms)
{
    const bool inside = d % 8 != 0;
    const int units = (d + 7) / 8;
    const int v = units > 2 * kMaxThreads ? 4
                  : units > kMaxThreads || (units > 160 && units <= (inside ? 384 : 448)) ? 2 : 1;
    const bool dense = fp8 && !inside && v == 1 && units > 448;
    const int regs = dense ? 64 : v == 4 ? 128 : 96;
    NormPlan p = plan_norm(T, d, v, gate_mode == kGateFull ? 3 : 2, fp8 || inside ? 3 : 4, regs, sms);
    p.dense = dense;
    return p;
}

// Backward, one unit a thread: two rows at a time in 128 registers up to 512
// threads, above that (up to 768) one row at a time in 80.  Many rows of 2056
// to 2560 columns are also taken one at a time: two CTAs then share an SM,
// where the two-row kernel's registers leave room for one of 288 or 320
// threads.  Measured, one against two rows: 8192 x 1024 30 and 26 us, 8192 x
// 2048 49 and 45, 8192 x 2304 58 and 64, 8192 x 2560 59 and 65, 4096 x 2560 36
// and 38, 2048 x 2560 22 and 21, 8192 x 2816 64 and 66 (with a full gate 75
// and 75), 8192 x 4096 94 and 76, 8192 x 2561 120 and 110; at 5120, 104 us
// against 167 with two units a thread.
constexpr int kWide = 768;
bool one_row(int64_t T, int d, int sms)
{
    return (d > 8 * kMaxThreads && d <= 8 * kWide) || (d > 2048 && d <= 2560 && d % 8 == 0 && T >= 24 * sms);
}

NormPlan plan_backward(int64_t T, int d, int gate_mode, int sms)
{
    const bool one = one_row(T, d, sms);
    const int units = (d + 7) / 8, v = one || units <= kMaxThreads ? 1 : units <= 2 * kMaxThreads ? 2 : 4;
    NormPlan p = plan_norm(T, d, v, gate_mode == kGateFull ? 5 : 4, 4, one ? 80 : 128, sms);
    p.one_row = one;
    return p;
}

// Two rows at a time where a thread has one unit.
constexpr int rows_at_once(int v) { return v == 1 ? 2 : 1; }

template <int V, int GATE, bool FP8, bool VEC, bool DENSE = false>
cudaError_t run_forward(const NormPlan &p, const NormForward &a, int device, cudaStream_t stream)
{
    if constexpr (V == 1 && FP8 && VEC && !DENSE)
        if (p.dense)
            return run_forward<V, GATE, FP8, VEC, true>(p, a, device, stream);
    static std::atomic<bool> set[kMaxDevices];
    cudaError_t e = ensure_smem(norm_forward_kernel<V, rows_at_once(V), GATE, FP8, VEC, DENSE>, kMaxSmem, device, set);
    if (e != cudaSuccess)
        return e;
    return launch_pdl(norm_forward_kernel<V, rows_at_once(V), GATE, FP8, VEC, DENSE>, dim3(p.grid), dim3(p.threads),
                      p.smem, stream,
                      static_cast<const uint16_t *>(a.y), static_cast<const uint16_t *>(a.h), a.g_post, a.g_pre,
                      a.gate, a.residual_scale, a.eps, a.T, static_cast<int>(a.d), p.slots,
                      static_cast<uint16_t *>(a.h_out), a.n_out, a.n_scale);
}

template <int V, int RPI, int MAXT, int GATE, bool VEC>
cudaError_t run_backward(const NormPlan &p, const NormBackward &a, int device, cudaStream_t stream)
{
    static std::atomic<bool> set[kMaxDevices];
    cudaError_t e = ensure_smem(norm_backward_kernel<V, RPI, MAXT, GATE, VEC>, kMaxSmem, device, set);
    if (e != cudaSuccess)
        return e;
    e = launch_pdl(norm_backward_kernel<V, RPI, MAXT, GATE, VEC>, dim3(p.grid), dim3(p.threads), p.smem, stream,
                   static_cast<const uint16_t *>(a.dn), static_cast<const uint16_t *>(a.dh_out),
                   static_cast<const uint16_t *>(a.y), static_cast<const uint16_t *>(a.h_out), a.g_post, a.g_pre,
                   a.gate, a.residual_scale, a.eps, a.T, static_cast<int>(a.d), p.slots,
                   static_cast<uint16_t *>(a.dy), static_cast<uint16_t *>(a.dh), a.dgate,
                   static_cast<float *>(a.workspace));
    if (e != cudaSuccess)
        return e;
    return launch_pdl(norm_gains_kernel, dim3(static_cast<unsigned>((a.d + 31) / 32)), dim3(512), 0, stream,
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

template <int V, int RPI, int MAXT, bool VEC>
cudaError_t backward_gate(const NormPlan &p, const NormBackward &a, int dev, cudaStream_t s)
{
    switch (a.gate_mode) {
    case kGateNone:
        return run_backward<V, RPI, MAXT, kGateNone, VEC>(p, a, dev, s);
    case kGateChannel:
        return run_backward<V, RPI, MAXT, kGateChannel, VEC>(p, a, dev, s);
    case kGateToken:
        return run_backward<V, RPI, MAXT, kGateToken, VEC>(p, a, dev, s);
    default:
        return run_backward<V, RPI, MAXT, kGateFull, VEC>(p, a, dev, s);
    }
}

template <bool VEC> cudaError_t backward_shape(const NormPlan &p, const NormBackward &a, int dev, cudaStream_t s)
{
    if (p.v == 1)
        return p.one_row ? backward_gate<1, 1, kWide, VEC>(p, a, dev, s)
                                              : backward_gate<1, 2, kMaxThreads, VEC>(p, a, dev, s);
    return p.v == 2 ? backward_gate<2, 1, kMaxThreads, VEC>(p, a, dev, s)
                    : backward_gate<4, 1, kMaxThreads, VEC>(p, a, dev, s);
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
    const NormPlan p = plan_forward(a.T, d, a.gate_mode, a.n_scale != nullptr, di.num_sms);
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
    return a.d % 8 == 0 ? backward_shape<true>(p, a, di.device, stream)
                        : backward_shape<false>(p, a, di.device, stream);
}

}  // namespace taco
