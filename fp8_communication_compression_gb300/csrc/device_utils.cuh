// Inline-PTX helpers for the sm_103a kernels: shared-memory mbarriers with
// time-limited waits, TMA tensor copies, and FP8 E4M3 / bf16 conversions.
#pragma once

#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

namespace taco {

// Every wait on another agent (TMA engine, producer warp) gives up after this
// many nanoseconds of %globaltimer, records a flag and lets the kernel exit.
constexpr uint64_t kWaitLimitNs = 1000000000ull;

__device__ __forceinline__ uint32_t smem_u32(const void *p)
{
    return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}

__device__ __forceinline__ uint64_t global_timer_ns()
{
    uint64_t t;
    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
    return t;
}

// ------------------------------------------- programmatic dependent launch --
// A kernel launched with programmatic stream serialization may start before
// the previous kernel in its stream has finished; it must not touch that
// kernel's outputs before pdl_wait() returns (which waits for the previous
// grid to complete and its memory to be visible).  Without that launch
// attribute the instruction is a no-op.
//
// No codec kernel triggers its dependents early (griddepcontrol.
// launch_dependents): a dependent grid is released when its predecessor
// completes.  Measured on GB300 in the back-to-back compress -> reduce ->
// decompress step at the GPT-6.7B size, an early trigger at the start of
// every kernel made the step slower: 122.1 us against 120.3 us with the
// 16-element shard reduce, and 132.7 us against 118.9 us with the
// 32-element one.
//
// Kernels of the FP8 linear layer and of the norms do, where their grid is
// small.  pdl_trigger() at the start of a kernel (of a product: once the CTA has
// its tensor memory) lets the next grid of the stream start as soon as this
// one's CTAs leave room; every kernel still waits for its predecessor's end in
// pdl_wait() before it touches memory.  It pays where a layer's kernels are
// short (a few us) and their launch latency shows.

__device__ __forceinline__ void pdl_trigger() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// -------------------------------------- rows that start inside granules --

// The first n of q's eight 16-bit elements, zeros after them.
__device__ __forceinline__ uint4 first_elements(const uint4 &q, int n)
{
    uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int j = 0; j < 4; ++j)
        w[j] &= 2 * j + 1 < n ? 0xFFFFFFFFu : 2 * j < n ? 0x0000FFFFu : 0u;
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// Elements e .. e + 7 of the sixteen in a, b (e the same in all lanes; both
// tests are then uniform).
__device__ __forceinline__ uint4 join(const uint4 &a, const uint4 &b, int e)
{
    uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    if (e & 4) {
#pragma unroll
        for (int j = 0; j < 6; ++j)
            w[j] = w[j + 2];
    }
    if (e & 2) {
#pragma unroll
        for (int j = 0; j < 5; ++j)
            w[j] = w[j + 1];
    }
    const uint32_t bits = 16 * (e & 1);
    return make_uint4(__funnelshift_r(w[0], w[1], bits), __funnelshift_r(w[1], w[2], bits),
                      __funnelshift_r(w[2], w[3], bits), __funnelshift_r(w[3], w[4], bits));
}

// ------------------------------------------------------------- mbarrier --

__device__ __forceinline__ void mbar_init(uint32_t bar, uint32_t count)
{
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}

__device__ __forceinline__ void fence_barrier_init()
{
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
}

__device__ __forceinline__ void mbar_arrive_expect_tx(uint32_t bar, uint32_t bytes)
{
    asm volatile("mbarrier.arrive.expect_tx.release.cta.shared::cta.b64 _, [%0], %1;" ::"r"(bar),
                 "r"(bytes)
                 : "memory");
}

__device__ __forceinline__ bool mbar_try_wait(uint32_t bar, uint32_t parity)
{
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cta.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}

// Waits for the phase with the given parity to complete.  Returns false if
// it has not completed within kWaitLimitNs.
__device__ __forceinline__ bool mbar_wait(uint32_t bar, uint32_t parity)
{
    if (mbar_try_wait(bar, parity))
        return true;
    const uint64_t t0 = global_timer_ns();
    for (;;) {
#pragma unroll 1
        for (int i = 0; i < 32; ++i)
            if (mbar_try_wait(bar, parity))
                return true;
        if (global_timer_ns() - t0 > kWaitLimitNs)
            return false;
    }
}

// mbar_wait with a hint that lets the warp sleep until the phase completes, for
// kernels all of whose warps wait for memory (in the policy loss polling took a
// tenth of the instructions).  CLUSTER: for what other CTAs have stored.
template <bool CLUSTER> __device__ __forceinline__ bool mbar_sleep(uint32_t bar, uint32_t parity)
{
    uint64_t t0 = 0;
    for (;;) {
        uint32_t ok;
        if (CLUSTER)
            asm volatile("{\n\t.reg .pred p;\n\t"
                         "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2, %3;\n\t"
                         "selp.u32 %0, 1, 0, p;\n\t}"
                         : "=r"(ok)
                         : "r"(bar), "r"(parity), "r"(10000000u)
                         : "memory");
        else
            asm volatile("{\n\t.reg .pred p;\n\t"
                         "mbarrier.try_wait.parity.acquire.cta.shared::cta.b64 p, [%1], %2, %3;\n\t"
                         "selp.u32 %0, 1, 0, p;\n\t}"
                         : "=r"(ok)
                         : "r"(bar), "r"(parity), "r"(10000000u)
                         : "memory");
        if (ok)
            return true;
        const uint64_t t = global_timer_ns();
        t0 = t0 ? t0 : t;
        if (t - t0 > kWaitLimitNs)
            return false;
    }
}

// ------------------------------------------------------------------- TMA --

// Copies `bytes` contiguous bytes (a multiple of 16, both addresses 16-byte
// aligned) to shared memory and reports them to the mbarrier at `bar`.
__device__ __forceinline__ void bulk_load(uint32_t dst, const void *src, uint32_t bytes, uint32_t bar)
{
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
                 "l"(src), "r"(bytes), "r"(bar)
                 : "memory");
}

// The same with an L2 cache policy.
__device__ __forceinline__ void bulk_load_hint(uint32_t dst, const void *src, uint32_t bytes, uint32_t bar, uint64_t pol)
{
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint"
                 " [%0], [%1], %2, [%3], %4;" ::"r"(dst),
                 "l"(src), "r"(bytes), "r"(bar), "l"(pol)
                 : "memory");
}

__device__ __forceinline__ void tma_prefetch_map(const CUtensorMap *map)
{
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(map)) : "memory");
}

// L2 cache policies (createpolicy) for data read or written exactly once.
__device__ __forceinline__ uint64_t policy_evict_first()
{
    uint64_t pol;
    asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(pol));
    return pol;
}

// 2-D tiled TMA copies with an L2 cache policy: a store shared -> global
// (as tma_store_2d), and a load global -> shared whose bytes complete on the
// mbarrier `bar`.
__device__ __forceinline__ void tma_store_2d_hint(const CUtensorMap *map, int32_t x, int32_t y, uint32_t src,
                                                  uint64_t pol)
{
    asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group.L2::cache_hint"
                 " [%0, {%1, %2}], [%3], %4;" ::"l"(reinterpret_cast<uint64_t>(map)),
                 "r"(x), "r"(y), "r"(src), "l"(pol)
                 : "memory");
}

__device__ __forceinline__ void tma_load_2d_hint(uint32_t dst, const CUtensorMap *map, int32_t x, int32_t y,
                                                 uint32_t bar, uint64_t pol)
{
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint"
        " [%0], [%1, {%2, %3}], [%4], %5;" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar), "l"(pol)
        : "memory");
}

// 2-D tiled store shared -> global (rows past the tensor end are clipped).
__device__ __forceinline__ void tma_store_2d(const CUtensorMap *map, int32_t x, int32_t y,
                                             uint32_t src)
{
    asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%1, %2}], [%3];" ::"l"(
                     reinterpret_cast<uint64_t>(map)),
                 "r"(x), "r"(y), "r"(src)
                 : "memory");
}

__device__ __forceinline__ void bulk_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }

// Wait until no bulk group of this thread is still reading shared memory.
__device__ __forceinline__ void bulk_wait_read_all()
{
    asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
}

// Wait until every bulk group of this thread has completed.
__device__ __forceinline__ void bulk_wait_all() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }

// Order this thread's generic-proxy shared-memory writes before later
// async-proxy (TMA) reads of them.
__device__ __forceinline__ void fence_proxy_async_smem()
{
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

// ---------------------------------------------------------- shared loads --

__device__ __forceinline__ uint4 lds128(uint32_t addr)
{
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(addr));
    return v;
}

__device__ __forceinline__ void sts128(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d)
{
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d)
                 : "memory");
}

// ---------------------------------------------------------- global loads --

// 16-byte streaming load through the non-coherent path (data read once).
__device__ __forceinline__ uint4 ldg128_stream(const void *p)
{
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}

// The same with an L2 cache policy (policy_evict_first() for inputs that
// nothing reads again, so that they do not displace data the next kernel
// reads).
__device__ __forceinline__ uint4 ldg128_stream_hint(const void *p, uint64_t pol)
{
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.L2::cache_hint.v4.u32 {%0, %1, %2, %3}, [%4], %5;"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p), "l"(pol));
    return v;
}

__device__ __forceinline__ void stg128_stream(void *p, uint4 v)
{
    asm volatile("st.global.L1::no_allocate.v4.u32 [%0], {%1, %2, %3, %4};" ::"l"(p), "r"(v.x), "r"(v.y),
                 "r"(v.z), "r"(v.w)
                 : "memory");
}

// ------------------------------------------- separately rounded products --
// a * b + c with the product rounded before the sum, on two lanes of a
// float2.  __fmul_rn / __fadd_rn are never contracted into a fused
// multiply-add, so terms that cancel exactly give exactly zero and the
// result is that of the stated arithmetic.

__device__ __forceinline__ float2 mul2_rounded(float2 a, float2 b)
{
    return make_float2(__fmul_rn(a.x, b.x), __fmul_rn(a.y, b.y));
}

__device__ __forceinline__ float2 add2_rounded(float2 a, float2 b)
{
    return make_float2(__fadd_rn(a.x, b.x), __fadd_rn(a.y, b.y));
}

// ------------------------------------------------------------ long sums --

// A sum in two fp32 parts: what each addition rounds off is kept (Knuth's
// two-sum).  As exact as fp64 for sums of some thousand terms, which the fp64
// units would take ten times as long for.
struct TwoPart {
    float hi = 0.0f, lo = 0.0f;
    __device__ __forceinline__ void add(float x)
    {
        const float t = __fadd_rn(hi, x), b = __fsub_rn(t, hi);
        lo = __fadd_rn(lo, __fadd_rn(__fsub_rn(hi, __fsub_rn(t, b)), __fsub_rn(x, b)));
        hi = t;
    }
    __device__ __forceinline__ void add(const TwoPart &x)
    {
        add(x.hi);
        lo += x.lo;
    }
    __device__ __forceinline__ void add_lanes()  // of a warp: in all of them
    {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            TwoPart x;
            x.hi = __shfl_xor_sync(~0u, hi, o);
            x.lo = __shfl_xor_sync(~0u, lo, o);
            add(x);
        }
    }
    // A sum that has left fp32's range, or of something that is no number, is hi.
    __device__ __forceinline__ float value() const { return fabsf(hi) <= 3.4028234e38f ? hi + lo : hi; }
};

// ----------------------------------------------------------- conversions --

// bf16 halves of a 32-bit word to fp32 (exact).
__device__ __forceinline__ float bf16lo_to_f32(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16hi_to_f32(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// Two fp32 -> two E4M3FN codes, round to nearest even, saturating to +-448.
// The low byte of the result holds `lo`, the high byte `hi`.
__device__ __forceinline__ uint32_t f32x2_to_e4m3x2(float lo, float hi)
{
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

// Four fp32 -> four E4M3FN codes packed little-endian into one word.
__device__ __forceinline__ uint32_t f32x4_to_e4m3x4(float a, float b, float c, float d)
{
    uint32_t r;
    asm("{\n\t.reg .b16 lo, hi;\n\tcvt.rn.satfinite.e4m3x2.f32 lo, %2, %1;\n\t"
        "cvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;\n\tmov.b32 %0, {lo, hi};\n\t}"
        : "=r"(r)
        : "f"(a), "f"(b), "f"(c), "f"(d));
    return r;
}

// Two E4M3FN codes (low byte = first element) -> two fp32 values (exact:
// every E4M3 value is an fp16 value, and every fp16 value an fp32 one).
__device__ __forceinline__ void e4m3x2_to_f32x2(uint32_t two_codes, float &lo, float &hi)
{
    uint32_t h2;
    uint16_t in = static_cast<uint16_t>(two_codes);
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"(in));
    asm("{\n\t.reg .f16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
        : "=f"(lo), "=f"(hi)
        : "r"(h2));
}

// Two fp32 -> two bf16 (round to nearest even), low half = lo.
__device__ __forceinline__ uint32_t f32x2_to_bf16x2(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

} // namespace taco
