// Inline PTX of the latent-attention kernels beyond ptx.cuh: 16-bit MMAs with
// either operand order, TMEM stores, TMA boxes of three dimensions, and the
// shared bounded wait.
#pragma once
#include <cstdint>

#include "ptx.cuh"

namespace sgq {
namespace lat {

// A value that is the same in all lanes, in a form that the compiler knows to be.
__device__ __forceinline__ uint32_t uniform(uint32_t x) { return __shfl_sync(0xFFFFFFFFu, x, 0); }

// A shared-memory matrix descriptor in halves: the low word holds the address
// (and the leading offset), the high word the stride and the layout.  Steps
// through shared memory only ever change the low word.
__device__ __forceinline__ uint32_t desc_lo(uint32_t saddr, uint32_t lbo_bytes) {
    return ((saddr >> 4) & 0x3FFFu) | ((lbo_bytes >> 4) << 16);
}
__host__ __device__ constexpr uint32_t desc_hi(uint32_t sbo_bytes, uint32_t layout) {
    return (sbo_bytes >> 4) | (1u << 14) | (layout << 29);
}

// Four MMAs D[tmem] (+)= A B^T of K = 16 each, 16-bit operands in shared
// memory, fp32 accumulator: descriptors kA and kB (units of 16 bytes) apart,
// the first one starting over where acc == 0.  Executed by a converged warp,
// issued by its elected lane.
template <int kA, int kB>
__device__ __forceinline__ void mma4_f16(uint32_t d, uint32_t a_lo, uint32_t a_hi, uint32_t b_lo, uint32_t b_hi,
                                         uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n.reg .pred e, q, t;\n.reg .b32 x, y;\n.reg .b64 a0, a1, a2, a3, b0, b1, b2, b3;\n"
        "elect.sync _|e, 0xffffffff;\n"
        "setp.ne.b32 q, %6, 0;\nsetp.eq.u32 t, %0, %0;\n"
        "mov.b64 a0, {%1, %2};\nmov.b64 b0, {%3, %4};\n"
        "add.u32 x, %1, %7;\nadd.u32 y, %3, %10;\nmov.b64 a1, {x, %2};\nmov.b64 b1, {y, %4};\n"
        "add.u32 x, %1, %8;\nadd.u32 y, %3, %11;\nmov.b64 a2, {x, %2};\nmov.b64 b2, {y, %4};\n"
        "add.u32 x, %1, %9;\nadd.u32 y, %3, %12;\nmov.b64 a3, {x, %2};\nmov.b64 b3, {y, %4};\n"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a0, b0, %5, q;\n"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a1, b1, %5, t;\n"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a2, b2, %5, t;\n"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a3, b3, %5, t;\n}" ::"r"(d),
        "r"(a_lo), "r"(a_hi), "r"(b_lo), "r"(b_hi), "r"(idesc), "r"(acc), "n"(kA), "n"(2 * kA), "n"(3 * kA), "n"(kB),
        "n"(2 * kB), "n"(3 * kB)
        : "memory");
}
// The same with A in TMEM (row i in lane i, two elements a 32-bit column).
template <int kB>
__device__ __forceinline__ void mma4_f16_ts(uint32_t d, uint32_t a, uint32_t b_lo, uint32_t b_hi, uint32_t idesc,
                                            uint32_t acc) {
    asm volatile(
        "{\n.reg .pred e, q, t;\n.reg .b32 a1, a2, a3, y;\n.reg .b64 b0, b1, b2, b3;\n"
        "elect.sync _|e, 0xffffffff;\n"
        "setp.ne.b32 q, %5, 0;\nsetp.eq.u32 t, %0, %0;\n"
        "add.u32 a1, %1, 8;\nadd.u32 a2, %1, 16;\nadd.u32 a3, %1, 24;\n"
        "mov.b64 b0, {%2, %3};\nadd.u32 y, %2, %6;\nmov.b64 b1, {y, %3};\n"
        "add.u32 y, %2, %7;\nmov.b64 b2, {y, %3};\nadd.u32 y, %2, %8;\nmov.b64 b3, {y, %3};\n"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b0, %4, q;\n"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a1], b1, %4, t;\n"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a2], b2, %4, t;\n"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a3], b3, %4, t;\n}" ::"r"(d),
        "r"(a), "r"(b_lo), "r"(b_hi), "r"(idesc), "r"(acc), "n"(kB), "n"(2 * kB), "n"(3 * kB)
        : "memory");
}
// Instruction descriptor, kind::f16: fp32 D; both operands bf16 or both fp16;
// an operand is K-major, or MN-major where its flag is set.
__host__ __device__ constexpr uint32_t idesc_f16(uint32_t M, uint32_t N, bool bf16, bool a_mn, bool b_mn) {
    return (1u << 4) | ((bf16 ? 1u : 0u) << 7) | ((bf16 ? 1u : 0u) << 10) | ((a_mn ? 1u : 0u) << 15) |
           ((b_mn ? 1u : 0u) << 16) | ((N >> 3) << 17) | ((M >> 4) << 24);
}
// Descriptor layout code of a row of 128, 64 or 32 bytes (its swizzle span).
__host__ __device__ constexpr uint32_t layout_of(uint32_t row_bytes) {
    return row_bytes == 128 ? 2u : row_bytes == 64 ? 4u : 6u;
}

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* m, int32_t x, int32_t y, int32_t z,
                                            uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(m)), "r"(x), "r"(y), "r"(z), "r"(bar)
        : "memory");
}

// `bytes` (a multiple of 16) from a 16-byte aligned address into L2.
__device__ __forceinline__ void bulk_prefetch(const void* p, uint32_t bytes) {
    asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(p), "r"(bytes) : "memory");
}

// Asks to take over a CTA of this grid that has not started: the answer (16
// bytes at a 16-byte aligned shared address) completes 16 bytes of
// transactions on `bar`.  Not to be asked again after an answer of no.
__device__ __forceinline__ void take_item(uint32_t answer, uint32_t bar) {
    asm volatile("clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(
                     answer),
                 "r"(bar)
                 : "memory");
}
// Whether the answer is yes, and then the block index (x) taken over.
__device__ __forceinline__ bool taken_item(uint32_t answer, uint32_t& x) {
    uint32_t yes, index;
    asm volatile(
        "{\n.reg .pred p;\n.reg .b128 r;\n"
        "ld.shared.b128 r, [%2];\n"
        "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, r;\n"
        "selp.u32 %0, 1, 0, p;\nmov.u32 %1, 0;\n"
        "@p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %1, r;\n}"
        : "=r"(yes), "=r"(index)
        : "r"(answer)
        : "memory");
    x = index;
    return yes != 0u;
}

// 32 lanes x N consecutive 32-bit columns; thread t writes lane (base_lane + t).
template <int N>
__device__ __forceinline__ void tmem_st(uint32_t taddr, const uint32_t (&r)[N]);
template <>
__device__ __forceinline__ void tmem_st<8>(uint32_t taddr, const uint32_t (&r)[8]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
        : "memory");
}
template <>
__device__ __forceinline__ void tmem_st<16>(uint32_t taddr, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// 2^x (flushing tiny results to zero); 2^-inf = 0.
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// Two fp32 operations in one instruction (both correctly rounded).
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;"
        : "=l"(d)
        : "l"(*reinterpret_cast<const uint64_t*>(&a)), "l"(*reinterpret_cast<const uint64_t*>(&b)),
          "l"(*reinterpret_cast<const uint64_t*>(&c)));
    return *reinterpret_cast<const float2*>(&d);
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;"
        : "=l"(d)
        : "l"(*reinterpret_cast<const uint64_t*>(&a)), "l"(*reinterpret_cast<const uint64_t*>(&b)));
    return *reinterpret_cast<const float2*>(&d);
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;"
        : "=l"(d)
        : "l"(*reinterpret_cast<const uint64_t*>(&a)), "l"(*reinterpret_cast<const uint64_t*>(&b)));
    return *reinterpret_cast<const float2*>(&d);
}
// Maximum over the warp, in every lane.
__device__ __forceinline__ float warp_max(float x) {
    float y;
    asm("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ void named_sync(int id, int threads) {
    asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

// The same barrier with a vote: true where some thread passes true.
__device__ __forceinline__ bool named_any(int id, int threads, bool x) {
    uint32_t r;
    asm volatile(
        "{\n.reg .pred p, q;\nsetp.ne.u32 q, %3, 0;\n"
        "bar.red.or.pred p, %1, %2, q;\nselp.u32 %0, 1, 0, p;\n}"
        : "=r"(r)
        : "r"(id), "r"(threads), "r"(x ? 1u : 0u)
        : "memory");
    return r != 0u;
}

// Bounded waits: a wait that runs out raises the CTA's abort flag and the
// device status; every other wait of the CTA then gives up as well.
constexpr uint32_t kStatusTimeout = 1u;
constexpr long long kTimeoutClocks = 4000000000ll;    // about 2 s
constexpr long long kTestTimeoutClocks = 1ll << 21;   // about 1 ms (SGQ_LATENT_TEST_TIMEOUT)
constexpr long long kAbortPollClocks = 2000000ll;
template <long long kLimit>
struct Sync {
    volatile uint32_t* abort_flag;
    uint32_t* status;
};
// The whole warp waits for a phase; false: gave up.  All lanes poll together:
// a warp whose lane 0 went through a polling loop alone stayed split in two
// afterwards, and its MMA issue slowed down three to four times.
template <long long kLimit>
static __device__ __noinline__ bool wait_slow(uint32_t bar, uint32_t parity, const Sync<kLimit>& s) {
    const long long t0 = clock64();
    for (uint32_t spins = 1;; ++spins) {
        if (__all_sync(0xFFFFFFFFu, ptx::mbar_try_wait(bar, parity))) return true;
        if ((spins & 63u) == 0) {
            const long long dt = clock64() - t0;
            if (__any_sync(0xFFFFFFFFu, dt > kLimit)) {
                *s.abort_flag = 1u;
                if ((threadIdx.x & 31) == 0) atomicOr(s.status, kStatusTimeout);
                __syncwarp();
                return false;
            }
            if (__any_sync(0xFFFFFFFFu, dt > kAbortPollClocks && *s.abort_flag)) return false;
        }
    }
}
template <long long kLimit>
__device__ __forceinline__ bool wait_warp(uint32_t bar, uint32_t parity, const Sync<kLimit>& s) {
    if (__all_sync(0xFFFFFFFFu, ptx::mbar_try_wait(bar, parity))) return true;
    return wait_slow(bar, parity, s);
}

}  // namespace lat
}  // namespace sgq
