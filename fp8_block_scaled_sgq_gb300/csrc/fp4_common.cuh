// The 4-bit form shared by its quantisers (fp4_quant.cu, norm.cu) and its
// GEMM (fp4_gemm.cu): E2M1 codes, two a byte, the even element in the low
// half, and one scale byte a group:
//   MXFP4  32 values, UE8M0 (2^(byte - 127)):  s = max(amax, 1e-10) / 6 rounded
//          up to a power of two, as the FP8 quantisers round theirs;
//   NVFP4  16 values, E4M3, and one fp32 scale t a tensor:  s = E4M3(amax / (6 t)),
//          at least 2^-9 and at most 448; the values are code * (s t).
// A code is E2M1(x / s) or E2M1(x / (s t)): an IEEE fp32 division, then round to
// nearest even, saturating at 6.  A group that holds a NaN or an infinity gets
// the NaN scale byte and codes of zero.
//
// Scale bytes lie in tiles of 128 rows x 4 groups, 512 bytes each, tiles of a
// row block one after the other along K: the byte of (row r, group j) is
// (r % 32) * 16 + (r % 128) / 32 * 4 + j % 4 of its tile, the order in which
// tcgen05.cp (32 lanes x 128 bits, copied to all four lane quarters) puts them
// where the block-scaled MMA looks for them.  Groups past K are 0; rows past
// the last one are never used and may hold anything.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cstdint>

#include "latent_common.cuh"
#include "latent_ptx.cuh"
#include "quant_math.cuh"

namespace sgq {
namespace fp4 {

using lat::Pair;

constexpr float kMax = 6.0f;            // largest E2M1 value
constexpr uint32_t kNanE8 = 0xFFu;      // NaN as UE8M0
constexpr uint32_t kNanE4 = 0x7Fu;      // NaN as E4M3
constexpr float kMaxE4 = 448.0f;        // the largest
constexpr uint32_t kInf = 0x7F800000u;

__host__ __device__ constexpr int group_of(bool nv) { return nv ? 16 : 32; }
// Tiles of scales along K.
__host__ __device__ constexpr int64_t scale_tiles(int64_t K, bool nv) { return (K + (nv ? 63 : 127)) / (nv ? 64 : 128); }

// Byte offset of a row's word of four groups (group j of it in byte j) in tile kb.
__device__ __forceinline__ int64_t scale_word_at(int64_t row, int64_t kb, int64_t tiles) {
    return ((row >> 7) * tiles + kb) * 512 + (row & 31) * 16 + ((row & 127) >> 5) * 4;
}

// Eight fp32 values -> eight E2M1 codes (saturating, to nearest even).
__device__ __forceinline__ uint32_t codes8(const float (&q)[8]) {
    uint32_t r;
    asm("{\n.reg .b8 a, b, c, d;\n"
        "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\ncvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n"
        "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\ncvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n"
        "mov.b32 %0, {a, b, c, d};\n}"
        : "=r"(r)
        : "f"(q[0]), "f"(q[1]), "f"(q[2]), "f"(q[3]), "f"(q[4]), "f"(q[5]), "f"(q[6]), "f"(q[7]));
    return r;
}
// And back: eight codes -> their values, as four fp16 pairs.
__device__ __forceinline__ void values8(uint32_t codes, uint32_t (&h)[4]) {
    asm("{\n.reg .b8 a, b, c, d;\nmov.b32 {a, b, c, d}, %4;\n"
        "cvt.rn.f16x2.e2m1x2 %0, a;\ncvt.rn.f16x2.e2m1x2 %1, b;\n"
        "cvt.rn.f16x2.e2m1x2 %2, c;\ncvt.rn.f16x2.e2m1x2 %3, d;\n}"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
        : "r"(codes));
}

// fp32 -> E4M3 byte (saturating) and back.
__device__ __forceinline__ uint32_t e4m3_of(float x) {
    return static_cast<uint32_t>(__nv_cvt_float_to_fp8(x, __NV_SATFINITE, __NV_E4M3));
}
__device__ __forceinline__ float of_e4m3(uint32_t b) {
    const __half_raw h = __nv_cvt_fp8_to_halfraw(static_cast<__nv_fp8_storage_t>(b), __NV_E4M3);
    return __half2float(*reinterpret_cast<const __half*>(&h));
}
// 2^(byte - 127); NaN for 255.
__device__ __forceinline__ float of_ue8m0(uint32_t b) {
    return b == kNanE8 ? __uint_as_float(0x7FFFFFFFu) : b == 0 ? __uint_as_float(0x400000u) : __uint_as_float(b << 23);
}

__device__ __forceinline__ bool in_range(float d) { return d >= 0x1p-60f && d <= 0x1p100f; }
// x / d correctly rounded, with r = 1/d rounded and d in range, as a product
// and two corrections by its exact remainder: after the first the quotient is
// within one unit, and after the second it is the rounded one (Markstein,
// "Computation of elementary functions on the IBM RISC System/6000 processor",
// 1990, theorem on the last step of a division).  Remainders are exact while
// nothing leaves fp32's normal range: other divisors take the division itself.
// A quotient past fp32's largest value comes out as NaN.
__device__ __forceinline__ float quotient(float x, float d, float r) {
    float q = __fmul_rn(x, r);
    q = __fmaf_rn(-__fmaf_rn(q, d, -x), r, q);
    return __fmaf_rn(-__fmaf_rn(q, d, -x), r, q);
}
// A tensor's scale t, 6 t, and the rounded reciprocal of that (0: divide).
struct TensorScale {
    float t, t6, r6;
    __device__ __forceinline__ explicit TensorScale(const float* p) {
        t = p ? __ldg(p) : 1.0f;
        t6 = __fmul_rn(t, kMax);
        r6 = in_range(t6) ? __frcp_rn(t6) : 0.0f;
    }
};

// A group's scale byte from the bits of its largest magnitude (NaN's bits are
// above infinity's, and those above every finite value's), and what its values
// are divided by: s itself, or s t.
template <bool kNv>
__device__ __forceinline__ uint32_t scale_byte(uint32_t amax_bits, const TensorScale& ts, float& div) {
    if (amax_bits >= kInf) {
        div = 0.0f;
        return kNv ? kNanE4 : kNanE8;
    }
    const float amax = __uint_as_float(amax_bits);
    if constexpr (kNv) {
        // (a quotient that the corrections do not settle is far below 2^-9, or past fp32's largest value: it is infinite
        // then, and the corrections make infinity - infinity of it, NaN, of which fminf takes the other operand)
        const float q = ts.r6 != 0.0f ? quotient(amax, ts.t6, ts.r6) : __fdiv_rn(amax, ts.t6);
        const uint32_t b = max(e4m3_of(fminf(q, kMaxE4)), 1u);
        div = __fmul_rn(of_e4m3(b), ts.t);
        return b;
    } else {
        uint32_t u = __float_as_uint(quotient(fmaxf(amax, qm::kEps), kMax, 1.0f / kMax));
        if (u & 0x7FFFFFu) u = (u & kInf) + 0x800000u;
        div = __uint_as_float(u);
        return u >> 23;
    }
}

// What eight values of a group are multiplied by, -1/div, where they are
// themselves results of fp32 arithmetic (a norm, silu): the quotients are
// within 1.5 units of the division's, far less than the values are off.
// (-1/2^e is exact, and so are those quotients.)
template <bool kNv>
__device__ __forceinline__ float minus_reciprocal(float div) {
    if constexpr (kNv) return -__frcp_rn(div);
    else return -__uint_as_float((254u - (__float_as_uint(div) >> 23)) << 23);
}
// Eight negated values -> codes, by divisions: for divisors outside in_range,
// whose reciprocals may leave fp32.  div == 0: the group is not finite.  (Out
// of line, and in registers.)
static __device__ __noinline__ uint32_t divided8(float4 a, float4 b, float div) {
    const float n[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    float q[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) q[i] = __fdiv_rn(n[i], -div);
    return div == 0.0f ? 0u : codes8(q);
}
__device__ __forceinline__ uint32_t divided8(const float (&n)[8], float div) {
    return divided8(make_float4(n[0], n[1], n[2], n[3]), make_float4(n[4], n[5], n[6], n[7]), div);
}
// Eight values of a group, negated, so that a zero keeps its sign -> codes.
// div == 0: the group is not finite.
template <bool kNv>
__device__ __forceinline__ uint32_t encode8(const float (&n)[8], float div) {
    if (kNv && !in_range(div)) return divided8(n, div);
    const float r = minus_reciprocal<kNv>(div);
    float q[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) q[i] = __fmul_rn(n[i], r);
    return div == 0.0f ? 0u : codes8(q);
}

// The largest magnitude of three; NaN where one is.
__device__ __forceinline__ float max3(float a, float b, float c) {
    float y;
    asm("{\n.reg .f32 x, y, z;\nabs.f32 x, %1;\nabs.f32 y, %2;\nabs.f32 z, %3;\nmax.NaN.f32 %0, x, y, z;\n}" : "=f"(y) : "f"(a), "f"(b), "f"(c));
    return y;
}
// The same without the NaNs among them (NaN where all are).
__device__ __forceinline__ float max3_of_numbers(float a, float b, float c) {
    float y;
    asm("{\n.reg .f32 x, y, z;\nabs.f32 x, %1;\nabs.f32 y, %2;\nabs.f32 z, %3;\nmax.f32 %0, x, y, z;\n}" : "=f"(y) : "f"(a), "f"(b), "f"(c));
    return y;
}
// The bits of the largest magnitude among eight, of those that are no NaN (0 where all are).
__device__ __forceinline__ uint32_t amax_bits8_of_numbers(const float (&v)[8]) {
    return __float_as_uint(max3_of_numbers(max3_of_numbers(v[0], v[1], v[2]), max3_of_numbers(v[3], v[4], v[5]), max3_of_numbers(v[6], v[7], 0.0f)));
}
// The bits of the largest magnitude among eight (above infinity's for NaN).
__device__ __forceinline__ uint32_t amax_bits8(const float (&v)[8]) {
    return __float_as_uint(max3(max3(v[0], v[1], v[2]), max3(v[3], v[4], v[5]), max3(v[6], v[7], v[7])));
}

template <typename T>
__device__ __forceinline__ void unpack8(const uint4& w, float (&v)[8]) {
    const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = Pair<T>::unpack(x[i]);
        v[2 * i] = f.x;
        v[2 * i + 1] = f.y;
    }
}
template <typename T>
__device__ __forceinline__ uint4 pack8(const float (&v)[8]) {
    return make_uint4(Pair<T>::pack(v[0], v[1]), Pair<T>::pack(v[2], v[3]), Pair<T>::pack(v[4], v[5]),
                      Pair<T>::pack(v[6], v[7]));
}

}  // namespace fp4
}  // namespace sgq
