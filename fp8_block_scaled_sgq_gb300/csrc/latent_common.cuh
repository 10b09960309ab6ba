// Shared by the latent-attention kernels (latent_rope.cu, latent_attn.cu,
// latent_prefill.cu): the two element types and the range of softmax weights.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cstdint>

namespace sgq {
namespace lat {

// Two elements of a 32-bit word <-> fp32.  Rounding is to nearest even, once,
// where a result leaves fp32.
template <typename T>
struct Pair;
template <>
struct Pair<__nv_bfloat16> {
    static __device__ __forceinline__ float2 unpack(uint32_t w) {
        return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
    }
    static __device__ __forceinline__ uint32_t pack(float a, float b) {
        const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
        return *reinterpret_cast<const uint32_t*>(&v);
    }
};
template <>
struct Pair<__half> {
    static __device__ __forceinline__ float2 unpack(uint32_t w) {
        return __half22float2(*reinterpret_cast<const __half2*>(&w));
    }
    static __device__ __forceinline__ uint32_t pack(float a, float b) {
        const __half2 v = __floats2half2_rn(a, b);
        return *reinterpret_cast<const uint32_t*>(&v);
    }
};

// Softmax weights as a product's operand: 2^(s - m) of a score s (in powers of
// two), rounded to the call's type.  A row's reference m is its running maximum
// less kLift, and follows it only when the maximum has grown by more than
// kGrow, so a row's largest weight is at least 2^kLift and none is above
// 2^(kLift + kGrow).  bf16 has fp32's exponents: any m does.  fp16 loses bits
// below 2^-14 and holds nothing below 2^-25, so weights are kept close below its
// 2^16: precise from 2^-23 of the row's largest weight on, and off by 2^-34 of
// it at most below.  (With m at the maximum, 131072 keys at 2^-26 of a dominant
// one vanished from a row, while its sum counted them.)  More lift leaves less
// growth, i.e. more rescaling.  kGrow, kLift of 8, 7 / 6, 9 / 5, 10 / 4, 11 for
// 131071 rows and 128 heads: 70.6, 70.6, 70.7, 74.7 us; expanded, 8 ragged
// prompts x 16 heads: 304.4, 304.7, 307.2, 322.2 us.
template <typename T>
struct Weights;
template <>
struct Weights<__nv_bfloat16> {
    static constexpr float kGrow = 8.0f, kLift = 0.0f;
};
template <>
struct Weights<__half> {
    static constexpr float kGrow = 6.0f, kLift = 9.0f;
};

}  // namespace lat
}  // namespace sgq
