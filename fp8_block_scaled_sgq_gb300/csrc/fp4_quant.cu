// 4-bit quantisation with microscales, and its way back, for sm_103a: the form
// and the rule are in fp4_common.cuh.
//
// Both kernels are bound by HBM: 2 bytes an element one way, 0.53 (MXFP4) or
// 0.56 (NVFP4) the other.  A thread holds 16 consecutive elements, i.e. one
// NVFP4 group or half an MXFP4 one; a warp takes a span of 512 elements of
// every so many rows, so that the four groups of a scale word lie in
// neighbouring lanes and leave as one store, and no index is divided on the way.
// Measured, 4099 x 7168, inputs from HBM: MXFP4 13.1 us (5.7 TB/s), NVFP4 15.3
// (4.9), of silu(gate) * up 23.6 and 23.8 (5.6), back to 16 bits 11.1 and 11.6
// (6.7 and 6.5).  The scale words, 4 bytes to a 32-byte sector, cost 1.3 us.
// What NVFP4 takes longer is instructions: its scales are no powers of two, so
// every quotient has its correction, two operations an element.
#include <cuda_runtime.h>

#include <type_traits>

#include "fp4_common.cuh"
#include "ptx.cuh"
#include "sgq_internal.h"

namespace sgq {
namespace {

using namespace fp4;

constexpr int kThreads = 256;
constexpr int kSpan = 512;   // elements of a warp's span

// -silu(g) * u of h = -g/4 and u in fp32, as h / (1/4 + exp(-g)/4) * u, so that
// the divisor stays below 2^126 and its reciprocal a normal number down to the
// last g whose exp(-g) is finite (-88.7; 0 below, as 1 + exp(-g) is infinite in
// fp32).  Within 2^-17 of its value: an
// exponent near 127 is off by half a unit, 2^-18, and the product with log2 e by
// as much.
__device__ __forceinline__ float minus_silu_mul(float h, float u) {
    constexpr float kLog2e = 1.44269504088896341f;
    float e, r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(__fmaf_rn(h, 4.0f * kLog2e, -2.0f)));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(e + 0.25f));
    return h * r * u;
}

// 16 elements, in one load where they start on 32 bytes.
template <bool kWide, typename T>
__device__ __forceinline__ void load16(const T* p, uint4& a, uint4& b) {
    if constexpr (kWide) {
        asm volatile("ld.global.nc.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                     : "=r"(a.x), "=r"(a.y), "=r"(a.z), "=r"(a.w), "=r"(b.x), "=r"(b.y), "=r"(b.z), "=r"(b.w)
                     : "l"(p));
    } else {
        a = __ldg(reinterpret_cast<const uint4*>(p));
        b = __ldg(reinterpret_cast<const uint4*>(p) + 1);
    }
}
// The fp32 bits of the largest magnitude among 16 values: magnitudes of one
// sign order as whole numbers do, NaN above infinity, two a comparison.
template <typename T>
__device__ __forceinline__ uint32_t amax_bits16(const uint4& a, const uint4& b) {
    const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    uint32_t m = w[0] & 0x7FFF7FFFu;
#pragma unroll
    for (int i = 1; i < 8; ++i) m = __vmaxu2(m, w[i] & 0x7FFF7FFFu);
    m = max(m & 0xFFFFu, m >> 16);
    return __float_as_uint(Pair<T>::unpack(m).x);
}

// A group under a tensor scale of an extreme size, or far past its tensor
// scale, by divisions: scale byte and codes.  (Out of line: with it inline the arrays of quant_rows went
// through local memory, 16.3 -> 21.4 us.)
template <typename T>
__device__ __noinline__ uint4 extreme_group(uint4 a, uint4 b, uint32_t amax, float t, float t6) {
    uint32_t byte = kNanE4;
    float div = 0.0f, x[2][8];
    if (amax < kInf) {
        byte = max(e4m3_of(__fdiv_rn(__uint_as_float(amax), t6)), 1u);
        div = __fmul_rn(of_e4m3(byte), t);
    }
    unpack8<T>(a, x[0]);
    unpack8<T>(b, x[1]);
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int j = 0; j < 8; ++j) x[h][j] = div == 0.0f ? 0.0f : __fdiv_rn(x[h][j], div);
    return make_uint4(byte, codes8(x[0]), codes8(x[1]), 0);
}

// kN rows' 16 elements of a lane, in steps that no branch divides, so that the
// rows' chains overlap (NVFP4, 4099 x 7168: 19.8 us with branches, 15.9 so).
//
// Values that are bf16 or fp16 as they are have at most 11 significant bits.
// Their codes are settled by one correction of the quotient by its remainder,
// even with an approximate reciprocal: compared with the division for each
// significand of x and of d, over quotients from 2^-4 to 2^5, no code differs
// (without the correction 319 of 8.6e9 do in bf16, 2202 of 6.9e10 in fp16; the
// tests repeat it for 1025 of the divisors).
// Divisors outside in_range divide, and so does what is so far past its tensor
// scale that a quotient leaves fp32.
template <typename T, bool kNv, int kN>
__device__ __forceinline__ void quant_rows(const uint4 (&raw)[kN][2], const TensorScale& ts, uint32_t (&byte)[kN], uint2 (&q)[kN]) {
    uint32_t amax[kN];
    float div[kN], r[kN];
    bool odd = kNv && ts.r6 == 0.0f;
#pragma unroll
    for (int i = 0; i < kN; ++i) amax[i] = amax_bits16<T>(raw[i][0], raw[i][1]);
#pragma unroll
    for (int i = 0; i < kN; ++i) {
        if constexpr (kNv) {
            // (NaN and infinity come out as the NaN byte, and so does a finite group whose quotient leaves fp32, which is divided)
            byte[i] = max(e4m3_of(quotient(__uint_as_float(amax[i]), ts.t6, ts.r6)), 1u);
            div[i] = __fmul_rn(of_e4m3(byte[i]), ts.t);
            asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r[i]) : "f"(div[i]));
            odd |= byte[i] == kNanE4 ? amax[i] < kInf : !in_range(div[i]);
        } else {
            amax[i] = max(amax[i], __shfl_xor_sync(0xFFFFFFFFu, amax[i], 1));
            byte[i] = scale_byte<false>(amax[i], ts, div[i]);
            r[i] = __uint_as_float((254u - byte[i]) << 23);   // 1 / 2^(byte - 127)
        }
    }
#pragma unroll
    for (int i = 0; i < kN; ++i) {
        const uint32_t keep = byte[i] == (kNv ? kNanE4 : kNanE8) ? 0u : 0xFFFFFFFFu;   // codes of zero beside a NaN scale
        uint32_t c[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            float x[8], v[8];
            unpack8<T>(raw[i][h], x);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                v[j] = __fmul_rn(x[j], r[i]);
                if constexpr (kNv) v[j] = __fmaf_rn(-__fmaf_rn(v[j], div[i], -x[j]), r[i], v[j]);
            }
            c[h] = codes8(v) & keep;
        }
        q[i] = make_uint2(c[0], c[1]);
    }
    if (kNv && __any_sync(0xFFFFFFFFu, odd)) {
#pragma unroll
        for (int i = 0; i < kN; ++i) {
            const uint4 g = extreme_group<T>(raw[i][0], raw[i][1], amax[i], ts.t, ts.t6);
            byte[i] = g.x;
            q[i] = make_uint2(g.y, g.z);
        }
    }
}
template <typename T, bool kNv>
__device__ __forceinline__ void silu_row(const uint4 (&raw)[4], const TensorScale& ts, uint32_t& byte, uint2& q) {
    float v[2][8];   // negated (encode8)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        float u[8];
        unpack8<T>(raw[h], v[h]);
        unpack8<T>(raw[2 + h], u);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[h][j] = minus_silu_mul(-0.25f * v[h][j], u[j]);
    }
    uint32_t amax = max(amax_bits8(v[0]), amax_bits8(v[1]));
    if constexpr (!kNv) amax = max(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 1));
    float div;
    byte = scale_byte<kNv>(amax, ts, div);
    q = make_uint2(encode8<kNv>(v[0], div), encode8<kNv>(v[1], div));
}

// kWhole: rows are whole spans, and (without silu) start on 32 bytes: nothing
// is asked on the way (3 to 7 % faster).
template <typename T, bool kNv, bool kSilu, bool kWhole>
__global__ void __launch_bounds__(kThreads) quant_fp4_kernel(const T* __restrict__ x, int64_t stride,
                                                             const float* __restrict__ tensor_scale, uint2* __restrict__ xq,
                                                             uint8_t* __restrict__ xs, uint32_t M, uint32_t K, uint32_t spans) {
    ptx::launch_dependents();
    ptx::grid_dependency_wait();
    const TensorScale ts(kNv ? tensor_scale : nullptr);
    const uint32_t lane = threadIdx.x & 31, warp = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
    const uint32_t nwarps = gridDim.x * (kThreads / 32);
    const int64_t tiles = scale_tiles(K, kNv);
    constexpr int kVecs = kSilu ? 4 : 2;
    // A warp keeps to one span of the rows (to every nwarps-th one, where rows have more spans than there are warps).
    const uint32_t step = spans < nwarps ? nwarps / spans : 1;   // rows between a warp's
    if (spans < nwarps && warp >= step * spans) return;
    for (uint64_t span = spans < nwarps ? warp % spans : warp; span < spans; span += nwarps) {
        const uint32_t col = static_cast<uint32_t>(span) * kSpan + lane * 16;
        const bool in = kWhole || col < K;
        const T* from = x + col;
        const int64_t word = int64_t(col / (kNv ? 64 : 128)) * 512;
        auto rows = [&](uint64_t row0, auto count) {
            constexpr int kN = decltype(count)::value;
            uint4 raw[kN][kVecs];
#pragma unroll
            for (int i = 0; i < kN; ++i) {
#pragma unroll
                for (int j = 0; j < kVecs; ++j) raw[i][j] = make_uint4(0, 0, 0, 0);
                if (in) {
                    const T* p = from + (row0 + uint64_t(step) * i) * stride;
                    load16<kWhole && !kSilu>(p, raw[i][0], raw[i][1]);
                    if constexpr (kSilu) load16<false>(p + K, raw[i][2], raw[i][3]);
                }
            }
            uint32_t byte[kN];
            uint2 q[kN];
            if constexpr (kSilu) silu_row<T, kNv>(raw[0], ts, byte[0], q[0]);
            else quant_rows<T, kNv, kN>(raw, ts, byte, q);
#pragma unroll
            for (int i = 0; i < kN; ++i) {
                const uint64_t row = row0 + uint64_t(step) * i;
                if (!in) byte[i] = 0;     // groups past K
                // the word of four groups, gathered in the first of their lanes
                constexpr int kStep = kNv ? 1 : 2;   // lanes a group
                byte[i] |= __shfl_down_sync(0xFFFFFFFFu, byte[i], kStep) << 8;
                byte[i] |= __shfl_down_sync(0xFFFFFFFFu, byte[i], 2 * kStep) << 16;
                if (in) {
                    xq[(row * K + col) / 16] = q[i];
                    if (lane % (4 * kStep) == 0)
                        *reinterpret_cast<uint32_t*>(xs + word + scale_word_at(static_cast<int64_t>(row), 0, tiles)) = byte[i];
                }
            }
        };
        uint64_t row = spans < nwarps ? warp / spans : 0;
        if constexpr (!kSilu)
            for (; row + step < M; row += 2 * uint64_t(step)) rows(row, std::integral_constant<int, 2>());
        for (; row < M; row += step) rows(row, std::integral_constant<int, 1>());
    }
}

template <typename T, bool kNv>
__global__ void __launch_bounds__(kThreads) dequant_fp4_kernel(const uint2* __restrict__ xq, const uint8_t* __restrict__ xs,
                                                               const float* __restrict__ tensor_scale, T* __restrict__ y,
                                                               uint32_t K, uint32_t spans, uint32_t total) {
    ptx::launch_dependents();
    ptx::grid_dependency_wait();
    const float t = kNv && tensor_scale ? __ldg(tensor_scale) : 1.0f;
    const int64_t tiles = scale_tiles(K, kNv);
    const uint32_t lane = threadIdx.x & 31;
    const uint32_t nwarps = gridDim.x * (kThreads / 32);
    const bool wide = (reinterpret_cast<uintptr_t>(y) & 31u) == 0;
    constexpr int kUnroll = 4;
    for (uint64_t w0 = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5); w0 < total; w0 += uint64_t(nwarps) * kUnroll) {
        uint2 q[kUnroll];
        uint32_t byte[kUnroll];
        int64_t at[kUnroll];
#pragma unroll
        for (int i = 0; i < kUnroll; ++i) {
            const uint64_t w = w0 + uint64_t(nwarps) * i;
            const uint32_t row = static_cast<uint32_t>(w) / spans;
            const uint32_t col = (static_cast<uint32_t>(w) - row * spans) * kSpan + lane * 16;
            at[i] = w < total && col < K ? row * int64_t(K) + col : -1;
            q[i] = make_uint2(0, 0);
            byte[i] = 0;
            if (at[i] >= 0) {
                const uint32_t g = kNv ? col / 16 : col / 32;
                q[i] = __ldg(xq + at[i] / 16);
                byte[i] = __ldg(xs + scale_word_at(row, g / 4, tiles) + g % 4);
            }
        }
#pragma unroll
        for (int i = 0; i < kUnroll; ++i) {
            if (at[i] < 0) continue;   // past the row, or past the end
            const float s = kNv ? __fmul_rn(of_e4m3(byte[i]), t) : of_ue8m0(byte[i]);
            const float2 s2 = make_float2(s, s);
            uint32_t out[8];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                uint32_t p[4];
                values8(h ? q[i].y : q[i].x, p);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float2 v = lat::mul2(Pair<__half>::unpack(p[j]), s2);
                    out[4 * h + j] = Pair<T>::pack(v.x, v.y);
                }
            }
            if (wide) {
                ptx::st_global_v8(y + at[i], out);
            } else {
                *reinterpret_cast<uint4*>(y + at[i]) = make_uint4(out[0], out[1], out[2], out[3]);
                *reinterpret_cast<uint4*>(y + at[i] + 8) = make_uint4(out[4], out[5], out[6], out[7]);
            }
        }
    }
}

cudaLaunchConfig_t config(cudaLaunchAttribute* attr, int64_t blocks, cudaStream_t st) {
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(blocks));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cfg;
}

template <typename T, bool kNv, bool kSilu, bool kWhole>
sgq_status launch_spans(const void* x, int64_t M, int64_t K, int64_t stride, const float* t, void* xq, void* xs, int sms,
                     cudaStream_t st) {
    const int64_t spans = (K + kSpan - 1) / kSpan, total = M * spans;
    const int64_t per = kThreads / 32, cap = int64_t(sms) * 8;
    const int64_t want = (total + per - 1) / per;
    cudaLaunchAttribute attr[1];
    cudaLaunchConfig_t cfg = config(attr, want < cap ? want : cap, st);
    if (cudaLaunchKernelEx(&cfg, quant_fp4_kernel<T, kNv, kSilu, kWhole>, static_cast<const T*>(x), stride, t,
                           static_cast<uint2*>(xq), static_cast<uint8_t*>(xs), static_cast<uint32_t>(M),
                           static_cast<uint32_t>(K), static_cast<uint32_t>(spans)) != cudaSuccess)
        return SGQ_ERR_CUDA;
    note_launch();
    return SGQ_OK;
}
template <typename T, bool kNv, bool kSilu>
sgq_status run_quant(const void* x, int64_t M, int64_t K, int64_t stride, const float* t, void* xq, void* xs, int sms,
                     cudaStream_t st) {
    const bool aligned = kSilu || ((reinterpret_cast<uintptr_t>(x) | static_cast<uintptr_t>(M > 1 ? stride : 0) * 2) & 31u) == 0;
    return K % kSpan == 0 && aligned ? launch_spans<T, kNv, kSilu, true>(x, M, K, stride, t, xq, xs, sms, st)
                                     : launch_spans<T, kNv, kSilu, false>(x, M, K, stride, t, xq, xs, sms, st);
}
template <typename T>
sgq_status pick_quant(const void* x, int64_t M, int64_t K, int64_t stride, bool nv, const float* t, bool silu, void* xq,
                      void* xs, int sms, cudaStream_t st) {
    if (nv)
        return silu ? run_quant<T, true, true>(x, M, K, stride, t, xq, xs, sms, st)
                    : run_quant<T, true, false>(x, M, K, stride, t, xq, xs, sms, st);
    return silu ? run_quant<T, false, true>(x, M, K, stride, t, xq, xs, sms, st)
                : run_quant<T, false, false>(x, M, K, stride, t, xq, xs, sms, st);
}
template <typename T, bool kNv>
sgq_status run_dequant(const void* xq, const void* xs, int64_t M, int64_t K, const float* t, void* y, int sms,
                       cudaStream_t st) {
    const int64_t spans = (K + kSpan - 1) / kSpan, total = M * spans;
    const int64_t per = kThreads / 32, cap = int64_t(sms) * 8;
    const int64_t want = (total + per - 1) / per;
    cudaLaunchAttribute attr[1];
    cudaLaunchConfig_t cfg = config(attr, want < cap ? want : cap, st);
    if (cudaLaunchKernelEx(&cfg, dequant_fp4_kernel<T, kNv>, static_cast<const uint2*>(xq), static_cast<const uint8_t*>(xs), t,
                           static_cast<T*>(y), static_cast<uint32_t>(K), static_cast<uint32_t>(spans),
                           static_cast<uint32_t>(total)) != cudaSuccess)
        return SGQ_ERR_CUDA;
    note_launch();
    return SGQ_OK;
}

}  // namespace

sgq_status launch_quant_fp4(const void* x, int64_t M, int64_t K, int64_t stride, int format, const float* t, int silu,
                            int dtype, void* xq, void* xs, cudaStream_t st) {
    DeviceInfo di;
    const sgq_status rc = device_info(&di);
    if (rc != SGQ_OK) return rc;
    if (!built_for(di)) return SGQ_ERR_UNSUPPORTED;
    return dtype == SGQ_BF16
               ? pick_quant<__nv_bfloat16>(x, M, K, stride, format == SGQ_NVFP4, t, silu != 0, xq, xs, di.sm_count, st)
               : pick_quant<__half>(x, M, K, stride, format == SGQ_NVFP4, t, silu != 0, xq, xs, di.sm_count, st);
}

sgq_status launch_dequant_fp4(const void* xq, const void* xs, int64_t M, int64_t K, int format, const float* t, int dtype,
                              void* y, cudaStream_t st) {
    DeviceInfo di;
    const sgq_status rc = device_info(&di);
    if (rc != SGQ_OK) return rc;
    if (!built_for(di)) return SGQ_ERR_UNSUPPORTED;
    if (format == SGQ_NVFP4)
        return dtype == SGQ_BF16 ? run_dequant<__nv_bfloat16, true>(xq, xs, M, K, t, y, di.sm_count, st)
                                 : run_dequant<__half, true>(xq, xs, M, K, t, y, di.sm_count, st);
    return dtype == SGQ_BF16 ? run_dequant<__nv_bfloat16, false>(xq, xs, M, K, t, y, di.sm_count, st)
                             : run_dequant<__half, false>(xq, xs, M, K, t, y, di.sm_count, st);
}

}  // namespace sgq
