// Expanded latent attention of ragged prompts: a simple form, one warp for
// each (query token, head).
//
// Softmax in one pass with a running maximum m and sum l: a key with score s
// (in powers of two) turns (m, l, o) into (m', l 2^(m-m') + 2^(s-m'),
// o 2^(m-m') + 2^(s-m') v), m' = max(m, s).  Lane i holds elements i, i + 32,
// ... of a row, so a key costs one row read and one warp sum.
#include <cuda_runtime.h>

#include "latent_common.cuh"
#include "sgq_internal.h"

namespace sgq {
namespace {

constexpr int kWarps = 8;
constexpr int kMaxPer = 6;   // (128 + 64) / 32 elements a lane

template <typename T>
__device__ __forceinline__ float to_f(T v);
template <>
__device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
template <>
__device__ __forceinline__ float to_f(__half v) { return __half2float(v); }
template <typename T>
__device__ __forceinline__ T from_f(float v);
template <>
__device__ __forceinline__ __nv_bfloat16 from_f(float v) { return __float2bfloat16_rn(v); }
template <>
__device__ __forceinline__ __half from_f(float v) { return __float2half_rn(v); }

struct RowState {
    float q[kMaxPer], o[kMaxPer], m = -INFINITY, l = 0.0f;
};
__device__ __forceinline__ void take(RowState& r, const float (&k)[kMaxPer], const float (&v)[kMaxPer], float scale2) {
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < kMaxPer; ++i) s = fmaf(r.q[i], k[i], s);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
    s *= scale2;
    const float m = fmaxf(r.m, s);
    const float a = exp2f(r.m - m), p = exp2f(s - m);
    r.l = r.l * a + p;
#pragma unroll
    for (int i = 0; i < kMaxPer; ++i) r.o[i] = r.o[i] * a + p * v[i];
    r.m = m;
}
template <typename T>
__device__ __forceinline__ void finish(const RowState& r, T* out, int width, float* lse) {
    const int lane = threadIdx.x & 31;
    const float inv = r.l > 0.0f ? 1.0f / r.l : 0.0f;
#pragma unroll
    for (int i = 0; i < kMaxPer; ++i)
        if (lane + 32 * i < width) out[lane + 32 * i] = from_f<T>(r.o[i] * inv);
    if (lse != nullptr && lane == 0) *lse = r.l > 0.0f ? r.m * 0.69314718055994531f + logf(r.l) : -INFINITY;
}

// The request that token t belongs to, in [0, B); starts clamped to [0, T].
__device__ __forceinline__ int64_t request_of(const int32_t* starts, int64_t B, int64_t t) {
    int64_t lo = 0, hi = B;
    while (hi - lo > 1) {
        const int64_t mid = (lo + hi) / 2;
        if (starts[mid] <= t) lo = mid;
        else hi = mid;
    }
    return lo;
}

template <typename T>
__global__ void __launch_bounds__(kWarps * 32) latent_prefill_simple(const PrefillArgs a) {
    const int64_t row = int64_t(blockIdx.x) * kWarps + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    if (row >= a.T * a.H) return;
    const int64_t t = row / a.H, h = row % a.H;
    const int64_t b = request_of(a.q_starts, a.B, t);
    const int64_t i = t - a.q_starts[b], n = a.q_starts[b + 1] - a.q_starts[b];
    const int64_t k0 = min(max(int64_t(a.kv_starts[b]), int64_t(0)), a.S);
    const int64_t m = min(max(int64_t(a.kv_starts[b + 1]), k0), a.S) - k0;
    const int W = a.N + a.R;
    RowState r;
    const T* q = static_cast<const T*>(a.q) + t * a.q_t + h * a.q_h;
#pragma unroll
    for (int e = 0; e < kMaxPer; ++e) {
        r.q[e] = lane + 32 * e < W ? to_f(q[lane + 32 * e]) : 0.0f;
        r.o[e] = 0.0f;
    }
    const int64_t end = a.causal ? min(m, m - n + i + 1) : m;
    for (int64_t j = k0; j < k0 + end; ++j) {
        const T* kp = static_cast<const T*>(a.k) + j * a.k_t + h * a.k_h;
        const T* rp = static_cast<const T*>(a.k_rot) + j * a.kr_t - a.N;
        const T* vp = static_cast<const T*>(a.v) + j * a.v_t + h * a.v_h;
        float k[kMaxPer], v[kMaxPer];
#pragma unroll
        for (int e = 0; e < kMaxPer; ++e) {
            const int c = lane + 32 * e;
            k[e] = c < a.N ? to_f(kp[c]) : (c < W ? to_f(rp[c]) : 0.0f);
            v[e] = c < a.N ? to_f(vp[c]) : 0.0f;
        }
        take(r, k, v, a.scale * 1.44269504088896341f);
    }
    finish(r, static_cast<T*>(a.out) + row * a.N, a.N, a.lse ? a.lse + row : nullptr);
}

}  // namespace

sgq_status launch_latent_prefill(const PrefillArgs& args, cudaStream_t st) {
    PrefillArgs a = args;
    const sgq_status rc = gemm::status_word(&a.status);
    if (rc != SGQ_OK) return rc;
    const int64_t blocks = (a.T * a.H + kWarps - 1) / kWarps;
    if (blocks > INT32_MAX) return SGQ_ERR_INVALID_ARG;
    if (a.dtype == SGQ_BF16) latent_prefill_simple<__nv_bfloat16><<<blocks, kWarps * 32, 0, st>>>(a);
    else latent_prefill_simple<__half><<<blocks, kWarps * 32, 0, st>>>(a);
    if (cudaGetLastError() != cudaSuccess) return SGQ_ERR_CUDA;
    note_launch();
    return SGQ_OK;
}

}  // namespace sgq
