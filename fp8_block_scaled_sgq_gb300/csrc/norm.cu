// The norm before a block, and what stands between two blocks: norm of a
// block's output, gate, scale, residual, next norm, with the result in 16 bits
// or quantised for the next linear, for sm_103a.
//
//   N(v, w) = v / sqrt(mean(v^2) + eps) * (w + offset)            per row
//   u = x, or N(x, w_post);   h = 16 bits of (r residual + s gate u)
//   y = N(h, w)   (without a residual: y = N(x, w))
//
// The second norm is of h as it is stored, so that it is the norm that a
// separate call would take.  Everything between is fp32; y is rounded once, to
// 16 bits, to FP8 groups (quant_math.cuh) or to the 4-bit form
// (fp4_common.cuh).
//
// Bound by HBM: each of x, residual, h and y passes once, a row stays in
// registers (8 elements a 16-byte load) between its one or two sums.
#include <cuda_runtime.h>

#include "fp4_common.cuh"
#include "ptx.cuh"
#include "sgq_internal.h"

namespace sgq {
namespace {

using namespace fp4;

enum Out : int { kNone, kSame, kFp8, kMx4, kNv4 };

struct Args {
    const void *x, *post, *gate, *residual, *weight;
    const float* tensor_scale;
    void *h, *y, *ys;
    int64_t M, x_s, r_s, h_s, gate_s, gate_rows;
    int K, group, scale_kind;   // FP8: values a group; scales fp32 (0), fp32 powers of two (1), UE8M0 bytes (2)
    float eps, offset, scale, residual_scale;
};

// Sum over the kRow threads of a row (whole warps), in every one of them.
template <int kRow>
__device__ __forceinline__ float row_sum(float s, float* part) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, off);
    if constexpr (kRow > 32) {
        if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = s;
        __syncthreads();
        constexpr int kWarps = kRow / 32;
        s = part[threadIdx.x & (kWarps - 1)];
#pragma unroll
        for (int off = kWarps / 2; off > 0; off >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, off);
    }
    return s;
}

// kRow threads a row, each with up to kVec columns of 8 elements, kRow columns apart.
template <typename T, int kRow, int kVec, Out kOut>
__global__ void __launch_bounds__(kRow == 32 ? 128 : kRow) norm_kernel(const Args a) {
    __shared__ float part[2][32];
    ptx::launch_dependents();
    ptx::grid_dependency_wait();
    const int tid = kRow == 32 ? threadIdx.x & 31 : threadIdx.x;
    const int64_t m = kRow == 32 ? int64_t(blockIdx.x) * 4 + (threadIdx.x >> 5) : int64_t(blockIdx.x);
    if (m >= a.M) return;   // (a whole warp, which meets no other)
    const int cols = a.K / 8;
    const float inv_k = 1.0f / static_cast<float>(a.K);
    // (x and residual may be h: plain loads)
    auto row_of = [&](const void* p, int64_t at, int c) { return reinterpret_cast<const uint4*>(static_cast<const T*>(p) + at)[c]; };
    auto load = [&](const void* p, int64_t at, int c) { return __ldg(reinterpret_cast<const uint4*>(static_cast<const T*>(p) + at) + c); };

    float v[kVec][8];
    uint4 r[kVec];
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
        const int c = tid + i * kRow;
        uint4 w = make_uint4(0, 0, 0, 0);
        r[i] = w;
        if (c < cols) {
            w = row_of(a.x, m * a.x_s, c);
            if (a.residual) r[i] = row_of(a.residual, m * a.r_s, c);
        }
        unpack8<T>(w, v[i]);
    }
    auto rstd_of = [&](float* p) {
        float s = 0.0f;
#pragma unroll
        for (int i = 0; i < kVec; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) s = fmaf(v[i][j], v[i][j], s);
        return __frsqrt_rn(row_sum<kRow>(s, p) * inv_k + a.eps);
    };
    if (a.residual) {
        if (a.post) {
            const float rstd = rstd_of(part[0]);
#pragma unroll
            for (int i = 0; i < kVec; ++i) {
                const int c = tid + i * kRow;
                if (c >= cols) continue;
                float w[8];
                unpack8<T>(load(a.post, 0, c), w);
#pragma unroll
                for (int j = 0; j < 8; ++j) v[i][j] = v[i][j] * rstd * (w[j] + a.offset);
            }
        }
        if (a.gate) {
            const int64_t at = m / a.gate_rows * a.gate_s;
#pragma unroll
            for (int i = 0; i < kVec; ++i) {
                const int c = tid + i * kRow;
                if (c >= cols) continue;
                float g[8];
                unpack8<T>(load(a.gate, at, c), g);
#pragma unroll
                for (int j = 0; j < 8; ++j) v[i][j] *= g[j];
            }
        }
#pragma unroll
        for (int i = 0; i < kVec; ++i) {
            const int c = tid + i * kRow;
            float f[8];
            unpack8<T>(r[i], f);
#pragma unroll
            for (int j = 0; j < 8; ++j) f[j] = fmaf(a.scale, v[i][j], a.residual_scale * f[j]);
            const uint4 h = pack8<T>(f);
            if (c < cols) reinterpret_cast<uint4*>(static_cast<T*>(a.h) + m * a.h_s)[c] = h;
            unpack8<T>(h, v[i]);   // what is stored
        }
    }
    if constexpr (kOut == kNone) return;

    const float rstd = rstd_of(part[1]);
    float t = 1.0f, t6 = kMax;
    if constexpr (kOut == kNv4) {
        if (a.tensor_scale) t = __ldg(a.tensor_scale);
        t6 = __fmul_rn(t, kMax);
    }
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
        const int c = tid + i * kRow;
        const bool in = c < cols;
        if (in) {
            float w[8];
            unpack8<T>(load(a.weight, 0, c), w);
#pragma unroll
            for (int j = 0; j < 8; ++j) v[i][j] = v[i][j] * rstd * (w[j] + a.offset);
        }
        // (groups are whole, and of neighbouring lanes: rows are whole warps' columns)
        if constexpr (kOut == kSame) {
            if (in) static_cast<uint4*>(a.y)[m * cols + c] = pack8<T>(v[i]);
        } else if constexpr (kOut == kFp8) {
            float amax = in ? qm::amax8(v[i]) : 0.0f;
            const int lanes = a.group / 8;
            amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 1));
            amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 2));
            if (lanes == 16) {
                amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 4));
                amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 8));
            }
            const bool pow2 = a.scale_kind != 0;
            const float s = qm::group_scale(amax, pow2);
            if (in) {
                static_cast<uint2*>(a.y)[m * cols + c] = qm::quantize8(v[i], s, pow2);
                if (c % lanes == 0) {
                    const int64_t g = (m * cols + c) / lanes;
                    if (a.scale_kind == 2) static_cast<uint8_t*>(a.ys)[g] = static_cast<uint8_t>(__float_as_uint(s) >> 23);
                    else static_cast<float*>(a.ys)[g] = s;
                }
            }
        } else {
            constexpr bool kNv = kOut == kNv4;
            constexpr int kLanes = kNv ? 2 : 4;   // a group's
            uint32_t amax = in ? amax_bits8(v[i]) : 0u;
            amax = max(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 1));
            if constexpr (!kNv) amax = max(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 2));
            float div;
            uint32_t byte = scale_byte<kNv>(amax, t, t6, div);
            if (!in) byte = 0;
            byte |= __shfl_down_sync(0xFFFFFFFFu, byte, kLanes) << 8;
            byte |= __shfl_down_sync(0xFFFFFFFFu, byte, 2 * kLanes) << 16;
            if (in) {
                static_cast<uint32_t*>(a.y)[m * cols + c] = encode8<kNv>(v[i], div);
                if (c % (4 * kLanes) == 0)
                    *reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(a.ys) +
                                                 scale_word_at(m, c / (4 * kLanes), scale_tiles(a.K, kNv))) = byte;
            }
        }
    }
}

template <typename T, int kRow, int kVec, Out kOut>
sgq_status run(const Args& a, cudaStream_t st) {
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(kRow == 32 ? (a.M + 3) / 4 : a.M));
    cfg.blockDim = dim3(kRow == 32 ? 128 : kRow);
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, norm_kernel<T, kRow, kVec, kOut>, a) != cudaSuccess) return SGQ_ERR_CUDA;
    note_launch();
    return SGQ_OK;
}
template <typename T, Out kOut>
sgq_status by_width(const Args& a, cudaStream_t st) {
    if (a.K <= 1024) return run<T, 32, 4, kOut>(a, st);
    if (a.K <= 4096) return run<T, 128, 4, kOut>(a, st);
    if (a.K <= 8192) return run<T, 256, 4, kOut>(a, st);
    if (a.K <= 16384) return run<T, 512, 4, kOut>(a, st);
    return run<T, 1024, 4, kOut>(a, st);
}
template <typename T>
sgq_status by_out(const Args& a, Out out, cudaStream_t st) {
    switch (out) {
        case kNone: return by_width<T, kNone>(a, st);
        case kSame: return by_width<T, kSame>(a, st);
        case kFp8: return by_width<T, kFp8>(a, st);
        case kMx4: return by_width<T, kMx4>(a, st);
        case kNv4: return by_width<T, kNv4>(a, st);
    }
    return SGQ_ERR_INVALID_ARG;
}

}  // namespace

sgq_status launch_norm(const NormArgs& n, cudaStream_t st) {
    DeviceInfo di;
    const sgq_status rc = device_info(&di);
    if (rc != SGQ_OK) return rc;
    if (!built_for(di)) return SGQ_ERR_UNSUPPORTED;
    Args a{};
    a.x = n.x; a.post = n.post; a.gate = n.gate; a.residual = n.residual; a.weight = n.weight;
    a.tensor_scale = n.tensor_scale; a.h = n.h; a.y = n.y; a.ys = n.ys;
    a.M = n.M; a.x_s = n.x_s; a.r_s = n.r_s; a.h_s = n.h_s; a.gate_s = n.gate_s;
    a.gate_rows = n.gate_rows; a.K = static_cast<int>(n.K);
    a.eps = n.eps; a.offset = n.offset; a.scale = n.scale; a.residual_scale = n.residual_scale;
    Out out = kNone;
    switch (n.out) {
        case SGQ_OUT_NONE: break;
        case SGQ_OUT_16: out = kSame; break;
        case SGQ_OUT_MXFP4: out = kMx4; break;
        case SGQ_OUT_NVFP4: out = kNv4; break;
        default:
            out = kFp8;
            a.group = n.out & SGQ_OUT_GROUP_128 ? 128 : 32;
            a.scale_kind = (n.out & SGQ_OUT_UE8M0) != 0 ? 2 : (n.out & SGQ_OUT_POW2) != 0 ? 1 : 0;
    }
    return n.dtype == SGQ_BF16 ? by_out<__nv_bfloat16>(a, out, st) : by_out<__half>(a, out, st);
}

}  // namespace sgq
