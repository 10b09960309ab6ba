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
// Each of x, residual, h and y passes once; a row stays in registers (8 elements
// a 16-byte load) between its one or two sums.  Measured, 4096 x 7168 in bf16,
// inputs from HBM: a norm 18.1 us (6.5 TB/s), residual alone 25.5 (6.9), with the
// next norm 40.1 (5.9): HBM.  A norm into FP8 groups 19.7 (4.5), MXFP4 22.0 (3.4),
// NVFP4 25.9 (2.9), and with every step before it 38.0 (5.4), 39.1, 42.4 (4.5):
// instructions beside it, 204 (FP8) to 227 (NVFP4) a warp for 8 elements a lane
// with every step.  One row: 3.0 us in a graph.
#include <cuda_runtime.h>

#include "fp4_common.cuh"
#include "ptx.cuh"
#include "resident.h"
#include "sgq_internal.h"

namespace sgq {
namespace {

using namespace fp4;

enum Out : int { kNone, kSame, kFp8, kMx4, kNv4 };

struct Args {
    const void *x, *post, *gate, *residual, *weight;
    const float* tensor_scale;
    void *h, *y, *ys;
    int64_t M, x_s, r_s, h_s, gate_s;
    uint32_t gate_rows;
    int depth;                  // rows under way (norm_walk_kernel)
    int K, group_shift, scale_kind;   // FP8: columns of 8 a group, as a power of two; scales fp32 (0), fp32 powers of two (1), UE8M0 bytes (2)
    float inv_k, eps, offset, scale, residual_scale;
};

// Sum over the kRow threads of a row (16 neighbouring lanes, or whole warps), in every one of them.
template <int kRow>
__device__ __forceinline__ float row_sum(float s, float* part) {
#pragma unroll
    for (int off = kRow < 32 ? kRow / 2 : 16; off > 0; off >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, off);
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

template <typename T>
__device__ __forceinline__ uint4 column(const void* p, int64_t at, int c) {
    return __ldg(reinterpret_cast<const uint4*>(static_cast<const T*>(p) + at) + c);
}
// Arithmetic on eight values, two an instruction.
__device__ __forceinline__ float2 two(const float (&v)[8], int j) { return make_float2(v[2 * j], v[2 * j + 1]); }
__device__ __forceinline__ void set(float (&v)[8], int j, float2 x) {
    v[2 * j] = x.x;
    v[2 * j + 1] = x.y;
}
template <int kVec>
__device__ __forceinline__ float squares(const float (&v)[kVec][8]) {
    float2 s = make_float2(0.0f, 0.0f);
#pragma unroll
    for (int i = 0; i < kVec; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) s = lat::fma2(two(v[i], j), two(v[i], j), s);
    return s.x + s.y;
}
__device__ __forceinline__ float rstd_of(float sum, const Args& a) {
    return __frsqrt_rn(fmaf(sum, a.inv_k, a.eps));
}
// v * factor * (weight + offset)
template <typename T>
__device__ __forceinline__ void weigh(float (&v)[8], float factor, const uint4& weight, float offset) {
    float w[8];
    unpack8<T>(weight, w);
    const float2 f = make_float2(factor, factor), o = make_float2(offset, offset);
#pragma unroll
    for (int j = 0; j < 4; ++j) set(v, j, lat::mul2(lat::mul2(two(v, j), f), lat::add2(two(w, j), o)));
}
// v * gate
template <typename T>
__device__ __forceinline__ void open(float (&v)[8], const uint4& gate) {
    float g[8];
    unpack8<T>(gate, g);
#pragma unroll
    for (int j = 0; j < 4; ++j) set(v, j, lat::mul2(two(v, j), two(g, j)));
}
// h = residual_scale * residual + scale * u: what is stored, and its values.
template <typename T>
__device__ __forceinline__ uint4 add_residual(float (&v)[8], const uint4& residual, const Args& a) {
    float r[8];
    unpack8<T>(residual, r);
    const float2 s = make_float2(a.scale, a.scale), t = make_float2(a.residual_scale, a.residual_scale);
#pragma unroll
    for (int j = 0; j < 4; ++j) set(r, j, lat::fma2(s, two(v, j), lat::mul2(t, two(r, j))));
    const uint4 h = pack8<T>(r);
    unpack8<T>(h, v);
    return h;
}

// qm::group_scale without the division's branches.  (An infinity stays one: its remainder is none.)
__device__ __forceinline__ float fp8_scale(float amax, bool pow2) {
    float s = quotient(fmaxf(amax, qm::kEps), qm::kFp8Max, 1.0f / qm::kFp8Max);
    if (__float_as_uint(amax) == kInf) s = amax;
    if (pow2) {
        uint32_t u = __float_as_uint(s);
        if (u & 0x7FFFFFu) u = (u & kInf) + 0x800000u;
        s = __uint_as_float(u);
    }
    return s;
}

// The codes of a column's eight quotients.
template <Out kOut>
__device__ __forceinline__ void store_codes(const Args& a, int64_t at, const float (&q)[8]) {
    if constexpr (kOut == kFp8) {
        uint32_t p[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
            p[j] = __nv_cvt_float2_to_fp8x2(make_float2(q[2 * j], q[2 * j + 1]), __NV_SATFINITE, __NV_E4M3);
        static_cast<uint2*>(a.y)[at] = make_uint2(p[0] | (p[1] << 16), p[2] | (p[3] << 16));
    } else {
        static_cast<uint32_t*>(a.y)[at] = codes8(q);
    }
}

// Columns tid, tid + step, ... of row m of y, in what `out` asks for.  v: their
// values, negated where they are to be quantised.  All lanes of a warp call
// it, those past the row's end (zeros) too: groups lie in neighbouring lanes,
// and are whole.  cols: the row's, or 0 for none.  The first kSure columns are within the row for every thread.
//
// A group's largest magnitude, its scale and the reciprocal of it are the same
// for all of its lanes, so they are taken once: lanes that meet in the maximum
// over a group each keep half of the columns, until a lane owns one (two of
// four where a group is two lanes), and hand the quotients' factors back.
template <typename T, Out kOut, int kVec, int kSure>
__device__ __forceinline__ void emit(const Args& a, int64_t m, int cols, int tid, int step, const float (&v)[kVec][8], const TensorScale& ts) {
    if constexpr (kOut == kSame) {
#pragma unroll
        for (int i = 0; i < kVec; ++i)
            if (i < kSure || tid + i * step < cols) static_cast<uint4*>(a.y)[m * cols + tid + i * step] = pack8<T>(v[i]);
    } else {
        constexpr unsigned kAll = 0xFFFFFFFFu;
        constexpr bool kNv = kOut == kNv4;
        constexpr int kOwn = kNv && kVec == 4 ? 2 : 1;
        static_assert(kVec == 1 || kVec == 2 || kVec == 4, "columns a thread");
        const int lane = threadIdx.x & 31;
        const bool odd1 = (lane & 1) != 0, odd2 = (lane & 2) != 0;
        uint32_t top[kVec], own[2];
#pragma unroll
        for (int i = 0; i < kVec; ++i) top[i] = kOut == kFp8 ? amax_bits8_of_numbers(v[i]) : amax_bits8(v[i]);
        int first;   // the first column that this lane owns
        if constexpr (kVec == 4) {
            own[0] = max(odd1 ? top[2] : top[0], __shfl_xor_sync(kAll, odd1 ? top[0] : top[2], 1));
            own[1] = max(odd1 ? top[3] : top[1], __shfl_xor_sync(kAll, odd1 ? top[1] : top[3], 1));
            first = odd1 ? 2 : 0;
            if constexpr (!kNv) {
                own[0] = max(odd2 ? own[1] : own[0], __shfl_xor_sync(kAll, odd2 ? own[0] : own[1], 2));
                first += odd2 ? 1 : 0;
            }
        } else {
            if constexpr (kVec == 2) own[0] = max(odd1 ? top[1] : top[0], __shfl_xor_sync(kAll, odd1 ? top[0] : top[1], 1));
            else own[0] = max(top[0], __shfl_xor_sync(kAll, top[0], 1));
            first = kVec == 2 && odd1 ? 1 : 0;
            if constexpr (!kNv) own[0] = max(own[0], __shfl_xor_sync(kAll, own[0], 2));
        }
        if (kOut == kFp8 && a.group_shift == 4) {
            own[0] = max(own[0], __shfl_xor_sync(kAll, own[0], 4));
            own[0] = max(own[0], __shfl_xor_sync(kAll, own[0], 8));
        }
        float rcp[kOwn];   // what the group's values are multiplied by; in 4 bits, not below 0: what they are divided by (divided8)
#pragma unroll
        for (int k = 0; k < kOwn; ++k) {
            const int c = tid + (first + k) * step;
            if constexpr (kOut == kFp8) {
                const float s = fp8_scale(__uint_as_float(own[k]), a.scale_kind != 0);
                rcp[k] = -__frcp_rn(s);
                // the first lanes of a group, one for each column
                if ((kSure == kVec || c < cols) && (lane & ((1 << a.group_shift) - 1)) < kVec) {
                    const int64_t g = m * (cols >> a.group_shift) + (c >> a.group_shift);
                    if (a.scale_kind == 2) static_cast<uint8_t*>(a.ys)[g] = static_cast<uint8_t>(__float_as_uint(s) >> 23);
                    else static_cast<float*>(a.ys)[g] = s;
                }
            } else {
                constexpr int kLanes = kNv ? 2 : 4;   // a group's; a scale word's are four times as many
                float div;
                uint32_t byte = scale_byte<kNv>(own[k], ts, div);
                rcp[k] = (kNv ? in_range(div) : div != 0.0f) ? minus_reciprocal<kNv>(div) : div;
                if (kSure < kVec && c >= cols) byte = 0;              // groups past the row's end
                byte |= __shfl_down_sync(kAll, byte, kLanes) << 8;
                byte |= __shfl_down_sync(kAll, byte, 2 * kLanes) << 16;
                if ((kSure == kVec || c < cols) && (lane & (4 * kLanes - 1)) < (kNv && kVec > 1 ? 2 : kVec))
                    *reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(a.ys) +
                                                 scale_word_at(m, c / (4 * kLanes), scale_tiles(a.K, kNv))) = byte;
            }
        }
#pragma unroll
        for (int i = 0; i < kVec; ++i) {
            const int c = tid + i * step;
            const int from = kVec == 1 ? lane : kVec == 2 ? (lane & ~1) | i : kNv ? (lane & ~1) | (i >> 1) : (lane & ~3) | (i >> 1) | ((i & 1) << 1);
            const float r = __shfl_sync(kAll, rcp[kVec == 4 && kNv ? i & 1 : 0], from);
            if (kOut != kFp8 && r >= 0.0f) {
                if (i < kSure || c < cols) static_cast<uint32_t*>(a.y)[m * cols + c] = divided8(v[i], r);
            } else {
                float q[8];
#pragma unroll
                for (int j = 0; j < 4; ++j) set(q, j, lat::mul2(two(v[i], j), make_float2(r, r)));
                if (i < kSure || c < cols) store_codes<kOut>(a, m * cols + c, q);
            }
        }
    }
}
__host__ __device__ constexpr bool negated(Out out) { return out == kFp8 || out == kMx4 || out == kNv4; }

// Narrow rows, up to 512 elements: kRow lanes a row (two rows a warp where they
// are 16), and kN steps of them at once, so that enough loads are under way.  A
// grid that fills the SMs walks over them: 234375 x 128 in 16 bits 21.6 us (5.6
// TB/s), with a residual 41.1, into FP8 28.6 (a warp a row in CTAs of four rows:
// 97.8, 130.9, 114.1), MXFP4 27.9, NVFP4 31.0.  Quantised, it is instructions: a
// thread has one column of up to 256 elements, so that each lane takes its group's
// maximum, scale and reciprocal for itself (emit).
template <typename T, int kRow, int kVec, int kN, Out kOut>
__global__ void __launch_bounds__(128, kVec == 2 ? 5 : 6) norm_rows_kernel(const Args a) {
    ptx::launch_dependents();
    ptx::grid_dependency_wait();
    const int lane = threadIdx.x & 31, tid = lane & (kRow - 1), cols = a.K / 8;
    constexpr int kRows = 32 / kRow;   // of a warp
    uint4 weight[kVec], post[kVec];
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
        const int c = tid + i * kRow;
        weight[i] = post[i] = make_uint4(0, 0, 0, 0);
        if (kOut != kNone && c < cols) weight[i] = column<T>(a.weight, 0, c);
        if (a.post && c < cols) post[i] = column<T>(a.post, 0, c);
    }
    const TensorScale ts(kOut == kNv4 ? a.tensor_scale : nullptr);
    const int64_t step = int64_t(gridDim.x) * 4 * kRows * kN;
    for (int64_t m0 = (int64_t(blockIdx.x) * 4 + (threadIdx.x >> 5)) * kRows * kN; m0 < a.M; m0 += step) {
        uint4 x[kN][kVec], r[kN][kVec];
#pragma unroll
        for (int n = 0; n < kN; ++n) {
            const int64_t m = m0 + n * kRows + lane / kRow;
#pragma unroll
            for (int i = 0; i < kVec; ++i) {
                const int c = tid + i * kRow;
                x[n][i] = r[n][i] = make_uint4(0, 0, 0, 0);
                if (m < a.M && c < cols) {   // (x and residual may be h: plain loads)
                    x[n][i] = reinterpret_cast<const uint4*>(static_cast<const T*>(a.x) + m * a.x_s)[c];
                    if (a.residual) r[n][i] = reinterpret_cast<const uint4*>(static_cast<const T*>(a.residual) + m * a.r_s)[c];
                }
            }
        }
#pragma unroll
        for (int n = 0; n < kN; ++n) {
            const int64_t m = m0 + n * kRows + lane / kRow;
            const int live = m < a.M ? cols : 0;
            float v[kVec][8];
#pragma unroll
            for (int i = 0; i < kVec; ++i) unpack8<T>(x[n][i], v[i]);
            if (a.residual) {
                if (a.post) {
                    const float rstd = rstd_of(row_sum<kRow>(squares(v), nullptr), a);
#pragma unroll
                    for (int i = 0; i < kVec; ++i) weigh<T>(v[i], rstd, post[i], a.offset);
                }
                if (a.gate) {
                    const int64_t at = static_cast<uint32_t>(m) / a.gate_rows * a.gate_s;
#pragma unroll
                    for (int i = 0; i < kVec; ++i)
                        if (tid + i * kRow < live) open<T>(v[i], column<T>(a.gate, at, tid + i * kRow));
                }
#pragma unroll
                for (int i = 0; i < kVec; ++i) {
                    const uint4 h = add_residual<T>(v[i], r[n][i], a);
                    if (tid + i * kRow < live) reinterpret_cast<uint4*>(static_cast<T*>(a.h) + m * a.h_s)[tid + i * kRow] = h;
                }
            }
            if constexpr (kOut != kNone) {
                float rstd = rstd_of(row_sum<kRow>(squares(v), nullptr), a);
                if constexpr (negated(kOut)) rstd = -rstd;
#pragma unroll
                for (int i = 0; i < kVec; ++i) weigh<T>(v[i], rstd, weight[i], a.offset);
                emit<T, kOut, kVec, 0>(a, m, live, tid, kRow, v, ts);
            }
        }
    }
}

// Few rows: a CTA of kRow threads each, with up to kVec columns of 8 elements a
// thread, kRow columns apart.  Rows past 16384 elements come here however many
// they are: four columns of 1024 threads, 64 registers each, of which some spill
// (up to 168 bytes, bf16), one CTA an SM and nothing fetched ahead.  They run at
// half of HBM's rate: 1365 x 21504 in 16 bits 37.8 us (3.1 TB/s), with every step
// 79.8, into FP8 41.8 and 83.9; 896 x 32768 34.1 (3.4 TB/s) and 68.3.  Residual and
// norm of 456 x 16384, which walks, 10.6 us, of 457 x 16392 16.8.
template <typename T, int kRow, int kVec, Out kOut>
__global__ void __launch_bounds__(kRow) norm_kernel(const Args a) {
    __shared__ float part[2][32];
    ptx::launch_dependents();
    ptx::grid_dependency_wait();
    const int tid = threadIdx.x;
    const int64_t m = blockIdx.x;
    const int cols = a.K / 8;

    float v[kVec][8];
    uint4 r[kVec];
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
        const int c = tid + i * kRow;
        uint4 w = make_uint4(0, 0, 0, 0);
        r[i] = w;
        if (c < cols) {   // (x and residual may be h: plain loads)
            w = reinterpret_cast<const uint4*>(static_cast<const T*>(a.x) + m * a.x_s)[c];
            if (a.residual) r[i] = reinterpret_cast<const uint4*>(static_cast<const T*>(a.residual) + m * a.r_s)[c];
        }
        unpack8<T>(w, v[i]);
    }
    if (a.residual) {
        if (a.post) {
            const float rstd = rstd_of(row_sum<kRow>(squares(v), part[0]), a);
#pragma unroll
            for (int i = 0; i < kVec; ++i)
                if (tid + i * kRow < cols) weigh<T>(v[i], rstd, column<T>(a.post, 0, tid + i * kRow), a.offset);
        }
        if (a.gate) {
            const int64_t at = static_cast<uint32_t>(m) / a.gate_rows * a.gate_s;
#pragma unroll
            for (int i = 0; i < kVec; ++i)
                if (tid + i * kRow < cols) open<T>(v[i], column<T>(a.gate, at, tid + i * kRow));
        }
#pragma unroll
        for (int i = 0; i < kVec; ++i) {
            const uint4 h = add_residual<T>(v[i], r[i], a);
            if (tid + i * kRow < cols) reinterpret_cast<uint4*>(static_cast<T*>(a.h) + m * a.h_s)[tid + i * kRow] = h;
        }
    }
    if constexpr (kOut != kNone) {
        float rstd = rstd_of(row_sum<kRow>(squares(v), part[1]), a);
        if constexpr (negated(kOut)) rstd = -rstd;
        const TensorScale ts(kOut == kNv4 ? a.tensor_scale : nullptr);
#pragma unroll
        for (int i = 0; i < kVec; ++i)
            if (tid + i * kRow < cols) weigh<T>(v[i], rstd, column<T>(a.weight, 0, tid + i * kRow), a.offset);
        emit<T, kOut, kVec, 0>(a, m, cols, tid, kRow, v, ts);
    }
}

// Many rows of 513 to 16384 elements (by_width): the grid fills the SMs once, and each
// CTA walks over rows, its weights in registers.  Every thread copies its own
// columns of the next rows into shared memory (cp.async, 16 bytes each, read
// back by that thread alone), so that `depth` rows of x, residual and gate are
// under way while one is summed.  Four columns a thread: what a row costs beside
// its elements (two sums over the CTA) falls with fewer warps, and the 14 warps of
// an SM's two CTAs keep HBM busy where nothing is quantised (with two columns and
// twice the warps every step into FP8 took 61.3 us instead of 58.4).  No
// branch stands between a thread's columns (48.7 -> 38.4 us for every step into
// FP8): only its last one may be none, which is zeros then.  kFull: it is none
// nowhere (K a multiple of 256 kVec).  kAlone: without a residual; the registers
// of a second norm's weights go to half as many warps again, which a norm into
// FP8 or 4 bits has work for (4096 x 7168, x in L2, to FP8 19.5 -> 17.6 us, NVFP4
// 25.2 -> 22.9; 80 registers each, of which bf16 spills 8 to 16 bytes).
__device__ __forceinline__ void copy16(uint32_t to, const void* from) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
}
__device__ __forceinline__ uint4 take16(uint32_t from) {
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(from) : "memory");
    return v;
}
// Sum over the CTA's threads (whole warps, up to kMost), in every one of them.
template <int kMost>
__device__ __forceinline__ float block_sum(float s, float* part) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, off);
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = s;
    __syncthreads();
    s = (threadIdx.x & 31) < (blockDim.x >> 5) ? part[threadIdx.x & 31] : 0.0f;
#pragma unroll
    for (int off = kMost > 512 ? 16 : 8; off > 0; off >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, off);
    return kMost > 512 ? s : __shfl_sync(0xFFFFFFFFu, s, 0);
}

template <typename T, int kThreads, int kVec, int kCtas, Out kOut, bool kFull, bool kAlone>
__global__ void __launch_bounds__(kThreads, kCtas) norm_walk_kernel(const Args a) {
    extern __shared__ uint4 ring[];
    __shared__ float part[4][32];
    ptx::launch_dependents();
    ptx::grid_dependency_wait();
    const int tid = threadIdx.x, threads = blockDim.x, cols = a.K / 8;
    const uint32_t ring0 = ptx::smem_u32(ring) + tid * 16;
    const int arrays = kAlone ? 1 : 1 + (a.residual != nullptr) + (a.gate != nullptr);
    const uint32_t array_bytes = kVec * threads * 16, row_bytes = arrays * array_bytes;
    // this thread's columns of a row: tid, tid + threads, ...
    const bool last = kFull || tid + (kVec - 1) * threads < cols;   // whether its last column is one
    auto fetch = [&](int64_t m, uint32_t slot) {
        if (m < a.M) {
            auto row = [&](const void* p, int64_t at, uint32_t to) {
                const T* from = static_cast<const T*>(p) + at + tid * 8;
#pragma unroll
                for (int i = 0; i < kVec; ++i)
                    if (i + 1 < kVec || last) copy16(to + i * threads * 16, from + i * threads * 8);
            };
            row(a.x, m * a.x_s, slot);
            if (!kAlone && a.residual) row(a.residual, m * a.r_s, slot + array_bytes);
            if (!kAlone && a.gate) row(a.gate, (a.gate_rows == 1 ? m : static_cast<uint32_t>(m) / a.gate_rows) * a.gate_s, slot + 2 * array_bytes);
        }
        ptx::cp_async_commit();
    };
    for (int d = 0; d < a.depth; ++d) fetch(blockIdx.x + int64_t(d) * gridDim.x, ring0 + d * row_bytes);
    uint4 weight[kVec], post[kVec];
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
        const int c = tid + i * threads;
        weight[i] = post[i] = make_uint4(0, 0, 0, 0);
        if (kOut != kNone && (i + 1 < kVec || last)) weight[i] = column<T>(a.weight, 0, c);
        if (!kAlone && a.post && (i + 1 < kVec || last)) post[i] = column<T>(a.post, 0, c);
    }
    const TensorScale ts(kOut == kNv4 ? a.tensor_scale : nullptr);
    int d = 0, turn = 0;
    for (int64_t m = blockIdx.x; m < a.M; m += gridDim.x, turn ^= 1) {
        ptx::cp_async_wait_pending(a.depth - 1);
        const uint32_t slot = ring0 + d * row_bytes;
        // this thread's column i of an array (zeros where it has none)
        auto taken = [&](uint32_t array, int i) {
            uint4 x = make_uint4(0, 0, 0, 0);
            if (i + 1 < kVec || last) x = take16(array + i * threads * 16);
            return x;
        };
        float v[kVec][8];
#pragma unroll
        for (int i = 0; i < kVec; ++i) unpack8<T>(taken(slot, i), v[i]);
        // (a row's first sum is met by all before the next row's is written: two sums take turns where there is no other)
        if (!kAlone && a.residual) {
            if (a.post) {
                const float rstd = rstd_of(block_sum<kThreads>(squares(v), part[2 * turn]), a);
#pragma unroll
                for (int i = 0; i < kVec; ++i) weigh<T>(v[i], rstd, post[i], a.offset);
            }
            if (a.gate) {
#pragma unroll
                for (int i = 0; i < kVec; ++i) open<T>(v[i], taken(slot + 2 * array_bytes, i));
            }
#pragma unroll
            for (int i = 0; i < kVec; ++i) {
                const uint4 h = add_residual<T>(v[i], taken(slot + array_bytes, i), a);
                if (i + 1 < kVec || last) reinterpret_cast<uint4*>(static_cast<T*>(a.h) + m * a.h_s)[tid + i * threads] = h;
            }
        }
        float rstd = 0.0f;
        if constexpr (kOut != kNone) rstd = rstd_of(block_sum<kThreads>(squares(v), part[2 * turn + 1]), a);
        fetch(m + int64_t(a.depth) * gridDim.x, slot);   // (what was in the slot has been used)
        if (++d == a.depth) d = 0;
        if constexpr (kOut != kNone) {
            if constexpr (negated(kOut)) rstd = -rstd;
#pragma unroll
            for (int i = 0; i < kVec; ++i) weigh<T>(v[i], rstd, weight[i], a.offset);
            emit<T, kOut, kVec, kFull ? kVec : kVec - 1>(a, m, cols, tid, threads, v, ts);
        }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
}

template <typename T, int kThreads, int kVec, int kCtas, Out kOut, bool kFull, bool kAlone>
sgq_status walk(Args a, int sms, cudaStream_t st) {
    const int cols = a.K / 8, threads = (cols + 32 * kVec - 1) / (32 * kVec) * 32;
    const int ctas = kThreads * kCtas / threads, share = 208 * 1024 / ctas;
    const int row_bytes = (1 + (a.residual != nullptr) + (a.gate != nullptr)) * kVec * threads * 16;
    a.depth = share / row_bytes < 4 ? share / row_bytes : 4;
    auto kern = norm_walk_kernel<T, kThreads, kVec, kCtas, kOut, kFull, kAlone>;
    static bool configured[64] = {};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return SGQ_ERR_CUDA;
    if (!configured[dev]) {
        if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, 208 * 1024) != cudaSuccess) return SGQ_ERR_CUDA;
        configured[dev] = true;
    }
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(sms * ctas));
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = static_cast<size_t>(a.depth) * row_bytes;
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, kern, a) != cudaSuccess) return SGQ_ERR_CUDA;
    note_launch();
    return SGQ_OK;
}

template <typename T, int kThreads, int kVec, int kCtas, Out kOut, bool kAlone>
sgq_status walk_rows(const Args& a, int sms, cudaStream_t st) {
    return a.K % (256 * kVec) == 0 ? walk<T, kThreads, kVec, kCtas, kOut, true, kAlone>(a, sms, st)
                                   : walk<T, kThreads, kVec, kCtas, kOut, false, kAlone>(a, sms, st);
}

template <typename T, int kRow, int kVec, Out kOut>
sgq_status run(const Args& a, cudaStream_t st) {
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(a.M));
    cfg.blockDim = dim3(kRow);
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, norm_kernel<T, kRow, kVec, kOut>, a) != cudaSuccess) return SGQ_ERR_CUDA;
    note_launch();
    return SGQ_OK;
}
template <typename T, int kRow, int kVec, int kN, Out kOut>
sgq_status narrow(const Args& a, int sms, cudaStream_t st) {
    // rows that all fit at once: one step of one row for each warp
    if (kN > 1 && a.M <= int64_t(sms) * 16 * (32 / kRow)) return narrow<T, kRow, kVec, 1, kOut>(a, sms, st);
    auto kern = norm_rows_kernel<T, kRow, kVec, kN, kOut>;
    static Resident resident;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return SGQ_ERR_CUDA;
    const int fit = resident.on(dev, [&] {   // CTAs an SM
        int n = 0;
        return cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kern, 128, 0) == cudaSuccess ? n : 0;
    });
    if (fit <= 0) return SGQ_ERR_CUDA;
    const int64_t rows = 4 * (32 / kRow) * kN, want = (a.M + rows - 1) / rows, most = int64_t(sms) * fit;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(want < most ? want : most));
    cfg.blockDim = dim3(128);
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, kern, a) != cudaSuccess) return SGQ_ERR_CUDA;
    note_launch();
    return SGQ_OK;
}
template <typename T, Out kOut>
sgq_status by_width(const Args& a, int sms, cudaStream_t st) {
    // CTAs walk where there are more rows than CTAs of norm_kernel at once, 1024 threads an SM; 513 to 2048 elements, where
    // the rows are more than L2 holds (a norm / residual and norm / every step into FP8 in a graph, us, a row each ->
    // walking: 456 x 5120 3.9 / 4.5 / 7.3 -> 3.1 / 3.6 / 4.6, 1024 x 4096 4.5 / 5.3 / 7.8 -> 4.1 / 5.3 / 7.6, 1024 x 7168
    // 7.1 / 8.5 / 13.3 -> 5.7 / 8.0 / 12.3, 456 x 16384 7.2 / 8.8 / 13.3 -> 5.7 / 8.1 / 10.7; but 304 x 7168 2.8 / 3.2 / 4.5
    // -> 3.0 / 3.5 / 4.7, 2432 x 2048 4.6 / 5.5 / 8.0 -> 4.7 / 6.0 / 9.6).
    const int64_t wave = int64_t(sms) * (a.K <= 4096 ? 4 : a.K <= 8192 ? 2 : 1);
    const bool many = a.K > 2048 ? a.K <= 16384 && a.M > wave : a.K > 512 && a.M * a.K > (int64_t(10) << 20);
    // (four columns a thread leave only the last one without some threads' part from 288 columns on)
    const bool four = a.K >= 288 * 8;
    if constexpr (negated(kOut)) {
        if (many && !a.residual && a.K <= 12288 && (four || a.K % 1024 == 0))
            return a.K <= 8192 ? walk_rows<T, 256, 4, 3, kOut, true>(a, sms, st) : walk_rows<T, 384, 4, 2, kOut, true>(a, sms, st);
    }
    if (many && !four) return walk_rows<T, 192, 2, 4, kOut, false>(a, sms, st);
    if (many && a.K <= 8192) return walk_rows<T, 256, 4, 2, kOut, false>(a, sms, st);
    // (9216 to 12288: two columns keep 18 to 24 warps busy, four 9 to 12; norm, residual, norm into NVFP4 of 3255 x 9216 45.7 -> 39.7 us)
    if (many && a.K <= 12288) return walk_rows<T, 768, 2, 1, kOut, false>(a, sms, st);
    if (many) return walk_rows<T, 512, 4, 1, kOut, false>(a, sms, st);
    if (a.K <= 128) return narrow<T, 16, 1, 4, kOut>(a, sms, st);
    if (a.K <= 256) return narrow<T, 32, 1, 4, kOut>(a, sms, st);
    if (a.K <= 512) return narrow<T, 32, 2, 2, kOut>(a, sms, st);
    if (a.K <= 1024) return run<T, 64, 2, kOut>(a, st);
    if (a.K <= 2048) return run<T, 128, 2, kOut>(a, st);
    if (a.K <= 4096) return run<T, 256, 2, kOut>(a, st);
    if (a.K <= 8192) return run<T, 512, 2, kOut>(a, st);
    if (a.K <= 16384) return run<T, 1024, 2, kOut>(a, st);
    return run<T, 1024, 4, kOut>(a, st);
}
template <typename T>
sgq_status by_out(const Args& a, Out out, int sms, cudaStream_t st) {
    switch (out) {
        case kNone: return by_width<T, kNone>(a, sms, st);
        case kSame: return by_width<T, kSame>(a, sms, st);
        case kFp8: return by_width<T, kFp8>(a, sms, st);
        case kMx4: return by_width<T, kMx4>(a, sms, st);
        case kNv4: return by_width<T, kNv4>(a, sms, st);
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
    a.gate_rows = static_cast<uint32_t>(n.gate_rows < n.M ? n.gate_rows : n.M); a.K = static_cast<int>(n.K);
    a.inv_k = 1.0f / static_cast<float>(n.K);
    a.eps = n.eps; a.offset = n.offset; a.scale = n.scale; a.residual_scale = n.residual_scale;
    Out out = kNone;
    switch (n.out) {
        case SGQ_OUT_NONE: break;
        case SGQ_OUT_16: out = kSame; break;
        case SGQ_OUT_MXFP4: out = kMx4; break;
        case SGQ_OUT_NVFP4: out = kNv4; break;
        default:
            out = kFp8;
            a.group_shift = n.out & SGQ_OUT_GROUP_128 ? 4 : 2;
            a.scale_kind = (n.out & SGQ_OUT_UE8M0) != 0 ? 2 : (n.out & SGQ_OUT_POW2) != 0 ? 1 : 0;
    }
    return n.dtype == SGQ_BF16 ? by_out<__nv_bfloat16>(a, out, di.sm_count, st) : by_out<__half>(a, out, di.sm_count, st);
}

}  // namespace sgq
