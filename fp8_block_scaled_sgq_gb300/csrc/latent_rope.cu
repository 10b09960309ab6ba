// Rotary positions and the append to a paged latent cache, for sm_103a.
//
// Rotation.  With (c, s) = table[pos][i], the cosine and sine of pair i's
// angle, pair i of a head's rotated part becomes
//     (a, b) -> (a c - b s, b c + a s)        inverse: s -> -s
// where pair i is elements (2i, 2i + 1) (interleaved) or (i, i + R/2) (half).
// The inverse is the transpose, i.e. the gradient (and the way back where the
// table's pairs have length 1).  The arithmetic is fp32 with one rounding on the
// way out.
//
// Both kernels are bound by HBM: every element is read and written once, and
// the table's rows (4 R bytes a token) are small beside a token's heads.  A
// thread keeps one 16-byte column of a row (half layout: the two columns that
// a pair spans, so that rotating in place has no race) and walks over heads,
// so its cosines and sines are loaded once for all of them.  Its first heads
// are on their way before it asks for the position, whose table row is two
// dependent loads away.  Four blocks an SM (a register bound of 64) keep
// enough of them in flight: 4096 x 128 x 192 fp16 (403 MB) in 70.0 us against
// 80.8 us without the bound, and 60.4 us at the measured copy rate; appending
// 4099 tokens of 128 heads (145 MB) in 23.9 us against 21.7 us.
#include <cuda_runtime.h>

#include "latent_common.cuh"
#include "ptx.cuh"
#include "sgq_internal.h"

namespace sgq {
namespace {

using lat::Pair;

constexpr int kThreads = 256;
constexpr int kHeadsInFlight = 4;   // independent 16-byte loads a thread keeps in flight

// cos/sin of the pairs that one unit (8 or 2 x 8 elements) rotates.
struct Turn {
    float c[8], s[8];
};
template <bool kInter>
__device__ __forceinline__ void load_turn(Turn& t, const float* __restrict__ row, int R, int unit, bool inverse) {
    constexpr int kPairs = kInter ? 4 : 8;
    const float4* c = reinterpret_cast<const float4*>(row + unit * kPairs);
    const float4* s = reinterpret_cast<const float4*>(row + R / 2 + unit * kPairs);
#pragma unroll
    for (int i = 0; i < kPairs / 4; ++i) {
        const float4 a = __ldg(c + i), b = __ldg(s + i);
        t.c[4 * i] = a.x; t.c[4 * i + 1] = a.y; t.c[4 * i + 2] = a.z; t.c[4 * i + 3] = a.w;
        t.s[4 * i] = b.x; t.s[4 * i + 1] = b.y; t.s[4 * i + 2] = b.z; t.s[4 * i + 3] = b.w;
    }
    if (inverse) {
#pragma unroll
        for (int i = 0; i < kPairs; ++i) t.s[i] = -t.s[i];
    }
}
__device__ __forceinline__ float2 turn(float a, float b, float c, float s) {
    return make_float2(fmaf(a, c, -b * s), fmaf(b, c, a * s));
}
template <typename T>
__device__ __forceinline__ uint4 rotate_inter(const uint4& v, const Turn& t) {
    uint4 r;
    const uint32_t* in = &v.x;
    uint32_t* out = &r.x;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 p = Pair<T>::unpack(in[i]);
        const float2 o = turn(p.x, p.y, t.c[i], t.s[i]);
        out[i] = Pair<T>::pack(o.x, o.y);
    }
    return r;
}
template <typename T>
__device__ __forceinline__ void rotate_half(uint4& lo, uint4& hi, const Turn& t) {
    uint32_t* a = &lo.x;
    uint32_t* b = &hi.x;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 p = Pair<T>::unpack(a[i]), q = Pair<T>::unpack(b[i]);
        const float2 x = turn(p.x, q.x, t.c[2 * i], t.s[2 * i]);
        const float2 y = turn(p.y, q.y, t.c[2 * i + 1], t.s[2 * i + 1]);
        a[i] = Pair<T>::pack(x.x, y.x);
        b[i] = Pair<T>::pack(x.y, y.y);
    }
}

// The table row of a token; a position outside the table is reported and
// clamped, so that nothing outside it is read.
__device__ __forceinline__ const float* table_row(const float* table, const int64_t* pos, int64_t t, int64_t max_pos,
                                                  int R, uint32_t* status) {
    int64_t p = __ldg(pos + t);
    if (p < 0 || p >= max_pos) {
        atomicOr(status, kStatusBadValue);
        p = p < 0 ? 0 : max_pos - 1;
    }
    return table + p * R;
}

struct HeadsArgs {
    const char* x;          // [T, H, .], byte strides
    char* y;
    int64_t x_t, x_h, y_t, y_h;
    int H, heads_per_block;
    int rot_lo, rot_units;  // first rotated unit of a row, number of rotated units
    int units, lanes;       // units a row: copied columns and rotated units; heads side by side
    int half_bytes;         // half layout: distance of a pair's two columns
    int inverse;
};

// One token's heads [h0, h0 + heads_per_block): thread (unit, head lane).
// Units are 16-byte columns in row order, a rotated unit of the half layout
// being the column of a pair's first elements and the one half_bytes further.
template <typename T, bool kInter>
__device__ __forceinline__ void rotate_heads(const HeadsArgs& a, const int64_t* pos, const float* table, int64_t max_pos,
                                             int R, uint32_t* status, int64_t t, int h0) {
    const int unit = threadIdx.x % a.units, hl = threadIdx.x / a.units;
    if (hl >= a.lanes) return;
    const bool rot = unit >= a.rot_lo && unit < a.rot_lo + a.rot_units;
    const int col = unit < a.rot_lo + a.rot_units ? unit * 16 : unit * 16 + (kInter ? 0 : a.half_bytes);
    const char* xp = a.x + t * a.x_t + col;
    char* yp = a.y + t * a.y_t + col;
    const int h1 = min(a.H, h0 + a.heads_per_block);
    uint4 v[kHeadsInFlight], w[kHeadsInFlight];
    auto fetch = [&](int h) {
#pragma unroll
        for (int i = 0; i < kHeadsInFlight; ++i) {
            const int hh = h + i * a.lanes;
            if (hh < h1) {
                v[i] = *reinterpret_cast<const uint4*>(xp + hh * a.x_h);
                if (!kInter && rot) w[i] = *reinterpret_cast<const uint4*>(xp + hh * a.x_h + a.half_bytes);
            }
        }
    };
    fetch(h0 + hl);
    Turn tn;
    if (rot) load_turn<kInter>(tn, table_row(table, pos, t, max_pos, R, status), R, unit - a.rot_lo, a.inverse != 0);
    for (int h = h0 + hl; h < h1; h += a.lanes * kHeadsInFlight) {
        if (h != h0 + hl) fetch(h);
#pragma unroll
        for (int i = 0; i < kHeadsInFlight; ++i) {
            const int hh = h + i * a.lanes;
            if (hh < h1) {
                if (rot) {
                    if constexpr (kInter) v[i] = rotate_inter<T>(v[i], tn);
                    else rotate_half<T>(v[i], w[i], tn);
                }
                *reinterpret_cast<uint4*>(yp + hh * a.y_h) = v[i];
                if (!kInter && rot) *reinterpret_cast<uint4*>(yp + hh * a.y_h + a.half_bytes) = w[i];
            }
        }
    }
}

template <typename T, bool kInter>
__global__ void __launch_bounds__(kThreads, 4) rotary_kernel(const HeadsArgs a, const int64_t* __restrict__ pos,
                                                          const float* __restrict__ table, int64_t max_pos, int R,
                                                          int blocks_per_token, uint32_t* status) {
    ptx::launch_dependents();
    ptx::grid_dependency_wait();
    const int64_t t = blockIdx.x / blocks_per_token;
    const int h0 = static_cast<int>(blockIdx.x % blocks_per_token) * a.heads_per_block;
    rotate_heads<T, kInter>(a, pos, table, max_pos, R, status, t, h0);
}

struct AppendArgs {
    HeadsArgs q;            // the rotated parts of the queries (H == 0: none)
    const char* k;          // [T, R]
    const char* latent;     // [T, L]
    char* k_out;            // [T, R] or null
    char* cache;            // [pages, page, L + R]
    int64_t k_t, l_t, ko_t, c_page, c_row;   // byte strides
    const int64_t* slots;
    int64_t T, slots_max;
    int page, q_blocks, L;
};

// Blocks [0, T * q_blocks) rotate the queries; every further block writes
// cache rows, a warp a token.
template <typename T, bool kInter>
__global__ void __launch_bounds__(kThreads, 4) latent_append_kernel(const AppendArgs a, const int64_t* __restrict__ pos,
                                                                 const float* __restrict__ table, int64_t max_pos,
                                                                 int R, uint32_t* status) {
    ptx::launch_dependents();
    ptx::grid_dependency_wait();
    const int64_t qb = a.T * a.q_blocks;
    if (blockIdx.x < qb) {
        const int64_t t = blockIdx.x / a.q_blocks;
        const int h0 = static_cast<int>(blockIdx.x % a.q_blocks) * a.q.heads_per_block;
        rotate_heads<T, kInter>(a.q, pos, table, max_pos, R, status, t, h0);
        return;
    }
    const int64_t t = (blockIdx.x - qb) * (blockDim.x >> 5) + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    if (t >= a.T) return;
    const int64_t slot = __ldg(a.slots + t);
    char* row = nullptr;
    if (slot >= 0 && slot < a.slots_max) row = a.cache + (slot / a.page) * a.c_page + (slot % a.page) * a.c_row;
    else if (slot >= a.slots_max && lane == 0) atomicOr(status, kStatusBadValue);
    if (row == nullptr && a.k_out == nullptr) return;
    if (row != nullptr) {
        const char* lp = a.latent + t * a.l_t;
        for (int c = lane; c < a.L / 8; c += 32)
            *reinterpret_cast<uint4*>(row + c * 16) = __ldg(reinterpret_cast<const uint4*>(lp + c * 16));
    }
    const int units = kInter ? R / 8 : R / 16;
    if (lane >= units) return;
    const float* trow = table_row(table, pos, t, max_pos, R, status);
    Turn tn;
    load_turn<kInter>(tn, trow, R, lane, false);
    const char* kp = a.k + t * a.k_t + lane * 16;
    uint4 v = *reinterpret_cast<const uint4*>(kp), w = make_uint4(0, 0, 0, 0);
    if constexpr (kInter) {
        v = rotate_inter<T>(v, tn);
    } else {
        w = *reinterpret_cast<const uint4*>(kp + R);
        rotate_half<T>(v, w, tn);
    }
    auto store = [&](char* dst) {
        *reinterpret_cast<uint4*>(dst + lane * 16) = v;
        if (!kInter) *reinterpret_cast<uint4*>(dst + lane * 16 + R) = w;
    };
    if (row != nullptr) store(row + 2 * a.L);
    if (a.k_out != nullptr) store(a.k_out + t * a.ko_t);
}

// Geometry of a head walk over `cols` 16-byte columns, R rotated elements
// from element `offset` on.  A block takes kHeadsInFlight heads a thread.
void plan_heads(HeadsArgs& h, int64_t H, int64_t cols, int R, int64_t offset, bool inter) {
    h.H = static_cast<int>(H);
    h.rot_lo = static_cast<int>(offset / 8);
    h.rot_units = inter ? R / 8 : R / 16;
    h.units = static_cast<int>(cols) - (inter ? 0 : R / 16);
    h.half_bytes = R;   // R / 2 elements of 2 bytes
    // As many heads side by side as leave every thread its loads in flight.
    const int most = kThreads / h.units, want = static_cast<int>((H + kHeadsInFlight - 1) / kHeadsInFlight);
    h.lanes = want < 1 ? 1 : want < most ? want : most;
    h.heads_per_block = h.lanes * kHeadsInFlight;
}

template <typename... Args, typename... Act>
sgq_status launch(void (*kern)(Args...), int64_t blocks, int threads, cudaStream_t st, Act... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(blocks));
    cfg.blockDim = dim3(static_cast<unsigned>(threads));
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, kern, args...) != cudaSuccess) return SGQ_ERR_CUDA;
    note_launch();
    return SGQ_OK;
}

}  // namespace

sgq_status launch_rotary(const void* x, int64_t T, int64_t H, int64_t D, int64_t x_t, int64_t x_h, const int64_t* pos,
                         const float* table, int64_t max_pos, int R, int64_t offset, int inter, int inverse, int dtype,
                         void* y, int64_t y_t, int64_t y_h, cudaStream_t st) {
    uint32_t* status = nullptr;
    const sgq_status rc = gemm::status_word(&status);
    if (rc != SGQ_OK) return rc;
    HeadsArgs h{};
    // In place the columns outside the rotated part stay as they are.
    const bool in_place = x == y;
    const int64_t skip = in_place ? offset : 0;
    h.x = static_cast<const char*>(x) + 2 * skip;
    h.y = static_cast<char*>(y) + 2 * skip;
    h.x_t = 2 * x_t; h.x_h = 2 * x_h; h.y_t = 2 * y_t; h.y_h = 2 * y_h;
    h.inverse = inverse;
    plan_heads(h, H, (in_place ? R : D) / 8, R, offset - skip, inter != 0);
    const int bpt = static_cast<int>((H + h.heads_per_block - 1) / h.heads_per_block);
    if (T * bpt > INT32_MAX) return SGQ_ERR_INVALID_ARG;
    auto kern = dtype == SGQ_BF16 ? (inter ? rotary_kernel<__nv_bfloat16, true> : rotary_kernel<__nv_bfloat16, false>)
                                  : (inter ? rotary_kernel<__half, true> : rotary_kernel<__half, false>);
    return launch(kern, T * bpt, (h.units * h.lanes + 31) / 32 * 32, st, h, pos, table, max_pos, R, bpt, status);
}

sgq_status launch_latent_append(const void* q, int64_t q_t, int64_t q_h, const void* k, int64_t k_t, const void* latent,
                                int64_t l_t, const int64_t* pos, const int64_t* slots, const float* table,
                                int64_t max_pos, int64_t T, int64_t H, int64_t L, int R, int inter, int dtype,
                                void* q_out, int64_t qo_t, int64_t qo_h, void* k_out, int64_t ko_t, void* cache,
                                int64_t pages, int64_t page, int64_t c_page, int64_t c_row, cudaStream_t st) {
    uint32_t* status = nullptr;
    const sgq_status rc = gemm::status_word(&status);
    if (rc != SGQ_OK) return rc;
    AppendArgs a{};
    a.q.x = static_cast<const char*>(q);
    a.q.y = static_cast<char*>(q_out);
    a.q.x_t = 2 * q_t; a.q.x_h = 2 * q_h; a.q.y_t = 2 * qo_t; a.q.y_h = 2 * qo_h;
    plan_heads(a.q, H, R / 8, R, 0, inter != 0);
    a.q_blocks = static_cast<int>((H + a.q.heads_per_block - 1) / a.q.heads_per_block);
    a.k = static_cast<const char*>(k);
    a.latent = static_cast<const char*>(latent);
    a.k_out = static_cast<char*>(k_out);
    a.cache = static_cast<char*>(cache);
    a.k_t = 2 * k_t; a.l_t = 2 * l_t; a.ko_t = 2 * ko_t; a.c_page = 2 * c_page; a.c_row = 2 * c_row;
    a.slots = slots;
    a.T = T;
    a.slots_max = pages * page;
    a.page = static_cast<int>(page);
    a.L = static_cast<int>(L);
    const int threads = H > 0 ? (a.q.units * a.q.lanes + 31) / 32 * 32 : kThreads, tokens = threads / 32;
    const int64_t blocks = T * a.q_blocks + (T + tokens - 1) / tokens;
    if (blocks > INT32_MAX) return SGQ_ERR_INVALID_ARG;
    auto kern = dtype == SGQ_BF16
                    ? (inter ? latent_append_kernel<__nv_bfloat16, true> : latent_append_kernel<__nv_bfloat16, false>)
                    : (inter ? latent_append_kernel<__half, true> : latent_append_kernel<__half, false>);
    return launch(kern, blocks, threads, st, a, pos, table, max_pos, R, status);
}

}  // namespace sgq
