// Block-scaled 4-bit GEMM for sm_103a: D = a w (Aq * As)(Wq * Ws)^T, E2M1
// operands with a scale every 16 (E4M3) or 32 (UE8M0) values along K, fp32
// accumulation, 16-bit output.  The form of the operands is in fp4_common.cuh.
#include <cuda.h>
#include <cuda_runtime.h>

#include "fp4_common.cuh"
#include "latent_ptx.cuh"
#include "ptx.cuh"
#include "sgq_internal.h"

namespace sgq {
namespace {

using namespace fp4;

constexpr int kRows = 128;        // rows of the MMA's M side
constexpr int kStageK = 256;      // elements of K a stage: one 128-byte swizzle row of codes
constexpr int kMmaK = 64;         // elements of K an MMA
constexpr int kRowBytes = kStageK / 2;

struct Args {
    void* D;
    const float *a_t, *w_t;   // tensor scales, or null for 1
    uint32_t* status;
    int M, N, K;
    int stages;      // K in stages
    int tiles_c;     // token tiles
    int tiles_n, tiles;   // pairs: weight tiles, and all tiles
    bool stream_out;      // pairs: D is large
    int splits;
    int ring;        // stages in shared memory
};

// kStall (SGQ_FP4_TEST_TIMEOUT): the first CTA never loads the second stage's
// weights, and waits run out early.
template <bool kStall>
using SyncOf = lat::Sync<kStall ? lat::kTestTimeoutClocks : lat::kTimeoutClocks>;

// Bytes of one row block's scales a stage (128 rows x 256 values).
constexpr int sf_bytes(bool nv) { return nv ? 2048 : 1024; }

// Instruction descriptor of kind::mxf4nvf4: E2M1 operands, both K-major, one
// scale word a row (UE8M0 or E4M3); the words' halves are chosen per MMA.
__host__ __device__ constexpr uint32_t idesc_fp4(uint32_t M, uint32_t N, bool nv) {
    return (1u << 7) | (1u << 10) | ((N >> 3) << 17) | ((nv ? 0u : 1u) << 23) | ((M >> 4) << 24);
}
__device__ __forceinline__ uint32_t elect() {
    uint32_t r;
    asm volatile("{\n.reg .pred e;\nelect.sync _|e, 0xffffffff;\nselp.u32 %0, 1, 0, e;\n}" : "=r"(r));
    return r;
}
// A stage's issue in two blocks of instructions for the elected lane of a
// converged warp.  An MMA of 256 x 192 x 64 lasts 50 ns; with addresses formed
// and predicates set anew for each, the warp took 66 ns to issue one.
//
// Scales of one row block (kTiles tiles of 128 rows x 4 groups, 512 bytes
// each) into TMEM, kStep columns apart.
#define SGQ_FP4_CP(CG)                                                                                            \
    "{\n.reg .pred e;\n.reg .b32 t1, t2, t3;\n.reg .b64 s1, s2, s3;\nelect.sync _|e, 0xffffffff;\n"             \
    "add.u32 t1, %0, %2;\nadd.u32 t2, %0, %3;\nadd.u32 t3, %0, %4;\n"                                             \
    "add.s64 s1, %1, 32;\nadd.s64 s2, %1, 64;\nadd.s64 s3, %1, 96;\n"                                             \
    "@e tcgen05.cp.cta_group::" CG ".32x128b.warpx4 [%0], %1;\n@e tcgen05.cp.cta_group::" CG ".32x128b.warpx4 [t1], s1;\n"
#define SGQ_FP4_CP2(CG) \
    "@e tcgen05.cp.cta_group::" CG ".32x128b.warpx4 [t2], s2;\n@e tcgen05.cp.cta_group::" CG ".32x128b.warpx4 [t3], s3;\n"
template <int CG, bool kNv, int kStep>
__device__ __forceinline__ void copy_scales(uint32_t t, uint64_t s) {
    if constexpr (CG == 1 && kNv)
        asm volatile(SGQ_FP4_CP("1") SGQ_FP4_CP2("1") "}" ::"r"(t), "l"(s), "n"(kStep), "n"(2 * kStep), "n"(3 * kStep) : "memory");
    else if constexpr (CG == 1)
        asm volatile(SGQ_FP4_CP("1") "}" ::"r"(t), "l"(s), "n"(kStep), "n"(2 * kStep), "n"(3 * kStep) : "memory");
    else if constexpr (kNv)
        asm volatile(SGQ_FP4_CP("2") SGQ_FP4_CP2("2") "}" ::"r"(t), "l"(s), "n"(kStep), "n"(2 * kStep), "n"(3 * kStep) : "memory");
    else
        asm volatile(SGQ_FP4_CP("2") "}" ::"r"(t), "l"(s), "n"(kStep), "n"(2 * kStep), "n"(3 * kStep) : "memory");
}
#undef SGQ_FP4_CP
#undef SGQ_FP4_CP2
// A stage's MMAs (n of four; the first one starts the sum over where acc == 0):
// operands 32 bytes further along K each; with two scales an MMA (MXFP4) a
// word of four serves two MMAs, its halves chosen in the instruction descriptor.
#define SGQ_FP4_MMA(CG, VEC)                                                                                       \
    "{\n.reg .pred e, q, t, f;\n.reg .b32 x1, x2, x3, y1, y2, y3;\n.reg .b64 a1, a2, a3, b1, b2, b3;\n"          \
    "elect.sync _|e, 0xffffffff;\nsetp.ne.b32 q, %6, 0;\nsetp.eq.u32 t, %0, %0;\n"                                 \
    "add.s64 a1, %1, 2;\nadd.s64 a2, %1, 4;\nadd.s64 a3, %1, 6;\nadd.s64 b1, %2, 2;\nadd.s64 b2, %2, 4;\nadd.s64 b3, %2, 6;\n" \
    "add.u32 x1, %4, %9;\nadd.u32 x2, %4, %10;\nadd.u32 x3, %4, %11;\nadd.u32 y1, %5, %12;\nadd.u32 y2, %5, %13;\nadd.u32 y3, %5, %14;\n" \
    "@e tcgen05.mma.cta_group::" CG ".kind::mxf4nvf4.block_scale.scale_vec::" VEC " [%0], %1, %2, %3, [%4], [%5], q;\n" \
    "setp.gt.and.u32 f, %8, 1, e;\n"                                                                              \
    "@f tcgen05.mma.cta_group::" CG ".kind::mxf4nvf4.block_scale.scale_vec::" VEC " [%0], a1, b1, %7, [x1], [y1], t;\n" \
    "setp.gt.and.u32 f, %8, 2, e;\n"                                                                              \
    "@f tcgen05.mma.cta_group::" CG ".kind::mxf4nvf4.block_scale.scale_vec::" VEC " [%0], a2, b2, %3, [x2], [y2], t;\n" \
    "setp.gt.and.u32 f, %8, 3, e;\n"                                                                              \
    "@f tcgen05.mma.cta_group::" CG ".kind::mxf4nvf4.block_scale.scale_vec::" VEC " [%0], a3, b3, %7, [x3], [y3], t;\n}"
template <int CG, bool kNv, int kStepA, int kStepB>
__device__ __forceinline__ void mma_stage(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sfa, uint32_t sfb,
                                          uint32_t acc, uint32_t n) {
    constexpr int A1 = kNv ? kStepA : 0, A2 = kNv ? 2 * kStepA : kStepA, A3 = kNv ? 3 * kStepA : kStepA;
    constexpr int B1 = kNv ? kStepB : 0, B2 = kNv ? 2 * kStepB : kStepB, B3 = kNv ? 3 * kStepB : kStepB;
    const uint32_t second = kNv ? idesc : ptx::idesc_sf_ids(idesc, 2, 2);
#define SGQ_FP4_OPS                                                                                                      \
    "r"(d), "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(acc), "r"(second), "r"(n), "n"(A1), "n"(A2), "n"(A3), "n"(B1), \
        "n"(B2), "n"(B3)
    if constexpr (CG == 1 && kNv) asm volatile(SGQ_FP4_MMA("1", "4X")::SGQ_FP4_OPS : "memory");
    else if constexpr (CG == 1) asm volatile(SGQ_FP4_MMA("1", "2X")::SGQ_FP4_OPS : "memory");
    else if constexpr (kNv) asm volatile(SGQ_FP4_MMA("2", "4X")::SGQ_FP4_OPS : "memory");
    else asm volatile(SGQ_FP4_MMA("2", "2X")::SGQ_FP4_OPS : "memory");
#undef SGQ_FP4_OPS
}
#undef SGQ_FP4_MMA

// 16 bytes to a shared-memory address of the cluster.
__device__ __forceinline__ void st_cluster_v4(uint32_t at, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    asm volatile("st.shared::cluster.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}
// Both tensor scales, as the factors that a sum is multiplied by, first and then
// second: their product and 1; or, where their product is no normal fp32
// number, the larger one and the smaller one, since what they make of the sum
// may be one all the same.  (MXFP4 has none.)
template <bool kNv>
struct Scales {
    float first = 1.0f, second = 1.0f;
    __device__ __forceinline__ explicit Scales(const Args& a) {
        if constexpr (kNv) {
            const float x = a.a_t ? __ldg(a.a_t) : 1.0f, w = a.w_t ? __ldg(a.w_t) : 1.0f, xw = x * w;
            const bool normal = fabsf(xw) >= 0x1p-126f && fabsf(xw) <= 0x1.fffffep127f, larger = fabsf(x) >= fabsf(w);
            first = normal ? xw : larger ? x : w;
            second = normal ? 1.0f : larger ? w : x;
        }
    }
    __device__ __forceinline__ float2 scaled(float u, float v) const {
        if constexpr (!kNv) return make_float2(u, v);
        return lat::mul2(lat::mul2(make_float2(u, v), make_float2(first, first)), make_float2(second, second));
    }
};

// ---------------------------------------------------------------- weights on the 128-row side
//
// One tile of 128 weight rows x BN tokens a cluster; the cluster's CTAs take
// equal parts of K and sum their accumulators through each other's shared
// memory in the order of the parts, each for its share of the tokens.
//
// Bound by latency: the first load, a stage every 0.31 us (the issuing warp's
// wait, scale copies and MMAs), and where K is split 1.3 us (64 tokens) to 3 (128)
// for the sum.  A CTA that has an SM to itself takes all of its shared memory for
// stages under way: weights at HBM's rate need some 60 KB an SM in flight (64
// tokens x 7168 x 7168: 13.7 us with 3 stages, 10.1 with 7).  Measured in a
// graph, other weights for each call, so that they come from HBM: 1 x 7168 x 2048
// NVFP4 4.8 us (1.7 TB/s), 64 x 7168 x 7168 NVFP4 9.9 (3.0), 64 x 24576 x 1536
// MXFP4 7.0 (3.3), 301 x 1536 x 7168 NVFP4 9.1.  With the same weights in L2: 3.9,
// 5.5 for 64 x 24576 x 1536, and 8.7.
//
// Warps: 0 loads (TMA), 1 issues, 2-5 read the accumulator (a TMEM lane
// quarter each).
constexpr int kTileThreads = 192;

template <int BN, bool kNv>
struct TileCfg {
    static constexpr int kSf = sf_bytes(kNv);
    static constexpr int kStageBytes = kRows * kRowBytes + BN * kRowBytes + 2 * kSf;
    static constexpr int kSfCols = kNv ? 16 : 8;                    // TMEM columns of one operand's scales a stage
    static constexpr uint32_t kSfAt = BN < 32 ? 32 : BN;            // after the accumulator; two stages' worth
    static constexpr uint32_t kTmem = kSfAt + 4 * kSfCols <= 128 ? 128 : 256;
    static_assert(kSfAt + 4 * kSfCols <= kTmem, "TMEM");
    static constexpr int kMaxRing = 12;
    static constexpr int kHead = 1024;                              // barriers and words, before the ring
    // At least the share of an SM's shared memory that the CTA takes of its
    // TMEM, so that CTAs of this file which fit together never wait for each
    // other's TMEM; and more than half of it for a CTA that waits for others (a
    // split tile's), so that no CTA of another cluster fits beside it: two clusters
    // that each hold the TMEM that the other's CTA waits for would never end.  (All
    // clusters of the library that hold TMEM take more than 111 KB a CTA, here and
    // in the FP8 GEMMs.  What does fit is a tile of 16 to 64 tokens without splits,
    // 57 KB and 128 columns, beside at most 256 of a split one: its columns are
    // there, and it waits for no other CTA.)
    static constexpr size_t kLeast = size_t(kTmem) * (228 * 1024 / 512) - 1024, kAlone = 116 * 1024;
    static size_t need(int ring, int splits) {
        return size_t(kHead) + size_t(ring) * kStageBytes + (splits > 1 ? size_t(BN < 4 * splits ? 4 * splits : BN) * kRows * 4 : 0) + 1024;
    }
    static size_t smem(int ring, int splits) {
        const size_t least = splits > 1 ? kAlone : kLeast, n = need(ring, splits);
        return n < least ? least : n;
    }
};

template <typename T, int BN, bool kNv, bool kStall = false>
__global__ void __launch_bounds__(kTileThreads)
    fp4_tile_kernel(const __grid_constant__ CUtensorMap tm_w, const __grid_constant__ CUtensorMap tm_x,
                    const __grid_constant__ CUtensorMap tm_ws, const __grid_constant__ CUtensorMap tm_xs, const Args a) {
    using C = TileCfg<BN, kNv>;
    extern __shared__ uint8_t raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem);                    // full[ring], empty[ring], acc, drain
    uint32_t* words = reinterpret_cast<uint32_t*>(smem + 512);             // TMEM base, abort flag
    uint8_t* ring = smem + C::kHead;
    const uint32_t ring0 = ptx::smem_u32(ring);
    const uint32_t w0 = ring0, x0 = w0 + a.ring * (kRows * kRowBytes), ws0 = x0 + a.ring * (BN * kRowBytes),
                   xs0 = ws0 + a.ring * C::kSf, red0 = xs0 + a.ring * C::kSf;
    const uint32_t bar0 = ptx::smem_u32(bars);
    auto full = [&](int s) { return bar0 + 8u * s; };
    auto empty = [&](int s) { return bar0 + 8u * (C::kMaxRing + s); };
    const uint32_t acc_bar = bar0 + 8u * (2 * C::kMaxRing), drain_bar = acc_bar + 8u;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const SyncOf<kStall> sync{words + 1, a.status};
    const int S = a.splits;
    const int rank = S > 1 ? static_cast<int>(ptx::cluster_rank()) : 0;
    const int tile = blockIdx.x / S;
    const int tw = tile / a.tiles_c, tx = tile - tw * a.tiles_c;
    const int kb0 = static_cast<int>(int64_t(a.stages) * rank / S), kb1 = static_cast<int>(int64_t(a.stages) * (rank + 1) / S);

    if (threadIdx.x == 0) {
        for (int s = 0; s < a.ring; ++s) {
            ptx::mbar_init(full(s), 1);
            ptx::mbar_init(empty(s), 1);
        }
        ptx::mbar_init(acc_bar, 1);
        ptx::mbar_init(drain_bar, 1);
        words[1] = 0;
        ptx::fence_mbar_init();
    }
    if (warp == 1) {
        ptx::tmem_alloc(ptx::smem_u32(words), C::kTmem);
        ptx::tmem_relinquish();
    }
    ptx::tc_fence_before();
    __syncthreads();
    if (S > 1) ptx::cluster_arrive_relaxed();   // waited for before the first remote store: every CTA has started
    ptx::tc_fence_after();
    const uint32_t tmem = words[0];
    ptx::launch_dependents();

    bool ok = true;
    if (warp == 0) {
        ptx::prefetch_tmap(&tm_w);
        const uint32_t e = elect();
        ptx::grid_dependency_wait();   // either operand may be the preceding kernel's output
        for (int kb = kb0, n = 0; kb < kb1; ++kb, ++n) {
            const int s = n % a.ring, r = n / a.ring;
            if (r > 0 && !lat::wait_warp(empty(s), (r - 1) & 1, sync)) break;
            ptx::mbar_arrive_expect_tx_if(e, full(s), C::kStageBytes);
            if (!(kStall && blockIdx.x == 0 && n == 1))
                ptx::tma_load_2d_if(e, w0 + s * (kRows * kRowBytes), &tm_w, kb * kRowBytes, tw * kRows, full(s));
            ptx::tma_load_2d_if(e, ws0 + s * C::kSf, &tm_ws, kb * (C::kSf / 8), tw, full(s));
            ptx::tma_load_2d_if(e, x0 + s * (BN * kRowBytes), &tm_x, kb * kRowBytes, tx * BN, full(s));
            ptx::tma_load_2d_if(e, xs0 + s * C::kSf, &tm_xs, kb * (C::kSf / 8), tx * BN / kRows, full(s));
        }
    } else if (warp == 1) {
        const uint32_t e = elect();
        ptx::grid_dependency_wait();   // (so that the limit of a wait below is not spent on the preceding kernel)
        constexpr uint32_t idesc = idesc_fp4(kRows, BN, kNv);
        const uint64_t wd = ptx::smem_desc(w0, 16, 1024, ptx::kLayoutSw128), xd = ptx::smem_desc(x0, 16, 1024, ptx::kLayoutSw128);
        const uint64_t wsd = ptx::smem_desc(ws0, 128, 128, ptx::kLayoutNone), xsd = ptx::smem_desc(xs0, 128, 128, ptx::kLayoutNone);
        // the tile's tokens may start inside their row block: two columns further for each 64
        const uint32_t sfx_off = static_cast<uint32_t>(tx * BN % kRows) / 32;
        for (int kb = kb0, n = 0; kb < kb1; ++kb, ++n) {
            const int s = n % a.ring, r = n / a.ring;
            if (!lat::wait_warp(full(s), r & 1, sync)) break;
            ptx::tc_fence_after();
            const uint32_t sfw = tmem + C::kSfAt + (n & 1) * 2 * C::kSfCols, sfx = sfw + C::kSfCols;
            copy_scales<1, kNv, 4>(sfw, wsd + s * (C::kSf >> 4));
            copy_scales<1, kNv, 4>(sfx, xsd + s * (C::kSf >> 4));
            const int left = a.K - kb * kStageK, mmas = left >= kStageK ? 4 : (left + kMmaK - 1) / kMmaK;
            mma_stage<1, kNv, 4, 4>(tmem, wd + s * (kRows * kRowBytes >> 4), xd + s * (BN * kRowBytes >> 4), idesc, sfw,
                                    sfx + sfx_off, n > 0, mmas);
            ptx::tc_commit_if(e, empty(s));
        }
        ptx::tc_commit_if(e, acc_bar);
    } else {
        ptx::grid_dependency_wait();   // the tensor scales; and D may still be read
        const int quad = warp & 3, row = quad * 32 + lane;
        const int n = tw * kRows + row;
        const Scales<kNv> scales(a);
        const int m0 = tx * BN;
        const uint32_t t_lane = tmem + (static_cast<uint32_t>(quad * 32) << 16);
        // Sums of four tokens for the lane's weight row -> D: lanes exchange with their neighbours, so that each
        // stores two weight rows of two tokens.
        T* const D = static_cast<T*>(a.D) + (n & ~1);
        auto store4 = [&](const float (&v)[4], int m) {
#pragma unroll
            for (int c = 0; c < 4; c += 2) {
                const float2 d = scales.scaled(v[c], v[c + 1]);
                const float other = __shfl_xor_sync(0xFFFFFFFFu, lane & 1 ? d.x : d.y, 1);
                const int token = m + c + (lane & 1);
                const uint32_t two = lane & 1 ? Pair<T>::pack(other, d.y) : Pair<T>::pack(d.x, other);
                if (n < a.N && token < a.M) *reinterpret_cast<uint32_t*>(D + int64_t(token) * a.N) = two;
            }
        };
        ok = lat::wait_warp(acc_bar, 0, sync);
        ptx::tc_fence_after();
        if (S > 1) ptx::cluster_wait();
        // A part's share of the tokens: whole fours, the last parts of a short tile may have none.
        const int cols = BN / S < 4 ? 4 : BN / S, shift = 31 - __clz(cols);
        // received sums: [part][four tokens][row][4]
        const uint32_t mine = red0 + (rank * cols * kRows + row * 4) * 4;
        if (ok) {
#pragma unroll 1
            for (int c0 = 0; c0 < BN && m0 + c0 < a.M; c0 += 16) {
                uint32_t v[16];
                ptx::tmem_ld<16>(t_lane + c0, v);
                ptx::tmem_wait_ld();
#pragma unroll
                for (int c = 0; c < 16; c += 4) {
                    if (S > 1) {
                        const int to = (c0 + c) >> shift, at = (c0 + c) & (cols - 1);
                        st_cluster_v4(ptx::mapa(mine + at * kRows * 4, to), v[c], v[c + 1], v[c + 2], v[c + 3]);
                    } else {
                        const float f[4] = {__uint_as_float(v[c]), __uint_as_float(v[c + 1]), __uint_as_float(v[c + 2]), __uint_as_float(v[c + 3])};
                        store4(f, m0 + c0 + c);
                    }
                }
            }
        }
        ptx::tc_fence_before();
        if (S > 1) {
            ptx::cluster_sync();
            // (the parts of a CTA that gave up are not there: its tile is undefined, as the status says)
            const float4* red = reinterpret_cast<const float4*>(ring + (red0 - ring0)) + row;
            for (int c = 0; c < cols; c += 4) {
                const int m = m0 + rank * cols + c;
                if (rank * cols >= BN || m >= a.M) break;
                float4 sum = red[c / 4 * kRows];
                for (int r = 1; r < S; ++r) {
                    const float4 x = red[(r * cols + c) / 4 * kRows];
                    sum.x += x.x;
                    sum.y += x.y;
                    sum.z += x.z;
                    sum.w += x.w;
                }
                const float f[4] = {sum.x, sum.y, sum.z, sum.w};
                store4(f, m);
            }
        }
    }
    if (S > 1 && warp < 2) {
        ptx::cluster_wait();
        ptx::cluster_sync();
    }
    __syncthreads();
    if (*sync.abort_flag != 0u) {
        // copies and MMAs in flight land before shared and tensor memory are given back (bounded, as every wait)
        if (warp == 0) {
            for (int s = 0; s < a.ring; ++s) {
                const int uses = (kb1 - kb0 - s + a.ring - 1) / a.ring;   // (an upper bound: later ones were not issued)
                for (int r = 0; r < uses; ++r) {
                    const long long t0 = clock64();
                    while (!ptx::mbar_try_wait(full(s), r & 1) && clock64() - t0 < (1ll << 22)) {
                    }
                }
            }
        } else if (warp == 1) {
            ptx::tc_commit_if(elect(), drain_bar);
            const long long t0 = clock64();
            while (!ptx::mbar_try_wait(drain_bar, 0) && clock64() - t0 < (1ll << 26)) {
            }
        }
        __syncthreads();
    }
    ptx::tc_fence_after();
    if (warp == 1) ptx::tmem_dealloc(tmem, C::kTmem);
}

// ---------------------------------------------------------------- many tokens: CTA pairs
//
// A pair of CTAs shares a tile of kHalves * 256 tokens x BN weight rows
// (.cta_group::2): each holds its tokens and half of the weight rows of every
// stage, and reads its tokens' sums.  What bounds this product is shared
// memory: at 4 bits an MMA of 256 x 192 x 64 lasts 96 cycles, in which its
// operands are read (10 KB an SM) and the next ones written (8.7 KB with one
// half, 6.5 KB with two that share the weights), at 128 bytes a cycle.
// Measured in a graph, two halves: 4096 x 7168 x 7168 NVFP4 58 us (7.2 PFLOP/s),
// MXFP4 56 us; 8192 x 24576 x 1536 MXFP4 108 us (115 with one half): its 402 MB of
// D take HBM 99 us by themselves (a fill), and the rest 81 without them.
//
// TMEM holds two accumulators.  One half: tiles take them in turn, and one is
// read while the next tile's sums form in the other.  Two halves: one each; a
// tile's end shows, so it pays where K is long.
//
// Warps: 0 loads (TMA; both CTAs' boxes land on the leader's barrier), 1 issues
// (the leader's), 4-7 and 8-11 read an accumulator each (a TMEM lane quarter a
// warp).
constexpr int kPairThreads = 384;

template <int BN, bool kNv, int kHalves>
struct PairCfg {
    static constexpr int kSf = sf_bytes(kNv);
    static constexpr int kWBlocks = BN > 128 ? 2 : 1;                // row blocks that a tile's weight rows touch
    static constexpr int kHalfBytes = kRows * kRowBytes;
    static constexpr int kXBytes = kHalves * kHalfBytes, kWBytes = BN / 2 * kRowBytes;
    static constexpr int kXSf = kHalves * kSf, kWSf = kWBlocks * kSf;
    static constexpr int kStageBytes = kXBytes + kWBytes + kXSf + kWSf;
    static constexpr int kRoom = 227 * 1024 - 2048;
    static constexpr int kRing = kRoom / kStageBytes < 8 ? kRoom / kStageBytes : 8;
    static constexpr int kWord = kNv ? 16 : 8;                       // TMEM columns of a row block's scales a stage
    static constexpr int kSfCols = kWord * (kHalves + kWBlocks);
    static constexpr uint32_t kSfAt = 2 * BN;
    static_assert(kSfAt + 2 * kSfCols <= 512, "TMEM");
    static_assert(BN % 64 == 0 && BN <= 192, "tiles start at a row block or in its middle");
    static constexpr int kTokens = kHalves * 256;                    // of a pair's tile
    static constexpr size_t kHead = 1024;
    static constexpr size_t kSmem = kHead + size_t(kRing) * kStageBytes + 1024;
};

// Arrives on a barrier of either CTA of the pair, publishing nothing: what it
// says is that TMEM has been read, which tcgen05.wait::ld and the fence before
// it have settled.  (With release semantics it waited for the warp's stores of
// the tile before: 8192 x 24576 x 1536 took 134.8 us, and 116.9 so.)
__device__ __forceinline__ void arrive_relaxed_if(uint32_t pred, uint32_t cluster_bar) {
    asm volatile(
        "{\n.reg .pred p;\nsetp.ne.b32 p, %1, 0;\n"
        "@p mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];\n}" ::"r"(cluster_bar), "r"(pred)
        : "memory");
}
// 32 bytes that L2 gives up first: what is written once and is larger than
// L2 has room for beside the operands makes way for them (116.9 -> 114.3 us).
__device__ __forceinline__ void st_global_v8_first(void* p, const uint32_t (&w)[8]) {
    asm volatile("st.global.L1::no_allocate.L2::evict_first.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]),
                 "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
}

// A whole warp waits for a phase that the other CTA of the pair may complete.
template <long long kLimit>
static __device__ __noinline__ bool pair_wait_slow(uint32_t bar, uint32_t parity, const lat::Sync<kLimit>& s) {
    const long long t0 = clock64();
    for (uint32_t spins = 1;; ++spins) {
        if (__all_sync(0xFFFFFFFFu, ptx::mbar_try_wait_cluster(bar, parity))) return true;
        if ((spins & 63u) == 0) {
            const long long dt = clock64() - t0;
            if (__any_sync(0xFFFFFFFFu, dt > kLimit)) {
                *s.abort_flag = 1u;
                if ((threadIdx.x & 31) == 0) atomicOr(s.status, lat::kStatusTimeout);
                __syncwarp();
                return false;
            }
            if (__any_sync(0xFFFFFFFFu, dt > lat::kAbortPollClocks && *s.abort_flag)) return false;
        }
    }
}
template <long long kLimit>
__device__ __forceinline__ bool pair_wait(uint32_t bar, uint32_t parity, const lat::Sync<kLimit>& s) {
    if (__all_sync(0xFFFFFFFFu, ptx::mbar_try_wait_cluster(bar, parity))) return true;
    return pair_wait_slow(bar, parity, s);
}
// Tile i: weight tiles of a group of 16 token tiles before the next group's, so
// that what runs together shares both operands in L2.
__device__ __forceinline__ void pair_tile(const Args& a, int i, int& tm, int& tn) {
    const int per = 16 * a.tiles_n, g = i / per, in = i - g * per;
    const int rows = min(16, a.tiles_c - g * 16);
    tn = in / rows;
    tm = g * 16 + in - tn * rows;
}

template <typename T, int BN, bool kNv, int kHalves, bool kStall = false>
__global__ void __launch_bounds__(kPairThreads, 1) __cluster_dims__(2, 1, 1)
    fp4_pair_kernel(const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_w,
                    const __grid_constant__ CUtensorMap tm_xs, const __grid_constant__ CUtensorMap tm_ws, const Args a) {
    using C = PairCfg<BN, kNv, kHalves>;
    extern __shared__ uint8_t raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
    uint32_t* words = reinterpret_cast<uint32_t*>(smem + 512);   // TMEM base, abort flag
    const uint32_t bar0 = ptx::smem_u32(smem), ring0 = bar0 + C::kHead;
    const uint32_t x0 = ring0, w0 = x0 + C::kRing * C::kXBytes, xs0 = w0 + C::kRing * C::kWBytes, ws0 = xs0 + C::kRing * C::kXSf;
    auto full = [&](int s) { return bar0 + 8u * s; };
    auto empty = [&](int s) { return bar0 + 8u * (8 + s); };
    auto acc_full = [&](int b) { return bar0 + 8u * (16 + b); };
    auto acc_empty = [&](int b) { return bar0 + 8u * (18 + b); };
    const uint32_t drain_bar = bar0 + 8u * 20;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const SyncOf<kStall> sync{words + 1, a.status};
    const uint32_t rank = ptx::cluster_rank();
    const int first = blockIdx.x >> 1, step = gridDim.x >> 1;

    if (threadIdx.x == 0) {
        for (int s = 0; s < C::kRing; ++s) {
            ptx::mbar_init(full(s), 1);
            ptx::mbar_init(empty(s), 1);
        }
        for (int b = 0; b < 2; ++b) {
            ptx::mbar_init(acc_full(b), 1);
            ptx::mbar_init(acc_empty(b), 8);   // the reading warps of both CTAs
        }
        ptx::mbar_init(drain_bar, 1);
        words[1] = 0;
        ptx::fence_mbar_init();
    }
    if (warp == 2) {
        ptx::tmem_alloc_g<2>(ptx::smem_u32(words), 512);
        ptx::tmem_relinquish_g<2>();
    }
    ptx::tc_fence_before();
    __syncthreads();
    ptx::cluster_sync();
    ptx::tc_fence_after();
    const uint32_t tmem = words[0];
    ptx::launch_dependents();

    if (warp == 0) {
        const uint32_t e = elect();
        if (e) {
            ptx::prefetch_tmap(&tm_x);
            ptx::prefetch_tmap(&tm_w);
            ptx::prefetch_tmap(&tm_xs);
            ptx::prefetch_tmap(&tm_ws);
        }
        __syncwarp();
        ptx::grid_dependency_wait();   // either operand may be the preceding kernel's output
        int n = 0;
        bool ok = true;
        for (int i = first; i < a.tiles && ok; i += step) {
            int tm, tn;
            pair_tile(a, i, tm, tn);
            const int row = tm * C::kTokens + static_cast<int>(rank) * (kHalves * kRows), wrow = tn * BN + static_cast<int>(rank) * (BN / 2);
            for (int kb = 0; kb < a.stages; ++kb, ++n) {
                const int s = n % C::kRing, r = n / C::kRing;
                if (r > 0 && !pair_wait(empty(s), (r - 1) & 1, sync)) {
                    ok = false;
                    break;
                }
                const uint32_t bar = ptx::mapa(full(s), 0u);
                ptx::mbar_arrive_expect_tx_if(e && rank == 0u, full(s), 2 * C::kStageBytes);
                ptx::tma_load_2d_pair_if(e, x0 + s * C::kXBytes, &tm_x, kb * kRowBytes, row, bar);
                if (!(kStall && blockIdx.x == 0 && n == 1))
                    ptx::tma_load_2d_pair_if(e, w0 + s * C::kWBytes, &tm_w, kb * kRowBytes, wrow, bar);
                ptx::tma_load_2d_pair_if(e, xs0 + s * C::kXSf, &tm_xs, kb * (C::kSf / 8), row / kRows, bar);
                ptx::tma_load_2d_pair_if(e, ws0 + s * C::kWSf, &tm_ws, kb * (C::kSf / 8), tn * BN / kRows, bar);
            }
        }
    } else if (warp == 1 && rank == 0u) {
        const uint32_t e = elect();
        ptx::grid_dependency_wait();   // (so that the limit of a wait below is not spent on the preceding kernel)
        constexpr uint32_t idesc = idesc_fp4(2 * kRows, BN, kNv);
        const uint64_t xd = ptx::smem_desc(x0, 16, 1024, ptx::kLayoutSw128), wd = ptx::smem_desc(w0, 16, 1024, ptx::kLayoutSw128);
        const uint64_t xsd = ptx::smem_desc(xs0, 128, 128, ptx::kLayoutNone), wsd = ptx::smem_desc(ws0, 128, 128, ptx::kLayoutNone);
        const int last = (a.K - (a.stages - 1) * kStageK + kMmaK - 1) / kMmaK;   // MMAs of a tile's last stage
        int n = 0, t = 0;
        bool ok = true;
        for (int i = first; i < a.tiles && ok; i += step, ++t) {
            int tm, tn;
            pair_tile(a, i, tm, tn);
            const uint32_t off = static_cast<uint32_t>(tn * BN % kRows) / 32;   // first weight row inside its row block
            // use u of accumulator b (of each half, or every other tile's)
            const int b0 = kHalves == 2 ? 0 : t & 1, u = kHalves == 2 ? t : t >> 1;
            for (int kb = 0; kb < a.stages; ++kb, ++n) {
                const int s = n % C::kRing, r = n / C::kRing;
                if (!(ok = pair_wait(full(s), r & 1, sync))) break;
                ptx::tc_fence_after();
                const uint32_t sfx = tmem + C::kSfAt + (n & 1) * C::kSfCols, sfw = sfx + kHalves * C::kWord;
                const int mmas = kb + 1 < a.stages ? 4 : last;
#pragma unroll
                for (int q = 0; q < C::kWBlocks; ++q)
                    copy_scales<2, kNv, 4 * C::kWBlocks>(sfw + 4 * q, wsd + s * (C::kWSf >> 4) + q * (C::kSf >> 4));
#pragma unroll
                for (int h = 0; h < kHalves; ++h) {
                    const int b = kHalves == 2 ? h : b0;
                    if (kb == 0) {   // the accumulator's last sums have been read
                        if (u > 0 && !(ok = pair_wait(acc_empty(b), (u - 1) & 1, sync))) break;
                        ptx::tc_fence_after();
                    }
                    const uint32_t sfh = sfx + h * C::kWord;
                    copy_scales<2, kNv, 4>(sfh, xsd + s * (C::kXSf >> 4) + h * (C::kSf >> 4));
                    mma_stage<2, kNv, 4, 4 * C::kWBlocks>(tmem + b * BN, xd + s * (C::kXBytes >> 4) + h * (C::kHalfBytes >> 4),
                                                          wd + s * (C::kWBytes >> 4), idesc, sfh, sfw + off, kb > 0, mmas);
                    if (kb + 1 == a.stages) ptx::tc_commit_g_if<2>(e, acc_full(b));
                }
                if (!ok) break;
                ptx::tc_commit_g_if<2>(e, empty(s));
            }
        }
        ptx::tc_commit_local_g_if<2>(e, drain_bar);
        if (!ptx::mbar_try_wait(drain_bar, 0)) lat::wait_warp(drain_bar, 0, sync);
    } else if (warp >= 4) {
        ptx::grid_dependency_wait();   // the tensor scales; and D may still be read
        const int quad = warp & 3, b = (warp - 4) >> 2;   // accumulator b
        const Scales<kNv> scales(a);
        const uint32_t acc = tmem + (static_cast<uint32_t>(quad * 32) << 16) + b * BN;
        T* const D = static_cast<T*>(a.D);
        const bool wide = ((reinterpret_cast<uintptr_t>(D) | (static_cast<uintptr_t>(a.N) * 2u)) & 31u) == 0;
        const int mine = kHalves == 2 ? step : 2 * step;
        int u = 0;
        for (int i = first + (kHalves == 2 ? 0 : b * step); i < a.tiles; i += mine, ++u) {
            int tm, tn;
            pair_tile(a, i, tm, tn);
            if (!pair_wait(acc_full(b), u & 1, sync)) break;
            ptx::tc_fence_after();
            // all of a row goes to registers before any of it is stored: the accumulator is free sooner
            uint32_t w[BN / 2];
#pragma unroll
            for (int c = 0; c < BN; c += 32) {
                uint32_t v[32];
                ptx::tmem_ld<32>(acc + c, v);
                ptx::tmem_wait_ld();
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    const float2 d = scales.scaled(__uint_as_float(v[2 * j]), __uint_as_float(v[2 * j + 1]));
                    w[c / 2 + j] = Pair<T>::pack(d.x, d.y);
                }
            }
            ptx::tc_fence_before();
            __syncwarp();
            arrive_relaxed_if(lane == 0 ? 1u : 0u, ptx::mapa(acc_empty(b), 0u));
            const int m = tm * C::kTokens + (static_cast<int>(rank) * kHalves + (kHalves == 2 ? b : 0)) * kRows + quad * 32 + lane;
            const int n0 = tn * BN;
            if (m < a.M) {
                T* row = D + int64_t(m) * a.N + n0;
#pragma unroll
                for (int c = 0; c < BN; c += 16) {
                    uint32_t q[8];
#pragma unroll
                    for (int j = 0; j < 8; ++j) q[j] = w[c / 2 + j];
                    if (wide && n0 + c + 16 <= a.N) {
                        if (a.stream_out) st_global_v8_first(row + c, q);
                        else ptx::st_global_v8(row + c, q);
                    } else {
                        if (n0 + c < a.N) *reinterpret_cast<uint4*>(row + c) = make_uint4(q[0], q[1], q[2], q[3]);
                        if (n0 + c + 8 < a.N) *reinterpret_cast<uint4*>(row + c + 8) = make_uint4(q[4], q[5], q[6], q[7]);
                    }
                }
            }
        }
    }
    __syncthreads();
    if (*sync.abort_flag != 0u) {
        // copies in flight land before the CTA leaves: each takes microseconds
        const long long t0 = clock64();
        while (clock64() - t0 < (1ll << 22)) {
        }
    }
    ptx::tc_fence_before();
    __syncthreads();
    ptx::cluster_sync();   // no remote operation targets a CTA that has left
    if (warp == 2) {
        ptx::tc_fence_after();
        ptx::tmem_dealloc_g<2>(tmem, 512);
    }
}

// ---------------------------------------------------------------- host

// Codes [rows, K / 2] in boxes of 128 bytes x `box` rows, 128-byte swizzle.
sgq_status code_map(gemm::TensorMapEncoder encode, CUtensorMap* m, const void* p, int64_t rows, int64_t K, int box) {
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(K / 2), static_cast<cuuint64_t>(rows)};
    const cuuint64_t strides[1] = {static_cast<cuuint64_t>(K / 2)};
    const cuuint32_t boxes[2] = {kRowBytes, static_cast<cuuint32_t>(box)}, ones[2] = {1, 1};
    return encode(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(p), dims, strides, boxes, ones,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
               ? SGQ_OK
               : SGQ_ERR_CUDA;
}
// Scale tiles [row blocks, tiles along K, 512 bytes] in boxes of a stage's
// tiles of `blocks` row blocks, as 8-byte elements (a box has at most 256 a
// side).  What lies past the last tile reads as zero.
sgq_status scale_map(gemm::TensorMapEncoder encode, CUtensorMap* m, const void* p, int64_t rows, int64_t K, bool nv,
                     int blocks) {
    const int64_t tiles = scale_tiles(K, nv);
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(tiles * 64), static_cast<cuuint64_t>((rows + 127) / 128)};
    const cuuint64_t strides[1] = {static_cast<cuuint64_t>(tiles * 512)};
    const cuuint32_t boxes[2] = {static_cast<cuuint32_t>(sf_bytes(nv) / 8), static_cast<cuuint32_t>(blocks)}, ones[2] = {1, 1};
    return encode(m, CU_TENSOR_MAP_DATA_TYPE_UINT64, 2, const_cast<void*>(p), dims, strides, boxes, ones,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
               ? SGQ_OK
               : SGQ_ERR_CUDA;
}

struct Maps {
    CUtensorMap w, x, ws, xs;
};

sgq_status device_of(int* dev) { return cudaGetDevice(dev) == cudaSuccess && *dev >= 0 && *dev < 64 ? SGQ_OK : SGQ_ERR_CUDA; }

// K splits of the tile kernel: doubled while every CTA still has an SM of its own and a stage to do.
int tile_splits(int64_t tiles, int stages, int sms) {
    int splits = 1;
    while (splits < 8 && splits * 2 <= stages && tiles * splits * 2 <= sms) splits *= 2;
    return splits;
}

// Which kernel serves more than 64 tokens: the one whose time, in us, is least
// by a model of a few terms.  A call costs 2.9 (tiles) or 3.2 (pairs); a stage
// costs an issuing warp 0.31, 0.48 with two halves; a pair's tile ends in 0.25
// and 1.2; the sum over the parts of a split tile takes 1.3 for 64 tokens and 3
// for 128; where tiles outnumber the SMs, two CTAs on an SM take 1.5 times one's
// time for 64 tokens and 2.6 for 128, whose loads already fill the SM's share of
// L2.  Measured in a graph (NVFP4; MXFP4 is 3 to 8 % faster), and by the model:
//   N, K, M              64 tokens  128 tokens  pairs, one half  two halves
//   1536, 7168, 128         6.4         7.2          11.8           15.5
//                          (6.4         7.1          12.1           17.8)
//   1536, 7168, 301         8.9         8.7          11.6           17.0
//                          (8.5         8.1          12.1           17.8)
//   7168, 2048, 301         6.8         8.0           7.1            9.3
//                          (6.6         9.3           5.9            8.2)
//   24576, 1536, 128       11.9         8.8           9.4           12.3
//                          (8.5         7.7           7.4           11.4)
//   7168, 7168, 1024       41.0        30.2          21.5           20.2
//                         (42.0        48.0          21.1           17.8)
//   7168, 7168, 4096      156.9        96.3          70.6           58.9
//                        (159.1       138.3          74.6           61.8)
//   24576, 1536, 8192       410         263           114            116
//                          (229         201           117            113)
// So it takes the fastest of four in four of these rows, and one that is 2 to 7 %
// slower in three: 301 x 7168 x 2048 and 128 x 24576 x 1536, where it holds pairs
// too short by 1.2 and 2.0, and 8192 x 24576 x 1536.  For many tiles it is far too
// short on tiles without pairs (to 1.8 times), which are not taken there.
enum Way { kTile64, kTile128, kPair1, kPair2 };
Way way_of(int64_t M, int64_t N, int stages, int sms) {
    auto tile = [&](int bn) {
        const int64_t tiles = (N + kRows - 1) / kRows * ((M + bn - 1) / bn);
        const int splits = tile_splits(tiles, stages, sms);
        const double waves = tiles * splits <= sms ? 1.0 : double((tiles + 2 * sms - 1) / (2 * sms)) * (bn == 64 ? 1.5 : 2.6);
        return 2.9 + waves * ((stages + splits - 1) / splits) * 0.31 + (splits == 1 ? 0.0 : bn == 64 ? 1.3 : 3.0);
    };
    auto pair = [&](int64_t tokens, double stage, double end) {
        const int64_t tiles = (M + tokens - 1) / tokens * ((N + 191) / 192), pairs = sms > 1 ? sms / 2 : 1;
        return 3.2 + double((tiles + pairs - 1) / pairs) * (stages * stage + end);
    };
    const double t[4] = {tile(64), tile(128), pair(256, 0.31, 0.25), pair(512, 0.48, 1.2)};
    int best = kPair1;
    for (int i = 0; i < 4; ++i)
        if (t[i] < t[best]) best = i;
    return static_cast<Way>(best);
}

template <typename T, int BN, bool kNv, bool kStall = false>
sgq_status run_tile(gemm::TensorMapEncoder encode, const Fp4GemmArgs& g, Args a, int sms, int smem_max, cudaStream_t st) {
    using C = TileCfg<BN, kNv>;
    Maps tm;
    if (code_map(encode, &tm.w, g.Wq, g.N, g.K, kRows) != SGQ_OK || code_map(encode, &tm.x, g.Aq, g.M, g.K, BN) != SGQ_OK ||
        scale_map(encode, &tm.ws, g.Ws, g.N, g.K, kNv, 1) != SGQ_OK || scale_map(encode, &tm.xs, g.As, g.M, g.K, kNv, 1) != SGQ_OK)
        return SGQ_ERR_CUDA;
    a.tiles_c = static_cast<int>((g.M + BN - 1) / BN);
    const int64_t tiles = (g.N + kRows - 1) / kRows * a.tiles_c;
    a.splits = tile_splits(tiles, a.stages, sms);
    const int per = (a.stages + a.splits - 1) / a.splits;
    a.ring = per < C::kMaxRing ? per : C::kMaxRing;
    const size_t room = (tiles * a.splits <= sms ? 226 : 113) * 1024;   // of an SM for one CTA, or for two
    while (a.ring > 2 && C::need(a.ring, a.splits) > room) --a.ring;
    if (tiles * a.splits > INT32_MAX) return SGQ_ERR_INVALID_ARG;
    auto kern = fp4_tile_kernel<T, BN, kNv, kStall>;
    int dev = 0;
    if (device_of(&dev) != SGQ_OK) return SGQ_ERR_CUDA;
    static bool configured[64] = {};
    if (!configured[dev]) {
        if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem_max) != cudaSuccess) return SGQ_ERR_CUDA;
        configured[dev] = true;
    }
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = a.splits;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(tiles * a.splits));
    cfg.blockDim = dim3(kTileThreads);
    cfg.dynamicSmemBytes = C::smem(a.ring, a.splits);
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = a.splits > 1 ? 2 : 1;
    if (cudaLaunchKernelEx(&cfg, kern, tm.w, tm.x, tm.ws, tm.xs, a) != cudaSuccess) return SGQ_ERR_CUDA;
    note_launch();
    return SGQ_OK;
}

template <typename T, int BN, bool kNv, int kHalves, bool kStall = false>
sgq_status run_pair(gemm::TensorMapEncoder encode, const Fp4GemmArgs& g, Args a, int sms, cudaStream_t st) {
    using C = PairCfg<BN, kNv, kHalves>;
    Maps tm;
    if (code_map(encode, &tm.w, g.Wq, g.N, g.K, BN / 2) != SGQ_OK ||
        code_map(encode, &tm.x, g.Aq, g.M, g.K, kHalves * kRows) != SGQ_OK ||
        scale_map(encode, &tm.ws, g.Ws, g.N, g.K, kNv, C::kWBlocks) != SGQ_OK ||
        scale_map(encode, &tm.xs, g.As, g.M, g.K, kNv, kHalves) != SGQ_OK)
        return SGQ_ERR_CUDA;
    const int64_t tiles_m = (g.M + C::kTokens - 1) / C::kTokens, tiles_n = (g.N + BN - 1) / BN;
    if (tiles_m * tiles_n > INT32_MAX || 16 * tiles_n > INT32_MAX) return SGQ_ERR_INVALID_ARG;
    a.tiles_c = static_cast<int>(tiles_m);
    a.tiles_n = static_cast<int>(tiles_n);
    a.tiles = static_cast<int>(tiles_m * tiles_n);
    a.stream_out = g.M * g.N * 2 > (int64_t(32) << 20);
    auto kern = fp4_pair_kernel<T, BN, kNv, kHalves, kStall>;
    int dev = 0;
    if (device_of(&dev) != SGQ_OK) return SGQ_ERR_CUDA;
    static bool configured[64] = {};
    if (!configured[dev]) {
        if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(C::kSmem)) != cudaSuccess)
            return SGQ_ERR_CUDA;
        configured[dev] = true;
    }
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    const int most = sms > 1 ? sms / 2 : 1, pairs = most < a.tiles ? most : a.tiles;
    cfg.gridDim = dim3(static_cast<unsigned>(2 * pairs));
    cfg.blockDim = dim3(kPairThreads);
    cfg.dynamicSmemBytes = C::kSmem;
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, kern, tm.x, tm.w, tm.xs, tm.ws, a) != cudaSuccess) return SGQ_ERR_CUDA;
    note_launch();
    return SGQ_OK;
}

template <typename T, bool kNv>
sgq_status pick(gemm::TensorMapEncoder encode, const Fp4GemmArgs& g, const Args& a, const DeviceInfo& di, cudaStream_t st) {
    if (g.M <= 16) return run_tile<T, 16, kNv>(encode, g, a, di.sm_count, di.max_smem_optin, st);
    if (g.M <= 32) return run_tile<T, 32, kNv>(encode, g, a, di.sm_count, di.max_smem_optin, st);
    if (g.M <= 64) return run_tile<T, 64, kNv>(encode, g, a, di.sm_count, di.max_smem_optin, st);
    switch (way_of(g.M, g.N, a.stages, di.sm_count)) {
        case kTile64: return run_tile<T, 64, kNv>(encode, g, a, di.sm_count, di.max_smem_optin, st);
        case kTile128: return run_tile<T, 128, kNv>(encode, g, a, di.sm_count, di.max_smem_optin, st);
        case kPair1: return run_pair<T, 192, kNv, 1>(encode, g, a, di.sm_count, st);
        case kPair2: return run_pair<T, 192, kNv, 2>(encode, g, a, di.sm_count, st);
    }
    return SGQ_ERR_INVALID_ARG;
}

}  // namespace

sgq_status launch_fp4_gemm(const Fp4GemmArgs& g, cudaStream_t st) {
    DeviceInfo di;
    sgq_status rc = device_info(&di);
    if (rc != SGQ_OK) return rc;
    if (!built_for(di)) return SGQ_ERR_UNSUPPORTED;
    gemm::TensorMapEncoder encode;
    rc = gemm::get_encoder(&encode);
    if (rc != SGQ_OK) return rc;
    Args a{};
    rc = gemm::status_word(&a.status);
    if (rc != SGQ_OK) return rc;
    a.D = g.D;
    a.a_t = g.a_t;
    a.w_t = g.w_t;
    a.M = static_cast<int>(g.M);
    a.N = static_cast<int>(g.N);
    a.K = static_cast<int>(g.K);
    a.stages = static_cast<int>((g.K + kStageK - 1) / kStageK);
    if (g.stall) {   // (the kernels of this flag: bf16, NVFP4)
        if (g.M <= 64) return run_tile<__nv_bfloat16, 64, true, true>(encode, g, a, di.sm_count, di.max_smem_optin, st);
        return g.M <= 512 ? run_pair<__nv_bfloat16, 192, true, 1, true>(encode, g, a, di.sm_count, st)
                          : run_pair<__nv_bfloat16, 192, true, 2, true>(encode, g, a, di.sm_count, st);
    }
    if (g.dtype == SGQ_BF16)
        return g.format == SGQ_NVFP4 ? pick<__nv_bfloat16, true>(encode, g, a, di, st)
                                     : pick<__nv_bfloat16, false>(encode, g, a, di, st);
    return g.format == SGQ_NVFP4 ? pick<__half, true>(encode, g, a, di, st) : pick<__half, false>(encode, g, a, di, st);
}

}  // namespace sgq
