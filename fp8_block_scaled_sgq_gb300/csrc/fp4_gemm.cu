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
constexpr long long kLimit = lat::kTimeoutClocks;
using Sync = lat::Sync<kLimit>;

struct Args {
    void* D;
    const float *a_t, *w_t;   // tensor scales, or null for 1
    uint32_t* status;
    int M, N, K;
    int stages;      // K in stages
    int tiles_c;     // token tiles
    int tiles_n, tiles;   // pairs: weight tiles, and all tiles
    int splits;
    int ring;        // stages in shared memory
};

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
template <bool kNv>
__device__ __forceinline__ void mma_fp4_if(uint32_t pred, uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sfa,
                                           uint32_t sfb, uint32_t acc) {
    if constexpr (kNv)
        asm volatile(
            "{\n.reg .pred p, q;\nsetp.ne.b32 p, %7, 0;\nsetp.ne.b32 q, %6, 0;\n"
            "@p tcgen05.mma.cta_group::1.kind::mxf4nvf4.block_scale.scale_vec::4X [%0], %1, %2, %3, [%4], [%5], q;\n}" ::"r"(
                d),
            "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(acc), "r"(pred)
            : "memory");
    else
        asm volatile(
            "{\n.reg .pred p, q;\nsetp.ne.b32 p, %7, 0;\nsetp.ne.b32 q, %6, 0;\n"
            "@p tcgen05.mma.cta_group::1.kind::mxf4nvf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], q;\n}" ::"r"(
                d),
            "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(acc), "r"(pred)
            : "memory");
}

__device__ __forceinline__ float tensor_scales(const Args& a) {
    return (a.a_t ? __ldg(a.a_t) : 1.0f) * (a.w_t ? __ldg(a.w_t) : 1.0f);
}
template <typename T>
__device__ __forceinline__ T round_to(float x);
template <>
__device__ __forceinline__ __nv_bfloat16 round_to(float x) { return __float2bfloat16_rn(x); }
template <>
__device__ __forceinline__ __half round_to(float x) { return __float2half_rn(x); }

// ---------------------------------------------------------------- weights on the 128-row side
//
// One tile of 128 weight rows x BN tokens a cluster; the cluster's CTAs take
// equal parts of K and sum their accumulators through each other's shared
// memory in the order of the parts, each for its share of the tokens.
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
    // TMEM: CTAs that fit together then never wait for each other's TMEM (a
    // cluster that did, while it holds what another one's peer waits for, would
    // never end).
    static constexpr size_t kLeast = size_t(kTmem) * (228 * 1024 / 512) - 1024;
    static size_t need(int ring, int splits) {
        return size_t(kHead) + size_t(ring) * kStageBytes + (splits > 1 ? size_t(BN) * kRows * 4 : 0) + 1024;
    }
    static size_t smem(int ring, int splits) { return need(ring, splits) < kLeast ? kLeast : need(ring, splits); }
};

template <typename T, int BN, bool kNv>
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
    const Sync sync{words + 1, a.status};
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
            ptx::tma_load_2d_if(e, w0 + s * (kRows * kRowBytes), &tm_w, kb * kRowBytes, tw * kRows, full(s));
            ptx::tma_load_2d_if(e, ws0 + s * C::kSf, &tm_ws, kb * (C::kSf / 8), tw, full(s));
            ptx::tma_load_2d_if(e, x0 + s * (BN * kRowBytes), &tm_x, kb * kRowBytes, tx * BN, full(s));
            ptx::tma_load_2d_if(e, xs0 + s * C::kSf, &tm_xs, kb * (C::kSf / 8), tx * BN / kRows, full(s));
        }
    } else if (warp == 1) {
        const uint32_t e = elect();
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
#pragma unroll
            for (int j = 0; j < C::kSf / 512; ++j) {
                ptx::tmem_cp_32x128b_x4_if(e, sfw + 4 * j, wsd + s * (C::kSf >> 4) + 32 * j);
                ptx::tmem_cp_32x128b_x4_if(e, sfx + 4 * j, xsd + s * (C::kSf >> 4) + 32 * j);
            }
            const int left = a.K - kb * kStageK, mmas = left >= kStageK ? 4 : (left + kMmaK - 1) / kMmaK;
            for (int j = 0; j < mmas; ++j) {
                const uint32_t id = kNv ? idesc : ptx::idesc_sf_ids(idesc, (j & 1) * 2, (j & 1) * 2);
                const uint32_t word = 4 * (kNv ? j : j / 2);
                mma_fp4_if<kNv>(e, tmem, wd + s * (kRows * kRowBytes >> 4) + 2 * j, xd + s * (BN * kRowBytes >> 4) + 2 * j, id,
                                sfw + word, sfx + word + sfx_off, n > 0 || j > 0);
            }
            ptx::tc_commit_if(e, empty(s));
        }
        ptx::tc_commit_if(e, acc_bar);
    } else {
        ptx::grid_dependency_wait();   // the tensor scales; and D may still be read
        const int quad = warp & 3, row = quad * 32 + lane;
        const int n = tw * kRows + row;
        const float scale = tensor_scales(a);
        T* D = static_cast<T*>(a.D) + n;
        const int m0 = tx * BN;
        const uint32_t t_lane = tmem + (static_cast<uint32_t>(quad * 32) << 16);
        ok = lat::wait_warp(acc_bar, 0, sync);
        ptx::tc_fence_after();
        if (S > 1) ptx::cluster_wait();
        const int cols = BN / S;
        if (ok) {
#pragma unroll 1
            for (int c0 = 0; c0 < BN; c0 += 16) {
                uint32_t v[16];
                ptx::tmem_ld<16>(t_lane + c0, v);
                ptx::tmem_wait_ld();
                if (S > 1) {
#pragma unroll
                    for (int c = 0; c < 16; ++c) {
                        const int to = (c0 + c) / cols;
                        const uint32_t at = red0 + ((rank * cols + (c0 + c) - to * cols) * kRows + row) * 4;
                        ptx::st_cluster_f32(ptx::mapa(at, to), __uint_as_float(v[c]));
                    }
                } else if (n < a.N) {
#pragma unroll
                    for (int c = 0; c < 16; ++c)
                        if (m0 + c0 + c < a.M) D[int64_t(m0 + c0 + c) * a.N] = round_to<T>(__uint_as_float(v[c]) * scale);
                }
            }
        }
        ptx::tc_fence_before();
        if (S > 1) {
            ptx::cluster_sync();
            // (the parts of a CTA that gave up are not there: its tile is undefined, as the status says)
            const float* red = reinterpret_cast<const float*>(ring + (red0 - ring0));
            if (n < a.N) {
                for (int c = 0; c < cols; ++c) {
                    const int m = m0 + rank * cols + c;
                    if (m >= a.M) break;
                    float sum = red[c * kRows + row];
                    for (int r = 1; r < S; ++r) sum += red[(r * cols + c) * kRows + row];
                    D[int64_t(m) * a.N] = round_to<T>(sum * scale);
                }
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
// A pair of CTAs shares a tile of 256 tokens x BN weight rows (.cta_group::2):
// each holds its 128 tokens and half of the weight rows of every stage, and
// reads its 128 tokens' sums.  What an SM takes in per operation bounds this
// product: at 4 bits the tensor cores ask for a 128 x 128 tile's stage every
// 0.14 us, 36 KB that take an SM 0.3 us.  A pair's tile halves the weights'
// share.  Two accumulators in TMEM: one is read and written out while the next
// tile's sums form in the other.
//
// Warps: 0 loads (TMA; both CTAs' boxes land on the leader's barrier), 1 issues
// (the leader's), 4-11 read (two a TMEM lane quarter, half of the columns each).
constexpr int kPairThreads = 384;
constexpr int kPairTokens = 256;

template <int BN, bool kNv>
struct PairCfg {
    static constexpr int kSf = sf_bytes(kNv);
    static constexpr int kWBlocks = BN > 128 ? 2 : 1;                // row blocks that a tile's weight rows touch
    static constexpr int kXBytes = kRows * kRowBytes, kWBytes = BN / 2 * kRowBytes;
    static constexpr int kStageBytes = kXBytes + kWBytes + kSf * (1 + kWBlocks);
    static constexpr int kRing = (226 * 1024 - 2048) / kStageBytes < 8 ? (226 * 1024 - 2048) / kStageBytes : 8;
    static constexpr int kSfCols = (kNv ? 16 : 8) * (1 + kWBlocks);  // TMEM columns of a stage's scales
    static constexpr uint32_t kSfAt = 2 * BN;
    static_assert(kSfAt + 2 * kSfCols <= 512, "TMEM");
    static_assert(BN % 64 == 0 && BN <= 192, "tiles start at a row block or in its middle");
    static constexpr size_t kHead = 1024;
    static constexpr size_t kSmem = kHead + size_t(kRing) * kStageBytes + 1024;
};

// A whole warp waits for a phase that the other CTA of the pair may complete.
static __device__ __noinline__ bool pair_wait_slow(uint32_t bar, uint32_t parity, const Sync& s) {
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
__device__ __forceinline__ bool pair_wait(uint32_t bar, uint32_t parity, const Sync& s) {
    if (__all_sync(0xFFFFFFFFu, ptx::mbar_try_wait_cluster(bar, parity))) return true;
    return pair_wait_slow(bar, parity, s);
}
template <bool kNv>
__device__ __forceinline__ void mma_fp4_pair_if(uint32_t pred, uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                                uint32_t sfa, uint32_t sfb, uint32_t acc) {
    if constexpr (kNv)
        asm volatile(
            "{\n.reg .pred p, q;\nsetp.ne.b32 p, %7, 0;\nsetp.ne.b32 q, %6, 0;\n"
            "@p tcgen05.mma.cta_group::2.kind::mxf4nvf4.block_scale.scale_vec::4X [%0], %1, %2, %3, [%4], [%5], q;\n}" ::"r"(
                d),
            "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(acc), "r"(pred)
            : "memory");
    else
        asm volatile(
            "{\n.reg .pred p, q;\nsetp.ne.b32 p, %7, 0;\nsetp.ne.b32 q, %6, 0;\n"
            "@p tcgen05.mma.cta_group::2.kind::mxf4nvf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], q;\n}" ::"r"(
                d),
            "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(acc), "r"(pred)
            : "memory");
}

// Tile i: weight tiles of a group of 16 token tiles before the next group's, so
// that what runs together shares both operands in L2.
__device__ __forceinline__ void pair_tile(const Args& a, int i, int& tm, int& tn) {
    const int per = 16 * a.tiles_n, g = i / per, in = i - g * per;
    const int rows = min(16, a.tiles_c - g * 16);
    tn = in / rows;
    tm = g * 16 + in - tn * rows;
}

template <typename T, int BN, bool kNv>
__global__ void __launch_bounds__(kPairThreads, 1) __cluster_dims__(2, 1, 1)
    fp4_pair_kernel(const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_w,
                    const __grid_constant__ CUtensorMap tm_xs, const __grid_constant__ CUtensorMap tm_ws, const Args a) {
    using C = PairCfg<BN, kNv>;
    extern __shared__ uint8_t raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
    uint32_t* words = reinterpret_cast<uint32_t*>(smem + 512);   // TMEM base, abort flag
    const uint32_t bar0 = ptx::smem_u32(smem), ring0 = bar0 + C::kHead;
    const uint32_t x0 = ring0, w0 = x0 + C::kRing * C::kXBytes, xs0 = w0 + C::kRing * C::kWBytes, ws0 = xs0 + C::kRing * C::kSf;
    auto full = [&](int s) { return bar0 + 8u * s; };
    auto empty = [&](int s) { return bar0 + 8u * (8 + s); };
    auto acc_full = [&](int b) { return bar0 + 8u * (16 + b); };
    auto acc_empty = [&](int b) { return bar0 + 8u * (18 + b); };
    const uint32_t drain_bar = bar0 + 8u * 20;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const Sync sync{words + 1, a.status};
    const uint32_t rank = ptx::cluster_rank();
    const int first = blockIdx.x >> 1, step = gridDim.x >> 1;

    if (threadIdx.x == 0) {
        for (int s = 0; s < C::kRing; ++s) {
            ptx::mbar_init(full(s), 1);
            ptx::mbar_init(empty(s), 1);
        }
        for (int b = 0; b < 2; ++b) {
            ptx::mbar_init(acc_full(b), 1);
            ptx::mbar_init(acc_empty(b), 16);   // the reading warps of both CTAs
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
            const int row = tm * kPairTokens + static_cast<int>(rank) * kRows, wrow = tn * BN + static_cast<int>(rank) * (BN / 2);
            for (int kb = 0; kb < a.stages; ++kb, ++n) {
                const int s = n % C::kRing, r = n / C::kRing;
                if (r > 0 && !pair_wait(empty(s), (r - 1) & 1, sync)) {
                    ok = false;
                    break;
                }
                const uint32_t bar = ptx::mapa(full(s), 0u);
                ptx::mbar_arrive_expect_tx_if(e && rank == 0u, full(s), 2 * C::kStageBytes);
                ptx::tma_load_2d_pair_if(e, x0 + s * C::kXBytes, &tm_x, kb * kRowBytes, row, bar);
                ptx::tma_load_2d_pair_if(e, w0 + s * C::kWBytes, &tm_w, kb * kRowBytes, wrow, bar);
                ptx::tma_load_2d_pair_if(e, xs0 + s * C::kSf, &tm_xs, kb * (C::kSf / 8), tm * 2 + static_cast<int>(rank), bar);
                ptx::tma_load_2d_pair_if(e, ws0 + s * C::kSf * C::kWBlocks, &tm_ws, kb * (C::kSf / 8), tn * BN / kRows, bar);
            }
        }
    } else if (warp == 1 && rank == 0u) {
        const uint32_t e = elect();
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
            const int b = t & 1;
            if (t > 1 && !pair_wait(acc_empty(b), ((t >> 1) - 1) & 1, sync)) break;
            ptx::tc_fence_after();
            const uint32_t d = tmem + b * BN;
            for (int kb = 0; kb < a.stages; ++kb, ++n) {
                const int s = n % C::kRing, r = n / C::kRing;
                if (!pair_wait(full(s), r & 1, sync)) {
                    ok = false;
                    break;
                }
                ptx::tc_fence_after();
                const uint32_t sfx = tmem + C::kSfAt + (n & 1) * C::kSfCols, sfw = sfx + (kNv ? 16 : 8);
#pragma unroll
                for (int j = 0; j < C::kSf / 512; ++j) {
                    ptx::tmem_cp_g_if<2>(e, sfx + 4 * j, xsd + s * (C::kSf >> 4) + 32 * j);
#pragma unroll
                    for (int q = 0; q < C::kWBlocks; ++q)
                        ptx::tmem_cp_g_if<2>(e, sfw + 4 * (j * C::kWBlocks + q),
                                             wsd + s * (C::kSf * C::kWBlocks >> 4) + q * (C::kSf >> 4) + 32 * j);
                }
                const int mmas = kb + 1 < a.stages ? 4 : last;
                for (int j = 0; j < mmas; ++j) {
                    const uint32_t id = kNv ? idesc : ptx::idesc_sf_ids(idesc, (j & 1) * 2, (j & 1) * 2);
                    const uint32_t word = 4 * (kNv ? j : j / 2);
                    mma_fp4_pair_if<kNv>(e, d, xd + s * (C::kXBytes >> 4) + 2 * j, wd + s * (C::kWBytes >> 4) + 2 * j, id, sfx + word,
                                         sfw + word * C::kWBlocks + off, kb > 0 || j > 0);
                }
                ptx::tc_commit_g_if<2>(e, empty(s));
            }
            if (ok) ptx::tc_commit_g_if<2>(e, acc_full(b));
        }
        ptx::tc_commit_local_g_if<2>(e, drain_bar);
        if (!ptx::mbar_try_wait(drain_bar, 0)) lat::wait_warp(drain_bar, 0, sync);
    } else if (warp >= 4) {
        ptx::grid_dependency_wait();   // the tensor scales; and D may still be read
        const int quad = warp & 3, half = (warp - 4) >> 2;
        const float scale = tensor_scales(a);
        const uint32_t t_lane = tmem + (static_cast<uint32_t>(quad * 32) << 16);
        T* const D = static_cast<T*>(a.D);
        const bool wide = ((reinterpret_cast<uintptr_t>(D) | (static_cast<uintptr_t>(a.N) * 2u)) & 31u) == 0;
        int t = 0;
        for (int i = first; i < a.tiles; i += step, ++t) {
            int tm, tn;
            pair_tile(a, i, tm, tn);
            const int b = t & 1;
            if (!pair_wait(acc_full(b), (t >> 1) & 1, sync)) break;
            ptx::tc_fence_after();
            constexpr int kCols = BN / 2;
            uint32_t w[kCols / 2];
#pragma unroll
            for (int c = 0; c < kCols; c += 16) {
                uint32_t v[16];
                ptx::tmem_ld<16>(t_lane + b * BN + half * kCols + c, v);
                ptx::tmem_wait_ld();
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    w[c / 2 + j] = Pair<T>::pack(__uint_as_float(v[2 * j]) * scale, __uint_as_float(v[2 * j + 1]) * scale);
            }
            ptx::tc_fence_before();
            __syncwarp();
            ptx::mbar_arrive_cluster_if(lane == 0 ? 1u : 0u, ptx::mapa(acc_empty(b), 0u));
            const int m = tm * kPairTokens + static_cast<int>(rank) * kRows + quad * 32 + lane;
            const int n0 = tn * BN + half * kCols;
            if (m < a.M) {
                T* row = D + int64_t(m) * a.N + n0;
#pragma unroll
                for (int c = 0; c < kCols; c += 16) {
                    uint32_t q[8];
#pragma unroll
                    for (int j = 0; j < 8; ++j) q[j] = w[c / 2 + j];
                    if (wide && n0 + c + 16 <= a.N) {
                        ptx::st_global_v8(row + c, q);
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

template <typename T, int BN, bool kNv>
sgq_status run_tile(gemm::TensorMapEncoder encode, const Fp4GemmArgs& g, Args a, int sms, int smem_max, cudaStream_t st) {
    using C = TileCfg<BN, kNv>;
    Maps tm;
    if (code_map(encode, &tm.w, g.Wq, g.N, g.K, kRows) != SGQ_OK || code_map(encode, &tm.x, g.Aq, g.M, g.K, BN) != SGQ_OK ||
        scale_map(encode, &tm.ws, g.Ws, g.N, g.K, kNv, 1) != SGQ_OK || scale_map(encode, &tm.xs, g.As, g.M, g.K, kNv, 1) != SGQ_OK)
        return SGQ_ERR_CUDA;
    a.tiles_c = static_cast<int>((g.M + BN - 1) / BN);
    const int64_t tiles = (g.N + kRows - 1) / kRows * a.tiles_c;
    a.splits = 1;
    while (a.splits < 8 && a.splits * 2 <= a.stages && tiles * a.splits * 2 <= sms) a.splits *= 2;
    const int per = (a.stages + a.splits - 1) / a.splits;
    a.ring = per < C::kMaxRing ? per : C::kMaxRing;
    while (a.ring > 2 && C::need(a.ring, a.splits) > 113 * 1024) --a.ring;
    if (tiles * a.splits > INT32_MAX) return SGQ_ERR_INVALID_ARG;
    auto kern = fp4_tile_kernel<T, BN, kNv>;
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

template <typename T, int BN, bool kNv>
sgq_status run_pair(gemm::TensorMapEncoder encode, const Fp4GemmArgs& g, Args a, int sms, cudaStream_t st) {
    using C = PairCfg<BN, kNv>;
    Maps tm;
    if (code_map(encode, &tm.w, g.Wq, g.N, g.K, BN / 2) != SGQ_OK || code_map(encode, &tm.x, g.Aq, g.M, g.K, kRows) != SGQ_OK ||
        scale_map(encode, &tm.ws, g.Ws, g.N, g.K, kNv, C::kWBlocks) != SGQ_OK ||
        scale_map(encode, &tm.xs, g.As, g.M, g.K, kNv, 1) != SGQ_OK)
        return SGQ_ERR_CUDA;
    const int64_t tiles_m = (g.M + kPairTokens - 1) / kPairTokens, tiles_n = (g.N + BN - 1) / BN;
    if (tiles_m * tiles_n > INT32_MAX || 16 * tiles_n > INT32_MAX) return SGQ_ERR_INVALID_ARG;
    a.tiles_c = static_cast<int>(tiles_m);
    a.tiles_n = static_cast<int>(tiles_n);
    a.tiles = static_cast<int>(tiles_m * tiles_n);
    auto kern = fp4_pair_kernel<T, BN, kNv>;
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
    const int pairs = sms / 2 < a.tiles ? sms / 2 : a.tiles;
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
    if (g.M > 512) return run_pair<T, 192, kNv>(encode, g, a, di.sm_count, st);
    return run_tile<T, 128, kNv>(encode, g, a, di.sm_count, di.max_smem_optin, st);
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
    if (g.dtype == SGQ_BF16)
        return g.format == SGQ_NVFP4 ? pick<__nv_bfloat16, true>(encode, g, a, di, st)
                                     : pick<__nv_bfloat16, false>(encode, g, a, di, st);
    return g.format == SGQ_NVFP4 ? pick<__half, true>(encode, g, a, di, st) : pick<__half, false>(encode, g, a, di, st);
}

}  // namespace sgq
