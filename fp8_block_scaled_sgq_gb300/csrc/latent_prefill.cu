// Expanded latent attention of ragged prompts, for sm_103a.
//
// A CTA takes two tiles of 128 queries of one head and walks over the keys in
// tiles of 128, each tile a pair of MMAs with an fp32 accumulator in TMEM:
//     S [128, 128] = Q K^T   over N + R columns (the R are shared by the heads)
//     O [128, N]  += P V     over 128 keys, P from TMEM (it overlays S)
// Softmax keeps a reference m and a sum l a row: p = 2^(s - m), s in powers of
// two.  m follows the running maximum only when that has grown by more than
// 2^kGrow (lat::Weights), so O is rescaled on few steps; sums are fp32.  P is
// rounded once, to the inputs' type, as the second product's operand; l sums
// the unrounded p.
//
// What bounds it: the tensor cores.  A tile of N + R = 192, N = 128 takes 1280
// cycles of MMAs at full rate; its exponentials take up to 1024 on the special
// function units.  So two query tiles share the CTA: one group of four warps
// does the softmax of its tile while the MMAs of the other run, and each has a
// warp of its own that issues them (one for both left the tensor cores idle in
// its waits).  Warps: 0 and 3 load (keys; values), 1 and 2 issue MMAs, 4 to 7
// and 8 to 11 softmax of a query tile each (thread = query row = TMEM lane).
// Keys and values share a ring of chunks of
// 128 rows x 64 columns: values of a tile arrive while the products before
// them run.
//
// Work: an item is a pair of query tiles of a head.  Heads go in groups whose
// keys and values fit L2 together, a group's items longest first: the last
// items of all are short.  The grid has a CTA for every item, but a CTA that
// runs takes over the next one that has not started yet (cluster launch
// control), asked for late in its item: its loads run ahead into the next one,
// and its barriers and tensor memory stay.
//
// Measured, 4096 tokens x 128 heads, causal, bf16: 427 us in bursts of 20 ms,
// 1610 TFLOP/s (0.87 of the measured bf16 burst rate); 466 to 478 us repeated for
// seconds, where the power limit holds the clock at 1.69 GHz (0.83 to 0.86 of
// what a library product sustains).  On the way, in bursts: CTAs that end with
// their item 492 us; taking over items 469; asking late 453; the order of the
// items 429.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <type_traits>

#include "latent_common.cuh"
#include "latent_ptx.cuh"
#include "sgq_internal.h"

namespace sgq {
namespace {

using lat::Pair;

constexpr int kThreads = 384;
constexpr int kTile = 128;
constexpr int kChunkBytes = kTile * 128;
constexpr int kSlots = 8;
constexpr float kLog2e = 1.44269504088896341f, kLn2 = 0.69314718055994531f;
constexpr int kOffQ = kSlots * kChunkBytes;
constexpr int kOffMisc = kOffQ + 6 * kChunkBytes;
constexpr int kMisc = 2048;
constexpr int kSmem = kOffMisc + kMisc + 1024;   // alignment slack
static_assert(kSmem <= 232448, "shared memory");

struct Args {
    const int32_t* q_starts;
    const int32_t* kv_starts;
    void* out;
    float* lse;
    uint32_t* status;
    int64_t T, S, B;
    int H, N, causal, span_size;
    float scale2;
};

struct Request {
    int q0, n, k0, m;   // queries [q0, q0 + n), keys [k0, k0 + m)
};
// An item: two query tiles of a head, what they see of the request's keys.
struct alignas(16) Item {
    Request r;
    int head, first, count0, count1;   // first query of the pair; key tiles of each query tile (first < r.n: it has rows)
    __device__ __forceinline__ int tiles() const { return max(count0, count1); }
    __device__ __forceinline__ int count(int g) const { return g == 0 ? count0 : count1; }
};
constexpr int64_t kGroupBytes = int64_t(48) << 20;
constexpr int kSpans = 256;
constexpr int kAskBefore = 3;          // tiles before an item's end at which its loader asks for another
struct Shared {
    uint64_t k_full[4], k_empty[4], v_full[4], v_empty[4];   // of the CTA's tile T: entry T % 4
    uint64_t q_full[2], q_empty[2], s_full[2], p_full[2], o_full[2], turn[2];
    uint64_t taken, item_full[2], item_empty[2], drain;
    alignas(16) uint32_t answer[4];    // to the request for another item
    Item item[2];                      // the CTA's items, in turn
    uint32_t tmem, abort;
    int64_t warp_sum[kThreads / 32];
    int span[kSpans];                  // items up to the end of each span of a.span_size requests
};
static_assert(sizeof(Shared) <= kMisc, "barriers");

__device__ __forceinline__ Request request(const Args& a, int64_t b, bool report) {
    const int64_t qs = a.q_starts[b], qe = a.q_starts[b + 1], ks = a.kv_starts[b], ke = a.kv_starts[b + 1];
    const int64_t q0 = min(max(qs, int64_t(0)), a.T), q1 = min(max(qe, q0), a.T);
    const int64_t k0 = min(max(ks, int64_t(0)), a.S), k1 = min(max(ke, k0), a.S);
    if (report && (q0 != qs || q1 != qe || k0 != ks || k1 != ke || (b == 0 && (qs != 0 || ks != 0)) ||
                   (b == a.B - 1 && (qe != a.T || ke != a.S))))
        atomicOr(a.status, kStatusBadValue);
    return Request{static_cast<int>(q0), static_cast<int>(q1 - q0), static_cast<int>(k0), static_cast<int>(k1 - k0)};
}

// Items of a request, and the prefix sums of all of them by spans of
// span_size requests; every thread takes part.  (The host has checked
// that an upper bound of the items fits 31 bits.)
__device__ __forceinline__ int items_of(const Args& a, const Request& r) { return (r.n + 2 * kTile - 1) / (2 * kTile) * a.H; }
__device__ __forceinline__ void sum_items(const Args& a, Shared& sh) {
    const int64_t b0 = min(a.B, int64_t(threadIdx.x) * a.span_size), b1 = min(a.B, b0 + a.span_size);
    int64_t scan = 0;   // (starts that do not rise are reported, and may make more items than there are CTAs)
    if (threadIdx.x < kSpans)
        for (int64_t i = b0; i < b1; ++i) scan += items_of(a, request(a, i, blockIdx.x == 0));
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t up = __shfl_up_sync(0xFFFFFFFFu, scan, o);
        if (lane >= o) scan += up;
    }
    if (lane == 31) sh.warp_sum[warp] = scan;
    __syncthreads();
    for (int w = 0; w < warp; ++w) scan += sh.warp_sum[w];
    if (threadIdx.x < kSpans) sh.span[threadIdx.x] = static_cast<int>(min(scan, int64_t(INT32_MAX)));
    __syncthreads();
}

// (Past the last item, where the grid is an upper bound: an item without rows.)
__device__ __forceinline__ Item find_item(const Args& a, const Shared& sh, int index) {
    Item it{Request{0, 0, 0, 0}, 0, 0, 0, 0};
    if (index >= sh.span[kSpans - 1]) return it;
    int lo = 0, hi = kSpans - 1;   // the first span that ends past the index
    while (lo < hi) {
        const int mid = (lo + hi) / 2;
        if (sh.span[mid] > index) hi = mid;
        else lo = mid + 1;
    }
    int at = lo > 0 ? sh.span[lo - 1] : 0;
    int64_t b = int64_t(lo) * a.span_size;
    for (; b < a.B; ++b) {
        it.r = request(a, b, false);
        const int n = items_of(a, it.r);
        if (index - at < n) break;
        at += n;
    }
    if (b >= a.B) return Item{Request{0, 0, 0, 0}, 0, 0, 0, 0};
    const int blocks = (it.r.n + 2 * kTile - 1) / (2 * kTile);
    // Heads in groups whose keys and values stay in L2 together; a group's items longest first, so that
    // the last ones are short.
    const int64_t head_bytes = int64_t(max(it.r.m, 1)) * 4 * a.N;
    const int most = static_cast<int>(max(int64_t(1), min(int64_t(a.H), kGroupBytes / head_bytes)));
    const int groups = (a.H + most - 1) / most, size = (a.H + groups - 1) / groups;
    const int group = (index - at) / (size * blocks), in = index - at - group * size * blocks;
    const int heads = min(size, a.H - group * size), nth = in / heads;
    it.head = group * size + in - nth * heads;
    it.first = (blocks - 1 - nth) * 2 * kTile;
#pragma unroll
    for (int g = 0; g < 2; ++g) {
        const int first = it.first + g * kTile, last = min(first + kTile, it.r.n) - 1;
        const int seen = first >= it.r.n ? 0 : (a.causal ? max(0, it.r.m - it.r.n + last + 1) : it.r.m);
        (g == 0 ? it.count0 : it.count1) = (seen + kTile - 1) / kTile;
    }
    return it;
}

// VC: chunks of 64 columns of the values (N / 64).  kStall: testing; CTA 0 never loads the keys of its second tile,
// and waits give up early.
template <typename T, int VC, bool kStall>
__global__ void __launch_bounds__(kThreads, 1)
    latent_prefill_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                          const __grid_constant__ CUtensorMap tm_r, const __grid_constant__ CUtensorMap tm_v, const Args a) {
    constexpr bool kBf16 = std::is_same<T, __nv_bfloat16>::value;
    constexpr float kLift = lat::Weights<T>::kLift, kMost = kLift + lat::Weights<T>::kGrow;   // powers of two of the weights
    // A tile's chunks follow one another in the ring: KC of keys (the rotated part last), then VC of
    // values.  Tile t's keys take the slots of what was loaded up to the values of tile t - kBackK,
    // its values those up to the keys of tile t - kBackV.
    constexpr int KC = VC + 1, kPer = KC + VC;
    constexpr int kBackK = VC == 2 ? 2 : 3, kBackV = VC == 2 ? 1 : 2;
    // (chunks from the first one still needed to the last one loaded, both included)
    static_assert((kBackK - 1) * kPer + KC <= kSlots && kBackV * kPer - KC + kPer <= kSlots, "the ring holds what is needed");
    extern __shared__ uint8_t raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
    Shared& sh = *reinterpret_cast<Shared*>(smem + kOffMisc);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const lat::Sync<kStall ? lat::kTestTimeoutClocks : lat::kTimeoutClocks> sync{&sh.abort, a.status};
    auto bar = [](uint64_t& b) { return ptx::smem_u32(&b); };
    const uint32_t s_ring = ptx::smem_u32(smem), s_q = s_ring + kOffQ;

    if (threadIdx.x == 0) {
        for (int i = 0; i < 4; ++i) {
            ptx::mbar_init(bar(sh.k_full[i]), 1);
            ptx::mbar_init(bar(sh.k_empty[i]), 2);   // a commit of each issuing warp
            ptx::mbar_init(bar(sh.v_full[i]), 1);
            ptx::mbar_init(bar(sh.v_empty[i]), 2);
        }
        ptx::mbar_init(bar(sh.taken), 1);
        for (int g = 0; g < 2; ++g) {
            ptx::mbar_init(bar(sh.item_full[g]), 1);
            ptx::mbar_init(bar(sh.item_empty[g]), kThreads / 32 - 1);
            ptx::mbar_init(bar(sh.q_full[g]), 1);
            ptx::mbar_init(bar(sh.q_empty[g]), 1);
            ptx::mbar_init(bar(sh.s_full[g]), 1);
            ptx::mbar_init(bar(sh.p_full[g]), 4);
            ptx::mbar_init(bar(sh.turn[g]), 1);
            ptx::mbar_init(bar(sh.o_full[g]), 1);
        }
        ptx::mbar_init(bar(sh.drain), 2);
        sh.abort = 0;
        ptx::fence_mbar_init();
        ptx::prefetch_tmap(&tm_q);
        ptx::prefetch_tmap(&tm_k);
        ptx::prefetch_tmap(&tm_r);
        ptx::prefetch_tmap(&tm_v);
    }
    if (warp == 1) {
        ptx::tmem_alloc(ptx::smem_u32(&sh.tmem), 512);
        ptx::tmem_relinquish();
    }
    ptx::launch_dependents();
    ptx::grid_dependency_wait();
    ptx::tc_fence_before();
    sum_items(a, sh);
    ptx::tc_fence_after();
    const uint32_t tmem = sh.tmem;
    // TMEM columns: S (and P) of the two query tiles at 0 and 128, O at 256 and 384.

    // Warp 0 finds the CTA's items and leaves them in sh.item, entry `number` % 2 (first < 0: no more);
    // the other warps take them from there.  False: no more, or a wait ran out.
    int number = 0;
    auto next_item = [&](Item& it) {
        const int e = number & 1;
        if (!lat::wait_warp(bar(sh.item_full[e]), (number >> 1) & 1, sync)) return false;
        it = sh.item[e];
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(bar(sh.item_empty[e]));
        ++number;
        return it.first >= 0;
    };
    Item it;
    uint32_t kt = 0;                                       // key tiles so far
    uint32_t q_used[2] = {0, 0};                           // query tiles loaded
    bool ok = true;
    if (warp == 0) {
        // ------------------------------------------------------------ loads: queries, keys
        uint32_t index = blockIdx.x;
        bool more = true;
        do {
            const int e = number & 1;
            ok = lat::wait_warp(bar(sh.item_empty[e]), ((number >> 1) & 1) ^ 1, sync);
            if (!ok) break;
            if (more) it = find_item(a, sh, static_cast<int>(index));
            else it.first = -1;
            if (lane == 0) {
                sh.item[e] = it;
                ptx::mbar_arrive(bar(sh.item_full[e]));
            }
            __syncwarp();
            ++number;
            if (!more) break;
            const int tiles = it.tiles();
            auto q_tile = [&](int g) {
                if (!ok || it.count(g) == 0) return;
                ok = lat::wait_warp(bar(sh.q_empty[g]), (q_used[g] & 1u) ^ 1u, sync);
                if (!ok) return;
                if (lane == 0) {
                    ptx::mbar_arrive_expect_tx(bar(sh.q_full[g]), KC * kChunkBytes);
#pragma unroll
                    for (int c = 0; c < KC; ++c)
                        lat::tma_load_3d(s_q + (g * 3 + c) * kChunkBytes, &tm_q, c * 64, it.head, it.r.q0 + it.first + g * kTile,
                                         bar(sh.q_full[g]));
                }
                __syncwarp();
                ++q_used[g];
            };
            // Asked late in the item, so that a CTA that is nearly done gets the next one; answered by its end.
            auto ask = [&]() {
                if (lane == 0) {
                    ptx::mbar_arrive_expect_tx(bar(sh.taken), 16);
                    lat::take_item(ptx::smem_u32(sh.answer), bar(sh.taken));
                }
                __syncwarp();
            };
            if (tiles == 0) ask();
            q_tile(1);   // (the one with the most keys first)
#pragma unroll 1
            for (int t = 0; t < tiles && ok; ++t, ++kt) {
                if (t == max(0, tiles - kAskBefore)) ask();
                const uint32_t n = kt * kPer, back = kt - kBackK;
                const int row = it.r.k0 + t * kTile;
                // (the first chunk's slot held the last keys of the tile kBackK before, the others' its values)
                const uint32_t full = bar(sh.k_full[kt & 3]);
                if (kt >= kBackK) ok = lat::wait_warp(bar(sh.k_empty[back & 3]), (back >> 2) & 1, sync);
                if (!ok) break;
                if (kStall && blockIdx.x == 0 && kt == 1) continue;
                if (lane == 0) {
                    ptx::mbar_arrive_expect_tx(full, KC * kChunkBytes);
                    lat::tma_load_3d(s_ring + (n % kSlots) * kChunkBytes, &tm_k, 0, it.head, row, full);
                }
                __syncwarp();
                if (kt >= kBackK) ok = lat::wait_warp(bar(sh.v_empty[back & 3]), (back >> 2) & 1, sync);
                if (lane == 0 && ok) {
#pragma unroll
                    for (int c = 1; c < VC; ++c) lat::tma_load_3d(s_ring + ((n + c) % kSlots) * kChunkBytes, &tm_k, c * 64, it.head, row, full);
                    ptx::tma_load_2d(s_ring + ((n + VC) % kSlots) * kChunkBytes, &tm_r, 0, row, full);
                }
                __syncwarp();
                if (t == 0) q_tile(0);
            }
            ok = ok && lat::wait_warp(bar(sh.taken), (number - 1) & 1, sync);
            more = ok && lat::taken_item(ptx::smem_u32(sh.answer), index);
            ptx::fence_proxy_async_smem();              // (the answer has been read before the next one is asked for)
            __syncwarp();
        } while (ok);
    } else if (warp == 3) {
        // ------------------------------------------------------------ loads: values
        while (ok && next_item(it)) {
            const int tiles = it.tiles();
#pragma unroll 1
            for (int t = 0; t < tiles; ++t, ++kt) {
                const uint32_t n = kt * kPer + KC, back = kt - kBackV;
                if (kt >= kBackV) ok = lat::wait_warp(bar(sh.k_empty[back & 3]), (back >> 2) & 1, sync);
                if (!ok) break;
                if (lane == 0) {
                    const uint32_t full = bar(sh.v_full[kt & 3]);
                    ptx::mbar_arrive_expect_tx(full, VC * kChunkBytes);
#pragma unroll
                    for (int c = 0; c < VC; ++c)
                        lat::tma_load_3d(s_ring + ((n + c) % kSlots) * kChunkBytes, &tm_v, c * 64, it.head, it.r.k0 + t * kTile, full);
                }
                __syncwarp();
            }
        }
    } else if (warp < 3) {
        // ------------------------------------------------------------ MMAs
        constexpr uint32_t kIdS = lat::idesc_f16(128, kTile, kBf16, false, false);
        constexpr uint32_t kIdO = lat::idesc_f16(128, VC * 64, kBf16, false, true);
        constexpr uint32_t kIdO64 = lat::idesc_f16(128, 64, kBf16, false, true);
        constexpr uint32_t kHi = lat::desc_hi(1024, ptx::kLayoutSw128), kChunk = kChunkBytes >> 4;
        const uint32_t lo_k = lat::uniform(lat::desc_lo(s_ring, 16)), lo_v = lat::uniform(lat::desc_lo(s_ring, kChunkBytes));
        const uint32_t lo_q = lat::uniform(lat::desc_lo(s_q, 16)), t_s = lat::uniform(tmem);
        auto scores = [&](int g, uint32_t n) {   // S of query tile g, keys in chunks n ... (zero from R columns on)
#pragma unroll
            for (int c = 0; c < KC; ++c)
                lat::mma4_f16<2, 2>(t_s + g * 128, lo_q + (g * 3 + c) * kChunk, kHi, lo_k + ((n + c) % kSlots) * kChunk, kHi, kIdS, c > 0);
            ptx::commit_elect(bar(sh.s_full[g]));
        };
        auto product = [&](int g, uint32_t n, uint32_t more) {   // O of query tile g, values in chunks n ...
            const uint32_t o = t_s + 256 + g * 128, p = t_s + g * 128, d0 = lo_v + n * kChunk;
            if (VC == 1 || n + 1 < kSlots) {
                lat::mma4_f16_ts<128>(o, p, d0, kHi, kIdO, more);
                lat::mma4_f16_ts<128>(o, p + 32, d0 + 512, kHi, kIdO, 1u);
            } else {   // the two chunks at the ring's two ends
                lat::mma4_f16_ts<128>(o, p, d0, kHi, kIdO64, more);
                lat::mma4_f16_ts<128>(o, p + 32, d0 + 512, kHi, kIdO64, 1u);
                lat::mma4_f16_ts<128>(o + 64, p, lo_v, kHi, kIdO64, more);
                lat::mma4_f16_ts<128>(o + 64, p + 32, lo_v + 512, kHi, kIdO64, 1u);
            }
        };
        const int g = lat::uniform(warp - 1);
        uint32_t p_used = 0;
        while (ok && next_item(it)) {
            const int tiles = it.tiles(), mine = it.count(g);
            if (tiles == 0) continue;
            ok = lat::wait_warp(bar(sh.k_full[kt & 3]), (kt >> 2) & 1, sync);
            if (ok && mine > 0) {
                ok = lat::wait_warp(bar(sh.q_full[g]), q_used[0] & 1u, sync);
                if (!ok) break;
                ++q_used[0];
                scores(g, lat::uniform(kt * kPer % kSlots));
                if (mine == 1) ptx::commit_elect(bar(sh.q_empty[g]));
            }
            if (!ok) break;
            ptx::commit_elect(bar(sh.k_empty[kt & 3]));
#pragma unroll 1
            for (int t = 0; t < tiles; ++t, ++kt) {
                // This tile's values, the next one's keys.  A tile that this query tile does not see is waited
                // for all the same before its release, so that no warp releases a slot's next use early.
                const uint32_t nv = lat::uniform((kt * kPer + KC) % kSlots), nk = lat::uniform((kt + 1) * kPer % kSlots);
                ok = lat::wait_warp(bar(sh.v_full[kt & 3]), (kt >> 2) & 1, sync);
                if (ok && t < mine) ok = lat::wait_warp(bar(sh.p_full[g]), p_used++ & 1u, sync);
                // The issuing warps take turns, the second query tile's first: MMAs of both at once would
                // make both query tiles wait, instead of one of them doing its softmax meanwhile.
                if (ok && (g == 0 || kt > 0)) ok = lat::wait_warp(bar(sh.turn[g]), (g == 0 ? kt : kt - 1) & 1u, sync);
                if (!ok) break;
                if (t < mine) {
                    ptx::tc_fence_after();
                    product(g, nv, lat::uniform(t > 0 ? 1u : 0u));
                    if (t + 1 == mine) ptx::commit_elect(bar(sh.o_full[g]));
                }
                ptx::commit_elect(bar(sh.v_empty[kt & 3]));
                if (t + 1 < tiles) {
                    ok = lat::wait_warp(bar(sh.k_full[(kt + 1) & 3]), ((kt + 1) >> 2) & 1, sync);
                    if (!ok) break;
                    if (t + 1 < mine) scores(g, nk);
                    if (t + 2 == mine) ptx::commit_elect(bar(sh.q_empty[g]));
                    ptx::commit_elect(bar(sh.k_empty[(kt + 1) & 3]));
                }
                if (lane == 0) ptx::mbar_arrive(bar(sh.turn[1 - g]));
                __syncwarp();
            }
        }
    } else {
        // ------------------------------------------------------------ softmax
        const int g = (warp - 4) >> 2, quarter = warp & 3;
        const int row = quarter * 32 + lane;
        const uint32_t t_s = tmem + (static_cast<uint32_t>(quarter * 32) << 16) + g * 128, t_o = t_s + 256;
        uint32_t s_used = 0, o_used = 0;
        while (ok && next_item(it)) {
            const Request& r = it.r;
            const int q = it.first + g * kTile + row;                  // query of the request
            const int mine = it.count(g);
            if (it.first + g * kTile < r.n) {
                const int sees = a.causal ? min(r.m, r.m - r.n + q + 1) : r.m;
                const int low = a.causal ? r.m - r.n + q - lane + 1 : r.m;   // what every row of the warp sees
                float ref = -INFINITY, l = 0.0f;
#pragma unroll 1
                for (int t = 0; t < mine; ++t) {
                    ok = lat::wait_warp(bar(sh.s_full[g]), s_used++ & 1u, sync);
                    if (!ok) break;
                    ptx::tc_fence_after();
                    // the second half arrives while the first one's maximum is taken
                    uint32_t s[4][32];
                    ptx::tmem_ld<32>(t_s, s[0]);
                    ptx::tmem_ld<32>(t_s + 32, s[1]);
                    ptx::tmem_wait_ld();
                    ptx::tmem_ld<32>(t_s + 64, s[2]);
                    ptx::tmem_ld<32>(t_s + 96, s[3]);
                    const bool edge = (t + 1) * kTile > low || (t + 1) * kTile > r.m;
                    const int end = sees - t * kTile;
                    float tops[4];
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        if (h == 1) ptx::tmem_wait_ld();
                        if (edge) {
#pragma unroll
                            for (int c = 2 * h; c < 2 * h + 2; ++c)
#pragma unroll
                                for (int j = 0; j < 32; ++j)
                                    if (c * 32 + j >= end) s[c][j] = __float_as_uint(-INFINITY);
                        }
#pragma unroll
                        for (int c = 2 * h; c < 2 * h + 2; ++c) {
                            tops[c] = __uint_as_float(s[c][0]);
#pragma unroll
                            for (int j = 1; j < 32; ++j) tops[c] = fmaxf(tops[c], __uint_as_float(s[c][j]));
                        }
                    }
                    const float top = fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3])) * a.scale2;
                    const bool grow = top > ref + kMost || (ref == -INFINITY && top > -INFINITY);
                    if (__any_sync(0xFFFFFFFFu, grow)) {
                        const float to = top - kLift, f = grow ? lat::ex2(ref - to) : 1.0f;
                        if (grow) ref = to;
                        l *= f;
                        if (t > 0) {
#pragma unroll 1
                            for (int c = 0; c < VC * 8; ++c) {
                                uint32_t o[8];
                                ptx::tmem_ld<8>(t_o + c * 8, o);
                                ptx::tmem_wait_ld();
#pragma unroll
                                for (int j = 0; j < 8; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * f);
                                lat::tmem_st<8>(t_o + c * 8, o);
                            }
                        }
                    }
                    const float base = ref == -INFINITY ? 0.0f : ref;
                    const float2 scale = make_float2(a.scale2, a.scale2), minus = make_float2(-base, -base);
                    float2 sum[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        uint32_t p[16];
#pragma unroll
                        for (int j = 0; j < 32; j += 2) {
                            float2 x = make_float2(__uint_as_float(s[c][j]), __uint_as_float(s[c][j + 1]));
                            x = lat::fma2(x, scale, minus);
                            x.x = lat::ex2(x.x);
                            x.y = lat::ex2(x.y);
                            sum[(j >> 1) & 1] = lat::add2(sum[(j >> 1) & 1], x);
                            p[j / 2] = Pair<T>::pack(x.x, x.y);
                        }
                        lat::tmem_st<16>(t_s + c * 16, p);
                    }
                    l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
                    // Weights past the request's keys are zero, but 0 times what lies there need not be: each
                    // group clears those rows of the values before its own product.
                    if ((t + 1) * kTile > r.m) {
                        ok = lat::wait_warp(bar(sh.v_full[(kt + t) & 3]), ((kt + t) >> 2) & 1, sync);
                        if (!ok) break;
                        if (t * kTile + row >= r.m) {
#pragma unroll
                            for (int c = 0; c < VC; ++c) {
                                uint4* z = reinterpret_cast<uint4*>(smem + (((kt + t) * kPer + KC + c) % kSlots) * kChunkBytes + row * 128);
#pragma unroll
                                for (int i = 0; i < 8; ++i) z[i] = make_uint4(0, 0, 0, 0);
                            }
                        }
                        ptx::fence_proxy_async_smem();
                    }
                    lat::tmem_wait_st();
                    ptx::tc_fence_before();
                    __syncwarp();
                    if (lane == 0) ptx::mbar_arrive(bar(sh.p_full[g]));
                }
                if (ok && mine > 0) {
                    ok = lat::wait_warp(bar(sh.o_full[g]), o_used++ & 1u, sync);
                    ptx::tc_fence_after();
                }
                if (ok) {
                    const float inv = l == 0.0f ? 0.0f : 1.0f / l;   // (0: nothing seen; NaN stays NaN)
                    const int64_t at = (int64_t(r.q0) + q) * a.H + it.head;
                    if (a.lse != nullptr && q < r.n) a.lse[at] = l == 0.0f ? -INFINITY : (ref + log2f(l)) * kLn2;
                    uint4* out = reinterpret_cast<uint4*>(static_cast<T*>(a.out) + at * a.N);
                    const bool wide = (reinterpret_cast<uintptr_t>(a.out) & 31u) == 0;
#pragma unroll 1
                    for (int c = 0; c < VC * 2; ++c) {
                        uint32_t o[32];
                        if (mine > 0) {
                            ptx::tmem_ld<32>(t_o + c * 32, o);
                            ptx::tmem_wait_ld();
                        } else {
#pragma unroll
                            for (int j = 0; j < 32; ++j) o[j] = 0u;
                        }
                        if (q < r.n) {
                            uint32_t w[16];
#pragma unroll
                            for (int j = 0; j < 16; ++j)
                                w[j] = Pair<T>::pack(__uint_as_float(o[2 * j]) * inv, __uint_as_float(o[2 * j + 1]) * inv);
                            if (wide) {   // a row a thread: whole sectors of 32 bytes
                                ptx::st_global_v8(out + c * 4, *reinterpret_cast<uint32_t (*)[8]>(w));
                                ptx::st_global_v8(out + c * 4 + 2, *reinterpret_cast<uint32_t (*)[8]>(w + 8));
                            } else {
#pragma unroll
                                for (int i = 0; i < 4; ++i) out[c * 4 + i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
                            }
                        }
                    }
                }
                ptx::tc_fence_before();
            }
            kt += it.tiles();
        }
    }
    __syncthreads();
    if (sh.abort) {
        // A wait ran out: copies in flight land and MMAs end (both bounded) before the CTA does.
        const uint64_t t0 = ptx::globaltimer();
        auto land = [&](uint64_t& x, uint32_t uses) {
            while (uses > 0 && !ptx::mbar_test_wait(bar(x), (uses - 1) & 1u) && ptx::globaltimer() - t0 < (1ull << 26)) {}
        };
        if (warp == 0 || warp == 3) {
            for (uint32_t i = 0; i < 4; ++i) land(warp == 0 ? sh.k_full[i] : sh.v_full[i], kt / 4 + (i < kt % 4 ? 1 : 0));
            if (warp == 0) {
                land(sh.q_full[0], q_used[0]);
                land(sh.q_full[1], q_used[1]);
                land(sh.taken, number);
            }
        } else if (threadIdx.x == 32 || threadIdx.x == 64) {
            ptx::tc_commit(bar(sh.drain));
            land(sh.drain, 1);
        }
        __syncthreads();
    }
    if (warp == 1) {
        ptx::tc_fence_after();
        ptx::tmem_dealloc(tmem, 512);
    }
}

// ---------------------------------------------------------------- host

// [rows, heads, width] as boxes of 64 columns x 128 rows of one head.
sgq_status head_map(gemm::TensorMapEncoder encode, CUtensorMap* m, const void* p, int64_t width, int64_t heads, int64_t rows, int64_t s_head,
                    int64_t s_row) {
    if (heads == 1) s_head = width;   // (a dimension of one entry has no stride that counts)
    if (rows == 1) s_row = width;
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(width), static_cast<cuuint64_t>(heads), static_cast<cuuint64_t>(rows)};
    const cuuint64_t strides[2] = {static_cast<cuuint64_t>(s_head) * 2, static_cast<cuuint64_t>(s_row) * 2};
    const cuuint32_t box[3] = {64, 1, kTile}, ones[3] = {1, 1, 1};
    return encode(m, CU_TENSOR_MAP_DATA_TYPE_UINT16, 3, const_cast<void*>(p), dims, strides, box, ones,
                     CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
               ? SGQ_OK
               : SGQ_ERR_CUDA;
}
sgq_status row_map(gemm::TensorMapEncoder encode, CUtensorMap* m, const void* p, int64_t width, int64_t rows, int64_t s_row) {
    if (rows == 1) s_row = width;
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(width), static_cast<cuuint64_t>(rows)};
    const cuuint64_t strides[1] = {static_cast<cuuint64_t>(s_row) * 2};
    const cuuint32_t box[2] = {64, kTile}, ones[2] = {1, 1};
    return encode(m, CU_TENSOR_MAP_DATA_TYPE_UINT16, 2, const_cast<void*>(p), dims, strides, box, ones,
                     CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
               ? SGQ_OK
               : SGQ_ERR_CUDA;
}

template <typename T, int VC, bool kStall = false>
sgq_status run(const CUtensorMap (&tm)[4], const Args& a, int64_t grid, cudaStream_t st) {
    auto kern = latent_prefill_kernel<T, VC, kStall>;
    static bool configured[64] = {};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return SGQ_ERR_CUDA;
    if (!configured[dev]) {
        if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem) != cudaSuccess) return SGQ_ERR_CUDA;
        configured[dev] = true;
    }
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(grid));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kSmem;
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, kern, tm[0], tm[1], tm[2], tm[3], a) != cudaSuccess) return SGQ_ERR_CUDA;
    note_launch();
    return SGQ_OK;
}

}  // namespace

sgq_status launch_latent_prefill(const PrefillArgs& x, cudaStream_t st) {
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
    a.q_starts = x.q_starts;
    a.kv_starts = x.kv_starts;
    a.out = x.out;
    a.lse = x.lse;
    a.T = x.T;
    a.S = x.S;
    a.B = x.B;
    a.H = x.H;
    a.N = x.N;
    a.causal = x.causal;
    a.scale2 = x.scale * kLog2e;
    a.span_size = static_cast<int>((x.B + kSpans - 1) / kSpans);
    const int64_t blocks = (x.T / (2 * kTile) + x.B) * x.H;   // at least the query tile pairs of any split of T
    if (blocks > INT32_MAX) return SGQ_ERR_INVALID_ARG;
    CUtensorMap tm[4];
    // (without keys nothing is loaded through the maps of keys and values: any address does)
    const bool none = x.S == 0;
    const int64_t W = x.N + x.R, S = none ? 1 : x.S;
    if (head_map(encode, &tm[0], x.q, W, x.H, x.T, x.q_h, x.q_t) != SGQ_OK ||
        head_map(encode, &tm[1], none ? x.q : x.k, x.N, x.H, S, none ? x.q_h : x.k_h, none ? x.q_t : x.k_t) != SGQ_OK ||
        row_map(encode, &tm[2], none ? x.q : x.k_rot, x.R, S, none ? x.q_t : x.kr_t) != SGQ_OK ||
        head_map(encode, &tm[3], none ? x.q : x.v, x.N, x.H, S, none ? x.q_h : x.v_h, none ? x.q_t : x.v_t) != SGQ_OK)
        return SGQ_ERR_CUDA;
    if (x.stall) return x.N == 128 ? run<__nv_bfloat16, 2, true>(tm, a, blocks, st) : run<__nv_bfloat16, 1, true>(tm, a, blocks, st);
    if (x.N == 128)
        return x.dtype == SGQ_BF16 ? run<__nv_bfloat16, 2>(tm, a, blocks, st) : run<__half, 2>(tm, a, blocks, st);
    return x.dtype == SGQ_BF16 ? run<__nv_bfloat16, 1>(tm, a, blocks, st) : run<__half, 1>(tm, a, blocks, st);
}

}  // namespace sgq
