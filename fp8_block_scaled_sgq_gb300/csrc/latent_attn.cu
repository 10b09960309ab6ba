// Absorbed latent attention over a paged cache, for sm_103a.
//
// All heads and all new tokens of a request read the same rows c_j of the
// cache, so a block of `NR` (token, head) rows q_i and a tile of 128 cached
// rows make two matrix products, written with the cache on the MMA's 128-row
// side and the queries on its N side (so few heads cost few columns):
//     S^T [128 tokens, NR] = C Q^T          over L + R columns
//     O^T [L, NR]         += C[:, :L]^T P^T over 128 tokens
// Softmax keeps a reference m and a sum l for every row i: p = 2^(s - m)
// with s in powers of two.  m follows the running maximum only when that has
// grown by more than 2^kGrow (lat::Weights): every sum is a sum of positive
// terms in fp32 with the same reference, and the accumulator in TMEM is
// rescaled only on those steps.  P is rounded once, to the cache's type, as the
// second product's operand; l sums the unrounded p.
//
// What bounds it.  A tile is 147 KB of cache (L + R = 576) and takes 68 steps
// of MMAs, of 40 cycles (NR = 16) to 49 (NR = 64, the operands' reads of shared
// memory).  With 16 rows a tile's MMAs and softmax take less than its share of
// HBM time, and HBM is the bound once a CTA is under way: 64 sequences of 130
// to 16384 rows with 16 heads (200 MB) in 49 us, of which 30 are the bytes at
// the measured copy rate and 7 the joining kernel and its launch.  With 64
// rows it is shared memory: reads by the MMAs and writes by TMA take 4470
// cycles a tile at least.  Only the tile in use fits beside the queries, so
// shared memory idles while softmax runs between the two products: 5250 cycles
// a tile.  128 sequences of 1024 to 8192 rows with 128 heads: 164 us (538 MB);
// one of 131071 rows: 69 us (151 MB); chunks: 373 us (728 TFLOP/s).  Between
// items code runs that a CTA executes once an item, and it comes cold (a
// hundred instructions take some 1000 cycles), so it is kept short.
//
// Layout.  A tile sits in shared memory once, as chunks of 128 rows x 64
// columns with 128-byte swizzle: read K-major for S^T and, by the descriptor's
// other operand order, MN-major for O^T.  Chunks of the latent part come in
// pairs (128 columns, one MMA's M) through a ring; the rotated part has a slot
// of its own, which takes P once S^T is done.  Warps: 0 issues MMAs, 1 to 3
// load (TMA, one box a run of rows inside a page), the others do softmax:
// thread = token, groups of four warps with a share of the columns each.
//
// Work: the tiles of all (request, row block) items, in order, are cut into
// equal runs, one a CTA, from the lengths on the device; an item counts
// kItemCost tiles more than it has, which is what starting and ending one
// takes.  An item that a cut splits leaves fp32 partial sums, which a second
// kernel joins in order: the result does not depend on timing.
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

constexpr int kTile = 128;                    // cached rows a tile
constexpr int kChunkBytes = kTile * 128;      // 64 columns of a tile
constexpr int kMaxPairs = 5, kMaxRope = 2;
constexpr int kLoaders = 3;                   // warps that issue loads: one alone keeps a third of this rate
constexpr int kItemCost = 2;                  // tiles that an item's start and end cost (chunks, 128 heads: 1 377 us, 2 373, 3 387; 128 requests: 168.5, 164.7, 163.3)
constexpr float kLog2e = 1.44269504088896341f, kLn2 = 0.69314718055994531f;
constexpr float kNone = -1.0e38f;             // reference of a row that has seen nothing

template <int NR>
struct Cfg {
    static constexpr int kPairs = NR == 64 ? 4 : 5;
    static constexpr int kRope = NR == 16 ? 2 : 1;
    static constexpr int kQChunk = NR * 128;
    static constexpr int kOffRope = kPairs * 2 * kChunkBytes;
    static constexpr int kOffQ = kOffRope + kRope * kChunkBytes;
    static constexpr int kOffMisc = kOffQ + 9 * kQChunk;
    static constexpr int kMisc = 3584;                     // barriers, schedule, statistics
    static constexpr int kSmem = kOffMisc + kMisc + 1024;  // alignment slack
    static constexpr int kGroups = NR == 64 ? 4 : 2;       // groups of four softmax warps, a share of the columns each
    static constexpr int kThreads = 128 + kGroups * 128;
    static constexpr int kHC = NR / kGroups;               // columns a softmax warp
    static constexpr int kRowBytes = NR * 2;               // a token's row of P
    static constexpr uint32_t kColS = 4 * NR;
    static_assert(kSmem <= 232448, "shared memory");
};

struct Args {
    const char* cache;
    const int32_t* table;
    const int32_t* kv_lens;
    const int32_t* q_starts;
    void* out;
    float* lse;
    float* partial;      // [2 grid][NR][L]
    float2* stats;       // [2 grid][NR]: reference, sum
    int4* joins;         // [grid]: first row, rows, parts (0: nothing to join)
    uint32_t* status;
    int64_t T, B, pages, width, c_page, c_row;   // strides in bytes
    uint32_t box_bytes;                          // a box's span, fetched ahead into L2 (0: not)
    int H, L, page, box;
    int tpn, hb;         // tokens a block, head blocks a token (one of them is 1)
    uint64_t inv_teams;  // 2^64 / teams, rounded up
    int team;            // CTAs that walk over the same tiles, a head block each: hb, or 1
    float scale2;        // scale log2(e)
};

// One request: its query tokens [t0, t0 + n) and cached rows m.
struct Request {
    int t0, n, m;
};
__device__ __forceinline__ Request request(const Args& a, int b, bool report) {
    Request r;
    if (a.q_starts == nullptr) {
        r.t0 = b;
        r.n = 1;
    } else {
        const int s = a.q_starts[b], e = a.q_starts[b + 1], T = static_cast<int>(a.T);
        r.t0 = min(max(s, 0), T);
        r.n = min(max(e, r.t0), T) - r.t0;
        if (report && (r.t0 != s || r.t0 + r.n != e || (b == 0 && s != 0) || (b == a.B - 1 && e != a.T)))
            atomicOr(a.status, kStatusBadValue);
    }
    const int m = a.kv_lens[b], most = static_cast<int>(a.width * a.page);
    r.m = min(max(m, 0), most);
    if (report && r.m != m) atomicOr(a.status, kStatusBadValue);
    return r;
}
// Rows of the cache that token t of the request sees, and the tiles of the
// token block i (its last token's rows; at least one tile, so that every item
// is visited and writes its result).
__device__ __forceinline__ int sees(const Request& r, int t) { return max(0, r.m - r.n + t + 1); }
__device__ __forceinline__ int tiles(const Request& r, int tpn, int i) {
    return max(1, (sees(r, min((i + 1) * tpn, r.n) - 1) + kTile - 1) / kTile);
}
// First token block whose tile count exceeds that of block i (or the number of blocks).
__device__ __forceinline__ int next_step(const Request& r, int tpn, int blocks, int c) {
    // block i counts more than c tiles from (i + 1) tpn > 128 c - (m - n) on
    // (c kTile is less than m + kTile, which fits: m is a table's width times its page)
    return min(blocks, max(c * kTile - (r.m - r.n), 0) / tpn);
}
__device__ __forceinline__ int64_t request_tiles(const Request& r, const Args& a) {
    const int blocks = (r.n + a.tpn - 1) / a.tpn;
    int64_t sum = 0;
    for (int i = 0; i < blocks;) {
        const int c = tiles(r, a.tpn, i);
        const int e = max(next_step(r, a.tpn, blocks, c), i + 1);
        sum += int64_t(c + kItemCost) * (e - i);
        i = e;
    }
    return sum * (a.hb / a.team);
}

// A CTA's run: item (b, block, head block), tile `at` of its `count`; a run's
// length counts each item's tiles and then its cost.
// The head blocks of a token read the same tiles: a team of CTAs takes them
// side by side, so that the second read finds them in L2 (read apart, B = 128
// with H = 128 moved 0.99 GB from HBM instead of 0.54).
struct Walk {
    int b, block, hblk, at, count;
    int64_t left;        // length of the run from here on
    Request r;
    __device__ __forceinline__ void settle(const Args& a) { count = tiles(r, a.tpn, block); }
    __device__ __forceinline__ int end() const { return static_cast<int>(min(int64_t(count), at + left)); }
    // The run's next item with tiles in it; false: the run is over.
    __device__ __forceinline__ bool next(const Args& a) {
        left -= count + kItemCost - at;
        if (left <= 0) return false;
        at = 0;
        if (++hblk == a.hb / a.team) {
            hblk = 0;
            if (++block * a.tpn >= r.n) {
                block = 0;
                do {
                    if (++b >= a.B) return false;
                    r = request(a, b, false);
                } while (r.n == 0);
            }
            settle(a);
        }
        return true;
    }
    __device__ __forceinline__ int64_t row0(const Args& a) const {
        return (int64_t(r.t0) + block * a.tpn) * a.H + head_block(a) * ((a.H + a.hb - 1) / a.hb);
    }
    __device__ __forceinline__ int head_block(const Args& a) const {
        return a.team == 1 ? hblk : static_cast<int>(blockIdx.x) % a.team;
    }
    __device__ __forceinline__ int rows(const Args& a) const {
        if (a.hb == 1) return min(a.tpn, r.n - block * a.tpn) * a.H;
        const int per = (a.H + a.hb - 1) / a.hb;
        return min(per, a.H - head_block(a) * per);
    }
};

// What the softmax warps need to know of an item.
struct alignas(16) Item {
    int64_t row0;
    int rows, at, end;   // rows (0: no more items), tiles [at, end)
    int m, n, first;     // the request's cached rows and tokens, the block's first token
    int parts;           // of its result: 1: this is all of it; 0: some other CTA's
};

struct Shared {
    uint64_t full[kMaxPairs], empty[kMaxPairs], rope_full[kMaxRope], rope_empty[kMaxRope];
    uint64_t q_full, q_empty, s_full, p_full, o_full, item_full[2], drain;
    Item item[2];        // the CTA's items, in turn
    uint32_t tmem, abort;
    // the schedule: totals of the threads' requests, then the CTA's start
    int64_t per, total;
    int b, block, hblk, at;
    Request r;
    int64_t warp_sum[20];
    alignas(16) float ref[4][16], fade[4][16];   // [column group][column]: new reference, 2^(old - new)
    float top[4][4][16], sum[4][4][16];          // [column group][lane quarter][column]
    alignas(16) int sees[64];                 // rows of the cache that each column's token sees
};
static_assert(sizeof(Shared) <= Cfg<16>::kMisc, "statistics");

// Where this CTA's run starts; every thread takes part.  Thread i adds up the
// requests [i k, (i + 1) k); the one whose span holds the start walks it again.
template <int kThreads>
__device__ __forceinline__ void plan(const Args& a, Shared& sh) {
    const int B = static_cast<int>(a.B), k = (B - 1) / kThreads + 1;
    const int b0 = static_cast<int>(min(int64_t(B), int64_t(threadIdx.x) * k)), b1 = min(B - b0, k) + b0;
    int64_t mine = 0;
    for (int b = b0; b < b1; ++b) mine += request_tiles(request(a, b, blockIdx.x == 0), a);
    int64_t scan = mine;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t up = __shfl_up_sync(0xFFFFFFFFu, scan, o);
        if (lane >= o) scan += up;
    }
    if (lane == 31) sh.warp_sum[warp] = scan;
    __syncthreads();
    int64_t total = 0;
    for (int w = 0; w < kThreads / 32; ++w) {
        if (w < warp) scan += sh.warp_sum[w];
        total += sh.warp_sum[w];
    }
    const int teams = gridDim.x / a.team;
    const int64_t per = __umul64hi(static_cast<uint64_t>(total + teams - 1), a.inv_teams) + (teams == 1 ? total : 0);   // / teams, exact below 2^40
    const int64_t start = per * (blockIdx.x / a.team);
    int64_t at = scan - mine;
    if (start >= at && start < scan) {
        for (int b = b0; b < b1; ++b) {
            const Request r = request(a, b, false);
            const int64_t n = request_tiles(r, a);
            if (start >= at + n) {
                at += n;
                continue;
            }
            const int blocks = (r.n + a.tpn - 1) / a.tpn;
            int i = 0, c = 1;
            while (i < blocks) {
                c = tiles(r, a.tpn, i);
                const int e = max(next_step(r, a.tpn, blocks, c), i + 1);
                const int64_t span = int64_t(c + kItemCost) * (e - i) * (a.hb / a.team);
                if (start < at + span) break;
                at += span;
                i = e;
            }
            const int64_t item = (start - at) / (c + kItemCost);
            sh.b = b;
            sh.r = r;
            sh.block = i + static_cast<int>(item / (a.hb / a.team));
            sh.hblk = static_cast<int>(item % (a.hb / a.team));
            sh.at = static_cast<int>((start - at) - item * (c + kItemCost));
            break;
        }
    }
    if (threadIdx.x == 0) {
        sh.per = per;
        sh.total = total;
    }
    __syncthreads();
}

// The columns' sums over the 32 lanes, column c of the N in lane c (and c + N ...).
template <int N>
__device__ __forceinline__ float lane_sums(float (&v)[N]) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int o = 16; o >= N; o >>= 1)
#pragma unroll
        for (int j = 0; j < N; ++j) v[j] += __shfl_xor_sync(0xFFFFFFFFu, v[j], o);
#pragma unroll
    for (int o = N / 2; o >= 1; o >>= 1) {
        const bool up = (lane & o) != 0;
#pragma unroll
        for (int j = 0; j < o; ++j) {
            const float send = up ? v[j] : v[j + o];
            const float keep = up ? v[j + o] : v[j];
            v[j] = keep + __shfl_xor_sync(0xFFFFFFFFu, send, o);
        }
    }
    return v[0];
}

// kStall: testing; CTA 0 never loads the first pair of its second tile, and waits give up early.
template <typename T, int NR, bool kStall>
__global__ void __launch_bounds__(Cfg<NR>::kThreads, 1)
    latent_attention_kernel(const __grid_constant__ CUtensorMap tm_cache, const __grid_constant__ CUtensorMap tm_q,
                            const Args a) {
    using C = Cfg<NR>;
    constexpr int HC = C::kHC;
    constexpr bool kBf16 = std::is_same<T, __nv_bfloat16>::value;
    constexpr float kLift = lat::Weights<T>::kLift, kMost = kLift + lat::Weights<T>::kGrow;   // powers of two of the weights
    extern __shared__ uint8_t raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
    Shared& sh = *reinterpret_cast<Shared*>(smem + C::kOffMisc);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const lat::Sync<kStall ? lat::kTestTimeoutClocks : lat::kTimeoutClocks> sync{&sh.abort, a.status};
    auto bar = [](uint64_t& b) { return ptx::smem_u32(&b); };
    const uint32_t s_pairs = ptx::smem_u32(smem), s_rope = s_pairs + C::kOffRope, s_q = s_pairs + C::kOffQ;

    if (threadIdx.x == 0) {
        for (int i = 0; i < C::kPairs; ++i) {
            ptx::mbar_init(bar(sh.full[i]), 1);
            ptx::mbar_init(bar(sh.empty[i]), 1);
        }
        for (int i = 0; i < C::kRope; ++i) {
            ptx::mbar_init(bar(sh.rope_full[i]), 1);
            ptx::mbar_init(bar(sh.rope_empty[i]), 1);
        }
        ptx::mbar_init(bar(sh.q_full), 1);
        ptx::mbar_init(bar(sh.q_empty), 1);
        ptx::mbar_init(bar(sh.s_full), 1);
        ptx::mbar_init(bar(sh.p_full), 4 * C::kGroups);
        ptx::mbar_init(bar(sh.o_full), 1);
        ptx::mbar_init(bar(sh.item_full[0]), 1);
        ptx::mbar_init(bar(sh.item_full[1]), 1);
        ptx::mbar_init(bar(sh.drain), 1);
        sh.abort = 0;
        ptx::fence_mbar_init();
        ptx::prefetch_tmap(&tm_cache);
        ptx::prefetch_tmap(&tm_q);
    }
    if (warp == 0) {
        ptx::tmem_alloc(ptx::smem_u32(&sh.tmem), 512);
        ptx::tmem_relinquish();
    }
    ptx::launch_dependents();
    ptx::grid_dependency_wait();
    ptx::tc_fence_before();
    plan<C::kThreads>(a, sh);
    ptx::tc_fence_after();
    const uint32_t tmem = sh.tmem;
    const int np = a.L / 128;                       // pairs of latent chunks a tile

    if (threadIdx.x == 128) a.joins[blockIdx.x] = make_int4(0, 0, 0, 0);
    Walk w;
    w.left = min(sh.per, sh.total - sh.per * (blockIdx.x / a.team));
    bool any = w.left > 0;
    if (any) {
        w.b = sh.b;
        w.block = sh.block;
        w.hblk = sh.hblk;
        w.at = sh.at;
        w.r = sh.r;
        w.settle(a);
        if (w.at >= w.count) any = w.next(a);       // the run starts in an item's cost
    }

    uint32_t pair = 0, rope = 0, seg = 0;            // slots and segments used so far
    if (warp >= 1 && warp < 1 + kLoaders && any) {
        // ------------------------------------------------------------ loads
        // Pairs go to the loading warps in turn, the rotated parts all to the last one.  A wait for a
        // slot's release tells phases apart by parity, so no loader may be two uses of a slot ahead:
        // the rotated parts' loader waits for every release in order; a loader of pair n has loaded
        // pair n - kLoaders, so pair n - kLoaders - kPairs is released, which is later than the
        // slot's use before the awaited one, n - 2 kPairs.
        static_assert(C::kPairs > kLoaders, "parity of the pairs' releases");
        const int id = warp - 1;
        int turn = 0;
        bool ok = true;
        // Lane i's box of a tile: rows [i box, (i + 1) box), inside one page.
        auto locate = [&](int tile, int& boxes, int& page, int& in_page) {
            const int rows = min(kTile, w.r.m - tile * kTile);
            boxes = rows > 0 ? (rows + a.box - 1) / a.box : 0;
            page = in_page = 0;
            if (lane < boxes) {
                const int j = tile * kTile + lane * a.box, in_table = j / a.page;
                page = __ldg(a.table + int64_t(w.b) * a.width + in_table);
                in_page = j - in_table * a.page;
            }
        };
        do {
            const int end = w.end();
            int boxes, page, in_page, next_boxes = 0, next_page = 0, next_in = 0;
            locate(w.at, boxes, page, in_page);
            if (id == 0) {
                ok = lat::wait_warp(bar(sh.q_empty), (seg & 1u) ^ 1u, sync);
                if (!ok) break;
                if (lane == 0) {
                    ptx::mbar_arrive_expect_tx(bar(sh.q_full), (2 * np + 1) * C::kQChunk);
                    const int row = static_cast<int>(w.row0(a));
#pragma unroll 1
                    for (int c = 0; c <= 2 * np; ++c)
                        ptx::tma_load_2d(s_q + c * C::kQChunk, &tm_q, c * 64, row, bar(sh.q_full));
                }
                __syncwarp();
            }
            ++seg;
#pragma unroll 1
            for (int tile = w.at; tile < end && ok; ++tile) {
                if (lane < boxes && (page < 0 || page >= a.pages)) {   // nowhere: the box past the last page reads as zeros
                    atomicOr(a.status, kStatusBadValue);
                    page = static_cast<int>(a.pages);
                }
                if (tile + 1 < end) locate(tile + 1, next_boxes, next_page, next_in);
                const uint32_t dst = lane * a.box * 128;
#pragma unroll 1
                for (int p = 0; p < np; ++p, ++pair, turn = turn + 1 == kLoaders ? 0 : turn + 1) {
                    if (turn != id) continue;
                    const uint32_t slot = pair % C::kPairs, full = bar(sh.full[slot]);
                    ok = lat::wait_warp(bar(sh.empty[slot]), ((pair / C::kPairs) & 1u) ^ 1u, sync);
                    if (!ok) break;
                    if (kStall && blockIdx.x == 0 && pair == static_cast<uint32_t>(np)) continue;
                    if (lane == 0) ptx::mbar_arrive_expect_tx(full, boxes * a.box * 256);
                    __syncwarp();
                    if (lane < boxes) {
                        const uint32_t to = s_pairs + slot * 2 * kChunkBytes + dst;
                        lat::tma_load_3d(to, &tm_cache, p * 128, in_page, page, full);
                        lat::tma_load_3d(to + kChunkBytes, &tm_cache, p * 128 + 64, in_page, page, full);
                    }
                    __syncwarp();
                }
                if (!ok) break;
                if (id == kLoaders - 1) {
                    const uint32_t slot = rope % C::kRope, full = bar(sh.rope_full[slot]);
                    ok = lat::wait_warp(bar(sh.rope_empty[slot]), ((rope / C::kRope) & 1u) ^ 1u, sync);
                    if (!ok) break;
                    if (lane == 0) ptx::mbar_arrive_expect_tx(full, boxes * a.box * 128);
                    __syncwarp();
                    if (lane < boxes) lat::tma_load_3d(s_rope + slot * kChunkBytes + dst, &tm_cache, a.L, in_page, page, full);
                    __syncwarp();
                }
                ++rope;
                // The next tile goes to L2 while its loads wait for their slots.
                if (id == 0 && a.box_bytes != 0 && tile + 1 < end && lane < next_boxes && next_page >= 0 && next_page < a.pages)
                    lat::bulk_prefetch(a.cache + next_page * a.c_page + next_in * a.c_row, a.box_bytes);
                __syncwarp();
                boxes = next_boxes;
                page = next_page;
                in_page = next_in;
            }
        } while (ok && w.next(a));
    } else if (warp == 0 && any) {
        // ------------------------------------------------------------ MMAs
        constexpr uint32_t kIdS = lat::idesc_f16(128, NR, kBf16, false, false);
        constexpr uint32_t kIdO = lat::idesc_f16(128, NR, kBf16, true, true);
        constexpr uint32_t kHiK = lat::desc_hi(1024, ptx::kLayoutSw128);                               // rows of 128 bytes
        constexpr uint32_t kHiP = lat::desc_hi(8 * C::kRowBytes, lat::layout_of(C::kRowBytes));
        constexpr uint32_t kPair = 2 * kChunkBytes >> 4, kChunk = kChunkBytes >> 4, kQ = C::kQChunk >> 4;
        constexpr int kStepP = C::kRowBytes;                       // 16 tokens of P, in units of 16 bytes
        const uint32_t lo_k = lat::uniform(lat::desc_lo(s_pairs, 16)), lo_v = lat::uniform(lat::desc_lo(s_pairs, kChunkBytes));
        const uint32_t lo_r = lat::uniform(lat::desc_lo(s_rope, 16)), lo_q = lat::uniform(lat::desc_lo(s_q, 16));
        const uint32_t t_o = lat::uniform(tmem), t_s = t_o + C::kColS;
        uint32_t tiles_done = 0;
        bool ok = true;
        Walk next = w;
        bool more = true;
        // An entry is written again two items later, after the first scores of the item between: by then the
        // softmax warps have taken it over.
        uint32_t items = 0;
        auto tell = [&]() {
            if (lane == 0) {
                Item& i = sh.item[items & 1];
                i.rows = more ? next.rows(a) : 0;
                i.row0 = next.row0(a);
                i.at = next.at;
                i.end = next.end();
                i.m = next.r.m;
                i.n = next.r.n;
                i.first = next.block * a.tpn;
                i.parts = i.at > 0 ? 0 : i.end == next.count ? 1 : static_cast<int>((next.count - next.left + sh.per - 1) / sh.per) + 1;
                ptx::mbar_arrive(bar(sh.item_full[items & 1]));
            }
            __syncwarp();
            ++items;
        };
        tell();
        do {
            ok = lat::wait_warp(bar(sh.q_full), seg & 1u, sync);
            if (!ok) break;
            ++seg;
            const int end = w.end();
#pragma unroll 1
            for (int tile = w.at; tile < end; ++tile) {
                const uint32_t first = lat::uniform(pair % C::kPairs), rope_slot = lat::uniform(rope % C::kRope);
                uint32_t slot = first, phase = (pair / C::kPairs) & 1u;
#pragma unroll 1
                for (int p = 0; p < np && ok; ++p) {               // S^T, 128 columns at a time
                    ok = lat::wait_warp(bar(sh.full[slot]), phase, sync);
                    const uint32_t da = lo_k + slot * kPair, db = lo_q + p * 2 * kQ;
                    lat::mma4_f16<2, 2>(t_s, da, kHiK, db, kHiK, kIdS, p > 0);
                    lat::mma4_f16<2, 2>(t_s, da + kChunk, kHiK, db + kQ, kHiK, kIdS, 1u);
                    if (++slot == C::kPairs) {
                        slot = 0;
                        phase ^= 1u;
                    }
                }
                if (ok) ok = lat::wait_warp(bar(sh.rope_full[rope_slot]), (rope / C::kRope) & 1u, sync);
                if (!ok) break;
                // (the rotated part is zero from R columns on)
                lat::mma4_f16<2, 2>(t_s, lo_r + rope_slot * kChunk, kHiK, lo_q + np * 2 * kQ, kHiK, kIdS, 1u);
                ptx::commit_elect(bar(sh.s_full));
                if (tile + 1 == end) ptx::commit_elect(bar(sh.q_empty));
                if (tile == w.at) {
                    more = next.next(a);
                    tell();
                }
                pair += np;
                ++rope;
                ok = lat::wait_warp(bar(sh.p_full), tiles_done & 1u, sync);
                if (!ok) break;
                ++tiles_done;
                ptx::tc_fence_after();
                const uint32_t more = lat::uniform(tile > w.at ? 1u : 0u), db = lat::uniform(lat::desc_lo(s_rope + rope_slot * kChunkBytes, 16));
                slot = first;
#pragma unroll 1
                for (int p = 0; p < np; ++p) {                     // O^T, 128 rows at a time
                    const uint32_t da = lo_v + slot * kPair, d = t_o + p * NR;
                    lat::mma4_f16<128, kStepP>(d, da, kHiK, db, kHiP, kIdO, more);
                    lat::mma4_f16<128, kStepP>(d, da + 4 * 128, kHiK, db + 4 * kStepP, kHiP, kIdO, 1u);
                    ptx::commit_elect(bar(sh.empty[slot]));
                    if (++slot == C::kPairs) slot = 0;
                }
                ptx::commit_elect(bar(sh.rope_empty[rope_slot]));
                if (tile + 1 == end) ptx::commit_elect(bar(sh.o_full));
            }
            w = next;
        } while (ok && more);
    } else if (warp > kLoaders && any) {
        // ------------------------------------------------------------ softmax
        const int quarter = warp & 3, group = (warp - 1 - kLoaders) >> 2;
        const int row = quarter * 32 + lane;                      // token of the tile
        const uint32_t lanes = static_cast<uint32_t>(quarter * 32) << 16;
        const uint32_t t_s = tmem + lanes + C::kColS + group * HC, t_o = tmem + lanes + group * HC;
        const int id = 1 + group;
        uint32_t tiles_done = 0;
        bool ok = true;
        for (;; ++seg) {
            ok = ok && lat::wait_warp(bar(sh.item_full[seg & 1u]), (seg >> 1) & 1u, sync);
            const Item it = sh.item[seg & 1u];
            // What the item's tiles find in shared memory: no reference, and what each column's token sees.
            if (quarter == 0 && lane < HC) {
                sh.ref[group][lane] = kNone;
                const int token = min(it.first + (a.hb == 1 ? (group * HC + lane) / a.H : 0), it.n - 1);
                sh.sees[group * HC + lane] = max(0, it.m - it.n + token + 1);
            }
            if (lat::named_any(id, 128, !ok) || it.rows == 0) break;
            const int low = max(0, it.m - it.n + it.first + 1);    // rows that every row of the block sees
            // l, ref: sum and reference of every column, the sums of this thread's token only
            float ref[HC], l[HC];
#pragma unroll
            for (int j = 0; j < HC; ++j) {
                l[j] = 0.0f;
                ref[j] = kNone;
            }
            bool failed = false;
#pragma unroll 1
            for (int tile = it.at; tile < it.end; ++tile) {
                ok = lat::wait_warp(bar(sh.s_full), tiles_done & 1u, sync);
                ++tiles_done;
                ptx::tc_fence_after();
                uint32_t raw_s[HC];
                ptx::tmem_ld<HC>(t_s, raw_s);
                ptx::tmem_wait_ld();
                const int token = tile * kTile + row;
                if ((tile + 1) * kTile > low) {
                    // rows past the request's, and rows newer than a query token, are not seen
#pragma unroll
                    for (int j = 0; j < HC; j += 4) {
                        const int4 s = *reinterpret_cast<const int4*>(&sh.sees[group * HC + j]);
                        if (token >= s.x) raw_s[j] = __float_as_uint(-INFINITY);
                        if (token >= s.y) raw_s[j + 1] = __float_as_uint(-INFINITY);
                        if (token >= s.z) raw_s[j + 2] = __float_as_uint(-INFINITY);
                        if (token >= s.w) raw_s[j + 3] = __float_as_uint(-INFINITY);
                    }
                }
                // Weights with the references as they are; if one is above 2^kMost (or the first one
                // seen), all of the group move them first.
                uint32_t packed[HC / 2];
                float p[HC];
                bool move = true;                                  // an item's first tile sets them
                if (tile > it.at) {
                    float most = -INFINITY;
#pragma unroll
                    for (int j = 0; j < HC; ++j) {
                        p[j] = fmaf(__uint_as_float(raw_s[j]), a.scale2, -ref[j]);
                        most = fmaxf(most, p[j]);
                    }
#pragma unroll
                    for (int j = 0; j < HC; ++j) p[j] = lat::ex2(p[j]);
                    move = lat::named_any(id, 128, most > kMost || !ok);
                }
                if (move) {
                    float top = kNone;                             // of column cl
                    const int cl = lane & (HC - 1);
#pragma unroll
                    for (int j = 0; j < HC; ++j) {
                        const float m = lat::warp_max(__uint_as_float(raw_s[j]) * a.scale2);
                        if (cl == j) top = fmaxf(top, m);
                    }
                    if (lane < HC) sh.top[group][quarter][lane] = top;
                    failed = lat::named_any(id, 128, !ok);
                    if (failed) break;
                    if (quarter == 0 && lane < HC) {
                        top = fmaxf(fmaxf(sh.top[group][0][cl], sh.top[group][1][cl]), fmaxf(sh.top[group][2][cl], sh.top[group][3][cl]));
                        const float old = sh.ref[group][cl], to = top > old + kMost ? top - kLift : old;
                        sh.ref[group][cl] = to;
                        sh.fade[group][cl] = lat::ex2(old - to);   // 0 where there was nothing before
                    }
                    lat::named_sync(id, 128);
#pragma unroll
                    for (int j = 0; j < HC; ++j) {
                        ref[j] = sh.ref[group][j];
                        l[j] *= sh.fade[group][j];
                        p[j] = lat::ex2(fmaf(__uint_as_float(raw_s[j]), a.scale2, -ref[j]));
                    }
                    if (tile > it.at) {
#pragma unroll 1
                        for (int b = 0; b < np; ++b) {
                            uint32_t o[HC];
                            ptx::tmem_ld<HC>(t_o + b * NR, o);
                            ptx::tmem_wait_ld();
#pragma unroll
                            for (int j = 0; j < HC; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * sh.fade[group][j]);
                            lat::tmem_st<HC>(t_o + b * NR, o);
                        }
                        lat::tmem_wait_st();
                    }
                    lat::named_sync(id, 128);                      // sh.ref and sh.fade have been read
                }
#pragma unroll
                for (int j = 0; j < HC; j += 2) {
                    l[j] += p[j];
                    l[j + 1] += p[j + 1];
                    packed[j / 2] = Pair<T>::pack(p[j], p[j + 1]);
                }
                uint8_t* prow = smem + C::kOffRope + (rope % C::kRope) * kChunkBytes;
#pragma unroll
                for (int c = 0; c < HC / 8; ++c) {
                    uint32_t off = row * C::kRowBytes + (group * HC / 8 + c) * 16;
                    off ^= ((off >> 7) & (C::kRowBytes / 16 - 1)) << 4;
                    *reinterpret_cast<uint4*>(prow + off) =
                        make_uint4(packed[4 * c], packed[4 * c + 1], packed[4 * c + 2], packed[4 * c + 3]);
                }
                // Weights past the request's rows are zero, but 0 times what lies there need not be.
                if (token >= it.m) {
#pragma unroll 1
                    for (int c = group; c < 2 * np; c += C::kGroups) {
                        uint4* z = reinterpret_cast<uint4*>(smem + ((pair + c / 2) % C::kPairs) * 2 * kChunkBytes +
                                                            (c & 1) * kChunkBytes + row * 128);
#pragma unroll
                        for (int i = 0; i < 8; ++i) z[i] = make_uint4(0, 0, 0, 0);
                    }
                }
                pair += np;
                ++rope;
                ptx::fence_proxy_async_smem();
                ptx::tc_fence_before();
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(bar(sh.p_full));
            }
            if (failed) break;
            // ---- the segment's result
            const float mine = lane_sums<HC>(l);
            if (lane < HC) sh.sum[group][quarter][lane] = mine;
            lat::named_sync(id, 128);
            const int cl = lane & (HC - 1);
            const float mine_ref = quarter == 0 ? sh.ref[group][cl] : kNone;   // (the warp that sets it)
            const float total = (sh.sum[group][0][cl] + sh.sum[group][1][cl]) + (sh.sum[group][2][cl] + sh.sum[group][3][cl]);
            const int rows = it.rows;
            const int col = group * HC + cl;                        // of the statistics
            const float inv = total == 0.0f ? 0.0f : 1.0f / total;   // (0: nothing seen; NaN stays NaN)
            float f[HC];
#pragma unroll
            for (int j = 0; j < HC; ++j) f[j] = __shfl_sync(0xFFFFFFFFu, inv, j);
            ok = lat::wait_warp(bar(sh.o_full), seg & 1u, sync);   // (the next vote ends it where this ran out)
            ptx::tc_fence_after();
            if (it.parts == 1) {
                if (a.lse != nullptr && quarter == 0 && lane < HC && col < rows)
                    a.lse[it.row0 + col] = total == 0.0f ? -INFINITY : (mine_ref + log2f(total)) * kLn2;
                const bool odd = (lane & 1) != 0;
                uint32_t* out = reinterpret_cast<uint32_t*>(a.out) +
                                (((it.row0 + group * HC + (odd ? 1 : 0)) * a.L + quarter * 32 + (lane & ~1)) >> 1);
                const int last = rows - group * HC - (odd ? 1 : 0);   // this lane's rows j < last exist
#pragma unroll 1
                for (int p = 0; p < np; ++p, out += 64) {
                    uint32_t o[HC];
                    ptx::tmem_ld<HC>(t_o + p * NR, o);
                    ptx::tmem_wait_ld();
#pragma unroll
                    for (int j = 0; j < HC; j += 2) {
                        // two rows, one element each -> one row, two elements: even lanes keep row j
                        const float v0 = __uint_as_float(o[j]) * f[j], v1 = __uint_as_float(o[j + 1]) * f[j + 1];
                        const float got = __shfl_xor_sync(0xFFFFFFFFu, odd ? v0 : v1, 1);
                        if (j < last) out[j * (a.L / 2)] = odd ? Pair<T>::pack(got, v1) : Pair<T>::pack(v0, got);
                    }
                }
            } else {
                // The part that begins an item owns its joining: parts up to the CTA of the item's last tile.
                if (it.parts > 1 && threadIdx.x == 128)
                    a.joins[blockIdx.x] = make_int4(static_cast<int>(it.row0), rows, it.parts, 0);
                const int64_t part = 2 * int64_t(blockIdx.x) + (it.at > 0 ? 0 : 1);
                if (quarter == 0 && lane < HC && col < rows) a.stats[part * NR + col] = make_float2(mine_ref, total);
                float* const dst = a.partial + (part * NR + group * HC) * a.L + quarter * 32 + lane;
#pragma unroll 1
                for (int c = 0; c < HC / 8 * np; ++c) {
                    const int p = HC == 8 ? c : c >> 1, j0 = HC == 8 ? 0 : (c & 1) * 8;
                    uint32_t o[8];
                    ptx::tmem_ld<8>(t_o + p * NR + j0, o);
                    ptx::tmem_wait_ld();
                    float* row = dst + j0 * a.L + p * 128;
#pragma unroll
                    for (int j = 0; j < 8; ++j, row += a.L) *row = __uint_as_float(o[j]);   // (rows that are none, too)
                }
            }
            ptx::tc_fence_before();
        }
    }
    __syncthreads();
    if (sh.abort) {
        // A wait ran out: copies in flight land and MMAs end (both bounded) before the CTA does.
        const uint64_t t0 = ptx::globaltimer();
        auto land = [&](uint64_t& b, uint32_t uses) {
            while (uses > 0 && !ptx::mbar_test_wait(bar(b), (uses - 1) & 1u) && ptx::globaltimer() - t0 < (1ull << 26)) {}
        };
        if (warp >= 1 && warp < 1 + kLoaders) {
            for (uint32_t i = 0; i < C::kPairs; ++i) land(sh.full[i], pair / C::kPairs + (i < pair % C::kPairs ? 1 : 0));
            for (uint32_t i = 0; i < C::kRope; ++i) land(sh.rope_full[i], rope / C::kRope + (i < rope % C::kRope ? 1 : 0));
            land(sh.q_full, seg);
        } else if (threadIdx.x == 0) {
            ptx::tc_commit(bar(sh.drain));
            land(sh.drain, 1);
        }
        __syncthreads();
    }
    if (warp == 0) {
        ptx::tc_fence_after();
        ptx::tmem_dealloc(tmem, 512);
    }
}

// Joins the parts of the items that the cuts split: row r of part i holds an
// unnormalised sum o_i with reference m_i and sum l_i, and
//     out = sum_i 2^(m_i - M) o_i / sum_i 2^(m_i - M) l_i,  M = max m_i,
// in a fixed order.  Rows of few parts take a warp each, eight rows a block;
// of rows of many parts, every 128 columns take a block, a warp every eighth
// part.
constexpr int kJoinThreads = 256, kJoinWarps = kJoinThreads / 32;
constexpr int kMaxGrid = 512;
constexpr int kFewParts = kJoinWarps;
template <typename T>
__global__ void __launch_bounds__(kJoinThreads) latent_join_kernel(const Args a, int grid, int NR) {
    ptx::launch_dependents();
    ptx::grid_dependency_wait();
    __shared__ int first[kMaxGrid + 1];                   // prefix sums of the CTAs' units of work
    __shared__ int sums[kJoinWarps];
    __shared__ alignas(16) float acc[kJoinWarps][128];
    __shared__ float acc_l[kJoinWarps];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int run = 0;
    for (int base = 0; base < grid; base += kJoinThreads) {
        const int c = base + threadIdx.x;
        int4 j = make_int4(0, 0, 0, 0);
        if (c < grid) j = a.joins[c];
        int v = j.z == 0 ? 0 : j.z <= kFewParts ? (j.y + kJoinWarps - 1) / kJoinWarps : j.y * (a.L / 128);
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int up = __shfl_up_sync(0xFFFFFFFFu, v, o);
            if (lane >= o) v += up;
        }
        __syncthreads();
        if (lane == 31) sums[warp] = v;
        __syncthreads();
        int all = run;
        for (int w = 0; w < kJoinWarps; ++w) {
            if (w < warp) v += sums[w];
            all += sums[w];
        }
        if (c < grid) first[c + 1] = run + v;
        run = all;
    }
    if (threadIdx.x == 0) first[0] = 0;
    __syncthreads();
    const int blocks = a.L / 128;                         // of 128 columns: four a lane
    for (int u = blockIdx.x; u < first[grid]; u += gridDim.x) {
        int lo = 0, hi = grid;
        while (hi - lo > 1) {
            const int mid = (lo + hi) / 2;
            if (first[mid] <= u) lo = mid;
            else hi = mid;
        }
        // (CTAs without work share their neighbour's prefix: the last one with first <= u has some)
        const int4 j = a.joins[lo];
        const bool few = j.z <= kFewParts;
        const int r = few ? (u - first[lo]) * kJoinWarps + warp : (u - first[lo]) / blocks, parts = j.z;
        const int q0 = few ? 0 : (u - first[lo]) % blocks, nq = few ? blocks : 1;   // this unit's column blocks
        const int step = few ? 1 : kJoinWarps;
        const bool mine = r < j.y;
        auto slot = [&](int i) { return (i == 0 ? int64_t(2) * lo + 1 : int64_t(2) * (lo + i * a.team)) * NR + r; };
        float m = kNone, l = 0.0f;
        float4 o[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) o[q] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (mine) {
            for (int i = lane; i < parts; i += 32) m = fmaxf(m, __ldcg(&a.stats[slot(i)]).x);
            m = lat::warp_max(m);
#pragma unroll 2
            for (int i = few ? 0 : warp; i < parts; i += step) {
                const int64_t s = slot(i);
                const float2 st = __ldcg(&a.stats[s]);
                const float4* src = reinterpret_cast<const float4*>(a.partial + s * a.L) + q0 * 32 + lane;
                const float f = lat::ex2(st.x - m);
                l = fmaf(f, st.y, l);
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    if (q < nq) {
                        const float4 v = __ldcg(src + q * 32);
                        o[q].x = fmaf(f, v.x, o[q].x);
                        o[q].y = fmaf(f, v.y, o[q].y);
                        o[q].z = fmaf(f, v.z, o[q].z);
                        o[q].w = fmaf(f, v.w, o[q].w);
                    }
                }
            }
        }
        const int64_t row = int64_t(j.x) + r;
        if (few) {
            if (mine) {
                const float inv = l == 0.0f ? 0.0f : 1.0f / l;
                uint2* out = reinterpret_cast<uint2*>(static_cast<T*>(a.out) + row * a.L) + lane;
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    if (q < nq)
                        out[q * 32] = make_uint2(Pair<T>::pack(o[q].x * inv, o[q].y * inv), Pair<T>::pack(o[q].z * inv, o[q].w * inv));
                if (a.lse != nullptr && lane == 0) a.lse[row] = l == 0.0f ? -INFINITY : (m + log2f(l)) * kLn2;
            }
            continue;
        }
        reinterpret_cast<float4*>(acc[warp])[lane] = o[0];
        if (lane == 0) acc_l[warp] = l;
        __syncthreads();
        l = 0.0f;
#pragma unroll
        for (int w = 0; w < kJoinWarps; ++w) l += acc_l[w];
        const float inv = l == 0.0f ? 0.0f : 1.0f / l;
        const int c = 2 * threadIdx.x;
        if (c < 128) {
            float x = 0.0f, y = 0.0f;
#pragma unroll
            for (int w = 0; w < kJoinWarps; ++w) {
                const float2 v = *reinterpret_cast<const float2*>(&acc[w][c]);
                x += v.x;
                y += v.y;
            }
            *reinterpret_cast<uint32_t*>(static_cast<T*>(a.out) + row * a.L + q0 * 128 + c) = Pair<T>::pack(x * inv, y * inv);
        }
        if (a.lse != nullptr && threadIdx.x == 0 && q0 == 0) a.lse[row] = l == 0.0f ? -INFINITY : (m + log2f(l)) * kLn2;
        __syncthreads();
    }
}

// ---------------------------------------------------------------- host

// Rows (token, head) of a block: as many as a request has on average, up to 64.
int row_block(int64_t rows) { return rows <= 16 ? 16 : rows <= 32 ? 32 : 64; }

struct Sizes {
    int64_t partial, stats, joins, total;
};
Sizes workspace_of(int64_t grid, int64_t NR, int64_t L) {
    Sizes s;
    s.partial = 2 * grid * NR * L * 4;
    s.stats = 2 * grid * NR * 8;
    s.joins = grid * 16;
    s.total = s.partial + s.stats + s.joins;
    return s;
}

template <typename T, int NR, bool kStall = false>
sgq_status run(const CUtensorMap& tm_cache, const CUtensorMap& tm_q, const Args& a, int grid, int join_grid,
               cudaStream_t st) {
    auto kern = latent_attention_kernel<T, NR, kStall>;
    static bool configured[64] = {};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return SGQ_ERR_CUDA;
    if (!configured[dev]) {
        if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg<NR>::kSmem) != cudaSuccess)
            return SGQ_ERR_CUDA;
        configured[dev] = true;
    }
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(grid));
    cfg.blockDim = dim3(Cfg<NR>::kThreads);
    cfg.dynamicSmemBytes = Cfg<NR>::kSmem;
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, kern, tm_cache, tm_q, a) != cudaSuccess) return SGQ_ERR_CUDA;
    note_launch();
    if (grid == a.team) return SGQ_OK;   // nothing is split
    cfg.gridDim = dim3(static_cast<unsigned>(join_grid));
    cfg.blockDim = dim3(kJoinThreads);
    cfg.dynamicSmemBytes = 0;
    if (cudaLaunchKernelEx(&cfg, latent_join_kernel<T>, a, grid, NR) != cudaSuccess) return SGQ_ERR_CUDA;
    note_launch();
    return SGQ_OK;
}
template <typename T, bool kStall = false>
sgq_status run_rows(int NR, const CUtensorMap& tm_cache, const CUtensorMap& tm_q, const Args& a, int grid,
                    int join_grid, cudaStream_t st) {
    if (NR == 16) return run<T, 16, kStall>(tm_cache, tm_q, a, grid, join_grid, st);
    if (NR == 32) return run<T, 32, kStall>(tm_cache, tm_q, a, grid, join_grid, st);
    return run<T, 64, kStall>(tm_cache, tm_q, a, grid, join_grid, st);
}

}  // namespace

sgq_status latent_attention_workspace(int64_t T, int64_t H, int64_t L, int64_t* bytes) {
    DeviceInfo di;
    const sgq_status rc = device_info(&di);
    if (rc != SGQ_OK) return rc;
    *bytes = workspace_of(std::min(di.sm_count, kMaxGrid), row_block(T * H), L).total;
    return SGQ_OK;
}

sgq_status launch_latent_attention(const LatentArgs& x, cudaStream_t st) {
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
    const int NR = row_block((x.T + x.B - 1) / x.B * x.H);
    a.cache = static_cast<const char*>(x.cache);
    a.c_page = 2 * x.c_page;
    a.c_row = 2 * x.c_row;
    a.table = x.page_table;
    a.kv_lens = x.kv_lens;
    a.q_starts = x.q_starts;
    a.out = x.out;
    a.lse = x.lse;
    a.T = x.T;
    a.B = x.B;
    a.pages = x.pages;
    a.width = x.table_width;
    a.H = x.H;
    a.L = x.L;
    a.page = x.page;
    a.box = std::min(x.page & -x.page, kTile);   // rows of a box: whole boxes in a page and in a tile
    // (rows that lie apart, as those of a layer between others, are not: what is between them is not wanted)
    const int64_t row_bytes = 2 * int64_t(x.L + x.R);
    a.box_bytes = a.c_row <= row_bytes + row_bytes / 8 ? static_cast<uint32_t>((a.box - 1) * a.c_row + row_bytes) : 0u;
    a.tpn = std::max(1, NR / x.H);
    a.hb = (x.H + NR - 1) / NR;
    // (more head blocks than that are a walk of one CTA: teams would leave CTAs over)
    a.team = a.hb <= 4 ? a.hb : 1;
    a.scale2 = x.scale * kLog2e;
    // No more CTAs than the tables could hold tiles (a request's counted up to the largest grid).
    const int64_t tiles = std::min<int64_t>(kMaxGrid, std::max<int64_t>(1, (x.table_width * x.page + kTile - 1) / kTile));
    const int64_t most = (x.T + x.B) * (a.hb / a.team) * tiles;
    const int sms = std::min(di.sm_count, kMaxGrid) / a.team * a.team;
    const int grid = static_cast<int>(std::min<int64_t>(sms, most * a.team));
    a.inv_teams = grid == a.team ? 0 : ~uint64_t(0) / static_cast<uint64_t>(grid / a.team) + 1;
    const Sizes s = workspace_of(grid, NR, x.L);
    char* ws = static_cast<char*>(x.workspace);
    a.partial = reinterpret_cast<float*>(ws);
    a.stats = reinterpret_cast<float2*>(ws + s.partial);
    a.joins = reinterpret_cast<int4*>(ws + s.partial + s.stats);

    const cuuint32_t ones[3] = {1, 1, 1};
    const cuuint64_t W = static_cast<cuuint64_t>(x.L + x.R);
    CUtensorMap tm_cache, tm_q;
    {
        const cuuint64_t dims[3] = {W, static_cast<cuuint64_t>(x.page), static_cast<cuuint64_t>(x.pages)};
        const cuuint64_t strides[2] = {static_cast<cuuint64_t>(x.c_row) * 2, static_cast<cuuint64_t>(x.c_page) * 2};
        const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(a.box), 1};
        if (encode(&tm_cache, CU_TENSOR_MAP_DATA_TYPE_UINT16, 3, const_cast<void*>(x.cache), dims, strides, box, ones,
                      CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                      CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
            return SGQ_ERR_CUDA;
    }
    {
        const cuuint64_t dims[2] = {W, static_cast<cuuint64_t>(x.T * x.H)};
        const cuuint64_t strides[1] = {static_cast<cuuint64_t>(x.q_row) * 2};
        const cuuint32_t box[2] = {64, static_cast<cuuint32_t>(NR)};
        if (encode(&tm_q, CU_TENSOR_MAP_DATA_TYPE_UINT16, 2, const_cast<void*>(x.q), dims, strides, box, ones,
                      CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                      CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
            return SGQ_ERR_CUDA;
    }
    const int join_grid = di.sm_count * 8;   // (a row's loads wait for one another: 2 / 4 / 8 an SM, one request of 131071 rows 77.5 / 71.7 / 70.9 us, 128 requests 171.7 / 166.3 / 165.3)
    if (x.stall) return run_rows<__nv_bfloat16, true>(NR, tm_cache, tm_q, a, grid, join_grid, st);
    return x.dtype == SGQ_BF16 ? run_rows<__nv_bfloat16>(NR, tm_cache, tm_q, a, grid, join_grid, st)
                               : run_rows<__half>(NR, tm_cache, tm_q, a, grid, join_grid, st);
}

}  // namespace sgq
